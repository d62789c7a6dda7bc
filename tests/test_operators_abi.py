"""CPU checks of the routing, few-token layer and 4-bit linear entry points: what they refuse, in
the C ABI (before any pointer is looked at) and in the binding, and their host-only queries."""

import ctypes as C
import math
import os

import pytest
import torch

from mxfp4_block_scaled_expert_amd import _lib as L
from mxfp4_block_scaled_expert_amd import ops

if not os.path.exists(L.LIB_PATH):
    pytest.skip("libmxq.so not built", allow_module_level=True)
LIB = L.load()
FAKE = C.c_void_p(1 << 20)  # never dereferenced: every call below is refused first


def _router(topk=2, scoring=0, n_group=1, topk_group=1, group_score=0, renormalize=0, scale=1.0):
    return C.byref(L.MoeRouter(topk, scoring, n_group, topk_group, group_score, renormalize, scale))


BAD_ROUTERS = [dict(topk=0), dict(topk=33), dict(topk=9), dict(scoring=2), dict(scoring=-1), dict(n_group=0),
               dict(n_group=3), dict(n_group=65), dict(topk_group=2), dict(n_group=4, topk_group=5),
               dict(n_group=4, topk_group=1, topk=3), dict(group_score=2), dict(renormalize=2),
               dict(scale=math.nan), dict(scale=math.inf)]


@pytest.mark.parametrize("bad", BAD_ROUTERS)
def test_router_fields_are_checked(bad):
    assert LIB.mxq_moe_route(FAKE, 1, 4, 8, 8, _router(**bad), None, FAKE, FAKE, None) == L.MXQ_ERR_ARG
    assert LIB.mxq_moe_layer_fp8(FAKE, 4, 256, 128, 8, 256, FAKE, 1, None, _router(**bad), None, FAKE, FAKE, FAKE,
                                 FAKE, None, 0, FAKE, 256, FAKE, 1 << 30, None) == L.MXQ_ERR_ARG


def test_route_refusals():
    f = LIB.mxq_moe_route
    r = _router()
    assert f(FAKE, 2, 4, 8, 8, r, None, FAKE, FAKE, None) == L.MXQ_ERR_DTYPE
    assert f(FAKE, 1, 4, 513, 513, r, None, FAKE, FAKE, None) == L.MXQ_ERR_SHAPE
    assert f(FAKE, 1, 4, 0, 8, r, None, FAKE, FAKE, None) == L.MXQ_ERR_SHAPE
    assert f(FAKE, 1, 4, 8, 7, r, None, FAKE, FAKE, None) == L.MXQ_ERR_SHAPE
    assert f(FAKE, 1, -1, 8, 8, r, None, FAKE, FAKE, None) == L.MXQ_ERR_SHAPE
    assert f(FAKE, 1, (1 << 25) + 1, 8, 8, r, None, FAKE, FAKE, None) == L.MXQ_ERR_SHAPE
    assert f(FAKE, 1, 4, 8, 8, None, None, FAKE, FAKE, None) == L.MXQ_ERR_NULL
    for args in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None)):
        assert f(args[0], 1, 4, 8, 8, r, None, args[1], args[2], None) == L.MXQ_ERR_NULL
    assert f(C.c_void_p((1 << 20) + 2), 1, 4, 8, 8, r, None, FAKE, FAKE, None) == L.MXQ_ERR_SHAPE
    assert f(None, 1, 0, 8, 8, r, None, None, None, None) == L.MXQ_OK


@pytest.mark.parametrize("mx", [False, True])
def test_layer_refusals(mx):
    fn = LIB.mxq_moe_layer_mxfp4 if mx else LIB.mxq_moe_layer_fp8

    def call(x=FAKE, M=4, H=256, I=128, E=8, ldx=256, gate=FAKE, gdt=0, router=_router(), w1=FAKE, s1=FAKE, w2=FAKE,
             s2=FAKE, layout=0, out=FAKE, ldo=256, ws=FAKE, n=1 << 30):
        return fn(x, M, H, I, E, ldx, gate, gdt, None, router, None, w1, s1, w2, s2, None, layout, out, ldo, ws, n,
                  None)

    assert call(gdt=2) == L.MXQ_ERR_DTYPE
    assert call(layout=2) == L.MXQ_ERR_ARG
    assert call(router=None) == L.MXQ_ERR_NULL
    assert call(M=0) == L.MXQ_OK
    for bad in (dict(M=-1), dict(M=17), dict(H=240, ldx=240, ldo=240), dict(I=100), dict(H=0), dict(I=0), dict(E=0),
                dict(E=513), dict(ldx=248), dict(ldx=260), dict(ldo=255), dict(H=1 << 21, ldx=1 << 21, ldo=1 << 21),
                dict(H=1 << 17, ldx=1 << 17, ldo=1 << 17), dict(I=1 << 21), dict(x=C.c_void_p((1 << 20) + 8)),
                dict(gate=C.c_void_p((1 << 20) + 8)), dict(w1=C.c_void_p((1 << 20) + 8)),
                dict(w2=C.c_void_p((1 << 20) + 8)), dict(ws=C.c_void_p((1 << 20) + 8))):
        assert call(**bad) == L.MXQ_ERR_SHAPE, bad
    for name in ("x", "gate", "w1", "s1", "w2", "s2", "out"):
        assert call(**{name: None}) == L.MXQ_ERR_NULL, name
    need = LIB.mxq_moe_layer_workspace_size(4, 256, 128, 8, 2, int(mx))
    assert need > 0
    assert call(ws=None) == L.MXQ_ERR_WORKSPACE
    assert call(n=need - 1) == L.MXQ_ERR_WORKSPACE


def test_layer_workspace_query():
    q = LIB.mxq_moe_layer_workspace_size
    for M in (1, 16):
        for (H, I, E, topk, w) in ((2880, 2880, 128, 4, 1), (7168, 2048, 256, 8, 0), (128, 128, 1, 1, 0)):
            assert q(M, H, I, E, topk, w) >= 4 * M * E
    for bad in ((0, 256, 128, 8, 2, 0), (17, 256, 128, 8, 2, 0), (4, 200, 128, 8, 2, 0), (4, 256, 96, 8, 2, 0),
                (4, 256, 128, 8, 9, 0), (4, 256, 128, 8, 2, 2), (4, 256, 128, 513, 2, 0)):
        assert q(*bad) == 0, bad
    assert q(4, 256, 96, 8, 2, 1) > 0  # MXFP4: multiples of 32


def test_int4_refusals():
    def call(A=FAKE, M=4, K=256, lda=256, W=FAKE, N=64, group=64, s=FAKE, sdt=1, z=None, b=None, bdt=1, out=FAKE,
             ldo=64, ws=FAKE, n=1 << 30):
        return LIB.mxq_int4_linear(A, M, K, lda, W, N, group, s, sdt, z, b, bdt, out, ldo, ws, n, None)

    for g in (0, 16, 48, 256, -64):
        assert call(group=g) == L.MXQ_ERR_BLOCK
    assert call(sdt=2) == L.MXQ_ERR_DTYPE
    assert call(b=FAKE, bdt=7) == L.MXQ_ERR_DTYPE
    for bad in (dict(K=224, group=64), dict(lda=248), dict(lda=260), dict(ldo=63), dict(M=-1), dict(N=-1),
                dict(K=0, lda=0), dict(M=(1 << 19) + 1), dict(N=(1 << 28) + 1, ldo=1 << 29),
                dict(A=C.c_void_p((1 << 20) + 8)), dict(W=C.c_void_p((1 << 20) + 8))):
        assert call(**bad) == L.MXQ_ERR_SHAPE, bad
    for name in ("A", "W", "s", "out"):
        assert call(**{name: None}) == L.MXQ_ERR_NULL, name
    assert call(M=0) == L.MXQ_OK and call(N=0) == L.MXQ_OK
    q = LIB.mxq_int4_linear_workspace_size
    assert q(0, 64, 256, 64) == 0 and q(4, 64, 256, 48) == 0 and q(4, 64, 224, 64) == 0 and q(4, 2048, 7168, 64) == 0
    assert q(4096, 4096, 4096, 128) >= 2 * 4096 * 4096
    for M, N, K in ((16, 2048, 7168), (64, 64, 16384), (2048, 512, 8192)):
        n = q(M, N, K, 64)
        assert M > 64 or (n % (4 * M * N) == 0 and n <= 16 << 20)
        if n:
            assert call(M=M, N=N, K=K, lda=K, ldo=N, ws=None) == L.MXQ_ERR_WORKSPACE
            assert call(M=M, N=N, K=K, lda=K, ldo=N, n=n - 1) == L.MXQ_ERR_WORKSPACE


def test_router_struct_matches_header():
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mxq.h")).read()
    body = re.search(r"typedef struct mxq_moe_router \{(.*?)\} mxq_moe_router;", src, re.S).group(1)
    assert [f for f, _ in L.MoeRouter._fields_] == re.findall(r"(?:int32_t|float) (\w+);", body)


def test_binding_refuses_before_the_library():
    bf, R = torch.bfloat16, ops.Router
    x, logits = torch.zeros(2, 256, dtype=bf), torch.zeros(2, 8)
    with pytest.raises(ValueError):
        ops.moe_route(logits.half(), R(2))
    with pytest.raises(ValueError):
        ops.moe_route(logits[0], R(2))
    with pytest.raises(ValueError):
        ops.moe_route(logits, (2, "softmax"))
    for r in (R(2, scoring="tanh"), R(2, group_score="sum")):
        with pytest.raises(ValueError):
            ops.moe_route(logits, r)
    with pytest.raises(ValueError):
        ops.moe_route(logits, R(2), correction_bias=torch.zeros(7))
    with pytest.raises(ValueError):
        ops.moe_route(logits, R(2))  # not on the GPU
    gate = torch.zeros(8, 256, dtype=bf)
    w1, w2 = torch.zeros(8, 256, 256, dtype=torch.uint8), torch.zeros(8, 256, 128, dtype=torch.uint8)
    s1, s2 = torch.ones(8, 2, 2), torch.ones(8, 2, 1)
    good = dict(x=x, gate=gate, router=R(2), w1=w1, w1_scale=s1, w2=w2, w2_scale=s2)
    for bad in (dict(x=x.float()), dict(x=x[0]), dict(gate=gate[:7]), dict(gate=gate.half()), dict(w1=w1[:, :, :128]),
                dict(w2=w2[:7]), dict(w1_scale=s1[:, :1]), dict(w1_scale=s1.to(bf)), dict(w2_scale=s2[:7]),
                dict(w1_bias=torch.zeros(8, 255)), dict(gate_bias=torch.zeros(7)),
                dict(correction_bias=torch.zeros(8, dtype=bf)), dict(weight_layout="packed"),
                dict(x=torch.zeros(17, 256, dtype=bf)), dict()):  # the last: not on the GPU
        with pytest.raises(ValueError):
            ops.moe_layer_fp8(**{**good, **bad})
    m1, m2 = torch.zeros(8, 256, 128, dtype=torch.uint8), torch.zeros(8, 256, 64, dtype=torch.uint8)
    e1, e2 = torch.zeros(8, 256, 8, dtype=torch.uint8), torch.zeros(8, 256, 4, dtype=torch.uint8)
    good = dict(x=x, gate=gate, router=R(2), w1=m1, w1_scale=e1, w2=m2, w2_scale=e2)
    for bad in (dict(w1=m1.float()), dict(w1_scale=e1[:, :, :7]), dict(w2=m2[:, :, :32]), dict(weight_layout="tiled"),
                dict()):
        with pytest.raises(ValueError):
            ops.moe_layer_mxfp4(**{**good, **bad})
    w, s = torch.zeros(16, 128, dtype=torch.uint8), torch.ones(16, 4)
    good = dict(x=x, weight=w, weight_scale=s)
    for bad in (dict(x=x.float()), dict(x=x[:, :128]), dict(weight=w.float()), dict(weight=w[0]),
                dict(weight_scale=torch.ones(16, 16)), dict(weight_scale=torch.ones(16, 3)),
                dict(weight_scale=torch.ones(15, 4)), dict(weight_scale=s.half()), dict(weight_scale=torch.ones(16, 0)),
                dict(weight_zero=torch.zeros(16, 1, dtype=torch.uint8)), dict(weight_zero=torch.zeros(16, 2)),
                dict(bias=torch.zeros(15)), dict()):
        with pytest.raises(ValueError):
            ops.int4_linear(**{**good, **bad})


@pytest.mark.parametrize("group", [32, 64, 128])
def test_int4_wide_weights_do_not_bring_prompt_tiles_to_few_rows(group):
    """The prompts' tiles of 256 rows need x laid out in the workspace (2 M K bytes and more); calls of up to
    128 rows take partial sums at most, however wide the weights are."""
    q = LIB.mxq_int4_linear_workspace_size
    for M in (5, 8, 32, 64, 128):
        for N in (16384, 28672, 131072):
            n = q(M, N, 4096, group)
            assert n <= 16 << 20 and n % (4 * M * N) == 0, (M, N)
    for M in (129, 512):
        assert q(M, 28672, 4096, group) >= 2 * M * 4096


def test_rows_reach_the_library_aligned():
    """Slices of one row and contiguous views at odd offsets, which contiguous() returns as they are."""
    bf = torch.bfloat16
    buf = torch.arange(2 * 128 + 1).to(bf)
    views = [torch.randn(6, 201).to(bf)[:1, :128], torch.randn(6, 320).to(bf)[:1, 3:131], torch.randn(6, 201).to(bf)[:, :128],
             buf[1:].view(2, 128), torch.randn(1, 128).to(bf).expand(3, 128), torch.randn(128, 4).to(bf).t(),
             torch.randn(4, 256).to(bf)[:, ::2]]
    for v in views:
        r, ld = ops._rows(v)
        assert torch.equal(r, v) and r.data_ptr() % 16 == 0 and r.stride(1) == 1 and ld % 8 == 0 and ld >= 128
        assert r.shape[0] == 1 or r.stride(0) == ld
    for v in (torch.zeros(6, 320, dtype=bf)[:, 64:192], torch.zeros(6, 201, dtype=bf)[:1, :128], torch.zeros(4, 128, dtype=bf)):
        assert ops._rows(v)[0].data_ptr() == v.data_ptr()  # read in place
    odd = torch.zeros(8 * 256 + 8, dtype=torch.uint8)[8:]
    with pytest.raises(ValueError, match="weight must start"):
        ops._laid_out(odd.view(8, 256), "weight")
    assert ops._laid_out(odd.view(8, 256)[:, ::2], "weight").is_contiguous()


def test_router_fields_reach_the_struct_whole():
    """Numbers that the C struct cannot hold are refused, not cut: 2^32 + 2 is not top-2, 2.5 neither."""
    logits = torch.zeros(2, 8)
    for bad in (dict(topk=2 ** 32 + 2), dict(topk=2.5), dict(topk=2, n_group=2 ** 32 + 1), dict(topk=2, n_group=2, topk_group=1.5),
                dict(topk=2, topk_group=2 ** 32 + 1), dict(topk="2"), dict(topk=None)):
        with pytest.raises(ValueError, match="32 bits"):
            ops.moe_route(logits, ops.Router(**bad))
    for bad in (dict(topk=torch.tensor(2)), dict(topk=2, scale=torch.tensor(2.0)), dict(topk=2, scale="1")):
        with pytest.raises(ValueError, match="must be"):
            ops.moe_route(logits, ops.Router(**bad))
    assert ops._router_struct(ops.Router(3, n_group=4, topk_group=2))._obj.topk == 3


def test_workspaces_are_whole():
    """An expanded or sliced workspace holds fewer bytes than its elements: it is refused before its size is."""
    args = (torch.zeros(2, 256, dtype=torch.bfloat16), torch.zeros(8, 256), ops.Router(2),
            torch.zeros(8, 256, 256, dtype=torch.uint8), torch.ones(8, 2, 2), torch.zeros(8, 256, 128, dtype=torch.uint8),
            torch.ones(8, 2, 1))
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(1 << 20, dtype=torch.uint8)[::2],
               torch.zeros(64, 1, dtype=torch.uint8).expand(64, 1 << 16)):
        with pytest.raises(ValueError, match="contiguous"):
            ops.moe_layer_fp8(*args, workspace=ws)
