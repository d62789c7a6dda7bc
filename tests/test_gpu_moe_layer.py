"""The few-token MoE layer against its float64 oracle: within half a bf16 step (2^-8 relative) of the
exact output plus the oracle's bound on what fp32 sums and the two-term intermediate can differ by."""

import math

import numpy as np
import pytest
import torch

from mxfp4_block_scaled_expert_amd import _lib as L
from mxfp4_block_scaled_expert_amd import ops, synth
from oracle.layer import layer
from tests._util import gpu, u8

pytestmark = pytest.mark.gpu
HALF = torch.finfo(torch.bfloat16).eps / 2
R = ops.Router


def make(mx, M, E, H, I, seed, gate_dtype=torch.bfloat16, w1_bias=True, gate_bias=False, bias=False):
    g = torch.Generator().manual_seed(seed)
    d = (synth.moe_mxfp4_weights if mx else synth.moe_fp8_weights)(E, H, I, seed=seed)
    d["mx"] = mx
    d["x"] = synth.bf16_randn((M, H), g, "cpu")
    d["gate"] = (torch.randn(E, H, generator=g) * (1.5 / math.sqrt(H))).to(gate_dtype)
    d["gate_bias"] = torch.randn(E, generator=g) * 0.1 if gate_bias else None
    d["bias"] = torch.randn(E, generator=g) * 0.1 if bias else None
    d["w1_bias"] = torch.randn(E, 2 * I, generator=g) if w1_bias else None
    return d


def on_gpu(d, layout="plain"):
    o = {k: (v.to(gpu()) if torch.is_tensor(v) else v) for k, v in d.items()}
    if layout == "tiled":
        o["w1"], o["w2"] = ops.moe_prepack(o["w1"]), ops.moe_prepack(o["w2"])
        if d["mx"]:
            o["w1_scale"], o["w2_scale"] = ops.moe_prepack_scales(o["w1_scale"]), ops.moe_prepack_scales(o["w2_scale"])
    return o


def call(o, router, layout="plain", **kw):
    fn = ops.moe_layer_mxfp4 if o["mx"] else ops.moe_layer_fp8
    return fn(kw.pop("x", o["x"]), o["gate"], router, o["w1"], o["w1_scale"], o["w2"], o["w2_scale"],
              w1_bias=o["w1_bias"], gate_bias=o["gate_bias"], correction_bias=o["bias"], weight_layout=layout, **kw)


def oracle(d, router):
    n = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    return layer(n(d["x"]), n(d["gate"]), u8(d["w1"]), d["w1_scale"].numpy(), u8(d["w2"]), d["w2_scale"].numpy(),
                 d["mx"], dict(topk=router.topk, sigmoid=router.scoring == "sigmoid", n_group=router.n_group,
                               topk_group=router.topk_group, top2=router.group_score == "top2",
                               renormalize=router.renormalize, scale=router.scale),
                 gate_bias=n(d["gate_bias"]), correction_bias=n(d["bias"]), b1=n(d["w1_bias"]))


def check(d, router, layouts=("plain", "tiled")):
    want, bound, ids, gap = oracle(d, router)
    assert gap > 1e-5  # the inputs leave no routing decision to fp32 rounding
    outs = []
    for lay in layouts:
        out = call(on_gpu(d, lay), router, lay)
        torch.cuda.synchronize()
        outs.append(out)
        got = out.double().cpu().numpy()
        assert (np.abs(got - want) <= HALF * np.abs(want) + bound).all(), (lay, np.abs(got - want).max())
    assert all(torch.equal(o.view(torch.int16), outs[0].view(torch.int16)) for o in outs)
    return outs[0], ids


CASES = [
    # M, E, H, I, router
    (1, 8, 256, 128, R(2, renormalize=True)),
    (1, 1, 128, 128, R(1)),
    (2, 4, 384, 256, R(4, scoring="sigmoid")),
    (3, 16, 128, 640, R(3, renormalize=True, scale=2.5)),
    (5, 8, 512, 256, R(2)),
    (8, 3, 256, 384, R(1, scoring="sigmoid", renormalize=True)),
    (9, 5, 256, 128, R(2)),
    (16, 2, 640, 128, R(1)),
    (16, 24, 256, 256, R(6, n_group=4, topk_group=2, group_score="top2", renormalize=True)),
    (16, 150, 128, 128, R(8, renormalize=True)),
    (7, 300, 128, 128, R(3, scoring="sigmoid")),
]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("M,E,H,I,router", CASES)
def test_matches_oracle(mx, M, E, H, I, router):
    check(make(mx, M, E, H, I, seed=M * 100 + E, w1_bias=M % 2 == 1, gate_bias=M % 3 == 0, bias=E % 2 == 0,
               gate_dtype=torch.float32 if M % 2 else torch.bfloat16), router)


@pytest.mark.parametrize("M,H,I", [(1, 32, 32), (3, 96, 160), (16, 288, 96), (2, 2880, 352), (4, 544, 1440)])
def test_mxfp4_ragged_steps(M, H, I):
    """H and I that end inside a 256-element step."""
    check(make(True, M, 6, H, I, seed=H + I), R(2, renormalize=True))


@pytest.mark.parametrize("M,H,I", [(1, 64, 64), (2, 2880, 192), (5, 320, 2880), (16, 448, 1088)])
def test_mxfp4_scale_codes_in_pairs(M, H, I):
    """Multiples of 64 that end inside a step; codes that differ between neighbouring groups; codes at an
    odd address."""
    d = make(True, M, 6, H, I, seed=H + I)
    g = torch.Generator().manual_seed(H)
    for k in ("w1_scale", "w2_scale"):
        d[k] = torch.randint(116, 124, d[k].shape, generator=g, dtype=torch.uint8)
    r = R(2, renormalize=True)
    out, _ = check(d, r)
    o = on_gpu(d)
    for k in ("w1_scale", "w2_scale"):
        odd = torch.empty(o[k].numel() + 1, dtype=torch.uint8, device=gpu())[1:].view(o[k].shape)
        odd.copy_(o[k])
        assert torch.equal(call(dict(o, **{k: odd}), r), out)


@pytest.mark.parametrize("mx", [False, True])
def test_many_batches_of_rows(mx):
    """16 tokens on the same two experts, and on all of many: row batches that cut experts, batches
    with few steps, column items with several batches."""
    check(make(mx, 16, 2, 256, 1024, seed=1), R(2))
    check(make(mx, 16, 12, 256, 2048, seed=2), R(8, renormalize=True))
    check(make(mx, 16, 32, 128, 128, seed=3), R(16, renormalize=True))


def test_more_column_items_than_workgroups():
    check(make(True, 2, 3, 4416, 64, seed=4), R(2), layouts=("plain",))
    check(make(False, 9, 3, 4352, 128, seed=5), R(3), layouts=("tiled",))


def test_tokens_in_several_passes():
    """Rows so long that the tokens' rows do not fit on-chip together."""
    check(make(False, 11, 3, 8192, 128, seed=6), R(1), layouts=("plain",))
    check(make(True, 16, 2, 16384, 32, seed=7), R(2), layouts=("plain",))


def test_fp32_router_weights_are_not_rounded():
    """Two experts whose fp32 router weights differ below bf16: the product has to tell them apart."""
    d = make(False, 4, 2, 256, 128, seed=8, gate_dtype=torch.float32)
    d["gate"][1] = d["gate"][0] + torch.where(d["x"][0].float() > 0, 1.0, -1.0) * 2.0 ** -14
    check(d, R(1))


@pytest.mark.parametrize("mx", [False, True])
def test_masked_experts_and_empty_tokens(mx):
    """gate_bias -inf masks experts; a NaN token finds no expert and gets zeros, the others are
    untouched by it."""
    d = make(mx, 5, 8, 256, 128, seed=9, gate_bias=True)
    d["gate_bias"][[0, 3, 4]] = -math.inf
    out, ids = check(d, R(2, renormalize=True))
    assert not np.isin(ids, [0, 3, 4]).any()
    o = on_gpu(d)
    x = o["x"].clone()
    x[2, 17] = float("nan")
    got = call(o, R(2, renormalize=True), x=x)
    assert (got[2] == 0).all()
    keep = [0, 1, 3, 4]
    assert torch.equal(got[keep].view(torch.int16), out[keep].view(torch.int16))
    # fewer live experts than topk; none at all
    d["gate_bias"][:7] = -math.inf
    check(d, R(3), layouts=("plain",))
    o["gate_bias"].fill_(-math.inf)
    assert (call(o, R(3)) == 0).all()


def test_non_finite_weights_stay_with_their_tokens():
    """NaN codes of an expert reach only the tokens that chose it."""
    d = make(False, 6, 4, 256, 128, seed=10)
    _, _, ids, _ = oracle(d, R(1))
    e = int(ids[0, 0])
    o = on_gpu(d)
    base = call(o, R(1))
    o["w2"][e, 5, 7] = 0x7F
    got = call(o, R(1))
    mine = torch.from_numpy((ids == e).any(1)).to(gpu())
    assert got[mine][:, 5].isnan().all()
    assert torch.equal(got[~mine].view(torch.int16), base[~mine].view(torch.int16))


def test_overflowing_intermediate():
    """An infinite intermediate gives infinite outputs, not NaN from its second term."""
    d = make(False, 1, 1, 128, 128, seed=11, w1_bias=True)
    d["w1_bias"][:] = 1e20
    d["w1_bias"][0, 128 + 3] = 3e38
    d["w2"][:] = 0x38  # 1.0
    out = call(on_gpu(d), R(1))
    assert (out == math.inf).all()


@pytest.mark.parametrize("mx", [False, True])
def test_strides_output_and_workspace(mx):
    d = make(mx, 3, 4, 256, 128, seed=12)
    o = on_gpu(d)
    r = R(2)
    want = call(o, r)
    wide = torch.zeros(5, 600, dtype=torch.bfloat16, device=gpu())
    wide[1:4, 8:264] = o["x"]
    assert torch.equal(call(o, r, x=wide[1:4, 8:264]), want)
    assert torch.equal(call(o, r, x=wide[1:2, 8:264].expand(3, 256)), call(o, r, x=o["x"][:1]).expand(3, 256))
    big = torch.full((4, 300), 5.0, dtype=torch.bfloat16, device=gpu())
    ws = ops.moe_layer_workspace(3, 256, 128, 4, 2, L.MXQ_WEIGHTS_MXFP4 if mx else L.MXQ_WEIGHTS_FP8_BLOCK, gpu())
    ws.fill_(0xFF)  # its contents do not matter
    got = call(o, r, out=big[:3, 7:263], workspace=ws)
    assert torch.equal(got, want)
    assert (big[3] == 5).all() and (big[:, :7] == 5).all() and (big[:, 263:] == 5).all()
    assert call(o, r, x=o["x"][:0]).shape == (0, 256)
    with pytest.raises(L.MxqError):
        call(o, r, workspace=ws[:-256])


@pytest.mark.parametrize("mx", [False, True])
def test_agrees_with_route_and_fused_moe(mx):
    """The operators together as they would be used: logits -> moe_route -> fused MoE gives the layer's
    output within the fused MoE's bf16 intermediates (1e-2, its own bar)."""
    d = make(mx, 12, 16, 512, 256, seed=13, gate_bias=True)
    o = on_gpu(d)
    r = R(4, renormalize=True)
    out = call(o, r).float()
    logits = o["x"].float() @ o["gate"].float().t() + o["gate_bias"]
    ids, w = ops.moe_route(logits, r)
    fn = ops.fused_moe_mxfp4 if mx else ops.fused_moe_fp8
    ref = fn(o["x"], ids, w, o["w1"], o["w1_scale"], o["w2"], o["w2_scale"], o["w1_bias"]).float()
    assert ((out - ref).abs() <= 1e-2 + 1e-2 * ref.abs()).all()


def test_decode_step_of_all_three_operators():
    """A decode step: 4-bit projection, routed layer, 4-bit projection, eager and as a captured graph
    replayed with new inputs between eager work, and two such steps on two streams at once."""
    d = make(True, 4, 8, 256, 128, seed=14)
    o = on_gpu(d)
    g = torch.Generator().manual_seed(15)
    w = torch.randint(0, 256, (256, 128), generator=g, dtype=torch.uint8).to(gpu())
    s = ((0.5 + torch.rand(256, 4, generator=g)) * 0.01).to(gpu())
    r = R(2, renormalize=True)

    def step(x):
        return ops.int4_linear(call(o, r, x=ops.int4_linear(x, w, s)), w, s)

    x = o["x"].clone()
    want = step(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x)
    for rep in range(4):
        x.copy_(torch.randn(4, 256, generator=g).to(torch.bfloat16).to(gpu()))
        graph.replay()
        torch.cuda.synchronize()
        first = got.clone()
        want = step(x)
        torch.cuda.synchronize()
        assert torch.equal(first.view(torch.int16), want.view(torch.int16)), rep
    xs = [x, x.flip(0).contiguous()]
    refs = [step(v) for v in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(4):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                outs[k].append(step(xs[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        for v in outs[k]:
            assert torch.equal(v.view(torch.int16), refs[k].view(torch.int16))


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("E,case", [(32, "saturated"), (64, "near"), (300, "saturated"), (512, "near"), (8, "near")])
def test_picks_closer_than_fp32_scores(mx, E, case):
    """Scores + bias that fp32 cannot tell apart choose the experts that moe_route chooses.  Token t's x
    is the t-th unit vector, so its logits are the router's t-th column, exact in fp32 in any order of
    summation.  saturated: sigmoids of logits in [17, 28], 1 - e^-17 at least, all 1 in fp32, largest
    logits last.  near: biases that leave only their own fp32 rounding between the picks."""
    M, H = 5, 256
    g = torch.Generator().manual_seed(E)
    logits = torch.randn(M, E, generator=g)
    bias = torch.zeros(E)
    if case == "saturated":
        n = E // 2
        logits[:, E - n:] = torch.sort(torch.rand(M, n, generator=g) * 11 + 17, dim=1)[0]
    else:
        logits = logits[:1].expand(M, E).contiguous()
    routers = [R(4, scoring="sigmoid", renormalize=True)]
    if E > 8:
        routers += [R(6, scoring="sigmoid", n_group=4, topk_group=2, group_score="top2")]
    if case == "near":
        routers += [R(4)]
    for r in routers:
        d = make(mx, M, E, H, 128, seed=E, gate_dtype=torch.float32)
        d["x"] = torch.eye(M, H).to(torch.bfloat16)
        d["gate"] = torch.zeros(E, H)
        d["gate"][:, :M] = logits.t()
        if case == "near":
            p = torch.softmax(logits[0].double(), 0) if r.scoring == "softmax" else torch.sigmoid(logits[0].double())
            bias = (0.7 - p).float()
        d["bias"] = bias
        want, bound, ids, _ = oracle(d, r)
        routed, _ = ops.moe_route(logits.to(gpu()), r, correction_bias=bias.to(gpu()))
        np.testing.assert_array_equal(routed.cpu().numpy(), ids)
        for lay in ("plain", "tiled"):
            got = call(on_gpu(d, lay), r, lay).double().cpu().numpy()
            assert (np.abs(got - want) <= HALF * np.abs(want) + bound).all(), (lay, r)


@pytest.mark.parametrize("mx", [False, True])
def test_infinite_activation_with_fp32_router(mx):
    """An infinite activation makes its token's logits +-inf by the sign of the router's weight there, with
    an fp32 router as with a bf16 one: the experts of +inf are chosen, and what they make of an infinity
    is no number -- while no expert (zeros) is only right where every logit is -inf."""
    d = make(mx, 6, 8, 256, 128, seed=21, gate_dtype=torch.float32)
    d["gate"][:, 70] = torch.tensor([1.1, -0.9, 1.3, -1.7, 0.7, -0.3, 2.9, -1.0])
    d["gate"][:, 71] = -d["gate"][:, 70].abs()
    r = R(2, renormalize=True)
    o = on_gpu(d)
    base = call(o, r)
    x = o["x"].clone()
    x[1, 70] = math.inf    # four experts of +inf
    x[2, 70] = -math.inf   # the other four
    x[3, 71] = math.inf    # none
    x[4, 71] = -math.inf   # all
    for gate in (o["gate"], o["gate"].to(torch.bfloat16)):
        out = call(dict(o, gate=gate), r, x=x)
        assert out[[1, 2, 4]].isnan().all() and (out[3] == 0).all()
        assert out[[0, 5]].isfinite().all()
    assert torch.equal(call(o, r, x=x)[[0, 5]], base[[0, 5]])
    # the product itself: one expert, whose weight's terms differ in sign; -inf leaves none
    one = make(mx, 2, 1, 256, 128, seed=22, gate_dtype=torch.float32)
    one["x"][:, 9] = math.inf
    for w, dead in ((1.0 + 2.0 ** -8 - 2.0 ** -20, False), (-1.0 - 2.0 ** -8 + 2.0 ** -20, True), (1.0, False)):
        one["gate"][0, 9] = w
        out = call(on_gpu(one), R(1))
        assert (out == 0).all() if dead else out.isnan().all(), w


def test_fp32_router_weights_above_bf16():
    """fp32 router weights beyond bf16's largest finite value stay finite; infinite and NaN ones do what they
    do in a bf16 router."""
    d = make(False, 2, 4, 256, 128, seed=23, gate_dtype=torch.float32)
    d["x"] = torch.zeros(2, 256, dtype=torch.bfloat16)
    d["x"][:, 3] = 2.0 ** -126
    d["x"][:, 4] = 1.0
    d["gate"] = torch.zeros(4, 256)
    d["gate"][:, 3] = torch.tensor([3.4e38, -3.4e38, 3.3e38, 1.0])  # logits 4.0, -4.0, 3.9, 0
    d["gate"][3, 4] = 5.0
    for k in (1, 2, 3):
        _, ids = check(d, R(k, renormalize=k > 1))
        assert ids[0].tolist() == [3, 0, 2][:k]
    o = on_gpu(d)
    o["gate"][0, 4], o["gate"][1, 4] = math.inf, -math.inf
    o["gate"][2, 4] = torch.tensor(0x7F800001, dtype=torch.int32).view(torch.float32)  # NaN in its last bit
    # the infinite one takes the whole weight, the NaN and -inf ones are out
    for r in (R(1), R(2, renormalize=True), R(4)):
        out = call(o, r)
        assert out.isfinite().all() and (out != 0).any()
        assert torch.equal(out, call(o, R(1)))
        assert torch.equal(out, call(dict(o, gate=o["gate"].clamp(-3.3e38, math.inf).to(torch.bfloat16)), r))


@pytest.mark.parametrize("mx", [False, True])
def test_one_row_slices_and_odd_offsets(mx):
    """A decoded token cut out of a wider or odd-strided buffer; contiguous rows at an odd offset; a
    misaligned weight or router is refused."""
    d = make(mx, 4, 4, 256, 128, seed=24)
    o = on_gpu(d)
    r = R(2)
    buf = torch.randn(6 * 520 + 1, device=gpu()).to(torch.bfloat16)
    for v in (buf[:6 * 301].view(6, 301)[:1, :256], buf[:3120].view(6, 520)[:1, 3:259], buf[1:513].view(2, 256),
              buf[5:261].view(1, 256), buf[:3 * 301].view(3, 301)[:, 8:264]):
        assert torch.equal(call(o, r, x=v), call(o, r, x=v.clone()))
    out = torch.full((1, 700), 3.0, dtype=torch.bfloat16, device=gpu())[:, 1:257]
    assert torch.equal(call(o, r, x=buf[None, 5:261], out=out), call(o, r, x=buf[None, 5:261].clone()))
    for name in ("gate", "w1", "w2"):
        t = o[name]
        odd = torch.zeros(t.numel() + 4, dtype=t.dtype, device=gpu())[4:].view(t.shape)
        with pytest.raises(ValueError, match=f"{name} must start"):
            call(dict(o, **{name: odd}), r)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_intermediate_above_bf16(sign):
    """A finite intermediate beyond bf16's largest value stays finite in its two terms.  (MXFP4, whose
    weights carry their scales; FP8 scales a block's fp32 sum of products with codes of up to 448,
    which overflows from intermediates of 3.4e38 / 448 on.)"""
    d = make(True, 2, 1, 256, 128, seed=25)
    d["w1_bias"][:] = 0.0
    d["w1_bias"][0, 7] = 1e20                # silu of it is itself
    d["w1_bias"][0, 128 + 7] = sign * 3.4e18  # their product 3.4e38, between bf16's largest and fp32's
    d["w2_scale"] = d["w2_scale"] - 20
    out, _ = check(d, R(1))
    assert out.isfinite().all() and out.abs().max() > 1e30


def _shares(d, chosen, topk):
    """Waves of a workgroup that share a gate/up item when `chosen` experts are chosen: the kernel's rule."""
    M, H = d["x"].shape
    E, tiles, steps = d["gate"].shape[0], d["w2"].shape[2] * (2 if d["mx"] else 1) // 16, -(-H // (256 if d["mx"] else 128))
    waves, n = 8 * min(256, -(-min(E, M * topk) * tiles // 8)), 1
    while n < 8 and 2 * n * chosen * tiles <= waves and 4 * n <= steps:
        n *= 2
    return 1 if n == 2 else n


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("M,E,H,I,topk,want", [
    (16, 16, 2048, 128, 1, 8), (8, 8, 2176, 256, 1, 8), (16, 16, 2176, 128, 1, 8), (16, 32, 2304, 128, 2, 8),
    (8, 8, 1024, 128, 1, 4), (4, 16, 1152, 256, 1, 4), (5, 8, 2048, 128, 2, 4), (16, 16, 640, 128, 1, 1), (2, 8, 2048, 128, 2, 1)])
def test_tokens_that_agree_on_few_experts(mx, M, E, H, I, topk, want):
    """Tokens on the same experts, which leave waves over that share items: eight, four or none, in steps that
    do and do not divide by their number.  (MXFP4 at twice the columns, whose steps are twice as wide.)"""
    H = H * 2 if mx else H
    d = make(mx, M, E, H, I, seed=M + E + H, w1_bias=True, gate_bias=False)
    d["x"] = d["x"][:1] * torch.exp2(torch.arange(M) % 4 - 2.0).to(torch.bfloat16)[:, None]
    out, ids = check(d, R(topk, renormalize=True))
    chosen = len(np.unique(ids))
    assert chosen == topk and _shares(d, chosen, topk) == want


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("M,E,topk", [(16, 32, 32), (16, 64, 31), (16, 40, 29), (15, 32, 32), (1, 32, 32)])
def test_largest_topk(mx, M, E, topk):
    """The most rows that a call can have: the sums of the down stage's rows fill a compute unit's LDS."""
    check(make(mx, M, E, 256, 128, seed=M + E + topk), R(topk, renormalize=True))


@pytest.mark.parametrize("mx", [False, True])
def test_one_workspace_for_calls_in_a_row(mx):
    """Calls one after the other on a stream may use one workspace, whatever their sizes; a call in several
    passes, captured and replayed; out may be x itself."""
    weights = L.MXQ_WEIGHTS_MXFP4 if mx else L.MXQ_WEIGHTS_FP8_BLOCK
    H = 16384 if mx else 8192
    big, small = on_gpu(make(mx, 16, 4, H, 128, seed=30)), on_gpu(make(mx, 3, 24, 256, 128, seed=31))
    r = R(2, renormalize=True)
    ws = ops.moe_layer_workspace(16, H, 128, 24, 2, weights, gpu())
    want = [call(big, r), call(small, r)]
    for _ in range(3):
        got = [call(big, r, workspace=ws), call(small, r, workspace=ws)]
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    x = big["x"].clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = call(big, r, x=x, workspace=ws)
    g = torch.Generator().manual_seed(32)
    for rep in range(4):
        x.copy_(torch.randn(16, H, generator=g))
        graph.replay()
        ref = call(big, r, x=x, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(out, ref), rep
    for o, w in ((big, want[0]), (small, want[1])):
        y = o["x"].clone()
        assert call(o, r, x=y, out=y).data_ptr() == y.data_ptr() and torch.equal(y, w)
