"""mxq_moe_route against the float64 oracle: ids and their order exactly, weights within fp32.

Tolerance of the weights: an fp32 exponential (2 ulp), a sum over at most 512 experts in a tree
(9 roundings), a division and the scale, each 2^-24 relative, on both sides of the renormalising
quotient: below 32 * 2^-24 = 2^-19.
"""

import math

import numpy as np
import pytest
import torch

from mxfp4_block_scaled_expert_amd import ops
from oracle.route import route
from tests._util import gpu

pytestmark = pytest.mark.gpu
RTOL = 2.0 ** -19


def _check(logits, router, bias=None, rtol=RTOL):
    """logits: CPU tensor.  Runs the operator and compares."""
    b = None if bias is None else bias.to(gpu())
    ids, w = ops.moe_route(logits.to(gpu()), router, correction_bias=b)
    torch.cuda.synchronize()
    want_ids, want_w, _ = route(logits.double().numpy(), router.topk, sigmoid=router.scoring == "sigmoid",
                                bias=None if bias is None else bias.double().numpy(), n_group=router.n_group,
                                topk_group=router.topk_group, top2=router.group_score == "top2",
                                renormalize=router.renormalize, scale=router.scale)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    np.testing.assert_allclose(w.double().cpu().numpy(), want_w, rtol=rtol, atol=1e-37)
    return ids, w


def _logits(M, E, seed, dtype=torch.float32, std=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, E, generator=g) * std).to(dtype)


R = ops.Router
CASES = [
    (1, 1, R(1)), (1, 2, R(2, renormalize=True)), (3, 5, R(5)), (1, 128, R(4, renormalize=True)),
    (32, 128, R(4)), (33, 60, R(6, scoring="sigmoid")), (7, 64, R(8, renormalize=True, scale=2.5)),
    (5, 65, R(3)), (9, 129, R(2, scoring="sigmoid", renormalize=True)), (6, 257, R(7)), (4, 511, R(32)),
    (130, 512, R(8, renormalize=True)),
    (17, 256, R(8, scoring="sigmoid", n_group=8, topk_group=4, group_score="top2", renormalize=True, scale=2.5)),
    (17, 160, R(6, n_group=8, topk_group=3)), (8, 72, R(4, n_group=36, topk_group=5, group_score="top2")),
    (8, 64, R(3, n_group=64, topk_group=3, group_score="top2")), (8, 512, R(8, n_group=2, topk_group=1)),
    (8, 510, R(5, scoring="sigmoid", n_group=3, topk_group=2, group_score="top2")),
]


@pytest.mark.parametrize("M,E,router", CASES)
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_matches_oracle(M, E, router, with_bias, dtype):
    g = torch.Generator().manual_seed(E)
    bias = torch.randn(E, generator=g) * 0.1 if with_bias else None
    _check(_logits(M, E, M * 1000 + E, dtype), router, bias)


def test_many_tokens_with_grouped_scores():
    r = R(8, scoring="sigmoid", n_group=8, topk_group=4, group_score="top2", renormalize=True, scale=2.5)
    g = torch.Generator().manual_seed(3)
    _check(_logits(3001, 256, 11), r, torch.randn(256, generator=g) * 0.1)


@pytest.mark.parametrize("router", [R(4), R(4, renormalize=True), R(4, scoring="sigmoid", renormalize=True),
                                    R(4, n_group=4, topk_group=2), R(4, n_group=4, topk_group=2, group_score="top2")])
def test_masked_logits(router):
    """-inf, NaN, +inf and the type's lowest value; rows with nothing, one and few live experts."""
    inf, nan, low = math.inf, math.nan, torch.finfo(torch.float32).min
    l = _logits(10, 16, 5)
    l[0] = -inf
    l[1] = nan
    l[2] = -inf
    l[2, 9] = 0.5
    l[3, ::2] = nan
    l[4, 5:] = -inf
    l[5] = low
    l[6, :] = -inf
    l[6, [1, 14]] = torch.tensor([low, 3.0])
    l[7, 3] = inf
    l[7, 12] = inf
    l[8] = 0.0
    l[9, :8] = -inf
    _check(l, router)


def test_masking_through_the_bias():
    """A bias of -inf (or NaN) takes its expert out, +inf puts it first."""
    l = _logits(6, 12, 8)
    bias = torch.zeros(12)
    bias[[2, 7]] = -math.inf
    bias[5] = math.inf
    _check(l, R(11, scoring="sigmoid", renormalize=True), bias)
    _check(l, R(3), bias)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_ties_go_to_the_lowest_index(scoring, group_score):
    g = torch.Generator().manual_seed(2)
    l = torch.randint(-2, 3, (64, 96), generator=g).float()
    for r in (R(6, scoring=scoring), R(6, scoring=scoring, n_group=8, topk_group=3, group_score=group_score)):
        _check(l, r)
        _check(l, r, torch.full((96,), 0.25))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_picks_closer_than_fp32_scores(scoring):
    """Biases that make all scores + bias nearly equal: only the fp32 rounding of the bias (2^-25
    relative, far below what an fp32 score resolves) tells them apart, and it has to."""
    for seed in range(4):
        l = _logits(1, 64, 40 + seed)
        p = torch.softmax(l.double(), 1) if scoring == "softmax" else torch.sigmoid(l.double())
        bias = (0.7 - p[0]).float()
        _check(l.expand(8, 64).contiguous(), R(8, scoring=scoring), bias)
        _check(l, R(8, scoring=scoring, n_group=8, topk_group=3, group_score="top2"), bias)


def test_extreme_logits():
    l = torch.tensor([[1e30, -1e30, 3e38, -3e38, 0.0, 88.0, -104.0, 1e-40]])
    for r in (R(8), R(8, scoring="sigmoid"), R(4, renormalize=True), R(8, scoring="sigmoid", renormalize=True)):
        _check(l, r)
    # sigmoid scores that underflow in fp32 keep their ratio when renormalised
    _check(torch.tensor([[-200.0, -201.0, -230.0, -199.5]]), R(3, scoring="sigmoid", renormalize=True))


def test_strides_views_and_empty():
    wide = _logits(9, 200, 3).to(gpu())
    view = wide[1:, 7:107]  # odd element offset, row stride 200
    ids, w = ops.moe_route(view, R(4))
    i2, w2 = ops.moe_route(view.contiguous(), R(4))
    assert torch.equal(ids, i2) and torch.equal(w, w2)
    t = ops.moe_route(wide.t()[:64], R(2))
    t2 = ops.moe_route(wide.t()[:64].contiguous(), R(2))
    assert torch.equal(t[0], t2[0]) and torch.equal(t[1], t2[1])
    e = ops.moe_route(wide[:1].expand(4, 200), R(2))
    assert torch.equal(e[0], ops.moe_route(wide[:1], R(2))[0].expand(4, 2))
    ids, w = ops.moe_route(wide[:0], R(4))
    assert ids.shape == (0, 4) and w.shape == (0, 4)


def test_rows_behind_the_last_are_left_alone():
    from mxfp4_block_scaled_expert_amd import _lib as L
    l = _logits(5, 40, 9).to(gpu())
    ids = torch.full((8, 3), -7, dtype=torch.int32, device=gpu())
    w = torch.full((8, 3), -7.0, device=gpu())
    st = L.load().mxq_moe_route(l.data_ptr(), L.MXQ_DTYPE_F32, 5, 40, 40, ops._router(R(3)), None, ids.data_ptr(),
                                w.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and (ids[5:] == -7).all() and (w[5:] == -7).all() and (ids[:5] >= 0).all()


@pytest.mark.parametrize("M,E,router", [
    (2049, 256, R(8, scoring="sigmoid", n_group=8, topk_group=4, group_score="top2", renormalize=True, scale=2.5)),
    (1027, 64, R(16, renormalize=True)), (1500, 60, R(6, scoring="sigmoid")), (1025, 3, R(3)),
    (1030, 128, R(4, scoring="sigmoid", renormalize=True)), (1201, 128, R(6, n_group=4, topk_group=2)),
    (1100, 257, R(7)), (1040, 512, R(8, n_group=2, topk_group=1, group_score="top2")), (1090, 510, R(17)),
    (1111, 160, R(6, n_group=8, topk_group=3)), (1033, 64, R(3, scoring="sigmoid", n_group=16, topk_group=5)),
    (1029, 40, R(3, n_group=5, topk_group=2, group_score="top2")), (1031, 20, R(2, n_group=5, topk_group=5))])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_tokens(M, E, router, with_bias, dtype):
    g = torch.Generator().manual_seed(E)
    bias = torch.randn(E, generator=g) * 0.1 if with_bias else None
    l = _logits(M, E, M + E, dtype)
    l[5] = -math.inf
    l[6] = math.nan
    l[7, 1:] = -math.inf
    l[8] = 0.0
    l[9, E // 2:] = -math.inf
    l[M - 1, 0] = math.inf
    l[M - 2] = torch.finfo(dtype).min
    _check(l, router, bias)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_many_tokens_ties_and_close_picks(scoring):
    g = torch.Generator().manual_seed(2)
    l = torch.randint(-2, 3, (1100, 96), generator=g).float()
    for r in (R(6, scoring=scoring), R(6, scoring=scoring, n_group=8, topk_group=3, group_score="top2"),
              R(6, scoring=scoring, n_group=4, topk_group=2)):
        _check(l, r)
        _check(l, r, torch.full((96,), 0.25))
    # half of the tokens have scores + bias nearer to each other than fp32 scores resolve
    one = _logits(1, 64, 40)
    p = torch.softmax(one.double(), 1) if scoring == "softmax" else torch.sigmoid(one.double())
    l = torch.cat([one.expand(600, 64), _logits(600, 64, 41)])[torch.randperm(1200, generator=g)].contiguous()
    for r in (R(8, scoring=scoring), R(8, scoring=scoring, n_group=8, topk_group=3, group_score="top2")):
        _check(l, r, (0.7 - p[0]).float())


def test_many_tokens_strides():
    wide = _logits(1100, 200, 3).to(gpu())
    for r in (R(4), R(4, n_group=5, topk_group=2)):
        for view in (wide[:, 7:107], wide[:, 8:108], wide[1:, :100]):  # unaligned and aligned rows
            a, b = ops.moe_route(view, r), ops.moe_route(view.contiguous(), r)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        # the same tokens in a call of few
        few = ops.moe_route(wide[:40, :100], r)
        many = ops.moe_route(wide[:, :100], r)
        assert torch.equal(few[0], many[0][:40])
        torch.testing.assert_close(few[1], many[1][:40], rtol=2 * RTOL, atol=0)


@pytest.mark.parametrize("M", [9, 1101])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("big", [30.0, 3e3, 1e4, 1e5, 1e7])
def test_group_scores_whose_terms_cancel(M, scoring, big):
    """Top-2 group scores of biases near +big and -big: what fp32 rounds off the terms is far above the
    distance of the sums, between neighbours in the order of groups and beyond them."""
    g = torch.Generator().manual_seed(int(big))
    E, n = 64, 8
    bias = torch.full((n, E // n), -2 * big)
    bias[:, 3] = big * (1 + torch.arange(n) * 0.25)
    bias[:, 6] = -big * (1 + torch.arange(n) * 0.25)
    bias = bias.reshape(-1)
    for topk_group in (1, 3, 7):
        _check(_logits(M, E, int(big) + M), R(topk_group, scoring=scoring, n_group=n, topk_group=topk_group,
                                             group_score="top2"), bias)
    bias[::8] += torch.randn(n, generator=g) * big  # some groups with ordinary scores among them
    _check(_logits(M, E, int(big) + M + 1), R(4, scoring=scoring, n_group=n, topk_group=4, group_score="top2"), bias)


@pytest.mark.parametrize("M", [5, 1030])
def test_group_scores_beyond_fp32(M):
    """Sums of two terms that overflow fp32, upward and downward, are told apart; infinite biases too."""
    big = torch.tensor([3.0e38, 3.2e38, 2.9e38, 3.3e38, -3.0e38, -3.2e38, -2.0e38, 1.0])
    bias = (big[:, None] * torch.tensor([0.9, 1.0, 0.8, 0.99])).reshape(-1)
    r = dict(scoring="sigmoid", n_group=8, group_score="top2")
    for topk_group in (1, 2, 3, 5, 6, 7):
        _check(_logits(M, 32, 60), R(4 * topk_group, topk_group=topk_group, **r), bias)
    _check(_logits(M, 32, 61), R(4, topk_group=1, **r), -bias.abs())
    bias = torch.zeros(32)
    bias[[5, 21]] = math.inf
    bias[9] = -math.inf
    for topk_group in (1, 2, 3):
        _check(_logits(M, 32, 62), R(2, topk_group=topk_group, **r), bias)


@pytest.mark.parametrize("M", [40, 1500])
@pytest.mark.parametrize("std", [4.0, 10.0])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_confident_routers(M, std, scoring):
    """Logits so large that most scores are near 0 or 1, with no, small and ordinary biases.  A weight's
    exponential takes the difference of two logits, which fp32 rounds by 2^-24 of it: that far apart,
    differences of up to D add D 2^-24 to the tolerance of a weight."""
    g = torch.Generator().manual_seed(M)
    for bias in (torch.zeros(256), torch.randn(256, generator=g) * 1e-6, torch.randn(256, generator=g) * 0.1):
        for r in (R(8, scoring=scoring, n_group=8, topk_group=4, group_score="top2", renormalize=True), R(8, scoring=scoring),
                  R(6, scoring=scoring, n_group=8, topk_group=3)):
            l = _logits(M, 256, M, std=std).clamp(max=30.0)
            _check(l, r, bias, rtol=RTOL + float(l.max() - l.min()) * 2.0 ** -24)


def test_captured_and_on_two_streams():
    """Captured calls of both kernels replayed with new logits between eager calls, and both on streams of
    their own at once."""
    r = R(8, scoring="sigmoid", n_group=8, topk_group=4, group_score="top2", renormalize=True)
    g = torch.Generator().manual_seed(7)
    bias = (torch.randn(256, generator=g) * 0.1).to(gpu())
    ls = [_logits(M, 256, 70 + M).to(gpu()) for M in (3, 2050)]
    graphs, outs = [], []
    for l in ls:
        ops.moe_route(l, r, correction_bias=bias)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(ops.moe_route(l, r, correction_bias=bias))
    for rep in range(4):
        for l, graph, out in zip(ls, graphs, outs):
            l.copy_(torch.randn(l.shape, generator=g) * (rep + 1))
            graph.replay()
            want = ops.moe_route(l, r, correction_bias=bias)
            torch.cuda.synchronize()
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), rep
    want = [ops.moe_route(l, r, correction_bias=bias) for l in ls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                got[k].append(ops.moe_route(ls[k], r, correction_bias=bias))
    torch.cuda.synchronize()
    for k in (0, 1):
        for ids, w in got[k]:
            assert torch.equal(ids, want[k][0]) and torch.equal(w, want[k][1])
