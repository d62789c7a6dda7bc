"""Pins for the oracles of the routing, the few-token layer and the 4-bit linear: a second
construction, closed forms and invariants."""

import itertools
import math

import numpy as np
import pytest

from oracle.int4 import int4_linear, unpack4
from oracle.layer import layer
from oracle.moe import fused_moe_fp8, fused_moe_mxfp4
from oracle.route import route, route_token


def _numpy_route(l, topk, sigmoid, bias, n_group, topk_group, top2, renormalize, scale):
    """The same routing written with arrays: stable descending argsorts."""
    l = np.asarray(l, np.float64)
    p = 1 / (1 + np.exp(-l)) if sigmoid else np.exp(l - l.max()) / np.exp(l - l.max()).sum()
    pick = p + bias if bias is not None else l
    if n_group > 1:
        val = (p + (bias if bias is not None else 0)) if top2 else pick
        grp = np.sort(val.reshape(n_group, -1), axis=1)[:, ::-1]
        gs = grp[:, :2].sum(axis=1) if top2 else grp[:, 0]
        keep = np.argsort(-gs, kind="stable")[:topk_group]
        mask = np.isin(np.arange(l.size) // (l.size // n_group), keep)
        pick = np.where(mask, pick, -np.inf)
    ids = np.argsort(-pick, kind="stable")[:topk]
    w = p[ids] / p[ids].sum() if renormalize else p[ids]
    return ids, w * scale


@pytest.mark.parametrize("sigmoid,with_bias,top2,renormalize", list(itertools.product((False, True), repeat=4)))
def test_route_matches_array_form(sigmoid, with_bias, top2, renormalize):
    rng = np.random.default_rng(5)
    for E, n_group, topk_group, topk in ((8, 1, 1, 2), (24, 4, 2, 5), (60, 6, 3, 4)):
        for _ in range(5):
            l = rng.normal(size=E) * 2
            b = rng.normal(size=E) * 0.2 if with_bias else None
            ids, w, _ = route_token(l, topk, sigmoid, b, n_group, topk_group, top2, renormalize, 1.5)
            ri, rw = _numpy_route(l, topk, sigmoid, b, n_group, topk_group, top2, renormalize, 1.5)
            assert list(ri) == ids
            np.testing.assert_allclose(w, rw, rtol=1e-12)


def test_route_masks_ties_and_empty_rows():
    inf, nan = math.inf, math.nan
    ids, w, _ = route([[1, 1, 1, 1], [-inf, 2, nan, 2], [-inf, -inf, nan, -inf], [3, inf, 0, inf]], 3)
    assert ids.tolist() == [[0, 1, 2], [1, 3, -1], [-1, -1, -1], [1, 3, 0]]
    np.testing.assert_allclose(w, [[.25, .25, .25], [.5, .5, 0], [0, 0, 0], [.5, .5, 0]])
    # renormalised weights of scores far below the maximum keep their ratio
    ids, w, _ = route([[500.0, 0.0, 0.0, -math.log(3)]], 2, bias=np.array([-9.0, 0, 0, 0.5]), renormalize=True)
    assert ids.tolist() == [[3, 1]]
    np.testing.assert_allclose(w, [[.25, .75]])


def test_unpack4_order():
    assert unpack4(np.array([[0x21, 0x43]], np.uint8), 3).tolist() == [[1, 2, 3]]


def test_int4_linear_by_loops():
    rng = np.random.default_rng(1)
    N, K, G = 3, 96, 32
    p = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    z = rng.integers(0, 256, (N, 2), dtype=np.uint8)
    s = rng.random((N, 3))
    x = rng.normal(size=(2, K))
    got = int4_linear(x, p, s, z, G, bias=np.arange(3))
    for m in range(2):
        for n in range(N):
            acc = 0.0
            for k in range(K):
                q = (int(p[n, k // 2]) >> (4 * (k % 2))) & 15
                g = k // G
                acc += x[m, k] * (q - ((int(z[n, g // 2]) >> (4 * (g % 2))) & 15)) * s[n, g]
            assert abs(got[m, n] - (acc + n)) < 1e-9
    # no zero points: 8 everywhere
    np.testing.assert_allclose(int4_linear(x, p, s, None, G),
                               int4_linear(x, p, s, np.full((N, 2), 0x88, np.uint8), G))


@pytest.mark.parametrize("mxfp4", [False, True])
def test_layer_agrees_with_route_and_fused_moe(mxfp4):
    """Layer = router product + routing + the fused MoE oracle, within that one's bf16 roundings."""
    import torch
    from mxfp4_block_scaled_expert_amd import synth
    from tests._util import bf16_bits, bits_to_float, u8
    E, H, I, topk, M = 6, 256, 128, 2, 5
    d = (synth.moe_mxfp4_weights if mxfp4 else synth.moe_fp8_weights)(E, H, I, seed=3)
    g = torch.Generator().manual_seed(4)
    x = synth.bf16_randn((M, H), g, "cpu")
    gate = torch.randn(E, H, generator=g) / 16
    b1 = d.get("w1_bias")
    args = [u8(d["w1"]), d["w1_scale"].numpy(), u8(d["w2"]), d["w2_scale"].numpy()]
    out, bound, ids, gap = layer(x.float().numpy(), gate.numpy(), *args, mxfp4,
                                 dict(topk=topk, renormalize=True), b1=None if b1 is None else b1.numpy())
    _, w, _ = route(x.double().numpy() @ gate.double().numpy().T, topk, renormalize=True)
    fn = fused_moe_mxfp4 if mxfp4 else fused_moe_fp8
    kw = {} if mxfp4 else {"act_quant": False}
    want = bits_to_float(fn(bf16_bits(x), ids, w.astype(np.float32), *args, None if b1 is None else b1.numpy(), **kw))
    assert np.abs(out - want).max() <= 2e-2 * np.abs(want).max()
    assert np.linalg.norm(out - want) <= 1e-2 * np.linalg.norm(want)
    assert (bound >= 0).all() and bound.max() < 2.0 ** -6 * np.abs(out).max() and gap > 0
