"""Oracle MoE layer (test infrastructure only): router product, routing, experts and combine of a few
tokens in float64, without intermediate roundings.

``out[t] = sum_j (w[t, j] * silu(g) * u) @ w2[e]^T`` with ``[g | u] = x[t] @ w1[e]^T + b1[e]`` and
``(e, w) = route(x @ gate^T + gate_bias)``.

``layer`` also returns, per output, a bound on what an implementation may differ by before its last
rounding: fp32 sums of n terms (n 2^-24 of the sum of magnitudes), the intermediate kept to 2^-16 of
itself (two bf16 terms, each rounded by at most 2^-8 of what it holds), and 2^-20 for the
exponential, the division and the routing weight.
"""

import numpy as np

from .moe import dequant_fp8_expert, dequant_mxfp4_expert
from .route import route


def expert_weight(codes, scale, mxfp4):
    f = dequant_mxfp4_expert if mxfp4 else dequant_fp8_expert
    return f(np.asarray(codes), np.asarray(scale)).astype(np.float64)


def router_logits(x, gate, gate_bias=None):
    l = np.asarray(x, np.float64) @ np.asarray(gate, np.float64).T
    return l if gate_bias is None else l + np.asarray(gate_bias, np.float64)[None, :]


def layer(x, gate, w1, s1, w2, s2, mxfp4, router, gate_bias=None, correction_bias=None, b1=None):
    """(out float64 [M, H], bound float64 [M, H], ids, smallest deciding routing gap)."""
    x = np.asarray(x, np.float64)
    M, H = x.shape
    ids, wt, gap = route(router_logits(x, gate, gate_bias), bias=correction_bias, **router)
    out, bound = np.zeros((M, H)), np.zeros((M, H))
    u24 = 2.0 ** -24
    for e in sorted(set(int(v) for v in ids.reshape(-1) if v >= 0)):
        t, j = np.nonzero(ids == e)
        W1 = expert_weight(w1[e], s1[e], mxfp4)
        W2 = expert_weight(w2[e], s2[e], mxfp4)
        I = W2.shape[1]
        v = x[t] @ W1.T
        mag = np.abs(x[t]) @ np.abs(W1).T
        if b1 is not None:
            v = v + np.asarray(b1[e], np.float64)[None, :]
            mag = mag + np.abs(np.asarray(b1[e], np.float64))[None, :]
        dv = (H + 8) * u24 * mag
        g, u = v[:, :I], v[:, I:]
        with np.errstate(over="ignore"):
            act = g / (1.0 + np.exp(-g))
        w = wt[t, j][:, None]
        h = w * act * u
        # |silu'| <= 1.1
        dh = np.abs(w) * (1.1 * dv[:, :I] * np.abs(u) + (np.abs(act) + 1.1 * dv[:, :I]) * dv[:, I:])
        dh = dh + np.abs(h) * (2.0 ** -16 + 2.0 ** -20)
        out[t] += h @ W2.T
        bound[t] += dh @ np.abs(W2).T + (I + 64) * u24 * (np.abs(h) @ np.abs(W2).T)
    return out, bound, ids, gap
