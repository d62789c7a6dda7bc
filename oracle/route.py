"""Oracle expert routing (test infrastructure only): one token at a time, float64 scalars.

Definition (the routing the fused MoE's ``topk_ids`` / ``topk_weights`` come from):

* an expert is live when its logit is greater than -inf (NaN is not);
* softmax scores ``exp(l - max l) / sum`` over the live experts, or sigmoid scores;
* the pick of an expert is its score plus the correction bias, or its logit without one;
* with groups, a group's score is its largest pick, or the sum of its two largest score + bias,
  and only the ``topk_group`` best groups (ties: the lower group) keep their experts;
* the ``topk`` largest picks, ties to the lower expert; missing ones get id -1, weight 0;
* weights are the scores, renormalised over the chosen experts or not, times ``scale``.  The
  renormalised weight is a ratio of scores, evaluated through their logarithms.
"""

import math

import numpy as np

NEG = -math.inf


def log_sigmoid(v: float) -> float:
    return -math.log1p(math.exp(-v)) if v >= 0 else v - math.log1p(math.exp(v))


def _scores(l, sigmoid):
    """{expert: (score, log score)} of the live experts."""
    live = [e for e, v in enumerate(l) if v > NEG]
    if sigmoid:
        return {e: (1.0 if l[e] == math.inf else math.exp(log_sigmoid(l[e])),
                    0.0 if l[e] == math.inf else log_sigmoid(l[e])) for e in live}
    if not live:
        return {}
    top = max(l[e] for e in live)
    rel = {e: 0.0 if l[e] == top else l[e] - top for e in live}
    total = math.fsum(math.exp(v) for v in rel.values())
    return {e: (math.exp(rel[e]) / total, rel[e] - math.log(total)) for e in live}


def route_token(logits, topk, sigmoid=False, bias=None, n_group=1, topk_group=1, top2=False, renormalize=False,
                scale=1.0):
    """(ids, weights, smallest gap between two picks or group scores that decide the result)."""
    l = [float(v) for v in logits]
    E = len(l)
    sc = _scores(l, sigmoid)
    pick = {e: (s[0] + float(bias[e]) if bias is not None else l[e]) for e, s in sc.items()}
    pick = {e: v for e, v in pick.items() if v > NEG}
    gap = math.inf
    if n_group > 1:
        size = E // n_group
        value = {}
        for g in range(n_group):
            own = [e for e in pick if e // size == g]
            if not own:
                continue
            if top2:
                v = sorted(((sc[e][0] + (float(bias[e]) if bias is not None else 0.0)) for e in own), reverse=True)
                value[g] = sum(v[:2])
            else:
                value[g] = max(pick[e] for e in own)
        order = sorted(value, key=lambda g: (-value[g], g))
        if len(order) > topk_group:
            gap = min(gap, value[order[topk_group - 1]] - value[order[topk_group]])
        kept = set(order[:topk_group])
        pick = {e: v for e, v in pick.items() if e // size in kept}
    order = sorted(pick, key=lambda e: (-pick[e], e))
    for a, b in zip(order[:topk], order[1:topk + 1]):
        gap = min(gap, pick[a] - pick[b])
    chosen = order[:topk]
    if renormalize and chosen:
        top = max(sc[e][1] for e in chosen)
        rel = [math.exp(sc[e][1] - top) for e in chosen]
        w = [v / math.fsum(rel) * scale for v in rel]
    else:
        w = [sc[e][0] * scale for e in chosen]
    pad = topk - len(chosen)
    return chosen + [-1] * pad, w + [0.0] * pad, gap


def route(logits, topk, **kw):
    """logits [M, E] -> (ids int32 [M, topk], weights float64 [M, topk], smallest deciding gap)."""
    rows = [route_token(r, topk, **kw) for r in np.asarray(logits, np.float64)]
    ids = np.array([r[0] for r in rows], np.int32).reshape(len(rows), topk)
    w = np.array([r[1] for r in rows], np.float64).reshape(len(rows), topk)
    return ids, w, min([r[2] for r in rows], default=math.inf)
