"""Oracle of the feed-forward operators (test infrastructure): the INT8 format, the
routing to experts and the experts' feed forward, in float64 from their definitions.
Inputs and outputs are exact values (float64 arrays).

INT8     per row: s = fl32(max |v| / 127), r = fl32(1 / s) (0 when s = 0, the largest
         finite float32 when it overflows), q = rint(fl32(v r)), ties to even; a row
         with a value that is not finite has scale NaN.
Route    an expert is available where its logit is neither NaN nor -inf (+inf counts
         as the largest finite float32), and can be chosen where its bias is neither,
         either. s = softmax over the available experts or the sigmoid. c = s + bias,
         without a bias the logit. Groups of neighbours: a
         group's score is the sum of its two largest c (s without a bias) over available
         experts, a lone one counting alone; only the best `top_groups` groups that have
         an available expert take part. The k largest c, ties to the lowest index;
         w = s, divided by their sum if asked (0 if the sum is 0), times scale. A place
         that no expert fills: expert -1, weight 0.
Experts  u = x_q Wu_e^T + bu_e, h = fl32(act(u)), d = h_q Wd_e^T + bd_e,
         y_t = residual_t + sum_j w_tj d_tj over the places whose expert is in [0, E).
"""

import math

import numpy as np

MAX32 = np.float32(3.4028234663852886e38)


def quant_int8(v):
    """(codes int8, scales float32) of float32 rows v [M, K]."""
    v = np.asarray(v, dtype=np.float32)
    a = np.abs(v).max(axis=-1)
    bad = ~np.isfinite(v).all(axis=-1)
    with np.errstate(all="ignore"):
        s = (a / np.float32(127)).astype(np.float32)
        r = np.where(s > 0, np.minimum(np.float32(1) / s, MAX32), np.float32(0)).astype(np.float32)
        q = np.rint((v * r[..., None]).astype(np.float32))
    q = np.where(bad[..., None], 0, q)
    return q.astype(np.int8), np.where(bad, np.float32(np.nan), s).astype(np.float32)


def dequant_int8(codes, scales):
    return codes.astype(np.float64) * scales.astype(np.float64)[..., None]


def route(logits, k, score="softmax", bias=None, groups=1, top_groups=1, renormalize=True, scale=1.0):
    """(weights float64 [T, k], experts int [T, k]) of float64 logits [T, E]."""
    T, E = logits.shape
    w, ids = np.zeros((T, k)), np.full((T, k), -1)
    for t in range(T):
        z = np.minimum(logits[t], float(MAX32))
        free = [e for e in range(E) if not np.isnan(z[e]) and z[e] > -np.inf]
        if not free:
            continue
        if score == "softmax":
            top = max(z[e] for e in free)
            total = math.fsum(math.exp(z[e] - top) for e in free)
            s = {e: math.exp(z[e] - top) / total for e in free}
        else:
            s = {e: 1 / (1 + math.exp(-z[e])) if z[e] > -700 else math.exp(max(z[e], -800)) for e in free}
        c = {e: s[e] + float(bias[e]) if bias is not None else z[e] for e in free}
        free = [e for e in free if c[e] > -np.inf]  # not where c is NaN
        if groups > 1:
            n = E // groups
            by = c if bias is not None else s
            best = []
            for g in range(groups):
                own = sorted((by[e] for e in free if e // n == g), reverse=True)[:2]
                if own:
                    best.append((-sum(own), g))
            keep = {g for _, g in sorted(best)[:top_groups]}
            free = [e for e in free if e // n in keep]
        chosen = sorted(free, key=lambda e: (-c[e], e))[:k]
        v = np.array([s[e] for e in chosen])
        if renormalize:
            v = v / v.sum() if v.sum() > 0 else 0 * v
        w[t, :len(chosen)], ids[t, :len(chosen)] = v * scale, chosen
    return w, ids
