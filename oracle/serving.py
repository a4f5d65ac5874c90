"""Oracle of the 8-bit serving operators (test infrastructure): the norm with
an 8-bit output, the fused epilogue, the paged 8-bit cache and the attention
over it, in float64 from their definitions. Inputs and outputs are exact
values (float64 arrays); codes come from the sibling formats' oracle.

Norm      h = x + r, y = h / sqrt(mean(h^2) + eps) * w.
Epilogue  y = act(z) + residual with z = alpha * (x_hat @ w_hat^T) + bias;
          swiglu pairs 16 gate columns with the 16 up columns after them.
Append    per (block, head): a = max |v| over the new finite values,
          e = min {e : a <= 448 2^e} in [-127, 127] (-127 for a = 0);
          E = e in a block that starts with new tokens, else max(E_old, e);
          codes = E4M3_RNE_satfinite(v 2^-E), NaN kept; codes held before are
          rounded again to 2^(E_old - E) times their value.
Attention o = sum_j p_j v_j / sum_j p_j over the visible keys, p_j =
          exp(s_j - max s), s_j = scale q . k_j; no visible key: o = 0,
          log-sum-exp = -inf.
"""

import math

import numpy as np

from . import formats as F


def rms_norm(x, w, eps, residual=None):
    """(y, h) float64 of x [M, K]."""
    h = x if residual is None else x + residual
    return h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * w, h


def _sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def activation(z, act):
    """act(z) for float64 z [M, N] (swiglu: [M, N/2])."""
    if act == "relu":
        return np.where(z > 0, z, 0.0)
    if act == "gelu":
        return z * 0.5 * (1.0 + np.vectorize(math.erf)(z / math.sqrt(2.0)))
    if act == "gelu_tanh":
        return z * 0.5 * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * _sigmoid(z)
    if act == "swiglu":
        gate, up = gate_up(z)
        return gate * _sigmoid(gate) * up
    return z


def gate_up(z):
    """The gate and up halves of interleaved columns, each [M, N/2]."""
    t = z.reshape(z.shape[0], -1, 2, 16)
    return t[:, :, 0].reshape(z.shape[0], -1), t[:, :, 1].reshape(z.shape[0], -1)


def cover_exponent(a):
    """min {e : a <= 448 2^e} clamped to [-127, 127]; -127 for a = 0."""
    if a == 0:
        return -127
    m, e = math.frexp(a)  # a = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
    return max(-127, min(127, e - 9 + (1 if m > 0.875 else 0)))


def encode(v, E):
    """E4M3 codes (uint8) of float64 v times 2^-E; NaN keeps 0x7F."""
    with np.errstate(over="ignore", invalid="ignore"):
        t = np.ldexp(v, -E)
        c = F.e4m3_encode(np.clip(np.where(np.isnan(t), 0.0, t), -1e30, 1e30).astype(np.float32))
    return np.where(np.isnan(v), np.uint8(0x7F), c)


class Cache:
    """Codes and exponents in logical order: k, v uint8 [blocks, heads, block_size, D]; ke, ve int
    [blocks, heads]."""

    def __init__(self, k, v, ke, ve):
        self.k, self.v, self.ke, self.ve = k, v, ke, ve
        self.block_size = k.shape[2]

    def append(self, k, v, table, lens, cu):
        """New tokens k, v float64 [T, heads, D]."""
        bs = self.block_size
        for codes, exps, new in ((self.k, self.ke, k), (self.v, self.ve, v)):
            for b, L in enumerate(lens):
                n = cu[b + 1] - cu[b]
                p0 = max(L - n, 0)
                if n == 0 or L <= 0:
                    continue
                for j in range(p0 // bs, (L - 1) // bs + 1):
                    blk = int(table[b][j])
                    if not 0 <= blk < codes.shape[0]:
                        continue
                    lo, hi = max(p0 - j * bs, 0), min(L - j * bs, bs)
                    r0 = cu[b + 1] - L + j * bs + lo
                    for h in range(codes.shape[1]):
                        t = new[r0:r0 + hi - lo, h]
                        mag = np.abs(t[np.isfinite(t)])
                        e = cover_exponent(mag.max() if mag.size else 0.0)
                        old = int(exps[blk, h])
                        if lo > 0:
                            e = max(e, old)
                            if e != old:
                                held = codes[blk, h, :lo]
                                codes[blk, h, :lo] = _same_nan(held, encode(np.ldexp(F.e4m3_decode(held), old), e))
                        exps[blk, h] = e
                        codes[blk, h, lo:hi] = encode(t, e)

    def values(self, pages, h):
        """(k, v) float64 [tokens, D] of a list of blocks (-1: absent, NaN) and one head."""
        out = []
        for codes, exps in ((self.k, self.ke), (self.v, self.ve)):
            t = [np.ldexp(F.e4m3_decode(codes[p, h]), int(exps[p, h])) if 0 <= p < codes.shape[0]
                 else np.full(codes.shape[2:], np.nan) for p in pages]
            out.append(np.concatenate(t))
        return out


def _same_nan(held, codes):
    return np.where((held & 0x7F) == 0x7F, np.uint8(0x7F), codes)


def attention(q, cache, table, lens, cu, scale, causal=True, window=0):
    """(out, lse, mass): out float64 [T, Hq, D]; lse [T, Hq]; mass = sum_j p_j |v_j| / sum_j p_j (the
    scale of out's rounding errors) and the largest scale * sum_d |q_d k_d| of a visible key."""
    T, Hq, D = q.shape
    H = cache.k.shape[1]
    G, bs = Hq // H, cache.block_size
    out, mass = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, size = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for b, L in enumerate(lens):
        n = cu[b + 1] - cu[b]
        pages = [int(p) for p in table[b][:-(-max(L, 0) // bs)]]
        if n == 0 or not pages:
            continue
        present = np.repeat([0 <= p < cache.k.shape[0] for p in pages], bs)[:L]
        pos = np.arange(L)
        for h in range(H):
            k, v = (t[:L] for t in cache.values(pages, h))
            for i in range(n):
                p = L - n + i
                seen = present & (pos <= p if causal else True)
                if window:
                    seen &= pos > p - window
                if not seen.any():
                    continue
                ks, vs = k[seen], v[seen]
                for r in range(h * G, h * G + G):
                    x = q[cu[b] + i, r]
                    s = scale * (ks @ x)
                    m = s.max()
                    w = np.exp(s - m)
                    out[cu[b] + i, r] = w @ vs / w.sum()
                    mass[cu[b] + i, r] = w @ np.abs(vs) / w.sum()
                    lse[cu[b] + i, r] = m + math.log(w.sum())
                    size[cu[b] + i, r] = abs(scale) * (np.abs(ks) @ np.abs(x)).max()
    return out, lse, mass, size
