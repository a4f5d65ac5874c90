"""Inputs, conversions and error bounds shared by the serving operators' tests (not a test module)."""

import numpy as np
import torch

from oracle import formats as F
from oracle import serving as S

DEV = "cuda:0"
HALF_BF16 = 2.0 ** -8   # bf16 rounding, relative: finfo(bfloat16).eps / 2


def bf16(a, dev=DEV):
    """float array -> bf16 tensor and its exact float64 values."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t.to(dev), t.to(torch.float64).numpy()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def strided(values, ld, off=0, dev=DEV):
    """A bf16 [M, K] view with row stride ld starting `off` elements into its storage."""
    M, K = values.shape
    flat = torch.full((off + M * ld + 8,), 3.0, dtype=torch.bfloat16)
    v = torch.as_strided(flat, (M, K), (ld, 1), off)
    v.copy_(torch.from_numpy(np.ascontiguousarray(values, dtype=np.float32)).to(torch.bfloat16))
    exact = v.to(torch.float64).numpy()
    return torch.as_strided(flat.to(dev), (M, K), (ld, 1), off), exact


def assert_e4m3_of(codes, v, rel):
    """Every code is the E4M3 rounding (nearest, saturating) of a value within rel of v: off by at most
    half a step of v's binade plus rel * |v|."""
    q = F.e4m3_decode(codes)
    t = np.clip(v, -448.0, 448.0)
    top = np.maximum(np.abs(t) * (1 + rel), 2.0 ** -6)
    half = np.exp2(np.floor(np.log2(top)) - 4)
    bad = ~(np.abs(q - t) <= half * (1 + 1e-12) + rel * np.abs(t))
    assert not bad.any(), (int(bad.sum()), q[bad][:4], v[bad][:4])


def tables(rng, B, cols, blocks, lens, bs, junk):
    """A block table whose used entries are distinct random blocks; unused entries hold `junk`."""
    order = rng.permutation(blocks)
    t = np.full((B, cols), junk, dtype=np.int32)
    at = 0
    for b, L in enumerate(lens):
        n = -(-L // bs)
        t[b, :n] = order[at:at + n]
        at += n
    assert at <= blocks
    return t


def random_cache(rng, blocks, H, bs, D, spread=3):
    """Oracle cache of N(0, 1) keys and values with exponents spread by a few powers of two."""
    out = []
    for _ in range(2):
        v = rng.standard_normal((blocks, H, bs, D))
        e = rng.integers(-7 - spread, -6 + spread, (blocks, H))
        codes = F.e4m3_encode(np.ldexp(v, -e[:, :, None, None]).astype(np.float32))
        # blocks of a large exponent hold small codes and the other way round
        out.append((codes, e))
    return S.Cache(out[0][0], out[1][0], out[0][1], out[1][1])


def poison(cache, table, lens):
    """NaN codes in every place no sequence's tokens occupy."""
    used = np.zeros((cache.k.shape[0], cache.block_size), dtype=bool)
    for b, L in enumerate(lens):
        for j in range(-(-L // cache.block_size)):
            p = int(table[b][j])
            if 0 <= p < used.shape[0]:
                used[p, :min(cache.block_size, L - j * cache.block_size)] = True
    mask = np.broadcast_to(~used[:, None, :, None], cache.k.shape)
    cache.k[mask] = 0x7F
    cache.v[mask] = 0xFF
    for e in (cache.ke, cache.ve):
        e[~used.any(axis=1)] = 128  # byte 255


def to_device(cache):
    """Oracle cache -> fql.KVCache8."""
    import fp8_quantized_linear_amd as fql

    nb, H, bs, D = cache.k.shape
    v = cache.v.reshape(nb, H, bs // 16, 16, D).swapaxes(3, 4)
    dev = [torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
           for a in (cache.k, v, (cache.ke + 127).astype(np.uint8), (cache.ve + 127).astype(np.uint8))]
    return fql.KVCache8(*dev)


def from_device(c):
    """fql.KVCache8 -> oracle arrays (k, v, ke, ve)."""
    nb, H, bs, D = c.num_blocks, c.kv_heads, c.block_size, c.head_dim
    k, v = c.k.cpu().numpy(), c.v.cpu().numpy()
    v = v.swapaxes(3, 4).reshape(nb, H, bs, D)
    return k, v, c.k_scale.cpu().numpy().astype(int) - 127, c.v_scale.cpu().numpy().astype(int) - 127


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def assert_attention(out, lse, ref, what):
    """Kernel output against the oracle's. Errors counted: the output's bf16 rounding (half a step,
    2^-8 |o|), the weights' (2^-8 of sum p |v|), and the float32 scores: a dot product of D <= 256
    terms in float32 is off by less than 2^-16 of sum |q k|, which moves every weight by e^that on
    both sides of the quotient."""
    o, l, mass, size = ref
    tol = HALF_BF16 * np.abs(o) + (HALF_BF16 + 2.0 ** -14 + 4 * 2.0 ** -16 * size[..., None]) * mass
    d = np.abs(f64(out) - o)
    bad = ~(d <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.size, np.argwhere(bad)[:4].tolist(), float(np.nanmax(d)))
    if lse is not None:
        got = f64(lse)
        empty = np.isneginf(l)
        assert np.array_equal(np.isneginf(got), empty), what
        tl = 2.0 ** -16 * size + 2.0 ** -18 * (1 + np.abs(np.where(empty, 0, l)))
        assert (np.abs(got - l)[~empty] <= tl[~empty]).all(), what
