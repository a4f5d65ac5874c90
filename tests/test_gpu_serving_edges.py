"""Edges of the 8-bit serving operators (GPU)."""

import numpy as np
import pytest

import fp8_quantized_linear_amd as fql
from oracle import serving as S

from gpu_helpers import announce
from serving_helpers import (HALF_BF16, assert_attention, bf16, f64, i32, poison, random_cache, tables, to_device)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 40, 90])
@pytest.mark.parametrize("absent", [4, 5, 6, 7])
def test_attention_nan_beside_an_absent_block(D, new, absent):
    """Blocks of 16 tokens, one of them absent, NaN values in the three others of the same 64 tokens,
    which every row sees: the NaN reach every row."""
    rng = np.random.default_rng([20, D, new, absent])
    bs, H, Hq, L = 16, 2, 4, 250
    table = tables(rng, 1, 17, 18, [L], bs, -1)
    cache = random_cache(rng, 18, H, bs, D)
    poison(cache, table, [L])
    for j in {4, 5, 6, 7} - {absent}:
        cache.v[table[0, j], 0, 3 * j % bs, 7 * j] = 0x7F
    table[0, absent] = -1
    q, q64 = bf16(rng.standard_normal((new, Hq, D)))
    announce(f"attention NaN beside an absent block D={D} new={new} absent={absent} "
             + fql.attention_kv8_plan(1, Hq, H, D, new, 17 * bs))
    out, _ = fql.attention_kv8(q, to_device(cache), i32(table), i32([L]), i32([0, new]), new, return_lse=True)
    o, _, mass, size = S.attention(q64, cache, table, [L], [0, new], D ** -0.5)
    got = f64(out)
    assert np.isnan(o).sum() == 3 * new * (Hq // H)
    assert np.array_equal(np.isnan(got), np.isnan(o))
    fin = ~np.isnan(o)
    tol = HALF_BF16 * np.abs(o) + (HALF_BF16 + 2.0 ** -14 + 4 * 2.0 ** -16 * size[..., None]) * mass
    assert (np.abs(got - o)[fin] <= tol[fin]).all()


@pytest.mark.parametrize("E", [118, 104, -104, -120])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_value_exponents_at_the_ends(E, new):
    """Values of 2^E, and scores that lie 7 (in powers of two) above those of the first 64 tokens: a
    running maximum that lags behind must not take the sums out of float32."""
    rng = np.random.default_rng([21, new])
    bs, H, Hq, D, L = 32, 1, 2, 128, 300
    table = tables(rng, 1, 11, 12, [L], bs, -1)
    cache = random_cache(rng, 12, H, bs, D)
    cache.ve[:] = E
    cache.ke[:] = 0
    cache.v[:] = np.where(rng.random(cache.v.shape) < 0.5, 0x38, 0xBA)  # 1, -1.25
    cache.k[:] = 0
    for t in range(64, L - new):
        if rng.random() < 0.5:
            cache.k[table[0, t // bs], 0, t % bs] = 0x2E  # 0.4375: 128 of them times 128^-1/2 are 7.1 log 2
    poison(cache, table, [L])
    q, q64 = bf16(np.ones((new, Hq, D)) + rng.integers(-2, 3, (new, Hq, 1)) / 64)
    announce(f"attention values of 2^{E} new={new} " + fql.attention_kv8_plan(1, Hq, H, D, new, 11 * bs))
    out, lse = fql.attention_kv8(q, to_device(cache), i32(table), i32([L]), i32([0, new]), new, return_lse=True)
    ref = S.attention(q64, cache, table, [L], [0, new], D ** -0.5)
    assert np.isfinite(f64(out)).all()
    assert_attention(out, lse, ref, f"2^{E}")
