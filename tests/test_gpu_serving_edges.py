"""Edges of the 8-bit serving operators (GPU)."""

import numpy as np
import pytest

import fp8_quantized_linear_amd as fql
from oracle import serving as S

from gpu_helpers import announce
from serving_helpers import (HALF_BF16, bf16, f64, i32, poison, random_cache, tables, to_device)

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
