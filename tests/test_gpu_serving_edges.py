"""Edges of the 8-bit serving operators (GPU)."""

import math

import numpy as np
import pytest
import torch

import fp8_quantized_linear_amd as fql
from oracle import serving as S

from gpu_helpers import announce
from serving_helpers import (DEV, HALF_BF16, assert_attention, bf16, f64, i32, poison, random_cache, tables, to_device)
from test_gpu_serving import FMTS, SCALE, Decoder, check_norm, layer, operand_rows

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


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------

NORM_SHAPES = [(7, 256), (7, 4096), (1, 256), (7, 14336), (7, 20480), (7, 70016)]


def rows_at_the_ends(rng, M, K):
    """Rows: ordinary, one NaN, one infinity, around 1e30, zeros, bf16 subnormals, ordinary."""
    x = rng.standard_normal((M, K))
    if M > 1:
        x[1, 9], x[2, 5] = np.nan, np.inf
        x[3] *= 1e30
        x[4] = 0.0
        x[5] *= 1e-39
    return x


def check_rows(fmt, codes, scales, y):
    """Codes are NaN exactly where y is; the others and the scales are those of y without its NaN."""
    nan = np.isnan(y)
    assert np.array_equal((codes & 0x7F) == 0x7F, nan), (fmt, [int(r.sum()) for r in (codes & 0x7F) == 0x7F])
    check_norm(fmt, np.where(nan, np.uint8(0), codes), scales, np.where(nan, 0.0, y))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("M,K", NORM_SHAPES)
def test_norm_rows_that_are_not_finite_or_at_the_ends_of_the_range(fmt, eps, M, K):
    """A y that is not a number has a NaN code (an all-zero row under eps = 0 too: 0 / 0), and rows
    whose squares leave float32's range are normed like any other."""
    announce(f"norm ends {fmt} {M}x{K} eps={eps}")
    rng = np.random.default_rng([22, M, K])
    x, x64 = bf16(rows_at_the_ends(rng, M, K))
    w, w64 = bf16(1 + 0.2 * rng.standard_normal(K))
    w[K - 3] = float("nan")  # a column of the weight
    w64[K - 3] = np.nan
    with np.errstate(invalid="ignore", divide="ignore"):
        y, _ = S.rms_norm(x64, w64, eps)
    sc = SCALE if fmt == "fp8" else None
    codes, scales, _ = fql.rms_norm_quant(x, w, fmt, eps=eps, scale=sc)
    codes = codes.cpu().numpy()
    check_rows(fmt, codes, None if scales is None else scales.cpu().numpy(), y)
    oc, os_ = operand_rows(fql.rms_norm_operand(x, w, fmt, eps=eps, scale=sc)[0])
    assert np.array_equal(oc, codes)
    assert os_ is None or np.array_equal(os_, scales.cpu().numpy())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [3, 80])
def test_a_row_that_is_not_finite_stays_so_through_the_linear_layer(fmt, M):
    announce(f"NaN row through the layer {fmt} M={M}")
    rng = np.random.default_rng([23, M])
    h, _ = bf16(rng.standard_normal((M, 512)))
    h[1, 100] = float("inf")
    r, _ = bf16(rng.standard_normal((M, 512)))
    w, _ = bf16(np.ones(512))
    g, _ = layer(fmt, rng.standard_normal((256, 512)) * 0.05)
    x, _ = fql.rms_norm_operand(h, w, fmt, residual=r, scale=0.1 if fmt == "fp8" else None)
    y = torch.isnan(fql.linear_fused(x, g))
    assert y[1].all() and not y[0].any() and not y[2:].any()


# ---------------------------------------------------------------------------
# fused linear
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt,M", [("mxfp8", 64), ("fp8_block", 20), ("mxfp4", 100), ("fp8", 4)])
def test_the_plan_names_the_kernels_that_run(fmt, M):
    announce(f"kernels of the plan {fmt} M={M}")
    g, _ = layer(fmt, np.random.default_rng(27).standard_normal((256, 512)))
    x, _ = bf16(np.ones((M, 512)))
    fql.linear_fused(x, g)
    torch.cuda.synchronize()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as p:
        fql.linear_fused(x, g)
        torch.cuda.synchronize()
    ran = [e.name for e in p.events() if "fql::" in e.name]
    named = [part.split("<")[0] for part in fql.linear_fused_plan(fmt, M, 256, 512).split(" + ")]
    assert len(ran) == len(named), (ran, named)
    for kernel, name in zip(ran, named):
        assert f":{name}<" in kernel, (kernel, name)


@pytest.mark.parametrize("M", [2, 80])
def test_gelu_tail(M):
    """The negative tail keeps its relative precision down to bf16's smallest normal values: its
    float32 evaluation is off by at most 1e-5 (a^2 / 2 <= 84 rounded, times 2^-23), bf16 by 2^-8."""
    announce(f"GELU tail M={M}")
    K, N = 128, 256
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    g, _ = layer("mxfp8", np.zeros((N, K)))
    b, z = bf16(-np.linspace(0.01, 12.9, N))
    y = f64(fql.linear_fused(x, g, activation="gelu", bias=b))
    want = np.array([[t / 2 * math.erfc(-t / math.sqrt(2)) for t in z]])  # 1 + erf cancels
    assert (np.abs(y - want) <= (HALF_BF16 + 1e-5) * np.abs(want)).all()


@pytest.mark.parametrize("M", [1, 5, 40])
def test_linear_reads_and_writes_columns_of_one_buffer(M):
    """x and out in the same rows of one buffer, side by side in either order, do not overlap."""
    announce(f"columns of one buffer M={M}")
    rng = np.random.default_rng([28, M])
    g, _ = layer("mxfp8", rng.standard_normal((64, 128)) * 0.1)
    x, _ = bf16(rng.standard_normal((M, 128)))
    want = fql.linear_fused(x, g)
    for x0, y0 in ((0, 128), (64, 0)):
        both = torch.full((M, 192), 3.0, dtype=torch.bfloat16, device=DEV)
        both[:, x0:x0 + 128] = x
        out = fql.linear_fused(both[:, x0:x0 + 128], g, out=both[:, y0:y0 + 64])
        assert torch.equal(out, want) and torch.equal(both[:, x0:x0 + 128], x)
    with pytest.raises(fql.FQLError, match="overlap"):
        fql.linear_fused(both[:, 64:], g, out=both[:, 32:96])


# ---------------------------------------------------------------------------
# no tokens
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
def test_calls_on_no_rows_give_empty_outputs(fmt):
    """A step in which no sequence has a token: a layer goes through it as the cache's calls do."""
    announce(f"no rows {fmt}")
    net = Decoder(fmt)
    h, _ = bf16(np.zeros((3, 512)))
    cache = fql.KVCache8.empty(2, 2, 16, 64, DEV)
    y = net(h[:0], cache, i32([[0, 1]]), i32([5]), i32([0, 0]), 1)
    assert y.shape == (0, 512) and y.dtype is torch.bfloat16 and y.device == h.device
    sc = 0.1 if fmt == "fp8" else None
    codes, scales, r = fql.rms_norm_quant(h[:0], net.w1, fmt, residual=h[:0], scale=sc)
    n = {"fp8": None, "fp8_block": 4, "mxfp8": 16}[fmt]
    assert codes.shape == (0, 512) and r.shape == (0, 512) and (scales is None if n is None else scales.shape == (0, n))
    assert fql.linear_fused(h.view(1, 3, 512)[:, :0], net.qkv).shape == (1, 0, 768)
    assert fql.linear_fused(fql.quant_operand(h[:0], fmt, scale=sc), net.gu, activation="swiglu").shape == (0, 1024)
    out = h[:0]
    assert fql.linear_fused(h[:0], net.o, residual=out, out=out) is out
    with pytest.raises(fql.FQLError, match="multiple"):  # what does not fit is refused all the same
        fql.rms_norm_quant(h[:0, :500], net.w1[:500], fmt, scale=sc)
    with pytest.raises(fql.FQLError, match="has K="):
        fql.linear_fused(h[:0, :256], net.qkv)


# ---------------------------------------------------------------------------
# workspaces under graph capture
# ---------------------------------------------------------------------------

def split_call(rng, lens, blocks, max_len):
    """Arguments of an attention call whose keys are split into ranges."""
    table = tables(rng, len(lens), max_len // 64, blocks, lens, 64, -1)
    q, _ = bf16(rng.standard_normal((len(lens), 8, 128)))
    assert "splits=1" not in fql.attention_kv8_plan(len(lens), 8, 2, 128, 1, max_len).split()
    return (q, to_device(random_cache(rng, blocks, 2, 64, 128)), i32(table), i32(lens), i32(range(len(lens) + 1)), 1)


def captured(s, args, warm):
    with torch.cuda.stream(s):
        if warm:
            fql.attention_kv8(*args)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = fql.attention_kv8(*args)
    return g, out


@pytest.mark.parametrize("warm", [False, True])
def test_a_graph_does_not_use_its_streams_eager_workspace(warm):
    """A replay on another stream beside eager calls on the capture's stream: the two must not share
    arrival counters. A call in flight is stood in for by counters that are not zero."""
    announce(f"workspace of a graph warm={warm}")
    rng = np.random.default_rng([24, warm])
    args = split_call(rng, [4000, 900], 90, 63 * 64)
    want = fql.attention_kv8(*args)
    torch.cuda.synchronize()
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    key = ("cuda", 0, s.cuda_stream)
    fql._workspaces.pop(key, None)
    g, got = captured(s, args, warm)
    with torch.cuda.stream(s):
        fql.attention_kv8(*args)
        s.synchronize()
    eager = fql._workspaces[key]
    for _ in range(4):
        got.zero_()
        eager[:65536].fill_(1)
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            g.replay()
        other.synchronize()
        assert (eager[:65536] == 1).all()
        eager[:65536].zero_()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        with torch.cuda.stream(s):
            assert torch.equal(fql.attention_kv8(*args), want)
        torch.cuda.synchronize()


def test_graphs_captured_on_one_stream_do_not_share_counters():
    announce("two graphs")
    rng = np.random.default_rng(25)
    cases = [split_call(rng, [4000, 900], 90, 63 * 64), split_call(rng, [3000, 2900, 10], 100, 63 * 64)]
    want = [fql.attention_kv8(*a) for a in cases]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graphs = [captured(s, a, True) for a in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for t, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(t):
                g.replay()
        torch.cuda.synchronize()
        for (_, got), w in zip(graphs, want):
            assert torch.equal(got, w)
            got.zero_()
        torch.cuda.synchronize()


def test_a_capture_clears_one_workspace_and_lets_go_of_it():
    """A whole layer captured on a stream without a workspace: one buffer, dropped when the stream is
    used again; replays give the eager results."""
    announce("one workspace a capture")
    net = Decoder("mxfp8")
    rng = np.random.default_rng(26)
    table, lens, cu = i32([[0, 1, 2, 3], [4, 5, 6, 7]]), i32([20, 30]), i32([0, 1, 2])
    start = random_cache(rng, 8, 2, 16, 64)
    caches = [to_device(start) for _ in range(2)]
    h, _ = bf16(rng.standard_normal((2, 512)))
    want = net(h, caches[0], table, lens, cu, 1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    key = ("cuda", 0, s.cuda_stream)
    for held in (fql._workspaces, fql._captured):
        held.pop(key, None)
    g = torch.cuda.CUDAGraph()
    seen = set()
    with torch.cuda.graph(g, stream=s):
        x, _ = fql.rms_norm_operand(h, net.w1, "mxfp8")
        for _ in range(2):
            y = fql.linear_fused(x, net.qkv)
            seen.add(fql._captured[key][1].data_ptr())
        got = net(h, caches[1], table, lens, cu, 1)
        fql.linear_mxfp8(h, net.qkv)
        seen.add(fql._captured[key][1].data_ptr())
    assert len(seen) == 1 and key not in fql._workspaces and y.shape == (2, 768)
    for _ in range(3):  # the cache is written with the same tokens each time
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    with torch.cuda.stream(s):
        fql.linear_fused(h, net.qkv)
    torch.cuda.synchronize()
    assert key not in fql._captured and key in fql._workspaces
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
