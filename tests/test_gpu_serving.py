"""The 8-bit serving operators against their float64 definitions (GPU)."""

import numpy as np
import pytest
import torch

import fp8_quantized_linear_amd as fql
from oracle import formats as F
from oracle import fp8 as P
from oracle import mx as X
from oracle import serving as S

from gpu_helpers import announce
from serving_helpers import (DEV, HALF_BF16, assert_attention, assert_e4m3_of, bf16, f64, from_device, i32, poison,
                             random_cache, strided, tables, to_device)

pytestmark = pytest.mark.gpu

FMTS = ("fp8", "fp8_block", "mxfp8")
SCALE = 0.03


def hidden(rng, M, K):
    x = rng.standard_normal((M, K))
    x[:, rng.random(K) < 0.02] *= 20
    return x


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------

# The kernel's y against the exact one. A thread adds at most 72 squares in order and the partial
# sums go through at most 6 + 16 more additions: the sum of squares is off by less than 96 * 2^-24,
# its root by half of that; the sum h, the mean, the root, the reciprocal and the products add less
# than 8 * 2^-24.
Y_REL = 64 * 2.0 ** -24


def check_norm(fmt, codes, scales, y):
    """Codes and scales of a float32 y within Y_REL of float64 y (and one float32 rounding of v * r)."""
    rel = Y_REL + 4 * 2.0 ** -24
    if fmt == "fp8":
        assert_e4m3_of(codes, y / float(np.float32(SCALE)), rel)
        return
    n = 128 if fmt == "fp8_block" else 32
    t = y.reshape(y.shape[0], -1, n)
    a = np.abs(t).max(axis=2)
    if fmt == "fp8_block":
        s = scales.astype(np.float64)
        assert (np.abs(s - a / 448) <= rel * a / 448).all()
    else:
        e = scales.astype(np.int64) - 127
        lo = np.maximum(np.floor(np.log2(np.maximum(a * (1 - rel), 1e-300))) - 8, -127)
        hi = np.maximum(np.floor(np.log2(np.maximum(a * (1 + rel), 1e-300))) - 8, -127)
        assert ((e >= lo) & (e <= hi)).all()
        s = np.ldexp(1.0, e)
    safe = np.where(s > 0, s, 1.0)
    v = np.where(s[..., None] > 0, t / safe[..., None], 0.0)
    assert_e4m3_of(codes.reshape(t.shape), v, 2 * rel)


def operand_rows(q):
    """A QuantizedActivation's codes [M, K] and its scales as the plain quantizer lays them out."""
    M, K, KC = q.M, q.K, -(-q.K // 128)
    Mp = -(-M // 256) * 256
    raw = q.data.cpu().numpy()
    half = 1 if q.fmt == "mxfp4" else 2
    c = raw[:Mp * KC * 64 * half].reshape(Mp // 16, KC, half, 4, 16, 16)  # tile, chunk, half, group, row, byte
    codes = c.transpose(0, 4, 1, 2, 3, 5).reshape(Mp, KC * 64 * half)
    pad = codes[:M, K * half // 2:]
    assert not pad.any()  # columns past K are zero codes
    rest = raw[Mp * KC * 64 * half:]
    scales = None
    if q.fmt in ("mxfp8", "mxfp4"):
        s = rest[:Mp * KC * 4].reshape(Mp // 64, KC, 4, 16, 4)  # quad, chunk, block, row, tile
        scales = s.transpose(0, 4, 3, 1, 2).reshape(Mp, KC * 4)[:M, :K // 32]
    elif q.fmt == "fp8_block":
        s = rest[:Mp * KC * 4].view(np.float32).reshape(Mp // 64, KC, 64)
        scales = s.transpose(0, 2, 1).reshape(Mp, KC)[:M]
    return codes[:M, :K * half // 2], scales


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K", [(1, 4096), (1, 128), (3, 256), (5, 1024), (17, 4096), (130, 5120), (2, 14336),
                                 (300, 2304), (2, 70016)])
def test_norm(fmt, M, K):
    announce(f"norm {fmt} {M}x{K}")
    rng = np.random.default_rng([M, K])
    x, x64 = bf16(hidden(rng, M, K))
    r, r64 = bf16(hidden(rng, M, K) * 3)
    w, w64 = bf16(1 + 0.2 * rng.standard_normal(K))
    sc = SCALE if fmt == "fp8" else None
    for residual, r_ in ((None, None), (r, r64)):
        y, h = S.rms_norm(x64, w64, 1e-5, r_)
        codes, scales, hout = fql.rms_norm_quant(x, w, fmt, eps=1e-5, residual=residual, scale=sc)
        check_norm(fmt, codes.cpu().numpy(), None if scales is None else scales.cpu().numpy(), y)
        if residual is None:
            assert hout is None
        else:
            assert (np.abs(f64(hout) - h) <= (HALF_BF16 + 2.0 ** -23) * np.abs(h)).all()
        q, h2 = fql.rms_norm_operand(x, w, fmt, eps=1e-5, residual=residual, scale=sc)
        oc, os_ = operand_rows(q)
        assert np.array_equal(oc, codes.cpu().numpy())
        assert os_ is None or np.array_equal(os_, scales.cpu().numpy())
        assert h2 is None or torch.equal(h2, hout)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp8"])
@pytest.mark.parametrize("M,K", [(700, 4096), (3000, 512), (40, 70016)])
def test_norm_codes_are_those_of_the_exact_values(fmt, M, K):
    """One rounding: every code is that of the float64 y (whose own error, some 2^-50, no value here
    is near enough to a tie to show)."""
    announce(f"norm exact codes {fmt} {M}x{K}")
    rng = np.random.default_rng([7, M, K])
    x, x64 = bf16(rng.standard_normal((M, K)))
    w, w64 = bf16(1 + 0.2 * rng.standard_normal(K))
    y, _ = S.rms_norm(x64, w64, float(np.float32(1e-5)), None)
    codes, scales, _ = fql.rms_norm_quant(x, w, fmt, eps=float(np.float32(1e-5)), scale=0.0625 if fmt == "fp8" else None)
    s = 0.0625 if fmt == "fp8" else np.repeat(np.ldexp(1.0, scales.cpu().numpy().astype(np.int64) - 127), 32, axis=1)
    got = codes.cpu().view(torch.float8_e4m3fn).double().numpy()
    v = np.clip(y / s, -448, 448)
    step = np.ldexp(1.0, np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -40))), -6).astype(np.int64) - 3)
    assert np.array_equal(got, np.rint(v / step) * step)


@pytest.mark.parametrize("fmt,K", [("fp8", 4096 + 32), ("mxfp8", 96), ("mxfp8", 4096 + 32), ("fp8", 32)])
def test_norm_columns_that_end_inside_a_chunk(fmt, K):
    announce(f"norm tail {fmt} K={K}")
    rng = np.random.default_rng(K)
    x, x64 = bf16(hidden(rng, 7, K))
    w, w64 = bf16(1 + 0.2 * rng.standard_normal(K))
    sc = SCALE if fmt == "fp8" else None
    codes, scales, _ = fql.rms_norm_quant(x, w, fmt, scale=sc)
    check_norm(fmt, codes.cpu().numpy(), None if scales is None else scales.cpu().numpy(),
               S.rms_norm(x64, w64, 1e-6)[0])
    oc, os_ = operand_rows(fql.rms_norm_operand(x, w, fmt, scale=sc)[0])
    assert np.array_equal(oc, codes.cpu().numpy())
    assert os_ is None or np.array_equal(os_, scales.cpu().numpy())


@pytest.mark.parametrize("ld,off", [(1024, 0), (1032, 8), (1025, 1)])
def test_norm_strides_and_in_place(ld, off):
    announce(f"norm strided ld={ld} off={off}")
    rng = np.random.default_rng(ld)
    x, x64 = strided(hidden(rng, 9, 1024), ld, off)
    r, r64 = strided(hidden(rng, 9, 1024), ld, off)
    w, w64 = bf16(1 + 0.2 * rng.standard_normal(1024))
    y, h = S.rms_norm(x64, w64, 1e-6, r64)
    want, ws, hw = fql.rms_norm_quant(x, w, "fp8_block", residual=r)
    check_norm("fp8_block", want.cpu().numpy(), ws.cpu().numpy(), y)
    for target in (r, x):  # the sum written over either input
        keep = target.clone()
        codes, scales, got = fql.rms_norm_quant(x, w, "fp8_block", residual=r, residual_out=target)
        assert got is target and torch.equal(target, hw) and torch.equal(codes, want) and torch.equal(scales, ws)
        target.copy_(keep)


def test_norm_zero_rows_and_extremes():
    announce("norm zeros")
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device=DEV)
    x[1, 3] = 1e30   # the sum of squares overflows float32: the row is 0 (1 / inf)
    x[2] = 1e-30     # vanishes below eps
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    for fmt in FMTS:
        codes, scales, _ = fql.rms_norm_quant(x, w, fmt, scale=SCALE if fmt == "fp8" else None)
        assert not codes[0].any() and not codes[1, 4:].any() and not codes[3].any()
        if fmt == "mxfp8":
            assert not scales[0].any()
        elif fmt == "fp8_block":
            assert not scales[0].any()
    # eps = 0 and a zero row: 0 * inf
    codes, scales, _ = fql.rms_norm_quant(x[3:], w, "mxfp8", eps=1e-6)
    assert not codes.any()


# ---------------------------------------------------------------------------
# fused linear
# ---------------------------------------------------------------------------

def layer(fmt, W, x_scale=0.1):
    """(GPU weight, exact float64 weight)."""
    wd = torch.from_numpy(W.astype(np.float32)).to(DEV)
    if fmt == "fp8":
        g = fql.FP8Weight.from_float(wd, input_scale=x_scale)
        return g, F.e4m3_decode(P.quant_fp8_tensor(W, g.weight_scale)) * g.weight_scale
    if fmt == "mxfp4":
        return fql.MXFP4Weight.from_float(wd), X.dequant_mxfp4(*X.quant_mxfp4(W))
    if fmt == "mxfp8":
        return fql.MXFP8Weight.from_float(wd), P.dequant_mxfp8(*P.quant_mxfp8(W))
    return fql.FP8BlockWeight.from_float(wd), P.dequant_fp8_block_weight(*P.quant_fp8_block_weight(W))


def activation_hat(fmt, x64, x_scale=0.1):
    x32 = x64.astype(np.float32)
    if fmt == "fp8":
        s = float(np.float32(x_scale))
        return F.e4m3_decode(P.quant_fp8_tensor(x32, np.float32(x_scale))) * s
    if fmt == "mxfp4":
        return X.dequant_mxfp4(*X.quant_mxfp4(x32))
    if fmt == "mxfp8":
        return P.dequant_mxfp8(*P.quant_mxfp8(x32))
    return P.dequant_fp8_block_act(*P.quant_fp8_block_act(x32))


def check_linear(y, xh, wh, bias, act, residual, what):
    """Errors counted: the products' sum (the FP8 matrix instruction keeps about 2^-13 of the sum of
    magnitudes; 2^-12 is allowed), the activation's slope (at most 1.13; swiglu by the product rule)
    and its float32 evaluation (2^-18), one bf16 rounding."""
    z = xh @ wh.T + (0 if bias is None else bias)
    e = 2.0 ** -12 * (np.abs(xh) @ np.abs(wh).T) + 2.0 ** -22 * np.abs(z)
    v = S.activation(z, act)
    if act == "swiglu":
        (g, u), (eg, eu) = S.gate_up(z), S.gate_up(e)
        tol = 1.13 * eg * (np.abs(u) + eu) + np.abs(g) * eu
    else:
        tol = 1.13 * e
    tol = tol + 2.0 ** -18 * np.abs(v) + 1e-30
    ref = v + (0 if residual is None else residual)
    tol = tol * (1 + HALF_BF16) + (HALF_BF16 + 2.0 ** -20) * np.abs(ref)
    d = np.abs(f64(y) - ref)
    bad = ~(d <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.size, np.argwhere(bad)[:4].tolist())


CASES = [(M, N, K) for M in (1, 9, 16, 17, 32) for N, K in ((512, 1024),)] + [
    (33, 384, 512), (100, 256, 2048), (129, 640, 384), (300, 256, 512), (600, 512, 256)]


@pytest.mark.parametrize("fmt", ("mxfp4",) + FMTS)
@pytest.mark.parametrize("M,N,K", CASES)
def test_linear_epilogues(fmt, M, N, K):
    rng = np.random.default_rng([M, N, K])
    x, x64 = bf16(rng.standard_normal((M, K)) * 2)
    g, wh = layer(fmt, rng.standard_normal((N, K)) * 0.05)
    b, b64 = bf16(rng.standard_normal(N))
    xh = activation_hat(fmt, x64)
    op = fql.quant_operand(x, fmt, scale=0.1)
    acts = ("none", "relu", "gelu", "gelu_tanh", "silu", "swiglu")
    for i, act in enumerate(acts):
        announce(f"linear {fmt} {M}x{N}x{K} {act}")
        res = i % 2 == 0
        No = N // 2 if act == "swiglu" else N
        r, r64 = bf16(rng.standard_normal((M, No)) * 4)
        bias, bias64 = (b, b64) if i % 3 else (None, None)
        args = dict(activation=act, bias=bias, residual=r if res else None)
        y = fql.linear_fused(x, g, **args)
        assert y.shape == (M, No)
        check_linear(y, xh, wh, bias64, act, r64 if res else None, (fmt, M, N, K, act))
        # the operand form holds the same codes: same products, same sums
        assert torch.equal(fql.linear_fused(op, g, **args), y)


@pytest.mark.parametrize("fmt,N", [("fp8", 200), ("mxfp8", 72), ("mxfp8", 224)])
@pytest.mark.parametrize("M", [1, 20, 70, 300])
def test_linear_ragged_columns_and_strides(fmt, N, M):
    announce(f"linear ragged {fmt} M={M} N={N}")
    rng = np.random.default_rng([M, N])
    K = 256
    x, x64 = strided(rng.standard_normal((M, K)), K + 3, 1)
    g, wh = layer(fmt, rng.standard_normal((N, K)) * 0.1)
    xh = activation_hat(fmt, x64)
    for act in ("silu", "swiglu"):
        if act == "swiglu" and N % 32:
            with pytest.raises(fql.FQLError):
                fql.linear_fused(x, g, activation=act)
            continue
        No = N // 2 if act == "swiglu" else N
        r, r64 = strided(rng.standard_normal((M, No)), No + 5, 3)
        flat = torch.full((2 + M * (No + 9) + 8,), -7.0, dtype=torch.bfloat16, device=DEV)
        out = torch.as_strided(flat, (M, No), (No + 9, 1), 2)
        fql.linear_fused(x, g, activation=act, residual=r, out=out)
        check_linear(out, xh, wh, None, act, r64, (fmt, M, N, act))
        gaps = flat.clone()
        torch.as_strided(gaps, (M, No), (No + 9, 1), 2).fill_(-7.0)
        assert (gaps == -7.0).all()  # nothing outside the view


@pytest.mark.parametrize("fmt", ("mxfp4",) + FMTS)
@pytest.mark.parametrize("M", [4, 64, 520])
def test_linear_residual_in_place(fmt, M):
    announce(f"linear in place {fmt} M={M}")
    rng = np.random.default_rng(M)
    x, _ = bf16(rng.standard_normal((M, 512)))
    g, _ = layer(fmt, rng.standard_normal((256, 512)) * 0.1)
    r, _ = bf16(rng.standard_normal((M, 256)))
    want = fql.linear_fused(x, g, activation="gelu_tanh", residual=r)
    got = r.clone()
    assert fql.linear_fused(x, g, activation="gelu_tanh", residual=got, out=got) is got
    assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", ("mxfp4",) + FMTS)
def test_linear_without_epilogue(fmt):
    announce(f"linear plain {fmt}")
    rng = np.random.default_rng(5)
    for M in (3, 40, 200):
        x, x64 = bf16(rng.standard_normal((M, 512)))
        g, wh = layer(fmt, rng.standard_normal((384, 512)) * 0.1)
        b, b64 = bf16(rng.standard_normal(384))
        y = fql.linear_fused(x, g, bias=b)
        check_linear(y, activation_hat(fmt, x64), wh, b64, "none", None, fmt)
        if M <= 32:  # one plan, one order of the sum: the plain layer bit for bit
            plain = {"mxfp4": fql.linear_mxfp4, "mxfp8": fql.linear_mxfp8, "fp8": fql.linear_fp8,
                     "fp8_block": fql.linear_fp8_block}[fmt]
            assert torch.equal(y, plain(x, g, bias=b))


# (M, N, K) whose plans are, in turn: 16 x 128, 64 x 64, 128 x 64, 128 x 128 and 256 x 128 tiles whole, and
# 64 x 64, 128 x 64 and 128 x 128 tiles with K in ranges (checked on rows and columns of a sample)
PLANNED = [(40, 1000, 1024, "MTW=1,NTW=2"), (250, 4096, 1024, "MTW=2,NTW=2"), (500, 4000, 512, "WM=4,WN=2,MTW=2"),
           (1000, 4096, 512, "WM=2,WN=4,MTW=4"), (1900, 4096, 512, "WM=4,WN=2,MTW=4"), (60, 4096, 14336, "splits=4"),
           (120, 4096, 14336, "splits"), (250, 5120, 12800, "splits")]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K,kind", PLANNED)
def test_linear_planned_tiles(fmt, M, N, K, kind):
    N = N // 128 * 128 if fmt == "fp8_block" else N
    announce(f"linear {fmt} {M}x{N}x{K} {fql.linear_fused_plan(fmt, M, N, K)}")
    rng = np.random.default_rng([M, N])
    x, x64 = bf16(rng.standard_normal((M, K), dtype=np.float32))
    W = rng.standard_normal((N, K), dtype=np.float32) * np.float32(0.05)
    wd = torch.from_numpy(W).to(DEV)
    g = {"fp8": lambda: fql.FP8Weight.from_float(wd, input_scale=0.1), "mxfp8": lambda: fql.MXFP8Weight.from_float(wd),
         "fp8_block": lambda: fql.FP8BlockWeight.from_float(wd)}[fmt]()
    r, r64 = bf16(rng.standard_normal((M, N), dtype=np.float32))
    y = fql.linear_fused(x, g, activation="silu", residual=r)
    rows = np.unique(np.concatenate([[0, 15, 16, 31, M // 2, M - 17, M - 1], rng.integers(0, M, 16)]))
    cols = np.arange(N) if N < 256 else np.unique(np.concatenate([np.arange(128), np.arange(N - 128, N)]))
    if fmt == "fp8":
        wh = F.e4m3_decode(P.quant_fp8_tensor(W[cols], g.weight_scale)) * g.weight_scale
    elif fmt == "mxfp8":
        wh = P.dequant_mxfp8(*P.quant_mxfp8(W[cols]))
    else:
        wh = P.dequant_fp8_block_weight(*P.quant_fp8_block_weight(W[cols]))
    check_linear(y[rows][:, cols], activation_hat(fmt, x64[rows]), wh, None, "silu", r64[np.ix_(rows, cols)],
                 (fmt, M, N, K))
    torch.cuda.synchronize()
    assert torch.equal(fql.linear_fused(x, g, activation="silu", residual=r), y)  # and again: counters are back at zero


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu", "swiglu"])
@pytest.mark.parametrize("M", [2, 80])
def test_activation_limits(act, M):
    """Large and infinite pre-activations (through the bias) reach the activation's limits."""
    announce(f"limits {act} M={M}")
    K, N = 128, 128
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    g, _ = layer("mxfp8", np.zeros((N, K)))
    z = np.zeros(N)
    z[:10] = [50, -50, 300, -300, 1e30, -1e30, np.inf, -np.inf, np.nan, -1e-3]
    if act == "swiglu":
        z[16:32] = 1.0
    b, z64 = bf16(z)
    y = f64(fql.linear_fused(x, g, activation=act, bias=b))[:, :10]
    with np.errstate(all="ignore"):
        want = S.activation(z64[None, :], act)[0, :10]
    want[7] = 0.0
    assert np.isnan(y[:, 8]).all()
    keep = [0, 1, 2, 3, 4, 5, 6, 7, 9]
    fin = [i for i in keep if i != 6]
    assert np.isposinf(y[:, 6]).all()
    tol = (HALF_BF16 + 2.0 ** -18) * np.abs(want[fin]) + 2.0 ** -20
    assert (np.abs(y[:, fin] - want[fin]) <= tol).all(), (y[0], want)


def test_interleave_gate_up_gives_silu_gate_times_up():
    announce("interleave")
    rng = np.random.default_rng(8)
    gate, up = rng.standard_normal((64, 256)) * 0.1, rng.standard_normal((64, 256)) * 0.1
    both = fql.interleave_gate_up(torch.from_numpy(gate), torch.from_numpy(up)).numpy()
    g, wh = layer("mxfp8", both)
    x, x64 = bf16(rng.standard_normal((40, 256)))
    y = fql.linear_fused(x, g, activation="swiglu")
    check_linear(y, activation_hat("mxfp8", x64), wh, None, "swiglu", None, "interleave")
    wg, wu = (P.dequant_mxfp8(*P.quant_mxfp8(t)) for t in (gate, up))
    xh = activation_hat("mxfp8", x64)
    ref = S.activation(xh @ wg.T, "silu") * (xh @ wu.T)
    assert np.linalg.norm(f64(y) - ref) <= 2 * HALF_BF16 * np.linalg.norm(ref)


# ---------------------------------------------------------------------------
# cache append
# ---------------------------------------------------------------------------

def spans(new, lens):
    cu = np.concatenate([[0], np.cumsum(new)])
    return list(new), list(lens), cu


def check_cache(dev, ref):
    k, v, ke, ve = from_device(dev)
    assert np.array_equal(ke, ref.ke) and np.array_equal(ve, ref.ve)
    for got, want in ((k, ref.k), (v, ref.v)):
        nan = (want & 0x7F) == 0x7F
        assert np.array_equal((got & 0x7F) == 0x7F, nan)
        assert np.array_equal(got[~nan], want[~nan])


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D,H", [(64, 3), (128, 2), (256, 1)])
def test_append(bs, D, H):
    rng = np.random.default_rng([bs, D])
    # empty sequences, one token, blocks begun, ended and crossed, a full prompt
    new, lens, cu = spans([1, 0, 1, 5, bs + 3, 2 * bs, 40, 1], [1, 30, 17, 5, bs + 30, 2 * bs, 300, 2 * bs])
    cols = max(-(-L // bs) for L in lens) + 2
    blocks = sum(-(-L // bs) for L in lens) + 3
    table = tables(rng, len(lens), cols, blocks, lens, bs, 10 ** 6)
    ref = random_cache(rng, blocks, H, bs, D)
    dev = to_device(ref)
    for step in range(2):  # the second call's tokens are larger: scales grow
        k = rng.standard_normal((cu[-1], H, D)) * 4.0 ** step
        v = rng.standard_normal((cu[-1], H, D)) * 8.0 ** step
        k[:, :, 5] *= 30
        kd, k64 = bf16(k)
        vd, v64 = bf16(v)
        announce(f"append bs={bs} D={D} step={step}")
        fql.kv_append(dev, kd, vd, i32(table), i32(lens), i32(cu), max(new))
        ref.append(k64, v64, table, lens, cu)
        check_cache(dev, ref)


def test_append_token_by_token_grows_scales():
    announce("append token by token")
    rng = np.random.default_rng(2)
    bs, H, D = 32, 2, 64
    ref = random_cache(rng, 6, H, bs, D)
    dev = to_device(ref)
    table = np.array([[4, 1], [0, 3]], dtype=np.int32)
    for t in range(40):
        k, k64 = bf16(rng.standard_normal((2, H, D)) * 2.0 ** (t % 7 - 3))
        v, v64 = bf16(rng.standard_normal((2, H, D)) * 2.0 ** (t // 5))
        lens = [t + 1, t + 20]
        fql.kv_append(dev, k, v, i32(table), i32(lens), i32([0, 1, 2]), 1)
        ref.append(k64, v64, table, lens, [0, 1, 2])
    check_cache(dev, ref)


def test_append_special_values():
    announce("append special")
    rng = np.random.default_rng(3)
    bs, H, D = 16, 4, 64
    ref = random_cache(rng, 3, H, bs, D)
    dev = to_device(ref)
    k = rng.standard_normal((20, H, D))
    k[3, 0, 1], k[4, 0, 2], k[5, 0, 3] = np.nan, np.inf, -np.inf
    k[:, 1] = 0.0
    k[:, 2] *= 1e-38
    k[0, 3, 0] = 3e38
    kd, k64 = bf16(k)
    vd, v64 = bf16(-k[::-1])
    table, lens, cu = np.array([[2, 0]], dtype=np.int32), [25], [0, 20]
    fql.kv_append(dev, kd, vd, i32(table), i32(lens), i32(cu), 20)
    ref.append(k64, v64, table, lens, cu)
    check_cache(dev, ref)


def test_append_strided_heads_of_one_projection():
    """k and v as views of one [tokens, (Hq + 2 H) D] projection, also at an odd offset."""
    rng = np.random.default_rng(4)
    bs, H, D, Hq, T = 64, 2, 128, 8, 50
    table, lens, cu = np.array([[1, 3], [0, 2]], dtype=np.int32), [70, 45], [0, 30, 50]
    for off in (0, 3):
        announce(f"append strided off={off}")
        w = (Hq + 2 * H) * D
        flat, f = bf16(rng.standard_normal(off + T * w))
        qkv = flat[off:].view(T, w)
        f = f[off:].reshape(T, w)
        k, v = qkv[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D)), qkv[:, (Hq + H) * D:].unflatten(1, (H, D))
        ref = random_cache(rng, 4, H, bs, D)
        dev = to_device(ref)
        fql.kv_append(dev, k, v, i32(table), i32(lens), i32(cu), 30)
        ref.append(f[:, Hq * D:(Hq + H) * D].reshape(T, H, D), f[:, (Hq + H) * D:].reshape(T, H, D), table, lens, cu)
        check_cache(dev, ref)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def attention_case(seed, new, lens, Hq, H, D, bs, causal=True, window=0, spread=3, q_scale=1.0, poisoned=True):
    rng = np.random.default_rng(seed)
    new, lens, cu = spans(new, lens)
    cols = max(1, max(-(-L // bs) for L in lens)) + 1
    blocks = sum(-(-L // bs) for L in lens) + 2
    table = tables(rng, len(lens), cols, blocks, lens, bs, -3)
    cache = random_cache(rng, blocks, H, bs, D, spread)
    if poisoned:
        poison(cache, table, lens)
    q, q64 = bf16(rng.standard_normal((cu[-1], Hq, D)) * q_scale)
    announce(f"attention new={new} lens={lens} Hq={Hq} H={H} D={D} bs={bs} causal={causal} window={window} "
             + fql.attention_kv8_plan(len(lens), Hq, H, D, max(new), cols * bs, window))
    out, lse = fql.attention_kv8(q, to_device(cache), i32(table), i32(lens), i32(cu), max(new), causal=causal,
                                 window=window, return_lse=True)
    torch.cuda.synchronize()
    ref = S.attention(q64, cache, table, lens, cu, D ** -0.5, causal, window)
    return out, lse, ref


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,H", [(8, 2), (3, 3), (16, 1), (14, 2), (24, 1)])
def test_attention_single_tokens(D, Hq, H):
    out, lse, ref = attention_case([1, D, Hq], [1] * 7, [1, 2, 63, 64, 65, 300, 1], Hq, H, D, 16)
    assert_attention(out, lse, ref, "single")


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_prompts(bs, D):
    out, lse, ref = attention_case([2, bs, D], [1, 70, 33, 5], [1, 70, 150, 201], 4, 2, D, bs)
    assert_attention(out, lse, ref, "prompt")


@pytest.mark.parametrize("window", [1, 5, 64, 100, 1000])
@pytest.mark.parametrize("new", [1, 3, 90])
def test_attention_window(window, new):
    out, lse, ref = attention_case([3, window, new], [new, 1, new], [new, 260, 333], 4, 2, 64, 32, window=window)
    assert_attention(out, lse, ref, "window")


@pytest.mark.parametrize("new", [1, 20, 150])
@pytest.mark.parametrize("window", [0, 40])
def test_attention_not_causal(new, window):
    out, lse, ref = attention_case([4, new], [new, 2], [200, 77], 6, 2, 128, 16, causal=False, window=window)
    assert_attention(out, lse, ref, "full")


def test_attention_empty_sequences_and_rows():
    """No new tokens, no tokens at all, and new tokens that no cached token precedes (lens < new:
    positions below zero see nothing)."""
    out, lse, ref = attention_case(5, [0, 3, 1, 0, 2], [0, 3, 40, 17, 2], 4, 4, 64, 16)
    assert_attention(out, lse, ref, "empty")
    out, lse, ref = attention_case(6, [5, 1, 4], [3, 0, 4], 4, 2, 64, 16)
    assert_attention(out, lse, ref, "short")
    assert not f64(out)[:2].any() and not f64(out)[5].any()


@pytest.mark.parametrize("new,lens", [([1, 1], [5000, 3000]), ([20], [4100]), ([2] * 3, [2049, 2048, 7])])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_split_over_keys(new, lens, D):
    out, lse, ref = attention_case([7, D, lens[0]], new, lens, 4, 1, D, 64)
    assert_attention(out, lse, ref, "split")


def test_attention_large_scores():
    """Scores of a few hundred: one key takes all, and the running maximum moves often."""
    for new in (1, 70):
        out, lse, ref = attention_case([8, new], [new], [700], 4, 2, 128, 32, spread=6, q_scale=8.0)
        assert_attention(out, lse, ref, "large")


@pytest.mark.parametrize("new", [1, 12, 80])
def test_attention_blocks_outside_the_cache_are_absent(new):
    rng = np.random.default_rng(9)
    bs, H, D, Hq, L = 16, 2, 64, 4, 190
    table = tables(rng, 1, 13, 15, [L], bs, -1)
    table[0, 2], table[0, 7], table[0, 8] = -1, 15, 2 ** 31 - 1
    cache = random_cache(rng, 15, H, bs, D)
    poison(cache, table, [L])
    q, q64 = bf16(rng.standard_normal((new, Hq, D)))
    announce(f"attention bad blocks new={new}")
    out, lse = fql.attention_kv8(q, to_device(cache), i32(table), i32([L]), i32([0, new]), new, return_lse=True)
    assert_attention(out, lse, S.attention(q64, cache, table, [L], [0, new], D ** -0.5), "blocks")


@pytest.mark.parametrize("new", [1, 5, 60])
def test_attention_blocks_below_the_window_may_hold_anything(new):
    rng = np.random.default_rng([12, new])
    bs, H, D, Hq, L, window = 16, 2, 128, 4, 300, 40
    table = tables(rng, 1, 19, 21, [L], bs, -1)
    cache = random_cache(rng, 21, H, bs, D)
    poison(cache, table, [L])
    for i in range((L - new - window + 1) // bs):  # blocks that no row sees
        blk = table[0, i]
        cache.k[blk], cache.v[blk], cache.ke[blk], cache.ve[blk] = 0x7F, 0x7F, 128, 128  # scale byte 255
    q, q64 = bf16(rng.standard_normal((new, Hq, D)))
    announce(f"attention stale blocks new={new}")
    out, lse = fql.attention_kv8(q, to_device(cache), i32(table), i32([L]), i32([0, new]), new, window=window,
                                 return_lse=True)
    assert_attention(out, lse, S.attention(q64, cache, table, [L], [0, new], D ** -0.5, window=window), "stale")


@pytest.mark.parametrize("new", [6, 40, 200])
@pytest.mark.parametrize("Hq", [1, 4])
def test_attention_nan_tokens_reach_only_rows_that_see_them(new, Hq):
    rng = np.random.default_rng([10, new])
    bs, D, L = 32, 64, 210
    table = tables(rng, 1, 8, 9, [L], bs, -1)
    cache = random_cache(rng, 9, 1, bs, D)
    poison(cache, table, [L])
    at = L - 3  # seen by the last three rows only
    cache.v[table[0][at // bs], 0, at % bs, 7] = 0x7F
    q, q64 = bf16(rng.standard_normal((new, Hq, D)))
    announce(f"attention NaN token new={new} Hq={Hq}")
    out, _ = fql.attention_kv8(q, to_device(cache), i32(table), i32([L]), i32([0, new]), new, return_lse=True)
    o, l, mass, size = S.attention(q64, cache, table, [L], [0, new], D ** -0.5)
    got = f64(out)
    assert np.array_equal(np.isnan(got), np.isnan(o)) and np.isnan(o).sum() == 3 * Hq
    fin = ~np.isnan(o)
    tol = HALF_BF16 * np.abs(o) + (HALF_BF16 + 2.0 ** -10) * mass
    assert (np.abs(got - o)[fin] <= tol[fin]).all()


def test_attention_strides_and_scale():
    rng = np.random.default_rng(11)
    bs, H, D, Hq, T, L = 64, 2, 128, 6, 30, 130
    table = tables(rng, 1, 3, 5, [L], bs, -1)
    cache = random_cache(rng, 5, H, bs, D)
    w = (Hq + 2 * H) * D
    for off in (0, 1):
        announce(f"attention strided off={off}")
        flat, f = bf16(rng.standard_normal(off + T * w))
        q = flat[off:].view(T, w)[:, :Hq * D].unflatten(1, (Hq, D))
        q64 = f[off:].reshape(T, w)[:, :Hq * D].reshape(T, Hq, D)
        store = torch.full((1 + T * (Hq * D + 2),), 5.0, dtype=torch.bfloat16, device=DEV)
        out = torch.as_strided(store, (T, Hq, D), (Hq * D + 2, D, 1), off)
        fql.attention_kv8(q, to_device(cache), i32(table), i32([L]), i32([0, T]), T, scale=0.05, out=out)
        ref = S.attention(q64, cache, table, [L], [0, T], 0.05)
        assert_attention(out, None, ref, "strided")
        gaps = store.clone()
        torch.as_strided(gaps, (T, Hq, D), (Hq * D + 2, D, 1), off).fill_(5.0)
        assert (gaps == 5.0).all()


def test_attention_max_len_only_changes_the_plan():
    rng = np.random.default_rng(12)
    bs, H, D, Hq, L = 64, 1, 128, 8, 900
    table = tables(rng, 1, 40, 16, [L], bs, -1)
    cache = to_device(random_cache(rng, 16, H, bs, D))
    q, _ = bf16(rng.standard_normal((1, Hq, D)))
    announce("attention max_len")
    # a bound below the true length (a caller's mistake) is slow, not wrong
    outs = [f64(fql.attention_kv8(q, cache, i32(table), i32([L]), i32([0, 1]), 1, max_len=m)) for m in (None, L, 256)]
    for o in outs[1:]:
        assert np.abs(o - outs[0]).max() <= 4 * HALF_BF16 * np.abs(outs[0]).max()


# ---------------------------------------------------------------------------
# streams, graphs, the whole chain
# ---------------------------------------------------------------------------

class Decoder:
    """One 8-bit decoder layer over the public entry points."""

    def __init__(self, fmt, K=512, H=2, G=4, D=64, FF=1024, seed=0):
        rng = np.random.default_rng(seed)
        self.fmt, self.K, self.H, self.Hq, self.D = fmt, K, H, H * G, D
        W = lambda n, k: rng.standard_normal((n, k)) * k ** -0.5  # noqa: E731
        both = fql.interleave_gate_up(torch.from_numpy(W(FF, K)), torch.from_numpy(W(FF, K))).numpy()
        mk = lambda w: layer(fmt, w)[0]  # noqa: E731
        self.qkv, self.o, self.gu, self.down = mk(W((self.Hq + 2 * H) * D, K)), mk(W(K, self.Hq * D)), mk(both), mk(W(K, FF))
        self.w1, self.w2 = (bf16(1 + 0.1 * rng.standard_normal(K))[0] for _ in range(2))
        self.s = 0.1 if fmt == "fp8" else None

    def __call__(self, h, cache, table, lens, cu, max_new):
        x, _ = fql.rms_norm_operand(h, self.w1, self.fmt, scale=self.s)
        qkv = fql.linear_fused(x, self.qkv)
        n = self.Hq * self.D
        q = qkv[:, :n].unflatten(1, (self.Hq, self.D))
        k, v = (t.unflatten(1, (self.H, self.D)) for t in qkv[:, n:].chunk(2, 1))
        fql.kv_append(cache, k, v, table, lens, cu, max_new)
        a = fql.attention_kv8(q, cache, table, lens, cu, max_new)
        y = fql.linear_fused(a.flatten(1), self.o)
        x, h = fql.rms_norm_operand(y, self.w2, self.fmt, residual=h, scale=self.s)
        return fql.linear_fused(fql.linear_fused(x, self.gu, activation="swiglu"), self.down, residual=h)


@pytest.mark.parametrize("fmt", FMTS)
def test_decoder_prompt_then_tokens_match_one_prompt(fmt):
    """A prompt followed by single tokens leaves the cache's values and outputs of one longer prompt,
    up to the scales' growth and the roundings after it."""
    announce(f"decoder {fmt}")
    net = Decoder(fmt)
    h, _ = bf16(np.random.default_rng(1).standard_normal((45, 512)))
    table = i32([[0, 1, 2, 3]])
    whole = net(h, fql.KVCache8.empty(4, 2, 16, 64, DEV), table, i32([45]), i32([0, 45]), 45)
    cache = fql.KVCache8.empty(4, 2, 16, 64, DEV)
    parts = [net(h[:40], cache, table, i32([40]), i32([0, 40]), 40)]
    for t in range(40, 45):
        parts.append(net(h[t:t + 1], cache, table, i32([t + 1]), i32([0, 1]), 1))
    a, b = f64(torch.cat(parts)), f64(whole)
    # E4M3 roundings of cached values (2^-4 each at most) reach the output through the residual
    # stream's attention and feed-forward branches
    assert np.linalg.norm(a - b) <= 2.0 ** -4 * np.linalg.norm(b)


def test_graph_replays_equal_eager_calls():
    announce("graph")
    net = Decoder("mxfp8")
    rng = np.random.default_rng(2)
    B = 3
    table, cu = i32([[0, 1, 2, 3], [4, 5, 6, 7], [8, 9, 10, 11]]), i32([0, 1, 2, 3])
    start = to_device(random_cache(rng, 12, 2, 16, 64))
    graph_cache = to_device(random_cache(rng, 12, 2, 16, 64))
    for a, b in zip((graph_cache.k, graph_cache.v, graph_cache.k_scale, graph_cache.v_scale),
                    (start.k, start.v, start.k_scale, start.v_scale)):
        a.copy_(b)
    h, lens = torch.zeros((B, 512), dtype=torch.bfloat16, device=DEV), i32([20, 30, 50])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        net(h, to_device(random_cache(rng, 12, 2, 16, 64)), table, lens, cu, 1)  # warms the workspace
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        y = net(h, graph_cache, table, lens, cu, 1)
    for step in range(4):
        x, _ = bf16(rng.standard_normal((B, 512)))
        h.copy_(x)
        lens.copy_(i32([20 + step, 30 + step, 50 + step]))
        g.replay()
        torch.cuda.synchronize()
        want = net(x, start, table, lens.clone(), cu, 1)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        assert torch.equal(graph_cache.k, start.k) and torch.equal(graph_cache.v, start.v)


def test_side_stream_and_repeats_are_bitwise_equal():
    announce("streams")
    rng = np.random.default_rng(3)
    bs, H, D, Hq = 64, 2, 128, 8
    lens = [4000, 1500]
    table = tables(rng, 2, 63, 90, lens, bs, -1)
    cache = to_device(random_cache(rng, 90, H, bs, D))
    q, _ = bf16(rng.standard_normal((2, Hq, D)))
    args = (cache, i32(table), i32(lens), i32([0, 1, 2]), 1)
    want = fql.attention_kv8(q, *args)
    for _ in range(5):
        assert torch.equal(fql.attention_kv8(q, *args), want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = fql.attention_kv8(q, *args)
    s.synchronize()
    assert torch.equal(got, want)


def test_expanded_tables_are_refused():
    """Rows of stride 0 are not what the kernels step by."""
    announce("expanded table")
    cache = fql.KVCache8.empty(4, 1, 16, 64, DEV)
    q, _ = bf16(np.zeros((2, 2, 64)))
    k, _ = bf16(np.zeros((2, 1, 64)))
    table, lens, cu = i32([[0, 1]]).expand(2, 2), i32([1, 1]), i32([0, 1, 2])
    with pytest.raises(fql.FQLError, match="overlap"):
        fql.attention_kv8(q, cache, table, lens, cu, 1)
    with pytest.raises(fql.FQLError, match="overlap"):
        fql.kv_append(cache, k, k, table, lens, cu, 1)
    assert fql.attention_kv8(q, cache, table.contiguous(), lens, cu, 1).shape == (2, 2, 64)


def test_a_graph_keeps_its_workspace_when_a_later_call_needs_a_larger_one():
    announce("outgrown workspace")
    rng = np.random.default_rng(4)
    bs, H, D, Hq = 64, 2, 128, 8

    def case(lens, blocks, max_len):
        table = tables(rng, len(lens), max_len // bs, blocks, lens, bs, -1)
        q, _ = bf16(rng.standard_normal((len(lens), Hq, D)))
        return (q, to_device(random_cache(rng, blocks, H, bs, D)), i32(table), i32(lens), i32(range(len(lens) + 1)), 1)

    small, large = case([900], 20, 1024), case([300 + 7 * i for i in range(40)], 400, 16384)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        want = fql.attention_kv8(*small)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = fql.attention_kv8(*small)
        key = ("cuda", 0, s.cuda_stream)
        before = fql._workspaces[key]
        fql._grow_workspace(key, 1, before.device)  # what a larger call does
        assert fql._workspaces[key].numel() >= 2 * before.numel() and any(w is before for w in fql._outgrown)
        for _ in range(4):
            fql.attention_kv8(*large)
            g.replay()
            s.synchronize()
            assert torch.equal(got, want)


@pytest.mark.parametrize("new", [5, 90])
def test_attention_window_wider_than_any_position(new):
    """The widest window hides nothing, also from a batch with more new tokens than its length."""
    out, lse, ref = attention_case([13, new], [new, 3], [new - 3, 60], 4, 2, 64, 16, window=2 ** 31 - 1)
    assert_attention(out, lse, ref, "wide window")


@pytest.mark.parametrize("new", [1, 70])
def test_caches_past_32_bits_of_offset(new):
    """Blocks beyond 4 GiB of keys hold and give what the same blocks of a small cache do."""
    announce(f"large cache new={new}")
    bs, H, D, Hq, blocks = 256, 8, 256, 16, 8200  # 4.3 GB of keys and of values each
    lens = [300, 700]
    rng = np.random.default_rng([14, new])
    small = fql.KVCache8.empty(8, H, bs, D, DEV)
    k = torch.empty((blocks, H, bs, D), dtype=torch.uint8, device=DEV)
    v = torch.empty((blocks, H, bs // 16, D, 16), dtype=torch.uint8, device=DEV)
    s = torch.zeros((2, blocks, H), dtype=torch.uint8, device=DEV)
    assert k.numel() > 2 ** 32
    large = fql.KVCache8(k, v, s[0], s[1])
    t_small = i32([[0, 1, 2], [3, 4, 5]])
    kv = [bf16(rng.standard_normal((sum(lens), H, D)))[0] for _ in range(2)]
    q, _ = bf16(rng.standard_normal((2 * new, Hq, D)))
    outs = []
    for cache, table in ((small, t_small), (large, t_small + (blocks - 8))):
        fql.kv_append(cache, *kv, table, i32(lens), i32([0, lens[0], sum(lens)]), max(lens))
        outs.append(fql.attention_kv8(q, cache, table, i32(lens), i32([0, new, 2 * new]), new))
    assert torch.equal(outs[0], outs[1])
    for i in (0, 3, 4):  # the blocks that are written whole
        assert torch.equal(large.k[i - 8], small.k[i]) and torch.equal(large.v[i - 8], small.v[i])
    for i in range(5):
        assert i == 2 or torch.equal(large.v_scale[i - 8], small.v_scale[i])


def test_a_capture_without_a_call_before_it_leaves_eager_calls_alone():
    announce("cold capture")
    rng = np.random.default_rng(15)
    lens = [4000, 900]
    table = tables(rng, 2, 63, 90, lens, 64, -1)
    q, _ = bf16(rng.standard_normal((2, 8, 128)))
    args = (q, to_device(random_cache(rng, 90, 2, 64, 128)), i32(table), i32(lens), i32([0, 1, 2]), 1)
    assert "splits=1" not in fql.attention_kv8_plan(2, 8, 2, 128, 1, 63 * 64).split()
    want = fql.attention_kv8(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    key = ("cuda", 0, s.cuda_stream)
    fql._workspaces.pop(key, None)  # the stream may be one that an earlier test used
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = fql.attention_kv8(*args)
    assert key not in fql._workspaces
    with torch.cuda.stream(s):
        assert torch.equal(fql.attention_kv8(*args), want)
        for _ in range(4):
            got.zero_()
            g.replay()
            s.synchronize()
            assert torch.equal(got, want)
            assert torch.equal(fql.attention_kv8(*args), want)
