"""INT8 on the GPU: the quantizer bit for bit, the norm in front of it, the linear layers against float64."""

import numpy as np
import pytest
import torch

import fp8_quantized_linear_amd as fql
from oracle import feedforward as O
from oracle import serving as S
from gpu_helpers import announce
from serving_helpers import DEV, HALF_BF16, bf16, f64, strided

pytestmark = pytest.mark.gpu


def weight(W):
    """(GPU weight, exact float64 weight)."""
    codes, scales = O.quant_int8(W)
    return fql.INT8Weight.from_float(torch.from_numpy(W.astype(np.float32)).to(DEV)), O.dequant_int8(codes, scales)


def x_hat(x64):
    return O.dequant_int8(*O.quant_int8(x64))


def check(y, xh, wh, bias, act, residual, what, alpha=1.0):
    """Errors counted: the sum over K is exact in integers; its conversion, the product of the scales, the
    product with them, alpha and the bias are a float32 rounding each (2^-24), a split K adds at most 16
    ranges' (2^-20 of the sum of magnitudes); the activation's slope (at most 1.13; swiglu by the product
    rule) and its float32 evaluation (2^-18, GELU 2^-16); one bf16 rounding."""
    z = alpha * (xh @ wh.T) + (0 if bias is None else bias)
    e = 2.0 ** -20 * abs(alpha) * (np.abs(xh) @ np.abs(wh).T) + 2.0 ** -22 * np.abs(z)
    v = S.activation(z, act)
    if act == "swiglu":
        (g, u), (eg, eu) = S.gate_up(z), S.gate_up(e)
        tol = 1.13 * eg * (np.abs(u) + eu) + np.abs(g) * eu
    else:
        tol = 1.13 * e
    tol = tol + 2.0 ** (-16 if act == "gelu" else -18) * np.abs(v) + 1e-30
    ref = v + (0 if residual is None else residual)
    tol = tol * (1 + HALF_BF16) + (HALF_BF16 + 2.0 ** -20) * np.abs(ref)
    d = np.abs(f64(y) - ref)
    bad = ~(d <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.size, np.argwhere(bad)[:4].tolist(), float((d / tol).max()))


SIZES = [(1, 32), (3, 96), (1, 4096), (17, 1024), (5, 14336), (130, 512), (2, 65536 + 32), (300, 160)]


@pytest.mark.parametrize("M,K", SIZES)
def test_quantizer(M, K):
    announce(f"int8 quant {M}x{K}")
    rng = np.random.default_rng([M, K])
    x, x64 = bf16(rng.standard_normal((M, K)) * np.exp2(rng.integers(-20, 20, (M, 1))))
    codes, scales = fql.quant_int8(x)
    want, ws = O.quant_int8(x64)
    assert codes.dtype == torch.int8 and codes.shape == (M, K) and scales.shape == (M,)
    assert np.array_equal(codes.cpu().numpy(), want) and np.array_equal(scales.cpu().numpy(), ws)
    W = rng.standard_normal((M, K)).astype(np.float32)
    wc, wsc = fql.quant_int8_weight(torch.from_numpy(W).to(DEV))
    want, ws = O.quant_int8(W)
    assert np.array_equal(wc.cpu().numpy(), want) and np.array_equal(wsc.cpu().numpy(), ws)


def test_quantizer_many_rows():
    """More rows than one dimension of the grid takes, through the codes and the packed operand."""
    M, K, N = (1 << 20) + 133, 32, 32
    announce(f"int8 quant {M}x{K}")
    rng = np.random.default_rng(5)
    x, x64 = bf16(rng.standard_normal((M, K)))
    codes, scales = fql.quant_int8(x)
    want, ws = O.quant_int8(x64)
    assert np.array_equal(codes.cpu().numpy(), want) and np.array_equal(scales.cpu().numpy(), ws)
    W, wh = weight(rng.standard_normal((N, K)))
    some = np.r_[0:200, (1 << 20) - 130:M]
    check(fql.linear_int8(x, W)[torch.from_numpy(some).to(DEV)], O.dequant_int8(want[some], ws[some]), wh, None, "none", None,
          "many rows")


def test_quantizer_extremes():
    """Zero rows, subnormal rows, ties, infinities and NaN."""
    announce("int8 quant extremes")
    x = np.zeros((9, 64), dtype=np.float32)
    x[1, 5] = 2.0 ** -133                    # a bf16 subnormal alone: 1 / s overflows
    x[2] = 2.0 ** -126
    x[3] = 3.3895313892515355e38             # the largest bf16
    x[4, :3] = [127, 0.5, 1.5]               # ties: s = 1
    x[4, 3:6] = [-127, -0.5, -2.5]
    x[5, 7] = np.inf
    x[6, 7] = -np.inf
    x[7, 63] = np.nan
    x[8] = -0.0
    t, x64 = bf16(x)
    codes, scales = (a.cpu().numpy() for a in fql.quant_int8(t))
    want, ws = O.quant_int8(x64)
    bad = np.isnan(ws)
    assert bad.tolist() == [False] * 5 + [True] * 3 + [False]
    assert np.array_equal(np.isnan(scales), bad) and np.array_equal(scales[~bad], ws[~bad])
    assert np.array_equal(codes[~bad], want[~bad])
    assert codes[4, :6].tolist() == [127, 0, 2, -127, 0, -2]
    # the rows' outputs: NaN where the scale is, in every plan
    g, _ = weight(np.random.default_rng(0).standard_normal((48, 64)))
    for rows in (9, 40, 200):
        y = fql.linear_int8(t.repeat(-(-rows // 9), 1)[:rows], g)
        assert np.array_equal(np.isnan(f64(y)).all(1), np.resize(bad, rows))
        assert np.array_equal(np.isnan(f64(y)).any(1), np.resize(bad, rows))


@pytest.mark.parametrize("M,K", [(1, 4096), (3, 256), (17, 5120), (130, 1024), (2, 70016)])
def test_norm(M, K):
    """Codes of y = h w / sqrt(mean h^2 + eps) within one rounding of y to float32 and one of the scale."""
    announce(f"int8 norm {M}x{K}")
    rng = np.random.default_rng([M, K, 1])
    x, x64 = bf16(rng.standard_normal((M, K)) * 3)
    r, r64 = bf16(rng.standard_normal((M, K)))
    w, w64 = bf16(1 + 0.1 * rng.standard_normal(K))
    op, h = fql.rms_norm_operand(x, w, "int8", residual=r)
    q, scales = operand_rows(op)
    y, h64 = S.rms_norm(x64, w64, float(np.float32(1e-6)), r64)
    assert torch.equal(h, (x.float() + r.float()).to(torch.bfloat16))
    # x + r is rounded to float32 (2^-24 a term), y once, the scale and its reciprocal once each
    s = np.abs(y).max(1) / 127
    assert (np.abs(scales - s) <= 2.0 ** -21 * s).all()
    assert (np.abs(q - y / s[:, None]) <= 0.5 + 127 * 2.0 ** -20).all()
    g, wh = weight(rng.standard_normal((64, K)))
    check(fql.linear_fused(op, g), q * scales[:, None], wh, None, "none", None, "norm")


def operand_rows(op):
    """(codes float64 [M, K], scales float64 [M]) of an INT8 operand."""
    KC, Mp = -(-op.K // 128), -(-op.M // 256) * 256
    d = op.data.cpu().numpy()
    q = d[:Mp * KC * 128].view(np.int8).reshape(Mp // 16, KC, 2, 4, 16, 16).transpose(0, 4, 1, 2, 3, 5)
    q = q.reshape(Mp, KC * 128)[:op.M]
    assert not q[:, op.K:].any()
    return q[:, :op.K].astype(np.float64), d[Mp * KC * 128:].view(np.float32)[:op.M].astype(np.float64)


def test_norm_in_place_and_bad_rows():
    announce("int8 norm in place")
    rng = np.random.default_rng(4)
    for K in (512, 70016):
        x, x64 = bf16(rng.standard_normal((4, K)))
        x[1, 3] = float("nan")
        x[2, 5] = float("inf")
        r, _ = bf16(rng.standard_normal((4, K)))
        w, _ = bf16(np.ones(K))
        want = operand_rows(fql.rms_norm_operand(x, w, "int8", residual=r)[0])
        a, b = x.clone(), r.clone()
        for into in (a, b):
            op, h = fql.rms_norm_operand(a if into is a else x, w, "int8", residual=b if into is b else r,
                                         residual_out=into)
            assert h is into
            got, ok = operand_rows(op), [0, 3]
            assert np.array_equal(got[0][ok], want[0][ok]) and np.array_equal(got[1][ok], want[1][ok])
            assert np.isnan(got[1][[1, 2]]).all()


CASES = [(M, 512, 1024) for M in (1, 9, 16, 17, 32)] + [
    (33, 384, 512), (100, 256, 2048), (129, 640, 384), (300, 256, 512), (600, 512, 256), (1, 200, 32), (40, 33, 96),
    (7, 1, 64), (530, 70, 160)]


@pytest.mark.parametrize("M,N,K", CASES)
def test_linear(M, N, K):
    rng = np.random.default_rng([M, N, K])
    x, x64 = bf16(rng.standard_normal((M, K)) * 2)
    W = rng.standard_normal((N, K)) * np.exp2(rng.integers(-6, 3, (N, 1)))
    g, wh = weight(W)
    b, b64 = bf16(rng.standard_normal(N))
    xh = x_hat(x64)
    announce(f"int8 linear {M}x{N}x{K}")
    check(fql.linear_int8(x, g), xh, wh, None, "none", None, "plain")
    check(fql.linear_int8(x, g, alpha=0.5, bias=b), xh, wh, b64, "none", None, "bias", alpha=0.5)
    op = fql.quant_operand(x, "int8")
    for i, act in enumerate(("none", "relu", "gelu", "gelu_tanh", "silu", "swiglu")):
        if act == "swiglu" and N % 32:
            continue
        No = N // 2 if act == "swiglu" else N
        r, r64 = bf16(rng.standard_normal((M, No)) * 4)
        res, bias = i % 2 == 0, i % 3 != 0
        args = dict(activation=act, bias=b if bias else None, residual=r if res else None)
        y = fql.linear_fused(x, g, **args)
        check(y, xh, wh, b64 if bias else None, act, r64 if res else None, (M, N, K, act))
        assert torch.equal(fql.linear_fused(op, g, **args), y)


# tiles whole and with K in ranges (16 x 128 .. 256 x 128)
PLANNED = [(40, 1000, 1024), (250, 4096, 1024), (500, 4000, 512), (1000, 4096, 512), (1900, 4096, 512),
           (60, 4096, 14336), (120, 4096, 14336), (250, 5120, 12800)]


@pytest.mark.parametrize("M,N,K", PLANNED)
def test_linear_planned_tiles(M, N, K):
    announce(f"int8 {M}x{N}x{K} {fql.linear_fused_plan('int8', M, N, K)}")
    rng = np.random.default_rng([M, N])
    x, x64 = bf16(rng.standard_normal((M, K), dtype=np.float32))
    W = rng.standard_normal((N, K), dtype=np.float32) * np.float32(0.05)
    g = fql.INT8Weight.from_float(torch.from_numpy(W).to(DEV))
    r, r64 = bf16(rng.standard_normal((M, N), dtype=np.float32))
    rows = np.unique(np.concatenate([[0, 15, 16, 31, M // 2, M - 17, M - 1], rng.integers(0, M, 16)]))
    cols = np.unique(np.concatenate([np.arange(128), np.arange(N - 128, N)]))
    wh = O.dequant_int8(*O.quant_int8(W[cols]))
    xh = x_hat(x64[rows])
    for plain in (False, True):
        y = fql.linear_int8(x, g) if plain else fql.linear_fused(x, g, activation="silu", residual=r)
        check(y[torch.from_numpy(rows).to(DEV)][:, torch.from_numpy(cols).to(DEV)], xh, wh, None,
              "none" if plain else "silu", None if plain else r64[np.ix_(rows, cols)], (M, N, K, plain))


@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_largest_sums_and_codes(M):
    """The longest K with every code at its end, -128 among the weight's: 2130706432 a sum."""
    announce(f"int8 largest sums M={M}")
    K = 131072
    x = torch.full((M, K), 127.0, dtype=torch.bfloat16, device=DEV)
    codes = torch.full((48, K), -128, dtype=torch.int8, device=DEV)
    codes[1::2] = 127
    scales = torch.full((48,), 2.0 ** -20, device=DEV)
    g = fql.INT8Weight(fql.pack_weight_int8(codes, scales), 48, K)
    y = f64(fql.linear_int8(x, g))
    want = np.where(np.arange(48) % 2 == 0, -128.0, 127.0) * 127 * K * 2.0 ** -20
    assert (np.abs(y - want) <= (HALF_BF16 + 2.0 ** -20) * np.abs(want)).all()


@pytest.mark.parametrize("M", [1, 20, 70, 300])
def test_strides_rows_and_in_place(M):
    announce(f"int8 strides M={M}")
    rng = np.random.default_rng(M)
    K, N = 288, 72
    x, x64 = strided(rng.standard_normal((M, K)), K + 3, 1)
    g, wh = weight(rng.standard_normal((N, K)) * 0.1)
    r, r64 = strided(rng.standard_normal((M, N)), N + 5, 3)
    flat = torch.full((2 + M * (N + 9) + 8,), -7.0, dtype=torch.bfloat16, device=DEV)
    out = torch.as_strided(flat, (M, N), (N + 9, 1), 2)
    fql.linear_fused(x, g, activation="silu", residual=r, out=out)
    check(out, x_hat(x64), wh, None, "silu", r64, "strided")
    gaps = flat.clone()
    torch.as_strided(gaps, (M, N), (N + 9, 1), 2).fill_(-7.0)
    assert (gaps == -7.0).all()
    want = out.clone()
    rr = r.clone()
    fql.linear_fused(x, g, activation="silu", residual=rr, out=rr)
    assert torch.equal(rr, want)
    assert fql.linear_fused(x[:0], g).shape == (0, N)


def test_repack_and_graph():
    """A captured call sees new weights and new inputs, and runs beside eager calls."""
    announce("int8 graph")
    rng = np.random.default_rng(8)
    x, _ = bf16(rng.standard_normal((5, 512)))
    g, _ = weight(rng.standard_normal((128, 512)))
    other, _ = weight(rng.standard_normal((128, 512)))
    fql.linear_int8(x, g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = fql.linear_fused(x, g, activation="silu")
    for i in range(4):
        x.copy_(bf16(rng.standard_normal((5, 512)))[0])
        if i == 2:
            W = torch.from_numpy(rng.standard_normal((128, 512)).astype(np.float32)).to(DEV)
            g.repack_(*fql.quant_int8_weight(W))
        graph.replay()
        fql.linear_int8(x, other)
        torch.cuda.synchronize()
        assert torch.equal(y, fql.linear_fused(x, g, activation="silu"))


def test_warmup_takes_int8_layers():
    announce("int8 warmup")
    g, _ = weight(np.random.default_rng(1).standard_normal((64, 128)))
    assert fql.warmup([g, g], [1, 40]) == 2


def check_relative(y, want, what):
    """`want` is what the exact sums of integers times the scales come to, all normal numbers of bf16, zeros or
    beyond its range. Counted: the sum's conversion and the scales' products a float32 rounding each (2^-24), the
    join of up to 16 ranges of K, whose terms all have one sign or cancel exactly (2^-20), one bf16 rounding."""
    y = f64(y)
    top = 3.3895313892515355e38
    past = np.abs(want) > top * (1 + 2.0 ** -9)
    assert np.array_equal(np.isinf(y), past), what
    assert (np.sign(y) == np.sign(want)).all(), what
    d = np.abs(np.where(past, 0.0, y) - np.where(past, 0.0, want))
    assert (d <= (HALF_BF16 + 2.0 ** -20) * np.where(past, 0.0, np.abs(want))).all(), (what, float(np.nanmax(d)))


# (row's scale 2^a, channel's scale 1.4 * 2^b): their product alone is below or above float32's range, or the
# sum times the row's scale is, while what comes of all three is a normal number
APART = [(-98, -51), (-75, -74), (-110, -30), (121, 8), (121, -30), (100, 40), (60, -60), (0, 0)]


@pytest.mark.parametrize("M", [1, 20, 70, 300])
def test_scales_of_any_size_beside_one_another(M):
    K, N = 4096, 64
    announce(f"int8 scales of any size M={M} {fql.linear_sc_plan('int8', M, N, K)}")
    rng = np.random.default_rng(M)
    codes = rng.integers(90, 128, (N, K))
    codes[3::4, 1::2] = -codes[3::4, 0::2]  # with equal neighbours in x these columns' sums are 0 in every range of K
    q = np.repeat(rng.integers(64, 127, (M, K // 2)), 2, axis=1)
    q[:, :2] = 127
    sums = q.astype(np.float64) @ codes.T
    wc = torch.from_numpy(codes.astype(np.int8)).to(DEV)
    for a, b in APART:
        x, x64 = bf16(np.ldexp(q.astype(np.float64), a))
        assert np.array_equal(x64, np.ldexp(q.astype(np.float64), a))
        sw = np.full(N, np.ldexp(np.float32(1.4), b), dtype=np.float32)
        g = fql.INT8Weight(fql.pack_weight_int8(wc, torch.from_numpy(sw).to(DEV)), N, K)
        with np.errstate(over="ignore"):
            want = np.ldexp(sums, a) * sw.astype(np.float64)
        check_relative(fql.linear_int8(x, g), want, ("plain", a, b))
        check_relative(fql.linear_fused(x, g, activation="relu"), want, ("fused", a, b))
        check_relative(fql.linear_fused(fql.quant_operand(x, "int8"), g, activation="relu"), want, ("operand", a, b))
        # gated, with ups of their own size: silu(z) is z where z is large, z / 2 where it is small
        if a + b > -40:
            continue
        up = sw.reshape(-1, 32).copy()
        up[:, 16:] = np.ldexp(np.float32(1.0), -a - 20)
        g = fql.INT8Weight(fql.pack_weight_int8(wc, torch.from_numpy(up.reshape(-1)).to(DEV)), N, K)
        z, u = (np.ldexp(v, a).reshape(M, -1, 16) for v in np.split(sums.reshape(M, -1, 32), 2, axis=2))
        want = (z * float(sw[0]) / 2 * u * 2.0 ** (-a - 20)).reshape(M, -1)
        y = f64(fql.linear_fused(x, g, activation="swiglu"))
        assert (np.abs(y - want) <= (HALF_BF16 + 2.0 ** -17) * np.abs(want)).all(), ("gated", a, b)
