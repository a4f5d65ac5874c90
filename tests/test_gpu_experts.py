"""The chosen experts' feed forward on the GPU against float64, with the inner activation's codes bounded by
what its float32 value may be off."""

import numpy as np
import pytest
import torch

import fp8_quantized_linear_amd as fql
from oracle import feedforward as O
from oracle import formats as F
from oracle import fp8 as P
from oracle import mx as X
from oracle import serving as S
from gpu_helpers import announce
from serving_helpers import DEV, HALF_BF16, bf16, f64, strided

pytestmark = pytest.mark.gpu

FMTS = ("fp8", "fp8_block", "mxfp8", "mxfp4", "int8")
SX, SH = 0.05, 0.03  # per-tensor FP8's static scales


def experts_of(fmt, W, scale):
    """(ExpertWeight, exact float64 weights) of float weights [E, N, K]."""
    g = fql.ExpertWeight.from_float(torch.from_numpy(W.astype(np.float32)).to(DEV), fmt,
                                    input_scale=scale if fmt == "fp8" else None)
    exact = []
    for e, w in enumerate(W.astype(np.float32)):
        if fmt == "fp8":
            s = np.float32(np.float64(np.float32(np.abs(w).max())) / 448)
            exact.append(F.e4m3_decode(P.quant_fp8_tensor(w, s)) * float(s))
        elif fmt == "mxfp4":
            exact.append(X.dequant_mxfp4(*X.quant_mxfp4(w)))
        elif fmt == "mxfp8":
            exact.append(P.dequant_mxfp8(*P.quant_mxfp8(w)))
        elif fmt == "int8":
            exact.append(O.dequant_int8(*O.quant_int8(w)))
        else:
            exact.append(P.dequant_fp8_block_weight(*P.quant_fp8_block_weight(w)))
    return g, np.stack(exact)


def hat(fmt, x64, scale):
    x32 = x64.astype(np.float32)
    if fmt == "fp8":
        return F.e4m3_decode(P.quant_fp8_tensor(x32, np.float32(scale))) * float(np.float32(scale))
    if fmt == "mxfp4":
        return X.dequant_mxfp4(*X.quant_mxfp4(x32))
    if fmt == "mxfp8":
        return P.dequant_mxfp8(*P.quant_mxfp8(x32))
    if fmt == "int8":
        return O.dequant_int8(*O.quant_int8(x32))
    return P.dequant_fp8_block_act(*P.quant_fp8_block_act(x32))


def code_values(fmt, v, tol, scale):
    """(dequantized codes of v, what they may be off when v is off by tol): a quantizer is monotone, so codes
    of a value within tol lie between those of v - tol and v + tol; a block's scale moves with its largest
    value, which shifts its quotients by as much relatively."""
    n = {"fp8": v.shape[1], "int8": v.shape[1], "fp8_block": 128, "mxfp8": 32, "mxfp4": 32}[fmt]
    t, d = v.reshape(v.shape[0], -1, n), tol.reshape(v.shape[0], -1, n)
    a = np.abs(t).max(2, keepdims=True)
    ta = d.max(2, keepdims=True)
    if fmt == "fp8":
        steps = [np.full_like(a, float(np.float32(scale)))]
    elif fmt in ("fp8_block", "int8"):
        steps = [np.maximum(a / (448 if fmt == "fp8_block" else 127), 1e-300)]
        d = d + np.abs(t) * (ta / np.maximum(a, 1e-300) + 2.0 ** -22)
    else:
        top = 8 if fmt == "mxfp8" else 2
        steps = [np.exp2(np.clip(np.floor(np.log2(np.maximum(b, 1e-300))) - top, -127, 127))
                 for b in (a, a - ta, a + ta)]

    def grid(q):
        q = np.clip(q, -1e30, 1e30)
        if fmt == "int8":
            return np.clip(np.rint(q), -127, 127)
        q32 = q.astype(np.float32)
        if fmt == "mxfp4":
            return F.e2m1_decode(F.e2m1_encode(np.clip(q32, -6, 6)))
        return F.e4m3_decode(F.e4m3_encode(np.clip(q32, -448, 448)))

    mid = grid(t / steps[0]) * steps[0]
    lo = np.min([grid((t - d) / s) * s for s in steps], 0)
    hi = np.max([grid((t + d) / s) * s for s in steps], 0)
    return mid.reshape(v.shape), np.maximum(hi - mid, mid - lo).reshape(v.shape)


def reference(fmt, xh, wu, wd, weights, ids, act, bu, bd, res):
    """(y, tolerance) of tokens xh [T, H]. Counted: the products' sums (2^-12 of the sum of magnitudes for the
    FP8 and FP4 matrix instructions, 2^-20 for integers), the activation as in the linear layers' tests, the
    codes of h (code_values), an fp16 rounding of each d, float32 sums, a bf16 rounding of y. d is divided by a
    power of two before it, so that the largest of 32 columns lies in 2^14 .. 2^15: an fp16 rounding is off by
    at most 2^-11 of the value, or by 2^-25 below 2^-14, which is 2^-39 of the largest."""
    rel = 2.0 ** -20 if fmt == "int8" else 2.0 ** -12
    E = wu.shape[0]
    y = np.zeros((xh.shape[0], wd.shape[1])) if res is None else res.copy()
    tol = np.zeros_like(y)
    mass = np.abs(y)
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if t.size == 0:
            continue
        z = xh[t] @ wu[e].T + (0 if bu is None else bu[e])
        ez = rel * (np.abs(xh[t]) @ np.abs(wu[e]).T) + 2.0 ** -22 * np.abs(z)
        h = S.activation(z, act)
        if act == "swiglu":
            (g, u), (eg, eu) = S.gate_up(z), S.gate_up(ez)
            eh = 1.13 * eg * (np.abs(u) + eu) + np.abs(g) * eu
        else:
            eh = 1.13 * ez
        eh = eh + 2.0 ** (-16 if act == "gelu" else -18) * np.abs(h) + 1e-30
        hq, off = code_values(fmt, h, eh, SH)
        d = hq @ wd[e].T + (0 if bd is None else bd[e])
        ed = off @ np.abs(wd[e]).T + rel * (np.abs(hq) + off) @ np.abs(wd[e]).T + 2.0 ** -22 * np.abs(d)
        top = np.abs(d) + ed
        top = np.pad(top, ((0, 0), (0, -top.shape[1] % 32))).reshape(top.shape[0], -1, 32).max(2)
        ed = ed * (1 + 2.0 ** -11) + 2.0 ** -11 * np.abs(d) + 2.0 ** -39 * np.repeat(top, 32, 1)[:, :d.shape[1]]
        w = weights[t, j][:, None]
        np.add.at(y, t, w * d)
        np.add.at(tol, t, np.abs(w) * ed)
        np.add.at(mass, t, np.abs(w * d))
    tol = tol + 2.0 ** -20 * mass
    return y, tol * (1 + HALF_BF16) + HALF_BF16 * np.abs(y) + 1e-30


def check(y, ref, tol, what):
    d = np.abs(f64(y) - ref)
    bad = ~(d <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.size, np.argwhere(bad)[:4].tolist(), float(np.nanmax(d / tol)))
    # the bounds are of the worst case; what is usual is far inside them
    assert np.linalg.norm(d) <= 0.05 * np.linalg.norm(ref) + 1e-30, what


class Layer:
    def __init__(self, fmt, E, H, I, Ho=None, act="swiglu", seed=0, bias=False):
        rng = np.random.default_rng([E, H, I, seed])
        Ho = Ho or H
        self.fmt, self.E, self.H, self.act = fmt, E, H, act
        N = 2 * I if act == "swiglu" else I
        self.up, self.wu = experts_of(fmt, rng.standard_normal((E, N, H)) * H ** -0.5, SX)
        self.down, self.wd = experts_of(fmt, rng.standard_normal((E, Ho, I)) * I ** -0.5, SH)
        self.bu = self.bd = self.bu64 = self.bd64 = None
        if bias:
            self.bu, self.bu64 = bf16(rng.standard_normal((E, N)))
            self.bd, self.bd64 = bf16(rng.standard_normal((E, Ho)))

    def __call__(self, x, w, e, **args):
        return fql.experts_fused(x, self.up, self.down, w, e, activation=self.act, bias_up=self.bu, bias_down=self.bd,
                                 **args)

    def reference(self, x64, w64, ids, res=None):
        return reference(self.fmt, hat(self.fmt, x64, SX), self.wu, self.wd, w64, ids, self.act, self.bu64, self.bd64, res)


def choice(rng, T, E, k, skew=0.0):
    """Weights and distinct experts; `skew` makes the first ones more popular."""
    s = rng.standard_normal((T, E)) - skew * np.arange(E)
    ids = np.argsort(-s, axis=1)[:, :k].astype(np.int32)
    w = rng.random((T, k)).astype(np.float32) + 0.1
    w /= w.sum(1, keepdims=True)
    return torch.from_numpy(w).to(DEV), torch.from_numpy(ids).to(DEV), w.astype(np.float64), ids


CASES = [(1, 4, 8, 256, 128), (5, 2, 4, 128, 384), (16, 8, 16, 384, 128), (40, 3, 5, 256, 256), (200, 2, 3, 256, 128),
         (333, 4, 4, 128, 256), (700, 1, 2, 256, 128)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k,E,H,I", CASES)
def test_experts(fmt, T, k, E, H, I):
    announce(f"experts {fmt} T={T} k={k} E={E} H={H} I={I} {fql.experts_fused_plan(fmt, T, k, E, H, 2 * I, H)}")
    rng = np.random.default_rng([T, k, E])
    layer = Layer(fmt, E, H, I)
    x, x64 = bf16(rng.standard_normal((T, H)))
    r, r64 = bf16(rng.standard_normal((T, H)))
    w, e, w64, ids = choice(rng, T, E, k, skew=0.3)
    y = layer(x, w, e, residual=r)
    check(y, *layer.reference(x64, w64, ids, r64), "residual")
    check(layer(x, w, e), *layer.reference(x64, w64, ids), "plain")
    # out over the residual, and over x
    rr = r.clone()
    assert layer(x, w, e, residual=rr, out=rr) is rr and torch.equal(rr, y)
    xx = x.clone()
    layer(xx, w, e, residual=r, out=xx)
    assert torch.equal(xx, y)


# (T, k, E, H, I, Ho) at which the products take tiles of 64, 128 and 256 rows, each of the formats
TILES = [(1500, 4, 16, 384, 256, 256), (6000, 2, 3, 384, 384, 640), (3000, 2, 8, 384, 640, 640),
         (800, 2, 32, 384, 256, 2176), (3000, 2, 4, 384, 384, 256), (300, 2, 3, 6784, 128, 256),
         (150, 2, 3, 256, 8192, 384)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k,E,H,I,Ho", TILES)
def test_tiles(fmt, T, k, E, H, I, Ho):
    """Many tokens, an expert's rows ending anywhere in a tile; some of the rows, and every row again."""
    announce(f"experts tiles {fmt} T={T} k={k} E={E} H={H} I={I} {fql.experts_fused_plan(fmt, T, k, E, H, 2 * I, Ho)}")
    rng = np.random.default_rng([T, E])
    layer = Layer(fmt, E, H, I, Ho=Ho, bias=True)
    x, x64 = bf16(rng.standard_normal((T, H)))
    w, e, w64, ids = choice(rng, T, E, k, skew=0.1)
    y = layer(x, w, e)
    rows = np.unique(np.concatenate([[0, T - 1], rng.integers(0, T, 150)]))
    check(y[torch.from_numpy(rows).to(DEV)], *layer.reference(x64[rows], w64[rows], ids[rows]), "tiles")
    # a token's result does not depend on where its pairs come to lie
    order = torch.from_numpy(rng.permutation(T)).to(DEV)
    assert torch.equal(layer(x[order].contiguous(), w[order].contiguous(), e[order].contiguous()), y[order])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [4, 70])
def test_rows_of_any_size_on_their_way(fmt, T):
    """Outputs of very different sizes beside one another, and columns whose weights are not finite: the rows of
    the second product keep 2^-11 of each or 2^-39 of the largest of 32, and infinities and NaN where they are."""
    announce(f"experts rows {fmt} T={T}")
    rng = np.random.default_rng(T)
    E, H, I, Ho = 3, 128, 128, 176 if fmt != "fp8_block" else 256
    layer = Layer(fmt, E, H, I, Ho=Ho)
    x, x64 = bf16(rng.standard_normal((T, H)))
    w, e, w64, ids = choice(rng, T, E, 2)
    big = np.zeros(Ho)
    big[5], big[40], big[41], big[75] = 3e38, np.inf, np.nan, -np.inf
    big[64:80] += 1e-39
    big[96:112] = 2.0 ** np.arange(-100, -52, 3)
    layer.bd, layer.bd64 = bf16(np.tile(big, (E, 1)))
    y = f64(layer(x, w, e))
    with np.errstate(invalid="ignore"):
        ref, _ = layer.reference(x64, w64, ids)
    odd = [40, 41, 75]
    assert np.isposinf(y[:, 40]).all() and np.isnan(y[:, 41]).all() and np.isneginf(y[:, 75]).all()
    layer.bd64 = np.where(np.isfinite(layer.bd64), layer.bd64, 0.0)
    ref, tol = layer.reference(x64, w64, ids)
    keep = [n for n in range(Ho) if n not in odd]
    d = np.abs(y - ref)[:, keep]
    assert (d <= tol[:, keep]).all(), np.argwhere(d > tol[:, keep])[:4]


FEW = [(1, 1, 1, 32, 32, 16), (1, 64, 64, 96, 160, 33), (1, 5, 9, 640, 544, 130), (2, 3, 40, 1120, 96, 77),
       (4, 16, 96, 128, 288, 48), (6, 2, 24, 224, 1184, 256), (3, 7, 64, 2080, 128, 20)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k,E,H,I,Ho", FEW)
def test_a_few_tokens(fmt, T, k, E, H, I, Ho):
    """Every pair for itself, without sorting: rows at odd addresses, columns and depths that end inside a tile
    and a wave's chunks, absent and repeated experts, an inner activation of every kind."""
    if fmt == "fp8_block":
        H, I, Ho = (-(-n // 128) * 128 for n in (H, I, Ho))
    announce(f"experts few {fmt} T={T} k={k} E={E} H={H} I={I} Ho={Ho}")
    rng = np.random.default_rng([T, k, E, H])
    act = ("silu", "swiglu", "none")[k % 3]
    N = 2 * I if act == "swiglu" else I
    assert "token_up" in fql.experts_fused_plan(fmt, T, k, E, H, N, Ho, act)
    layer = Layer(fmt, E, H, I, Ho=Ho, act=act, bias=k % 2 == 1)
    x, x64 = strided(rng.standard_normal((T, H)), H + 3, 1)
    r, r64 = strided(rng.standard_normal((T, Ho)), Ho + 5, 3)
    w, _, w64, ids = choice(rng, T, E, k)
    check(layer(x, w, torch.from_numpy(ids).to(DEV), residual=r), *layer.reference(x64, w64, ids, r64), "all")
    ids[0, -1] = ids[0, 0]
    if k > 1:
        ids[-1, 1] = E if T % 2 else -1
    e = torch.from_numpy(ids).to(DEV)
    y = layer(x, w, e)
    check(y, *layer.reference(x64, w64, ids), "absent and repeated")
    for _ in range(2):
        assert torch.equal(layer(x, w, e), y)
    ids[:] = -7
    assert torch.equal(layer(x, w, torch.from_numpy(ids).to(DEV), residual=r), r)


@pytest.mark.parametrize("fmt", FMTS)
def test_a_few_tokens_keep_to_themselves(fmt):
    """A row of NaN and a NaN weight reach their own token alone; an unchosen expert's NaN weights reach none."""
    announce(f"experts few NaN {fmt}")
    rng = np.random.default_rng(3)
    E, H = 32, 256
    layer = Layer(fmt, E, H, 128)
    assert "token_up" in fql.experts_fused_plan(fmt, 4, 2, E, H, 256, H)
    x, _ = bf16(rng.standard_normal((4, H)))
    w, e, _, ids = choice(rng, 4, E, 2)
    want = layer(x, w, e)
    idle = [i for i in range(E) if i not in ids][0]
    layer.up.packed[idle] = 0xFF
    layer.down.packed[idle] = 0xFF
    assert torch.equal(layer(x, w, e), want)
    w2, x2 = w.clone(), x.clone()
    w2[1, 0] = float("nan")
    x2[3] = float("nan")
    got = layer(x2, w2, e)
    assert torch.equal(got[[0, 2]], want[[0, 2]])
    assert torch.isnan(got[1]).all()
    if fmt == "int8":  # the other formats' quantizers saturate a NaN
        assert torch.isnan(got[3]).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"])
def test_activations_and_biases(fmt, act):
    for T in (3, 90):
        announce(f"experts {fmt} {act} T={T}")
        rng = np.random.default_rng(T)
        layer = Layer(fmt, 3, 128, 256, act=act, bias=True)
        x, x64 = bf16(rng.standard_normal((T, 128)))
        w, e, w64, ids = choice(rng, T, 3, 2)
        check(layer(x, w, e), *layer.reference(x64, w64, ids), (fmt, act))


@pytest.mark.parametrize("fmt", ("fp8", "mxfp8", "mxfp4", "int8"))
@pytest.mark.parametrize("T", [1, 7, 60, 400])
def test_odd_sizes_and_strides(fmt, T):
    """Columns that end inside a chunk or a tile, rows with gaps that stay as they are."""
    announce(f"experts odd {fmt} T={T}")
    rng = np.random.default_rng(T)
    H, I, Ho, E = 96, 160, 77, 3
    layer = Layer(fmt, E, H, I, Ho=Ho)
    x, x64 = strided(rng.standard_normal((T, H)), H + 3, 1)
    r, r64 = strided(rng.standard_normal((T, Ho)), Ho + 5, 3)
    w, e, w64, ids = choice(rng, T, E, 2)
    flat = torch.full((2 + T * (Ho + 9) + 8,), -7.0, dtype=torch.bfloat16, device=DEV)
    out = torch.as_strided(flat, (T, Ho), (Ho + 9, 1), 2)
    layer(x, w, e, residual=r, out=out)
    check(out, *layer.reference(x64, w64, ids, r64), "strided")
    gaps = flat.clone()
    torch.as_strided(gaps, (T, Ho), (Ho + 9, 1), 2).fill_(-7.0)
    assert (gaps == -7.0).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [2, 70, 600])
def test_absent_repeated_and_lone_experts(fmt, T):
    """Experts out of range, one expert in both places, one expert for all, none at all."""
    announce(f"experts absent {fmt} T={T}")
    rng = np.random.default_rng(T)
    E, H = 6, 128
    layer = Layer(fmt, E, H, 128)
    x, x64 = bf16(rng.standard_normal((T, H)))
    r, r64 = bf16(rng.standard_normal((T, H)))
    w, _, w64, _ = choice(rng, T, E, 3)
    for kind in ("absent", "repeated", "lone", "none"):
        ids = rng.integers(-2, E + 2, (T, 3)).astype(np.int32)
        if kind == "absent":
            ids[0] = [-1, E, 2 ** 31 - 1]
            ids[1, 0] = -2 ** 31
        elif kind == "repeated":
            ids[:, 1] = ids[:, 0] = rng.integers(0, E, T)
        elif kind == "lone":
            ids[:] = 4
        else:
            ids[:] = -1
        y = layer(x, w, torch.from_numpy(ids).to(DEV), residual=r)
        check(y, *layer.reference(x64, w64, ids, r64), kind)
        if kind == "none":
            assert torch.equal(y, r)
            assert (layer(x, w, torch.from_numpy(ids).to(DEV)) == 0).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_a_token_does_not_reach_another(fmt):
    """A row of NaN reaches its own output alone, and a NaN weight likewise."""
    for T in (6, 150):
        announce(f"experts NaN {fmt} T={T}")
        rng = np.random.default_rng(T)
        layer = Layer(fmt, 3, 256, 128)
        x, _ = bf16(rng.standard_normal((T, 256)))
        w, e, _, _ = choice(rng, T, 3, 2)
        want = layer(x, w, e)
        w2, x2 = w.clone(), x.clone()
        w2[1, 0] = float("nan")
        x2[4] = float("nan")
        x2[2, 7] = float("inf")
        got = layer(x2, w2, e)
        same = [t for t in range(T) if t not in (1, 2, 4)]
        assert torch.equal(got[same], want[same])
        assert torch.isnan(got[1]).all()
        if fmt == "int8":
            assert torch.isnan(got[[2, 4]]).all()


@pytest.mark.parametrize("fmt", ("mxfp8", "int8"))
def test_many_experts_and_places(fmt):
    announce(f"experts many {fmt}")
    rng = np.random.default_rng(1)
    E, H, T, k = 200, 64, 37, 16
    layer = Layer(fmt, E, H, 64)
    x, x64 = bf16(rng.standard_normal((T, H)))
    w, e, w64, ids = choice(rng, T, E, k)
    check(layer(x, w, e), *layer.reference(x64, w64, ids), "many")


def test_passes_over_tokens():
    """More tokens than one pass of the workspace takes."""
    T, k, E, H, I = 2600, 8, 8, 128, 14336
    plan = fql.experts_fused_plan("mxfp8", T, k, E, H, 2 * I, H)
    announce(f"experts passes {plan}")
    rng = np.random.default_rng(2)
    layer = Layer("mxfp8", E, H, I)
    x, x64 = bf16(rng.standard_normal((T, H), dtype=np.float32))
    w, e, w64, ids = choice(rng, T, E, k)
    y = layer(x, w, e, out=x.clone())
    rows = np.unique(np.concatenate([[0, T - 1], rng.integers(0, T, 20), np.arange(1400, 1900, 50)]))
    check(y[torch.from_numpy(rows).to(DEV)], *layer.reference(x64[rows], w64[rows], ids[rows]), "passes")
    xx = x.clone()
    layer(xx, w, e, out=xx)
    assert torch.equal(xx, y)


@pytest.mark.parametrize("fmt", FMTS)
def test_codes_and_repack(fmt):
    announce(f"experts repack {fmt}")
    rng = np.random.default_rng(3)
    layer, other = Layer(fmt, 3, 128, 128), Layer(fmt, 3, 128, 128, seed=9)
    x, x64 = bf16(rng.standard_normal((20, 128)))
    w, e, w64, ids = choice(rng, 20, 3, 2)
    W = torch.from_numpy(other.wd[1].astype(np.float32)).to(DEV)
    if fmt == "fp8":
        s = fql.fp8_scale_from_amax(W.abs().max().item())
        layer.down.repack_(1, fql.quant_fp8_weight(W, s), s)
    else:
        quant = {"mxfp4": fql.quant_mxfp4_weight, "mxfp8": fql.quant_mxfp8_weight, "int8": fql.quant_int8_weight,
                 "fp8_block": fql.quant_fp8_block_weight}[fmt]
        layer.down.repack_(1, *quant(W))
    layer.wd[1] = experts_of(fmt, other.wd[1:2], SH)[1][0]
    check(layer(x, w, e), *layer.reference(x64, w64, ids), "repacked")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [3, 130])
def test_graph_and_streams(fmt, T):
    """Replays of a captured call beside eager ones, other choices each time; a call on another stream."""
    announce(f"experts graph {fmt} T={T}")
    rng = np.random.default_rng(4)
    layer = Layer(fmt, 4, 256, 128)
    x, _ = bf16(rng.standard_normal((T, 256)))
    w, e, _, _ = choice(rng, T, 4, 2)
    layer(x, w, e)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(x, w, e)
    for i in range(4):
        x.copy_(bf16(rng.standard_normal((T, 256)))[0])
        e.copy_(choice(rng, T, 4, 2)[1])
        if i == 3:
            e.fill_(-1)
        graph.replay()
        eager = layer(x, w, e)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            aside = layer(x, w, e)
        torch.cuda.synchronize()
        assert torch.equal(y, eager) and torch.equal(aside, eager)


def test_no_tokens_and_leading_dimensions():
    announce("experts shapes")
    layer = Layer("mxfp8", 4, 128, 128)
    rng = np.random.default_rng(5)
    x, _ = bf16(rng.standard_normal((6, 128)))
    w, e, _, _ = choice(rng, 6, 4, 2)
    assert layer(x[:0], w[:0], e[:0]).shape == (0, 128)
    y = layer(x.view(2, 3, 128), w.view(2, 3, 2), e.view(2, 3, 2))
    assert y.shape == (2, 3, 128) and torch.equal(y.view(6, 128), layer(x, w, e))
    one = layer(x[0], w[0], e[0])
    assert one.shape == (128,) and torch.equal(one, layer(x[:1], w[:1], e[:1])[0])


@pytest.mark.parametrize("fmt", ("fp8_block", "mxfp8", "int8"))
@pytest.mark.parametrize("T", [1, 33])
def test_decoder_feed_forward(fmt, T):
    """The operators as a layer runs them: INT8 or dense projection, router, experts, residual stream."""
    announce(f"feed forward {fmt} T={T}")
    rng = np.random.default_rng([T, 6])
    E, k, H, I = 8, 2, 256, 128
    layer = Layer(fmt, E, H, I)
    dense = fql.INT8Weight.from_float(torch.from_numpy(rng.standard_normal((H, H)).astype(np.float32) * H ** -0.5).to(DEV))
    router = bf16(rng.standard_normal((E, H)) * H ** -0.5)[0]
    norm, _ = bf16(np.ones(H))
    h0, _ = bf16(rng.standard_normal((T, H)))
    bias = torch.from_numpy((0.1 * rng.standard_normal(E)).astype(np.float32)).to(DEV)

    def step(h0):
        a, _ = fql.rms_norm_operand(h0, norm, "int8")
        x = fql.linear_fused(a, dense, activation="silu")
        logits = x @ router.t().contiguous()
        w, e = fql.route_experts(logits, k, score="sigmoid", bias=bias, groups=4, top_groups=2, scale=2.0)
        return x, logits, w, e, fql.experts_fused(x, layer.up, layer.down, w, e, residual=h0)

    x, logits, w, e, y = step(h0)
    w64, ids = O.route(f64(logits), k, score="sigmoid", bias=f64(bias), groups=4, top_groups=2, scale=2.0)
    assert np.array_equal(e.cpu().numpy(), ids)
    check(y, *layer.reference(f64(x), f64(w), ids, f64(h0)), "feed forward")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gy = step(h0)[-1]
    for _ in range(3):
        h0.copy_(bf16(rng.standard_normal((T, H)))[0])
        graph.replay()
        eager = step(h0)[-1]
        torch.cuda.synchronize()
        assert torch.equal(gy, eager)


@pytest.mark.parametrize("T", [1, 19, 40, 6000])
def test_int8_scales_of_any_size_beside_one_another(T):
    """A row's scale times a channel's below or above float32's range where the product with the sum is not:
    single tokens, and tiles of every kind, in both products."""
    H, I, Ho = 1024, 2048, 64
    announce(f"experts int8 scales T={T} {fql.experts_fused_plan('int8', T, 1, 1, H, I, Ho, 'none')}")

    def pack(codes, scale):
        sw = torch.full((1, codes.shape[0]), 1.4 * 2.0 ** scale, dtype=torch.float32)
        return fql.ExpertWeight.from_codes("int8", torch.from_numpy(codes[None].astype(np.int8)).to(DEV), sw.to(DEV))

    rng = np.random.default_rng(T)
    uc = rng.integers(90, 128, (I, H))
    dc = rng.integers(90, 128, (Ho, I))
    dc[3::4] = 0
    w, e = torch.ones((T, 1), device=DEV), torch.zeros((T, 1), dtype=torch.int32, device=DEV)
    q = rng.integers(64, 128, (T, H))
    q[:, 0] = 127
    for a, b, c in ((-98, -48, 30), (-40, -60, -67), (121, 8, -60), (100, -20, 60), (0, 0, 0)):
        x, x64 = bf16(np.ldexp(q.astype(np.float64), a))
        assert np.array_equal(x64, np.ldexp(q.astype(np.float64), a))
        y = f64(fql.experts_fused(x, pack(uc, b), pack(dc, c), w, e, activation="none"))
        s = float(np.float32(1.4))
        h = np.ldexp(q.astype(np.float64) @ uc.T * s, a + b)
        past = (h > 3.4e38).any(1)
        assert not past.any() or past.all()
        # counted: h's roundings (2^-22) move its scale by as much, and rare codes by a step, of I * 64 steps a sum
        # and more; an fp16 rounding of a row (2^-11); y's own rounding
        hq, hs = O.quant_int8(np.minimum(h, 3.4e38).astype(np.float32))
        want = np.ldexp(hq.astype(np.float64) @ dc.T * (hs.astype(np.float64)[:, None] * s), c)
        if past.all():
            assert np.isnan(y).all()  # an inner activation beyond float32: the row's scale is NaN
            continue
        assert (y[:, 3::4] == 0).all(), (a, b, c)
        over = want > 3.41e38
        assert over[:, 0].all() == over.any() == (c == 60) and np.isposinf(y[over]).all()
        y, want = np.where(over, 0.0, y), np.where(over, 0.0, want)
        assert (np.abs(y - want) <= (HALF_BF16 + 2.0 ** -11 + 2.0 ** -16) * want).all(), (a, b, c)


def parts_of(plan):
    return int(plan.rsplit("tokens=", 1)[1])


# (format, T, k, E, H, I, Ho): tiles with the inner activation quantized in registers; INT8 on large tiles, whose
# inner activation is float32; 16-row tiles of both, whose second product's rows are float32 too
PASSES = [("mxfp8", 2100, 8, 8, 128, 14336, 160), ("fp8_block", 2100, 8, 8, 128, 14336, 256),
          ("int8", 2100, 8, 8, 128, 14336, 160), ("mxfp8", 130, 64, 1024, 32, 32768, 48),
          ("int8", 130, 64, 400, 32, 32768, 48)]


@pytest.mark.parametrize("fmt,T,k,E,H,I,Ho", PASSES)
def test_every_workspace_layout_over_passes(fmt, T, k, E, H, I, Ho):
    """More tokens than a pass takes, with rows of x, residual and out at strides of their own."""
    plan = fql.experts_fused_plan(fmt, T, k, E, H, I, Ho, "relu")
    announce(f"experts passes {fmt} T={T} {plan}")
    first = parts_of(plan)
    assert 0 < first < T and ("16x128" in plan) == (E >= 400)
    rng = np.random.default_rng([T, E])
    D = 3  # different experts; expert e has the weights of e % D
    layer = Layer(fmt, D, H, I, Ho=Ho, act="relu")
    at = torch.arange(E, device=DEV) % D
    for name in ("up", "down"):
        g = getattr(layer, name)
        setattr(layer, name, fql.ExpertWeight(fmt, g.packed[at].contiguous(), g.N, g.K))
    x, x64 = strided(rng.standard_normal((T, H)), H + 3, 1)
    r, r64 = strided(rng.standard_normal((T, Ho)), Ho + 5, 3)
    w, e, w64, ids = choice(rng, T, E, k)
    flat = torch.full((2 + T * (Ho + 9) + 8,), -7.0, dtype=torch.bfloat16, device=DEV)
    out = torch.as_strided(flat, (T, Ho), (Ho + 9, 1), 2)
    layer(x, w, e, residual=r, out=out)
    rows = np.unique(np.concatenate([[0, first - 1, first, min(2 * first, T - 1), T - 1], rng.integers(0, T, 12)]))
    check(out[torch.from_numpy(rows).to(DEV)], *layer.reference(x64[rows], w64[rows], ids[rows] % D, r64[rows]), "passes")
    gaps = flat.clone()
    torch.as_strided(gaps, (T, Ho), (Ho + 9, 1), 2).fill_(-7.0)
    assert (gaps == -7.0).all()


# the forms of the two products: a few tokens, 16-row tiles, tiles of 64, 128 and 256 rows (test_tiles)
EXACT = [(3, 2, 16, 256, 384, 160), (30, 2, 16, 256, 384, 160), (6000, 2, 3, 384, 768, 640)] + TILES


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k,E,H,I,Ho", EXACT)
def test_whole_numbers_come_out_exactly(fmt, T, k, E, H, I, Ho):
    """Values that every format holds and sums of few bits: nothing is rounded before y, whose bits are those of
    the exact result. The inner activation picks elements of x; the second product's rows are whole numbers below
    2^11, which fp16 with a power of two holds and bf16 does not."""
    if fmt == "fp8_block":
        Ho = -(-Ho // 128) * 128
    announce(f"experts exact {fmt} T={T} {fql.experts_fused_plan(fmt, T, k, E, H, I, Ho, 'none')}")
    rng = np.random.default_rng([T, E, I])
    values = np.array([0, 1, 2, 3, 4, 6, -1, -2, -3, -4, -6])
    # a scale that is a quotient of a largest value is a power of two where that is 7 * 2^n (448 / 7 = 64), 127:
    # it stands in the first column of every 128 of x and of h, and in the second column of a weight, where x and
    # h are 0
    top = {"fp8": 4, "fp8_block": 7, "mxfp8": 4, "mxfp4": 4, "int8": 127}[fmt]
    setter = {"fp8": 7, "fp8_block": 7, "int8": 127}.get(fmt, 0)
    x = rng.choice(values, (T, H))
    x[:, 0::128], x[:, 1::128] = top, 0
    free = np.array([c for c in range(H) if c % 128 > 1])
    wu = np.zeros((E, I, H), dtype=np.float32)
    pick, sign = rng.choice(free, (E, I)), rng.choice([1, -1], (E, I))
    pick[:, 0::128], sign[:, 0::128] = 0, 1
    pick[:, 1::128] = 1
    np.put_along_axis(wu, pick[:, :, None], sign[:, :, None].astype(np.float32), 2)
    wd = np.zeros((E, Ho, I), dtype=np.float32)
    inner = np.array([c for c in range(I) if c % 128 > 1])
    cols = rng.choice(inner, (E, Ho, 40))
    np.put_along_axis(wd, cols, rng.choice(values, cols.shape).astype(np.float32), 2)
    if setter:
        wu[:, :, 1::128] = setter
        wd[:, :, 1::128] = setter
    one = dict(input_scale=1.0) if fmt == "fp8" else {}
    up, down = (fql.ExpertWeight.from_float(torch.from_numpy(v).to(DEV), fmt, **one) for v in (wu, wd))
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    weights = rng.choice([1.0, -1.0, 0.5], (T, k)).astype(np.float32)
    want = np.zeros((T, Ho))
    for ex in range(E):
        t, j = np.nonzero(ids == ex)
        h = x[t][:, pick[ex]] * sign[ex]
        d = h.astype(np.float64) @ wd[ex].T
        assert np.abs(d).max(initial=0) < 2 ** 11
        np.add.at(want, t, weights[t, j][:, None] * d)
    y = fql.experts_fused(bf16(x)[0], up, down, torch.from_numpy(weights).to(DEV), torch.from_numpy(ids).to(DEV),
                          activation="none")
    want = torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16)
    bad = (y.cpu() != want).nonzero()
    assert bad.numel() == 0, (bad.shape[0], bad[:4].tolist())


USUAL = [(1, 8, 64, 2048, 1024), (100, 4, 16, 1024, 512), (1000, 2, 4, 512, 2048)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k,E,H,I", USUAL)
def test_usual_error(fmt, T, k, E, H, I):
    """The norm of the error of all outputs, of normally distributed inputs. The output's bf16 rounding is 2^-8 at
    most and 0.0017 of the norm on average; codes of h that the FP8 matrix instruction's internal sums move to a
    neighbour bring the largest of measured cases to 0.0021. Twice that is allowed: an inner activation in bf16
    alone would double it."""
    announce(f"experts usual error {fmt} T={T}")
    rng = np.random.default_rng([T, E, 7])
    D = min(E, 4)
    layer = Layer(fmt, D, H, I)
    at = torch.arange(E, device=DEV) % D
    for name in ("up", "down"):
        g = getattr(layer, name)
        args = dict(input_scale=g.input_scale, alpha=g.alpha[at].contiguous()) if fmt == "fp8" else {}
        setattr(layer, name, fql.ExpertWeight(fmt, g.packed[at].contiguous(), g.N, g.K, **args))
    x, x64 = bf16(rng.standard_normal((T, H)))
    w, e, w64, ids = choice(rng, T, E, k)
    ref, _ = layer.reference(x64, w64, ids % D)
    d = np.linalg.norm(f64(layer(x, w, e)) - ref) / np.linalg.norm(ref)
    print(f"usual error {fmt} T={T}: {d:.5f}", flush=True)
    assert d <= 0.0042
