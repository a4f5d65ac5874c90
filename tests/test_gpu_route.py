"""Routing to experts on the GPU against float64: choices equal, weights within one float32 rounding."""

import numpy as np
import pytest
import torch

import fp8_quantized_linear_amd as fql
from oracle import feedforward as O
from gpu_helpers import announce
from serving_helpers import DEV, f64

pytestmark = pytest.mark.gpu


def check(logits, k, what, **args):
    """Weights: a float64 evaluation (under 2^-40 of the weight) rounded to float32 once, half a step 2^-24."""
    bias = args.get("bias")
    dev = {**args, "bias": None if bias is None else torch.from_numpy(bias).to(DEV)}
    w, e = fql.route_experts(logits, k, **dev)
    assert w.dtype == torch.float32 and e.dtype == torch.int32 and w.shape == e.shape == logits.shape[:-1] + (k,)
    z = f64(logits).reshape(-1, logits.shape[-1])
    G = args.get("groups", 1)
    ww, we = O.route(z, k, **{**args, "top_groups": args.get("top_groups", G)})
    got, ids = f64(w).reshape(-1, k), e.cpu().numpy().reshape(-1, k)
    assert np.array_equal(ids, we), (what, np.argwhere(ids != we)[:4])
    assert (np.abs(got - ww) <= (2.0 ** -24 + 2.0 ** -40) * np.abs(ww) + 2.0 ** -149).all(), what
    return got, ids


def logits(rng, T, E, dtype, std=1.5):
    return torch.from_numpy((rng.standard_normal((T, E)) * std).astype(np.float32)).to(dtype).to(DEV)


SIZES = [(1, 1, 1), (1, 64, 6), (3, 8, 2), (7, 60, 4), (5, 65, 64), (33, 128, 8), (4, 160, 6), (9, 256, 8), (2, 384, 10),
         (3, 512, 33), (2, 1000, 8), (2, 1024, 64), (130, 16, 16)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_choices_and_weights(T, E, k, score):
    announce(f"route {T}x{E} k={k} {score}")
    rng = np.random.default_rng([T, E, k])
    for dtype in (torch.bfloat16, torch.float32):
        x = logits(rng, T, E, dtype)
        bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
        check(x, k, "plain", score=score)
        check(x, k, "raw", score=score, renormalize=False, scale=-1.5)
        check(x, k, "bias", score=score, bias=bias, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G", [(8, 2), (64, 64), (60, 5), (256, 8), (160, 4), (512, 2), (1024, 64), (9, 3), (128, 33 - 1)])
def test_groups(E, G, score):
    announce(f"route groups {E}/{G} {score}")
    rng = np.random.default_rng([E, G])
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    for top in sorted({1, (G + 1) // 2, G - 1, G}):
        k = min(8, top * (E // G))
        for dtype in (torch.bfloat16, torch.float32):
            x = logits(rng, 11, E, dtype)
            check(x, k, "groups", score=score, groups=G, top_groups=top)
            check(x, k, "groups bias", score=score, groups=G, top_groups=top, bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [6, 64, 200, 777])
def test_ties_go_to_the_lowest_index(E, score):
    announce(f"route ties {E} {score}")
    rng = np.random.default_rng(E)
    x = torch.from_numpy(rng.integers(-1, 2, (40, E)).astype(np.float32)).to(DEV)
    x[0] = 0.5
    x[1] = torch.where(torch.arange(E, device=DEV) % 2 == 0, 0.0, -0.0)
    for dtype in (torch.bfloat16, torch.float32):
        check(x.to(dtype), min(E, 6), "ties", score=score)
        check(x.to(dtype), min(E, 6), "ties", score=score, bias=np.zeros(E, dtype=np.float32))
        if E % 4 == 0:
            check(x.to(dtype), 3, "ties", score=score, groups=4, top_groups=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_unavailable_experts(score):
    """NaN, infinities, rows with too few experts and with none, scores that underflow."""
    announce(f"route masks {score}")
    E, k, inf, nan = 70, 5, np.inf, np.nan
    x = np.random.default_rng(3).standard_normal((12, E)).astype(np.float32)
    x[0] = -inf
    x[1] = nan
    x[2], x[2, 68] = -inf, 0.25
    x[3, ::2] = -inf
    x[4, 3:] = nan
    x[5, 40] = inf
    x[6, [5, 66]] = inf
    x[7] = np.finfo(np.float32).min
    x[8], x[8, 9] = -3e38, 3e38
    x[9] = -800.0
    x[10, :] = -90.0
    x[11, 0:69] = -inf
    t = torch.from_numpy(x).to(DEV)
    for dtype in (torch.bfloat16, torch.float32):
        for renorm in (True, False):
            w, e = check(t.to(dtype), k, "masks", score=score, renormalize=renorm)
            assert (e[:2] == -1).all() and (w[:2] == 0).all()
            assert e[2].tolist() == [68, -1, -1, -1, -1]
            check(t.to(dtype), k, "masks", score=score, renormalize=renorm, groups=7, top_groups=2)
            bias = np.zeros(E, dtype=np.float32)
            bias[:4], bias[4:6], bias[60:62] = -inf, nan, inf
            check(t.to(dtype), k, "masks bias", score=score, renormalize=renorm, bias=bias)
            check(t.to(dtype), k, "masks bias", score=score, renormalize=renorm, bias=bias, groups=7, top_groups=2)


def test_strides_shapes_and_no_rows():
    announce("route strides")
    rng = np.random.default_rng(5)
    x = logits(rng, 24, 100, torch.bfloat16)
    check(x[:, 3:67], 4, "columns")
    check(x[::2, :64], 4, "every other row")
    check(x.view(2, 3, 4, 100), 4, "leading dimensions")
    check(x[0], 4, "one row")
    w, e = fql.route_experts(x[:0], 4)
    assert w.shape == e.shape == (0, 4)


def test_many_tokens_streams_and_graph():
    announce("route many")
    rng = np.random.default_rng(6)
    x = logits(rng, 5000, 256, torch.float32)
    bias = torch.from_numpy((0.05 * rng.standard_normal(256)).astype(np.float32)).to(DEV)
    args = dict(score="sigmoid", bias=bias, groups=8, top_groups=4, scale=2.5)
    w, e = fql.route_experts(x, 8, **args)
    rows = rng.integers(0, 5000, 60)
    ww, we = O.route(f64(x)[rows], 8, **{**args, "bias": f64(bias)})
    assert np.array_equal(e.cpu().numpy()[rows], we)
    assert (np.abs(f64(w)[rows] - ww) <= (2.0 ** -24 + 2.0 ** -40) * ww).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gw, ge = fql.route_experts(x, 8, **args)
    for _ in range(3):
        x.copy_(logits(rng, 5000, 256, torch.float32))
        graph.replay()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            w, e = fql.route_experts(x, 8, **args)
        torch.cuda.synchronize()
        assert torch.equal(gw, w) and torch.equal(ge, e)
