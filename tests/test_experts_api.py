"""Refusals and sizes of the mixture of experts (CPU): every call here fails validation before any launch, or
only plans."""

import ctypes

import numpy as np
import pytest
import torch

import fp8_quantized_linear_amd as fql
from oracle import feedforward as O

P, NULL = ctypes.c_void_p(1 << 20), ctypes.c_void_p(0)


def refused(status, *words, code=-1):
    msg = fql.lib().fql_last_error().decode()
    assert status == code, (status, msg)
    assert all(w in msg for w in words), msg


def route(kind=1, x=P, T=4, E=64, ld=64, score=1, bias=NULL, groups=1, top=1, k=4, scale=1.0, w=P, e=P):
    return fql.lib().fql_route_experts(kind, x, T, E, ld, score, bias, groups, top, k, 1, scale, w, e, NULL)


def test_route_refusals():
    refused(route(kind=0), "bf16", code=-2)
    refused(route(score=3), "score")
    refused(route(T=-1), "T")
    refused(route(T=(1 << 30) + 1), "T")
    refused(route(T=(1 << 24) + 1), "T")
    refused(route(E=0), "experts", code=-2)
    refused(route(E=1025, ld=1025), "1024", code=-2)
    refused(route(ld=63), "stride")
    refused(route(groups=3), "groups")
    refused(route(groups=0), "groups")
    refused(route(E=128, ld=128, groups=128), "groups")
    refused(route(groups=4, top=5), "top_groups")
    refused(route(groups=4, top=0), "top_groups")
    refused(route(groups=8, top=1, k=9), "k must")
    refused(route(k=0), "k must")
    refused(route(E=128, ld=128, k=65), "64")
    refused(route(scale=float("inf")), "scale")
    refused(route(x=NULL), "null")
    refused(route(w=NULL), "null")
    refused(route(e=NULL), "null")
    refused(route(kind=2, x=ctypes.c_void_p((1 << 20) + 2)), "aligned")
    refused(route(bias=ctypes.c_void_p((1 << 20) + 2)), "aligned")
    assert route(T=0, x=NULL, w=NULL, e=NULL) == 0


def test_binding_refusals_without_a_gpu():
    with pytest.raises(fql.FQLError, match="CUDA"):
        fql.route_experts(torch.zeros(4, 8), 2)


def test_oracle_route():
    z = np.array([[0.0, 2.0, 1.0, 2.0], [-np.inf, np.nan, 1.0, -np.inf], [np.nan] * 4, [5.0, 4.0, 4.9, 4.8]])
    w, e = O.route(z, 2)
    assert e.tolist() == [[1, 3], [2, -1], [-1, -1], [0, 2]]
    assert w[:2].tolist() == [[0.5, 0.5], [1.0, 0.0]] and w[2].tolist() == [0, 0]
    w, e = O.route(z[3:], 2, score="sigmoid", renormalize=False, bias=np.array([-9.0, 0, 0, 0]), scale=2.0)
    assert e.tolist() == [[2, 3]] and np.allclose(w, 2 / (1 + np.exp(-z[3:, [2, 3]])))


class Weight(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("stride", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("alpha", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("input_scale", ctypes.c_float)]


FP8, BLOCK, MXFP8, MXFP4, INT8, NVFP4 = (fql.FMT_FP8, fql.FMT_FP8_BLOCK, fql.FMT_MXFP8, fql.FMT_MXFP4, fql.FMT_INT8,
                                         fql.FMT_NVFP4)


def experts(fmt=MXFP8, x=1 << 20, T=4, H=256, ldx=None, N=512, I=256, Ho=256, E=8, act=5, k=2, w=P, e=P, res=0, ldr=256,
            y=1 << 24, ldy=None, ws=P, size=1 << 40, up={}, down={}):
    u = Weight(**{**dict(packed=1 << 20, stride=1 << 30, N=N, K=H, input_scale=0.1), **up})
    d = Weight(**{**dict(packed=1 << 20, stride=1 << 30, N=Ho, K=I, input_scale=0.1), **down})
    return fql.lib().fql_experts_fused(fmt, ctypes.c_void_p(x), T, H if ldx is None else ldx, ctypes.byref(u),
                                       ctypes.byref(d), E, act, w, e, k, ctypes.c_void_p(res), ldr, ctypes.c_void_p(y),
                                       Ho if ldy is None else ldy, ws, size, NULL)


def test_experts_refusals():
    refused(experts(fmt=NVFP4), "format", code=-2)
    refused(experts(act=6), "activation")
    refused(experts(E=0), "experts", code=-2)
    refused(experts(E=1025), "1024", code=-2)
    refused(experts(k=0), "k must")
    refused(experts(k=65), "64")
    refused(experts(T=-1), "T must")
    refused(experts(T=(1 << 24) + 1), "T must")
    refused(experts(H=40), "32")
    refused(experts(fmt=BLOCK, N=640), "128")
    refused(experts(fmt=BLOCK, H=160), "128")
    refused(experts(N=48, I=24), "32")
    refused(experts(N=528, I=264), "multiple of 32")
    refused(experts(I=512), "down")
    refused(experts(act=0, I=256), "down")
    refused(experts(N=1 << 19, I=1 << 18), "2^18")
    refused(experts(fmt=INT8, act=0, H=1 << 18, Ho=64, I=512), "131072")
    refused(experts(ldx=255), "stride")
    refused(experts(ldy=255), "ldy")
    refused(experts(res=1 << 22, ldr=255), "residual")
    refused(experts(x=0), "null")
    refused(experts(w=NULL), "null")
    refused(experts(e=NULL), "null")
    refused(experts(y=0), "null")
    refused(experts(ws=NULL), "null")
    refused(experts(up=dict(packed=0)), "null")
    refused(experts(up=dict(packed=(1 << 20) + 8)), "up", "16-byte")
    refused(experts(down=dict(stride=256 * 256 + 8)), "down", "16-byte")
    refused(experts(down=dict(stride=256 * 256)), "down", "smaller")
    refused(experts(up=dict(alpha=(1 << 20) + 2)), "aligned")
    refused(experts(down=dict(bias=(1 << 20) + 1)), "aligned")
    refused(experts(fmt=FP8, up=dict(input_scale=0.0)), "input_scale")
    refused(experts(fmt=FP8, down=dict(input_scale=float("nan"))), "input_scale")
    refused(experts(ws=ctypes.c_void_p((1 << 20) + 16)), "256")
    refused(experts(size=1 << 10), "workspace", code=-4)
    refused(experts(y=(1 << 20) + 512), "overlaps")             # x one row on
    refused(experts(Ho=128, y=1 << 20), "overlaps")             # another width over x
    refused(experts(res=(1 << 24) + 2), "overlaps")
    assert experts(T=0, x=0, w=NULL, e=NULL, y=0, ws=NULL, size=0) == 0


def test_experts_sizes_and_plans():
    n = ctypes.c_size_t()
    for fmt, code in (("mxfp4", MXFP4), ("mxfp8", MXFP8), ("fp8", FP8), ("fp8_block", BLOCK), ("int8", INT8)):
        last = 0
        for T in (1, 16, 100, 1000, 4096, 100000, 1 << 24):
            args = (code, T, 8, 64, 4096, 2048, 4096, 5)
            assert fql.lib().fql_experts_workspace_bytes(*args, ctypes.byref(n)) == 0
            assert last <= n.value < 3 << 30  # tokens are taken in passes
            last = n.value
            assert "tokens=" in fql.experts_fused_plan(fmt, T, 8, 64, 4096, 2048, 4096)
    refused(fql.lib().fql_experts_workspace_bytes(NVFP4, 1, 1, 1, 64, 64, 64, 0, ctypes.byref(n)), "format", code=-2)
    refused(fql.lib().fql_experts_workspace_bytes(MXFP8, 1, 1, 1, 60, 64, 64, 0, ctypes.byref(n)), "32")


def test_experts_binding_refusals_without_a_gpu():
    with pytest.raises(fql.FQLError, match="ExpertWeight"):
        fql.experts_fused(None, None, None, None, None)
    with pytest.raises(fql.FQLError, match="activation"):
        fql.experts_fused(None, None, None, None, None, activation="tanh")
    with pytest.raises(fql.FQLError, match="unknown format"):
        fql.ExpertWeight.from_codes("nvfp4", None, None)
    with pytest.raises(fql.FQLError, match="CUDA"):
        fql.ExpertWeight("int8", torch.zeros(2, 4096, dtype=torch.uint8), 16, 128)
    with pytest.raises(fql.FQLError, match="CUDA"):
        fql.ExpertWeight.from_codes("mxfp8", torch.zeros(2, 16, 128), None)


def test_the_gpu_tests_reach_every_tile():
    import test_gpu_experts as G
    for fmt in G.FMTS:
        plans = [fql.experts_fused_plan(fmt, T, k, E, H, 2 * I, Ho) for T, k, E, H, I, Ho in G.TILES]
        plans += [fql.experts_fused_plan(fmt, T, k, E, H, 2 * I, H) for T, k, E, H, I in G.CASES]
        for product in ("up", "down"):
            of = [p.split(" down ")[product == "down"] for p in plans if " down " in p]
            for tile in ("16x128", "64x256", "128x256", "256x256"):
                assert any(f"tiles={tile}" in p for p in of), (fmt, product, tile)
        assert any("token" in p for p in plans)


@pytest.mark.parametrize("fmt", (MXFP4, MXFP8, FP8, BLOCK, INT8))
@pytest.mark.parametrize("k,E,H,N,Ho", [(8, 64, 4096, 2048, 4096), (2, 8, 4096, 28672, 4096), (4, 32, 2048, 2816, 2048),
                                        (1, 1, 128, 256, 128), (64, 1024, 256, 512, 384), (8, 128, 128, 256, 16384)])
def test_a_workspace_of_the_largest_batch_serves_every_smaller_one(fmt, k, E, H, N, Ho):
    n = ctypes.c_size_t()
    sizes = []
    batches = sorted({*range(1, 700), *(int(1.07 ** i) for i in range(246)), *(E * r // k + d for r in (8, 20)
                     for d in (-1, 0, 1)), 1 << 24})
    for T in (t for t in batches if 0 < t <= 1 << 24):
        assert fql.lib().fql_experts_workspace_bytes(fmt, T, k, E, H, N, Ho, 5, ctypes.byref(n)) == 0
        sizes.append((n.value, T))
    assert sizes == sorted(sizes), next((a, b) for a, b in zip(sizes, sizes[1:]) if a > b)
