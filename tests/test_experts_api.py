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
