"""Mixture of experts: the routing of tokens to experts and the chosen experts' feed forward.

    route_experts     scores, groups, top-k and weights from a router's logits

Like the rest of the binding this module only marshals arguments; every step
runs in the library's HIP kernels (include/fql.h has the formulas).

    w, e = route_experts(logits, 8)                               # logits [tokens, experts]
"""

import torch

from . import FQLError, _check, _rows_view, lib
from .serving import _f32, _new, _same_device, _stream, _within

_TYPES = {torch.bfloat16: 1, torch.float32: 2}  # FQL_TYPE_BF16, FQL_TYPE_F32
SCORES = {"softmax": 1, "sigmoid": 2}
_I32_MAX = 2 ** 31 - 1


def route_experts(logits, top_k, score="softmax", bias=None, groups=1, top_groups=None, renormalize=True, scale=1.0):
    """The top_k experts of each token and their weights: (weights float32 [..., top_k], experts int32
    [..., top_k], best first).

    logits: bf16 or float32 [..., E], any row stride. score: "softmax" or "sigmoid". bias: float32 [E], added
    to the scores for the choice alone. groups, top_groups: only experts of the best top_groups of `groups`
    groups of neighbours can be chosen. renormalize: the weights sum to 1; scale: a factor on them. An expert
    whose logit is NaN or -inf is not available (nor one whose bias is); places that no expert fills get
    expert -1 and weight 0. Ties go to the lowest index."""
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda:
        raise FQLError("logits must be a CUDA (HIP) tensor")
    kind = _TYPES.get(logits.dtype)
    if kind is None:
        raise FQLError("logits must be bfloat16 or float32")
    how = SCORES.get(score)
    if how is None:
        raise FQLError(f"unknown score {score!r} (one of {', '.join(SCORES)})")
    x, ld = _rows_view(logits, "logits")
    T, E = x.shape
    index = logits.get_device()
    bp = 0
    if bias is not None:
        if not isinstance(bias, torch.Tensor) or not bias.is_cuda or bias.dtype is not _f32:
            raise FQLError("bias must be a float32 CUDA (HIP) tensor")
        _same_device(bias, "bias", index, "logits")
        if bias.shape != (E,) or not bias.is_contiguous():
            raise FQLError(f"bias must be a contiguous tensor of {E} elements")
        bp = bias.data_ptr()
    k = _within(top_k, "top_k", 1, _I32_MAX)
    groups = _within(groups, "groups", 1, _I32_MAX)
    top_groups = groups if top_groups is None else _within(top_groups, "top_groups", 1, _I32_MAX)
    shape = logits.shape[:-1] + (k,)
    dev = logits.device
    weights, experts = _new(shape, _f32, dev), _new(shape, torch.int32, dev)
    _check(lib().fql_route_experts(kind, x.data_ptr(), T, E, ld, how, bp, groups, top_groups, k, bool(renormalize),
                                   scale, weights.data_ptr(), experts.data_ptr(), _stream(index)))
    return weights, experts
