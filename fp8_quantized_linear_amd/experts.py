"""Mixture of experts: the routing of tokens to experts and the chosen experts' feed forward.

    route_experts     scores, groups, top-k and weights from a router's logits
    ExpertWeight      the packed weights of all experts' one projection
    experts_fused     both projections of every token's experts, weighted and added

Like the rest of the binding this module only marshals arguments; every step
runs in the library's HIP kernels (include/fql.h has the formulas).

The feed forward of a decoder layer, all tensors on the GPU (x: the normed hidden states, h: the residual
stream):

    w, e = route_experts(x @ router.T, 8)                         # logits [tokens, experts]
    h = experts_fused(x, up, down, w, e, residual=h)

with up = ExpertWeight.from_float(gate and up projections [E, 2 I, H], interleaved, "mxfp8") and
down = ExpertWeight.from_float([E, H, I], "mxfp8").
"""

import ctypes
import struct

import torch

from . import (FQLError, _CODES, _SCALES, _check, _one_of, _pack_sc, _rows_view, _size_query, fp8_output_scale,
               fp8_scale_from_amax, lib)
from . import quant_fp8_block_weight, quant_fp8_weight, quant_int8_weight, quant_mxfp4_weight, quant_mxfp8_weight
from .serving import (ACTIVATIONS, FORMATS, _bf16, _cuda, _f32, _format, _i32, _new, _query, _rows, _same_device, _stream,
                      _u8, _within, _workspace)

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


# ---------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------

_QUANT = {"mxfp4": quant_mxfp4_weight, "mxfp8": quant_mxfp8_weight, "fp8_block": quant_fp8_block_weight,
          "int8": quant_int8_weight}


class ExpertWeight:
    """The packed weights [N, K] of E experts' one projection, in one format.

    packed: uint8 [E, bytes]; alpha: float32 [E] of per-tensor FP8, input_scale * weight_scale of each expert
    (None otherwise); input_scale: per-tensor FP8's static scale of the projection's input.
    """

    def __init__(self, fmt, packed, N, K, input_scale=None, alpha=None):
        _format(fmt)
        self.fmt, self.N, self.K = fmt, int(N), int(K)
        _cuda(packed, "packed", _u8)
        if packed.dim() != 2 or packed.shape[0] < 1 or not packed.is_contiguous():
            raise FQLError("packed must be a contiguous tensor [E, bytes]")
        self.packed, self.E = packed, packed.shape[0]
        if fmt == "fp8":
            if input_scale is None or alpha is None:
                raise FQLError("per-tensor FP8 needs its input_scale and alpha")
            _cuda(alpha, "alpha", _f32)
            _same_device(alpha, "alpha", packed.get_device(), "packed")
            if alpha.shape != (self.E,) or not alpha.is_contiguous():
                raise FQLError("alpha must be float32 [E]")
            input_scale = ctypes.c_float(float(input_scale)).value
        elif input_scale is not None or alpha is not None:
            raise FQLError("input_scale and alpha belong to per-tensor FP8")
        self.input_scale, self.alpha = input_scale, alpha
        need = _size_query(f"fql_packed_{fmt}_bytes", self.N, self.K)
        if packed.shape[1] < need or packed.shape[1] % 16 != 0:
            raise FQLError(f"an expert's packed weight has {need} bytes, and rows of packed a multiple of 16")

    @classmethod
    def from_codes(cls, fmt, codes, scales, input_scale=None):
        """From canonical codes [E, N, K] (MXFP4: [E, N, K/2]) and the format's scales of each expert, stacked
        (per-tensor FP8: the weight scales, float32 [E])."""
        _format(fmt)
        if not isinstance(codes, torch.Tensor) or not codes.is_cuda or codes.dim() != 3 or codes.shape[0] < 1:
            raise FQLError("codes must be a CUDA (HIP) tensor [E, N, K]")
        _one_of(codes, "codes", _CODES[fmt], fmt)
        if fmt != "fp8":
            _one_of(scales, "scales", _SCALES[fmt], fmt)
        E, N, K = codes.shape
        K *= 2 if fmt == "mxfp4" else 1
        if not isinstance(scales, torch.Tensor) or scales.shape[:1] != (E,) or scales.device != codes.device:
            raise FQLError("scales must be the experts' scales, stacked, on the codes' device")
        size = -(-_size_query(f"fql_packed_{fmt}_bytes", N, K) // 256) * 256
        packed = torch.empty((E, size), dtype=_u8, device=codes.device)
        for e in range(E):
            _pack_sc(fmt, codes[e], None if fmt == "fp8" else scales[e], packed[e])
        alpha = None
        if fmt == "fp8":
            if input_scale is None:
                raise FQLError("per-tensor FP8 needs its input_scale")
            alpha = torch.tensor([fp8_output_scale(input_scale, s) for s in scales.tolist()], dtype=_f32,
                                 device=codes.device)
        return cls(fmt, packed, N, K, input_scale, alpha)

    @classmethod
    def from_float(cls, w, fmt, input_scale=None):
        """From float32 weights [E, N, K]."""
        _format(fmt)
        if not isinstance(w, torch.Tensor) or w.dim() != 3 or w.shape[0] < 1:
            raise FQLError("w must be a tensor [E, N, K]")
        if fmt == "fp8":
            scales = [fp8_scale_from_amax(m) for m in w.abs().amax((1, 2)).tolist()]
            codes = [quant_fp8_weight(w[e], s) for e, s in enumerate(scales)]
            return cls.from_codes(fmt, torch.stack(codes), torch.tensor(scales, dtype=_f32, device=w.device), input_scale)
        both = [_QUANT[fmt](w[e]) for e in range(w.shape[0])]
        return cls.from_codes(fmt, torch.stack([c for c, _ in both]), torch.stack([s for _, s in both]), input_scale)

    def repack_(self, expert, codes, scales):
        """New canonical weights of one expert into the same storage (per-tensor FP8: scales is its weight scale)."""
        expert = _within(expert, "expert", 0, self.E - 1)
        K = codes.shape[-1] * (2 if self.fmt == "mxfp4" else 1)
        if codes.dim() != 2 or (codes.shape[0], K) != (self.N, self.K):
            raise FQLError(f"codes must be an expert's [{self.N}, {self.K}]")
        _pack_sc(self.fmt, codes, None if self.fmt == "fp8" else scales, self.packed[expert])
        if self.fmt == "fp8":
            self.alpha[expert].fill_(fp8_output_scale(self.input_scale, float(scales)))
        return self


def _expert_struct(w, bias, name, index):
    """A packed fql_expert_weight."""
    if w.packed.get_device() != index:
        _same_device(w.packed, name, index)
    bp = 0
    if bias is not None:
        _cuda(bias, f"bias of {name}", _bf16)
        _same_device(bias, f"bias of {name}", index)
        if bias.shape != (w.E, w.N) or not bias.is_contiguous():
            raise FQLError(f"bias of {name} must be a contiguous bf16 tensor [{w.E}, {w.N}]")
        bp = bias.data_ptr()
    return struct.pack("PqqqPPf4x", w.packed.data_ptr(), w.packed.shape[1], w.N, w.K,
                       0 if w.alpha is None else w.alpha.data_ptr(), bp, w.input_scale or 0.0)


def experts_fused_plan(fmt, tokens, top_k, experts, hidden, up_columns, out_columns, activation="swiglu"):
    """One-line description of the launch plan of an experts_fused call."""
    buf = ctypes.create_string_buffer(256)
    _check(lib().fql_experts_describe(_format(fmt), int(tokens), int(top_k), int(experts), int(hidden), int(up_columns),
                                      int(out_columns), ACTIVATIONS[activation], buf, 256))
    return buf.value.decode()


def experts_fused(x, up, down, weights, experts, activation="swiglu", bias_up=None, bias_down=None, residual=None,
                  out=None, workspace=None):
    """y = bf16(residual + sum_j weights[:, j] * down_e(act(up_e(x)))), e = experts[:, j].

    x: bf16 [..., H]. up, down: ExpertWeight of one format, [N, H] and [Ho, I] (I = N; "swiglu", whose rows are
    interleaved by interleave_gate_up: N / 2). weights float32 [..., k], experts int32 [..., k] as route_experts
    gives them; a place whose expert is not in 0 .. E - 1 adds nothing. bias_up, bias_down: bf16 [E, N].
    residual: bf16 [..., Ho]. out may be residual or x itself. The inner activation is quantized from float32."""
    if activation not in ACTIVATIONS:
        raise FQLError(f"unknown activation {activation!r}")
    if not isinstance(up, ExpertWeight) or not isinstance(down, ExpertWeight):
        raise FQLError("up and down must be ExpertWeight")
    if up.fmt != down.fmt or up.E != down.E:
        raise FQLError(f"up is {up.fmt} of {up.E} experts, down {down.fmt} of {down.E}")
    xp, T, H, ld = _rows(x, "x")
    if H != up.K:
        raise FQLError(f"x has K={H}, up has K={up.K}")
    dev = x.device
    index = dev.index
    lead = x.shape[:-1]
    k = weights.shape[-1] if isinstance(weights, torch.Tensor) and weights.dim() else 0
    for t, name, dtype in ((weights, "weights", _f32), (experts, "experts", _i32)):
        if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index:
            _cuda(t, name, dtype)
            _same_device(t, name, index)
        if t.shape != lead + (k,) or not t.is_contiguous():
            raise FQLError(f"{name} must be contiguous with shape {tuple(lead) + ('k',)}")
    shape = lead + (down.N,)
    rp = ldr = 0
    if residual is not None:
        rp, _, _, ldr = _rows(residual, "residual", shape, index)
    if out is None:
        out = _new(shape, _bf16, dev)
        yp, ldy = out.data_ptr(), down.N
    else:
        yp, _, _, ldy = _rows(out, "out", shape, index)
    f, act = FORMATS[up.fmt], ACTIVATIONS[activation]
    u, d = _expert_struct(up, bias_up, "up", index), _expert_struct(down, bias_down, "down", index)
    need = _query("fql_experts_workspace_bytes", f, T, k, up.E, H, up.N, down.N, act)
    wp = size = 0
    if workspace is not None:
        _same_device(workspace, "workspace", index)
        wp, size = workspace.data_ptr(), workspace.numel()
    elif T > 0:
        workspace = _workspace(dev, need)
        wp, size = workspace.data_ptr(), workspace.numel()
    _check(lib().fql_experts_fused(f, xp, T, ld, u, d, up.E, act, weights.data_ptr(), experts.data_ptr(), k, rp, ldr, yp,
                                   ldy, wp, size, _stream(index)))
    return out
