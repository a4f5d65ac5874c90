"""8-bit serving operators: what stands between the 8-bit linear layers of a decoder.

    rms_norm_quant / rms_norm_operand   residual + root-mean-square norm + 8-bit output
    linear_fused                        linear layer with bias, activation, residual in its epilogue
    KVCache8, kv_append, attention_kv8  paged 8-bit cache, the write into it, attention over it

Like the rest of the binding this module only marshals arguments; every step
runs in the library's HIP kernels (include/fql.h has the formulas).

One layer of a decoder, all tensors on the GPU:

    xq, h = rms_norm_operand(y, w1, "mxfp8", residual=h)     # h: the residual stream
    qkv = linear_fused(xq, w_qkv)
    q, k, v = (t.unflatten(-1, (-1, 128)) for t in qkv.split([4096, 1024, 1024], -1))
    kv_append(cache, k, v, table, lens, cu, max_new)
    o = attention_kv8(q, cache, table, lens, cu, max_new)
    h = linear_fused(o.flatten(1), w_o, residual=h, out=h)
    xq, _ = rms_norm_operand(h, w2, "mxfp8")
    y = linear_fused(linear_fused(xq, w_gate_up, activation="swiglu"), w_down)
"""

import ctypes

import torch

from . import (FMT_FP8, FMT_FP8_BLOCK, FMT_MXFP4, FMT_MXFP8, FQLError, KvBatchStruct, KvCacheStruct,
               _check, _ptr, _require_cuda, _rows_view, _size_query, _stream, _workspace, lib,
               linear_sc_workspace_bytes)

FORMATS = {"mxfp4": FMT_MXFP4, "mxfp8": FMT_MXFP8, "fp8": FMT_FP8, "fp8_block": FMT_FP8_BLOCK}
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "swiglu": 5}


def _format(fmt):
    if fmt not in FORMATS:
        raise FQLError(f"unknown format {fmt!r} (one of {', '.join(FORMATS)})")
    return FORMATS[fmt]


def _bf16_rows(t, name, shape):
    _require_cuda(t, name)
    if t.dtype != torch.bfloat16 or tuple(t.shape) != tuple(shape):
        raise FQLError(f"{name} must be a bfloat16 tensor of shape {tuple(shape)}")
    return _rows_view(t, name)


def _scale_arg(fmt, scale):
    if fmt != "fp8":
        return 0
    if scale is None:
        raise FQLError("per-tensor FP8 needs its static scale")
    return ctypes.c_float(float(scale)).value


def _bf16_vector(t, name, n):
    _require_cuda(t, name)
    if t.dtype != torch.bfloat16 or t.numel() != n or not t.is_contiguous():
        raise FQLError(f"{name} must be a contiguous bf16 tensor of {n} elements")


# ---------------------------------------------------------------------------
# norm, operands
# ---------------------------------------------------------------------------

class QuantizedActivation:
    """A quantized activation [..., K] in the order the linear kernels read it.

    Made by rms_norm_operand or quant_operand, taken by linear_fused in place of
    the bf16 activation. data: the device buffer; fmt: its format; scale: the
    static scale it was quantized with (per-tensor FP8).
    """

    def __init__(self, data, fmt, lead, K, scale=None):
        self.data, self.fmt, self.scale = data, fmt, scale
        self.lead, self.K = tuple(lead), int(K)
        self.M = 1
        for n in self.lead:
            self.M *= n


def _new_operand(x, fmt, scale):
    K = x.shape[-1]
    lead = tuple(x.shape[:-1])
    q = QuantizedActivation(None, fmt, lead, K, scale if fmt == "fp8" else None)
    nbytes = _size_query("fql_operand_bytes", _format(fmt), q.M, K)
    q.data = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    return q


def _norm_args(x, weight, residual, residual_out):
    _require_cuda(x, "x")
    if x.dtype != torch.bfloat16:
        raise FQLError("x must be bfloat16")
    x2, ld = _rows_view(x, "x")
    _bf16_vector(weight, "weight", x.shape[-1])
    r2, ldr, h, h2, ldh = None, 0, None, None, 0
    if residual is not None:
        r2, ldr = _bf16_rows(residual, "residual", x.shape)
        h = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device) if residual_out is None else residual_out
        h2, ldh = _bf16_rows(h, "residual_out", x.shape)
    elif residual_out is not None:
        raise FQLError("residual_out needs a residual")
    return x2, ld, r2, ldr, h, h2, ldh


def rms_norm_quant(x, weight, fmt, eps=1e-6, residual=None, scale=None, residual_out=None):
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight, quantized to fmt ("fp8", "fp8_block"
    or "mxfp8"). x, residual bf16 [..., K], weight bf16 [K]; scale: per-tensor FP8's static scale.
    Returns (codes uint8 [..., K], scales as quant_<fmt> gives them or None, h bf16 or None without a
    residual). residual_out may be x or residual itself."""
    f = _format(fmt)
    x2, ld, r2, ldr, h, h2, ldh = _norm_args(x, weight, residual, residual_out)
    M, K = x2.shape
    lead = tuple(x.shape[:-1])
    codes = torch.empty(lead + (K,), dtype=torch.uint8, device=x.device)
    scales = None
    if fmt == "mxfp8":
        scales = torch.empty(lead + (K // 32,), dtype=torch.uint8, device=x.device)
    elif fmt == "fp8_block":
        scales = torch.empty(lead + (K // 128,), dtype=torch.float32, device=x.device)
    _check(lib().fql_rms_norm_quant(f, _ptr(x2), M, K, ld, _ptr(r2), ldr, _ptr(weight), float(eps),
                                    _scale_arg(fmt, scale), _ptr(codes), _ptr(scales), _ptr(h2), ldh,
                                    _stream(x.device)))
    return codes, scales, h


def rms_norm_operand(x, weight, fmt, eps=1e-6, residual=None, scale=None, residual_out=None):
    """rms_norm_quant with the quantized activation as a QuantizedActivation for linear_fused;
    returns (activation, h or None)."""
    f = _format(fmt)
    x2, ld, r2, ldr, h, h2, ldh = _norm_args(x, weight, residual, residual_out)
    M, K = x2.shape
    s = _scale_arg(fmt, scale)
    q = _new_operand(x, fmt, s)
    _check(lib().fql_rms_norm_operand(f, _ptr(x2), M, K, ld, _ptr(r2), ldr, _ptr(weight), float(eps), s,
                                      _ptr(q.data), q.data.numel(), _ptr(h2), ldh, _stream(x.device)))
    return q, h


def quant_operand(x, fmt, scale=None):
    """bf16 x [..., K] quantized once for several linear_fused calls (also "mxfp4")."""
    f = _format(fmt)
    _require_cuda(x, "x")
    if x.dtype != torch.bfloat16:
        raise FQLError("x must be bfloat16")
    x2, ld = _rows_view(x, "x")
    M, K = x2.shape
    s = _scale_arg(fmt, scale)
    q = _new_operand(x, fmt, s)
    _check(lib().fql_quant_operand(f, _ptr(x2), M, K, ld, s, _ptr(q.data), q.data.numel(), _stream(x.device)))
    return q


# ---------------------------------------------------------------------------
# linear layer with a fused epilogue
# ---------------------------------------------------------------------------

def interleave_gate_up(gate, up):
    """Rows of a gate and an up projection (or their biases, [N] tensors) in the order
    linear_fused's "swiglu" takes them: 16 gate rows, their 16 up rows, and so on. N % 16 == 0.
    Block FP8 weights are interleaved before they are quantized."""
    if gate.shape != up.shape or gate.shape[0] % 16 != 0:
        raise FQLError("gate and up must have the same shape and a multiple of 16 rows")
    both = torch.stack([gate.unflatten(0, (-1, 16)), up.unflatten(0, (-1, 16))], 1)
    return both.flatten(0, 2).contiguous()


def linear_fused(x, weight, activation=None, bias=None, residual=None, alpha=None, out=None, workspace=None):
    """y = bf16(act(alpha * x_q @ W_q^T + bias) + residual), rounded once.

    x: bf16 [..., K], quantized in the call as linear_<fmt> does, or a QuantizedActivation.
    weight: MXFP4Weight, MXFP8Weight, FP8Weight or FP8BlockWeight. activation: None, "relu",
    "gelu", "gelu_tanh", "silu", or "swiglu" (rows interleaved by interleave_gate_up, output
    [..., N/2]). bias bf16 [N]. residual: bf16 of y's shape; may be `out` itself."""
    if activation not in ACTIVATIONS:
        raise FQLError(f"unknown activation {activation!r}")
    fmt = getattr(weight, "fmt", None)
    if fmt not in FORMATS:
        raise FQLError("linear_fused takes MXFP4, MXFP8, FP8 and block FP8 weights")
    N, K = weight.N, weight.K
    quantized = isinstance(x, QuantizedActivation)
    if quantized:
        if x.fmt != fmt:
            raise FQLError(f"the activation is {x.fmt}, the weight {fmt}")
        if fmt == "fp8" and x.scale != weight.input_scale:
            raise FQLError("the activation was quantized with another scale than the weight's input_scale")
        if x.K != K:
            raise FQLError(f"x has K={x.K}, weight has K={K}")
        lead, M, ld, x2, op, dev = x.lead, x.M, 0, None, x.data, x.data.device
    else:
        _require_cuda(x, "x")
        if x.dtype != torch.bfloat16:
            raise FQLError("linear_fused takes bfloat16 activations or a QuantizedActivation")
        if x.shape[-1] != K:
            raise FQLError(f"x has K={x.shape[-1]}, weight has K={K}")
        lead, dev, op = tuple(x.shape[:-1]), x.device, None
        x2, ld = _rows_view(x, "x")
        M = x2.shape[0]
    if bias is not None:
        _bf16_vector(bias, "bias", N)
    shape = lead + (N // 2 if activation == "swiglu" else N,)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    y2, ldy = _bf16_rows(out, "out", shape)
    r2, ldr = (None, 0) if residual is None else _bf16_rows(residual, "residual", shape)
    if workspace is None:
        workspace = _workspace(dev, linear_sc_workspace_bytes(fmt, M, N, K))
    alpha_dev = weight.alpha_dev if fmt == "fp8" and alpha is None else None
    _check(lib().fql_linear_fused(FORMATS[fmt], _ptr(x2), M, K, ld, getattr(weight, "input_scale", 0), _ptr(op),
                                  _ptr(weight.packed), N, 1.0 if alpha is None else float(alpha), _ptr(alpha_dev),
                                  _ptr(bias), ACTIVATIONS[activation], _ptr(r2), ldr, _ptr(y2), ldy,
                                  _ptr(workspace), workspace.numel(), _stream(dev)))
    return out


# ---------------------------------------------------------------------------
# paged 8-bit cache
# ---------------------------------------------------------------------------

class KVCache8:
    """A paged key/value cache of E4M3 codes with one power-of-two scale per (block, head).

    k uint8 [blocks, kv_heads, block_size, head_dim]; v uint8 [blocks, kv_heads, block_size / 16,
    head_dim, 16]; k_scale, v_scale uint8 [blocks, kv_heads] (value = code * 2^(scale - 127)).
    block_size 16, 32, 64, 128 or 256; head_dim 64, 128 or 256.
    """

    def __init__(self, k, v, k_scale, v_scale):
        for t, name in ((k, "k"), (v, "v"), (k_scale, "k_scale"), (v_scale, "v_scale")):
            _require_cuda(t, name)
            if t.dtype != torch.uint8 or not t.is_contiguous() or t.device != k.device:
                raise FQLError(f"{name} must be a contiguous uint8 tensor on the cache's device")
        if k.dim() != 4 or k.shape[2] % 16 != 0:
            raise FQLError("k must be [blocks, kv_heads, block_size, head_dim], block_size a multiple of 16")
        self.num_blocks, self.kv_heads, self.block_size, self.head_dim = k.shape
        if tuple(v.shape) != (self.num_blocks, self.kv_heads, self.block_size // 16, self.head_dim, 16):
            raise FQLError("v must be [blocks, kv_heads, block_size / 16, head_dim, 16]")
        if not tuple(k_scale.shape) == tuple(v_scale.shape) == (self.num_blocks, self.kv_heads):
            raise FQLError("scales must be [blocks, kv_heads]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self._struct = KvCacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                     self.num_blocks, self.kv_heads, self.block_size, self.head_dim)

    @classmethod
    def empty(cls, num_blocks, kv_heads, block_size, head_dim, device="cuda"):
        """A cache of zeros."""
        k = torch.zeros((num_blocks, kv_heads, block_size, head_dim), dtype=torch.uint8, device=device)
        v = torch.zeros((num_blocks, kv_heads, block_size // 16, head_dim, 16), dtype=torch.uint8, device=device)
        s = torch.zeros((2, num_blocks, kv_heads), dtype=torch.uint8, device=device)
        return cls(k, v, s[0], s[1])


def _heads(t, name, tokens, heads, head_dim):
    """(tensor, token stride, head stride) of a bf16 [tokens, heads, head_dim] tensor."""
    _require_cuda(t, name)
    if t.dtype != torch.bfloat16 or t.dim() != 3 or tuple(t.shape[1:]) != (heads, head_dim):
        raise FQLError(f"{name} must be a bfloat16 tensor [tokens, {heads}, {head_dim}]")
    if tokens is not None and t.shape[0] != tokens:
        raise FQLError(f"{name} must have {tokens} tokens")
    if t.stride(2) != 1:
        raise FQLError(f"{name} must have unit stride in its last dimension")
    return t, t.stride(0), t.stride(1)


def _batch(cache, block_table, lens, cu_seqlens, max_new, tokens):
    for t, name in ((block_table, "block_table"), (lens, "lens"), (cu_seqlens, "cu_seqlens")):
        _require_cuda(t, name)
        if t.dtype != torch.int32 or t.device != cache.k.device:
            raise FQLError(f"{name} must be an int32 tensor on the cache's device")
    B = lens.shape[0] if lens.dim() == 1 else -1
    if B < 1 or tuple(cu_seqlens.shape) != (B + 1,) or block_table.dim() != 2 or block_table.shape[0] != B:
        raise FQLError("block_table must be [batch, columns], lens [batch], cu_seqlens [batch + 1]")
    if block_table.stride(1) != 1 or not lens.is_contiguous() or not cu_seqlens.is_contiguous():
        raise FQLError("block_table's rows, lens and cu_seqlens must be contiguous")
    cols = block_table.shape[1]
    ld = block_table.stride(0) if B > 1 else max(cols, block_table.stride(0))
    return KvBatchStruct(block_table.data_ptr(), ld, lens.data_ptr(), cu_seqlens.data_ptr(), tokens, cols, B,
                         min(int(max_new), tokens))


def kv_append(cache, k, v, block_table, lens, cu_seqlens, max_new):
    """Write new keys and values (bf16 [tokens, kv_heads, head_dim], any token and head strides) into
    the cache. block_table int32 [B, columns], lens int32 [B] (tokens of each sequence with the new
    ones), cu_seqlens int32 [B + 1] (first row of each sequence's new tokens), max_new: an upper bound
    of a sequence's new tokens. Nothing is read back to the host."""
    k, kt, kh = _heads(k, "k", None, cache.kv_heads, cache.head_dim)
    v, vt, vh = _heads(v, "v", k.shape[0], cache.kv_heads, cache.head_dim)
    b = _batch(cache, block_table, lens, cu_seqlens, max_new, k.shape[0])
    if k.shape[0] == 0:
        return
    _check(lib().fql_kv_append(ctypes.byref(cache._struct), ctypes.byref(b), _ptr(k), kt, kh, _ptr(v), vt, vh,
                               _stream(cache.k.device)))


def attention_kv8_plan(batch, q_heads, kv_heads, head_dim, max_new, max_len, window=0):
    """One-line description of the launch plan of an attention_kv8 call."""
    buf = ctypes.create_string_buffer(256)
    _check(lib().fql_attention_kv8_describe(int(batch), int(q_heads), int(kv_heads), int(head_dim), int(max_new),
                                            int(max_len), int(window), buf, 256))
    return buf.value.decode()


def attention_kv8(q, cache, block_table, lens, cu_seqlens, max_new, causal=True, window=0, scale=None,
                  max_len=None, out=None, return_lse=False, workspace=None):
    """Attention of the new tokens q (bf16 [tokens, q_heads, head_dim]) over the cache, which holds
    them already. Batch arguments as kv_append. window > 0: a token sees the last `window` keys up to
    itself. scale: of the scores (default 1 / sqrt(head_dim)). max_len: an upper bound of lens when one
    is known on the host (the launch is planned by it). Returns out [tokens, q_heads, head_dim] bf16, or
    (out, lse float32 [tokens, q_heads]). Rows outside cu_seqlens' ranges are not written."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise FQLError("q must be [tokens, q_heads, head_dim]")
    T, Hq = q.shape[0], q.shape[1]
    q, qt, qh = _heads(q, "q", None, Hq, cache.head_dim)
    if out is None:
        out = torch.empty((T, Hq, cache.head_dim), dtype=torch.bfloat16, device=q.device)
    out, ot, oh = _heads(out, "out", T, Hq, cache.head_dim)
    lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device) if return_lse else None
    b = _batch(cache, block_table, lens, cu_seqlens, max_new, T)
    if T > 0:
        if max_len is None:
            max_len = b.table_cols * cache.block_size
        if workspace is None:
            workspace = _workspace(q.device, _size_query("fql_attention_kv8_workspace_bytes", b.batch, Hq,
                                                         cache.kv_heads, cache.head_dim, b.max_new, max_len, window))
        s = cache.head_dim ** -0.5 if scale is None else float(scale)
        _check(lib().fql_attention_kv8(ctypes.byref(cache._struct), ctypes.byref(b), _ptr(q), qt, qh, Hq, s,
                                       int(bool(causal)), int(window), int(max_len), _ptr(out), ot, oh, _ptr(lse),
                                       _ptr(workspace), workspace.numel(), _stream(q.device)))
    return (out, lse) if return_lse else out
