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
import functools
import struct

import torch

from . import (FMT_FP8, FMT_FP8_BLOCK, FMT_MXFP4, FMT_MXFP8, FQLError, _captured, _captured_workspace, _capturing,
               _check, _grow_workspace, _rows_view, _size_query, _workspaces, lib)

FORMATS = {"mxfp4": FMT_MXFP4, "mxfp8": FMT_MXFP8, "fp8": FMT_FP8, "fp8_block": FMT_FP8_BLOCK}
_I32_MAX = 2 ** 31 - 1
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "swiglu": 5}

# A decode step's calls take a few microseconds on the GPU, so what Python does
# around them counts: addresses go to the library as plain integers, the
# structs of include/fql.h as packed bytes, sizes that depend on shapes alone
# are remembered (until set_plan_override changes the plans).
_stream = torch._C._cuda_getCurrentRawStream  # device index -> hipStream_t of torch's current stream
_bf16, _u8, _i32, _f32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
_query = functools.lru_cache(4096)(_size_query)


def _workspace(device, nbytes):
    """The binding's workspace of this device and stream, or of its capture (shared with the linear calls)."""
    index = device.index
    key = ("cuda", index, _stream(index))
    if _captured or _capturing():
        ws = _captured_workspace(key, nbytes, device)
        if ws is not None:
            return ws
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = _grow_workspace(key, nbytes, device)
    return ws


def _new(shape, dtype, dev):
    """torch.empty of a contiguous tensor, a microsecond sooner for two dimensions (given as a
    torch.Size, it takes 2.2 us; so, 1.3)."""
    if len(shape) == 2:
        M, n = shape
        return torch.empty_strided((M, n), (n, 1), dtype=dtype, device=dev)
    return torch.empty(shape, dtype=dtype, device=dev)


def _format(fmt):
    if fmt not in FORMATS:
        raise FQLError(f"unknown format {fmt!r} (one of {', '.join(FORMATS)})")
    return FORMATS[fmt]


def _cuda(t, name, dtype):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise FQLError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype is not dtype:
        raise FQLError(f"{name} must be {dtype}")


def _same_device(t, name, index, of="x"):
    if t.get_device() != index:
        raise FQLError(f"{name} must be on {of}'s device")


def _rows(t, name, shape=None, index=None):
    """(address, rows, columns, row stride) of a bf16 [..., K] tensor, of the given shape and on the
    given device if any."""
    if shape is None:
        _cuda(t, name, _bf16)
    elif not isinstance(t, torch.Tensor) or t.dtype is not _bf16 or t.get_device() != index or t.shape != shape:
        _cuda(t, name, _bf16)
        _same_device(t, name, index)
        raise FQLError(f"{name} must have shape {tuple(shape)}")
    if t.dim() == 2:
        M, K = t.shape
        ld, unit = t.stride()
        if unit == 1:
            return t.data_ptr(), M, K, ld if M > 1 or ld > K else K
    t2, ld = _rows_view(t, name)
    return t2.data_ptr(), t2.shape[0], t2.shape[1], ld


def _scale_arg(fmt, scale):
    if fmt != "fp8":
        return 0
    if scale is None:
        raise FQLError("per-tensor FP8 needs its static scale")
    return ctypes.c_float(float(scale)).value


def _vector(t, name, n, index):
    if not isinstance(t, torch.Tensor) or t.dtype is not _bf16 or t.get_device() != index:
        _cuda(t, name, _bf16)
        _same_device(t, name, index)
    if t.numel() != n or not t.is_contiguous():
        raise FQLError(f"{name} must be a contiguous bf16 tensor of {n} elements")
    return t.data_ptr()


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
    """An operand of x's shape, without any bytes where x has no rows."""
    K = x.shape[-1]
    q = QuantizedActivation(None, fmt, x.shape[:-1], K, scale if fmt == "fp8" else None)
    n = _query("fql_operand_bytes", _format(fmt), q.M or 1, K)
    q.data = torch.empty_strided((n if q.M else 0,), (1,), dtype=_u8, device=x.device)
    return q


def _norm_args(x, weight, residual, residual_out):
    """(address, M, K, ld of x, of the residual: address, ld, weight's address, h, its address and ld)."""
    xp, M, K, ld = _rows(x, "x")
    index = x.get_device()
    wp = _vector(weight, "weight", K, index)
    if residual is None:
        if residual_out is not None:
            raise FQLError("residual_out needs a residual")
        return xp, M, K, ld, 0, 0, wp, None, 0, 0
    rp, _, _, ldr = _rows(residual, "residual", x.shape, index)
    if residual_out is None:
        h = _new(x.shape, _bf16, x.device)
        return xp, M, K, ld, rp, ldr, wp, h, h.data_ptr(), K
    hp, _, _, ldh = _rows(residual_out, "residual_out", x.shape, index)
    return xp, M, K, ld, rp, ldr, wp, residual_out, hp, ldh


def rms_norm_quant(x, weight, fmt, eps=1e-6, residual=None, scale=None, residual_out=None):
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight, quantized to fmt ("fp8", "fp8_block"
    or "mxfp8"). x, residual bf16 [..., K], weight bf16 [K]; scale: per-tensor FP8's static scale.
    Returns (codes uint8 [..., K], scales as quant_<fmt> gives them or None, h bf16 or None without a
    residual). residual_out may be x or residual itself. No rows give empty outputs."""
    f = _format(fmt)
    xp, M, K, ld, rp, ldr, wp, h, hp, ldh = _norm_args(x, weight, residual, residual_out)
    dev = x.device
    codes = _new(x.shape, _u8, dev)
    scales, sp = None, 0
    if fmt == "mxfp8":
        scales = _new(x.shape[:-1] + (K // 32,), _u8, dev)
    elif fmt == "fp8_block":
        scales = _new(x.shape[:-1] + (K // 128,), _f32, dev)
    if scales is not None:
        sp = scales.data_ptr()
    s = _scale_arg(fmt, scale)
    if M == 0:
        _query("fql_operand_bytes", f, 1, K)  # refuses what any other call on this K would
    else:
        _check(lib().fql_rms_norm_quant(f, xp, M, K, ld, rp, ldr, wp, eps, s, codes.data_ptr(), sp, hp, ldh,
                                        _stream(dev.index)))
    return codes, scales, h


def rms_norm_operand(x, weight, fmt, eps=1e-6, residual=None, scale=None, residual_out=None):
    """rms_norm_quant with the quantized activation as a QuantizedActivation for linear_fused;
    returns (activation, h or None)."""
    f = _format(fmt)
    xp, M, K, ld, rp, ldr, wp, h, hp, ldh = _norm_args(x, weight, residual, residual_out)
    s = _scale_arg(fmt, scale)
    q = _new_operand(x, fmt, s)
    if M > 0:
        _check(lib().fql_rms_norm_operand(f, xp, M, K, ld, rp, ldr, wp, eps, s, q.data.data_ptr(), q.data.numel(), hp,
                                          ldh, _stream(x.device.index)))
    return q, h


def quant_operand(x, fmt, scale=None):
    """bf16 x [..., K] quantized once for several linear_fused calls (also "mxfp4")."""
    f = _format(fmt)
    xp, M, K, ld = _rows(x, "x")
    s = _scale_arg(fmt, scale)
    q = _new_operand(x, fmt, s)
    if M > 0:
        _check(lib().fql_quant_operand(f, xp, M, K, ld, s, q.data.data_ptr(), q.data.numel(), _stream(x.device.index)))
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


def linear_fused_plan(fmt, M, N, K):
    """One-line description of the launch plan of a linear_fused call."""
    buf = ctypes.create_string_buffer(256)
    _check(lib().fql_linear_fused_describe(_format(fmt), int(M), int(N), int(K), buf, 256))
    return buf.value.decode()


def linear_fused(x, weight, activation=None, bias=None, residual=None, alpha=None, out=None, workspace=None):
    """y = bf16(act(alpha * x_q @ W_q^T + bias) + residual), rounded once.

    x: bf16 [..., K], quantized in the call as linear_<fmt> does, or a QuantizedActivation.
    weight: MXFP4Weight, MXFP8Weight, FP8Weight or FP8BlockWeight. activation: None, "relu",
    "gelu", "gelu_tanh", "silu", or "swiglu" (rows interleaved by interleave_gate_up, output
    [..., N/2]). bias bf16 [N]. residual: bf16 of y's shape; may be `out` itself, `x` may not. No rows
    give an empty output."""
    if activation not in ACTIVATIONS:
        raise FQLError(f"unknown activation {activation!r}")
    fmt = getattr(weight, "fmt", None)
    if fmt not in FORMATS:
        raise FQLError("linear_fused takes MXFP4, MXFP8, FP8 and block FP8 weights")
    N, K = weight.N, weight.K
    xp = op = ld = 0
    if isinstance(x, QuantizedActivation):
        if x.fmt != fmt:
            raise FQLError(f"the activation is {x.fmt}, the weight {fmt}")
        if fmt == "fp8" and x.scale != weight.input_scale:
            raise FQLError("the activation was quantized with another scale than the weight's input_scale")
        lead, M, xK, op, dev = x.lead, x.M, x.K, x.data.data_ptr(), x.data.device
    else:
        xp, M, xK, ld = _rows(x, "x")
        lead, dev = x.shape[:-1], x.device
    if xK != K:
        raise FQLError(f"x has K={xK}, weight has K={K}")
    index = dev.index
    packed = weight.packed
    if packed.get_device() != index:
        _same_device(packed, "weight", index)
    bp = 0 if bias is None else _vector(bias, "bias", N, index)
    No = N // 2 if activation == "swiglu" else N
    shape = lead + (No,)
    rp = ldr = 0
    if residual is not None:
        rp, _, _, ldr = _rows(residual, "residual", shape, index)
    if out is None:
        out = _new(shape, _bf16, dev)
        yp, ldy = out.data_ptr(), No
    else:
        yp, _, _, ldy = _rows(out, "out", shape, index)
    if M == 0:
        return out
    if workspace is None:
        workspace = _workspace(dev, _query("fql_linear_fused_workspace_bytes", FORMATS[fmt], M, N, K))
    else:
        _same_device(workspace, "workspace", index)
    scale, ap = 0, 0
    if fmt == "fp8":
        scale = weight.input_scale
        if alpha is None:
            _same_device(weight.alpha_dev, "alpha_dev", index)
            ap = weight.alpha_dev.data_ptr()
    _check(lib().fql_linear_fused(FORMATS[fmt], xp, M, K, ld, scale, op, packed.data_ptr(), N,
                                  1.0 if alpha is None else alpha, ap, bp, ACTIVATIONS[activation], rp, ldr, yp, ldy,
                                  workspace.data_ptr(), workspace.numel(), _stream(index)))
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
            _cuda(t, name, _u8)
            if not t.is_contiguous() or t.device != k.device:
                raise FQLError(f"{name} must be contiguous and on the cache's device")
        if k.dim() != 4 or k.shape[2] % 16 != 0:
            raise FQLError("k must be [blocks, kv_heads, block_size, head_dim], block_size a multiple of 16")
        self.num_blocks, self.kv_heads, self.block_size, self.head_dim = k.shape
        if tuple(v.shape) != (self.num_blocks, self.kv_heads, self.block_size // 16, self.head_dim, 16):
            raise FQLError("v must be [blocks, kv_heads, block_size / 16, head_dim, 16]")
        if not tuple(k_scale.shape) == tuple(v_scale.shape) == (self.num_blocks, self.kv_heads):
            raise FQLError("scales must be [blocks, kv_heads]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self._index = k.get_device()
        self._struct = struct.pack("PPPPqiii4x", k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                   self.num_blocks, self.kv_heads, self.block_size, self.head_dim)  # fql_kv_cache

    @classmethod
    def empty(cls, num_blocks, kv_heads, block_size, head_dim, device="cuda"):
        """A cache of zeros."""
        k = torch.zeros((num_blocks, kv_heads, block_size, head_dim), dtype=torch.uint8, device=device)
        v = torch.zeros((num_blocks, kv_heads, block_size // 16, head_dim, 16), dtype=torch.uint8, device=device)
        s = torch.zeros((2, num_blocks, kv_heads), dtype=torch.uint8, device=device)
        return cls(k, v, s[0], s[1])


def _heads(t, name, shape, index):
    """(address, token stride, head stride) of a bf16 [tokens, heads, head_dim] tensor on the cache's device."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _bf16 or t.get_device() != index:
        _cuda(t, name, _bf16)
        raise FQLError(f"{name} must be on the cache's device")
    if t.shape != shape:
        raise FQLError(f"{name} must have shape {shape}")
    ld_token, ld_head, unit = t.stride()
    if unit != 1:
        raise FQLError(f"{name} must have unit stride in its last dimension")
    return t.data_ptr(), ld_token, ld_head


def _is_i32(t, index):
    return isinstance(t, torch.Tensor) and t.dtype is _i32 and t.get_device() == index


def _batch(cache, block_table, lens, cu_seqlens, max_new, tokens):
    """A packed fql_kv_batch, the batch size and its bound of new tokens."""
    index = cache._index
    if not (_is_i32(block_table, index) and _is_i32(lens, index) and _is_i32(cu_seqlens, index)):
        for t, name in ((block_table, "block_table"), (lens, "lens"), (cu_seqlens, "cu_seqlens")):
            _cuda(t, name, _i32)
            if t.get_device() != index:
                raise FQLError(f"{name} must be on the cache's device")
    if lens.dim() != 1 or cu_seqlens.dim() != 1 or block_table.dim() != 2:
        raise FQLError("block_table must be [batch, columns], lens [batch], cu_seqlens [batch + 1]")
    B = lens.shape[0]
    rows, cols = block_table.shape
    if B < 1 or rows != B or cu_seqlens.shape[0] != B + 1:
        raise FQLError("block_table must be [batch, columns], lens [batch], cu_seqlens [batch + 1]")
    ld, unit = block_table.stride()
    if (unit != 1 and cols > 1) or not lens.is_contiguous() or not cu_seqlens.is_contiguous():
        raise FQLError("block_table's rows, lens and cu_seqlens must be contiguous")
    if B == 1:
        ld = cols
    elif ld < cols:
        raise FQLError("block_table's rows must not overlap (copy an expanded table)")
    new = int(max_new)
    if new < 0:
        raise FQLError("max_new must be >= 0")
    new = new if new < tokens else tokens
    return struct.pack("PqPPqiii4x", block_table.data_ptr(), ld, lens.data_ptr(), cu_seqlens.data_ptr(), tokens, cols, B,
                       new), B, cols, new


def kv_append(cache, k, v, block_table, lens, cu_seqlens, max_new):
    """Write new keys and values (bf16 [tokens, kv_heads, head_dim], any token and head strides) into
    the cache. block_table int32 [B, columns], lens int32 [B] (tokens of each sequence with the new
    ones), cu_seqlens int32 [B + 1] (first row of each sequence's new tokens), max_new: an upper bound
    of a sequence's new tokens. Nothing is read back to the host."""
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise FQLError("k must be a tensor [tokens, kv_heads, head_dim]")
    T = k.shape[0]
    shape = (T, cache.kv_heads, cache.head_dim)
    kp, kt, kh = _heads(k, "k", shape, cache._index)
    vp, vt, vh = _heads(v, "v", shape, cache._index)
    b, _, _, _ = _batch(cache, block_table, lens, cu_seqlens, max_new, T)
    if T > 0:
        _check(lib().fql_kv_append(cache._struct, b, kp, kt, kh, vp, vt, vh, _stream(cache._index)))


def _within(value, name, lo, hi):
    """A whole number that the library's C argument holds."""
    value = int(value)
    if not lo <= value <= hi:
        raise FQLError(f"{name} must be in {lo} .. {hi}")
    return value


def attention_kv8_plan(batch, q_heads, kv_heads, head_dim, max_new, max_len, window=0):
    """One-line description of the launch plan of an attention_kv8 call."""
    buf = ctypes.create_string_buffer(256)
    _check(lib().fql_attention_kv8_describe(int(batch), int(q_heads), int(kv_heads), int(head_dim), int(max_new),
                                            int(max_len), _within(window, "window", 0, _I32_MAX), buf, 256))
    return buf.value.decode()


def attention_kv8(q, cache, block_table, lens, cu_seqlens, max_new, causal=True, window=0, scale=None,
                  max_len=None, out=None, return_lse=False, workspace=None):
    """Attention of the new tokens q (bf16 [tokens, q_heads, head_dim]) over the cache, which holds
    them already. Batch arguments as kv_append. window > 0: a token sees the last `window` keys up to
    itself. scale: of the scores (default 1 / sqrt(head_dim)). max_len: an upper bound of lens when one
    is known on the host (the launch is planned by it). Returns out [tokens, q_heads, head_dim] bf16, or
    (out, lse float32 [tokens, q_heads]). Rows outside cu_seqlens' ranges are not written."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise FQLError("q must be a tensor [tokens, q_heads, head_dim]")
    T, Hq, _ = q.shape
    D, dev = cache.head_dim, q.device
    shape = (T, Hq, D)
    qp, qt, qh = _heads(q, "q", shape, cache._index)
    if out is None:
        out = torch.empty_strided(shape, (Hq * D, D, 1), dtype=_bf16, device=dev)
        op, ot, oh = out.data_ptr(), Hq * D, D
    else:
        op, ot, oh = _heads(out, "out", shape, cache._index)
    lse, lp = None, 0
    if return_lse:
        lse = _new((T, Hq), _f32, dev)
        lp = lse.data_ptr()
    b, B, cols, new = _batch(cache, block_table, lens, cu_seqlens, max_new, T)
    if T > 0:
        if window:
            window = _within(window, "window", 0, _I32_MAX)
        if max_len is None:
            max_len = cols * cache.block_size
        else:
            max_len = _within(max_len, "max_len", 1, 1 << 30)
        if workspace is None:
            workspace = _workspace(dev, _query("fql_attention_kv8_workspace_bytes", B, Hq, cache.kv_heads, D, new,
                                               max_len, window))
        else:
            _same_device(workspace, "workspace", cache._index, "the cache")
        _check(lib().fql_attention_kv8(cache._struct, b, qp, qt, qh, Hq, D ** -0.5 if scale is None else scale,
                                       bool(causal), window, max_len, op, ot, oh, lp, workspace.data_ptr(),
                                       workspace.numel(), _stream(cache._index)))
    return (out, lse) if return_lse else out
