"""Refusals, sizes and plans of the 8-bit serving operators (CPU): every call here fails validation
before any launch, or only plans."""

import ctypes

import pytest
import torch

import fp8_quantized_linear_amd as fql

P, NULL = ctypes.c_void_p(1 << 20), ctypes.c_void_p(0)
FP8, BLOCK, MXFP8, MXFP4, NVFP4 = (fql.FMT_FP8, fql.FMT_FP8_BLOCK, fql.FMT_MXFP8, fql.FMT_MXFP4, fql.FMT_NVFP4)


def refused(status, *words, code=-1):
    msg = fql.lib().fql_last_error().decode()
    assert status == code, (status, msg)
    assert all(w in msg for w in words), msg


def norm(fmt=MXFP8, x=P, M=4, K=256, ldx=256, res=P, ldr=256, w=P, eps=1e-6, scale=0.1, codes=P, scales=P, h=P, ldh=256):
    return fql.lib().fql_rms_norm_quant(fmt, x, M, K, ldx, res, ldr, w, eps, scale, codes, scales, h, ldh, NULL)


def test_norm_refusals():
    refused(norm(fmt=NVFP4), "format", code=-2)
    refused(norm(fmt=MXFP4), "format", code=-2)
    refused(norm(fmt=99), code=-2)
    refused(norm(M=0), "M")
    refused(norm(K=240), "32")
    refused(norm(fmt=BLOCK, K=160), "128")
    refused(norm(ldx=255), "stride")
    refused(norm(ldr=255), "residual")
    refused(norm(ldh=255), "h_out")
    refused(norm(res=NULL), "h_out")
    refused(norm(eps=-1.0), "eps")
    refused(norm(eps=float("nan")), "eps")
    refused(norm(fmt=FP8, scale=0.0), "scale")
    refused(norm(fmt=FP8, scale=float("inf")), "scale")
    refused(norm(codes=ctypes.c_void_p((1 << 20) + 4)), "aligned")
    for null in ("x", "w", "codes", "scales"):
        refused(norm(**{null: NULL}), "null")


def test_operand_sizes_and_refusals():
    n = ctypes.c_size_t()
    lib = fql.lib()
    for fmt, code, scale in ((FP8, 1, 0), (BLOCK, 1, 4), (MXFP8, 1, 4)):
        for M, K in ((1, 128), (256, 4096), (257, 4096)):
            assert lib.fql_operand_bytes(fmt, M, K, ctypes.byref(n)) == 0
            Mp = -(-M // 256) * 256
            assert n.value == Mp * K * code + Mp * (K // 128) * scale
    assert lib.fql_operand_bytes(MXFP4, 1, 128, ctypes.byref(n)) == 0 and n.value == 256 * 64 + 256 * 4
    refused(lib.fql_operand_bytes(NVFP4, 1, 128, ctypes.byref(n)), code=-2)
    refused(lib.fql_operand_bytes(FP8, 0, 128, ctypes.byref(n)), "M")
    q = lambda op, size, scale=1.0, fmt=MXFP8: lib.fql_quant_operand(fmt, P, 4, 128, 128, scale, op, size, NULL)  # noqa: E731
    refused(q(P, 100), "holds")
    refused(q(ctypes.c_void_p((1 << 20) + 16), 1 << 30), "256")
    refused(q(NULL, 1 << 30), "null")
    refused(q(P, 1 << 30, scale=-1.0, fmt=FP8), "scale")
    refused(lib.fql_rms_norm_operand(MXFP8, P, 4, 128, 128, NULL, 0, P, 1e-6, 0.0, P, 100, NULL, 0, NULL), "holds")


def linear(fmt=MXFP8, x=P, M=4, K=256, ldx=256, s=0.1, op=NULL, w=P, N=64, alpha=1.0, act=0, res=NULL, ldr=0, y=P,
           ldy=64, ws=P, size=1 << 30):
    return fql.lib().fql_linear_fused(fmt, x, M, K, ldx, s, op, w, N, alpha, NULL, NULL, act, res, ldr, y, ldy, ws, size,
                                      NULL)


def test_linear_refusals():
    refused(linear(fmt=NVFP4), "epilogue", code=-2)
    refused(linear(op=P), "either")
    refused(linear(x=NULL), "either")
    refused(linear(act=6), "activation")
    refused(linear(act=-1), "activation")
    refused(linear(act=5, N=48, ldy=48), "32")
    refused(linear(act=5, N=64, ldy=31), "ldy")
    refused(linear(ldy=63), "ldy")
    refused(linear(res=P, ldr=63), "residual")
    refused(linear(act=5, ldy=32, res=P, ldr=31), "residual")
    refused(linear(alpha=float("nan")), "alpha")
    refused(linear(fmt=FP8, s=0.0), "input_scale")
    refused(linear(K=200), "32")
    refused(linear(ldx=200), "stride")
    refused(linear(fmt=BLOCK, N=100, ldy=100), "128")
    refused(linear(w=NULL), "null")
    refused(linear(y=NULL), "null")
    refused(linear(x=NULL, op=ctypes.c_void_p(1 << 20 | 16)), "256")
    refused(linear(size=16), "workspace", code=-4)


def test_linear_plans():
    """The planner's tiles over the range; workspaces hold the activation operand and the partial sums."""
    n = ctypes.c_size_t()
    seen = set()
    for fmt, code in (("mxfp4", MXFP4), ("mxfp8", MXFP8), ("fp8", FP8), ("fp8_block", BLOCK)):
        for M in (1, 16, 33, 64, 100, 128, 250, 500, 1000, 1900, 4096):
            for N, K in ((128, 128), (4096, 4096), (28672, 4096), (4096, 14336), (5120, 25600)):
                assert fql.lib().fql_linear_fused_workspace_bytes(code, M, N, K, ctypes.byref(n)) == 0
                assert n.value >= 65536 + M * K // (2 if fmt == "mxfp4" else 1)
                plan = fql.linear_fused_plan(fmt, M, N, K)
                if fmt == "mxfp4" or M <= 32:
                    assert plan == fql.linear_sc_plan(fmt, M, N, K)
                seen.add(plan.split("<")[-1].split(">")[0].split(",", 1)[1])
    assert {"WM=2,WN=2,MTW=2,NTW=2,ST=4", "WM=4,WN=2,MTW=2,NTW=2,ST=4", "WM=2,WN=4,MTW=4,NTW=2,ST=4",
            "WM=4,WN=2,MTW=4,NTW=4,ST=3", "WM=1,WN=4,MTW=1,NTW=2,ST=4"} <= seen, seen
    refused(fql.lib().fql_linear_fused_workspace_bytes(NVFP4, 4, 64, 128, ctypes.byref(n)), "format", code=-2)
    refused(fql.lib().fql_linear_fused_workspace_bytes(MXFP8, 4, 64, 100, ctypes.byref(n)), "32")


class CacheStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] + [("num_blocks", ctypes.c_int64)] + [
        (n, ctypes.c_int32) for n in ("kv_heads", "block_size", "head_dim")]


class BatchStruct(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("ld_table", ctypes.c_int64), ("lens", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p), ("tokens", ctypes.c_int64), ("table_cols", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("max_new", ctypes.c_int32)]


def cache(**kw):
    d = dict(k=1 << 20, v=1 << 20, k_scale=1 << 20, v_scale=1 << 20, num_blocks=8, kv_heads=2, block_size=16, head_dim=64)
    d.update(kw)
    return CacheStruct(**d)


def batch(**kw):
    d = dict(block_table=1 << 20, ld_table=4, lens=1 << 20, cu_seqlens=1 << 20, tokens=3, table_cols=4, batch=2, max_new=2)
    d.update(kw)
    return BatchStruct(**d)


def test_binding_packs_the_structs_as_the_header_lays_them_out():
    import struct

    c = struct.pack("PPPPqiii4x", 1, 2, 3, 4, 5, 6, 7, 8)
    assert c[:ctypes.sizeof(CacheStruct)] == bytes(CacheStruct(1, 2, 3, 4, 5, 6, 7, 8)) and len(c) == ctypes.sizeof(CacheStruct)
    b = struct.pack("PqPPqiii4x", 1, 2, 3, 4, 5, 6, 7, 8)
    assert b == bytes(BatchStruct(1, 2, 3, 4, 5, 6, 7, 8))


def append(c=None, b=None, k=P, v=P, st=128):
    return fql.lib().fql_kv_append(ctypes.byref(c or cache()), ctypes.byref(b or batch()), k, st, 64, v, 128, 64, NULL)


def attend(c=None, b=None, q=P, Hq=4, scale=0.1, window=0, max_len=64, out=P, ws=P, size=1 << 30, st=256):
    return fql.lib().fql_attention_kv8(ctypes.byref(c or cache()), ctypes.byref(b or batch()), q, st, 64, Hq, scale, 1,
                                       window, max_len, out, 256, 64, NULL, ws, size, NULL)


@pytest.mark.parametrize("call", [append, attend])
def test_cache_and_batch_refusals(call):
    for null in ("k", "v", "k_scale", "v_scale"):
        refused(call(c=cache(**{null: 0})), "null")
    for null in ("block_table", "lens", "cu_seqlens"):
        refused(call(b=batch(**{null: 0})), "null")
    refused(call(c=cache(k=(1 << 20) + 8)), "aligned")
    for d in (0, 32, 96, 512):
        refused(call(c=cache(head_dim=d)), "head_dim", code=-2)
    for bs in (0, 8, 24, 512, -16):
        refused(call(c=cache(block_size=bs)), "block_size", code=-2)
    refused(call(c=cache(kv_heads=0)), "kv_heads")
    refused(call(c=cache(num_blocks=0)), "num_blocks")
    refused(call(c=cache(num_blocks=1 << 40)), "num_blocks")
    refused(call(b=batch(batch=0)), "batch")
    refused(call(b=batch(batch=1 << 17)), "batch")
    refused(call(b=batch(table_cols=5)), "table_cols")
    refused(call(b=batch(table_cols=0)), "table_cols")
    refused(call(c=cache(block_size=256), b=batch(ld_table=1 << 24, table_cols=1 << 23)), "2^30")
    refused(call(b=batch(tokens=-1)), "tokens")
    refused(call(b=batch(max_new=-1)), "max_new")
    refused(call(st=-1), "stride")
    # nothing to do: no launch, no error
    assert call(b=batch(tokens=0)) == 0
    assert call(b=batch(max_new=0)) == 0


def test_append_and_attention_refusals():
    refused(append(k=NULL), "null")
    refused(append(v=NULL), "null")
    refused(attend(q=NULL), "null")
    refused(attend(out=NULL), "null")
    refused(attend(ws=NULL), "null")
    refused(attend(Hq=3), "q_heads")
    refused(attend(Hq=0), "q_heads")
    refused(attend(scale=float("inf")), "scale")
    refused(attend(scale=-0.1), "scale")
    refused(attend(scale=0.0), "scale")
    refused(attend(window=-1), "window")
    refused(attend(max_len=0), "max_len")
    refused(attend(ws=ctypes.c_void_p((1 << 20) + 16)), "256")
    refused(attend(size=1000), "workspace", code=-4)
    refused(attend(b=batch(tokens=1 << 29, max_new=1 << 24), Hq=256), "rows", code=-2)


def test_attention_plans():
    """Few rows stream with the keys split until the card is full; the workspace holds the plan's
    partial results."""
    n = ctypes.c_size_t()
    for B in (1, 2, 7, 64, 300):
        for Hq, H in ((32, 8), (64, 8), (16, 16), (28, 4), (24, 1)):
            for D in (64, 128, 256):
                for new in (1, 2, 5, 33, 2000):
                    for max_len in (1, 64, 1000, 16384, 131072):
                        for window in (0, 100):
                            args = (B, Hq, H, D, new, max_len, window)
                            assert fql.lib().fql_attention_kv8_workspace_bytes(*args, ctypes.byref(n)) == 0
                            assert 65536 <= n.value < 1 << 32
                            plan = fql.attention_kv8_plan(*args)
                            f = dict(w.split("=") for w in plan.replace("<", " ").replace(">", " ").replace(",", " ").split()
                                     if "=" in w)
                            assert int(f["chunk"]) % 64 == 0
                            span = min(max_len, window + new + 62) if window else max_len
                            assert int(f["splits"]) * int(f["chunk"]) >= span, plan
    assert "splits=1 " not in fql.attention_kv8_plan(1, 32, 8, 128, 1, 16384)
    assert "splits=1 " in fql.attention_kv8_plan(1, 32, 8, 128, 1, 200)


def test_binding_refusals_without_a_gpu():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.ones(256, dtype=torch.bfloat16)
    with pytest.raises(fql.FQLError, match="unknown format"):
        fql.rms_norm_quant(x, w, "int8")
    with pytest.raises(fql.FQLError, match="CUDA"):
        fql.rms_norm_quant(x, w, "mxfp8")
    with pytest.raises(fql.FQLError, match="CUDA"):
        fql.quant_operand(x, "mxfp8")
    with pytest.raises(fql.FQLError, match="activation"):
        fql.linear_fused(x, None, activation="tanh")
    with pytest.raises(fql.FQLError, match="weights"):
        fql.linear_fused(x, None)
    with pytest.raises(fql.FQLError, match="CUDA"):
        fql.KVCache8.empty(2, 1, 16, 64, device="cpu")
    with pytest.raises(fql.FQLError, match="16 rows"):
        fql.interleave_gate_up(torch.zeros(8, 4), torch.zeros(8, 4))
    g, u = torch.arange(32), torch.arange(32) + 100
    both = fql.interleave_gate_up(g, u)
    assert both.tolist() == [*range(16), *range(100, 116), *range(16, 32), *range(116, 132)]
