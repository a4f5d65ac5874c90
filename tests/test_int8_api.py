"""Refusals, sizes and plans of INT8 (CPU): every call here fails validation before any launch, or only plans."""

import ctypes

import numpy as np

import fp8_quantized_linear_amd as fql
from oracle import feedforward as O

P, NULL = ctypes.c_void_p(1 << 20), ctypes.c_void_p(0)


def refused(status, *words, code=-1):
    msg = fql.lib().fql_last_error().decode()
    assert status == code, (status, msg)
    assert all(w in msg for w in words), msg


def test_can_implement():
    assert fql.can_implement(100, 4096 + 32, 0, fmt=fql.FMT_INT8) == (True, "")
    assert fql.can_implement(1, 131072, 0, fmt=fql.FMT_INT8)[0]
    for N, K, hb, word in ((64, 131072 + 32, 0, "131072"), (64, 40, 0, "32"), (0, 64, 0, "N"), (64, 64, 32, "rotation")):
        ok, why = fql.can_implement(N, K, hb, fmt=fql.FMT_INT8)
        assert not ok and word in why


def test_sizes_and_plans():
    n = ctypes.c_size_t()
    lib = fql.lib()
    for N, K in ((1, 32), (100, 4096), (4096, 14336)):
        assert lib.fql_packed_int8_bytes(N, K, ctypes.byref(n)) == 0
        Np, Kp = -(-N // 16) * 16, -(-K // 128) * 128
        assert n.value == Np * Kp + -(-Np * 4 // 256) * 256
    assert lib.fql_operand_bytes(fql.FMT_INT8, 257, 4096, ctypes.byref(n)) == 0 and n.value == 512 * 4096 + 512 * 4
    for M in (1, 17, 33, 128, 512, 4096):
        for N, K in ((128, 128), (4096, 4096), (28672, 4096), (4096, 14336)):
            assert fql.linear_sc_workspace_bytes("int8", M, N, K) >= 65536 + M * K
            assert "int8" in fql.linear_sc_plan("int8", M, N, K) and "int8" in fql.linear_fused_plan("int8", M, N, K)
    assert "FQ=1" in fql.linear_sc_plan("int8", 1, 4096, 4096)  # single tokens are quantized in the product's launch


def test_refusals():
    lib = fql.lib()
    quant = lambda x=P, M=4, K=256, ld=256, codes=P, scales=P: lib.fql_quant_int8(x, M, K, ld, codes, scales, NULL)  # noqa: E731
    refused(quant(M=0), "M")
    refused(quant(K=48, ld=48), "32")
    refused(quant(K=131072 + 32, ld=1 << 20), "131072")
    refused(quant(ld=255), "stride")
    refused(quant(x=NULL), "null")
    refused(quant(scales=NULL), "null")
    refused(quant(codes=ctypes.c_void_p((1 << 20) + 4)), "8-byte")
    refused(quant(scales=ctypes.c_void_p((1 << 20) + 2)), "aligned")
    pack = lambda c=P, s=P, N=64, K=128, p=P, size=1 << 30: lib.fql_pack_weight_int8(c, s, N, K, p, size, NULL)  # noqa: E731
    refused(pack(size=100), "holds")
    refused(pack(s=NULL), "null")
    refused(pack(c=ctypes.c_void_p((1 << 20) + 8)), "16-byte")
    refused(pack(s=ctypes.c_void_p((1 << 20) + 1)), "aligned")

    def linear(x=P, M=4, K=256, ldx=256, w=P, N=64, alpha=1.0, y=P, ldy=64, ws=P, size=1 << 30):
        return lib.fql_linear_int8(x, M, K, ldx, w, N, alpha, NULL, y, ldy, ws, size, NULL)

    refused(linear(K=40), "32")
    refused(linear(K=262144, ldx=262144), "131072")
    refused(linear(ldy=63), "ldy")
    refused(linear(alpha=float("nan")), "alpha")
    refused(linear(w=NULL), "null")
    refused(linear(size=16), "workspace", code=-4)
    refused(lib.fql_rms_norm_quant(fql.FMT_INT8, P, 4, 64, 64, NULL, 0, P, 1e-6, 0.0, P, P, NULL, 0, NULL), "operand",
            code=-2)


def test_oracle_codes():
    x = np.array([[127, 0.5, 1.5, -2.5], [0, 0, 0, 0], [np.inf, 1, 1, 1], [2.54, -1.27, 0.01, 0.03]], dtype=np.float32)
    q, s = O.quant_int8(x)
    assert q[0].tolist() == [127, 0, 2, -2] and s[0] == 1.0
    assert q[1].tolist() == [0] * 4 and s[1] == 0.0 and np.isnan(s[2])
    assert (np.abs(O.dequant_int8(q, s)[3] - x[3]) <= s[3] * (0.5 + 1e-5)).all()
