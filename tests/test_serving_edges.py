"""Edges of the 8-bit serving operators that need no GPU: host queries, checks of arguments."""

import ctypes

import fp8_quantized_linear_amd as fql

from test_serving_api import refused


def test_capture_id_refusals():
    refused(fql.lib().fql_stream_capture_id(None, ctypes.POINTER(ctypes.c_uint64)()), "null")


def test_a_remembered_workspace_size_follows_the_launch_plan_override():
    def size():
        return fql.serving._query("fql_linear_fused_workspace_bytes", fql.FMT_MXFP8, 256, 4096, 4096)

    def asked():
        n = ctypes.c_size_t()
        assert fql.lib().fql_linear_fused_workspace_bytes(fql.FMT_MXFP8, 256, 4096, 4096, ctypes.byref(n)) == 0
        return n.value

    plain = size()
    with fql.plan_override("2,2,4,4,3,4", which="sc_gemm"):
        assert size() == asked() > 4 * plain
    assert size() == asked() == plain
