"""Edges of the 8-bit serving operators that need no GPU: host queries, checks of arguments."""

import ctypes

import fp8_quantized_linear_amd as fql

from test_serving_api import refused


def test_capture_id_refusals():
    refused(fql.lib().fql_stream_capture_id(None, ctypes.POINTER(ctypes.c_uint64)()), "null")
