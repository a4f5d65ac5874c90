"""Edges of the 8-bit serving operators that need no GPU: host queries, checks of arguments."""

import ctypes
import types
import weakref

import numpy as np
import pytest
import torch

import fp8_quantized_linear_amd as fql

from test_serving_api import FP8, NULL, P, batch, cache, linear, norm, refused


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


# ---------------------------------------------------------------------------
# tensors of another device
# ---------------------------------------------------------------------------

class OnDevice(torch.Tensor):
    """A host tensor that says it lies on a GPU: enough for checks that come before any launch."""

    @staticmethod
    def make(t, index):
        t = t.as_subclass(OnDevice)
        t.index = index
        return t

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index


def bf16(index, *shape):
    return OnDevice.make(torch.zeros(shape, dtype=torch.bfloat16), index)


def weight(index, fmt="mxfp8", alpha_index=0):
    w = types.SimpleNamespace(fmt=fmt, N=64, K=128, packed=OnDevice.make(torch.zeros(64, dtype=torch.uint8), index))
    if fmt == "fp8":
        w.input_scale, w.alpha_dev = 0.5, OnDevice.make(torch.zeros(1), alpha_index)
    return w


@pytest.mark.parametrize("call", [fql.rms_norm_quant, fql.rms_norm_operand])
def test_norm_refuses_tensors_of_another_device(call):
    x = bf16(0, 4, 128)
    for name, args in (("weight", dict(weight=bf16(1, 128))), ("residual", dict(residual=bf16(1, 4, 128))),
                       ("residual_out", dict(residual=bf16(0, 4, 128), residual_out=bf16(1, 4, 128)))):
        args = {"weight": bf16(0, 128), **args}
        with pytest.raises(fql.FQLError, match=f"{name} must be on x's device"):
            call(x, fmt="mxfp8", **args)


def test_linear_refuses_tensors_of_another_device():
    x = bf16(0, 4, 128)
    op = fql.QuantizedActivation(OnDevice.make(torch.zeros(64, dtype=torch.uint8), 0), "mxfp8", (4,), 128)
    ws = OnDevice.make(torch.zeros(64, dtype=torch.uint8), 1)
    for a in (x, op):
        for name, w, args in (("weight", weight(1), {}), ("bias", weight(0), dict(bias=bf16(1, 64))),
                              ("residual", weight(0), dict(residual=bf16(1, 4, 64))),
                              ("out", weight(0), dict(out=bf16(1, 4, 64))),
                              ("workspace", weight(0), dict(out=bf16(0, 4, 64), workspace=ws))):
            with pytest.raises(fql.FQLError, match=f"{name} must be on x's device"):
                fql.linear_fused(a, w, **args)
    with pytest.raises(fql.FQLError, match="alpha_dev must be on x's device"):
        fql.linear_fused(x, weight(0, "fp8", 1), out=bf16(0, 4, 64), workspace=OnDevice.make(ws.as_subclass(torch.Tensor), 0))


def test_attention_refuses_a_workspace_of_another_device():
    def u8(*shape):
        return OnDevice.make(torch.zeros(shape, dtype=torch.uint8), 0)

    def i32(*values):
        return OnDevice.make(torch.tensor(values, dtype=torch.int32), 0)

    cache = fql.KVCache8(u8(2, 1, 16, 64), u8(2, 1, 1, 64, 16), u8(2, 1), u8(2, 1))
    q = bf16(0, 1, 2, 64)
    with pytest.raises(fql.FQLError, match="workspace must be on the cache's device"):
        fql.attention_kv8(q, cache, i32([0, 1]), i32(1), i32(0, 1), 1, out=bf16(0, 1, 2, 64),
                          workspace=OnDevice.make(torch.zeros(1 << 20, dtype=torch.uint8), 1))


# ---------------------------------------------------------------------------
# attention's output rows and its host arguments
# ---------------------------------------------------------------------------

def attend_out(tokens, heads, ld_token, ld_head):
    return fql.lib().fql_attention_kv8(
        ctypes.byref(cache()), ctypes.byref(batch(tokens=tokens, max_new=min(tokens, 2))), P, heads * 64, 64, heads, 0.1, 1,
        0, 64, P, ld_token, ld_head, NULL, P, 16, NULL)  # a workspace of 16 bytes: what passes is refused for that


@pytest.mark.parametrize("tokens", [1, 2, 5])
@pytest.mark.parametrize("heads", [2, 6])
def test_attention_refuses_output_rows_that_overlap(tokens, heads):
    D = 64
    for lt in (0, 1, 32, 63, 64, 65, 96, 128, 129, 160, 192, 320, 384, 400, 640):
        for lh in (0, 1, 48, 63, 64, 65, 96, 128, 192, 320, 321, 640):
            starts = sorted(t * lt + h * lh for t in range(tokens) for h in range(heads))
            apart = all(b - a >= D for a, b in zip(starts, starts[1:]))
            if apart:
                refused(attend_out(tokens, heads, lt, lh), "workspace", code=-4)
            else:
                refused(attend_out(tokens, heads, lt, lh), "overlap")
    big = 1 << 62  # no overflow on the way
    refused(attend_out(tokens, heads, big, 64), "workspace", code=-4)
    refused(attend_out(tokens, heads, 64 * heads, big), "workspace", code=-4)
    refused(attend_out(tokens, heads, big, 0), "overlap")


def test_attention_host_arguments_do_not_wrap(monkeypatch):
    """window and max_len reach the library as C integers: what those cannot hold is refused, and any
    kind of whole number is taken."""
    def u8(*shape):
        return OnDevice.make(torch.zeros(shape, dtype=torch.uint8), 0)

    def i32(*values):
        return OnDevice.make(torch.tensor(values, dtype=torch.int32), 0)

    c = fql.KVCache8(u8(2, 1, 16, 64), u8(2, 1, 1, 64, 16), u8(2, 1), u8(2, 1))
    args = (bf16(0, 1, 2, 64), c, i32([0, 1]), i32(1), i32(0, 1), 1)
    for bad in (2 ** 32, 2 ** 32 + 5, 2 ** 31, -1, -2 ** 40):
        with pytest.raises(fql.FQLError, match="window"):
            fql.attention_kv8(*args, out=bf16(0, 1, 2, 64), window=bad)
        with pytest.raises(fql.FQLError, match="window"):
            fql.attention_kv8_plan(1, 2, 1, 64, 1, 32, window=bad)
    for bad in (0, -1, 2 ** 64 + 5, 2 ** 31):
        with pytest.raises(fql.FQLError, match="max_len"):
            fql.attention_kv8(*args, out=bf16(0, 1, 2, 64), max_len=bad)
    # numpy's and torch's numbers: as far as the workspace, which is too small
    ws = u8(4096)
    monkeypatch.setattr(fql.serving, "_stream", lambda index: 0)
    for number in (np.int64, torch.tensor):
        with pytest.raises(fql.FQLError, match="workspace"):
            fql.attention_kv8(*args, out=bf16(0, 1, 2, 64), window=number(8), max_len=number(32), workspace=ws)


def test_a_replaced_workspace_is_given_back():
    """Growing keeps nothing of the old buffer: no graph uses an eager workspace."""
    key, device = ("cpu", None, -1), torch.device("cpu")
    try:
        sizes = []
        for need in (1 << 20, 3 << 20, 4 << 20, 1):
            old = fql._workspaces.get(key)
            gone = [] if old is None else [weakref.ref(old)]
            sizes.append(fql._grow_workspace(key, need, device).numel())
            del old
            assert all(r() is None for r in gone)
        assert sizes == [1 << 20, 3 << 20, 6 << 20, 12 << 20]
    finally:
        fql._workspaces.pop(key, None)


@pytest.mark.parametrize("M", [1, 4, 40])
def test_linear_refuses_an_output_that_overlaps_its_input(M):
    """x [M, 128] and y [M, 64] at distances (in elements) and strides where they share elements."""
    def at(offset):
        return ctypes.c_void_p((1 << 20) + 2 * offset)

    def call(y, ldx, ldy):
        return fql.lib().fql_linear_fused(fql.FMT_MXFP8, at(0), M, 128, ldx, 0.0, NULL, ctypes.c_void_p(1 << 24), 64, 1.0, NULL,
                                          NULL, 0, NULL, 0, at(y), ldy, ctypes.c_void_p(1 << 25), 1 << 26, NULL)

    for y, ldx, ldy in ((0, 128, 64), (127, 128, 64), (-63, 128, 64), (0, 128, 128), (64, 192, 192)):
        refused(call(y, ldx, ldy), "overlaps")
    if M > 1:
        for y, ldx, ldy in ((192 - 1, 192, 192), (-64, 191, 191), (128 + 1, 192, 192), (130, 192, 200), (191, 256, 64)):
            refused(call(y, ldx, ldy), "overlaps")


def test_outputs_that_are_an_input_shifted_are_refused():
    """h_out may be x or residual itself and y may be residual itself, not a neighbouring row or column of it."""
    def at(offset):
        return ctypes.c_void_p((1 << 20) + 2 * offset)

    far = ctypes.c_void_p(1 << 28)
    for h, ldh in ((1, 256), (256, 256), (-256, 256), (0, 257), (300, 512), (255, 511)):
        for args in (dict(x=at(0), res=far), dict(x=far, res=at(0))):
            refused(norm(**args, h=at(h), ldh=ldh), "h_out overlaps")
    for y, ldy in ((1, 64), (64, 64), (-64, 64), (0, 65), (80, 128)):
        refused(linear(x=far, res=at(0), ldr=64, y=at(y), ldy=ldy), "y overlaps")
    # itself, as far as the next check
    for args in (dict(x=at(0), res=far), dict(x=far, res=at(0)), dict(x=at(0), res=at(0))):
        refused(norm(**args, h=at(0), fmt=FP8, scale=0.0), "scale")
    refused(linear(x=at(0), ldx=256, res=at(0), ldr=64, y=at(0)), "y overlaps x")
