"""Tensors of the linear calls (CPU): host tensors that say they lie on a GPU, and a library that is not called. A
refused call must not reach it, since the kernels write and read at the addresses that they are given."""

import types

import pytest
import torch

import fp8_quantized_linear_amd as fql
from test_packing_api import FMTS, Gpu0, Gpu1, on

M, N, K = 6, 64, 128
LINEAR = {f: getattr(fql, f"linear_{f}") for f in FMTS}


def bf16(*shape, kind=Gpu0):
    return on(kind, torch.zeros(shape, dtype=torch.bfloat16))


def u8(n, kind=Gpu0):
    return on(kind, torch.empty(n, dtype=torch.uint8))


def weight(fmt, kind=Gpu0, alpha_kind=Gpu0):
    w = types.SimpleNamespace(fmt=fmt, N=N, K=K, packed=u8(64, kind), hadamard_block=0, transform=None,
                              input_global_scale=1.0, weight_global_scale=1.0, input_scale=1.0, alpha=1.0)
    if fmt in ("nvfp4", "fp8"):
        w.alpha_dev = on(alpha_kind, torch.zeros(1))
    return w


@pytest.fixture
def calls(monkeypatch):
    made = []
    real = fql.lib()

    class Lib:
        def __getattr__(self, name):
            if not name.startswith("fql_linear_") or name.endswith("_bytes"):
                return getattr(real, name)
            return lambda *args: made.append(name) or 0

    handle = Lib()
    monkeypatch.setattr(fql, "lib", lambda: handle)
    monkeypatch.setattr(fql, "_stream", lambda device=None: None)
    return made


@pytest.mark.parametrize("fmt", FMTS)
def test_outputs_of_another_shape_or_type_are_refused(fmt, calls):
    """The kernel writes M rows of N bf16 values whatever the output is."""
    x, ws = bf16(2, 3, K), u8(1 << 20)
    for out in (bf16(2, 3, N - 1), bf16(M - 1, N), bf16(M, N + 1), bf16(2, 2, N), bf16(N), bf16(M, N).to(torch.float32),
                bf16(M, N).to(torch.int8)):
        with pytest.raises(fql.FQLError, match="out must"):
            LINEAR[fmt](x, weight(fmt), out=out, workspace=ws)
    if fmt == "nvfp4":
        for call in (lambda out: fql.linear_nvfp4_noalloc(x, weight(fmt), out),
                     lambda out: fql.linear_nvfp4_gemm(M, weight(fmt), ws, 1.0, out=out)):
            for out in (bf16(M - 1, N), bf16(M, N).to(torch.float32)):
                with pytest.raises(fql.FQLError, match="out must"):
                    call(out)
    assert calls == []
    for out in (bf16(2, 3, N), bf16(M, N), bf16(M, N + 5)[:, :N]):
        assert LINEAR[fmt](x, weight(fmt), out=out, workspace=ws) is out
    assert len(calls) == 3


@pytest.mark.parametrize("fmt", FMTS)
def test_tensors_of_another_device_are_refused(fmt, calls):
    """The kernel would use an address that is the host's or another GPU's."""
    x, out, ws = bf16(M, K), bf16(M, N), u8(1 << 20)
    good = dict(weight=weight(fmt), out=out, workspace=ws, bias=bf16(N))
    for kind in (torch.Tensor, Gpu1):
        bad = [("weight", weight(fmt, kind=kind)), ("out", bf16(M, N, kind=kind)), ("workspace", u8(1 << 20, kind)),
               ("bias", bf16(N, kind=kind))]
        for name, t in bad:
            with pytest.raises(fql.FQLError, match=f"{name} must be"):
                LINEAR[fmt](x, **{**good, name: t})
        if fmt in ("nvfp4", "fp8"):
            with pytest.raises(fql.FQLError, match="alpha_dev must be"):
                LINEAR[fmt](x, **{**good, "weight": weight(fmt, alpha_kind=kind)})
        if fmt == "nvfp4":
            for name, t in bad:
                if name != "workspace":
                    with pytest.raises(fql.FQLError, match=f"{name} must be"):
                        fql.linear_nvfp4_noalloc(x, **{**{k: v for k, v in good.items() if k != "workspace"}, name: t})
    assert calls == []
    assert LINEAR[fmt](x, **good) is out and len(calls) == 1
