"""Arguments of the weight packers (CPU): host tensors that say they lie on a GPU, and a library that is not
called. A refused call must not reach it, since the kernels take addresses as they come."""

import pytest
import torch

import fp8_quantized_linear_amd as fql


class Gpu0(torch.Tensor):
    """A host tensor that says it lies on the first GPU, and so do its views."""
    index = 0
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index


class Gpu1(Gpu0):
    index = 1


N, K = 128, 128  # (small: torch starts no threads, which other tests' forked workers would inherit halfway)


def on(kind, t):
    return t.as_subclass(kind)


def operands(fmt, kind=Gpu0):
    """Well-formed (codes, scales) of an [N, K] weight; per-tensor FP8: no scales."""
    u8 = torch.uint8
    codes = torch.zeros((N, K // 2 if fmt in ("nvfp4", "mxfp4") else K), dtype=torch.int8 if fmt == "int8" else u8)
    scales = {"nvfp4": torch.zeros((N, K // 16), dtype=u8), "mxfp4": torch.zeros((N, K // 32), dtype=u8),
              "mxfp8": torch.zeros((N, K // 32), dtype=u8), "fp8": None, "int8": torch.zeros(N),
              "fp8_block": torch.zeros((N // 128, K // 128))}[fmt]
    return on(kind, codes), None if scales is None else on(kind, scales)


def storage(fmt, kind=Gpu0):
    return on(kind, torch.empty(fql._size_query(f"fql_packed_{fmt}_bytes", N, K), dtype=torch.uint8))


def pack(fmt, codes, scales, out):
    args = (codes,) if fmt == "fp8" else (codes, scales)
    return getattr(fql, f"pack_weight_{fmt}")(*args, out=out)


FMTS = ("nvfp4", "mxfp4", "mxfp8", "fp8", "fp8_block", "int8")
SCALED = tuple(f for f in FMTS if f != "fp8")


def weight(fmt, kind=Gpu0):
    cls = {"nvfp4": fql.NVFP4Weight, "mxfp4": fql.MXFP4Weight, "mxfp8": fql.MXFP8Weight, "fp8": fql.FP8Weight,
           "fp8_block": fql.FP8BlockWeight, "int8": fql.INT8Weight}[fmt]
    w = cls.__new__(cls)  # what repack_ reads, without a device scalar
    w.packed, w.N, w.K, w.weight_global_scale = storage(fmt, kind), N, K, 1.0
    return w


def experts(fmt, kind=Gpu0):
    size = -(-storage(fmt).numel() // 256) * 256
    args = dict(input_scale=0.5, alpha=on(kind, torch.zeros(2))) if fmt == "fp8" else {}
    return fql.ExpertWeight(fmt, on(kind, torch.empty((2, size), dtype=torch.uint8)), N, K, **args)


@pytest.fixture
def calls(monkeypatch):
    """The library calls of packers that would have been made; none reaches the library."""
    made = []

    def stub(name):
        def call(*args):
            made.append(name)
            return 0
        return call

    real = fql.lib()

    class Lib:
        def __getattr__(self, name):
            return stub(name) if "pack_weight" in name else getattr(real, name)

    handle = Lib()
    monkeypatch.setattr(fql, "lib", lambda: handle)
    monkeypatch.setattr(fql, "_stream", lambda device=None: None)
    return made


@pytest.mark.parametrize("fmt", FMTS)
def test_well_formed_calls_reach_the_library(fmt, calls):
    out = storage(fmt)
    assert pack(fmt, *operands(fmt), out) is out
    w = weight(fmt)
    codes, scales = operands(fmt)
    assert w.repack_(codes, scales) is w
    assert calls == [f"fql_pack_weight_{fmt}"] * 2
    if fmt != "nvfp4":
        g = experts(fmt)
        assert g.repack_(1, codes, 0.25 if fmt == "fp8" else scales) is g
        assert len(calls) == 3


@pytest.mark.parametrize("fmt", SCALED)
@pytest.mark.parametrize("where", ("host", "another GPU"))
def test_scales_of_another_device_are_refused(fmt, where, calls):
    """The packing kernel would read them at an address of the host, or of another GPU."""
    codes, _ = operands(fmt)
    scales = operands(fmt, torch.Tensor if where == "host" else Gpu1)[1]
    bad = [lambda: pack(fmt, codes, scales, storage(fmt)), lambda: weight(fmt).repack_(codes, scales),
           lambda: weight(fmt).repack_(codes, None)]
    if fmt != "nvfp4":
        bad.append(lambda: experts(fmt).repack_(0, codes, scales))
    for call in bad:
        with pytest.raises(fql.FQLError, match="scales must be"):
            call()
    assert calls == []


@pytest.mark.parametrize("fmt", FMTS)
def test_storage_of_another_device_or_with_gaps_is_refused(fmt, calls):
    """The packing kernel would write through an address that is not its device's, or over the gaps of a view."""
    codes, scales = operands(fmt)
    n = storage(fmt).numel()
    for out in (on(torch.Tensor, storage(fmt)), storage(fmt, Gpu1), on(Gpu0, torch.empty(2 * n, dtype=torch.uint8))[::2]):
        with pytest.raises(fql.FQLError, match="out must be"):
            pack(fmt, codes, scales, out)
    with pytest.raises(fql.FQLError, match="out must be"):
        weight(fmt, Gpu1).repack_(codes, scales)
    if fmt != "nvfp4":
        with pytest.raises(fql.FQLError, match="out must be"):
            experts(fmt, Gpu1).repack_(0, codes, 0.25 if fmt == "fp8" else scales)
    assert calls == []


@pytest.mark.parametrize("fmt", ("nvfp4", "mxfp4", "mxfp8", "fp8", "fp8_block"))
def test_codes_of_wider_types_are_refused(fmt, calls):
    """Their first bytes would be packed as codes."""
    codes, scales = operands(fmt)
    for dtype in (torch.bfloat16, torch.float32, torch.int32, torch.float8_e5m2, torch.float8_e4m3fnuz):
        wide = codes.to(dtype)
        bad = [lambda: pack(fmt, wide, scales, storage(fmt)), lambda: weight(fmt).repack_(wide, scales)]
        if fmt != "nvfp4":
            bad.append(lambda: experts(fmt).repack_(0, wide, 0.25 if fmt == "fp8" else scales))
            bad.append(lambda: fql.ExpertWeight.from_codes(fmt, torch.stack([wide] * 2), torch.stack([codes] * 2)))
        for call in bad:
            with pytest.raises(fql.FQLError, match="codes must be"):
                call()
    assert calls == []
    bytes_ = [torch.uint8, torch.int8] + ([torch.float8_e4m3fn] if "fp8" in fmt else [])
    for dtype in bytes_:
        pack(fmt, codes.view(dtype), scales, storage(fmt))
    assert len(calls) == len(bytes_)


@pytest.mark.parametrize("fmt", ("nvfp4", "mxfp4", "mxfp8"))
def test_one_byte_scales_of_another_type_are_refused(fmt, calls):
    """A checkpoint's scales as float32, of the right shape, would be packed byte by byte."""
    codes, scales = operands(fmt)
    own = torch.float8_e4m3fn if fmt == "nvfp4" else torch.float8_e8m0fnu
    other = torch.float8_e8m0fnu if fmt == "nvfp4" else torch.float8_e4m3fn
    for wide in (scales.to(torch.float32), scales.to(torch.bfloat16), scales.to(torch.int32), scales.view(other)):
        bad = [lambda: pack(fmt, codes, wide, storage(fmt)), lambda: weight(fmt).repack_(codes, wide)]
        if fmt != "nvfp4":
            bad.append(lambda: experts(fmt).repack_(0, codes, wide))
            bad.append(lambda: fql.ExpertWeight.from_codes(fmt, torch.stack([codes] * 2), torch.stack([wide] * 2)))
        for call in bad:
            with pytest.raises(fql.FQLError, match="scales must be"):
                call()
    assert calls == []
    for dtype in (torch.uint8, own):
        pack(fmt, codes, scales.view(dtype), storage(fmt))
    assert len(calls) == 2


@pytest.mark.parametrize("fmt", FMTS)
def test_codes_that_are_no_matrix_are_refused(fmt, calls):
    """The codes of several experts, or one row's, are no [N, K] weight."""
    codes, scales = operands(fmt)
    for bad in (torch.stack([codes, codes]), codes[0]):
        with pytest.raises(fql.FQLError, match="codes must have two dimensions"):
            pack(fmt, bad, scales, storage(fmt))
        with pytest.raises(fql.FQLError, match="codes must"):
            weight(fmt).repack_(bad, scales)
    assert calls == []


@pytest.mark.parametrize("fmt", FMTS)
def test_repacking_another_shape_is_refused(fmt, calls):
    """A smaller weight fits the storage, whose layout goes by the old shape."""
    codes, scales = operands(fmt)
    half = codes[:N // 2].contiguous(), None if scales is None else scales[:(scales.shape[0]) // 2].contiguous()
    narrow = codes[:, :codes.shape[1] // 2].contiguous(), (
        None if scales is None else scales if fmt == "int8" else scales[:, :scales.shape[1] // 2].contiguous())
    for bad in (half, narrow):
        with pytest.raises(fql.FQLError, match="codes must be"):
            weight(fmt).repack_(*bad)
    assert calls == []
