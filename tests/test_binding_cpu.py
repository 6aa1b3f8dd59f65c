"""The library handle of load_library: the C signatures as ctypes types."""

import ctypes

import pytest
import torch

from moe_grouped_gemm_x128_amd import binding


def _tensors():
    x, q, sf = torch.zeros(4, 256), torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 3)  # (one scale too many)
    return [binding.describe(t) for t in (x, q, sf)]


@pytest.mark.parametrize("how", [lambda d: d, ctypes.byref, ctypes.pointer])
def test_descriptors_by_structure_reference_and_pointer(how):
    lib = binding.load_library()
    x, q, sf = (how(d) for d in _tensors())
    assert lib.per_token_cast_to_fp8(x, q, sf, 0, None) == binding.DG_INVALID_ARG
    assert b"sf" in lib.dg_last_error()
    assert lib.moe_combine(x, None, None, None, None) == binding.DG_INVALID_ARG


@pytest.mark.parametrize("wrong", [12345, b"not a descriptor", ctypes.c_void_p(12345), ctypes.byref(ctypes.c_int(0))])
def test_what_is_no_descriptor_is_refused(wrong):
    lib = binding.load_library()
    x, q, _ = _tensors()
    with pytest.raises(ctypes.ArgumentError):
        lib.per_token_cast_to_fp8(x, q, wrong, 0, None)
    for name in ("moe_route_topk_bwd", "paged_attention_fp8", "kv_append_fp8"):
        fn = getattr(lib, name)
        args = [wrong] + [0 if t in (ctypes.c_int, ctypes.c_int32, ctypes.c_float) else None for t in fn.argtypes[1:]]
        with pytest.raises(ctypes.ArgumentError):
            fn(*args)


def test_a_library_of_its_own_path():
    lib = binding.load_library(binding.LIB_PATH)
    assert lib.per_token_cast_to_fp8(*_tensors(), 0, None) == binding.DG_INVALID_ARG
