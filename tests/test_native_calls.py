"""The native module's argument marshalling, without a GPU: what it refuses itself, and
what it hands on for the library to refuse (nothing of either reaches a launch)."""
import gc
import sys

import pytest
import torch

from mixture_experts_grouped_router_gb300 import _lib as L
from mixture_experts_grouped_router_gb300 import _native


class NoStream:  # the null stream, without asking CUDA for the current one
    cuda_stream = 0


def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def q8(*s):
    return torch.zeros(*s, dtype=torch.int8)


def test_tensors_are_row_major_matrices():
    with pytest.raises(AssertionError, match="row-major"):
        _native.act8_quantize(bf(64, 8).t(), q8(8, 64), bf(8, 2), None, 0)
    with pytest.raises(AssertionError, match="matrices"):
        _native.act8_quantize(bf(8, 64), q8(512), bf(8, 2), None, 0)
    with pytest.raises(ValueError, match="matrices"):
        _native.act8_quantize(bf(2, 8, 64), q8(8, 64), bf(8, 2), None, 0)


@pytest.mark.parametrize("bad", [None, 3, "x", object()])
def test_what_is_no_tensor(bad):
    with pytest.raises(AttributeError):
        _native.act8_quantize(bad, q8(8, 64), bf(8, 2), None, 0)
    with pytest.raises(AttributeError):
        _native.act8_dequantize(q8(8, 64), bf(8, 2), bad, None, 0)


def test_numbers():
    with pytest.raises(TypeError):
        _native.act8_quantize(bf(8, 64), q8(8, 64), bf(8, 2), None, "0")
    with pytest.raises(TypeError, match="5 arguments"):
        _native.act8_quantize(bf(8, 64), q8(8, 64), bf(8, 2), None)
    sf = torch.zeros(L.moe_fp4_scale_bytes(8, 64, 0, 3), dtype=torch.uint8)
    q = torch.zeros(8, 32, dtype=torch.uint8)
    with pytest.raises(OverflowError):
        _native.fp4_quantize(bf(8, 64), 2 ** 40, q, sf, 3, None, 1, None, 1, None, None, None, 0)
    with pytest.raises(TypeError):
        _native.fp4_dequantize(q, sf, 0.5, bf(8, 64), 3, None, 1, None, 0)


def test_the_library_refuses_the_rest():
    with pytest.raises(L.MoEError, match="too small") as e:
        L.moe_act8_swiglu_fwd(bf(8, 64), bf(8, 32), q8(8, 32), bf(8, 2),
                              stream=NoStream)  # codes of half of h
    assert e.value.status == L.MOE_ERR_INVALID_ARG
    with pytest.raises(L.MoEError, match="bad fmt") as e:
        L.moe_fp4_quantize(bf(8, 64), 7, torch.zeros(8, 32, dtype=torch.uint8),
                           torch.zeros(4096, dtype=torch.uint8), row_map=L.FP4_ROWS_EXPERTS, stream=NoStream)
    assert e.value.status == L.MOE_ERR_INVALID_ARG


def test_empty_matrices_are_no_work():
    L.moe_act8_quantize(bf(0, 64), q8(0, 64), bf(0, 2), stream=NoStream)
    L.moe_act8_swiglu_bwd(q8(0, 64), bf(0, 2), bf(0, 32), bf(0, 64), stream=NoStream)
    L.moe_fp4_quantize(bf(4, 64), 1, torch.zeros(0, 32, dtype=torch.uint8),
                       torch.zeros(0, dtype=torch.uint8), group_offsets=torch.zeros(3, dtype=torch.int32),
                       stream=NoStream)


def test_no_reference_is_lost_or_kept():
    x, q, s = bf(0, 64), q8(0, 64), bf(0, 2)
    bad = bf(64, 8).t()
    before = [sys.getrefcount(t) for t in (x, q, s, bad)]
    for _ in range(100):
        L.moe_act8_quantize(x, q, s, stream=NoStream)
        with pytest.raises(AssertionError):
            _native.act8_quantize(bad, q8(8, 64), bf(8, 2), None, 0)
    gc.collect()
    assert [sys.getrefcount(t) for t in (x, q, s, bad)] == before
