"""What the low-bit calls refuse by their operands' shapes and types, before anything is
launched: a matrix of too few rows or another type would be read or written past its end.
On the host, with tensors of its memory."""
import pytest
import torch

from mixture_experts_grouped_router_gb300 import _lib as L
from mixture_experts_grouped_router_gb300 import lowbit

E, D, F = 3, 64, 96


def u8(*s):
    return torch.zeros(*s, dtype=torch.uint8)


def f32(*s):
    return torch.zeros(*s)


def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


# ------------------------------------------------------------ a checkpoint's codes
def codes(fmt, **change):
    blk = 16 if fmt == "nv" else 32
    a = dict(wi_q=u8(E, 2 * F, D // 2), wi_s=u8(E, 2 * F, D // blk), wi_scale=f32(E),
             wo_q=u8(E, D, F // 2), wo_s=u8(E, D, F // blk), wo_scale=f32(E))
    a.update(change)
    return lowbit.Fp4Experts.from_codes(fmt, **a)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_from_codes_scales(fmt):
    blk, other = (16, 32) if fmt == "nv" else (32, 16)
    for name, rows, cols in (("wi_s", 2 * F, D), ("wo_s", D, F)):
        for bad in (u8(E, rows, cols // other),          # the other format's
                    u8(E, rows // 2, 2 * cols // blk),   # as many bytes in other rows
                    u8(E * rows, cols // blk), u8(E + 1, rows, cols // blk),
                    torch.zeros(E, rows, cols // blk, dtype=torch.bfloat16),
                    u8(E, cols // blk, rows).transpose(1, 2)):
            with pytest.raises(ValueError, match=name):
                codes(fmt, **{name: bad})


def test_from_codes_codes():
    for name, bad in (("wi_q", u8(E, 2 * F, D)), ("wi_q", u8(E, F, D // 2)), ("wi_q", f32(E, 2 * F, D // 2)),
                      ("wo_q", u8(E * D, F // 2)), ("wo_q", u8(E, F // 2, D).transpose(1, 2))):
        with pytest.raises(ValueError, match="w[io]_q"):
            codes("mx", **{name: bad})


def test_arranged_scales_are_whole_rows():
    with pytest.raises(ValueError, match="no rows of 4"):
        L.moe_fp4_arrange_scales(u8(67), 64, L.FP4_NV, L.FP4_ROWS_EXPERTS, 1, u8(4096))
