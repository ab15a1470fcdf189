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


def experts(**change):
    nb = L.moe_fp4_scale_bytes
    a = dict(fmt=L.FP4_NV, wi_q=u8(E, 2 * F, D // 2),
             wi_sf=u8(nb(E * 2 * F, D, L.FP4_NV, L.FP4_ROWS_SWIGLU, E)), wi_scale=f32(E),
             wo_q=u8(E, D, F // 2), wo_sf=u8(nb(E * D, F, L.FP4_NV, L.FP4_ROWS_EXPERTS, E)),
             wo_scale=f32(E), x_scale=f32(1), act_scale=f32(1))
    a.update(change)
    return lowbit.Fp4Experts(**a)


def test_experts():
    w = experts()
    assert (w.E, w.d, w.f) == (E, D, F)
    experts(wi_scale=None, wo_scale=None, x_scale=None, act_scale=None)
    for name in ("wi_scale", "wo_scale"):  # one for all experts would be read past its end
        for bad in (f32(1), f32(E + 1), f32(E).double(), f32(E).bfloat16(), f32(2 * E)[::2]):
            with pytest.raises(ValueError, match=name):
                experts(**{name: bad})
    for name in ("x_scale", "act_scale"):
        for bad in (f32(E), f32(1).half(), f32(0)):
            with pytest.raises(ValueError, match=name):
                experts(**{name: bad})
    for name in ("wi_sf", "wo_sf"):
        for bad in (u8(512), f32(1 << 20), u8(1 << 20)[::2], u8(1024, 1024)):
            with pytest.raises(ValueError, match=name):
                experts(**{name: bad})
    with pytest.raises(ValueError, match="fmt"):
        experts(fmt="nv")
    with pytest.raises(ValueError, match="one device"):
        experts(x_scale=torch.empty(1, device="meta"))


def test_from_weights():
    make = lowbit.Fp4Experts.from_weights
    for wi, wo in ((bf(E, D, F), bf(E, F, D)), (bf(E, D, 2 * F), bf(E, F, D).half()),
                   (bf(E, D, 2 * F).float(), bf(E, F, D)), (bf(E, 2 * F, D).transpose(1, 2), bf(E, F, D)),
                   (bf(E + 1, D, 2 * F), bf(E, F, D)), (bf(E, D, 2 * F), bf(F, D))):
        with pytest.raises(ValueError, match="w[io]: "):
            make("mx", wi, wo)


def test_arranged_scales_are_whole_rows():
    with pytest.raises(ValueError, match="no rows of 4"):
        L.moe_fp4_arrange_scales(u8(67), 64, L.FP4_NV, L.FP4_ROWS_EXPERTS, 1, u8(4096))
