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


# ------------------------------------------------------- rows, columns and elements
class NoStream:  # the null stream, without asking CUDA for the current one
    cuda_stream = 0


def i32(n):
    return torch.zeros(n, dtype=torch.int32)


def i8(*s):
    return torch.zeros(*s, dtype=torch.int8)


def refuses(f, good, **bad):
    """f(**good, changed by one of bad) names the operand that is too small."""
    for name, values in bad.items():
        for v in values:
            with pytest.raises(ValueError, match=name + "(:| is| has)"):
                f(stream=NoStream, **dict(good, **{name: v}))


def test_act8_rows():
    x = bf(8, 72)
    refuses(L.moe_act8_quantize, dict(x=x, q=i8(8, 72), scales=bf(8, 3)), q=[i8(7, 72), i8(8, 128)[:, :64]],
            scales=[bf(7, 3), bf(1, 3), bf(8, 4)[:, :2]], group_offsets=[i32(6)[::2]])
    refuses(L.moe_act8_dequantize, dict(x=x, q=i8(8, 72), scales=bf(8, 3)), q=[i8(7, 72)],
            scales=[bf(7, 3)])
    good = dict(h=bf(8, 144), act=bf(8, 72), q=i8(8, 144), scales=bf(8, 6))
    refuses(L.moe_act8_swiglu_fwd, good, h=[bf(7, 144), bf(8, 200)[:, :72]], q=[i8(5, 144)],
            scales=[bf(7, 6), bf(8, 6)[:, :5]])
    good = dict(q=i8(8, 144), scales=bf(8, 6), dact=bf(8, 72), dh=bf(8, 144), act=bf(8, 72))
    refuses(L.moe_act8_swiglu_bwd, good, q=[i8(5, 144)], scales=[bf(7, 6)], dh=[bf(7, 144)],
            act=[bf(7, 72), bf(8, 144)[:, :64]])


@pytest.mark.parametrize("fmt", [0, 1])
def test_fp4_rows(fmt):
    nb = L.moe_fp4_scale_bytes(8, 64, fmt, L.FP4_ROWS_GROUPED, 2)
    good = dict(x=bf(8, 64), fmt=fmt, q=u8(8, 32), sf=u8(nb), group_offsets=i32(3))
    refuses(L.moe_fp4_quantize, good, row_index=[i32(0), i32(7), i32(16)[::2]], sf=[u8(2 * nb)[::2]],
            workspace=[u8(8192)[::2]], dev_status=[i32(0)], q=[u8(8, 64)[:, :16]])
    good = dict(q=u8(8, 32), sf=u8(nb), fmt=fmt, x=bf(8, 64), group_offsets=i32(3))
    refuses(L.moe_fp4_dequantize, good, q=[u8(7, 32)], sf=[u8(2 * nb)[::2]])
    nw = L.moe_fp4_scale_bytes(2 * 64, 64, fmt, L.FP4_ROWS_EXPERTS, 2)
    w = dict(row_map=L.FP4_ROWS_EXPERTS, groups=2)
    if fmt == L.FP4_NV:  # one scale an expert
        refuses(L.moe_fp4_quantize, dict(w, x=bf(128, 64), fmt=fmt, q=u8(128, 32), sf=u8(nw)), scale=[f32(1)])
        refuses(L.moe_fp4_dequantize, dict(w, x=bf(128, 64), fmt=fmt, q=u8(128, 32), sf=u8(nw)),
                scale=[f32(1)])


def test_weights_and_products():
    w = dict(w=bf(2, 64, 128), fmt=1, row_map=L.FP4_ROWS_EXPERTS, q=u8(2, 128, 32), sf=u8(1 << 16))
    refuses(L.moe_fp4_quantize_weights, w, q=[u8(1, 128, 32)], scale=[f32(1)])
    nb = L.moe_fp4_scale_bytes
    A = dict(A=u8(8, 32), sfa=u8(nb(8, 64, 1, L.FP4_ROWS_GROUPED, 2)), B=u8(2, 128, 32),
             sfb=u8(nb(256, 64, 1, L.FP4_ROWS_EXPERTS, 2)), fmt=1, group_offsets=i32(3), C=bf(8, 128))
    refuses(L.moe_gmm_fp4, A, sfa=[u8(512)], sfb=[u8(512)], group_offsets=[i32(2), i32(6)[::2]],
                C=[bf(7, 128), bf(8, 256)[:, :120]], b_scale=[f32(1), f32(4)[::2]])
    A.update(C=None, epilogue=L.EPI_SWIGLU_FWD, Q2=u8(8, 32), sf2=u8(1 << 16),
             sfb=u8(nb(256, 64, 1, L.FP4_ROWS_SWIGLU, 2)))
    refuses(L.moe_gmm_fp4, A, Q2=[u8(7, 32)], C=[bf(7, 128)], sf2=[u8(1 << 17)[::2]], sfb=[u8(512)])


def test_experts_call():
    w = experts()
    arg = L.Fp4BuffersArg(12)  # of 12 rows
    call = lambda x, s2f, off: L.moe_fp4_experts(w.arg, arg, x, s2f, 2, off, NoStream)  # noqa: E731
    for x, s2f, off in ((bf(6, D)[:, :32], i32(12), i32(E + 1)), (bf(6, D), i32(11), i32(E + 1)),
                        (bf(6, D), i32(12), i32(E)), (bf(6, D), i32(24)[::2], i32(E + 1))):
        with pytest.raises(ValueError, match="x is|sorted_to_flat|group_offsets"):
            call(x, s2f, off)


# ------------------------------------------------------------------------- types
def test_types_of_the_native_calls():
    """Elements of another type would be read as bf16, int32 or fp32."""
    i64 = lambda n: i32(n).long()  # noqa: E731
    a = dict(x=bf(8, 64), q=i8(8, 64), scales=bf(8, 2), group_offsets=i32(3))
    refuses(L.moe_act8_quantize, a, x=[f32(8, 64), bf(8, 64).half()], q=[f32(8, 64)],
            scales=[f32(8, 2)], group_offsets=[i64(3)])
    refuses(L.moe_act8_dequantize, a, x=[f32(8, 64)], q=[bf(8, 64)], scales=[f32(8, 2)])
    a = dict(h=bf(8, 128), act=bf(8, 64), q=i8(8, 128), scales=bf(8, 4))
    refuses(L.moe_act8_swiglu_fwd, a, h=[f32(8, 128)], act=[f32(8, 64)], q=[i32(1024).view(8, 128)],
            scales=[bf(8, 4).half()])
    a = dict(q=i8(8, 128), scales=bf(8, 4), dact=bf(8, 64), dh=bf(8, 128), act=bf(8, 64))
    refuses(L.moe_act8_swiglu_bwd, a, q=[f32(8, 128)], scales=[f32(8, 4)], dact=[f32(8, 64)],
            dh=[f32(8, 128)], act=[f32(8, 64)])
    sf = u8(L.moe_fp4_scale_bytes(8, 64, 1, 1, 2))
    a = dict(x=bf(8, 64), fmt=1, q=u8(8, 32), sf=sf, group_offsets=i32(3))
    refuses(L.moe_fp4_quantize, a, x=[f32(8, 64)], q=[bf(8, 32)], sf=[sf.float()],
            group_offsets=[i64(3)], row_index=[i64(8)], scale=[f32(1).double(), bf(1)],
            dev_status=[i64(1)])
    refuses(L.moe_fp4_dequantize, a, x=[f32(8, 64)], q=[f32(8, 32)], sf=[sf.float()], scale=[bf(1)])
    w, arg = experts(), L.Fp4BuffersArg(12)
    for x, s2f, off in ((f32(6, D), i32(12), i32(E + 1)), (bf(6, D), i64(12), i32(E + 1)),
                        (bf(6, D), i32(12), i64(E + 1))):
        with pytest.raises(ValueError, match="is torch"):
            L.moe_fp4_experts(w.arg, arg, x, s2f, 2, off, NoStream)


def test_codes_are_any_bytes():
    """What checkpoints call them does not matter: no work here, and no refusal either."""
    L.moe_act8_quantize(bf(0, 64), u8(0, 64), bf(0, 2), stream=NoStream)
    L.moe_fp4_dequantize(i8(0, 32), torch.zeros(0, dtype=torch.float8_e4m3fn), 1, bf(0, 64),
                         group_offsets=i32(3), stream=NoStream)


def test_types_of_weights_and_products():
    w = dict(w=bf(2, 64, 128), fmt=1, row_map=L.FP4_ROWS_EXPERTS, q=u8(2, 128, 32), sf=u8(1 << 16))
    refuses(L.moe_fp4_quantize_weights, w, w=[f32(2, 64, 128)], q=[f32(2, 128, 32)], scale=[bf(2)])
    refuses(L.moe_fp4_arrange_scales, dict(scales=u8(128, 4), cols=64, fmt=1, row_map=3, E=1, sf=u8(4096)),
            scales=[f32(128, 4)], sf=[f32(4096)])
    nb = L.moe_fp4_scale_bytes
    a = dict(A=u8(8, 32), sfa=u8(nb(8, 64, 1, L.FP4_ROWS_GROUPED, 2)), B=u8(2, 128, 32),
             sfb=u8(nb(256, 64, 1, L.FP4_ROWS_EXPERTS, 2)), fmt=1, group_offsets=i32(3), C=bf(8, 128))
    refuses(L.moe_gmm_fp4, a, A=[bf(8, 32)], B=[bf(2, 128, 32)], C=[bf(8, 128).half()],
            group_offsets=[i32(3).long()], a_scale=[bf(1)], b_scale=[bf(2)], dev_status=[i32(1).long()])


def test_types_of_the_serving_layer():
    from mixture_experts_grouped_router_gb300 import layer
    m = lowbit.Fp4Layer(experts(), layer.LayerShape(8, D, F, E, 2))
    for x, logits, bias in ((f32(4, D), f32(4, E), None), (bf(4, D), bf(4, E), None),
                            (bf(4, D), f32(4, E), bf(E)), (bf(4, D), f32(4, E), f32(1)),
                            (bf(4, D + 32)[:, :32], f32(4, E), None)):
        with pytest.raises(ValueError, match="is torch|x is|expert_bias"):
            m.forward(x, logits, expert_bias=bias, stream=NoStream)


@pytest.mark.parametrize("option", [dict(fp8=True), dict(mxfp8=True), dict(num_chunks=2),
                                    dict(aux_coeff=1e-3), dict(bias=True)])
def test_the_serving_layer_refuses_what_it_does_not_serve(option):
    from mixture_experts_grouped_router_gb300 import layer
    with pytest.raises(ValueError, match=list(option)[0]):
        lowbit.Fp4Layer(experts(), layer.LayerShape(8, D, F, E, 2, **option))


def test_tensors_are_not_exchanged_behind_the_calls_arguments():
    """A scale calibrated anew goes into the tensor: the calls hold its address."""
    w = experts()
    b = lowbit.Fp4Buffers(w, 12, save_h=True)
    for o, names in ((w, ("x_scale", "act_scale", "wi_q", "wo_sf", "fmt")), (b, ("h", "y", "x", "rows_cap"))):
        for n in names:
            with pytest.raises(AttributeError, match=n):
                setattr(o, n, getattr(o, n))
    w.x_scale.fill_(2.0)
    assert w.arg.x_scale == w.x_scale.data_ptr() and b.arg.y == b.y.data_ptr()
