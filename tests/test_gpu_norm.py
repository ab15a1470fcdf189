"""RMS norm with the residual's addition and 8-bit outputs, and its backward, against the fp64
oracle.  Tolerances: the one rounding of a result (half its type's spacing) and the fp32
arithmetic: sums of squares over at most 32 products a lane and 11 additions across lanes lose 43
half-ulps, the reciprocal root 2^-22, products one each: 2^-18 of the terms' size in all.  The
columns' sums of dw take at most 1 + rows / (blocks of a GB300) + 64 additions: 2^-16."""
import numpy as np
import pytest
import torch

from oracle import block_ref as R
from oracle.lowbit_ref import bf16_half_step

pytestmark = pytest.mark.gpu

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def block():
    from mixture_experts_grouped_router_gb300 import block
    return block


@pytest.fixture(scope="module")
def L():
    from mixture_experts_grouped_router_gb300 import _lib
    return _lib


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def half_step(v, dtype):
    return bf16_half_step(v) if dtype == torch.bfloat16 else np.abs(v) * 2.0 ** -24 + 2.0 ** -149


def rows_of(shape, dtype, pad, fill, gen, size=1.0):
    """A matrix with `pad` spare columns of `fill` behind each row, and the whole."""
    whole = torch.full((shape[0], shape[1] + pad), fill, dtype=dtype, device="cuda")
    whole[:, :shape[1]] = (size * torch.randn(*shape, generator=gen, device="cuda")).to(dtype)
    return whole[:, :shape[1]], whole


SHAPES = [(1, 8), (3, 40), (1, 7168), (2, 16384), (5, 8192), (7, 8200), (33, 256), (64, 1000),
          (305, 520), (330, 4096), (700, 128), (400, 16384)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("stream", ["bf16", "fp32"])
@pytest.mark.parametrize("w_type,pad", [("fp32", 0), ("bf16", 16)])
def test_forward_and_backward(block, rows, cols, stream, w_type, pad):
    g = torch.Generator(device="cuda").manual_seed(rows * 31 + cols)
    st = TYPES[stream]
    x, _ = rows_of((rows, cols), torch.bfloat16, pad, 1e30, g)
    res, _ = rows_of((rows, cols), st, pad, 1e30, g, 3.0)
    x[0], res[0] = 0.0, 0.0           # a row of zeros: y = 0, dh = dy w / sqrt(eps)
    w = (1.0 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(TYPES[w_type])
    h, hw = rows_of((rows, cols), st, pad, 7.0, g)
    y, yw = rows_of((rows, cols), torch.bfloat16, pad, 7.0, g)
    assert block.rms_norm(x, w, EPS, y, residual=res, h=h) is y
    want_h = f64(x) + f64(res)
    # fp32 adds the two, its sum is rounded to the stream's type
    assert (np.abs(f64(h) - want_h) <= half_step(want_h, st) + 2.0 ** -24 * np.abs(want_h)).all()
    hv, wv = f64(h), f64(w)
    want, _ = R.rms_norm(hv, wv, EPS)
    assert (np.abs(f64(y) - want) <= bf16_half_step(want) + 2.0 ** -18 * np.abs(want)).all()
    assert (hw[:, cols:] == 7.0).all() and (yw[:, cols:] == 7.0).all()

    dy, _ = rows_of((rows, cols), torch.bfloat16, pad, 1e30, g)
    d_res, _ = rows_of((rows, cols), st, pad, 1e30, g)
    dh, dhw = rows_of((rows, cols), st, pad, 7.0, g)
    dx, dxw = rows_of((rows, cols), torch.bfloat16, pad, 7.0, g)
    dw = torch.full((cols + 1,), 7.0, device="cuda")
    ws = block.rms_norm_bwd_workspace(rows, cols)
    ws.fill_(0xFF)
    block.rms_norm_bwd(dy, h, w, EPS, dh, dw[:cols], ws, d_residual=d_res, dx=dx)
    dyv, rv = f64(dy), f64(d_res)
    want_dh, want_dw = R.rms_norm_bwd(dyv, hv, wv, EPS, rv)
    _, r = R.rms_norm(hv, wv, EPS)
    size = (np.abs(r * dyv * wv) + r ** 3 * np.abs(dyv * wv * hv).mean(1, keepdims=True) * np.abs(hv)
            + np.abs(rv))
    tol = half_step(want_dh, st) + 2.0 ** -17 * size
    assert (np.abs(f64(dh) - want_dh) <= tol).all()
    assert (np.abs(f64(dx) - want_dh) <= bf16_half_step(want_dh) + 2.0 ** -17 * size).all()
    assert (np.abs(f64(dw)[:cols] - want_dw) <= 2.0 ** -16 * np.abs(dyv * hv * r).sum(0) + 1e-30).all()
    assert (dhw[:, cols:] == 7.0).all() and (dxw[:, cols:] == 7.0).all() and dw[cols] == 7.0
    # without the residual's gradient, without dx and dw
    first = dh.clone()
    block.rms_norm_bwd(dy, h, w, EPS, dh, d_residual=None)
    want_0 = want_dh - rv
    assert (np.abs(f64(dh) - want_0) <= half_step(want_0, st) + 2.0 ** -17 * size).all()
    # added to dw; the same numbers each time
    again = dw[:cols].clone()
    block.rms_norm_bwd(dy, h, w, EPS, dh, again, ws, d_residual=d_res, accumulate=True)
    assert torch.equal(dh, first)
    assert (np.abs(f64(again) - 2 * f64(dw)[:cols]) <= 2.0 ** -23 * np.abs(f64(dw)[:cols])).all()


@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 7168), (129, 256), (700, 1024), (310, 4096)])
@pytest.mark.parametrize("keep_y", [True, False])
def test_codes_are_the_quantisers(block, L, rows, cols, keep_y):
    """Both formats: bit for bit what the framework's quantisers make of the bf16 y."""
    g = torch.Generator(device="cuda").manual_seed(cols + rows)
    x = torch.randn(rows, cols, generator=g, device="cuda").bfloat16()
    x[rows // 2, cols // 2] = 300.0  # an outlier
    x[-1, :64] = 0.0
    w = torch.randn(cols, generator=g, device="cuda")
    w[64:96] = 1e-30
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    block.rms_norm(x, w, EPS, y)
    for fmt in ("mx", "act8"):
        c, want = block.Codes8(rows, cols, fmt), block.Codes8(rows, cols, fmt)
        c.scales.view(torch.uint8).fill_(0x33), want.scales.view(torch.uint8).fill_(0x33)
        block.rms_norm(x, w, EPS, y2 if keep_y else None, codes=c)
        if fmt == "mx":
            L.moe_mx_quantize(y, L.FP8_E4M3, want.q, want.scales)
        else:
            L.moe_act8_quantize(y, want.q, want.scales)
        assert torch.equal(c.q, want.q) and torch.equal(c.scales.view(torch.uint8), want.scales.view(torch.uint8))
        if keep_y:
            assert torch.equal(y, y2)
        out = torch.full_like(x, 5.0)
        assert c.dequantize(out) is out
        worst = f64(y).reshape(rows, -1, 32)
        worst = np.repeat(np.abs(worst).max(2), 32, 1)
        # a step of the largest magnitude's (2^-4 of a power of two up to twice it: 448 of 512 is
        # saturated to an eighth; or half of the scale, which is 1 / 127 rounded up by at most one
        # bf16 spacing, 2^-7 of it; blocks under 2^-100 read as zeros there), and bf16's at the value that is
        # rounded, which may lie in the next binade
        bound = worst * 0.126 + 1e-37 if fmt == "mx" else worst * (1 + 2.0 ** -7) / 254 + 2.0 ** -100
        top = np.maximum(np.abs(f64(out)), np.abs(f64(y)))
        assert (np.abs(f64(out) - f64(y)) <= bound + bf16_half_step(top)).all()


@pytest.mark.parametrize("cols", [8, 40, 1000, 8200])
def test_act8_of_odd_widths(block, L, cols):
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(37, cols, generator=g, device="cuda").bfloat16()
    w = torch.ones(cols, device="cuda")
    y = torch.empty_like(x)
    c, want = block.Codes8(37, cols, "act8"), block.Codes8(37, cols, "act8")
    block.rms_norm(x, w, EPS, y, codes=c)
    L.moe_act8_quantize(y, want.q, want.scales)
    assert torch.equal(c.q, want.q) and torch.equal(c.scales, want.scales)


@pytest.mark.parametrize("fmt", ["E4M3", "E5M2"])
@pytest.mark.parametrize("rows,cols", [(1, 128), (130, 384), (2, 7168)])
def test_mx_dequantize(L, fmt, rows, cols):
    """Every code and scale code, against PyTorch's 8-bit floats."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    q = torch.randint(0, 256, (rows, cols), generator=g, device="cuda").to(torch.uint8)
    sf = torch.randint(0, 256, (L.moe_mx_scale_bytes(rows, cols, L.MX_ROWS_PLAIN),), generator=g,
                       device="cuda").to(torch.uint8)
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    L.moe_mx_dequantize(q, sf, getattr(L, "FP8_" + fmt), out)
    f8 = torch.float8_e4m3fn if fmt == "E4M3" else torch.float8_e5m2
    v = q.cpu().view(f8).double()
    r, b = torch.arange(rows).unsqueeze(1), torch.arange(cols // 32).unsqueeze(0)
    at = ((r // 128) * (cols // 128) + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4
    code = sf.cpu()[at].double()
    s = torch.where(code == 255, torch.nan, torch.pow(torch.tensor(2.0, dtype=torch.float64), code - 127))
    want = (v * s.repeat_interleave(32, 1)).float()  # 4 bits: exact in fp32, subnormals too
    torch.testing.assert_close(out.cpu(), want.bfloat16(), rtol=0, atol=0, equal_nan=True)


def test_codes_feed_the_block_scaled_product(block, L):
    """The norm's codes as the A operand of moe_gmm_mx: the product of their values."""
    T, d, N = 200, 256, 192
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    wn = torch.ones(d, device="cuda")
    c = block.Codes8(T, d, "mx")
    block.rms_norm(x, wn, EPS, codes=c)
    B = torch.randn(N, d, generator=g, device="cuda").bfloat16()
    qb = torch.empty(1, N, d, dtype=torch.uint8, device="cuda")
    sb = torch.empty(L.moe_mx_scale_bytes(N, d, L.MX_ROWS_TILES, 1), dtype=torch.uint8, device="cuda")
    L.moe_mx_quantize(B, L.FP8_E4M3, qb[0], sb, L.MX_ROWS_TILES)
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out = torch.empty(T, N, device="cuda")
    L.moe_gmm_mx(c.q, c.scales, L.FP8_E4M3, qb, sb, False, L.FP8_E4M3, off, out)
    a = f64(c.dequantize(torch.empty_like(x)))
    from oracle import moe_mx_ref
    b = moe_mx_ref.mx_qdq(f64(B), "e4m3")
    want = a @ b.T
    assert (np.abs(f64(out) - want) <= 2.0 ** -14 * (np.abs(a) @ np.abs(b).T)).all()


@pytest.mark.parametrize("stream", ["bf16", "fp32"])
def test_in_place(block, stream):
    """h over the residual, y over x; dh over the residual's gradient, dx over dy."""
    g = torch.Generator(device="cuda").manual_seed(9)
    st = TYPES[stream]
    x = torch.randn(50, 1024, generator=g, device="cuda").bfloat16()
    res = torch.randn(50, 1024, generator=g, device="cuda").to(st)
    w = torch.randn(1024, generator=g, device="cuda")
    h, y = torch.empty_like(res), torch.empty_like(x)
    block.rms_norm(x, w, EPS, y, residual=res, h=h)
    x2, r2 = x.clone(), res.clone()
    block.rms_norm(x2, w, EPS, x2, residual=r2, h=r2)
    assert torch.equal(x2, y) and torch.equal(r2, h)
    dy, d_res = x, res
    dh, dx, dw = torch.empty_like(h), torch.empty_like(y), torch.empty(1024, device="cuda")
    ws = block.rms_norm_bwd_workspace(50, 1024)
    block.rms_norm_bwd(dy, h, w, EPS, dh, dw, ws, d_residual=d_res, dx=dx)
    dy2, r2, dw2 = dy.clone(), d_res.clone(), torch.empty_like(dw)
    block.rms_norm_bwd(dy2, h, w, EPS, r2, dw2, ws, d_residual=r2, dx=dy2)
    assert torch.equal(dy2, dx) and torch.equal(r2, dh) and torch.equal(dw2, dw)


def test_one_addend_alone(block):
    g = torch.Generator(device="cuda").manual_seed(10)
    w = torch.ones(256, device="cuda")
    x = torch.randn(5, 256, generator=g, device="cuda").bfloat16()
    y, y2, h = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    block.rms_norm(x, w, EPS, y, h=h)
    block.rms_norm(None, w, EPS, y2, residual=x)
    assert torch.equal(y, y2) and torch.equal(h, x)
    r = torch.randn(5, 256, generator=g, device="cuda")
    block.rms_norm(None, w, EPS, y, residual=r)
    want, _ = R.rms_norm(f64(r), f64(w), EPS)
    assert (np.abs(f64(y) - want) <= bf16_half_step(want) + 2.0 ** -18 * np.abs(want)).all()


def test_bad_values_stay_in_their_row(block):
    x = torch.ones(4, 512, device="cuda").bfloat16()
    x[1, 3], x[2, 500] = float("nan"), float("inf")
    w = torch.ones(512, device="cuda")
    y = torch.empty_like(x)
    c = block.Codes8(4, 512, "mx")
    block.rms_norm(x, w, 1e-6, y, codes=c)
    out = f64(c.dequantize(torch.empty_like(x)))
    assert np.isnan(f64(y)[1]).all() and np.isnan(f64(y)[2, 500]) and np.isnan(out[1]).all()
    assert (f64(y)[[0, 3]] == 1.0).all() and (out[[0, 3]] == 1.0).all()
    huge = torch.full((1, 512), 1e30, device="cuda").bfloat16()
    block.rms_norm(huge, w, 1e-6, y[:1])
    assert (y[:1] == 0).all()  # squares past fp32: as the header says


def test_no_rows(block):
    x = torch.empty(0, 256, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(256, device="cuda")
    c = block.Codes8(0, 256, "mx")
    block.rms_norm(x, w, EPS, torch.empty_like(x), residual=x, h=torch.empty_like(x), codes=c)
    c.dequantize(torch.empty_like(x))
    dw = torch.full((256,), 3.0, device="cuda")
    ws = block.rms_norm_bwd_workspace(0, 256)
    block.rms_norm_bwd(x, x, w, EPS, torch.empty_like(x), dw, ws, accumulate=True)
    assert (dw == 3.0).all()
    block.rms_norm_bwd(x, x, w, EPS, torch.empty_like(x), dw, ws)
    assert (dw == 0.0).all()


def test_gradient_by_differences(block):
    """dh and dw against differences of the fp64 forward at the stored h."""
    g = torch.Generator(device="cuda").manual_seed(11)
    h = torch.randn(2, 16, generator=g, device="cuda")
    w, dy = torch.randn(16, generator=g, device="cuda"), torch.randn(2, 16, generator=g, device="cuda").bfloat16()
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    block.rms_norm_bwd(dy, h, w, EPS, dh, dw, block.rms_norm_bwd_workspace(2, 16))
    hv, wv, dv = f64(h), f64(w), f64(dy)
    f = lambda h, w: (R.rms_norm(h, w, EPS)[0] * dv).sum()  # noqa: E731
    for i in np.ndindex(2, 16):
        e = np.zeros_like(hv)
        e[i] = 1e-5
        assert abs((f(hv + e, wv) - f(hv - e, wv)) / 2e-5 - f64(dh)[i]) <= 1e-4
    for j in range(16):
        e = np.zeros_like(wv)
        e[j] = 1e-5
        assert abs((f(hv, wv + e) - f(hv, wv - e)) / 2e-5 - f64(dw)[j]) <= 1e-4


def test_rows_past_32_bit_offsets(block):
    """Leading dimensions that put the last row past 2^31 elements."""
    rows, cols, ld = 3, 64, (1 << 30) + 8
    whole = torch.empty(2 * ld + cols, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(whole, (rows, cols), (ld, 1))
    x.copy_(torch.randn(rows, cols, device="cuda"))
    want, y = torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16), x.clone()
    w = torch.ones(cols, device="cuda")
    block.rms_norm(x.contiguous(), w, EPS, want)
    block.rms_norm(x, w, EPS, y)
    assert torch.equal(y, want)
    block.rms_norm(x, w, EPS, x)
    assert torch.equal(x, want)


@pytest.mark.parametrize("cols", [256, 1000, 4096, 5000, 16384])
@pytest.mark.parametrize("stream", ["bf16", "fp32"])
@pytest.mark.parametrize("eps", [1e-20, 1e-30, 1e-37])
def test_small_eps(block, cols, stream, eps):
    """Rows of zeros and of values about the root of eps, where the reciprocal root's third power
    passes fp32's range.  Tolerances as above."""
    rows = 9
    g = torch.Generator(device="cuda").manual_seed(cols)
    st, eps = TYPES[stream], float(np.float32(eps))
    h = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.float64)
    h *= torch.tensor([1, 0, eps ** 0.5, 0.1 * eps ** 0.5, 30 * eps ** 0.5, 0, 1e-3, 0, 1], device="cuda",
                      dtype=torch.float64)[:, None]
    h[7, 3] = eps ** 0.5
    h = h.to(st)
    w = 1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")
    dy = (0.1 * torch.randn(rows, cols, generator=g, device="cuda")).bfloat16()
    res = torch.randn(rows, cols, generator=g, device="cuda").to(st)
    y, dh, dw = torch.empty_like(dy), torch.empty_like(h), torch.empty(cols, device="cuda")
    block.rms_norm(None, w, eps, y, residual=h)
    block.rms_norm_bwd(dy, h, w, eps, dh, dw, block.rms_norm_bwd_workspace(rows, cols), d_residual=res)
    hv, wv, dv, rv = f64(h), f64(w), f64(dy), f64(res)
    want, r = R.rms_norm(hv, wv, eps)
    assert (np.abs(f64(y) - want) <= half_step(want, torch.bfloat16) + 2.0 ** -18 * np.abs(want)).all()
    want, want_dw = R.rms_norm_bwd(dv, hv, wv, eps, rv)
    gr = np.abs(dv * wv) * r
    terms = gr + r * np.abs(hv) * r * r * np.abs(dv * wv * hv).mean(1, keepdims=True) + np.abs(rv)
    assert (np.abs(f64(dh) - want) <= half_step(want, st) + 2.0 ** -18 * terms).all()
    assert (np.abs(f64(dw) - want_dw) <= 2.0 ** -16 * np.abs(dv * hv * r).sum(0)).all()


@pytest.mark.parametrize("cols", [256, 4096, 16384])
@pytest.mark.parametrize("stream", ["bf16", "fp32"])
def test_backward_of_rows_past_fp32(block, cols, stream):
    """Rows whose squares pass fp32's range read as zeros in y: nothing but d_residual reaches them,
    and they add nothing to dw."""
    g = torch.Generator(device="cuda").manual_seed(5)
    st = TYPES[stream]
    h = torch.randn(4, cols, generator=g, device="cuda")
    h[1] = 3e38 * torch.sign(h[1])
    h[2, 7] = 2e19
    h = h.to(st)
    w = torch.ones(cols, device="cuda")
    dy = (10.0 * torch.randn(4, cols, generator=g, device="cuda")).bfloat16()
    res = torch.randn(4, cols, generator=g, device="cuda").to(st)
    y, dh, dw = torch.empty_like(dy), torch.empty_like(h), torch.empty(cols, device="cuda")
    ws = block.rms_norm_bwd_workspace(4, cols)
    block.rms_norm(None, w, EPS, y, residual=h)
    block.rms_norm_bwd(dy, h, w, EPS, dh, dw, ws, d_residual=res)
    assert (y[1:3] == 0).all() and torch.equal(dh[1:3], res[1:3])
    hv, dv = f64(h)[::3], f64(dy)[::3]
    _, want_dw = R.rms_norm_bwd(dv, hv, f64(w), EPS)
    size = np.abs(dv * hv / np.sqrt((hv * hv).mean(1, keepdims=True) + EPS)).sum(0)
    assert (np.abs(f64(dw) - want_dw) <= 2.0 ** -16 * size).all()
