"""Pins of the low-bit oracle on hand-worked blocks (CPU)."""
import numpy as np

from oracle import lowbit_ref as R


def test_e2m1_ties_go_to_even_codes():
    x = np.zeros((1, 32))
    x[0, :9] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0]
    el, code, val = R.fp4_quantize(x, "mx")
    assert code[0, 0] == 127  # floor(log2 6) - 2 = 0
    assert val[0, :9].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -4.0]
    assert el[0, :9].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 14]


def test_mx_saturates_and_handles_empty_and_bad_blocks():
    x = np.zeros((1, 96))
    x[0, 0] = 7.9          # scale 1: saturates at 6
    x[0, 64:] = 1.0
    x[0, 70] = np.inf
    el, code, val = R.fp4_quantize(x, "mx")
    assert code[0].tolist() == [127, 0, 255]
    assert val[0, 0] == 6.0 and (val[0, 32:64] == 0).all() and np.isnan(val[0, 64:]).all()


def test_nv_scales():
    x = np.zeros((1, 48))
    x[0, 0] = 6.0 * 1.1          # 1.1 -> E4M3 1.125 (steps of 1/8)
    x[0, 16] = 6.0 * 2000.0      # past 448: saturates
    x[0, 32] = 6.0 * 2.0 ** -11  # under half of the smallest scale 2^-9: zero
    el, code, val = R.fp4_quantize(x, "nv")
    assert R.e4m3_value(code[0]).tolist() == [1.125, 448.0, 0.0]
    assert val[0, 0] == 6.0 * 1.125 and val[0, 16] == 6.0 * 448.0 and val[0, 32] == 0.0
    el2, code2, val2 = R.fp4_quantize(x * 0.5, "nv", 0.5)  # g scales everything
    assert (code2 == code).all() and (val2 == 0.5 * val).all()


def test_e4m3_codes_round_trip():
    codes = np.arange(0x7F, dtype=np.uint8)
    v = R.e4m3_value(codes)
    assert (R.e4m3_code(v) == codes).all() and (R.round_e4m3(v) == v).all()
    assert R.round_e4m3(np.array([1.0625, 1.1875, 460.0])).tolist() == [1.0, 1.25, 448.0]


def test_padded_rows_are_distinct():
    for G, E, m in ((200, 3, "experts"), (192, 2, "swiglu"), (2 * 224, 2, "swiglu")):
        rows = [R.padded_row(r, G, m) for r in range(E * G)]
        assert len(set(rows)) == E * G
    assert R.scale_byte(128 + 33, 5, 2) == (1 * 2 + 1) * 512 + 16 + 4 + 1


def test_act8():
    x = np.zeros((1, 72))
    x[0, 0], x[0, 1], x[0, 2] = 127.0, 0.5, 1.5   # scale 1: ties to even
    x[0, 32] = 128.0                              # 128 / 127 = 1.00787.. up to bf16: 1.015625
    x[0, 64] = 2.0 ** -101                        # too small: zeros
    q, s, v = R.act8_quantize(x)
    assert s[0].tolist() == [1.0, 1.015625, 0.0]
    assert q[0, :3].tolist() == [127.0, 0.0, 2.0] and q[0, 32] == 126.0 and q[0, 64] == 0.0
    x[0, 5] = np.nan
    assert np.isnan(R.act8_quantize(x)[2][0, :32]).all()


def test_swiglu_gradient_matches_differences():
    rng = np.random.default_rng(0)
    h, da = rng.standard_normal((3, 8)), rng.standard_normal((3, 4))
    dh, act = R.swiglu_bwd(h, da)
    assert np.allclose(act, R.swiglu(h), rtol=1e-14, atol=0)
    eps = 1e-6
    for i in range(3):
        for j in range(8):
            d = np.zeros_like(h)
            d[i, j] = eps
            num = ((R.swiglu(h + d) - R.swiglu(h - d)) * da).sum() / (2 * eps)
            assert abs(num - dh[i, j]) < 1e-8  # eps^2 and rounding 1e-16 / eps
