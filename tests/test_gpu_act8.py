"""8-bit activation checkpoints on the GPU against the fp64 oracle: codes and
scales bit-exact; the SwiGLU forward and the backward from the codes to one
rounding to bf16 (half its spacing) plus 2^-18 of the terms' size for the fp32
exponential, reciprocal and products (each within a few 2^-23)."""
import numpy as np
import pytest
import torch

from oracle import lowbit_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from mixture_experts_grouped_router_gb300 import _lib
    return _lib


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().cuda()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def values(rng, rows, cols):
    """bf16 values of many magnitudes, with zeros and ties of the code grid."""
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, 1)))
    x[rng.random((rows, cols)) < 0.05] = 0.0
    tie = rng.random((rows, 1)) < 0.3  # scale 1: halves are ties
    x = np.where(tie, rng.integers(-254, 255, (rows, cols)) / 2.0, x)
    x[:, ::32] = np.where(tie, 127.0, x[:, ::32])
    return f64(bf16(x))


SHAPES = [(1, 8), (3, 32), (5, 40), (17, 264), (2, 1000), (300, 7168)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("live", ["all", "some", "none"])
def test_round_trip(L, rows, cols, strided, live):
    rng = np.random.default_rng(rows + cols)
    x = values(rng, rows, cols)
    nb = -(-cols // 32)
    pad = 24 if strided else 0
    xt = torch.full((rows, cols + pad), 3.0, dtype=torch.bfloat16, device="cuda")[:, :cols]
    xt.copy_(bf16(x))
    q = torch.full((rows, cols + pad), 77, dtype=torch.int8, device="cuda")
    s = torch.full((rows, nb + pad), 5.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full((rows, cols + pad), 9.0, dtype=torch.bfloat16, device="cuda")
    n = {"all": rows, "some": rows // 2, "none": 0}[live]
    off = None if live == "all" else torch.tensor([0, n // 3, n], dtype=torch.int32, device="cuda")
    L.moe_act8_quantize(xt, q[:, :cols], s[:, :nb], off)
    L.moe_act8_dequantize(q[:, :cols], s[:, :nb], out[:, :cols], off)
    cq, cs, cv = R.act8_quantize(x[:n]) if n else (np.zeros((0, cols)),) * 3
    assert (f64(q)[:n, :cols] == cq).all()
    if n:
        assert (f64(s)[:n, :nb] == cs).all()
    assert (f64(out)[:n, :cols] == f64(bf16(cv))).all()
    assert (q[n:] == 77).all() and (s[n:] == 5.0).all() and (out[n:] == 9.0).all()
    assert (q[:, cols:] == 77).all() and (s[:, nb:] == 5.0).all() and (out[:, cols:] == 9.0).all()
    err = np.abs(f64(out)[:n, :cols] - x[:n])  # half a code step, and bf16's rounding
    if n:
        half = np.repeat(cs, 32, 1)[:, :cols] * 0.5
        assert (err <= half + R.bf16_half_step(cv) + 2.0 ** -100).all()


def test_bad_values_poison_their_block_alone(L):
    x = np.ones((4, 96))
    x[0, 3], x[1, 40], x[2, 95], x[3] = np.nan, np.inf, -np.inf, 0.0
    x[3, 0] = 2.0 ** -120
    q = torch.empty(4, 96, dtype=torch.int8, device="cuda")
    s = torch.empty(4, 3, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(4, 96, dtype=torch.bfloat16, device="cuda")
    L.moe_act8_quantize(bf16(x), q, s)
    L.moe_act8_dequantize(q, s, out)
    want = R.act8_quantize(x)[2]
    got = f64(out)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and int(np.isnan(got).sum()) == 96
    assert (got[3] == 0).all()
    ok = ~np.isnan(want)
    assert (got[ok] == f64(bf16(np.where(ok, want, 0)))[ok]).all()


@pytest.mark.parametrize("rows,F", [(1, 8), (2, 40), (33, 256), (5, 1000), (130, 2048)])
@pytest.mark.parametrize("live", ["all", "some"])
@pytest.mark.parametrize("want_act", [True, False])
def test_swiglu_forward_and_backward(L, rows, F, live, want_act):
    rng = np.random.default_rng(rows * F)
    h = f64(bf16(2.0 * rng.standard_normal((rows, 2 * F))))
    h[0, 0], h[0, F] = 90.0, -120.0   # the sigmoid's ends
    h[-1, F - 1] = -200.0
    da = f64(bf16(rng.standard_normal((rows, F))))
    nb = -(-F // 32)
    n = rows if live == "all" else rows // 2
    off = None if live == "all" else torch.tensor([0, n], dtype=torch.int32, device="cuda")
    act = torch.full((rows, F), 9.0, dtype=torch.bfloat16, device="cuda")
    act2, dh = act.clone(), torch.full((rows, 2 * F), 9.0, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(rows, 2 * F, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, 2 * nb, dtype=torch.bfloat16, device="cuda")
    L.moe_act8_swiglu_fwd(bf16(h), act, q, s, off)
    L.moe_act8_swiglu_bwd(q, s, bf16(da), dh, act2 if want_act else None, off)
    if n == 0:
        assert (act == 9.0).all() and (dh == 9.0).all()
        return
    qg, sg, vg = R.act8_quantize(h[:n, :F])
    qu, su, vu = R.act8_quantize(h[:n, F:])
    assert (f64(q)[:n] == np.concatenate([qg, qu], 1)).all()
    assert (f64(s)[:n] == np.concatenate([sg, su], 1)).all()
    a = R.swiglu(h[:n])
    tiny = 2.0 ** -120  # results under bf16's normal range
    assert (np.abs(f64(act)[:n] - a) <= R.bf16_half_step(a) + 2.0 ** -18 * np.abs(a) + tiny).all()
    hv = np.concatenate([vg, vu], 1)
    wdh, wact = R.swiglu_bwd(hv, da[:n])
    sig = 1.0 / (1.0 + np.exp(-vg))
    size = np.concatenate([np.abs(da[:n] * vu) * sig * (1 + np.abs(vg)), np.abs(wdh[:, F:])], 1)
    assert (np.abs(f64(dh)[:n] - wdh) <= R.bf16_half_step(wdh) + 2.0 ** -18 * size + tiny).all()
    if want_act:
        assert (np.abs(f64(act2)[:n] - wact) <= R.bf16_half_step(wact) + 2.0 ** -18 * np.abs(wact) + tiny).all()
    else:
        assert (act2 == 9.0).all()
    assert (act[n:] == 9.0).all() and (dh[n:] == 9.0).all()


def test_backward_is_the_forwards_derivative(L):
    """dh against differences of the fp64 forward at the saved values."""
    rng = np.random.default_rng(7)
    rows, F = 2, 32
    h, da = f64(bf16(rng.standard_normal((rows, 2 * F)))), f64(bf16(rng.standard_normal((rows, F))))
    q = torch.empty(rows, 2 * F, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, 2, dtype=torch.bfloat16, device="cuda")
    act, dh = bf16(da), bf16(h)
    L.moe_act8_swiglu_fwd(bf16(h), act, q, s)
    L.moe_act8_swiglu_bwd(q, s, bf16(da), dh)
    v = f64(q) * np.repeat(f64(s), 32, 1)
    got, eps = f64(dh), 1e-5
    for i in range(rows):
        for j in range(2 * F):
            d = np.zeros_like(v)
            d[i, j] = eps
            num = ((R.swiglu(v + d) - R.swiglu(v - d)) * da).sum() / (2 * eps)
            # bf16's rounding, the fp32 terms, and the difference's own eps^2
            assert abs(num - got[i, j]) <= R.bf16_half_step(num) + 1e-4


def test_another_stream(L):
    x = torch.randn(64, 512, device="cuda").bfloat16()
    st = torch.cuda.Stream()
    q = torch.empty(64, 512, dtype=torch.int8, device="cuda")
    s = torch.empty(64, 16, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    L.moe_act8_quantize(x, q, s, stream=st)
    L.moe_act8_dequantize(q, s, out, stream=st)
    st.synchronize()
    assert (f64(out) == f64(bf16(R.act8_quantize(f64(x))[2]))).all()
