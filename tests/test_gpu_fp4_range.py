"""4-bit blocks at the ends of the number range: bf16's largest values, its subnormals, and
scales of every size, bit for bit against the fp64 oracle.

fp32 scales have 8 significant bits here, so that whether a ratio is a tie is decided exactly.
A block scale past E4M3's 448 saturates there and its elements at 6; only a NaN or an infinity
takes the NaN scale."""
import numpy as np
import pytest
import torch

from oracle import lowbit_ref as R
from test_gpu_fp4 import (FMT, bf16, f64, gemm_case, grouped_scales, i32, offsets_of, padded_rows)

pytestmark = pytest.mark.gpu

SCALES = [1.0, 2.0 ** -64, 2.0 ** 100, 1.2578125 * 2.0 ** -9, 1.109375 * 2.0 ** -100]


@pytest.fixture(scope="module")
def L():
    from mixture_experts_grouped_router_gb300 import _lib
    return _lib


def whole_range(rng, rows, cols):
    """bf16 values: rows of one magnitude each, from 2^-133 to 2^128, a third of them with a
    magnitude an element, zeros among them."""
    e = np.linspace(-133, 127, rows)[:, None]
    x = (0.5 + 0.496 * rng.random((rows, cols))) * np.exp2(np.floor(e) + 1)
    each = rng.random((rows, 1)) < 0.33
    x = np.where(each, x * np.exp2(rng.integers(-12, 1, (rows, cols))), x)
    x *= rng.choice([-1.0, 1.0], (rows, cols))
    x[rng.random((rows, cols)) < 0.05] = 0.0
    return f64(bf16(x))


def check(q, sf, at, x, fmt, g):
    """Codes q [rows, cols / 2] and the scales of padded rows `at` against the oracle."""
    el, code, val = R.fp4_quantize(x, fmt, g)
    atom = 64 if fmt == "nv" else 128
    s = grouped_scales(sf.cpu().numpy(), at, code.shape[1], -(-x.shape[1] // atom))
    assert (s == code).all()
    got = R.unpack(q.cpu().numpy())
    assert ((got == el) | ((el & 7 == 0) & (got & 7 == 0))).all()  # a zero's sign is not kept
    return val


def some_saturate(x, g):
    return (np.abs(x).max() / (6.0 * g)) > 2.0 ** 128


@pytest.mark.parametrize("fmt,g", [("mx", 1.0)] + [("nv", g) for g in SCALES])
def test_quantize_over_the_whole_range(L, fmt, g):
    rng = np.random.default_rng(11)
    sizes, cols = [200, 0, 61], 96
    n = sum(sizes)
    x = whole_range(rng, n, cols)
    assert (g >= 0.125) or some_saturate(x, g)  # the ratio passes fp32's range
    q = torch.empty(n, cols // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(L.moe_fp4_scale_bytes(n, cols, FMT[fmt], 1, 3), dtype=torch.uint8, device="cuda")
    off, gt = i32(offsets_of(sizes)), torch.tensor([g], device="cuda")
    L.moe_fp4_quantize(bf16(x), FMT[fmt], q, sf, group_offsets=off, scale=gt)
    val = check(q, sf, padded_rows(sizes), x, fmt, g)
    out = torch.empty(n, cols, dtype=torch.bfloat16, device="cuda")
    L.moe_fp4_dequantize(q, sf, FMT[fmt], out, group_offsets=off, scale=gt)
    assert (f64(out) == f64(bf16(val))).all()


@pytest.mark.parametrize("fmt,g", [("mx", 1.0), ("nv", 1.0), ("nv", SCALES[3])])
def test_linked_gather_over_the_whole_range(L, fmt, g):
    """Each source row taken eight times: quantised once, against the oracle."""
    rng = np.random.default_rng(12)
    src, k, cols = 512, 8, 4096
    x = whole_range(rng, src, cols)
    idx = rng.permutation(src * k).astype(np.int32)
    sizes = [1000, 0, 3000, 96]
    assert sum(sizes) == src * k
    q = torch.empty(src * k, cols // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(L.moe_fp4_scale_bytes(src * k, cols, FMT[fmt], 1, 4), dtype=torch.uint8,
                     device="cuda")
    ws = torch.empty(L.moe_fp4_quantize_workspace_bytes(src, src * k), dtype=torch.uint8, device="cuda")
    L.moe_fp4_quantize(bf16(x), FMT[fmt], q, sf, group_offsets=i32(offsets_of(sizes)),
                       row_index=i32(idx), index_div=k, scale=torch.tensor([g], device="cuda"),
                       workspace=ws)
    el, code, _ = R.fp4_quantize(x, fmt, g)
    got = R.unpack(q.cpu().numpy())
    el, code = el[idx // k], code[idx // k]
    assert ((got == el) | ((el & 7 == 0) & (got & 7 == 0))).all()
    nb, ac = code.shape[1], cols // (64 if fmt == "nv" else 128)
    p = np.array(padded_rows(sizes))[:, None]
    b = np.arange(nb)[None]
    at = ((p // 128) * ac + b // 4) * 512 + (p % 32) * 16 + (p % 128 // 32) * 4 + b % 4
    assert (sf.cpu().numpy()[at] == code).all()


@pytest.mark.parametrize("fmt,g", [("mx", 1.0)] + [("nv", g) for g in SCALES])
def test_weights_over_the_whole_range(L, fmt, g):
    rng = np.random.default_rng(13)
    E, K, N = 2, 96, 128
    wt = whole_range(rng, E * N, K)
    w = wt.reshape(E, N, K).transpose(0, 2, 1)
    gt = torch.full((E,), g, device="cuda")
    q = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(L.moe_fp4_scale_bytes(E * N, K, FMT[fmt], 3, E), dtype=torch.uint8, device="cuda")
    L.moe_fp4_quantize_weights(bf16(w), FMT[fmt], 3, q, sf, gt)
    check(q.view(E * N, K // 2), sf, [R.padded_row(r, N, "experts") for r in range(E * N)], wt, fmt, g)


@pytest.mark.parametrize("sizes,K", [([40, 3], 96), ([515], 96)])  # weights as M, tokens as M
def test_act_saturates_in_the_epilogue(L, sizes, K):
    """A scale of Act so small that ratios pass fp32's range: the largest codes."""
    F, g2 = 96, 2.0 ** -124
    c = gemm_case(L, "nv", sizes, K, 2 * F, swiglu=True)
    n, cap, E = c["n"], c["cap"], len(sizes)
    S = 16.0 * c["S"]
    blocks = np.abs(R.swiglu(S)).reshape(n, -1, 16).max(-1)
    # every block saturates, some of them past 2^128; no sigmoid is flushed to zero
    assert blocks.min() > 448 * 6 * g2 and blocks.max() > 6 * g2 * 2.0 ** 128 and np.abs(S).max() < 84
    q2 = torch.empty(cap, F // 2, dtype=torch.uint8, device="cuda")
    sf2 = torch.empty(L.moe_fp4_scale_bytes(cap, F, 1, 1, E), dtype=torch.uint8, device="cuda")
    L.moe_gmm_fp4(c["A"], c["sfa"], c["B"], c["sfb"], 1, c["off"], epilogue=L.EPI_SWIGLU_FWD, Q2=q2,
                  sf2=sf2, a_scale=16.0 * c["a_scale"], b_scale=c["b_scale"],
                  q2_scale=torch.tensor([g2], device="cuda"))
    s = grouped_scales(sf2.cpu().numpy(), padded_rows(sizes), F // 16, -(-F // 64))
    assert (s == 0x7E).all()
    got = R.unpack(q2.cpu().numpy()[:n])
    err = 2.0 ** -16 * c["mag"]  # of the fp32 sums
    gate, up = c["S"][:, :F], c["S"][:, F:]
    sure = (np.abs(gate) > err[:, :F]) & (np.abs(up) > err[:, F:])  # both signs are certain
    assert sure.mean() > 0.9
    assert (got[sure] == np.where((gate < 0) != (up < 0), 15, 7)[sure]).all()
