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


TIES = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])


def beside_ties(n, seed):
    """n blocks [n, 16] and their fp32 scales g [n] of 24 bits: in each block some values whose
    quotient by the block's scale S g lies 2^-22 to 2^-18 (relative) beside a tie.  S g and the
    quotient are rounded to 2^-24 each on the way: the side is certain."""
    rng = np.random.default_rng(seed)
    S = 1.0 + rng.integers(0, 8, n) / 8
    tie = rng.choice(TIES, n)
    x = f64(bf16((1.0 + rng.random(n)) * np.exp2(rng.integers(-6, 7, n))))
    g = (x / (tie * S)).astype(np.float32)
    g = (g.view(np.int32) + (rng.choice([-1, 1], n) * rng.integers(8, 17, n)).astype(np.int32)).view(np.float32)
    d = np.abs(x / (tie * S * g.astype(np.float64)) - 1)
    assert (d >= 2.0 ** -22).all() and (d <= 2.0 ** -18).all()
    b = np.zeros((n, 16))
    b[:, 0] = f64(bf16(6.0 * S * g))  # the block's largest: its scale is S
    b[:, 3], b[:, 4], b[:, 15] = x, -x, x
    el, code, _ = R.fp4_quantize(b[:1], "nv", float(g[0]))
    assert R.e4m3_value(code[0, 0]) == S[0]
    return b, g


def test_quotients_beside_a_tie(L):
    """A scale of 24 bits (one an expert): the side that the quotient is on decides."""
    n = 4096
    b, g = beside_ties(2 * n, 21)
    x, gg = b.reshape(n, 32), g.reshape(n, 2)
    x = np.stack([x, x[:, np.r_[16:32, 0:16]]], 1)  # two rows an expert: each scale's blocks
    for half in (0, 1):
        gt = torch.from_numpy(np.ascontiguousarray(gg[:, half])).cuda()
        q = torch.empty(2 * n, 16, dtype=torch.uint8, device="cuda")
        sf = torch.empty(L.moe_fp4_scale_bytes(2 * n, 32, 1, 3, n), dtype=torch.uint8, device="cuda")
        L.moe_fp4_quantize(bf16(x.reshape(2 * n, 32)), 1, q, sf, row_map=3, groups=n, scale=gt)
        got = R.unpack(q.cpu().numpy()).reshape(n, 2, 2, 16)
        want = np.stack([R.fp4_quantize(b.reshape(n, 2, 16)[i, half][None], "nv", float(gg[i, half]))[0][0]
                         for i in range(n)])
        assert (got[:, 0, half] == want).all() and (got[:, 1, 1 - half] == want).all()
        # the same as weights that are laid out
        q2, sf2 = torch.empty(n, 2, 16, dtype=torch.uint8, device="cuda"), torch.empty_like(sf)
        L.moe_fp4_quantize_weights(bf16(x.transpose(0, 2, 1)), 1, 3, q2, sf2, gt)
        assert (q2.view(2 * n, 16) == q).all()


@pytest.mark.parametrize("i", range(12))
def test_quotients_beside_a_tie_of_the_tensors_scale(L, i):
    """As activations, one scale for all rows, directly and gathered."""
    b, g = beside_ties(12, 22)
    g = float(g[i])
    x = np.repeat(b[i][None], 8, 0).reshape(4, 32)
    el, code, _ = R.fp4_quantize(x, "nv", g)
    gt = torch.tensor([g], device="cuda")
    for idx in (None, i32([3, 1, 0, 2])):
        q = torch.empty(4, 16, dtype=torch.uint8, device="cuda")
        sf = torch.empty(L.moe_fp4_scale_bytes(4, 32, 1, 1, 1), dtype=torch.uint8, device="cuda")
        L.moe_fp4_quantize(bf16(x), 1, q, sf, group_offsets=i32([0, 4]), row_index=idx, scale=gt)
        assert (R.unpack(q.cpu().numpy()) == el).all()


@pytest.mark.parametrize("g", [0.0137, 6.0 / 2688, 1.1e-30, 3.3e20])
def test_scales_of_24_bits_over_the_whole_range(L, g):
    """Bit for bit but for ratios 2^-22 beside a tie, of which there are next to none."""
    g = float(np.float32(g))
    rng = np.random.default_rng(23)
    n, cols = 261, 96
    x = whole_range(rng, n, cols)
    q = torch.empty(n, cols // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(L.moe_fp4_scale_bytes(n, cols, 1, 1, 1), dtype=torch.uint8, device="cuda")
    L.moe_fp4_quantize(bf16(x), 1, q, sf, group_offsets=i32([0, n]), scale=torch.tensor([g], device="cuda"))
    el, code, _ = R.fp4_quantize(x, "nv", g)
    s = grouped_scales(sf.cpu().numpy(), list(range(n)), cols // 16, -(-cols // 64))
    a = np.abs(x).reshape(n, -1, 16).max(-1) / (6.0 * g)
    step = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    sure = np.abs(np.mod(a / step, 1.0) - 0.5) > 2.0 ** -19  # 16 steps to a binade at most
    sure |= a > 448
    assert sure.mean() > 0.99 and (s == code)[sure].all()
    t = np.repeat(R.e4m3_value(code) * g, 16, 1)
    r = np.abs(x) / np.where(t > 0, t, 1.0)
    near = (np.abs(r[..., None] / TIES - 1) < 2.0 ** -22).any(-1)
    ok = np.repeat(sure, 16, 1) & ~near
    got = R.unpack(q.cpu().numpy())
    assert ok.mean() > 0.98 and ((got == el) | ((el & 7 == 0) & (got & 7 == 0)))[ok].all()
