"""4-bit block-scaled formats on the GPU: quantisers, scale atoms and the grouped
GEMM against the fp64 oracle of the formats.

Tolerances.  Codes and scales are bit-exact on bf16 inputs (with fp32 scales of
few significant bits, so that a ratio's ties are ties in fp32 too).  A product's
bf16 output differs from fp64 by one rounding (half bf16's spacing) and the fp32
sums' error, at most K 2^-23 of sum |a b|, taken as 2^-16 for K up to 4096 (the
tensor cores add in fp32 with truncation).  Act is quantised from fp32 values off
by that much: a code moves where a value lies that near a tie, under 1 in 1000."""
import numpy as np
import pytest
import torch

from oracle import lowbit_ref as R

pytestmark = pytest.mark.gpu

FMT = {"mx": 0, "nv": 1}


@pytest.fixture(scope="module")
def L():
    from mixture_experts_grouped_router_gb300 import _lib
    return _lib


@pytest.fixture(scope="module")
def lowbit():
    from mixture_experts_grouped_router_gb300 import lowbit
    return lowbit


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).bfloat16().cuda()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def offsets_of(sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)


def values(rng, rows, cols):
    """bf16 values over many magnitudes, zeros, and ties of the code grid."""
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-12, 12, (rows, 1)))
    x[rng.random((rows, cols)) < 0.05] = 0.0
    tie = rng.random((rows, cols)) < 0.1
    x[tie] = (rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], tie.sum())
              * np.exp2(rng.integers(-3, 3, tie.sum())))
    return f64(bf16(x))


def grouped_scales(sf, rows_at, nb, ac):
    """Scale codes [len(rows_at), nb] at padded rows of the atoms."""
    idx = np.array([[R.scale_byte(p, b, ac) for b in range(nb)] for p in rows_at])
    return sf[idx]


def padded_rows(sizes):
    out, p = [], 0
    for s in sizes:
        out += list(range(p, p + s))
        p += -(-s // 128) * 128
    return out


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("sizes,cols", [([1], 32), ([0, 3, 0], 64), ([130, 0, 1, 127], 96),
                                        ([5, 300], 1056), ([7], 7168)])
def test_quantize_grouped_is_bit_exact(L, fmt, sizes, cols):
    rng = np.random.default_rng(cols + len(sizes))
    off = offsets_of(sizes)
    n, E, cap = int(off[-1]), len(sizes), int(off[-1]) + 5
    x = values(rng, n + 2, cols)
    idx = rng.integers(-1, 3 * (n + 2), cap)
    g = float(torch.tensor(0.0137).bfloat16())
    q = torch.full((cap, cols // 2), 0xAB, dtype=torch.uint8, device="cuda")
    sf = torch.full((L.moe_fp4_scale_bytes(cap, cols, FMT[fmt], 1, E),), 0xCD, dtype=torch.uint8,
                    device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.moe_fp4_quantize(bf16(x), FMT[fmt], q, sf, group_offsets=i32(off), row_index=i32(idx),
                       index_div=3, scale=torch.tensor([g], device="cuda"), dev_status=st)
    rows = np.where((idx >= 0)[:, None], x[np.maximum(idx, 0) // 3], 0.0)[:n]
    el, code, val = R.fp4_quantize(rows, fmt, g)
    assert int(st.item()) == 0
    got = q.cpu().numpy()
    assert (R.unpack(got[:n]) & 7 == el & 7).all()
    nz = (el & 7) != 0
    assert ((R.unpack(got[:n]) == el) | ~nz).all()     # a zero's sign is not kept
    assert (got[n:] == 0xAB).all()                     # rows past the groups: not written
    atom = 64 if fmt == "nv" else 128
    ac, nb = -(-cols // atom), code.shape[1]
    s = grouped_scales(sf.cpu().numpy(), padded_rows(sizes), 4 * ac, ac)
    assert (s[:, :nb] == code).all() and (s[:, nb:] == 0).all()
    out = torch.full((cap, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    L.moe_fp4_dequantize(q, sf, FMT[fmt], out, group_offsets=i32(off),
                         scale=torch.tensor([g], device="cuda"))
    want = val if fmt == "mx" else f64(bf16(val))
    assert (f64(out)[:n] == want).all() and (f64(out)[n:] == 7.0).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("sizes,src,cols", [([0, 4000, 1, 900], 1500, 4096),
                                            ([20000, 130], 5000, 928)])
def test_gather_of_repeated_rows_quantises_them_once(L, fmt, sizes, src, cols):
    """The same codes and scales with the workspace of a repeating gather as without:
    repeats, rows of zeros (a long run of them), unused and missing source rows."""
    rng = np.random.default_rng(src)
    off = offsets_of(sizes)
    cap, E = int(off[-1]) + 7, len(sizes)
    x = bf16(rng.standard_normal((src, cols)))
    idx = rng.integers(0, 4 * (src - 9), cap)
    idx[rng.random(cap) < 0.1] = -1
    idx[100:400] = -1
    idx[3] = 4 * src  # not there
    g = torch.tensor([0.015625], device="cuda")
    res = []
    for ws in (None, torch.empty(L.moe_fp4_quantize_workspace_bytes(src, cap), dtype=torch.uint8,
                                 device="cuda")):
        q = torch.full((cap, cols // 2), 0xAB, dtype=torch.uint8, device="cuda")
        sf = torch.full((L.moe_fp4_scale_bytes(cap, cols, FMT[fmt], 1, E),), 0xCD,
                        dtype=torch.uint8, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        for _ in range(2):
            L.moe_fp4_quantize(x, FMT[fmt], q, sf, group_offsets=i32(off), row_index=i32(idx),
                               index_div=4, scale=g, workspace=ws, dev_status=st)
        assert int(st.item()) == L.MOE_ERR_DEVICE
        res.append((q, sf))
    assert (res[0][0] == res[1][0]).all() and (res[0][1] == res[1][1]).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_nan_blocks_and_bad_rows(L, fmt):
    x = np.ones((4, 64))
    x[0, 3], x[1, 40], x[2, 0], x[3] = np.nan, np.inf, -np.inf, 0.0
    q = torch.empty(6, 32, dtype=torch.uint8, device="cuda")
    sf = torch.empty(L.moe_fp4_scale_bytes(6, 64, FMT[fmt], 1, 1), dtype=torch.uint8,
                     device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = i32([0, 1, 2, 3, 4, -1])  # row 4 is not there
    L.moe_fp4_quantize(bf16(x), FMT[fmt], q, sf, group_offsets=i32([0, 6]), row_index=idx,
                       dev_status=st)
    out = torch.empty(6, 64, dtype=torch.bfloat16, device="cuda")
    L.moe_fp4_dequantize(q, sf, FMT[fmt], out, group_offsets=i32([0, 6]))
    got = f64(out)
    assert int(st.item()) == L.MOE_ERR_DEVICE
    _, _, val = R.fp4_quantize(x, fmt)
    assert np.array_equal(got[:4], val, equal_nan=True)
    assert (got[4:] == 0).all() and int(np.isnan(got).sum()) == int(np.isnan(val).sum()) > 0


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("offs", [[0, 9, 4, 8], [3, 5, 8, 8], [-7, 2, 90, 8]])
def test_bad_offset_tables_touch_nothing_outside(L, fmt, offs):
    rows, cols = 8, 64
    nb = L.moe_fp4_scale_bytes(rows, cols, FMT[fmt], 1, 3)
    buf = torch.full((nb + 8192,), 0xCD, dtype=torch.uint8, device="cuda")
    q = torch.full((rows + 8, 32), 0xAB, dtype=torch.uint8, device="cuda")
    L.moe_fp4_quantize(torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda"), FMT[fmt],
                       q[:rows], buf[:nb], group_offsets=i32(offs))
    assert (buf[nb:] == 0xCD).all() and (q[rows:] == 0xAB).all()
    if offs[0] > 0:
        assert (q[:offs[0]] == 0xAB).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("row_map", ["experts", "swiglu"])
@pytest.mark.parametrize("E,K,N", [(1, 32, 64), (2, 96, 192), (3, 160, 448)])
def test_weights_and_arranged_scales(L, fmt, row_map, E, K, N):
    rng = np.random.default_rng(K + N)
    m = 3 if row_map == "experts" else 2
    w = f64(bf16(rng.standard_normal((E, K, N)) * 0.02))
    g = np.exp2(-6.0 - np.arange(E)).astype(np.float32)
    gt = torch.from_numpy(g).cuda()
    nbytes = L.moe_fp4_scale_bytes(E * N, K, FMT[fmt], m, E)
    q = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    sf, sf2, sf3 = (torch.full((nbytes,), 0xEE, dtype=torch.uint8, device="cuda")
                    for _ in range(3))
    L.moe_fp4_quantize_weights(bf16(w), FMT[fmt], m, q, sf, gt)
    wt = w.transpose(0, 2, 1).reshape(E * N, K)
    parts = [R.fp4_quantize(wt[e * N:(e + 1) * N], fmt, float(g[e])) for e in range(E)]
    el, code, val = (np.concatenate(p) for p in zip(*parts))
    got = R.unpack(q.view(E * N, K // 2).cpu().numpy())
    assert ((got == el) | ((el & 7 == 0) & (got & 7 == 0))).all()
    ac = -(-K // (64 if fmt == "nv" else 128))
    at = [R.padded_row(r, N, row_map) for r in range(E * N)]
    s = grouped_scales(sf.cpu().numpy(), at, 4 * ac, ac)
    nb = code.shape[1]
    assert (s[:, :nb] == code).all() and (s[:, nb:] == 0).all()
    # the same atoms from row-order scales, and from K-major bf16 weights
    L.moe_fp4_arrange_scales(torch.from_numpy(np.ascontiguousarray(code)).cuda(), K, FMT[fmt], m, E, sf2)
    assert (grouped_scales(sf2.cpu().numpy(), at, 4 * ac, ac) == s).all()
    q3 = torch.empty(E * N, K // 2, dtype=torch.uint8, device="cuda")
    L.moe_fp4_quantize(bf16(wt), FMT[fmt], q3, sf3, row_map=m, groups=E, scale=gt)
    assert (q3 == q.view(E * N, K // 2)).all()
    assert (grouped_scales(sf3.cpu().numpy(), at, 4 * ac, ac) == s).all()
    out = torch.empty(E * N, K, dtype=torch.bfloat16, device="cuda")
    L.moe_fp4_dequantize(q3, sf3, FMT[fmt], out, row_map=m, groups=E, scale=gt)
    assert (f64(out) == val).all()  # powers of two as g: exact in bf16


def gemm_case(L, fmt, sizes, K, N, seed=0, swiglu=False):
    rng = np.random.default_rng(seed)
    off = offsets_of(sizes)
    E, cap = len(sizes), int(off[-1]) + 3
    x = f64(bf16(rng.standard_normal((cap, K))))
    w = f64(bf16(rng.standard_normal((E * N, K)) * K ** -0.5))
    ga, gb = np.float32(0.0625), np.exp2(-8.0 - np.arange(E)).astype(np.float32)
    m = 2 if swiglu else 3
    A = torch.empty(cap, K // 2, dtype=torch.uint8, device="cuda")
    sfa = torch.empty(L.moe_fp4_scale_bytes(cap, K, FMT[fmt], 1, E), dtype=torch.uint8,
                      device="cuda")
    B = torch.empty(E * N, K // 2, dtype=torch.uint8, device="cuda")
    sfb = torch.empty(L.moe_fp4_scale_bytes(E * N, K, FMT[fmt], m, E), dtype=torch.uint8,
                      device="cuda")
    o = i32(off)
    gat, gbt = torch.tensor([float(ga)], device="cuda"), torch.from_numpy(gb).cuda()
    if fmt == "mx":
        gat = gbt = None
        ga, gb = 1.0, np.ones(E)
    L.moe_fp4_quantize(bf16(x), FMT[fmt], A, sfa, group_offsets=o, scale=gat)
    L.moe_fp4_quantize(bf16(w), FMT[fmt], B, sfb, row_map=m, groups=E, scale=gbt)
    xv = R.fp4_quantize(x, fmt, float(ga))[2]
    wv = np.concatenate([R.fp4_quantize(w[e * N:(e + 1) * N], fmt, float(gb[e]))[2]
                         for e in range(E)]).reshape(E, N, K)
    S, mag = np.zeros((int(off[-1]), N)), np.zeros((int(off[-1]), N))
    for e in range(E):
        r = slice(off[e], off[e + 1])
        S[r] = xv[r] @ wv[e].T
        mag[r] = np.abs(xv[r]) @ np.abs(wv[e]).T
    return dict(A=A, sfa=sfa, B=B.view(E, N, K // 2), sfb=sfb, off=o, a_scale=gat, b_scale=gbt,
                S=S, mag=mag, n=int(off[-1]), cap=cap)


CASES = [([5], 32, 8), ([1, 0, 2], 64, 24), ([130, 1, 127, 0, 300], 512, 200),
         ([3, 256], 1056, 384), ([40], 4096, 576)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("sizes,K,N", CASES)
def test_gmm_plain(L, fmt, f32, sizes, K, N):
    c = gemm_case(L, fmt, sizes, K, N)
    C = torch.full((c["cap"], N), 9.0, dtype=torch.float32 if f32 else torch.bfloat16,
                   device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.moe_gmm_fp4(c["A"], c["sfa"], c["B"], c["sfb"], FMT[fmt], c["off"], C=C,
                  a_scale=c["a_scale"], b_scale=c["b_scale"], dev_status=st)
    got = f64(C)
    assert int(st.item()) == 0
    tol = (0.0 if f32 else R.bf16_half_step(c["S"])) + 2.0 ** -16 * c["mag"]
    assert (np.abs(got[:c["n"]] - c["S"]) <= tol).all()
    assert (got[c["n"]:] == 9.0).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("save_h", [False, True])
@pytest.mark.parametrize("sizes,K,F", [([5], 32, 32), ([1, 0, 2], 64, 96), ([130, 1, 300], 512, 416),
                                       ([40], 4096, 288), ([515], 160, 96),
                                       ([700, 0, 3, 1345], 544, 416)])
def test_gmm_swiglu_quantises_act(L, fmt, save_h, sizes, K, F):
    c = gemm_case(L, fmt, sizes, K, 2 * F, swiglu=True)
    n, cap, E = c["n"], c["cap"], len(sizes)
    q2 = torch.full((cap, F // 2), 0xAB, dtype=torch.uint8, device="cuda")
    sf2 = torch.full((L.moe_fp4_scale_bytes(cap, F, FMT[fmt], 1, E),), 0xCD, dtype=torch.uint8,
                     device="cuda")
    H = torch.full((cap, 2 * F), 9.0, dtype=torch.bfloat16, device="cuda") if save_h else None
    g2 = 0.03125
    g2t = torch.tensor([g2], device="cuda") if fmt == "nv" else None
    L.moe_gmm_fp4(c["A"], c["sfa"], c["B"], c["sfb"], FMT[fmt], c["off"],
                  epilogue=L.EPI_SWIGLU_FWD, C=H, Q2=q2, sf2=sf2, a_scale=c["a_scale"],
                  b_scale=c["b_scale"], q2_scale=g2t)
    act = R.swiglu(c["S"])
    el, code, val = R.fp4_quantize(act, fmt, g2)
    ac = -(-F // (64 if fmt == "nv" else 128))
    s = grouped_scales(sf2.cpu().numpy(), padded_rows(sizes), 4 * ac, ac)
    nb = code.shape[1]
    assert (s[:, nb:] == 0).all()
    got_el = R.unpack(q2.cpu().numpy()[:n])
    got = R.fp4_values(got_el, s[:, :nb], fmt, g2)
    off_codes = np.mean(got != val)
    assert off_codes <= 1e-3 + 64.0 / val.size and np.mean(s[:, :nb] != code) <= 1e-3 + 2.0 / code.size
    assert np.linalg.norm(got - val) <= 1e-2 * np.linalg.norm(val)
    assert (q2.cpu().numpy()[n:] == 0xAB).all()
    if save_h:
        h = f64(H)
        assert (np.abs(h[:n] - c["S"]) <= R.bf16_half_step(c["S"]) + 2.0 ** -16 * c["mag"]).all()
        assert (h[n:] == 9.0).all()


# three to four tiles a pair of CTAs (on 76 of them), token tiles of every kind: one
# token, exactly 128, 192 and 256, one more, two and three like ones
ROUNDS = [([300, 0, 256, 193, 515], 288, 8448), ([256, 256, 257, 128], 32, 8448),
          ([1, 192, 640, 31, 385], 544, 6400), ([130, 300], 2848, 6600)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("sizes,K,N", ROUNDS)
def test_gmm_plain_over_many_tiles(L, fmt, sizes, K, N):
    """Accumulators and their shared columns handed on from tile to tile."""
    c = gemm_case(L, fmt, sizes, K, N, seed=N)
    C = torch.full((c["cap"], N), 9.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        C.fill_(9.0)
        L.moe_gmm_fp4(c["A"], c["sfa"], c["B"], c["sfb"], FMT[fmt], c["off"], C=C,
                      a_scale=c["a_scale"], b_scale=c["b_scale"])
        got = f64(C)
        tol = R.bf16_half_step(c["S"]) + 2.0 ** -16 * c["mag"]
        assert (np.abs(got[:c["n"]] - c["S"]) <= tol).all()
        assert (got[c["n"]:] == 9.0).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("sizes,K,F", [([300, 0, 256, 193, 515], 2848, 2080),
                                       ([1, 192, 270, 31, 385], 96, 3296),
                                       ([300, 0, 700, 193, 515], 96, 3296)])
def test_gmm_swiglu_over_many_tiles(L, fmt, sizes, K, F):
    """Both forms (weights as M: long K or few rows; tokens as M), H in bf16: every
    value within a rounding and the fp32 sums' error."""
    c = gemm_case(L, fmt, sizes, K, 2 * F, seed=F, swiglu=True)
    n, cap, E = c["n"], c["cap"], len(sizes)
    q2 = torch.full((cap, F // 2), 0xAB, dtype=torch.uint8, device="cuda")
    sf2 = torch.empty(L.moe_fp4_scale_bytes(cap, F, FMT[fmt], 1, E), dtype=torch.uint8, device="cuda")
    H = torch.full((cap, 2 * F), 9.0, dtype=torch.bfloat16, device="cuda")
    g2 = 0.03125
    L.moe_gmm_fp4(c["A"], c["sfa"], c["B"], c["sfb"], FMT[fmt], c["off"],
                  epilogue=L.EPI_SWIGLU_FWD, C=H, Q2=q2, sf2=sf2, a_scale=c["a_scale"],
                  b_scale=c["b_scale"],
                  q2_scale=torch.tensor([g2], device="cuda") if fmt == "nv" else None)
    h = f64(H)
    assert (np.abs(h[:n] - c["S"]) <= R.bf16_half_step(c["S"]) + 2.0 ** -16 * c["mag"]).all()
    assert (h[n:] == 9.0).all()
    val = R.fp4_quantize(R.swiglu(c["S"]), fmt, g2)[2]
    ac = -(-F // (64 if fmt == "nv" else 128))
    s = grouped_scales(sf2.cpu().numpy(), padded_rows(sizes), -(-F // (16 if fmt == "nv" else 32)), ac)
    got = R.fp4_values(R.unpack(q2.cpu().numpy()[:n]), s, fmt, g2)
    assert np.mean(got != val) <= 1e-3
    assert np.linalg.norm(got - val) <= 1e-2 * np.linalg.norm(val)
    assert (q2.cpu().numpy()[n:] == 0xAB).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_a_nan_block_reaches_its_row_alone(L, fmt):
    c = gemm_case(L, fmt, [6], 256, 64)
    ac = 256 // (64 if fmt == "nv" else 128)
    sfa = c["sfa"].clone()
    sfa[R.scale_byte(2, 3, ac)] = 0x7F if fmt == "nv" else 0xFF
    C = torch.empty(c["cap"], 64, dtype=torch.float32, device="cuda")
    L.moe_gmm_fp4(c["A"], sfa, c["B"], c["sfb"], FMT[fmt], c["off"], C=C, a_scale=c["a_scale"],
                  b_scale=c["b_scale"])
    got = f64(C)[:6]
    assert np.isnan(got[2]).all() and np.isfinite(np.delete(got, 2, 0)).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T,d,f,E,k", [(1, 64, 32, 4, 2), (33, 160, 224, 5, 2), (300, 256, 512, 8, 3)])
def test_experts_on_another_stream(lowbit, L, fmt, T, d, f, E, k):
    """The whole FFN, weights quantised from bf16, launched on a stream of its own."""
    rng = np.random.default_rng(T)
    x, wi = rng.standard_normal((T, d)), 0.3 * rng.standard_normal((E, d, 2 * f)) * d ** -0.5
    wo = 0.3 * rng.standard_normal((E, f, d)) * f ** -0.5
    x, wi, wo = (f64(bf16(a)) for a in (x, wi, wo))
    idx = np.array([rng.permutation(E)[:k] for _ in range(T)])
    flat = idx.reshape(-1)
    order = np.argsort(flat, kind="stable")
    off = offsets_of(np.bincount(flat, minlength=E))
    gx, gact = (0.0078125, 0.0009765625) if fmt == "nv" else (1.0, 1.0)
    t = lambda v: torch.tensor([v], dtype=torch.float32, device="cuda")  # noqa: E731
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        w = lowbit.Fp4Experts.from_weights(fmt, bf16(wi), bf16(wo), t(gx), t(gact))
        b = lowbit.Fp4Buffers(w, T * k)
        y = lowbit.fp4_experts(w, b, bf16(x), i32(order), k, i32(off))
    s.synchronize()
    assert int(b.dev_status.item()) == 0
    gi = f64(w.wi_scale) if fmt == "nv" else np.ones(E)
    go = f64(w.wo_scale) if fmt == "nv" else np.ones(E)
    xq = R.fp4_quantize(x, fmt, gx)[2][order // k]
    want = np.zeros((T * k, d))
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        act = R.swiglu(xq[r] @ R.fp4_quantize(wi[e].T, fmt, gi[e])[2].T)
        want[r] = R.fp4_quantize(act, fmt, gact)[2] @ R.fp4_quantize(wo[e].T, fmt, go[e])[2].T
    got = f64(y)
    # Act's codes may move as above
    assert np.linalg.norm(got - want) <= 1e-2 * np.linalg.norm(want)


def test_no_rows(L):
    c = gemm_case(L, "nv", [4], 64, 64)
    C = torch.full((c["cap"], 64), 9.0, dtype=torch.bfloat16, device="cuda")
    L.moe_gmm_fp4(c["A"], c["sfa"], c["B"], c["sfb"], 1, i32([0, 0]), C=C)
    L.moe_gmm_fp4(c["A"][:0], c["sfa"], c["B"], c["sfb"], 1, i32([0, 0]), C=C[:0])
    assert (C == 9.0).all()


def test_a_wait_that_runs_out_is_reported(L):
    c = gemm_case(L, "mx", [40], 512, 192)
    C = torch.empty(c["cap"], 192, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.moe_set_wait_limit_ns(5_000_000)
    L.moe_test_stall_loads(True)
    try:
        L.moe_gmm_fp4(c["A"], c["sfa"], c["B"], c["sfb"], 0, c["off"], C=C, dev_status=st)
        torch.cuda.synchronize()
    finally:
        L.moe_test_stall_loads(False)
        L.moe_set_wait_limit_ns(2_000_000_000)
    assert int(st.item()) == L.MOE_ERR_TIMEOUT
    st.zero_()
    L.moe_gmm_fp4(c["A"], c["sfa"], c["B"], c["sfb"], 0, c["off"], C=C, dev_status=st)
    assert int(st.item()) == 0
