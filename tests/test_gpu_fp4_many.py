"""4-bit operators with more experts than a warp has lanes, and with padded leading dimensions.

Tolerances: codes and scales of bf16 inputs bit for bit (fp32 scales of few bits).  A product is
within one rounding to bf16 (half its spacing) and 2^-16 of sum |a b| for the fp32 sums.  An Act
value differs from the 64-bit one by what those sums' error makes of it (silu has slopes under
1.1) and 2^-20 of itself for the exponential, the reciprocal and the products; its code may
differ only where a tie lies that near, and only by one, and a block's scale likewise."""
import numpy as np
import pytest
import torch

from oracle import lowbit_ref as R
from test_gpu_fp4 import FMT, bf16, f64, i32, offsets_of, padded_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from mixture_experts_grouped_router_gb300 import _lib
    return _lib


def ragged(E, seed, most=9):
    """Sizes of E groups: many empty, a few rows, some that fill an atom of 128 rows or pass
    it by one, on both sides of every 32nd; the last ones empty."""
    rng = np.random.default_rng(seed)
    s = rng.integers(0, most, E) * (rng.random(E) < 0.6)
    for e in range(0, E, 32):
        s[e] = rng.choice([127, 128, 129])
        if e:
            s[e - 1] = rng.choice([1, 128, 129])
    s[-2:] = 0
    return [int(v) for v in s]


def codes_at(sf, rows_at, nb, ac):
    p, b = np.array(rows_at)[:, None], np.arange(nb)[None]
    return sf.cpu().numpy()[((p // 128) * ac + b // 4) * 512 + (p % 32) * 16 + (p % 128 // 32) * 4 + b % 4]


def padded(rows, cols, pad, dtype, fill):
    t = torch.full((rows, cols + pad), fill, dtype=dtype, device="cuda")
    return t, t[:, :cols]


def untouched(t, cols, fill, rows=None):
    """Nothing past the columns, nor past the rows, has been written."""
    t = t.view(torch.int16) if t.dtype == torch.bfloat16 else t
    fill = int(torch.tensor(fill).bfloat16().view(torch.int16)) if t.dtype == torch.int16 else fill
    return bool((t[:, cols:] == fill).all()) and (rows is None or bool((t[rows:] == fill).all()))


MANY = [33, 64, 65, 256]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("E", MANY)
@pytest.mark.parametrize("pad", [0, 32])
def test_quantize_and_dequantize(L, fmt, E, pad):
    sizes = ragged(E, E)
    n, cols = sum(sizes), 160
    cap = n + 5
    rng = np.random.default_rng(E)
    x = f64(bf16(rng.standard_normal((n // 2 + 1, cols)) * np.exp2(rng.integers(-9, 9, (n // 2 + 1, 1)))))
    xt, xv = padded(len(x), cols, pad, torch.bfloat16, 3.0)
    xv.copy_(bf16(x))
    idx = rng.integers(-1, 2 * len(x), cap)
    g = torch.tensor([0.015625], device="cuda")
    qt, q = padded(cap, cols // 2, pad, torch.uint8, 0xAB)
    sf = torch.full((L.moe_fp4_scale_bytes(cap, cols, FMT[fmt], 1, E),), 0xCD, dtype=torch.uint8, device="cuda")
    off = i32(offsets_of(sizes))
    L.moe_fp4_quantize(xv, FMT[fmt], q, sf, group_offsets=off, row_index=i32(idx), index_div=2, scale=g)
    rows = np.where((idx >= 0)[:, None], x[np.maximum(idx, 0) // 2], 0.0)[:n]
    el, code, val = R.fp4_quantize(rows, fmt, 0.015625)
    got = R.unpack(q.cpu().numpy()[:n])
    assert ((got == el) | ((el & 7 == 0) & (got & 7 == 0))).all()
    ac = -(-cols // (64 if fmt == "nv" else 128))
    s = codes_at(sf, padded_rows(sizes), 4 * ac, ac)
    assert (s[:, :code.shape[1]] == code).all() and (s[:, code.shape[1]:] == 0).all()
    assert untouched(qt, cols // 2, 0xAB, n)
    ot, o = padded(cap, cols, pad, torch.bfloat16, 7.0)
    L.moe_fp4_dequantize(q, sf, FMT[fmt], o, group_offsets=off, scale=g)
    assert (f64(o)[:n] == f64(bf16(val))).all() and untouched(ot, cols, 7.0, n)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("E", MANY)
def test_linked_gather(L, fmt, E):
    sizes = ragged(E, E + 1)
    n, src, cols = sum(sizes), 60, 17408
    sizes[1] += max(0, 1000 - n)
    n = sum(sizes)
    assert n >= 2 * src and n * cols >= 1 << 24
    rng = np.random.default_rng(E)
    x = f64(bf16(rng.standard_normal((src, cols))))
    idx = rng.integers(-1, 3 * src, n)
    q = torch.empty(n, cols // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(L.moe_fp4_scale_bytes(n, cols, FMT[fmt], 1, E), dtype=torch.uint8, device="cuda")
    ws = torch.empty(L.moe_fp4_quantize_workspace_bytes(src, n), dtype=torch.uint8, device="cuda")
    L.moe_fp4_quantize(bf16(x), FMT[fmt], q, sf, group_offsets=i32(offsets_of(sizes)), row_index=i32(idx),
                       index_div=3, scale=torch.tensor([0.015625], device="cuda"), workspace=ws)
    el, code, _ = R.fp4_quantize(np.concatenate([x, np.zeros((1, cols))]), fmt, 0.015625)
    at = np.where(idx >= 0, idx // 3, src)
    el, code = el[at], code[at]
    got = R.unpack(q.cpu().numpy())
    assert ((got == el) | ((el & 7 == 0) & (got & 7 == 0))).all()
    s = codes_at(sf, padded_rows(sizes), code.shape[1], cols // (64 if fmt == "nv" else 128))
    assert (s == code).all()


def product(L, fmt, sizes, K, N, swiglu, pad=0, seed=0, cap=None):
    """Operands (leading dimensions `pad` longer), the 64-bit product S and sum |a b|."""
    rng = np.random.default_rng(seed)
    off = offsets_of(sizes)
    E, n = len(sizes), int(off[-1])
    cap = n + 3 if cap is None else cap
    x = f64(bf16(rng.standard_normal((cap, K))))
    w = f64(bf16(rng.standard_normal((E * N, K)) * K ** -0.5))
    ga, gb = 0.0625, np.exp2(-8.0 - np.arange(E) % 5)
    m = 2 if swiglu else 3
    nb = L.moe_fp4_scale_bytes
    A = padded(cap, K // 2, pad, torch.uint8, 0x77)[1]
    sfa = torch.full((nb(cap, K, FMT[fmt], 1, E),), 0x38, dtype=torch.uint8, device="cuda")
    Bt = torch.full((E, N + (2 if pad else 0), K // 2 + pad), 0x77, dtype=torch.uint8, device="cuda")
    B = Bt[:, :N, :K // 2]
    q = torch.empty(E * N, K // 2, dtype=torch.uint8, device="cuda")
    sfb = torch.full((nb(E * N, K, FMT[fmt], m, E),), 0x38, dtype=torch.uint8, device="cuda")
    gat, gbt = torch.tensor([ga], device="cuda"), torch.tensor(gb, dtype=torch.float32, device="cuda")
    L.moe_fp4_quantize(bf16(x), FMT[fmt], A, sfa, group_offsets=i32(off), scale=gat)
    L.moe_fp4_quantize(bf16(w), FMT[fmt], q, sfb, row_map=m, groups=E, scale=gbt)
    B.copy_(q.view(E, N, K // 2))
    if fmt == "mx":  # the products take the factors all the same
        xq = R.fp4_quantize(x, fmt)[2] * ga
        wq = R.fp4_quantize(w, fmt)[2].reshape(E, N, K) * gb[:, None, None]
    else:
        xq = R.fp4_quantize(x, fmt, ga)[2]
        wq = np.concatenate([R.fp4_quantize(w[e * N:(e + 1) * N], fmt, gb[e])[2] for e in range(E)])
        wq = wq.reshape(E, N, K)
    S, mag = np.zeros((n, N)), np.zeros((n, N))
    for e in range(E):
        r = slice(off[e], off[e + 1])
        S[r], mag[r] = xq[r] @ wq[e].T, np.abs(xq[r]) @ np.abs(wq[e]).T
    return dict(args=(A, sfa, B, sfb, FMT[fmt], i32(off)), scales=dict(a_scale=gat, b_scale=gbt),
                S=S, mag=mag, n=n, cap=cap, E=E)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("E,K,N,pad", [(33, 96, 72, 0), (64, 288, 264, 48), (65, 64, 136, 16),
                                       (256, 96, 40, 0), (256, 64, 512, 16)])
@pytest.mark.parametrize("f32", [False, True])
def test_plain(L, fmt, E, K, N, pad, f32):
    c = product(L, fmt, ragged(E, E + 2), K, N, False, pad, seed=E)
    Ct, C = padded(c["cap"], N, pad, torch.float32 if f32 else torch.bfloat16, 9.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.moe_gmm_fp4(*c["args"], C=C, dev_status=st, **c["scales"])
    assert int(st.item()) == 0
    tol = (0.0 if f32 else R.bf16_half_step(c["S"])) + 2.0 ** -16 * c["mag"]
    assert (np.abs(f64(C)[:c["n"]] - c["S"]) <= tol).all() and untouched(Ct, N, 9.0, c["n"])
    again = C.clone()
    L.moe_gmm_fp4(*c["args"], C=C, **c["scales"])
    assert torch.equal(again, C)  # the order of the sums is fixed


def check_act(c, F, fmt, g2, q, s):
    """Codes q [n, F] and scale codes s of Act against the 64-bit product's."""
    S, n = c["S"], c["n"]
    g, u, eg, eu = S[:, :F], S[:, F:], *np.split(2.0 ** -16 * c["mag"], 2, axis=1)
    act = R.swiglu(S)
    err = (1.1 * eg * (np.abs(u) + eu) + np.abs(g / (1 + np.exp(-g))) * eu) + 2.0 ** -20 * np.abs(act)
    blk = 16 if fmt == "nv" else 32
    el, code, _ = R.fp4_quantize(act, fmt, g2)
    a, ea = (np.abs(v).reshape(n, -1, blk).max(-1) for v in (act, err))
    if fmt == "nv":  # both ends of the largest magnitude round to neighbours
        lo, hi = (R.e4m3_code(R.round_e4m3(np.maximum(a + d, 0) / (6 * g2))).astype(int) for d in (-ea, ea))
    else:
        lo, hi = (np.clip(np.frexp(np.maximum(a + d, 2.0 ** -126))[1] - 3, -127, 127) + 127 for d in (-ea, ea))
    assert ((s >= lo) & (s <= hi)).all()
    t = R.e4m3_value(s) * g2 if fmt == "nv" else R.e8m0_value(s)
    t = np.repeat(np.where(a > 0, t, 1.0), blk, axis=1)
    def code_of(v):  # of a magnitude
        m = np.minimum(np.maximum(v, 0) / t, 6.0)
        step = np.exp2(np.floor(np.log2(np.maximum(m, 1.0))) - 1)
        return np.searchsorted(R.E2M1, np.rint(m / step) * step)
    mag = q & 7
    assert ((mag >= code_of(np.abs(act) - err)) & (mag <= code_of(np.abs(act) + err))).all()
    assert (((q >= 8) == (act < 0)) | (mag == 0) | (np.abs(act) <= err)).all()
    zeros = (mag == 0) & (el & 7 == 0)  # a zero's sign is not kept
    # fp32 sums of a few hundred terms are within 2^-19 of |a b|: some 10^-5 of the values
    assert np.mean((q != el) & ~zeros) <= 1e-4


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("E,K,F,pad,save_h", [(33, 96, 96, 0, True), (64, 288, 160, 48, False),
                                              (65, 64, 32, 16, True), (256, 96, 64, 0, False),
                                              (5, 544, 416, 16, True), (1, 4096, 288, 0, False)])
def test_swiglu(L, fmt, E, K, F, pad, save_h):
    c = product(L, fmt, ragged(E, E + 3) if E > 5 else [130, 0, 1, 300, 65][:E], K, 2 * F, True, pad, seed=E)
    run_swiglu(L, c, fmt, F, pad, save_h)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("E,K,F,pad,save_h", [(2, 160, 96, 0, False), (3, 544, 416, 48, True),
                                              (33, 64, 32, 0, True), (64, 96, 96, 16, False)])
def test_swiglu_with_tokens_as_m(L, fmt, E, K, F, pad, save_h):
    """As many rows an expert as take the other form, of groups of every size."""
    rng = np.random.default_rng(E)
    sizes = [int(v) for v in rng.integers(0, 400, E) * (rng.random(E) < 0.8)]
    sizes[0] = 1
    c = product(L, fmt, sizes, K, 2 * F, True, pad, seed=E, cap=max(256 * E, sum(sizes)) + 3)
    run_swiglu(L, c, fmt, F, pad, save_h)


def run_swiglu(L, c, fmt, F, pad, save_h):
    n, cap, E = c["n"], c["cap"], c["E"]
    qt, q2 = padded(cap, F // 2, pad, torch.uint8, 0xAB)
    sf2 = torch.full((L.moe_fp4_scale_bytes(cap, F, FMT[fmt], 1, E),), 0xCD, dtype=torch.uint8, device="cuda")
    ht, H = padded(cap, 2 * F, pad, torch.bfloat16, 9.0)
    g2 = 0.03125 if fmt == "nv" else 1.0
    L.moe_gmm_fp4(*c["args"], epilogue=L.EPI_SWIGLU_FWD, C=H if save_h else None, Q2=q2, sf2=sf2,
                  q2_scale=torch.tensor([g2], device="cuda"), **c["scales"])
    off = c["args"][5].cpu().numpy()
    ac, nb = -(-F // (64 if fmt == "nv" else 128)), F // (16 if fmt == "nv" else 32)
    s = codes_at(sf2, padded_rows(list(np.diff(off))), 4 * ac, ac).astype(int)
    assert (s[:, nb:] == 0).all()
    check_act(c, F, fmt, g2, R.unpack(q2.cpu().numpy()[:n]), s[:, :nb])
    assert untouched(qt, F // 2, 0xAB, n)
    if save_h:
        assert (np.abs(f64(H)[:n] - c["S"]) <= R.bf16_half_step(c["S"]) + 2.0 ** -16 * c["mag"]).all()
    assert untouched(ht, 2 * F, 9.0, n if save_h else 0)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("E,k,T", [(40, 8, 5), (64, 8, 200), (256, 8, 300)])
def test_serving_layer(fmt, E, k, T):
    """Against the fp64 layer on the values of the 4-bit weights, tokens and Act (relative
    Frobenius 1e-2: codes of Act that move across a tie)."""
    import moe_synth
    from gpu_helpers import dev_bf16
    from mixture_experts_grouped_router_gb300 import layer, lowbit
    from oracle import moe_ref
    cfg = moe_synth.MoEConfig("many", T=T, d=96, f=64, E=E, k=k)
    inp = moe_synth.make_inputs(cfg, seed=E)
    x, wi, wo = (moe_synth.bits_to_f64(inp[n]) for n in ("x", "wi", "wo"))
    gx, ga = (0.0078125, 0.0009765625) if fmt == "nv" else (1.0, 1.0)
    t = lambda v: torch.tensor([v], dtype=torch.float32, device="cuda")  # noqa: E731
    w = lowbit.Fp4Experts.from_weights(fmt, dev_bf16(inp["wi"]), dev_bf16(inp["wo"]), t(gx), t(ga))
    m = lowbit.Fp4Layer(w, layer.LayerShape(T, cfg.d, cfg.f, E, k))
    out = m.forward(dev_bf16(inp["x"]), torch.from_numpy(inp["logits"]).cuda())
    assert int(m.bufs.dev_status.item()) == 0
    gi, go = (f64(v) if fmt == "nv" else np.ones(E) for v in (w.wi_scale, w.wo_scale))
    fw = moe_ref.forward(x, inp["logits"], wi, wo, k, 0, 1, 0, 0)
    off, s2f = fw["layout"]["group_offsets"], np.asarray(fw["layout"]["sorted_to_flat"])
    xq, want = R.fp4_quantize(x, fmt, gx)[2], np.zeros((T, cfg.d))
    for e in range(E):
        r = s2f[off[e]:off[e + 1]]
        if len(r) == 0:
            continue
        a = R.swiglu(xq[r // k] @ R.fp4_quantize(wi[e].T, fmt, gi[e])[2].T)
        y = R.fp4_quantize(a, fmt, ga)[2] @ R.fp4_quantize(wo[e].T, fmt, go[e])[2].T
        np.add.at(want, r // k, fw["topk_w"].reshape(-1)[r][:, None] * y)
    assert np.linalg.norm(f64(out) - want) <= 1e-2 * np.linalg.norm(want)
