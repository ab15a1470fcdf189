"""The global gradient norm and clipping against the fp64 oracle.  Tolerances: squares are summed
in fp32 8 at a time (4 additions and a product: 5 half-ulps of a sum of positive terms), then in
64 bits; the root halves that, one rounding to fp32 at the end: 2^-21.  A clipped value is off by the
norm's error, the products' and the rounding to its type."""
import numpy as np
import pytest
import torch

from oracle import block_ref as R
from oracle.lowbit_ref import bf16_half_step

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def block():
    from mixture_experts_grouped_router_gb300 import block
    return block


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64).ravel()


def check_outs(grads, outs, factor, slack=2.0 ** -20):
    for g, o in zip(grads, outs):
        want = g * factor
        half = bf16_half_step(want) if o.dtype == BF else np.abs(want) * 2.0 ** -24 + 2.0 ** -149
        assert (np.abs(f64(o) - want) <= half + slack * np.abs(want)).all()


SETS = [[1], [8], [0, 3], [4096, 1, 1023, 1024, 1025, 7, 0, 33], [100000], [1 << 21, 12345],
        [(1 << 24) + 1000, 17]]


@pytest.mark.parametrize("sizes", SETS, ids=str)
@pytest.mark.parametrize("types", ["bf16", "fp32", "mixed"])
@pytest.mark.parametrize("into", ["place", "same", "fp32", "bf16"])
def test_norm_and_clip(block, sizes, types, into):
    gen = torch.Generator(device="cuda").manual_seed(len(sizes))
    t = {"bf16": [BF], "fp32": [F32], "mixed": [BF, F32]}[types]
    grads = [torch.randn(n, generator=gen, device="cuda").to(t[i % len(t)]) for i, n in enumerate(sizes)]
    values = [f64(g) for g in grads]
    outs = None
    if into != "place":
        want_t = {"same": None, "fp32": F32, "bf16": BF}[into]
        outs = [torch.full_like(g, 9.0, dtype=want_t or g.dtype) for g in grads]
    c = block.GradClip(grads, outs)
    norm, _ = R.clip(values, 1.0, 0.25)
    assert abs(float(c.norm(0.25)) - norm) <= 2.0 ** -21 * norm
    assert all((f64(g) == v).all() for g, v in zip(grads, values))
    most = 0.3 * norm
    want_norm, factor = R.clip(values, most, 0.25)
    assert abs(float(c.clip(most, 0.25)) - want_norm) <= 2.0 ** -21 * want_norm
    check_outs(values, grads if outs is None else outs, factor)


@pytest.mark.parametrize("shift", [1, 2, 3, 5, 7])
@pytest.mark.parametrize("out_shift", [None, 0, 1, 4])
@pytest.mark.parametrize("g_type,o_type", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_views_at_odd_offsets(block, shift, out_shift, g_type, o_type):
    n = 5000
    gen = torch.Generator(device="cuda").manual_seed(shift)
    whole = torch.randn(n + 16, generator=gen, device="cuda").to(g_type)
    g = whole[shift:shift + n]
    v, before = f64(g), whole.clone()
    outs, ow = None, None
    if out_shift is not None:
        ow = torch.full((n + 16,), 9.0, dtype=o_type, device="cuda")
        outs = [ow[out_shift:out_shift + n]]
    elif g_type != o_type:
        pytest.skip("in place with one type")
    c = block.GradClip([g], outs)
    norm, factor = R.clip([v], 2.0, 1.0)
    assert abs(float(c.clip(2.0)) - norm) <= 2.0 ** -21 * norm
    check_outs([v], [g if outs is None else outs[0]], factor)
    if outs is None:  # what lies around the view stays
        assert torch.equal(whole[:shift], before[:shift]) and torch.equal(whole[shift + n:], before[shift + n:])
    else:
        assert torch.equal(whole, before)
        assert (ow[:out_shift] == 9.0).all() and (ow[out_shift + n:] == 9.0).all()


def test_small_norms_are_not_clipped(block):
    g = torch.tensor([3.0, 4.0], device="cuda")
    out = torch.empty_like(g)
    assert float(block.GradClip([g], [out]).clip(5.1)) == 5.0 and torch.equal(out, g)
    assert float(block.GradClip([g]).clip(float("inf"))) == 5.0 and g.tolist() == [3.0, 4.0]
    assert float(block.GradClip([g], [out]).clip(float("inf"), 0.5)) == 2.5 and out.tolist() == [1.5, 2.0]
    assert float(block.GradClip([g], [out]).clip(0.0)) == 5.0 and out.tolist() == [0.0, 0.0]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-22, 1e-12, 1e18, 1e25, 1e35])
def test_squares_past_fp32(block, dtype, size):
    """Values whose squares are over or under fp32's range, alone and beside ordinary ones."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    base = torch.randn(3001, generator=gen, device="cuda").double().clamp(-2.5, 2.5)
    g = (base * size).to(dtype)
    v = f64(g)
    norm = float(np.sqrt((v * v).sum()))
    got = float(block.GradClip([g]).norm())
    # (a subnormal norm's own spacing)
    assert abs(got - norm) <= 2.0 ** -21 * norm + 2.0 ** -149
    mixed = block.GradClip([g, torch.zeros(5000, dtype=BF, device="cuda"), torch.ones(100, device="cuda")])
    both = float(np.sqrt((v * v).sum() + 100.0))
    assert abs(float(mixed.norm()) - both) <= 2.0 ** -21 * both
    out = torch.empty_like(g)
    float(block.GradClip([g], [out]).clip(0.5 * norm if norm > 1e-4 else 1.0))
    if norm > 1e-4:
        check_outs([v], [out], 0.5 / (1 + 1e-6 / norm))
    else:
        assert torch.equal(out, g)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_norm_that_is_no_number_clips_nothing(block, bad):
    g = torch.ones(3000, device="cuda").to(BF)
    g[1234] = bad
    before = g.clone()
    c = block.GradClip([g])
    n = float(c.clip(1.0))
    assert (np.isnan(n) if np.isnan(bad) else n == np.inf)
    torch.testing.assert_close(g, before, rtol=0, atol=0, equal_nan=True)


def test_same_numbers_each_time_and_zeros(block):
    gen = torch.Generator(device="cuda").manual_seed(8)
    g = [torch.randn(n, generator=gen, device="cuda").to(BF) for n in (70001, 300000, 5)]
    c = block.GradClip(g)
    assert len({float(c.norm()) for _ in range(5)}) == 1
    z = torch.zeros(9999, device="cuda")
    assert float(block.GradClip([z]).clip(1.0)) == 0.0 and (z == 0).all()


def test_many_tensors(block):
    gen = torch.Generator(device="cuda").manual_seed(9)
    g = [torch.randn(1 + (i * 37) % 500, generator=gen, device="cuda").to(BF if i % 3 else F32) for i in range(1500)]
    v = [f64(t) for t in g]
    norm, factor = R.clip(v, 1.0, 1.0)
    assert abs(float(block.GradClip(g).clip(1.0)) - norm) <= 2.0 ** -21 * norm
    check_outs(v, g, factor)


def test_a_tensor_past_32_bits(block):
    n = (1 << 32) + 4099
    g = torch.zeros(n, dtype=BF, device="cuda")
    at = torch.tensor([0, (1 << 31) + 1, (1 << 32) + 4098], device="cuda")
    g[at] = torch.tensor([3.0, 4.0, 12.0], device="cuda").to(BF)
    c = block.GradClip([g])
    assert float(c.clip(6.5)) == 13.0
    assert g[at].tolist() == [1.5, 2.0, 6.0] and int(torch.count_nonzero(g)) == 3


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("low,high", [(-38, 38), (-38, -10), (-20, -8), (8, 38), (-15, -13), (17, 20)])
def test_neighbours_of_any_size(block, dtype, low, high):
    """Values of up to 76 powers of ten side by side, some of them 0.  At most 32 squares are added
    one after the other in fp32, which the root halves; its own and two more roundings."""
    gen = torch.Generator(device="cuda").manual_seed(high - low)
    e = torch.rand(20003, generator=gen, device="cuda", dtype=torch.float64) * (high - low) + low
    sign = torch.randint(-1, 2, (20003,), generator=gen, device="cuda")
    for n in (20003, 4099, 31, 1):
        g = (10.0 ** e * sign)[:n].to(dtype)
        v = f64(g)
        norm = float(np.sqrt((v * v).sum()))
        got = float(block.GradClip([g]).norm())
        if norm > 3.4e38:
            assert got == float("inf") or got >= 3.4e38 * (1 - 2.0 ** -20)
        else:
            assert abs(got - norm) <= 20 * 2.0 ** -24 * norm + 2.0 ** -149


@pytest.mark.parametrize("n", [1, 6, 9, 255, 2047, 2049, 70001])
@pytest.mark.parametrize("shifts", [(1, 0), (0, 1), (4, 0), (3, 5), (8, 1)], ids=str)
@pytest.mark.parametrize("g_type,o_type", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_views_that_start_apart(block, n, shifts, g_type, o_type):
    """Slices of a flat buffer of gradients written to tensors of their own, and the other way."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    whole = torch.randn(n + 24, generator=gen, device="cuda").to(g_type)
    ow = torch.full((n + 24,), 9.0, dtype=o_type, device="cuda")
    g, o = whole[shifts[0]:][:n], ow[shifts[1]:][:n]
    v = f64(g)
    small = torch.ones(3, device="cuda")
    c = block.GradClip([g, small], [o, torch.empty(3, device="cuda")])
    want, factor = R.clip([v, np.ones(3)], 0.5, 1.0)
    assert abs(float(c.clip(0.5)) - want) <= 20 * 2.0 ** -24 * want
    check_outs([v], [o], factor)
    assert (ow[:shifts[1]] == 9).all() and (ow[shifts[1] + n:] == 9).all()
    c.clip(1e9)
    assert torch.equal(o, g.to(o_type))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_norm_past_fp32_clips_nothing(block, dtype):
    """The norm that is returned is infinite: nothing is clipped, as where a gradient is."""
    g = torch.full((3000,), 3e38, device="cuda").to(dtype)
    g[::7] = 1.0
    before = g.clone()
    assert float(block.GradClip([g]).clip(1.0)) == float("inf") and torch.equal(g, before)
    out = torch.empty_like(g)
    assert float(block.GradClip([g], [out]).clip(1.0, 0.5)) == float("inf") and torch.equal(out, 0.5 * g)


@pytest.mark.parametrize("g_type,o_type", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("size,scale,most", [(1e36, 1.0, 1e-3), (1e38, 2.0 ** -3, 1e-2), (1e14, 1.0, 1e-30),
                                             (1e30, 1e-30, 1e-15), (3e37, 1e-8, 1e-12), (1e20, 1.0, 1e-19)])
@pytest.mark.parametrize("shift", [0, 1])
def test_factors_under_fp32(block, g_type, o_type, size, scale, most, shift):
    """Factors that fp32 holds with few bits or not at all, of gradients large enough that the
    clipped ones are ordinary numbers; also into a tensor that starts apart.  The norm's error and one
    half-ulp more, as elsewhere: 2^-20."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    n = 5003
    g = (size * torch.randn(n, generator=gen, device="cuda").clamp(-2, 2)).to(g_type)
    g[5], g[6] = 0.0, 1e-30
    whole = torch.empty(n + 8, dtype=o_type, device="cuda")
    v, s = f64(g), float(np.float32(scale))
    c = block.GradClip([g], [whole[shift:shift + n]])
    norm, factor = R.clip([v], float(np.float32(most)), s)
    got = float(c.clip(most, scale))
    if norm > 3.402823466e38:  # as documented: infinite, and not clipped
        assert got == float("inf")
        factor = s
    else:
        assert abs(got - norm) <= 20 * 2.0 ** -24 * norm
    check_outs([v], [whole[shift:shift + n]], factor)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_scale_that_brings_the_norm_back(block, dtype):
    """The norm of these values is past fp32, the scaled one is not: clipped, by a factor under fp32."""
    g = torch.full((3000,), 3e38, device="cuda").to(dtype)
    g[::7] = 1.0
    out = torch.empty_like(g)
    want, factor = R.clip([f64(g)], 1.0, 2.0 ** -20)  # a scale that brings it back
    assert abs(float(block.GradClip([g], [out]).clip(1.0, 2.0 ** -20)) - want) <= 20 * 2.0 ** -24 * want
    check_outs([f64(g)], [out], factor)
