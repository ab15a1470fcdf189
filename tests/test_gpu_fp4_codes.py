"""Experts from a 4-bit checkpoint's codes: the same atoms, and the same outputs bit for bit, as
experts quantised from the bf16 weights that the codes stand for."""
import numpy as np
import pytest
import torch

from oracle import lowbit_ref as R
from test_gpu_fp4 import bf16, f64, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("E,d,f", [(1, 64, 32), (5, 160, 224)])
@pytest.mark.parametrize("typed", [False, True])
def test_from_codes_is_from_weights(fmt, E, d, f, typed):
    from mixture_experts_grouped_router_gb300 import lowbit
    rng = np.random.default_rng(E)
    wi = f64(bf16(rng.standard_normal((E, d, 2 * f)) * d ** -0.5))
    wo = f64(bf16(rng.standard_normal((E, f, d)) * f ** -0.5))
    t = torch.tensor([0.0078125], device="cuda") if fmt == "nv" else None
    want = lowbit.Fp4Experts.from_weights(fmt, bf16(wi), bf16(wo), t, t)

    def checkpoint(w, g):  # codes and scales in row order, by the oracle
        parts = [R.fp4_quantize(w[e].T, fmt, 1.0 if g is None else float(g[e])) for e in range(E)]
        q = np.ascontiguousarray([R.pack(p[0]) for p in parts])
        s = torch.from_numpy(np.ascontiguousarray([p[1] for p in parts])).cuda()
        if typed and fmt == "nv":
            s = s.view(torch.float8_e4m3fn)
        return torch.from_numpy(q).cuda(), s

    (qi, si), (qo, so) = checkpoint(wi, want.wi_scale), checkpoint(wo, want.wo_scale)
    got = lowbit.Fp4Experts.from_codes(fmt, qi, si, want.wi_scale, qo, so, want.wo_scale, t, t)
    T, k = 37, min(2, E)
    x = bf16(rng.standard_normal((T, d)))
    idx = np.array([rng.permutation(E)[:k] for _ in range(T)]).reshape(-1)
    order = i32(np.argsort(idx, kind="stable"))
    off = i32(np.concatenate([[0], np.cumsum(np.bincount(idx, minlength=E))]))
    ys = []
    for w in (want, got):
        b = lowbit.Fp4Buffers(w, T * k)
        ys.append(lowbit.fp4_experts(w, b, x, order, k, off).clone())
        assert int(b.dev_status.item()) == 0
    assert ys[0].abs().max() > 0 and torch.equal(*ys)
    # the atoms of every row that there is
    for sf, sw, N, K, m in ((got.wi_sf, want.wi_sf, 2 * f, d, "swiglu"), (got.wo_sf, want.wo_sf, d, f, "experts")):
        nb = K // (16 if fmt == "nv" else 32)
        ac = -(-nb // 4)
        at = [R.scale_byte(R.padded_row(r, N, m), b, ac) for r in range(E * N) for b in range(4 * ac)]
        at = torch.tensor(at, device="cuda")
        assert torch.equal(sf[at], sw[at])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_a_short_permutation_in_larger_buffers(fmt):
    """rows below the buffers' rows_cap, with a sorted_to_flat of just as many: the same outputs
    as buffers of that size give, the rest of y untouched."""
    from mixture_experts_grouped_router_gb300 import lowbit
    rng = np.random.default_rng(5)
    E, d, f, T = 4, 96, 64, 21
    w = lowbit.Fp4Experts.from_weights(fmt, bf16(rng.standard_normal((E, d, 2 * f))),
                                       bf16(rng.standard_normal((E, f, d))))
    x = bf16(rng.standard_normal((T, d)))
    order, off = i32(rng.permutation(T)), i32([0, 3, 3, 15, T])
    want = lowbit.fp4_experts(w, lowbit.Fp4Buffers(w, T), x, order, 1, off)
    b = lowbit.Fp4Buffers(w, 300)
    b.y.fill_(9.0)
    got = lowbit.fp4_experts(w, b, x, order, 1, off, rows=T)
    assert torch.equal(got[:T], want) and (got[T:] == 9.0).all()
    assert int(b.dev_status.item()) == 0
    for rows, s2f in ((T, order[:-1]), (301, order), (-1, order), (None, order)):
        with pytest.raises(ValueError, match="rows"):
            lowbit.fp4_experts(w, b, x, s2f, 1, off, rows=rows)
