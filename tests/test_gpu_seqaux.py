"""The balance loss of sequences with the z loss against the fp64 oracle.  Tolerances: e^x of a
logit is within |x| 2^-24 + 2^-22 of itself (logits here are within 6 of 0: 2^-20.6), reciprocals
within 2^-23, a token's sums take at most 8 values a lane and 5 lanes' additions, each half an ulp:
2^-19 of a probability, twice that of the gradient's terms (2^-18 of their size); lse also half an
ulp of its own size and 2^-22 of the largest logit.  Means over tokens take at most `adds`
additions: adds 2^-24."""
import numpy as np
import pytest
import torch

from oracle import block_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def block():
    from mixture_experts_grouped_router_gb300 import block
    return block


@pytest.fixture(scope="module")
def L():
    from mixture_experts_grouped_router_gb300 import _lib
    return _lib


def f64(t):
    return t.detach().cpu().numpy().astype(np.float64)


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def case(T, E, k, seed=0):
    rng = np.random.default_rng(seed + 7 * T + E)
    x = (rng.standard_normal((T, E)) + 0.7 * rng.standard_normal(E)).astype(np.float32)
    return rng, x, np.argsort(-x, 1, kind="stable")[:, :k].astype(np.int32)


def check(got, want, E, T, factor=1.0):
    loss, counts, tokens, probs, d = got
    assert (counts.cpu().numpy() == want["counts"]).all()
    assert (tokens.cpu().numpy() == want["tokens"]).all()
    mean = 2.0 ** -19 + (T / 152.0 + 64) * 2.0 ** -24
    assert (np.abs(f64(probs) - want["probs"]) <= mean * want["probs"] + 1e-37).all()
    assert (np.abs(f64(loss) - want["loss"]) <= 2 * mean * np.abs(want["loss"]) + 1e-37).all()
    if d is not None:
        assert (np.abs(f64(d) - factor * want["d_logits"])
                <= 2.0 ** -18 * abs(factor) * want["size"] + 1e-37).all()


SHAPES = [(1, 2, 1), (5, 7, 3), (256, 8, 2), (1000, 16, 4), (257, 32, 8), (300, 60, 6), (2000, 64, 1),
          (777, 100, 2), (130, 160, 8), (500, 255, 5), (1111, 256, 16)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("sigmoid", [0, 1])
@pytest.mark.parametrize("B,masked", [(1, False), (4, True), (40, False)])
def test_loss_and_gradient(block, T, E, k, sigmoid, B, masked):
    rng, x, idx = case(T, E, k, B)
    cut = np.sort(rng.integers(0, T + 1, B + 1))
    if B == 1:
        cut = np.array([0, T])
    if B == 4:
        cut[2] = cut[1]                # an empty sequence
    mask = rng.random(T) > 0.3 if masked else None
    if masked:
        mask[cut[0]:cut[1]] = False    # and one without live tokens
    m = None if mask is None else torch.tensor(mask, device="cuda")
    want = R.seq_aux(x, idx, cut, mask, bool(sigmoid), 0.3, 0.05)
    lx, li, off = torch.tensor(x, device="cuda"), i32(idx), i32(cut)
    s = block.SeqAuxLoss(T + 3, E, k, B, sigmoid, 0.3, 0.05)
    s.workspace.fill_(0xFF)
    d = torch.full((T, E), 9.0, device="cuda")
    assert s.forward(lx, li, off, m, d_logits=d) is s.loss
    check((s.loss, s.counts, s.tokens, s.probs, d), want, E, T)
    # the gradient by itself is the same one
    d2 = torch.full_like(d, 9.0)
    s.backward(lx, off, d2, m, accumulate=False)
    assert torch.equal(d, d2)
    # scaled, and added: tokens that are not live keep theirs
    base = torch.randn(T, E, device="cuda")
    d3 = base.clone()
    s.backward(lx, off, d3, m, d_loss=-2.0)
    sum_ = f64(base) - 2.0 * want["d_logits"]
    assert (np.abs(f64(d3) - sum_) <= 2.0 ** -17 * want["size"] + 2.0 ** -23 * np.abs(sum_) + 1e-37).all()
    dead = np.ones(T, bool)
    dead[np.concatenate(R.live_tokens(T, cut, mask))] = False
    dead = torch.tensor(dead, device="cuda")
    assert torch.equal(d3[dead], base[dead]) and (d[dead] == 0).all()
    # the loss alone; the same numbers each time
    first = [t.clone() for t in (s.loss, s.counts, s.tokens, s.probs)]
    s.forward(lx, li, off, m)
    assert all(torch.equal(a, b) for a, b in zip(first, (s.loss, s.counts, s.tokens, s.probs)))
    d4 = base.clone()
    s.forward(lx, li, off, m, d_logits=d4, d_loss=-2.0, accumulate=True)
    assert torch.equal(d3, d4)


@pytest.mark.parametrize("sigmoid", [0, 1])
def test_one_sequence_is_moe_aux_loss(L, block, sigmoid):
    T, E, k = 500, 32, 4
    _, x, idx = case(T, E, k)
    lx, li = torch.tensor(x, device="cuda"), i32(idx)
    s = block.SeqAuxLoss(T, E, k, 1, sigmoid, 0.1)
    d, d_old = torch.empty_like(lx), torch.empty_like(lx)
    s.forward(lx, li, i32([0, T]), d_logits=d)
    counts, probs, loss = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(L.moe_aux_loss_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
    L.moe_aux_loss(lx, li, sigmoid, 0.1, counts, probs, loss, ws)
    L.moe_aux_loss_bwd(lx, counts, k, sigmoid, 0.1, d_old, accumulate=False)
    assert torch.equal(s.counts[0], counts) and s.loss[1] == 0
    torch.testing.assert_close(s.loss[:1], loss, rtol=1e-5, atol=0)
    torch.testing.assert_close(s.probs[0], probs, rtol=1e-5, atol=0)
    torch.testing.assert_close(d, d_old, rtol=1e-4, atol=float(d_old.abs().max()) * 1e-5)


@pytest.mark.parametrize("E,pad", [(8, 4), (60, 4), (64, 3), (33, 2), (256, 8)])
def test_strided_rows(block, E, pad):
    """Leading dimensions that keep rows on 16 bytes and that do not; spare columns stay."""
    T, k = 300, 2
    _, x, idx = case(T, E, k)
    want = R.seq_aux(x, idx, [10, 200, 290], None, False, 0.3, 0.05)
    whole = torch.full((T, E + pad), 1e30, device="cuda")
    whole[:, :E] = torch.tensor(x)
    dw = torch.full((T, E + pad), 9.0, device="cuda")
    s = block.SeqAuxLoss(T, E, k, 2, 0, 0.3, 0.05)
    s.forward(whole[:, :E], i32(idx), i32([10, 200, 290]), d_logits=dw[:, :E])
    check((s.loss, s.counts, s.tokens, s.probs, dw[:, :E]), want, E, T)
    assert (dw[:, E:] == 9.0).all()
    # a base address off 16 bytes
    flat = torch.empty(T * E + 1, device="cuda")
    odd = flat[1:].view(T, E)
    odd.copy_(torch.tensor(x))
    s.forward(odd, i32(idx), i32([10, 200, 290]), d_logits=dw[:, :E])
    check((s.loss, s.counts, s.tokens, s.probs, dw[:, :E]), want, E, T)


@pytest.mark.parametrize("sigmoid", [0, 1])
def test_odd_logits_and_choices(block, sigmoid):
    """-inf for closed experts, rows of -inf alone, NaN, huge logits; choices out of range."""
    T, E, k = 64, 12, 2
    _, x, idx = case(T, E, k)
    x[:, 5] = -np.inf
    x[3] = -np.inf
    x[4] = np.nan
    x[5, 2] = np.nan
    x[6] = np.where(np.arange(E) == 1, 1e4, -1e4)
    x[7] = np.finfo(np.float32).min
    idx[8, 0], idx[9, 1], idx[10, 0] = -1, E, 2 ** 31 - 1
    off = [0, 30, T]
    want = R.seq_aux(x, idx, off, None, bool(sigmoid), 0.3, 0.0)
    s = block.SeqAuxLoss(T, E, k, 2, sigmoid, 0.3)
    d = torch.empty(T, E, device="cuda")
    s.forward(torch.tensor(x, device="cuda"), i32(idx), i32(off), d_logits=d)
    check((s.loss, s.counts, s.tokens, s.probs, d), want, E, T)
    assert torch.isfinite(d).all()


def test_offsets_out_of_range_stay_in_bounds(block):
    """Offsets past T or below 0 are clamped."""
    T, E, k = 100, 8, 2
    _, x, idx = case(T, E, k)
    s = block.SeqAuxLoss(T, E, k, 3, 0, 0.3, 0.05)
    d = torch.empty(T, E, device="cuda")
    off = [-5, 20, 90, 5000]
    s.forward(torch.tensor(x, device="cuda"), i32(idx), i32(off), d_logits=d)
    check((s.loss, s.counts, s.tokens, s.probs, d), R.seq_aux(x, idx, off, None, False, 0.3, 0.05), E, T)


@pytest.mark.parametrize("T", [0, 40])
def test_nothing_live(block, T):
    E, k, B = 8, 2, 3
    s = block.SeqAuxLoss(T, E, k, B, 0, 0.3, 0.05)
    x = torch.randn(T, E, device="cuda")
    d = torch.full((T, E), 9.0, device="cuda")
    for mask, off in ((torch.zeros(T, dtype=torch.bool, device="cuda"), [0, 10, 20, T]), (None, [T] * 4)):
        s.loss.fill_(5.0), s.counts.fill_(5), s.tokens.fill_(5), s.probs.fill_(5.0)
        s.forward(x, torch.zeros(T, k, dtype=torch.int32, device="cuda"), i32(off), mask, d_logits=d)
        assert all((t == 0).all() for t in (s.loss, s.counts, s.tokens, s.probs, d))
        s.backward(x, i32(off), d, mask, accumulate=False)
        assert (d == 0).all()


@pytest.mark.parametrize("T,E,k,B", [(40000, 8, 2, 1), (9000, 256, 8, 1), (5000, 16, 2, 3000)])
def test_long_and_many_sequences(block, T, E, k, B):
    """One sequence over every block (its choices counted by a cluster), and more sequences than
    blocks, most of a token or none."""
    rng, x, idx = case(T, E, k)
    cut = np.array([0, T]) if B == 1 else np.sort(rng.integers(0, T + 1, B + 1))
    want = R.seq_aux(x, idx, cut, None, True, 0.3, 0.05)
    s = block.SeqAuxLoss(T, E, k, B, 1, 0.3, 0.05)
    d = torch.empty(T, E, device="cuda")
    s.forward(torch.tensor(x, device="cuda"), i32(idx), i32(cut), d_logits=d)
    check((s.loss, s.counts, s.tokens, s.probs, d), want, E, T)


def test_gradient_by_differences(block):
    T, E, k = 6, 5, 2
    rng, x, idx = case(T, E, k)
    s = block.SeqAuxLoss(T, E, k, 2, 0, 0.9, 0.4)
    d = torch.empty(T, E, device="cuda")
    s.forward(torch.tensor(x, device="cuda"), i32(idx), i32([0, 2, 6]), d_logits=d)
    f = lambda v: R.seq_aux(v, idx, [0, 2, 6], None, False, 0.9, 0.4)["loss"].sum()  # noqa: E731
    for i in np.ndindex(T, E):
        e = np.zeros((T, E))
        e[i] = 1e-5
        assert abs((f(x + e) - f(x - e)) / 2e-5 - f64(d)[i]) <= 1e-5


@pytest.mark.parametrize("E,sigmoid", [(64, 0), (256, 1), (30, 1), (8, 0)])
def test_odd_logits_among_others(block, E, sigmoid):
    """Steps that hold closed experts, far logits and rows without any, in ragged masked sequences;
    written and added to."""
    T, k = 3001, 2
    rng, x, idx = case(T, E, k, 5)
    x[rng.random(T) < 0.05] += 40.0
    x[rng.random(T) < 0.05] -= 300.0
    closed = rng.random((T, E)) < 0.3
    x = np.where((rng.random(T) < 0.1)[:, None] & closed, -np.inf, x).astype(np.float32)
    x[rng.integers(0, T, 5)] = -np.inf
    cut = np.sort(rng.integers(0, T + 1, 18))
    mask = rng.random(T) > 0.2
    want = R.seq_aux(x, idx, cut, mask, bool(sigmoid), 0.3, 0.0)
    lx, li, off, m = torch.tensor(x, device="cuda"), i32(idx), i32(cut), torch.tensor(mask, device="cuda")
    s = block.SeqAuxLoss(T, E, k, 17, sigmoid, 0.3)
    d = torch.full((T, E), 9.0, device="cuda")
    s.forward(lx, li, off, m, d_logits=d)
    check((s.loss, s.counts, s.tokens, s.probs, d), want, E, T)
    base = torch.randn(T, E, device="cuda") * 1e-3
    added = base.clone()
    s.backward(lx, off, added, m)
    sum_ = f64(base) + want["d_logits"]
    assert (np.abs(f64(added) - sum_) <= 2.0 ** -18 * want["size"] + 2.0 ** -23 * np.abs(sum_) + 1e-37).all()


@pytest.mark.parametrize("masked", [False, True])
def test_a_million_tokens(block, masked):
    """More tokens a block than it keeps the mask of."""
    T, E, k, B = 1_100_003, 2, 1, 3
    rng, x, idx = case(T, E, k)
    cut = np.array([7, 300_000, 300_000, T - 5])
    mask = rng.random(T) > 0.5 if masked else None
    want = R.seq_aux(x, idx, cut, mask, False, 0.3, 0.05)
    s = block.SeqAuxLoss(T, E, k, B, 0, 0.3, 0.05)
    d = torch.full((T, E), 9.0, device="cuda")
    s.forward(torch.tensor(x, device="cuda"), i32(idx), i32(cut),
              None if mask is None else torch.tensor(mask, device="cuda"), d_logits=d)
    # (two experts: lse may lie near 0, where it is off by half an ulp of the logits' size)
    want["size"] += 2.0 * 0.05 / want["tokens"].sum() * 2.0 ** -4
    check((s.loss, s.counts, s.tokens, s.probs, d), want, E, T)


def test_the_gradient_is_that_of_the_last_forward(block):
    s = block.SeqAuxLoss(10, 8, 2, 1, 0, 0.3)
    x, off = torch.randn(6, 8, device="cuda"), i32([0, 6])
    with pytest.raises(ValueError, match="last forward"):
        s.backward(x, off, torch.empty_like(x))
    s.forward(x, x.topk(2, 1).indices.to(torch.int32), off)
    s.backward(x, off, torch.empty_like(x))
    with pytest.raises(ValueError, match="last forward"):
        s.backward(x[:5], off, torch.empty(5, 8, device="cuda"))


@pytest.mark.parametrize("T,E,k,B", [(145, 16, 4, 273), (394, 32, 2, 180), (17, 128, 2, 166), (1, 8, 2, 40),
                                     (60, 256, 8, 60), (2000, 8, 2, 900), (300, 33, 3, 100), (100, 8, 2, 100)])
@pytest.mark.parametrize("masked", [False, True])
def test_sequences_of_few_tokens(block, T, E, k, B, masked):
    """Sequences shorter than a step, many of them empty, and tokens on both sides of all; one that
    holds nearly every token."""
    for long in (False, True):
        rng, x, idx = case(T, E, k, B + long)
        cut = np.sort(rng.integers(0, T + 1, B + 1))
        if long:
            cut = np.sort(np.where(rng.random(B + 1) < 0.5, cut.min(), T - T // 8))
        mask = rng.random(T) > 0.4 if masked else None
        want = R.seq_aux(x, idx, cut, mask, True, 0.3, 0.05)
        lx, off = torch.tensor(x, device="cuda"), i32(cut)
        m = None if mask is None else torch.tensor(mask, device="cuda")
        s = block.SeqAuxLoss(T, E, k, B, 1, 0.3, 0.05)
        s.workspace.fill_(0xFF)
        for t in (s.probs, s.loss):
            t.fill_(9.0)
        d = torch.full((T, E), 9.0, device="cuda")
        s.forward(lx, i32(idx), off, m, d_logits=d)
        check((s.loss, s.counts, s.tokens, s.probs, d), want, E, T)
        d2 = torch.full((T, E), 9.0, device="cuda")
        s.backward(lx, off, d2, m, accumulate=False)
        assert torch.equal(d, d2)
        base = torch.randn(T, E, device="cuda")
        added = base.clone()
        s.backward(lx, off, added, m, d_loss=2.0)
        sum_ = f64(base) + 2.0 * want["d_logits"]
        assert (np.abs(f64(added) - sum_) <= 2.0 ** -17 * want["size"] + 2.0 ** -23 * np.abs(sum_) + 1e-37).all()
        dead = (want["d_logits"] == 0).all(1)
        assert torch.equal(added[torch.tensor(dead, device="cuda")], base[torch.tensor(dead, device="cuda")])


def ragged(rng, T, kind):
    """Offsets of a batch with runs of sequences of no, one or a few tokens among long ones."""
    lens = {"few": lambda: int(rng.integers(0, 4)), "mixed": lambda: int(rng.choice([0, 0, 1, 1, 2, 5, 17, 300])),
            "ones": lambda: 1}[kind]
    cut = [int(rng.integers(0, 3))]
    if kind == "ones":
        cut += [cut[0] + T // 3]
    while cut[-1] < T - 2 and len(cut) < 3000:
        cut.append(min(T, cut[-1] + lens()))
    if kind == "ones" and T > 1000:  # and a long one behind them
        cut = [c for c in cut if c < T // 3 + 400] + [T]
    return np.array(cut)


@pytest.mark.parametrize("T,E,k", [(700, 8, 2), (3001, 16, 1), (2500, 30, 4), (1500, 64, 6), (900, 100, 2),
                                   (800, 160, 8), (1203, 256, 8), (40000, 8, 4)])
@pytest.mark.parametrize("kind", ["few", "mixed", "ones"])
@pytest.mark.parametrize("sigmoid,masked,odd", [(0, True, False), (1, False, True), (1, True, False)])
def test_short_sequences_among_long_ones(block, T, E, k, kind, sigmoid, masked, odd):
    rng, x, idx = case(T, E, k, len(kind))
    cut = ragged(rng, T, kind)
    B = len(cut) - 1
    mask = rng.random(T) > 0.4 if masked else None
    if odd:  # logits far from 0, which a step takes in another way
        x[::97] += 30.0
    m = None if mask is None else torch.tensor(mask, device="cuda")
    want = R.seq_aux(x, idx, cut, mask, bool(sigmoid), 0.3, 0.0 if odd else 0.05)
    lx, li, off = torch.tensor(x, device="cuda"), i32(idx), i32(cut)
    s = block.SeqAuxLoss(T, E, k, B, sigmoid, 0.3, 0.0 if odd else 0.05)
    s.workspace.fill_(0xFF)
    d = torch.full((T, E), 9.0, device="cuda")
    s.forward(lx, li, off, m, d_logits=d)
    check((s.loss, s.counts, s.tokens, s.probs, d), want, E, T)
    first = [t.clone() for t in (s.loss, s.counts, s.tokens, s.probs)]
    d2 = torch.full_like(d, 9.0)
    s.backward(lx, off, d2, m, accumulate=False)
    assert torch.equal(d, d2)
    base = torch.randn(T, E, device="cuda")
    d3 = base.clone()
    s.forward(lx, li, off, m, d_logits=d3, d_loss=-2.0, accumulate=True)
    assert all(torch.equal(a, b) for a, b in zip(first, (s.loss, s.counts, s.tokens, s.probs)))
    sum_ = f64(base) - 2.0 * want["d_logits"]
    assert (np.abs(f64(d3) - sum_) <= 2.0 ** -17 * want["size"] + 2.0 ** -23 * np.abs(sum_) + 1e-37).all()


@pytest.mark.parametrize("T,E,k,B", [(3000, 8, 2, 65536), (200, 64, 4, 1500), (64, 256, 2, 9000), (300, 16, 2, 700)])
@pytest.mark.parametrize("masked", [False, True])
def test_more_sequences_than_a_block_each_pays_for(block, T, E, k, B, masked):
    """Thousands of sequences of few tokens or none, the loss with its gradient and the gradient alone."""
    rng, x, idx = case(T, E, k, B)
    cut = np.sort(rng.integers(0, T + 1, B + 1))
    mask = rng.random(T) > 0.4 if masked else None
    want = R.seq_aux(x, idx, cut, mask, True, 0.3, 0.05)
    lx, off = torch.tensor(x, device="cuda"), i32(cut)
    m = None if mask is None else torch.tensor(mask, device="cuda")
    s = block.SeqAuxLoss(T, E, k, B, 1, 0.3, 0.05)
    s.workspace.fill_(0xFF)
    for t in (s.probs, s.loss):
        t.fill_(9.0)
    d, d2 = (torch.full((T, E), 9.0, device="cuda") for _ in range(2))
    s.forward(lx, i32(idx), off, m, d_logits=d)
    check((s.loss, s.counts, s.tokens, s.probs, d), want, E, T)
    s.backward(lx, off, d2, m, accumulate=False)
    assert torch.equal(d, d2)


def cut_of(kind, T, B, rng):
    """Offsets of B sequences: of equal lengths; one that holds all but a few tokens of the others; or
    runs of one token and of none among long ones, with tokens before the first and behind the last."""
    if kind == "even":
        return np.arange(B + 1) * T // B
    if kind == "one":
        lens = np.where(np.arange(B) < B // 2, 1, 0)
        lens[B // 3] = T - lens.sum()
        return np.concatenate(([0], np.cumsum(lens)))
    lens = rng.integers(0, 2, B)
    lens[:: max(1, B // 5)] = (T - 40 - B) // 6
    return 17 + np.concatenate(([0], np.cumsum(lens)))


@pytest.mark.parametrize("T,E,k,B", [(9000, 256, 8, 60), (9000, 256, 8, 200), (20000, 64, 8, 300), (70000, 8, 1, 900),
                                     (40000, 33, 1, 100), (16384, 64, 4, 500), (2048, 128, 16, 64), (8000, 16, 4, 250)])
@pytest.mark.parametrize("kind", ["even", "one", "runs"])
@pytest.mark.parametrize("masked", [False, True])
def test_counts_by_lengths(block, T, E, k, B, kind, masked):
    """Around 2^15 and 2^17 choices: sequences counted by a block each, by several blocks, and several
    in a block, with and without a cell of its shared memory for each sequence and expert."""
    rng, x, idx = case(T, E, k, B)
    cut = cut_of(kind, T, B, rng)
    assert cut[0] >= 0 and cut[-1] <= T and (np.diff(cut) >= 0).all()
    idx[rng.integers(0, T, 20), 0] = -1
    mask = rng.random(T) > 0.3 if masked else None
    want = R.seq_aux(x, idx, cut, mask, False, 0.3, 0.05)
    s = block.SeqAuxLoss(T, E, k, B, 0, 0.3, 0.05)
    for t in (s.counts, s.tokens):
        t.fill_(77)
    s.workspace.fill_(0xFF)
    d = torch.full((T, E), 9.0, device="cuda")
    args = (torch.tensor(x, device="cuda"), i32(idx), i32(cut), None if mask is None else torch.tensor(mask, device="cuda"))
    s.forward(*args, d_logits=d)
    check((s.loss, s.counts, s.tokens, s.probs, d), want, E, T)
    first = [t.clone() for t in (s.loss, s.counts, s.tokens, s.probs, d)]
    s.forward(*args, d_logits=d)
    assert all(torch.equal(a, b) for a, b in zip(first, (s.loss, s.counts, s.tokens, s.probs, d)))
