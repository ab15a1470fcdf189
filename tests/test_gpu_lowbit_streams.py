"""The weights' layout on a stream that is given, with work queued on both streams: every step
runs there, in order, and in memory that the current stream is done with."""
import pytest
import torch

pytestmark = pytest.mark.gpu

LONG = 50_000_000  # clock cycles, some 25 ms: far longer than the host takes to queue a call


@pytest.fixture(scope="module")
def lowbit():
    from mixture_experts_grouped_router_gb300 import lowbit
    return lowbit


def parts(w):
    return [t for t in (w.wi_q, w.wi_sf, w.wi_scale, w.wo_q, w.wo_sf, w.wo_scale) if t is not None]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(parts(a), parts(b)))


E_, D, F = 6, 128, 128  # whole atoms: every byte of them is written


def weights():
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    size = torch.arange(1, E_ + 1, device="cuda").view(-1, 1, 1)
    return (rnd(E_, D, 2 * F) * size).bfloat16(), (rnd(E_, F, D) / size).bfloat16()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("busy", ["given", "current", "both"])
def test_from_weights(lowbit, fmt, busy):
    wi, wo = weights()
    want = lowbit.Fp4Experts.from_weights(fmt, wi, wo)
    s = torch.cuda.Stream()
    # small blocks that the allocator hands out again, with a wrong maximum in them
    stale = [torch.full((E_,), 1e4, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del stale
    if busy in ("given", "both"):
        with torch.cuda.stream(s):
            torch.cuda._sleep(LONG)
    if busy in ("current", "both"):
        torch.cuda._sleep(2 * LONG)
    got = lowbit.Fp4Experts.from_weights(fmt, wi, wo, stream=s)
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_from_codes(lowbit, fmt):
    """The atoms come from memory that the current stream is still to write: a block freed
    there may be given to the current stream's next tensor, not to another stream's."""
    blk = 16 if fmt == "nv" else 32
    g = torch.Generator(device="cuda").manual_seed(4)
    byte = lambda hi, *s: torch.randint(0, hi, s, device="cuda", generator=g).to(torch.uint8)  # noqa: E731
    wi, wo = byte(256, E_, 2 * F, D // 2), byte(256, E_, D, F // 2)
    si, so = byte(127, E_, 2 * F, D // blk), byte(127, E_, D, F // blk)
    scale = torch.ones(E_, device="cuda") if fmt == "nv" else None
    make = lambda st: lowbit.Fp4Experts.from_codes(fmt, wi, si, scale, wo, so, scale, stream=st)  # noqa: E731
    want = make(None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = [want.wi_sf.numel(), want.wo_sf.numel()]
    torch.cuda._sleep(LONG)
    late = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    for t in late:
        t.fill_(0xEE)
    del late, t
    got = make(s)
    torch.cuda.synchronize()
    assert same(got, want)
