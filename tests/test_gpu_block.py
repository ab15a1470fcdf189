"""The operators around the expert layer as a step uses them: a pre-norm block forward and backward
against the fp64 oracle, captured into CUDA graphs, on other streams, between other kernels."""
import numpy as np
import pytest
import torch

from gpu_helpers import assert_close, host_f64
from oracle import block_ref as R
from oracle import moe_ref

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def mods():
    from mixture_experts_grouped_router_gb300 import _lib, block, layer
    return _lib, block, layer


class Step:
    """One block: h = x + r, y = norm(h), logits = y Wr, out = experts(y); the gradient of
    <out, g_out> + <h, g_h> + balance and z losses, clipped."""

    def __init__(self, mods, stream, T=200, d=128, f=192, E=8, k=2, B=3, score_fn=1):
        L, block, layer = mods
        self.block, self.layer = block, layer
        g = torch.Generator(device="cuda").manual_seed(17)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.k, self.score_fn = k, score_fn
        self.x, self.r = rnd(T, d).bfloat16(), rnd(T, d).to(stream)
        self.w = 1.0 + 0.1 * rnd(d)
        self.wr = 0.3 * rnd(d, E)
        self.wi, self.wo = (rnd(E, d, 2 * f) * d ** -0.5).bfloat16(), (rnd(E, f, d) * f ** -0.5).bfloat16()
        self.g_out, self.g_h = rnd(T, d).bfloat16(), rnd(T, d).to(stream)
        self.off = torch.tensor([0, 70, 150, T], dtype=torch.int32, device="cuda")
        self.mask = torch.rand(T, generator=g, device="cuda") > 0.2
        self.h, self.y = torch.empty_like(self.r), torch.empty_like(self.x)
        self.dh, self.dw = torch.empty_like(self.r), torch.empty(d, device="cuda")
        self.dx, self.dwr = torch.empty_like(self.x), torch.empty_like(self.wr)
        self.ws = block.rms_norm_bwd_workspace(T, d)
        self.b = layer.MoEBuffers(layer.LayerShape(T, d, f, E, k, score_fn=score_fn))
        self.aux = block.SeqAuxLoss(T, E, k, B, score_fn, coeff=0.5, z_coeff=0.1)
        self.clip = block.GradClip.of(self.b, self.dwr, self.dw)
        self.logits = torch.empty(T, E, device="cuda")
        self.max_norm = 3.0

    def run(self):
        blk, b = self.block, self.b
        blk.rms_norm(self.x, self.w, EPS, self.y, residual=self.r, h=self.h)
        torch.mm(self.y.float(), self.wr, out=self.logits)
        self.layer.forward(b, self.y, self.logits, self.wi, self.wo)
        self.layer.backward(b, self.g_out, self.wi, self.wo)
        self.aux.forward(self.logits, b.topk_idx, self.off, self.mask, d_logits=b.d_logits, accumulate=True)
        torch.mm(self.y.float().t(), b.d_logits, out=self.dwr)
        dy = (b.dx.float() + b.d_logits @ self.wr.t()).bfloat16()
        blk.rms_norm_bwd(dy, self.h, self.w, EPS, self.dh, self.dw, self.ws, d_residual=self.g_h, dx=self.dx)
        self.norm = self.clip.clip(self.max_norm)
        return self.results()

    def results(self):
        return [self.h, self.y, self.b.out, self.aux.loss, self.b.d_logits, self.dh, self.dx, self.norm,
                self.b.dwi, self.b.dwo, self.dwr, self.dw]


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score_fn", [0, 1])
def test_step(mods, stream, score_fn):
    s = Step(mods, stream, score_fn=score_fn)
    # the layer's own tolerance (1e-2 of the 2-norm) for what passes through its bf16 products
    got = [t.clone() for t in s.run()]
    h, y, out, loss, d_logits, dh, dx, norm, dwi, dwo, dwr, dw = got
    x, r, w, wr = (host_f64(t) for t in (s.x, s.r, s.w, s.wr))
    wi, wo, g_out, g_h = (host_f64(t) for t in (s.wi, s.wo, s.g_out, s.g_h))
    assert_close("h", h, x + r)
    hv = host_f64(h)
    assert_close("y", y, R.rms_norm(hv, w, EPS)[0])
    yv = host_f64(y)
    logits = s.logits.cpu().numpy()
    assert_close("logits", s.logits, yv @ wr, 1e-4, 1e-3)
    fw = moe_ref.forward(yv, logits, wi, wo, s.k, s.score_fn, 1)
    assert_close("out", out, fw["out"])
    bw = moe_ref.backward(fw, g_out, wi, wo, s.k)
    off, mask = s.off.cpu().numpy(), s.mask.cpu().numpy()
    aux = R.seq_aux(logits, fw["topk_idx"], off, mask, bool(s.score_fn), 0.5, 0.1)
    assert_close("loss", loss, aux["loss"], 1e-5, 1e-5)
    assert (s.aux.counts.cpu().numpy() == aux["counts"]).all()
    dl = moe_ref.route_topk_bwd(logits, fw["topk_idx"], bw["d_topk_w"], s.score_fn, 1) + aux["d_logits"]
    assert_close("d_logits", d_logits, dl)
    dy = bw["dx"] + dl @ wr.T
    want_dh, want_dw = R.rms_norm_bwd(dy, hv, w, EPS, g_h)
    assert_close("dh", dh, want_dh)
    assert_close("dx", dx, want_dh)
    grads = [bw["d_wi"], bw["d_wo"], yv.T @ dl, want_dw]
    n, factor = R.clip(grads, s.max_norm, 1.0)
    assert n > s.max_norm  # something to clip
    assert abs(float(norm) - n) <= 1e-2 * n
    for name, t, g in zip(("dwi", "dwo", "dwr", "dw"), (dwi, dwo, dwr, dw), grads):
        assert_close(name, t, factor * g)


def test_step_in_a_graph(mods):
    s = Step(mods, torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (s.x, s.r, s.g_out):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        s.mask.copy_(torch.rand(s.mask.shape, generator=g, device="cuda") > 0.5)
        s.off.copy_(torch.tensor([5, 5 + seed, 100, 190], dtype=torch.int32))
        want = [t.clone() for t in s.run()]
        for t in s.results():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, s.results()):
            assert torch.equal(a, b)


def test_two_graphs_share_what_a_program_keeps(mods):
    """Replayed in turn on one stream, two graphs may use the same workspaces."""
    s = Step(mods, torch.bfloat16)
    s.run()
    other = [torch.randn_like(t.float()).to(t.dtype) for t in (s.x, s.r)]
    graphs, wants, ins = [], [], [(s.x, s.r), tuple(other)]
    for x, r in ins:
        s.x, s.r = x, r
        wants.append([t.clone() for t in s.run()])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
        assert all(torch.equal(a, b) for a, b in zip(wants[i], s.results()))


def test_given_streams(mods):
    """Work on a stream that is given, with the current one and the given one busy."""
    L, block, _ = mods
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(300, 1024, generator=g, device="cuda").bfloat16()
    w = torch.randn(1024, generator=g, device="cuda")
    lg = torch.randn(300, 16, generator=g, device="cuda")
    idx = lg.topk(2, 1).indices.to(torch.int32)
    off = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    h, y, dh, dw = x.clone(), x.clone(), x.clone(), w.clone()
    c = block.Codes8(300, 1024, "mx")
    back = torch.empty_like(x)
    ws = block.rms_norm_bwd_workspace(300, 1024)
    aux = block.SeqAuxLoss(300, 16, 2, 2, 1, 0.1, 0.1)
    d, grad, out = lg.clone(), lg.clone(), lg.clone()
    clip = block.GradClip([grad], [out])

    def run(st):
        block.rms_norm(x, w, EPS, y, residual=x, h=h, codes=c, stream=st)
        c.dequantize(back, stream=st)
        block.rms_norm_bwd(y, h, w, EPS, dh, dw, ws, d_residual=x, stream=st)
        aux.forward(lg, idx, off, d_logits=d, stream=st)
        aux.backward(lg, off, d, stream=st)
        clip.norm(stream=st)
        clip.clip(1.0, stream=st)
        return [t.clone() if st is None else t for t in (h, y, back, dh, dw, d, aux.loss, out, clip.total)]
    want = run(None)
    st = torch.cuda.Stream()
    for t in (h, y, back, dh, dw, d, aux.loss, out):
        t.zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    with torch.cuda.stream(st):
        torch.cuda._sleep(5_000_000)
    got = run(st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_two_streams_at_once(mods):
    """Two programs with what is theirs, on two streams at the same time."""
    a, b = Step(mods, torch.bfloat16), Step(mods, torch.float32, T=150, d=256, score_fn=0)
    b.off.copy_(torch.tensor([0, 10, 90, 150], dtype=torch.int32))
    want = [[t.clone() for t in s.run()] for s in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    for s, w in zip((a, b), want):
        assert all(torch.equal(p, q) for p, q in zip(w, s.results()))


def test_between_other_kernels(mods):
    """Inputs written by the kernel before and read by the kernel after, call on call: nothing is
    read early or late."""
    L, block, _ = mods
    T, E, k, B, d = 6000, 32, 4, 5, 512
    gen = torch.Generator(device="cuda").manual_seed(6)
    base = torch.randn(T, E, generator=gen, device="cuda")
    bx = torch.randn(T, d, generator=gen, device="cuda")
    lg, idx = torch.empty_like(base), torch.empty(T, k, dtype=torch.int32, device="cuda")
    off = torch.empty(B + 1, dtype=torch.int32, device="cuda")
    mask = torch.empty(T, dtype=torch.bool, device="cuda")
    x, w = torch.empty(T, d, dtype=torch.bfloat16, device="cuda"), torch.empty(d, device="cuda")
    h, y, dh, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    ws, aux = block.rms_norm_bwd_workspace(T, d), block.SeqAuxLoss(T, E, k, B, 1, 0.1, 0.1)
    g = torch.empty(T, E, device="cuda")
    clip = block.GradClip([g, dw])
    cuts = torch.arange(B + 1, device="cuda") * (T // B)

    def turn(i, wait):
        sync = torch.cuda.synchronize if wait else (lambda: None)
        lg.copy_(base * (1.0 + 0.1 * i))
        idx.copy_((torch.arange(T * k, device="cuda").view(T, k) * (i + 1)) % E)
        off.copy_(cuts - i)
        mask.copy_(base[:, 0] > -0.1 * i)
        sync()
        aux.forward(lg, idx, off, mask, d_logits=g)
        sync()
        g.mul_(3.0)
        x.copy_(bx + i)
        w.fill_(1.0 + i)
        sync()
        block.rms_norm(x, w, EPS, y, residual=x, h=h)
        sync()
        block.rms_norm_bwd(y, h, w, EPS, dh, dw, ws)
        sync()
        n = clip.clip(0.5)
        sync()
        return [t.clone() for t in (aux.loss, aux.probs, aux.counts, y, dh, dw, g, n)]
    want = [turn(i, True) for i in range(6)]
    for _ in range(5):
        got = [turn(i, False) for i in range(6)]
        assert all(torch.equal(p, q) for a, b in zip(want, got) for p, q in zip(a, b))


def test_fewer_tokens_than_the_instance_is_for(mods):
    _, block, _ = mods
    s = block.SeqAuxLoss(1000, 8, 2, 2, 0, 0.1, 0.1)
    rng = np.random.default_rng(3)
    for T in (1000, 300, 1, 7):
        x = rng.standard_normal((T, 8)).astype(np.float32)
        idx = np.argsort(-x, 1)[:, :2].astype(np.int32)
        want = R.seq_aux(x, idx, [0, T // 2, T], None, False, 0.1, 0.1)
        s.forward(torch.tensor(x, device="cuda"), torch.tensor(idx, device="cuda"),
                  torch.tensor([0, T // 2, T], dtype=torch.int32, device="cuda"))
        assert (s.counts.cpu().numpy() == want["counts"]).all()
        assert_close("loss", s.loss, want["loss"], 1e-5, 1e-5)
