"""Refusals of the operators around the expert layer (host checks, nothing is launched): the C
ABI's, and what the Python calls check of their tensors.  No GPU."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__._build_module().build()
    from mixture_experts_grouped_router_gb300 import _lib
    return _lib


@pytest.fixture(scope="module")
def block(L):
    from mixture_experts_grouped_router_gb300 import block
    return block


def P(v=4096):
    return ctypes.c_void_p(v)


BIG = 1 << 40


def norm(L, x=P(), ldx=128, res=P(), ldr=128, st=0, rows=10, cols=128, w=P(), wt=1, eps=1e-5, h=P(),
         ldh=128, y=P(), ldy=128, codes=0, q=P(), ldq=128, s=P(), lds=4, nb=BIG):
    return L.LIB.moe_rms_norm(x, ldx, res, ldr, st, rows, cols, w, wt, eps, h, ldh, y, ldy, codes, q,
                              ldq, s, lds, nb, None)


def test_rms_norm(L):
    bad, uns = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED
    assert norm(L, rows=-1) == bad and norm(L, cols=0) == bad
    assert norm(L, cols=100, ldx=104) == uns and "multiple of 8" in L.last_error()
    assert norm(L, cols=16392) == uns and norm(L, rows=1 << 31) == uns
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert norm(L, eps=eps) == bad and "eps" in L.last_error()
    assert norm(L, st=2) == bad and norm(L, wt=7) == bad and norm(L, codes=3) == bad
    assert norm(L, w=None) == bad and norm(L, w=P(4100)) == uns
    assert norm(L, x=None, res=None) == bad and "neither x nor residual" in L.last_error()
    assert norm(L, y=None) == bad and "neither y nor codes" in L.last_error()
    for ld in ("ldx", "ldr", "ldh", "ldy"):
        assert norm(L, **{ld: 120}) == bad and norm(L, **{ld: 132}) == uns
    assert norm(L, st=1, ldr=130) == uns and norm(L, st=1, ldr=132, ldh=130) == uns
    for p in ("x", "res", "h", "y"):
        assert norm(L, **{p: P(4104)}) == uns and "16 bytes" in L.last_error()
    assert norm(L, codes=1, cols=120) == uns and "128" in L.last_error()
    assert norm(L, codes=1, ldq=136) == uns and norm(L, codes=2, ldq=132) == uns
    for c in (1, 2):
        assert norm(L, codes=c, q=None) == bad and norm(L, codes=c, s=None) == bad
        assert norm(L, codes=c, ldq=120) == bad
    assert norm(L, codes=1, nb=511) == bad and "511" in L.last_error()
    assert norm(L, codes=2, lds=3) == bad and norm(L, codes=2, nb=(9 * 4 + 4) * 2 - 1) == bad
    assert norm(L, codes=2, s=P(4097)) == uns and norm(L, codes=1, s=P(4104)) == uns
    assert norm(L, rows=0, x=None, res=None, y=None, h=None) == L.MOE_OK


def norm_bwd(L, dy=P(), ldy=128, h=P(), ldh=128, st=0, rows=10, cols=128, w=P(), wt=1, eps=1e-5,
             res=P(), ldr=128, dh=P(), lddh=128, dx=P(), lddx=128, dw=P(), ws=P(), nb=BIG):
    return L.LIB.moe_rms_norm_bwd(dy, ldy, h, ldh, st, rows, cols, w, wt, eps, res, ldr, dh, lddh, dx,
                                  lddx, dw, 0, ws, nb, None)


def test_rms_norm_bwd(L):
    bad, uns = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED
    for p in ("dy", "h", "dh", "w"):
        assert norm_bwd(L, **{p: None}) == bad
    for p in ("dy", "h", "res", "dh", "dx", "w"):
        assert norm_bwd(L, **{p: P(4104)}) == uns
    for ld in ("ldy", "ldh", "ldr", "lddh", "lddx"):
        assert norm_bwd(L, **{ld: 120}) == bad and norm_bwd(L, **{ld: 132}) == uns
    assert norm_bwd(L, cols=12) == uns and norm_bwd(L, eps=0.0) == bad and norm_bwd(L, st=5) == bad
    need = L.moe_rms_norm_bwd_workspace_bytes(10, 128)
    assert need > 0
    assert norm_bwd(L, nb=need - 1) == bad and "workspace" in L.last_error()
    assert norm_bwd(L, ws=None) == bad and norm_bwd(L, ws=P(4104)) == uns and norm_bwd(L, dw=P(4098)) == uns
    assert norm_bwd(L, rows=0, dw=None, ws=None, dy=None, h=None, dh=None) == L.MOE_OK
    f = L.moe_rms_norm_bwd_workspace_bytes
    assert f(-1, 128) == 0 and f(4, 0) == 0 and f(4, 16392) == 0 and f(0, 128) > 0
    assert f(1 << 30, 4096) < 1 << 24


def test_mx_dequantize(L):
    bad, uns = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED

    def d(q=P(), ldq=128, sf=P(), nb=BIG, rows=10, cols=128, fmt=0, x=P(), ldx=128):
        return L.LIB.moe_mx_dequantize(q, ldq, sf, nb, rows, cols, fmt, x, ldx, None)
    assert d(cols=64) == uns and d(fmt=2) == bad and d(rows=-1) == bad and d(nb=511) == bad
    assert d(ldq=120) == bad and d(ldq=132) == uns and d(ldx=120) == bad and d(ldx=132) == uns
    assert d(q=None) == bad and d(sf=None) == bad and d(x=None) == bad and d(x=P(4104)) == uns
    assert d(q=P(4100)) == uns and d(rows=0, q=None) == L.MOE_OK


def seq(L, lg=P(1 << 16), ld=8, T=10, E=8, k=2, fn=0, idx=P(), off=P(), B=3, c=0.1, z=0.1, cnt=P(), tok=P(),
        pr=P(), loss=P(), d=P(), ldd=8, ws=P(), nb=BIG):
    return L.LIB.moe_seq_aux_loss(lg, ld, T, E, k, fn, idx, off, B, None, c, z, cnt, tok, pr, loss, 1.0,
                                  d, ldd, 0, ws, nb, None)


def test_seq_aux_loss(L):
    bad, uns = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED
    assert seq(L, T=-1) == bad and seq(L, k=9) == bad and seq(L, k=0) == bad and seq(L, B=0) == bad
    assert seq(L, E=257, ld=257, ldd=257) == uns and seq(L, E=20, ld=20, ldd=20, k=17) == uns
    assert seq(L, T=(1 << 30) + 1) == uns and seq(L, B=65537) == uns
    assert seq(L, fn=2) == bad and seq(L, ld=7) == bad and seq(L, ldd=7) == bad
    assert seq(L, d=P(1 << 16)) == bad and "d_logits are logits" in L.last_error()
    for p in ("lg", "idx", "off", "cnt", "tok", "pr", "loss", "ws"):
        assert seq(L, **{p: None}) == bad
    for v in (float("nan"), float("inf")):
        assert seq(L, c=v) == bad and seq(L, z=v) == bad and "finite" in L.last_error()
    need = L.moe_seq_aux_loss_workspace_bytes(10, 8, 3)
    assert need > 0 and seq(L, nb=need - 1) == bad and seq(L, ws=P(4098)) == uns
    f = L.moe_seq_aux_loss_workspace_bytes
    assert f(-1, 8, 1) == 0 and f(8, 0, 1) == 0 and f(8, 257, 1) == 0 and f(8, 8, 0) == 0

    def bwd(lg=P(1 << 16), ld=8, T=10, E=8, k=2, fn=0, off=P(), B=3, cnt=P(), tok=P(), d=P(), ldd=8):
        return L.LIB.moe_seq_aux_loss_bwd(lg, ld, T, E, k, fn, off, B, None, 0.1, 0.1, cnt, tok, 1.0, d,
                                          ldd, 0, None)
    for p in ("lg", "off", "cnt", "tok", "d"):
        assert bwd(**{p: None}) == bad
    assert bwd(d=P(1 << 16)) == bad and bwd(ldd=7) == bad and bwd(E=300, ld=300, ldd=300) == uns and bwd(fn=-1) == bad
    assert bwd(T=0, lg=None, d=None) == L.MOE_OK


def test_clip(L):
    bad, uns = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED
    nb = L.moe_clip_workspace_bytes()

    def c(plan=P(), n=1, most=1.0, scale=1.0, norm=P(), ws=P(), nb=nb):
        return L.LIB.moe_clip_grads(plan, n, most, scale, norm, ws, nb, None)
    assert c(plan=None) == bad and c(n=-1) == bad and c(norm=None) == bad and c(ws=None) == bad
    for v in (0.0, -1.0, float("nan"), float("inf")):
        assert c(scale=v) == bad
    assert c(most=-1.0) == bad and c(most=float("nan")) == bad and c(nb=nb - 1) == bad
    assert c(plan=P(4104)) == uns and c(ws=P(4100)) == uns and c(norm=P(4098)) == uns

    G = L.GradArg

    def chunks(*g):
        return L.LIB.moe_clip_plan_chunks((G * len(g))(*g), len(g))
    assert chunks(G(4096, 4096, 10, 0, 0)) == 1 and chunks(G(4096, 4096, 1025, 0, 0)) == 2
    assert chunks(G(4098, 4098, 1025, 0, 0)) == 2  # 7 elements up to the next 16 bytes, 1018
    assert chunks(G(None, None, 0, 0, 1)) == 0
    assert chunks(G(4096, 4096, -1, 0, 0)) == -1 and chunks(G(None, 4096, 1, 0, 0)) == -1
    assert chunks(G(4096, 4096, 1, 2, 0)) == -1 and chunks(G(4096, 4096, 1, 0, 1)) == -1
    assert chunks(G(4097, 4096, 1, 0, 0)) == -1 and chunks(G(4096, 8194, 1, 0, 1)) == -1
    out = (ctypes.c_uint8 * 64)()
    g = (G * 1)(G(4096, 4096, 1025, 0, 0))
    assert L.LIB.moe_clip_plan(g, 1, out, 63) == bad and L.LIB.moe_clip_plan(g, 1, out, 64) == L.MOE_OK


def test_a_plan_covers_every_element_once(L):
    """Chunks of tensors of any size, type and alignment: in order, whole, accesses of 8 elements
    only where both sides of a chunk start on the size of 8 (16 or 32 bytes)."""
    import struct
    for g_at, o_at, gt, ot, n in [(4096, 8192, 0, 0, 5000), (4098, 8194, 0, 0, 5000), (4098, 8192, 0, 1, 3000),
                                  (4100, 8200, 1, 1, 4097), (4104, 8208, 0, 1, 9000), (4110, 8196, 0, 1, 7),
                                  (4096, 8192, 0, 1, (1 << 24) + 5), (4096, 4096, 1, 1, 1)]:
        g = (L.GradArg * 1)(L.GradArg(g_at, o_at, n, gt, ot))
        k = L.LIB.moe_clip_plan_chunks(g, 1)
        out = (ctypes.c_uint8 * (32 * k))()
        assert L.LIB.moe_clip_plan(g, 1, out, 32 * k) == L.MOE_OK
        at = 0
        gs, os = (4 if gt else 2), (4 if ot else 2)
        for p, o, m, kind in struct.iter_unpack("<QQii8x", bytes(out)):
            assert p == g_at + at * gs and o == o_at + at * os and m > 0
            assert (kind & 1) == gt and (kind >> 1 & 1) == ot
            if not kind & 4:
                assert p % (8 * gs) == 0 and o % (8 * os) == 0
            at += m
        assert at == n


class NoStream:  # the null stream of GPU 0, without asking CUDA for the current one
    cuda_stream = 0
    device_index = 0


def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def f32(*s):
    return torch.zeros(*s)


S = NoStream()


def test_tensors_of_the_norm(block):
    w = f32(128)
    ok = dict(residual=bf(4, 128), h=bf(4, 128), stream=S)
    with pytest.raises(ValueError, match="x is not on a GPU"):
        block.rms_norm(bf(4, 128), w, 1e-5, bf(4, 128), **ok)
    with pytest.raises(ValueError, match="residual"):
        block.rms_norm(bf(4, 128), w, 1e-5, bf(4, 128), residual=bf(5, 128), stream=S)
    with pytest.raises(ValueError, match="h is"):
        block.rms_norm(bf(4, 128), w, 1e-5, bf(4, 128), residual=bf(4, 128), h=f32(4, 128), stream=S)
    with pytest.raises(ValueError, match="residual is torch.float16"):
        block.rms_norm(bf(4, 128), w, 1e-5, bf(4, 128), residual=f32(4, 128).half(), stream=S)
    with pytest.raises(ValueError, match="x is torch.float32"):
        block.rms_norm(f32(4, 128), w, 1e-5, bf(4, 128), stream=S)
    with pytest.raises(ValueError, match="y is"):
        block.rms_norm(bf(4, 128), w, 1e-5, bf(4, 120), stream=S)
    with pytest.raises(ValueError, match="w has 64"):
        block.rms_norm(bf(4, 128), f32(64), 1e-5, bf(4, 128), stream=S)
    with pytest.raises(ValueError, match="w is torch.int32"):
        block.rms_norm(bf(4, 128), w.int(), 1e-5, bf(4, 128), stream=S)
    with pytest.raises(ValueError, match="neither"):
        block.rms_norm(None, w, 1e-5, bf(4, 128), stream=S)
    with pytest.raises(AssertionError, match="row-major"):
        block.rms_norm(bf(128, 4).t(), w, 1e-5, bf(4, 128), stream=S)
    with pytest.raises(ValueError, match="matrices"):
        block.rms_norm(bf(2, 4, 128), w, 1e-5, bf(4, 128), stream=S)
    with pytest.raises(ValueError, match="fmt"):
        block.Codes8(4, 128, "fp8", device="cpu")
    with pytest.raises(ValueError, match="128"):
        block.Codes8(4, 64, "mx", device="cpu")
    c = block.Codes8(3, 128, "mx", device="cpu")
    with pytest.raises(ValueError, match="q is"):
        block.rms_norm(bf(4, 128), w, 1e-5, codes=c, stream=S)
    with pytest.raises(ValueError, match="out is"):
        c.dequantize(bf(4, 128), stream=S)
    for fmt in ("mx", "act8"):
        with pytest.raises(ValueError, match="GPU"):
            block.Codes8(3, 128, fmt, device="cpu").dequantize(bf(3, 128), stream=S)


def test_tensors_of_the_norms_backward(block):
    w = f32(128)
    a = lambda **k: block.rms_norm_bwd(*[{**dict(dy=bf(4, 128), h=bf(4, 128)), **k}.pop(n) for n in ("dy", "h")],  # noqa: E731
                                       w, 1e-5, k.get("dh", bf(4, 128)), k.get("dw"), k.get("ws"),
                                       d_residual=k.get("res"), dx=k.get("dx"), stream=S)
    with pytest.raises(ValueError, match="dy is not on a GPU"):
        a()
    with pytest.raises(ValueError, match="h is"):
        a(h=bf(3, 128))
    with pytest.raises(ValueError, match="dh is torch.float32"):
        a(dh=f32(4, 128))
    with pytest.raises(ValueError, match="d_residual"):
        a(res=f32(4, 128))
    with pytest.raises(ValueError, match="dx is"):
        a(dx=f32(4, 128))
    with pytest.raises(ValueError, match="dw has"):
        a(dw=f32(120))
    with pytest.raises(ValueError, match="dw is torch.bfloat16"):
        a(dw=bf(128))
    with pytest.raises(ValueError, match="needed"):
        block.rms_norm_bwd(bf(4, 128), bf(4, 128), w, 1e-5, None, stream=S)


def test_tensors_of_the_loss(block):
    with pytest.raises(ValueError):
        block.SeqAuxLoss(4, 8, 9, 1, device="cpu")
    with pytest.raises(ValueError):
        block.SeqAuxLoss(4, 257, 2, 1, device="cpu")
    s = block.SeqAuxLoss(16, 8, 2, 3, device="cpu")
    i32 = dict(dtype=torch.int32)
    off, idx = torch.zeros(4, **i32), torch.zeros(16, 2, **i32)
    with pytest.raises(ValueError, match="GPU"):
        s.forward(f32(16, 8), idx, off, stream=S)
    with pytest.raises(ValueError, match="at most 16 tokens"):
        s.forward(f32(17, 8), idx, off, stream=S)
    with pytest.raises(ValueError, match="8 experts"):
        s.forward(f32(16, 7), idx, off, stream=S)
    with pytest.raises(ValueError, match="offsets"):
        s.forward(f32(16, 8), idx, torch.zeros(3, **i32), stream=S)
    with pytest.raises(ValueError, match="choices"):
        s.forward(f32(16, 8), torch.zeros(16, 3, **i32), off, stream=S)
    with pytest.raises(ValueError, match="topk_idx of 15"):
        s.forward(f32(16, 8), idx[:15], off, stream=S)
    with pytest.raises(ValueError, match="topk_idx is torch.int64"):
        s.forward(f32(16, 8), idx.long(), off, stream=S)
    with pytest.raises(ValueError, match="logits is torch.bfloat16"):
        s.forward(bf(16, 8), idx, off, stream=S)
    with pytest.raises(ValueError, match="token_mask"):
        s.forward(f32(16, 8), idx, off, torch.ones(15, dtype=torch.bool), stream=S)
    with pytest.raises(ValueError, match="token_mask is torch.float32"):
        s.forward(f32(16, 8), idx, off, torch.ones(16), stream=S)
    with pytest.raises(ValueError, match="d_logits"):
        s.forward(f32(16, 8), idx, off, d_logits=f32(15, 8), stream=S)
    with pytest.raises(ValueError, match="last forward was of None"):
        s.backward(f32(16, 8), off, f32(16, 8), stream=S)
    s.seen = 16  # as after a forward
    with pytest.raises(ValueError, match="of 15 tokens, the last forward was of 16"):
        s.backward(f32(15, 8), off, f32(15, 8), stream=S)
    with pytest.raises(ValueError, match="d_logits"):
        s.backward(f32(16, 8), off, f32(16, 9), stream=S)
    with pytest.raises(ValueError, match="GPU"):
        s.backward(f32(16, 8), off, f32(16, 8), stream=S)


def test_tensors_of_the_clipping(block):
    with pytest.raises(ValueError, match="0 gradients"):
        block.GradClip([])
    with pytest.raises(ValueError, match="1 gradients, 2 outputs"):
        block.GradClip([f32(3)], [f32(3), f32(3)])
    with pytest.raises(ValueError, match="not on the GPU"):
        block.GradClip([f32(3)])
    with pytest.raises(ValueError, match="float16"):
        block.GradClip([f32(3).half()])
    with pytest.raises(ValueError, match="strides"):
        block.GradClip([f32(4, 4).t()])


class Gpu0:
    """Stands for a tensor on GPU 0, for the checks that need an address alone."""

    def __init__(self, at, n, dtype=torch.float32):
        self.at, self.n, self.dtype = at, n, dtype

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.n

    def element_size(self):
        return self.dtype.itemsize


def test_tensors_that_share_memory(block):
    def apart(grads, outs=None):
        c = block.GradClip.__new__(block.GradClip)
        c.grads = tuple(grads)
        c.outs = c.grads if outs is None else tuple(outs)
        c._apart()
    a, b = Gpu0(4096, 100), Gpu0(4496, 100)
    apart([a, b])
    apart([a, a], [b, Gpu0(8192, 100)])      # read twice
    apart([Gpu0(4096, 0), a])
    for grads, outs in (([a, a], None), ([a, Gpu0(4492, 5)], None), ([a, b], [Gpu0(9000, 100), a]),
                        ([a], [Gpu0(4100, 100)]), ([a], [Gpu0(4096, 100, torch.bfloat16)]),
                        ([a, b], [Gpu0(9000, 100), Gpu0(9200, 100)]),
                        ([Gpu0(4096, 1000), b], [Gpu0(9000, 1000), Gpu0(4700, 100)])):
        with pytest.raises(ValueError, match="shares memory"):
            apart(grads, outs)


def test_codes_on_another_device(block):
    """Codes that were made on the host are not read by a call on GPU 0."""
    class Out:  # stands for a bf16 tensor [3, 128] on GPU 0, up to the call itself
        shape, dtype, device, is_cuda = (3, 128), torch.bfloat16, "cuda:0", True
        get_device = staticmethod(lambda: 0)
        stride = staticmethod(lambda: (128, 1))
        is_contiguous = staticmethod(lambda: True)
        data_ptr = staticmethod(lambda: 4096)
    for fmt in ("act8", "mx"):
        with pytest.raises(ValueError, match="q is (on cpu|not on a GPU)"):
            block.Codes8(3, 128, fmt, device="cpu").dequantize(Out(), stream=S)
