"""The expert FFN at few bits: experts served from 4-bit codes, and training
steps whose saved activations take 8 bits.

4-bit experts (MXFP4 or NVFP4, see include/moe_gb300.h for the formats):
:class:`Fp4Experts` holds both weights as codes and scale atoms, made from the
layer's bf16 weights or loaded from a 4-bit checkpoint; :func:`fp4_experts`
takes the router's permutation and runs gather + quantise, the up-projection
with the SwiGLU and the quantisation of Act in its epilogue, and the
down-projection.  :class:`Fp4Layer` is the serving layer around it (route,
permute, experts, combine), for prompts and for single tokens.

8-bit activation checkpoints: :func:`act8_swiglu_fwd` / :func:`act8_swiglu_bwd`
and :func:`act8_quantize` / :func:`act8_dequantize`.  :class:`Checkpoint8` keeps
what the bf16 layer's backward needs of a forward in 8 bits, so that layers share
one workspace: ``layer.forward(bufs, ...)``, ``ck.save(bufs)``, other layers'
forwards in the same ``bufs``, then ``ck.backward(bufs, ...)``.  The codes of H
feed the SwiGLU backward as they are, Act is recomputed there, and the permuted
tokens and the expert outputs are restored for the weight gradient and the
routing weights' gradient.

Every function launches on the given or current stream and returns without
waiting; each arithmetic step runs in libmoe_gb300.so.
"""
from __future__ import annotations

import torch

from . import _lib as L

FORMATS = {"mx": L.FP4_MX, "nv": L.FP4_NV}


def _fmt(fmt: str) -> int:
    if fmt not in FORMATS:
        raise ValueError("fmt is 'mx' (MXFP4) or 'nv' (NVFP4), not %r" % (fmt,))
    return FORMATS[fmt]


def _block(fmt: int) -> int:
    """Columns of a scale."""
    return 16 if fmt == L.FP4_NV else 32


def _expect(name, t, shape, what, ok):
    """t is a contiguous tensor of `shape` (None: any length) whose type passes `ok`."""
    got = tuple(t.shape)
    if len(got) != len(shape) or any(n is not None and n != m for n, m in zip(shape, got)) \
            or not ok(t) or not t.is_contiguous():
        raise ValueError("%s: %s %s, strides %s, for contiguous %s %s"
                         % (name, t.dtype, got, t.stride(), what, tuple(shape)))


def _bytes(t):  # codes and scales, whatever type of one byte they are called
    return t.element_size() == 1


def _bf16(t):
    return t.dtype == torch.bfloat16


def _expect_scale(name, t, n):
    """An fp32 scale of n elements, or None."""
    if t is not None and (t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous()):
        raise ValueError("%s: %s %s for %d contiguous fp32" % (name, t.dtype, tuple(t.shape), n))


# ------------------------------------------------------------------ 4-bit rows
class Fp4Rows:
    """Codes and scale atoms of grouped activation rows [rows, cols] (E groups)."""

    def __init__(self, rows: int, cols: int, E: int, fmt: str, device="cuda"):
        self.rows, self.cols, self.E, self.fmt = rows, cols, E, _fmt(fmt)
        nb = L.moe_fp4_scale_bytes(rows, cols, self.fmt, L.FP4_ROWS_GROUPED, E)
        self.q = torch.empty(rows, cols // 2, dtype=torch.uint8, device=device)
        self.sf = torch.empty(nb, dtype=torch.uint8, device=device)
        # scratch of a gather from up to rows / 2 source rows (others do without)
        self.workspace = torch.empty(L.moe_fp4_quantize_workspace_bytes(rows // 2, rows),
                                     dtype=torch.uint8, device=device)


def fp4_quantize(x, rows: Fp4Rows, group_offsets, row_index=None, index_div=1, scale=None,
                 dev_status=None, stream=None):
    """Rows of x bf16 into `rows`; with row_index int32 [rows] row p is
    x[row_index[p] / index_div] (the permute's sorted_to_flat with index_div = k),
    zeros where it is negative.  scale: fp32 [1] (nv)."""
    L.moe_fp4_quantize(x, rows.fmt, rows.q, rows.sf, L.FP4_ROWS_GROUPED, group_offsets,
                       row_index=row_index, index_div=index_div, scale=scale,
                       workspace=rows.workspace, dev_status=dev_status, stream=stream)


def fp4_dequantize(rows: Fp4Rows, group_offsets, out, scale=None, stream=None):
    """The values of `rows` into out bf16 [rows, cols] (rows past group_offsets[-1] are not
    written)."""
    L.moe_fp4_dequantize(rows.q, rows.sf, rows.fmt, out, L.FP4_ROWS_GROUPED, group_offsets,
                         scale=scale, stream=stream)


# --------------------------------------------------------------- 4-bit experts
class _Fixed:
    """Attributes are set once: the calls' arguments hold the tensors' addresses, and another
    tensor in their place would not be read."""

    def __setattr__(self, name, value):
        if name in self.__dict__:
            raise AttributeError("%s is fixed; write into the tensor, or make another %s"
                                 % (name, type(self).__name__))
        super().__setattr__(name, value)


class Fp4Experts(_Fixed):
    """The weights of E experts in 4 bits: wi [E, 2f, d] ([gate | up]) and wo [E, d, f], both
    K-major codes with scale atoms and (nv) one fp32 scale an expert; x_scale and act_scale
    (fp32 [1], nv) are the calibrated scales of the experts' input and of Act."""

    def __init__(self, fmt, wi_q, wi_sf, wi_scale, wo_q, wo_sf, wo_scale, x_scale=None,
                 act_scale=None):
        self.E, self.d, self.f = self._sizes(fmt, wi_q, wo_q)
        for name, t, rows, cols, m in (("wi_sf", wi_sf, 2 * self.f, self.d, L.FP4_ROWS_SWIGLU),
                                       ("wo_sf", wo_sf, self.d, self.f, L.FP4_ROWS_EXPERTS)):
            _expect(name, t, (None,), "atoms of one-byte scales", _bytes)
            nb = L.moe_fp4_scale_bytes(self.E * rows, cols, fmt, m, self.E)
            if t.numel() < nb:
                raise ValueError("%s: %d bytes of scale atoms, not %d" % (name, t.numel(), nb))
        for name, t, n in (("wi_scale", wi_scale, self.E), ("wo_scale", wo_scale, self.E),
                           ("x_scale", x_scale, 1), ("act_scale", act_scale, 1)):
            _expect_scale(name, t, n)
        tensors = (wi_q, wi_sf, wi_scale, wo_q, wo_sf, wo_scale, x_scale, act_scale)
        if any(t is not None and t.device != wo_q.device for t in tensors):
            raise ValueError("codes and scales on one device")
        self.fmt = fmt
        self.wi_q, self.wi_sf, self.wi_scale = wi_q, wi_sf, wi_scale
        self.wo_q, self.wo_sf, self.wo_scale = wo_q, wo_sf, wo_scale
        self.x_scale, self.act_scale = x_scale, act_scale
        self.arg = L.Fp4WeightsArg(
            self.E, self.d, self.f, fmt, *(None if t is None else t.data_ptr() for t in tensors))

    @staticmethod
    def _sizes(fmt, wi_q, wo_q):
        """(E, d, f) of the weights' codes."""
        if fmt not in FORMATS.values():
            raise ValueError("fmt is FP4_MX or FP4_NV, not %r" % (fmt,))
        _expect("wo_q", wo_q, (None, None, None), "one-byte codes", _bytes)
        E, d, f = wo_q.shape[0], wo_q.shape[1], 2 * wo_q.shape[2]
        _expect("wi_q", wi_q, (E, 2 * f, d // 2), "one-byte codes", _bytes)
        return E, d, f

    @classmethod
    def from_codes(cls, fmt, wi_q, wi_s, wi_scale, wo_q, wo_s, wo_scale, x_scale=None,
                   act_scale=None, stream=None):
        """From a 4-bit checkpoint: codes uint8 [E, 2f, d / 2] and [E, d, f / 2], scales in row
        order uint8 [E, 2f, d / block] and [E, d, f / block], fp32 [E] scales or None."""
        f = _fmt(fmt)
        E, d, ff = cls._sizes(f, wi_q, wo_q)
        _expect("wi_s", wi_s, (E, 2 * ff, d // _block(f)), "one-byte scales", _bytes)
        _expect("wo_s", wo_s, (E, d, ff // _block(f)), "one-byte scales", _bytes)

        def atoms(q, s, row_map):
            E, N, kb = q.shape
            nb = L.moe_fp4_scale_bytes(E * N, 2 * kb, f, row_map, E)
            sf = torch.empty(nb, dtype=torch.uint8, device=q.device)
            L.moe_fp4_arrange_scales(s, 2 * kb, f, row_map, E, sf)
            return sf

        with torch.cuda.stream(stream):  # (the allocations too)
            wi_sf, wo_sf = atoms(wi_q, wi_s, L.FP4_ROWS_SWIGLU), atoms(wo_q, wo_s, L.FP4_ROWS_EXPERTS)
        return cls(f, wi_q, wi_sf, wi_scale, wo_q, wo_sf, wo_scale, x_scale, act_scale)

    @classmethod
    def from_weights(cls, fmt, wi, wo, x_scale=None, act_scale=None, stream=None):
        """From the layer's bf16 weights wi [E, d, 2f], wo [E, f, d]; nv: each expert's fp32
        scale is its weight's max |w| / (6 * 448), kept in 8 significant bits, so that whether
        a ratio of two weights is a tie of the E4M3 or E2M1 grid does not hang on its last bit."""
        f = _fmt(fmt)
        _expect("wo", wo, (None, None, None), "bf16", _bf16)
        E, ff, d = wo.shape
        _expect("wi", wi, (E, d, 2 * ff), "bf16", _bf16)

        def quantise(w, row_map):
            E, K, N = w.shape
            scale = None
            if f == L.FP4_NV:
                amax = torch.empty(E, dtype=torch.float32, device=w.device)
                L.moe_fp8_amax(w.view(E * K, N), amax, groups=E)
                scale = (amax / (6.0 * 448.0)).bfloat16().float().clamp_(min=2.0 ** -64)
            nb = L.moe_fp4_scale_bytes(E * N, K, f, row_map, E)
            q = torch.empty(E, N, K // 2, dtype=torch.uint8, device=w.device)
            sf = torch.empty(nb, dtype=torch.uint8, device=w.device)
            L.moe_fp4_quantize_weights(w, f, row_map, q, sf, scale)
            return q, sf, scale

        with torch.cuda.stream(stream):  # (torch's own steps and the allocations too)
            parts = *quantise(wi, L.FP4_ROWS_SWIGLU), *quantise(wo, L.FP4_ROWS_EXPERTS)
        return cls(f, *parts, x_scale, act_scale)


class Fp4Buffers(_Fixed):
    """Device buffers of the 4-bit experts for up to rows_cap permuted rows."""

    def __init__(self, w: Fp4Experts, rows_cap: int, save_h=False):
        dev = w.wo_q.device
        name = {v: k for k, v in FORMATS.items()}[w.fmt]
        self.rows_cap = rows_cap
        self.x = Fp4Rows(rows_cap, w.d, w.E, name, device=dev)
        self.act = Fp4Rows(rows_cap, w.f, w.E, name, device=dev)
        self.h = torch.empty(rows_cap, 2 * w.f, dtype=torch.bfloat16,
                             device=dev) if save_h else None
        self.y = torch.empty(rows_cap, w.d, dtype=torch.bfloat16, device=dev)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.arg = L.Fp4BuffersArg(
            rows_cap, self.x.q.data_ptr(), self.x.sf.data_ptr(), self.x.sf.numel(),
            self.act.q.data_ptr(), self.act.sf.data_ptr(), self.act.sf.numel(),
            None if self.h is None else self.h.data_ptr(), self.y.data_ptr(),
            self.x.workspace.data_ptr(), self.x.workspace.numel(), self.dev_status.data_ptr())


def fp4_experts(w: Fp4Experts, b: Fp4Buffers, x, sorted_to_flat, k, group_offsets, stream=None,
                rows=None):
    """Expert outputs y bf16 [rows_cap, d] of the permuted rows of x bf16 [T, d]
    (sorted_to_flat int32 [rows], group_offsets int32 [E + 1] as moe_permute leaves them;
    rows past group_offsets[E] are not written).  With b.h also H = [gate | up] in bf16.
    rows: the first so many rows hold every group (rows_cap, or fewer where x is short of what
    the buffers are for); group_offsets past them are clamped."""
    cap = b.rows_cap if rows is None else rows
    if not 0 <= cap <= b.rows_cap:
        raise ValueError("rows = %d of %d" % (cap, b.rows_cap))
    if sorted_to_flat.shape[0] < cap or group_offsets.shape[0] != w.E + 1:
        raise ValueError("sorted_to_flat of %d rows (%d), group_offsets of %d (E %d)"
                         % (sorted_to_flat.shape[0], cap, group_offsets.shape[0], w.E))
    if x.shape[1] != w.d or b.y.shape[1] != w.d or b.act.cols != w.f:
        raise ValueError("x of %d columns, buffers for (%d, %d), experts (%d, %d)"
                         % (x.shape[1], b.y.shape[1], b.act.cols, w.d, w.f))
    arg = b.arg
    if cap != b.rows_cap:
        arg = L.Fp4BuffersArg.from_buffer_copy(b.arg)
        arg.rows_cap = cap
    L.moe_fp4_experts(w.arg, arg, x, sorted_to_flat, k, group_offsets, stream)
    return b.y


class Fp4Layer:
    """The serving layer for up to T tokens: routing (a LayerShape's router, alignment and
    capacity options; biases, other precisions, K-chunks and the auxiliary loss are refused),
    the 4-bit experts and the combine.  ``forward(x, logits)`` -> out bf16 [T', d] for x bf16 [T', d],
    logits fp32 [T', E], T' <= T (a view of the layer's buffer)."""

    def __init__(self, w: Fp4Experts, s):
        if (s.E, s.d, s.f) != (w.E, w.d, w.f):
            raise ValueError("shape (E, d, f) = (%d, %d, %d) for experts (%d, %d, %d)"
                             % (s.E, s.d, s.f, w.E, w.d, w.f))
        if s.bias:
            raise ValueError("the 4-bit experts take no biases")
        # the products' precision and schedule and the training loss are not the serving layer's
        if s.fp8 or s.mxfp8 or s.num_chunks > 1 or s.aux_coeff:
            raise ValueError("the 4-bit serving layer takes no fp8, mxfp8, num_chunks or aux_coeff")
        dev = w.wo_q.device
        i32 = dict(dtype=torch.int32, device=dev)
        self.w, self.s = w, s
        R = L.moe_rows_cap(s.T, s.E, s.k, s.align, s.capacity)
        self.bufs = Fp4Buffers(w, R)
        self.topk_idx = torch.empty(s.T, s.k, **i32)
        self.topk_w = torch.empty(s.T, s.k, dtype=torch.float32, device=dev)
        self.sizes, self.kept = torch.empty(s.E, **i32), torch.empty(s.E, **i32)
        self.offsets = torch.empty(s.E + 1, **i32)
        self.s2f, self.f2s = torch.empty(R, **i32), torch.empty(s.T * s.k, **i32)
        # the permute gathers no more than 8 columns: the experts gather codes themselves
        self.head = torch.empty(R, 8, dtype=torch.bfloat16, device=dev)
        self.ws = torch.empty(L.moe_permute_workspace_bytes(s.T, s.E), dtype=torch.uint8,
                              device=dev)
        self.out = torch.empty(s.T, s.d, dtype=torch.bfloat16, device=dev)

    def forward(self, x, logits, expert_bias=None, stream=None):
        s, T = self.s, x.shape[0]
        if T > s.T or logits.shape != (T, s.E):
            raise ValueError("x of %d tokens (at most %d), logits of shape %s"
                             % (T, s.T, tuple(logits.shape)))
        L._need_matrix("x", x, T, s.d, torch.bfloat16)
        L._need_type("logits", logits, torch.float32)
        L._need("expert_bias", expert_bias, s.E, torch.float32)
        idx, w, f2s, out = self.topk_idx[:T], self.topk_w[:T], self.f2s[:T * s.k], self.out[:T]
        if T == 0:
            return out
        L.moe_route_topk(logits, s.k, s.score_fn, s.renorm, idx, w, stream,
                         expert_bias=expert_bias, num_groups=s.num_groups, topk_group=s.topk_group)
        L.moe_permute(x[:, :8], idx, s.E, s.align, s.capacity, self.head, self.sizes, self.kept,
                      self.offsets, self.s2f, f2s, self.ws, self.bufs.dev_status, stream)
        # the kernels take their tiles by the rows that T tokens can fill
        R = L.moe_rows_cap(T, s.E, s.k, s.align, s.capacity)
        y = fp4_experts(self.w, self.bufs, x, self.s2f, s.k, self.offsets, stream, rows=R)
        L.moe_combine(y, f2s, w, out, s.k, stream)
        return out


# --------------------------------------------------- 8-bit activation checkpoints
# x bf16 [rows, cols] <-> q int8 [rows, cols], scales bf16 [rows, ceil(cols / 32)]; h bf16
# [rows, 2F] -> act and its codes; codes and dact -> dh and act (see the functions' own words)
act8_quantize = L.moe_act8_quantize
act8_dequantize = L.moe_act8_dequantize
act8_swiglu_fwd = L.moe_act8_swiglu_fwd
act8_swiglu_bwd = L.moe_act8_swiglu_bwd


class Checkpoint8:
    """What the bf16 layer's backward needs of one forward, in 8 bits: codes of the permuted
    tokens, of H and of the expert outputs, and the routing decision.  One for each layer of a
    model; all of them may share one MoEBuffers."""

    def __init__(self, b):
        s = b.s
        if s.fp8 or s.mxfp8 or s.wgrad_colwise:
            raise ValueError("8-bit checkpoints are of the bf16 layer without column-wise copies")
        if s.d % 8 or s.f % 8:
            raise ValueError("d=%d and f=%d must be multiples of 8" % (s.d, s.f))
        self.s = s
        dev = b.workspace.device
        R, nf = b.rows_cap, -(-s.f // 32)

        def codes(cols, blocks):
            return (torch.empty(R, cols, dtype=torch.int8, device=dev),
                    torch.empty(R, blocks, dtype=torch.bfloat16, device=dev))

        self.xs, self.y = codes(s.d, -(-s.d // 32)), codes(s.d, -(-s.d // 32))
        self.h = codes(2 * s.f, 2 * nf)
        self.nf = nf
        names = ("topk_idx", "topk_w", "group_offsets", "s2f", "f2s") + (
            ("aux_counts",) if s.aux_coeff else ())
        self.routing = {n: torch.empty_like(getattr(b, n)) for n in names}
        self.logits = torch.empty(s.T, s.E, dtype=torch.float32, device=dev)
        self.saved = False

    def nbytes(self) -> int:
        """Bytes of the codes and the routing decision (the logits, 4 T E, beside them)."""
        ts = [*self.xs, *self.h, *self.y, *self.routing.values()]
        return sum(t.numel() * t.element_size() for t in ts)

    def _same_shape(self, b):
        if b.s != self.s:
            raise ValueError("a checkpoint of %r for buffers of %r" % (self.s, b.s))

    def save(self, b, stream=None):
        """After layer.forward(b, ...): afterwards b is free for another layer's forward."""
        self._same_shape(b)
        if b.logits is None:
            raise ValueError("Checkpoint8.save before a forward")
        f, nf = b.s.f, self.nf
        off = b.group_offsets
        self.saved = True
        with torch.cuda.stream(stream):
            self.logits.copy_(b.logits)  # the caller's tensor may hold the next layer's soon
            for n, t in self.routing.items():
                t.copy_(getattr(b, n))
        act8_quantize(b.xs, *self.xs, off, stream)
        act8_quantize(b.y, *self.y, off, stream)
        q, sc = self.h
        if f % 32 == 0:  # no block straddles the halves
            act8_quantize(b.h, q, sc, off, stream)
        else:
            act8_quantize(b.h[:, :f], q[:, :f], sc[:, :nf], off, stream)
            act8_quantize(b.h[:, f:], q[:, f:], sc[:, nf:], off, stream)

    def backward(self, b, dout, wi, wo, stream=None):
        """layer.backward of the saved forward: (dx, dwi, dwo, d_topk_w) in b's buffers, the
        router-logit gradient in b.d_logits, bias gradients in b.dbi and b.dbo.  A forward that
        b still holds is lost (save it first): its state gives way."""
        self._same_shape(b)
        if not self.saved:
            raise ValueError("Checkpoint8.backward before save")
        b.logits = None  # layer.backward and save of that forward are refused
        s, r = b.s, self.routing
        off, f2s, st = r["group_offsets"], r["f2s"], b.dev_status
        act8_dequantize(*self.y, b.y, off, stream)
        L.moe_unpermute_bwd(dout, b.y, f2s, r["s2f"], off, r["topk_w"], b.dy, b.d_topk_w, stream)
        L.moe_route_topk_bwd(self.logits, r["topk_idx"], r["topk_w"], b.d_topk_w, s.score_fn,
                             s.renorm, b.d_logits, stream)
        if s.aux_coeff:
            L.moe_aux_loss_bwd(self.logits, r["aux_counts"], s.k, s.score_fn, s.aux_coeff,
                               b.d_logits, stream=stream)
        dact = b.h[:, :s.f]  # H itself is not needed: its codes are
        L.moe_gmm(b.dy, wo, 1, off, dact, dev_status=st, stream=stream)
        act8_swiglu_bwd(*self.h, dact, b.dh, b.act, off, stream)
        L.moe_tgmm(b.act, b.dy, off, b.dwo, dev_status=st, stream=stream)
        if s.bias:
            L.moe_group_colsum(b.dy, off, b.dbo, stream)
            L.moe_group_colsum(b.dh, off, b.dbi, stream)
        L.moe_gmm(b.dh, wi, 1, off, b.dxs, dev_status=st, stream=stream)
        act8_dequantize(*self.xs, b.xs, off, stream)
        L.moe_tgmm(b.xs, b.dh, off, b.dwi, dev_status=st, stream=stream)
        L.moe_combine(b.dxs, f2s, None, b.dx, s.k, stream)
        return b.dx, b.dwi, b.dwo, b.d_topk_w
