"""What a training or serving step has around the expert layer, on the library's kernels.

Before it: :func:`rms_norm` adds the residual and normalises, in one pass, with the output in
bf16, in 8 bits (:class:`Codes8`), or both; :func:`rms_norm_bwd` is its backward.
Beside it: :class:`SeqAuxLoss`, the load-balancing loss of every sequence of a ragged batch with
the router's z loss, its gradient from the same pass over the logits or by itself.  (The
layer's own ``aux_coeff`` is one loss for the whole batch.)
After it: :class:`GradClip`, the norm of all gradients together and their clipping.

A step of a pre-norm block: ``rms_norm(x, w, eps, y, residual=r, h=h)``, the router's logits from
y, ``layer.forward(b, y, logits, ...)``; then ``layer.backward(b, dout, ...)``,
``loss.forward(logits, b.topk_idx, seq_offsets, d_logits=b.d_logits, accumulate=True)``,
``rms_norm_bwd(dy, h, w, eps, dh, dw, ws, d_residual=...)`` and ``clip.clip(max_norm)``.

Every function launches on the given or current stream and returns without waiting; each
arithmetic step runs in libmoe_gb300.so.  Tensors that the caller passes have to lie on the
stream's GPU (ValueError).
"""
from __future__ import annotations

import torch

from . import _lib as L

CODES = {"mx": L.CODES_MX, "act8": L.CODES_ACT8}


class Codes8:
    """8-bit codes and scales of [rows, cols]: "mx" (E4M3 with a power of two for 32 columns, the A
    operand of moe_gmm_mx with one group; cols % 128 == 0) or "act8" (int8 with a bf16 scale for 32
    columns, as the checkpoints keep activations)."""

    def __init__(self, rows: int, cols: int, fmt: str, device="cuda"):
        if fmt not in CODES:
            raise ValueError("fmt is 'mx' or 'act8', not %r" % (fmt,))
        if rows < 0 or cols <= 0 or cols % (128 if fmt == "mx" else 8):
            raise ValueError("%d rows of %d columns: multiples of %d for %s"
                             % (rows, cols, 128 if fmt == "mx" else 8, fmt))
        self.rows, self.cols, self.fmt = rows, cols, fmt
        self.q = torch.empty(rows, cols, dtype=torch.uint8 if fmt == "mx" else torch.int8,
                             device=device)
        if fmt == "mx":
            nb = L.moe_mx_scale_bytes(rows, cols, L.MX_ROWS_PLAIN)
            self.scales = torch.empty(nb, dtype=torch.uint8, device=device)
        else:
            self.scales = torch.empty(rows, -(-cols // 32), dtype=torch.bfloat16, device=device)

    def dequantize(self, out, stream=None):
        """The values, rounded once to bf16, in out [rows, cols]."""
        if tuple(out.shape) != (self.rows, self.cols):
            raise ValueError("out is %s, not [%d, %d]" % (tuple(out.shape), self.rows, self.cols))
        if self.fmt == "mx":
            L.moe_mx_dequantize(self.q, self.scales, L.FP8_E4M3, out, stream)
        else:
            for name, t in (("q", self.q), ("scales", self.scales), ("out", out)):
                L._need_device(name, t, stream)
            L.moe_act8_dequantize(self.q, self.scales, out, None, stream)
        return out


def rms_norm(x, w, eps, y=None, residual=None, h=None, codes=None, stream=None):
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * w over the last of two dimensions.

    x bf16 [rows, cols] or None (the residual alone is normalised); residual and h bf16 or fp32, of
    one type (the residual stream's; h may be residual); w bf16 or fp32 [cols]; y bf16 or None;
    codes: a Codes8 of [rows, cols] that takes y in 8 bits, or None.  Returns y."""
    if codes is None:
        L.moe_rms_norm(x, residual, w, eps, h, y, 0, None, None, stream)
    else:
        L.moe_rms_norm(x, residual, w, eps, h, y, CODES[codes.fmt], codes.q, codes.scales, stream)
    return y


def rms_norm_bwd_workspace(rows: int, cols: int, device="cuda"):
    """Scratch of rms_norm_bwd for up to so many rows."""
    return torch.empty(L.moe_rms_norm_bwd_workspace_bytes(rows, cols), dtype=torch.uint8, device=device)


def rms_norm_bwd(dy, h, w, eps, dh, dw=None, workspace=None, d_residual=None, dx=None,
                 accumulate=False, stream=None):
    """From dy bf16 and the h that the forward kept: dh (h's type) = the norm's gradient +
    d_residual, the gradient of x and of the residual; dx: the same in bf16 too; dw fp32 [cols]
    (added to with accumulate; needs a workspace)."""
    L.moe_rms_norm_bwd(dy, h, w, eps, dh, dw, workspace, d_residual, dx, accumulate, stream)
    return dh


class SeqAuxLoss:
    """The balance loss of up to B ragged sequences of up to T tokens, and the router's z loss.

    After ``forward``: ``loss`` fp32 [2] (balance, z), ``counts`` int32 [B, E], ``tokens`` int32 [B]
    (live ones), ``probs`` fp32 [B, E], all on the device.  One instance serves one batch at a time."""

    def __init__(self, T: int, E: int, k: int, B: int, score_fn=L.SCORE_SOFTMAX, coeff=0.0,
                 z_coeff=0.0, device="cuda"):
        nb = L.moe_seq_aux_loss_workspace_bytes(T, E, B)
        if nb == 0 or not 0 < k <= E:
            raise ValueError("T=%d E=%d k=%d B=%d" % (T, E, k, B))
        self.T, self.E, self.k, self.B = T, E, k, B
        self.score_fn, self.coeff, self.z_coeff = score_fn, float(coeff), float(z_coeff)
        i32, f32 = (dict(dtype=t, device=device) for t in (torch.int32, torch.float32))
        self.counts, self.tokens = torch.empty(B, E, **i32), torch.empty(B, **i32)
        self.probs, self.loss = torch.empty(B, E, **f32), torch.empty(2, **f32)
        self.workspace = torch.empty(nb, dtype=torch.uint8, device=device)
        self.seen = None  # tokens of the last forward

    def _shape(self, logits, seq_offsets):
        if logits.dim() != 2 or logits.shape[0] > self.T or logits.shape[1] != self.E \
                or seq_offsets.numel() != self.B + 1:
            raise ValueError("logits %s and %d offsets for at most %d tokens, %d experts, %d sequences"
                             % (tuple(logits.shape), seq_offsets.numel(), self.T, self.E, self.B))

    def forward(self, logits, topk_idx, seq_offsets, token_mask=None, d_logits=None, d_loss=1.0,
                accumulate=False, stream=None):
        """logits fp32 [T', E] (T' <= T), topk_idx int32 [T', k], seq_offsets int32 [B + 1], token_mask
        bool or uint8 [T'] or None -> loss.  With d_logits fp32 [T', E] the gradient (times d_loss)
        is written there, or added with accumulate, in the same pass."""
        self._shape(logits, seq_offsets)
        if topk_idx.shape[-1] != self.k:
            raise ValueError("topk_idx of %d choices, not %d" % (topk_idx.shape[-1], self.k))
        L.moe_seq_aux_loss(logits, topk_idx, seq_offsets, self.score_fn, self.coeff, self.z_coeff,
                           self.counts, self.tokens, self.probs, self.loss, self.workspace,
                           token_mask, d_logits, d_loss, accumulate, stream)
        self.seen = logits.shape[0]
        return self.loss

    def backward(self, logits, seq_offsets, d_logits, token_mask=None, d_loss=1.0, accumulate=True,
                 stream=None):
        """The gradient of the last forward into d_logits: of the same logits, offsets and mask, as
        the counts are those of that forward (no other batch in between, of the same size either)."""
        self._shape(logits, seq_offsets)
        if logits.shape[0] != self.seen:
            raise ValueError("SeqAuxLoss.backward of %d tokens, the last forward was of %s"
                             % (logits.shape[0], self.seen))
        L.moe_seq_aux_loss_bwd(logits, self.k, seq_offsets, self.score_fn, self.coeff, self.z_coeff,
                               self.counts, self.tokens, d_logits, token_mask, d_loss, accumulate, stream)
        return d_logits


class GradClip:
    """The norm of `grads` together (bf16 / fp32 tensors, contiguous, on one GPU), and their
    clipping, in place or into `outs` (of the same sizes, bf16 or fp32).  The tensors' addresses are
    laid out once: the instance keeps the tensors, and what is written into them counts.
    ``GradClip.of(b)``: the gradients of an expert layer's buffers (layer.MoEBuffers)."""

    def __init__(self, grads, outs=None):
        self.grads = tuple(grads)
        self.outs = self.grads if outs is None else tuple(outs)
        if not self.grads or len(self.grads) != len(self.outs):
            raise ValueError("%d gradients, %d outputs" % (len(self.grads), len(self.outs)))
        dev = self.grads[0].device
        for i, (g, o) in enumerate(zip(self.grads, self.outs)):
            for name, t in (("gradient", g), ("output", o)):
                if t.dtype not in (torch.bfloat16, torch.float32) or not t.is_contiguous():
                    raise ValueError("%s %d: %s, strides %s, for contiguous bf16 or fp32"
                                     % (name, i, t.dtype, t.stride()))
                if t.device != dev or not t.is_cuda:
                    raise ValueError("%s %d is on %s, not on the GPU of the first gradient" % (name, i, t.device))
            if g.numel() != o.numel():
                raise ValueError("output %d of %d elements for %d" % (i, o.numel(), g.numel()))
        self._apart()
        plan, self.chunks = L.moe_clip_plan(self.grads, self.outs)
        self.plan = plan.to(dev)
        self.workspace = torch.empty(L.moe_clip_workspace_bytes(), dtype=torch.uint8, device=dev)
        self.total = torch.empty(1, dtype=torch.float32, device=dev)

    def _apart(self):
        """No memory that is written is another tensor's."""
        spans = []
        for i, (g, o) in enumerate(zip(self.grads, self.outs)):
            for t, written in ((g, False), (o, True)):
                if t.numel() and not (not written and g.data_ptr() == o.data_ptr() and g.dtype == o.dtype):
                    spans.append((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), written, i))
        spans.sort()
        end, end_written, last = 0, 0, None
        for lo, hi, written, i in spans:
            if lo < (end if written else end_written):
                raise ValueError("tensor %d shares memory with tensor %d" % (i, last))
            if hi > end:
                end, last = hi, i
            if written:
                end_written = max(end_written, hi)

    @classmethod
    def of(cls, b, *more):
        """The weight gradients of one layer's buffers, those of its biases, and `more` tensors."""
        return cls([t for t in (b.dwi, b.dwo, b.dbi, b.dbo) if t is not None] + list(more))

    def norm(self, scale=1.0, stream=None):
        """scale * sqrt(sum of squares), fp32 [1] on the device; nothing else is written."""
        L.moe_grad_norm(self.plan, self.chunks, scale, self.total, self.workspace, stream)
        return self.total

    def clip(self, max_norm, scale=1.0, stream=None):
        """outs = grads * scale * min(1, max_norm / (norm + 1e-6)); returns the norm (of the scaled
        gradients; the same tensor each time).  A norm that is not finite clips nothing: leave the step out."""
        L.moe_clip_grads(self.plan, self.chunks, max_norm, scale, self.total, self.workspace, stream)
        return self.total
