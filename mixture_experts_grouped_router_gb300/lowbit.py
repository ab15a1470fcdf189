"""The expert FFN at few bits: experts served from 4-bit codes, and training
steps whose saved activations take 8 bits.

4-bit experts (MXFP4 or NVFP4, see include/moe_gb300.h for the formats):
:class:`Fp4Experts` holds both weights as codes and scale atoms, made from the
layer's bf16 weights or loaded from a 4-bit checkpoint; :func:`fp4_experts`
takes the router's permutation and runs gather + quantise, the up-projection
with the SwiGLU and the quantisation of Act in its epilogue, and the
down-projection.  :func:`fp4_layer` is the whole serving layer around it (route,
permute, experts, combine).

8-bit activation checkpoints: :func:`act8_swiglu_fwd` / :func:`act8_swiglu_bwd`
and :func:`act8_quantize` / :func:`act8_dequantize`.

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
class Fp4Experts:
    """The weights of E experts in 4 bits: wi [E, 2f, d] ([gate | up]) and wo [E, d, f], both
    K-major codes with scale atoms and (nv) one fp32 scale an expert; x_scale and act_scale
    (fp32 [1], nv) are the calibrated scales of the experts' input and of Act."""

    def __init__(self, fmt, wi_q, wi_sf, wi_scale, wo_q, wo_sf, wo_scale, x_scale=None,
                 act_scale=None):
        self.fmt = fmt
        self.wi_q, self.wi_sf, self.wi_scale = wi_q, wi_sf, wi_scale
        self.wo_q, self.wo_sf, self.wo_scale = wo_q, wo_sf, wo_scale
        self.x_scale, self.act_scale = x_scale, act_scale
        self.E, self.d, self.f = wo_q.shape[0], wo_q.shape[1], 2 * wo_q.shape[2]
        if wi_q.shape != (self.E, 2 * self.f, self.d // 2):
            raise ValueError("wi codes of shape %s do not match wo's %s"
                             % (tuple(wi_q.shape), tuple(wo_q.shape)))
        if not (wi_q.is_contiguous() and wo_q.is_contiguous()):
            raise ValueError("the weights' codes are contiguous")
        self.arg = L.Fp4WeightsArg(
            self.E, self.d, self.f, fmt, *(None if t is None else t.data_ptr() for t in (
                wi_q, wi_sf, wi_scale, wo_q, wo_sf, wo_scale, x_scale, act_scale)))

    @classmethod
    def from_codes(cls, fmt, wi_q, wi_s, wi_scale, wo_q, wo_s, wo_scale, x_scale=None,
                   act_scale=None, stream=None):
        """From a 4-bit checkpoint: codes uint8 [E, 2f, d / 2] and [E, d, f / 2], scales in row
        order uint8 [E, 2f, d / block] and [E, d, f / block], fp32 [E] scales or None."""
        f = _fmt(fmt)

        def atoms(q, s, row_map):
            E, N, kb = q.shape
            nb = L.moe_fp4_scale_bytes(E * N, 2 * kb, f, row_map, E)
            sf = torch.empty(nb, dtype=torch.uint8, device=q.device)
            L.moe_fp4_arrange_scales(s, 2 * kb, f, row_map, E, sf, stream)
            return sf

        return cls(f, wi_q, atoms(wi_q, wi_s, L.FP4_ROWS_SWIGLU), wi_scale,
                   wo_q, atoms(wo_q, wo_s, L.FP4_ROWS_EXPERTS), wo_scale, x_scale, act_scale)

    @classmethod
    def from_weights(cls, fmt, wi, wo, x_scale=None, act_scale=None, stream=None):
        """From the layer's bf16 weights wi [E, d, 2f], wo [E, f, d]; nv: each expert's fp32
        scale is its weight's max |w| / (6 * 448), kept in 8 significant bits, so that whether
        a ratio of two weights is a tie of the E4M3 or E2M1 grid does not hang on its last bit."""
        f = _fmt(fmt)

        def quantise(w, row_map):
            E, K, N = w.shape
            scale = None
            if f == L.FP4_NV:
                amax = torch.empty(E, dtype=torch.float32, device=w.device)
                L.moe_fp8_amax(w.view(E * K, N), amax, groups=E, stream=stream)
                scale = (amax / (6.0 * 448.0)).bfloat16().float().clamp_(min=2.0 ** -64)
            nb = L.moe_fp4_scale_bytes(E * N, K, f, row_map, E)
            q = torch.empty(E, N, K // 2, dtype=torch.uint8, device=w.device)
            sf = torch.empty(nb, dtype=torch.uint8, device=w.device)
            L.moe_fp4_quantize_weights(w, f, row_map, q, sf, scale, stream)
            return q, sf, scale

        return cls(f, *quantise(wi, L.FP4_ROWS_SWIGLU), *quantise(wo, L.FP4_ROWS_EXPERTS), x_scale,
                   act_scale)


class Fp4Buffers:
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


def fp4_experts(w: Fp4Experts, b: Fp4Buffers, x, sorted_to_flat, k, group_offsets, stream=None):
    """Expert outputs y bf16 [rows_cap, d] of the permuted rows of x bf16 [T, d]
    (sorted_to_flat int32 [rows_cap], group_offsets int32 [E + 1] as moe_permute leaves them;
    rows past group_offsets[E] are not written).  With b.h also H = [gate | up] in bf16."""
    if sorted_to_flat.shape[0] < b.rows_cap or group_offsets.shape[0] != w.E + 1:
        raise ValueError("sorted_to_flat of %d rows (rows_cap %d), group_offsets of %d (E %d)"
                         % (sorted_to_flat.shape[0], b.rows_cap, group_offsets.shape[0], w.E))
    if x.shape[1] != w.d or b.y.shape[1] != w.d or b.act.cols != w.f:
        raise ValueError("x of %d columns, buffers for (%d, %d), experts (%d, %d)"
                         % (x.shape[1], b.y.shape[1], b.act.cols, w.d, w.f))
    L.moe_fp4_experts(w.arg, b.arg, x, sorted_to_flat, k, group_offsets, stream)
    return b.y


# --------------------------------------------------- 8-bit activation checkpoints
# x bf16 [rows, cols] <-> q int8 [rows, cols], scales bf16 [rows, ceil(cols / 32)]; h bf16
# [rows, 2F] -> act and its codes; codes and dact -> dh and act (see the functions' own words)
act8_quantize = L.moe_act8_quantize
act8_dequantize = L.moe_act8_dequantize
act8_swiglu_fwd = L.moe_act8_swiglu_fwd
act8_swiglu_bwd = L.moe_act8_swiglu_bwd
