"""fp64 oracle of the low-bit formats: 4-bit block-scaled floats (MXFP4 as in
the OCP Microscaling (MX) v1.0 definition, NVFP4's 16-element blocks with E4M3
scales) and 8-bit activation checkpoints.  NumPy, written from the formats'
definitions; test infrastructure only."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _pow2(e):
    return np.ldexp(1.0, np.asarray(e, np.int64))


def _floor_log2(v):
    return np.frexp(v)[1] - 1


def round_e4m3(v):
    """v >= 0 to the nearest E4M3 value (ties to even), saturated at 448."""
    v = np.minimum(v, 448.0)
    step = _pow2(_floor_log2(np.maximum(v, 2.0 ** -6)) - 3)
    return np.rint(v / step) * step


def e4m3_code(v):
    """Code of an E4M3 value v >= 0."""
    e = np.maximum(_floor_log2(np.maximum(v, 2.0 ** -6)), -6)
    m = np.rint(v / _pow2(e - 3)).astype(np.int64)  # 8..15, below 8 for subnormals
    return np.where(m >= 8, ((e + 7) << 3) + (m - 8), m).astype(np.uint8)


def e4m3_value(code):
    c = np.asarray(code).astype(np.int64)
    ex, man = (c >> 3) & 15, c & 7
    v = np.where(ex > 0, (1 + man / 8) * _pow2(ex - 7), man / 8 * 2.0 ** -6)
    return np.where(c == 0x7F, np.nan, v)


def e8m0_value(code):
    c = np.asarray(code).astype(np.int64)
    return np.where(c == 255, np.nan, _pow2(c - 127))


def fp4_quantize(x, fmt, g=1.0):
    """x [rows, cols] -> (element codes uint8 [rows, cols] (4 bits), scale codes uint8 [rows,
    cols / block], values [rows, cols])."""
    x = np.asarray(x, np.float64)
    blk = 16 if fmt == "nv" else 32
    b = x.reshape(x.shape[0], -1, blk)
    finite = np.isfinite(b).all(-1)
    a = np.where(finite[..., None], np.abs(b), 0.0).max(-1)
    if fmt == "nv":
        s = round_e4m3(a / (6.0 * g))
        code = e4m3_code(s)
        t = s * g
        nan_code = 0x7F
    else:
        e = np.clip(_floor_log2(np.where(a > 0, a, 1.0)) - 2, -127, 127)
        e = np.where(a > 0, e, -127)
        code = (e + 127).astype(np.uint8)
        t = np.where(a > 0, _pow2(e), 0.0)
        nan_code = 0xFF
    r = np.where((t > 0)[..., None] & finite[..., None], b, 0.0) / np.where(t > 0, t, 1.0)[..., None]
    m = np.minimum(np.abs(r), 6.0)
    step = _pow2(_floor_log2(np.maximum(m, 1.0)) - 1)
    mag = np.rint(m / step) * step
    el = np.searchsorted(E2M1, mag).astype(np.uint8) + 8 * ((r < 0).astype(np.uint8))
    val = np.sign(r) * mag * t[..., None]
    code = np.where(finite, code, nan_code).astype(np.uint8)
    val = np.where(finite[..., None], val, np.nan)
    return el.reshape(x.shape), code, val.reshape(x.shape)


def fp4_values(el, code, fmt, g=1.0):
    """Values of element codes [rows, cols] and scale codes [rows, cols / block]."""
    v = E2M1[el & 7] * np.where(el & 8, -1.0, 1.0)
    t = e4m3_value(code) * g if fmt == "nv" else e8m0_value(code)
    return v * np.repeat(t, v.shape[1] // t.shape[1], axis=1)


def pack(el):
    return (el[:, ::2] | (el[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    return np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)


def padded_row(r, G, row_map):
    """Padded row ("experts", "swiglu") of row r of E groups of G rows."""
    e, n = divmod(r, G)
    if row_map == "swiglu":
        up, m = divmod(n, G // 2)
        n = m // 32 * 64 + 32 * up + m % 32
    return e * (-(-G // 128) * 128) + n


def scale_byte(pr, blk, ac):
    """Byte of (padded row, block) in atoms of `ac` atom columns."""
    rw = pr % 128
    return ((pr // 128) * ac + blk // 4) * 512 + (rw % 32) * 16 + (rw // 32) * 4 + blk % 4


# ------------------------------------------------- 8-bit activation checkpoints
def bf16_up(v):
    """v >= 0 rounded up to bf16 (8 significant bits; no subnormals needed)."""
    step = _pow2(_floor_log2(np.maximum(v, 2.0 ** -126)) - 7)
    return np.ceil(v / step) * step


def bf16_half_step(v):
    """Half the spacing of bf16 numbers at v: what one rounding to nearest may move it."""
    return _pow2(_floor_log2(np.maximum(np.abs(v), 2.0 ** -126)) - 8)


def act8_quantize(x):
    """x [rows, cols] -> (codes [rows, cols], scales [rows, ceil(cols / 32)], values)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb = -(-cols // 32)
    b = np.zeros((rows, nb * 32))
    b[:, :cols] = x
    b = b.reshape(rows, nb, 32)
    finite = np.isfinite(b).all(-1)
    a = np.where(finite[..., None], np.abs(b), 0.0).max(-1)
    s = np.where(a >= 2.0 ** -100, bf16_up(a / 127.0), 0.0)
    ok = (s > 0) & finite
    q = np.rint(np.where(ok[..., None], b, 0.0) / np.where(ok, s, 1.0)[..., None])
    s = np.where(finite, s, np.nan)
    v = q * s[..., None]
    return (q.reshape(rows, -1)[:, :cols], s, v.reshape(rows, -1)[:, :cols])


def swiglu(h):
    F = h.shape[1] // 2
    g, u = h[:, :F], h[:, F:]
    return g / (1.0 + np.exp(-g)) * u


def swiglu_bwd(h, dact):
    """(dh, act) at h = [gate | up]."""
    F = h.shape[1] // 2
    g, u = h[:, :F], h[:, F:]
    s = 1.0 / (1.0 + np.exp(-g))
    return (np.concatenate([dact * u * s * (1.0 + g * (1.0 - s)), dact * g * s], 1), g * s * u)
