"""Timed cases of the low-bit expert operators: 4-bit block-scaled quantisation, the expert FFN on
4-bit codes, and 8-bit activation checkpoints with the backward pass that reads them.

Each case is one call sequence of a program around the MoE layer.  With ``own`` false the operators
are computed in elementary torch operations in 32 bits; with it true through this package.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def _round(name, fmt, T, d, E, k):
    return dict(name=name, kind="fp4_round", fmt=fmt, T=T, d=d, E=E, k=k)


def _experts(name, fmt, T, d, f, E, k):
    return dict(name=name, kind="fp4_experts", fmt=fmt, T=T, d=d, f=f, E=E, k=k)


def _swiglu(name, rows, f):
    return dict(name=name, kind="act8_swiglu", rows=rows, f=f)


def _saved(name, rows, d):
    return dict(name=name, kind="act8_saved", rows=rows, d=d)


def listed():
    return [
        # a prompt batch's tokens gathered by expert into 4-bit codes and read back
        _round("fp4_round_nv_prompt", "nv", 16384, 4096, 8, 2),
        # the same of an odd number of tokens, top-8 of many experts
        _round("fp4_round_mx_odd", "mx", 777, 7168, 32, 8),
        # one token decoded through the Mixtral-like experts: the weights' bytes are the cost
        _experts("experts_nv_token", "nv", 1, 4096, 14336, 8, 2),
        # a small decoding batch through the DeepSeek-like experts
        _experts("experts_mx_decode", "mx", 13, 7168, 2048, 32, 8),
        # the tiny layer: latency
        _experts("experts_mx_tiny", "mx", 256, 128, 256, 8, 2),
        # a prompt's chunk through the DeepSeek-like experts
        _experts("experts_nv_prompt", "nv", 1024, 7168, 2048, 32, 8),
        # the Mixtral-like layer's batch, an odd number of tokens
        _experts("experts_mx_batch", "mx", 16381, 4096, 14336, 8, 2),
        # a training step's activation function from its 8-bit saved input: the Mixtral-like layer
        _swiglu("act8_swiglu_train", 32768, 14336),
        # ragged live rows, DeepSeek-like width
        _swiglu("act8_swiglu_odd", 1237, 2048),
        # the tiny layer's rows
        _swiglu("act8_swiglu_tiny", 512, 256),
        # permuted tokens saved for the weight gradient and restored before it
        _saved("act8_saved_train", 32768, 4096),
        _saved("act8_saved_odd", 2047, 7168),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    kind = rng.choice(("fp4_round", "fp4_experts", "fp4_experts", "act8_swiglu", "act8_saved"))
    if kind == "act8_swiglu":
        return dict(kind=kind, rows=_log(rng, 1, 32768), f=_log(rng, 64, 14336, 8))
    if kind == "act8_saved":
        return dict(kind=kind, rows=_log(rng, 1, 32768), d=_log(rng, 64, 7168, 8))
    fmt = rng.choice(("mx", "nv"))
    E = rng.choice((4, 8, 16, 32, 64))
    k = rng.choice([v for v in (1, 2, 4, 8) if v <= E // 2])
    d = _log(rng, 128, 7168, 32)
    if kind == "fp4_round":
        return dict(kind=kind, fmt=fmt, T=_log(rng, 1, 32768 // k), d=d, E=E, k=k)
    f = _log(rng, 128, min(14336, 500_000_000 // (E * d)), 32)
    most = max(1, min(32768, int(1.1e13 / (6.0 * d * f))))  # rows of the largest listed case's work
    return dict(kind=kind, fmt=fmt, T=_log(rng, 1, max(1, most // k)), d=d, f=f, E=E, k=k)


# --------------------------------------------------- 4-bit and 8-bit formats
def _e2m1_code(v):
    """Codes of v (fp32), round to nearest, ties to the even code, saturated: 3 bits and a sign."""
    a = v.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
         + (a >= 3.5) + (a > 5.0))
    return c + 8 * (v < 0).to(torch.uint8)


def _quantize4(x, fmt, g):
    """Codes [.., cols], scale codes uint8 [.., cols / block] and block scales (fp32, without g)
    of x (fp32); g: fp32 scalar tensor (nv)."""
    blk = 16 if fmt == "nv" else 32
    b = x.unflatten(-1, (-1, blk))
    a = b.abs().amax(-1)
    if fmt == "nv":
        code = (a / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
        scale = code.float()
        code = code.view(torch.uint8)
        t = scale * g
    else:
        e = torch.where(a > 0, torch.frexp(a).exponent - 3, torch.full_like(a, -127).int())
        e = e.clamp(-127, 127)
        code = (e + 127).to(torch.uint8)
        t = scale = _scale_value(code, fmt)
    q = torch.where(t.unsqueeze(-1) > 0, b / t.unsqueeze(-1), torch.zeros_like(b))
    return _e2m1_code(q).flatten(-2), code, scale


def _scale_value(code, fmt):
    if fmt == "nv":
        return code.view(torch.float8_e4m3fn).float()
    bits = code.int()  # 2^(code - 127) from its bits: exact, where a power function need not be
    return torch.where(bits > 0, bits << 23, torch.full_like(bits, 1 << 22)).view(torch.float32)


def _value4(device):
    t = torch.tensor(E2M1, device=device)
    return torch.cat((t, -t))


def _dequantize4(codes, scale):
    """codes uint8 [.., cols] times scale fp32 [.., cols / block], in fp32."""
    v = torch.index_select(_value4(codes.device), 0, codes.flatten().int()).view(codes.shape)
    return (v.unflatten(-1, (scale.shape[-1], -1)) * scale.unsqueeze(-1)).flatten(-2)


def _dequantize_packed(q, scode, fmt):
    """Packed codes uint8 [.., cols / 2] (low nibble first) and scale codes, in fp32."""
    v = _value4(q.device)
    both = torch.stack((v.repeat(16), v.repeat_interleave(16)), 1)  # byte -> its two values
    w = torch.index_select(both, 0, q.flatten().int()).view(*q.shape[:-1], 2 * q.shape[-1])
    s = _scale_value(scode, fmt)
    return w.unflatten(-1, (s.shape[-1], -1)).mul_(s.unsqueeze(-1)).flatten(-2)


def _round8(x):
    """x (fp32 [rows, cols]) through 8-bit codes, one bf16 scale per 32 columns."""
    cols = x.shape[-1]
    p = torch.nn.functional.pad(x, (0, -cols % 32)).unflatten(-1, (-1, 32))
    a = p.abs().amax(-1, keepdim=True)
    s = (((a / 127.0).view(torch.int32) + 0xFFFF) & -65536).view(torch.float32)  # bf16, rounded up
    s = torch.where(a >= 2.0 ** -100, s, torch.zeros_like(s))
    q = torch.where(s > 0, torch.round(p / s), torch.zeros_like(p))
    return (q * s).flatten(-2)[..., :cols]


# ------------------------------------------------------------------ inputs
def _rng(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _routing(T, E, k, gen):
    """Top-k routing of T tokens as the layer's permute leaves it: group offsets [E + 1] and the
    flat assignment (token * k + slot) of each permuted row."""
    idx = torch.rand(T, E, generator=gen, device=DEV).topk(k, dim=1).indices
    flat = idx.flatten()
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return offsets, order.to(torch.int32)


def _activations(rows, cols, gen):
    """bf16 hidden states: unit normal, a few channels several times larger."""
    big = 1.0 + 5.0 * (torch.rand(cols, generator=gen, device=DEV) > 0.99)
    return (torch.randn(rows, cols, generator=gen, device=DEV) * big).bfloat16()


def _scale8(amax):
    if amax is None:
        return torch.ones(1, device=DEV)
    return (amax / (6.0 * 448.0)).bfloat16().float()


def _weights(E, N, K, fmt, gen):
    """A 4-bit checkpoint's weight [E, N, K], K the contraction: packed codes, scale codes in row
    order and each expert's fp32 scale."""
    q = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
    s = torch.empty(E, N, K // (16 if fmt == "nv" else 32), dtype=torch.uint8, device=DEV)
    g = torch.ones(E, device=DEV)
    for e in range(E):
        w = 0.02 * torch.randn(N, K, generator=gen, device=DEV)
        if fmt == "nv":
            g[e] = w.abs().amax() / (6.0 * 448.0)
        c, s[e], _ = _quantize4(w, fmt, g[e])
        q[e] = c[:, ::2] | (c[:, 1::2] << 4)
    return q, s, g


def prepare(case, seed):
    gen = _rng(seed)
    kind = case["kind"]
    st = dict(case=case)
    if kind in ("act8_swiglu", "act8_saved"):
        rows = case["rows"]
        # the layer's buffers hold rows_cap rows, of which group_offsets[E] are live
        st["offsets"] = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device=DEV)
        cols = 2 * case["f"] if kind == "act8_swiglu" else case["d"]
        st["x"] = _activations(rows, cols, gen)
        st["q"] = torch.empty(rows, cols, dtype=torch.int8, device=DEV)
        st["s"] = torch.empty(rows, -(-cols // 32) if kind == "act8_saved"
                              else 2 * -(-case["f"] // 32), dtype=torch.bfloat16, device=DEV)
        if kind == "act8_swiglu":
            st["dact"] = (0.1 * torch.randn(rows, case["f"], generator=gen, device=DEV)).bfloat16()
            st["act"], st["act2"] = torch.empty_like(st["dact"]), torch.empty_like(st["dact"])
            st["dh"] = torch.empty_like(st["x"])
        else:
            st["out"] = torch.empty_like(st["x"])
        return st
    T, d, E, k, fmt = (case[n] for n in ("T", "d", "E", "k", "fmt"))
    R = T * k
    st["x"] = _activations(T, d, gen)
    st["offsets"], st["s2f"] = _routing(T, E, k, gen)
    # calibrated scales of the activations (nv), kept in 8 significant bits: with more, a ratio
    # that is a tie up to the scale's own rounding falls one way in 32 bits, the other in 64
    st["g"] = _scale8(st["x"].float().abs().amax().reshape(1) if fmt == "nv" else None)
    if kind == "fp4_round":
        st["out"] = torch.empty(R, d, dtype=torch.bfloat16, device=DEV)
        if own:
            from mixture_experts_grouped_router_gb300 import lowbit
            st["codes"] = lowbit.Fp4Rows(R, d, E, fmt, device=DEV)
        return st
    f = case["f"]
    st["g_act"] = _scale8(torch.full((1,), 32.0, device=DEV) if fmt == "nv" else None)
    st["wi"] = _weights(E, 2 * f, d, fmt, gen)   # [gate rows | up rows]
    st["wo"] = _weights(E, d, f, fmt, gen)
    if own:
        from mixture_experts_grouped_router_gb300 import lowbit
        st["experts"] = lowbit.Fp4Experts.from_codes(fmt, *st["wi"], *st["wo"], x_scale=st["g"],
                                                     act_scale=st["g_act"])
        st["bufs"] = lowbit.Fp4Buffers(st["experts"], R)
        return st
    # the plain form multiplies the experts that have rows, each group padded to the longest one
    off = st["offsets"].cpu().long()
    sizes = off[1:] - off[:-1]
    live = torch.nonzero(sizes).flatten()
    most = int(sizes.max())
    at = torch.arange(most).unsqueeze(0)
    pad = torch.where(at < sizes[live].unsqueeze(1), off[:-1][live].unsqueeze(1) + at, R)
    st["live"], st["pad"] = live.to(DEV), pad.to(DEV)
    return st


# -------------------------------------------------------------------- runs
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    from mixture_experts_grouped_router_gb300 import lowbit
    case = st["case"]
    kind = case["kind"]
    if kind == "fp4_round":
        c = st["codes"]
        lowbit.fp4_quantize(st["x"], c, st["offsets"], row_index=st["s2f"], index_div=case["k"],
                            scale=st["g"])
        lowbit.fp4_dequantize(c, st["offsets"], st["out"], scale=st["g"])
        return st["out"]
    if kind == "fp4_experts":
        return lowbit.fp4_experts(st["experts"], st["bufs"], st["x"], st["s2f"], case["k"],
                                  st["offsets"])
    if kind == "act8_swiglu":
        lowbit.act8_swiglu_fwd(st["x"], st["act"], st["q"], st["s"], st["offsets"])
        lowbit.act8_swiglu_bwd(st["q"], st["s"], st["dact"], st["dh"], st["act2"], st["offsets"])
        return dict(act=st["act"], dh=st["dh"], act_again=st["act2"])
    lowbit.act8_quantize(st["x"], st["q"], st["s"], st["offsets"])
    lowbit.act8_dequantize(st["q"], st["s"], st["out"], st["offsets"])
    return st["out"]


def _run_plain(st):
    case = st["case"]
    kind = case["kind"]
    if kind == "act8_saved":
        return _round8(st["x"].float()).bfloat16()
    if kind == "act8_swiglu":
        h = st["x"].float()
        g, u = h.chunk(2, dim=1)
        act = g / (1.0 + torch.exp(-g)) * u
        g, u = _round8(g), _round8(u)
        sig = 1.0 / (1.0 + torch.exp(-g))
        da = st["dact"].float()
        dh = torch.cat((da * u * sig * (1.0 + g * (1.0 - sig)), da * g * sig), 1)
        return dict(act=act.bfloat16(), dh=dh.bfloat16(), act_again=(g * sig * u).bfloat16())
    fmt = case["fmt"]
    rows = torch.div(st["s2f"], case["k"], rounding_mode="floor").long()
    codes, _, scale = _quantize4(st["x"].float(), fmt, st["g"])
    x = _dequantize4(codes, scale)
    if kind == "fp4_round":
        return (x * st["g"]).bfloat16()[rows]
    live, pad = st["live"], st["pad"]
    xs = torch.cat((x[rows], x.new_zeros(1, x.shape[1])))[pad]          # [live, most, d]
    wi = _dequantize_packed(st["wi"][0][live], st["wi"][1][live], fmt)  # [live, 2f, d]
    h = torch.bmm(xs, wi.transpose(1, 2)) * (st["g"] * st["wi"][2][live]).view(-1, 1, 1)
    del wi
    g, u = h.chunk(2, dim=2)
    codes, _, scale = _quantize4(g / (1.0 + torch.exp(-g)) * u, fmt, st["g_act"])
    wo = _dequantize_packed(st["wo"][0][live], st["wo"][1][live], fmt)  # [live, d, f]
    y = torch.bmm(_dequantize4(codes, scale), wo.transpose(1, 2))
    y = y * (st["g_act"] * st["wo"][2][live]).view(-1, 1, 1)
    out = y.new_zeros(rows.numel() + 1, y.shape[2])
    out[pad.flatten()] = y.flatten(0, 1)
    return out[:-1].bfloat16()


# -------------------------------------------------------------------- work
def work(case):
    kind = case["kind"]
    if kind == "act8_saved":  # bf16 read, codes written and read, bf16 written
        n = case["rows"] * case["d"]
        return dict(bytes=n * (2 + 2 * (1 + 2 / 32) + 2), flops=4.0 * n)
    if kind == "act8_swiglu":  # forward: h read, act and codes written; backward reads codes, dact
        n = case["rows"] * case["f"]
        return dict(bytes=n * (4 + 2 + 4 * (1 + 2 / 32) + 2 + 4 + 2), flops=40.0 * n)
    bits = 0.5 + (1 / 16 if case["fmt"] == "nv" else 1 / 32)
    T, d, k, E = case["T"], case["d"], case["k"], case["E"]
    R = T * k
    if kind == "fp4_round":
        return dict(bytes=T * d * 2 + R * d * (2 * bits + 2) + 4 * R, flops=4.0 * R * d)
    f = case["f"]
    live = E * (1.0 - (1.0 - k / E) ** T)  # experts that meet a token, on average
    weights = live * 3 * d * f * bits
    return dict(bytes=weights + T * d * 2 + R * d * 2 + 4 * R, flops=6.0 * R * d * f)


# ------------------------------------------------------------------- exact
def _pow2(e):
    """2^e of whole numbers e (float64), exact."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _floor_log2(v):
    return torch.frexp(v).exponent.double() - 1


def _exact4(x, fmt, g):
    """Values of x (float64 [rows, cols]) in 4-bit blocks, by the formats' definition."""
    blk = 16 if fmt == "nv" else 32
    b = x.reshape(x.shape[0], -1, blk)
    a = b.abs().amax(-1, keepdim=True)
    if fmt == "nv":
        # E4M3: 3 bits after the leading one, exponents from -6 on, at most 448
        r = (a / (6.0 * g)).clamp(max=448.0)
        step = _pow2(_floor_log2(r.clamp(min=2.0 ** -6)) - 3)
        t = torch.round(r / step) * step * g
    else:
        t = _pow2((_floor_log2(a.clamp(min=2.0 ** -140)) - 2).clamp(-127, 127))
    r = (b / torch.where(t > 0, t, torch.ones_like(t))).abs().clamp(max=6.0)
    step = _pow2(_floor_log2(r.clamp(min=1.0)) - 1)  # E2M1: one bit after it
    v = torch.round(r / step) * step * torch.sign(b) * t
    return v.reshape(x.shape)


def _exact8(x):
    cols = x.shape[1]
    b = torch.nn.functional.pad(x, (0, -cols % 32)).reshape(x.shape[0], -1, 32)
    a = b.abs().amax(-1, keepdim=True)
    r = a / 127.0
    step = _pow2(_floor_log2(r.clamp(min=2.0 ** -120)) - 7)  # bf16: 7 bits
    s = torch.ceil(r / step) * step * (a >= 2.0 ** -100)
    v = torch.round(b / torch.where(s > 0, s, torch.ones_like(s))) * s
    return v.reshape(x.shape[0], -1)[:, :cols]


def _exact_weight(w, e, fmt):
    q, s, g = w
    byte = q[e].long()
    c = torch.stack((byte & 15, byte >> 4), -1).flatten(-2)
    m = torch.tensor(E2M1, dtype=torch.float64, device=q.device)[c & 7]
    v = torch.where(c >= 8, -m, m)
    sc = s[e].long()
    if fmt == "nv":
        ex, man = (sc >> 3) & 15, (sc & 7).double()
        t = torch.where(ex > 0, (1 + man / 8) * _pow2(ex - 7), man / 8 * 2.0 ** -6)
        t = t * g[e].double()
    else:
        t = _pow2(sc - 127)
    return v * t.repeat_interleave(v.shape[1] // t.shape[1], dim=1)


def exact(case, seed):
    kind = case["kind"]
    flops = work(case)["flops"]
    if kind == "fp4_experts" and flops > 6e12:
        return None  # the products in 64 bits would take too long
    st = prepare(case, seed)
    if kind in ("act8_saved", "act8_swiglu"):
        out = []
        for x, da in zip(st["x"].split(4096), (st["dact"] if "dact" in st else st["x"]).split(4096)):
            x, da = x.double(), da.double()
            if kind == "act8_saved":
                out.append((_exact8(x).float(),))
                continue
            g, u = x[:, :case["f"]], x[:, case["f"]:]
            act = g * torch.sigmoid(g) * u
            g, u = _exact8(g), _exact8(u)
            p = torch.sigmoid(g)
            dg, du = da * u * (p + g * p * (1 - p)), da * g * p
            out.append((act.float(), torch.cat((dg, du), 1).float(), (g * p * u).float()))
        out = [torch.cat(t).double() if st["x"].numel() < 2 ** 26 else torch.cat(t)
               for t in zip(*out)]
        return out[0] if kind == "act8_saved" else dict(act=out[0], dh=out[1], act_again=out[2])
    fmt, k = case["fmt"], case["k"]
    g = st["g"].double()
    rows = st["s2f"].long() // k
    x = torch.cat([_exact4(t.double(), fmt, g) for t in st["x"].split(4096)])
    if kind == "fp4_round":
        return x.float()[rows]
    off = st["offsets"].tolist()
    y = torch.zeros(rows.numel(), case["d"], dtype=torch.float64, device=DEV)
    for e in range(case["E"]):
        if off[e] == off[e + 1]:
            continue
        h = x[rows[off[e]:off[e + 1]]] @ _exact_weight(st["wi"], e, fmt).T
        a = h[:, :case["f"]] * torch.sigmoid(h[:, :case["f"]]) * h[:, case["f"]:]
        a = _exact4(a, fmt, st["g_act"].double())
        y[off[e]:off[e + 1]] = a @ _exact_weight(st["wo"], e, fmt).T
    return y
