"""Timed cases of what a training or serving step has around the expert layer: the RMS norm with the
residual's addition and 8-bit outputs, the balance loss of every sequence with the router's z loss,
and the clipping of all gradients by their global norm.

Each case is one call sequence of a program.  With ``own`` false the operators are computed in
elementary torch operations; with it true through this package.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------- cases
def _norm(name, T, d, stream, codes, train):
    """stream: type of the residual stream; codes: format of the 8-bit output ("mx", "act8") or
    "none" (y in bf16); train: y in bf16 too, and the backward pass."""
    return dict(name=name, kind="norm", T=T, d=d, stream=stream, codes=codes, train=train)


def _balance(name, T, E, k, B, sigmoid, masked, split):
    """B ragged sequences; masked: some tokens of each count for nothing; split: the gradient by a
    backward call of its own, else in the same call as the loss."""
    return dict(name=name, kind="balance", T=T, E=E, k=k, B=B, sigmoid=sigmoid, masked=masked,
                split=split)


def _clip(name, d, f, E, extra, out, scale):
    """Gradients of a layer (d, f, E), its router and norm, and `extra` odd-sized vectors; out:
    type that the clipped weight gradients are written in; scale: 1 / loss scale."""
    return dict(name=name, kind="clip", d=d, f=f, E=E, extra=extra, out=out, scale=scale)


def listed():
    return [
        # one decoded token before the DeepSeek-like experts, block-scaled codes: latency
        _norm("norm_token_mx", 1, 7168, "bf16", "mx", False),
        # a small decoding batch on an fp32 residual stream
        _norm("norm_decode_fp32", 77, 7168, "fp32", "none", False),
        # a prompt batch before the Mixtral-like experts, block-scaled codes in the place of bf16
        _norm("norm_prompt_mx", 16384, 4096, "bf16", "mx", False),
        # a training step's norm at that size, forward and backward
        _norm("norm_train", 16384, 4096, "bf16", "none", True),
        # an odd number of tokens on an fp32 stream, the output saved in 8 bits too
        _norm("norm_train_act8_odd", 2047, 7168, "fp32", "act8", True),
        # the tiny layer's router: latency
        _balance("balance_tiny", 256, 8, 2, 1, False, False, False),
        # the DeepSeek-like router's batch: two sequences and padding
        _balance("balance_sigmoid", 8192, 32, 8, 2, True, True, False),
        # packed documents over many experts, loss and gradient by themselves
        _balance("balance_packed", 65521, 256, 8, 37, True, True, True),
        # a long batch of packed documents, softmax scores
        _balance("balance_long", 131072, 64, 1, 500, False, False, False),
        # the tiny layer's gradients and some vectors: latency
        _clip("clip_tiny", 128, 256, 8, 5, "bf16", 1.0),
        # the DeepSeek-like layer's gradients with a loss scale, into the optimiser's fp32
        _clip("clip_dsv3_fp32", 7168, 2048, 8, 41, "fp32", 2.0 ** -10),
        # the Mixtral-like layer's gradients
        _clip("clip_mixtral", 4096, 14336, 8, 0, "bf16", 1.0),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    kind = rng.choice(("norm", "norm", "balance", "balance", "clip"))
    if kind == "norm":
        codes = rng.choice(("none", "mx", "act8"))
        d = _log(rng, 128, 16384, 128 if codes == "mx" else 8)
        T = _log(rng, 1, min(32768, 16384 * 4096 // d))
        return dict(kind=kind, T=T, d=d, stream=rng.choice(("bf16", "fp32")), codes=codes,
                    train=rng.random() < 0.5)
    if kind == "balance":
        E = rng.choice((8, 16, 32, 60, 64, 128, 160, 256))
        k = rng.choice([v for v in (1, 2, 4, 6, 8) if v <= E // 2])
        T = _log(rng, 1, min(131072, 65521 * 256 // E))
        return dict(kind=kind, T=T, E=E, k=k, B=_log(rng, 1, 500), sigmoid=rng.random() < 0.5,
                    masked=rng.random() < 0.5, split=rng.random() < 0.5)
    d, f = _log(rng, 64, 7168, 8), _log(rng, 64, 14336, 8)
    E = max(1, min(_log(rng, 1, 64), 400_000_000 // (3 * d * f)))
    return dict(kind=kind, d=d, f=f, E=E, extra=rng.randrange(0, 50),
                out=rng.choice(("bf16", "fp32")), scale=rng.choice((1.0, 2.0 ** -10)))


# ------------------------------------------------------------------ inputs
def _type(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _prepare_norm(case, gen, st):
    T, d, stream = case["T"], case["d"], _type(case["stream"])

    def rnd(*s):
        return torch.randn(*s, generator=gen, device=DEV)

    big = 1.0 + 5.0 * (torch.rand(d, generator=gen, device=DEV) > 0.99)  # a few larger channels
    st["x"] = (rnd(T, d) * big).bfloat16()
    st["residual"] = (2.0 * rnd(T, d) * big).to(stream)
    st["w"] = 1.0 + 0.1 * rnd(d)
    st["h"] = torch.empty(T, d, dtype=stream, device=DEV)
    st["y"] = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    if case["codes"] != "none":
        st["restored"] = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    if case["train"]:
        st["dy"] = (0.1 * rnd(T, d)).bfloat16()
        st["d_res"] = (0.1 * rnd(T, d)).to(stream)  # from the layers above, past the block
        st["dh"] = torch.empty(T, d, dtype=stream, device=DEV)
        st["dw"] = torch.empty(d, device=DEV)
    if own:
        from mixture_experts_grouped_router_gb300 import block
        if case["codes"] != "none":
            st["codes"] = block.Codes8(T, d, case["codes"], device=DEV)
        if case["train"]:
            st["ws"] = block.rms_norm_bwd_workspace(T, d, device=DEV)


def _prepare_balance(case, gen, st):
    T, E, k, B = (case[n] for n in ("T", "E", "k", "B"))
    # some experts are liked more than others
    st["logits"] = (torch.randn(T, E, generator=gen, device=DEV)
                    + 0.5 * torch.randn(E, generator=gen, device=DEV))
    st["idx"] = st["logits"].topk(k, dim=1).indices.to(torch.int32)
    # lengths as of documents (some empty), a tail that belongs to none where there is a mask
    cut = torch.rand(B - 1, generator=gen, device=DEV).sort().values
    used = T - T // 16 if case["masked"] else T
    off = torch.cat((torch.zeros(1, device=DEV), (cut * used).floor(),
                     torch.full((1,), float(used), device=DEV)))
    st["offsets"] = off.to(torch.int32)
    st["mask"] = (torch.rand(T, generator=gen, device=DEV) > 0.1) if case["masked"] else None
    st["d_logits"] = torch.empty(T, E, device=DEV)
    if own:
        from mixture_experts_grouped_router_gb300 import _lib, block
        st["loss"] = block.SeqAuxLoss(
            T, E, k, B, score_fn=_lib.SCORE_SIGMOID if case["sigmoid"] else _lib.SCORE_SOFTMAX,
            coeff=COEFF, z_coeff=Z_COEFF, device=DEV)


COEFF, Z_COEFF = 1e-2, 1e-3


def _sizes(case):
    """(elements, type) of each gradient: the experts' weights, the router's, the norm's weight, and
    vectors of odd sizes."""
    d, f, E = case["d"], case["f"], case["E"]
    odd = [(1 + (7919 * (i + 1) ** 2) % 20011, ("bf16", "fp32")[i % 2]) for i in range(case["extra"])]
    return [(E * d * 2 * f, "bf16"), (E * f * d, "bf16"), (d * E, "fp32"), (d, "fp32"), *odd]


def _prepare_clip(case, gen, st):
    def grad(n, t):
        g = torch.empty(n, dtype=_type(t), device=DEV)
        for lo in range(0, n, 1 << 28):  # the noise in pieces: it is fp32 first
            hi = min(n, lo + (1 << 28))
            g[lo:hi] = (0.01 / case["scale"]) * torch.randn(hi - lo, generator=gen, device=DEV)
        return g

    sizes = _sizes(case)
    st["grads"] = [grad(n, t) for n, t in sizes]
    st["outs"] = [torch.empty(n, dtype=_type("fp32" if "fp32" in (t, case["out"]) else t), device=DEV)
                  for n, t in sizes]
    st["norm"] = torch.empty(1, device=DEV)
    # a good third of what the norm will be about: the gradients are clipped
    st["max_norm"] = 0.37 * 0.01 * math.sqrt(sum(n for n, _ in sizes))
    if own:
        from mixture_experts_grouped_router_gb300 import block
        st["clip"] = block.GradClip(st["grads"], st["outs"])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = dict(case=case)
    {"norm": _prepare_norm, "balance": _prepare_balance, "clip": _prepare_clip}[case["kind"]](
        case, gen, st)
    return st


# -------------------------------------------------------------------- runs
def run(st):
    kind = st["case"]["kind"]
    if own:
        return {"norm": _own_norm, "balance": _own_balance, "clip": _own_clip}[kind](st)
    return {"norm": _plain_norm, "balance": _plain_balance, "clip": _plain_clip}[kind](st)


def _own_norm(st):
    from mixture_experts_grouped_router_gb300 import block
    case = st["case"]
    codes, train = st.get("codes"), case["train"]
    y = st["y"] if train or codes is None else None
    block.rms_norm(st["x"], st["w"], EPS, y, residual=st["residual"], h=st["h"], codes=codes)
    out = dict(h=st["h"])
    if y is not None:
        out["y"] = y
    if codes is not None:
        out["restored"] = codes.dequantize(st["restored"])
    if train:
        block.rms_norm_bwd(st["dy"], st["h"], st["w"], EPS, st["dh"], st["dw"], st["ws"],
                           d_residual=st["d_res"])
        out.update(dh=st["dh"], dw=st["dw"])
    return out


def _own_balance(st):
    loss, split = st["loss"], st["case"]["split"]
    loss.forward(st["logits"], st["idx"], st["offsets"], token_mask=st["mask"],
                 d_logits=None if split else st["d_logits"])
    if split:
        loss.backward(st["logits"], st["offsets"], st["d_logits"], token_mask=st["mask"],
                      accumulate=False)
    return dict(loss=loss.loss, counts=loss.counts, tokens=loss.tokens, probs=loss.probs,
                d_logits=st["d_logits"])


def _own_clip(st):
    norm = st["clip"].clip(st["max_norm"], scale=st["case"]["scale"])
    return dict(norm=norm, outs=st["outs"])


def _plain_norm(st):
    case = st["case"]
    h = (st["x"].float() + st["residual"].float()).to(st["h"].dtype)
    hf = h.float()
    r = 1.0 / torch.sqrt((hf * hf).mean(1, keepdim=True) + EPS)
    y = (hf * r * st["w"]).bfloat16()
    out = dict(h=h)
    if case["train"] or case["codes"] == "none":
        out["y"] = y
    if case["codes"] == "mx":
        out["restored"] = _through_mx(y.float()).bfloat16()
    elif case["codes"] == "act8":
        out["restored"] = _through_act8(y.float()).bfloat16()
    if case["train"]:
        dy = st["dy"].float()
        n = hf * r
        g = dy * st["w"]
        dh = r * (g - n * (g * n).mean(1, keepdim=True)) + st["d_res"].float()
        out.update(dh=dh.to(h.dtype), dw=(dy * n).sum(0))
    return out


def _through_mx(x):
    """x through E4M3 codes with one power of two for 32 columns."""
    b = x.unflatten(-1, (-1, 32))
    a = b.abs().amax(-1, keepdim=True)
    e = torch.where(a > 0, torch.frexp(a).exponent - 9, torch.full_like(a, -127).int())
    e = e.clamp(-126, 127)  # (values under 2^-120 are none of the path's)
    s = ((e + 127) << 23).view(torch.float32)
    q = (b / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    return (q * s).flatten(-2)


def _through_act8(x):
    """x through signed 8-bit codes with one bf16 scale for 32 columns."""
    cols = x.shape[-1]
    p = torch.nn.functional.pad(x, (0, -cols % 32)).unflatten(-1, (-1, 32))
    a = p.abs().amax(-1, keepdim=True)
    s = (((a / 127.0).view(torch.int32) + 0xFFFF) & -65536).view(torch.float32)  # bf16, rounded up
    q = torch.where(s > 0, torch.round(p / s), torch.zeros_like(p))
    return (q * s).flatten(-2)[..., :cols]


def _plain_balance(st):
    case = st["case"]
    T, E, k, B = (case[n] for n in ("T", "E", "k", "B"))
    logits, off = st["logits"], st["offsets"]
    at = torch.arange(T, dtype=torch.int32, device=DEV)
    seq = (at.unsqueeze(1) >= off[1:]).sum(1)  # B: of no sequence
    live = seq < B
    if st["mask"] is not None:
        live = live & st["mask"]
    seq = torch.where(live, seq, torch.full_like(seq, B))  # a bin of its own for the others
    tokens = torch.zeros(B + 1, dtype=torch.int32, device=DEV).index_add_(
        0, seq, torch.ones_like(at))
    cell = (seq.unsqueeze(1) * E + st["idx"]).flatten()
    counts = torch.zeros((B + 1) * E, dtype=torch.int32, device=DEV).index_add_(
        0, cell, torch.ones_like(cell, dtype=torch.int32)).view(B + 1, E)
    m = logits.amax(1, keepdim=True)
    ex = torch.exp(logits - m)
    total = ex.sum(1, keepdim=True)
    soft, lse = ex / total, m + torch.log(total)
    if case["sigmoid"]:
        s = 1.0 / (1.0 + torch.exp(-logits))
        size = s.sum(1, keepdim=True)
        p, jac = s / size, s * (1.0 - s) / size
    else:
        p = jac = soft
    n = tokens.clamp(min=1).float().unsqueeze(1)
    probs = torch.zeros(B + 1, E, dtype=torch.float64, device=DEV).index_add_(0, seq, p.double())
    probs = (probs / n).float()
    f = counts * (E / k) / n
    sequences = (tokens[:B] > 0).sum().clamp(min=1).float()
    count = tokens[:B].sum().clamp(min=1).float()
    loss = torch.stack((COEFF / sequences * (f * probs)[:B].sum(),
                        Z_COEFF / count * torch.where(live, lse.squeeze(1) ** 2, 0.0).sum()))
    ft = f[seq]
    c = (ft * p).sum(1, keepdim=True)
    g = COEFF / (sequences * n[seq]) * jac * (ft - c) + Z_COEFF * 2.0 / count * lse * soft
    return dict(loss=loss, counts=counts[:B], tokens=tokens[:B], probs=probs[:B],
                d_logits=torch.where(live.unsqueeze(1), g, 0.0))


def _plain_clip(st):
    scale = st["case"]["scale"]
    squares = torch.stack([(g.float() ** 2).sum(dtype=torch.float64) for g in st["grads"]])
    norm = (scale * torch.sqrt(squares.sum())).float().reshape(1)
    c = scale * (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    return dict(norm=norm, outs=[(g.float() * c).to(o.dtype) for g, o in zip(st["grads"], st["outs"])])


# -------------------------------------------------------------------- work
def work(case):
    if case["kind"] == "norm":
        n, wide = case["T"] * case["d"], 4 if case["stream"] == "fp32" else 2
        code = {"none": 0.0, "mx": 1 + 1 / 32, "act8": 1 + 2 / 32}[case["codes"]]
        b = 2 + 2 * wide + (2 if case["train"] or not code else 0)  # x, residual, h, y
        b += 2 * code + (2 if code else 0)                          # codes written, read; restored
        b += 2 + 3 * wide if case["train"] else 0                   # dy, h, d_res, dh
        return dict(bytes=n * b + 8.0 * case["d"], flops=n * (30.0 if case["train"] else 10.0))
    if case["kind"] == "balance":
        T, E = case["T"], case["E"]
        b = T * (4.0 * E * (3 if case["split"] else 2) + 4 * case["k"] + (1 if case["masked"] else 0))
        return dict(bytes=b + 8.0 * case["B"] * E, flops=25.0 * T * E)
    b = n = 0
    for m, t in _sizes(case):
        wide = 4 if "fp32" in (t, case["out"]) else 2
        b, n = b + m * ((4 if t == "fp32" else 2) + wide), n + m
    return dict(bytes=float(b), flops=3.0 * n)


# ------------------------------------------------------------------- exact
def _pow2(e):
    """2^e of whole numbers e (float64), exact."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _floor_log2(v):
    return torch.frexp(v).exponent.double() - 1


def _exact_codes(y, fmt):
    """Values of y (float64) in blocks of 32 columns, by the formats' definition."""
    cols = y.shape[1]
    b = torch.nn.functional.pad(y, (0, -cols % 32)).reshape(y.shape[0], -1, 32)
    a = b.abs().amax(-1, keepdim=True)
    if fmt == "mx":  # E4M3: 3 bits after the leading one, exponents from -6 on, at most 448
        s = _pow2((_floor_log2(a.clamp(min=2.0 ** -115)) - 8).clamp(min=-127))
        r = (b / s).abs().clamp(max=448.0)
        step = _pow2(_floor_log2(r.clamp(min=2.0 ** -6)) - 3)
        v = (torch.round(r / step) * step).clamp(max=448.0) * torch.sign(b) * s
    else:
        r = a / 127.0
        step = _pow2(_floor_log2(r.clamp(min=2.0 ** -110)) - 7)  # bf16: 7 bits
        s = torch.ceil(r / step) * step
        v = torch.round(b / torch.where(s > 0, s, torch.ones_like(s))) * s
    return v.reshape(y.shape[0], -1)[:, :cols]


def _exact_norm(case, st):
    parts, w = [], st["w"].double()
    dw = torch.zeros_like(w)
    for lo in range(0, case["T"], 2048):
        rows = slice(lo, lo + 2048)
        h = (st["x"][rows].double() + st["residual"][rows].double()).to(st["h"].dtype).double()
        r = (h.square().mean(1, keepdim=True) + EPS).rsqrt()
        y = h * r * w
        p = dict(h=h)
        if case["train"] or case["codes"] == "none":
            p["y"] = y
        if case["codes"] != "none":  # the codes are those of y as it is kept, in bf16
            p["restored"] = _exact_codes(y.bfloat16().double(), case["codes"])
        if case["train"]:
            dy = st["dy"][rows].double()
            along = (dy * w * h).mean(1, keepdim=True)
            p["dh"] = r * dy * w - r ** 3 * along * h + st["d_res"][rows].double()
            dw += torch.einsum("td,td->d", dy, h * r)
        parts.append(p)
    out = {n: torch.cat([p[n] for p in parts]) for n in parts[0]}
    if case["train"]:
        out["dw"] = dw
    return out


def _exact_balance(case, st):
    T, E, k, B = (case[n] for n in ("T", "E", "k", "B"))
    off = st["offsets"].tolist()
    d_logits = torch.zeros(T, E, dtype=torch.float64, device=DEV)
    probs = torch.zeros(B, E, dtype=torch.float64, device=DEV)
    counts = torch.zeros(B, E, dtype=torch.int32, device=DEV)
    tokens = torch.zeros(B, dtype=torch.int32, device=DEV)
    rows = []
    for b in range(B):
        t = torch.arange(off[b], off[b + 1], device=DEV)
        rows.append(t if st["mask"] is None else t[st["mask"][t]])
    S = max(1, sum(r.numel() > 0 for r in rows))
    N = max(1, sum(r.numel() for r in rows))
    balance = z = torch.zeros((), dtype=torch.float64, device=DEV)
    for b, r in enumerate(rows):
        if not r.numel():
            continue
        x = st["logits"][r].double()
        lse = torch.logsumexp(x, 1, keepdim=True)
        soft = torch.exp(x - lse)
        p = jac = soft
        if case["sigmoid"]:
            s = torch.sigmoid(x)
            p, jac = s / s.sum(1, keepdim=True), s * torch.sigmoid(-x) / s.sum(1, keepdim=True)
        counts[b] = torch.bincount(st["idx"][r].flatten(), minlength=E)
        tokens[b] = r.numel()
        probs[b] = p.mean(0)
        f = counts[b].double() * E / (k * r.numel())
        balance = balance + COEFF / S * torch.dot(f, probs[b])
        z = z + Z_COEFF / N * lse.square().sum()
        d_logits[r] = (COEFF / (S * r.numel()) * jac * (f - (p @ f).unsqueeze(1))
                       + 2.0 * Z_COEFF / N * lse * soft)
    return dict(loss=torch.stack((balance, z)), counts=counts, tokens=tokens, probs=probs,
                d_logits=d_logits)


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "norm":
        return _exact_norm(case, st)
    if case["kind"] == "balance":
        return _exact_balance(case, st)
    total = torch.zeros((), dtype=torch.float64, device=DEV)
    for g in st["grads"]:
        for part in g.split(1 << 27):
            v = part.double()
            total = total + torch.dot(v, v)
    norm = case["scale"] * total.sqrt()
    c = case["scale"] * (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    return dict(norm=norm.reshape(1), outs=[g.double() * c for g in st["grads"]])
