"""The low-bit operators as a program uses them: the layer's backward from 8-bit
checkpoints, the 4-bit serving layer, and the example that runs both.

Tolerances.  A code is off by at most half a step s / 2 with s about max|block| /
127: uniform errors of max / (254 sqrt 3), max about 2.1 sigma for blocks of 32
normal values, so 0.5% of a saved tensor's norm.  A gradient is a product of a saved
tensor with exact operands, or an elementwise function with slope near 1 of two of
them: at most 2 x 0.5%, beside the layer's own 1e-2.  The checkpointed backward is
held to 2e-2 of the layer's (relative Frobenius)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import moe_synth
from gpu_helpers import dev_bf16, layer_shape, run_gpu_layer
from oracle import lowbit_ref as R
from oracle import moe_ref

pytestmark = pytest.mark.gpu

C = moe_synth.CONFIGS
CASES = {
    "tiny": C["tiny"],
    "dsv3": moe_synth.scaled(C["dsv3"], T=512, d=448, f=256),
    "skewed": moe_synth.scaled(C["skewed"], T=4096, d=256, f=128, capacity=64),
    "odd_sizes": moe_synth.MoEConfig("odd_sizes", T=999, d=200, f=136, E=7, k=3, score_fn=1,
                                     renorm=0, align=16, capacity=300),
}


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("biased", [False, True])
def test_backward_from_checkpoint(name, biased):
    from mixture_experts_grouped_router_gb300 import layer, lowbit
    cfg = CASES[name]
    inp = moe_synth.make_inputs(cfg, seed=3)
    biases = moe_synth.make_biases(cfg, seed=4) if biased else None
    aux = 1e-2 if biased else 0.0
    ref = run_gpu_layer(cfg, inp, biases=biases, aux_coeff=aux)
    want = {n: getattr(ref, n).clone() for n in ("dx", "dwi", "dwo", "d_topk_w", "d_logits") + (
        ("dbi", "dbo") if biased else ())}
    x, wi, wo, dout = (dev_bf16(inp[n]) for n in ("x", "wi", "wo", "dout"))
    logits = torch.from_numpy(inp["logits"]).cuda()
    b = layer.MoEBuffers(layer_shape(cfg, biased, aux_coeff=aux))
    bi, bo = (dev_bf16(biases["bi"]), dev_bf16(biases["bo"])) if biased else (None, None)
    ck = lowbit.Checkpoint8(b)
    layer.forward(b, x, logits, wi, wo, bi=bi, bo=bo)
    ck.save(b)
    # another layer's forward and backward overwrite the workspace
    layer.forward(b, -x, -logits, wi, wo, bi=bi, bo=bo)
    layer.backward(b, -dout, wi, wo)
    ck.backward(b, dout, wi, wo)
    assert int(b.dev_status.item()) == 0
    for n, w in want.items():
        got, w = f64(getattr(b, n)), f64(w)
        assert np.linalg.norm(got - w) <= 2e-2 * np.linalg.norm(w), n
    R_, d, f = b.rows_cap, cfg.d, cfg.f
    assert ck.nbytes() <= 0.54 * 2 * R_ * (2 * d + 2 * f) + 16 * R_ + 8 * cfg.T * cfg.k + 8192


def test_checkpoint_outlives_the_callers_logits():
    """Every layer's logits in one buffer of the caller: the saved layer's router-logit
    gradient is that of its own."""
    from mixture_experts_grouped_router_gb300 import layer, lowbit
    cfg = CASES["odd_sizes"]
    inp = moe_synth.make_inputs(cfg, seed=5)
    x, wi, wo, dout = (dev_bf16(inp[n]) for n in ("x", "wi", "wo", "dout"))
    logits = torch.from_numpy(inp["logits"]).cuda()
    b = layer.MoEBuffers(layer_shape(cfg, False))
    ck = lowbit.Checkpoint8(b)
    with pytest.raises(ValueError, match="before a forward"):
        ck.save(b)
    layer.forward(b, x, logits, wi, wo)
    ck.save(b)
    ck.backward(b, dout, wi, wo)
    want = b.d_logits.clone()
    logits.copy_(torch.randn_like(logits))
    layer.forward(b, x, logits, wi, wo)
    ck.backward(b, dout, wi, wo)
    assert torch.equal(b.d_logits, want)


def test_checkpoint_refusals():
    from mixture_experts_grouped_router_gb300 import layer, lowbit
    b = layer.MoEBuffers(layer.LayerShape(64, 128, 128, 4, 2, mxfp8=True))
    with pytest.raises(ValueError, match="bf16 layer"):
        lowbit.Checkpoint8(b)
    b = layer.MoEBuffers(layer.LayerShape(64, 128, 128, 4, 2))
    with pytest.raises(ValueError, match="before save"):
        lowbit.Checkpoint8(b).backward(b, None, None, None)
    w = lowbit.Fp4Experts.from_weights("mx", torch.zeros(4, 128, 256, device="cuda").bfloat16(),
                                       torch.zeros(4, 128, 128, device="cuda").bfloat16())
    with pytest.raises(ValueError, match="experts"):
        lowbit.Fp4Layer(w, layer.LayerShape(64, 128, 256, 4, 2))
    m = lowbit.Fp4Layer(w, layer.LayerShape(8, 128, 128, 4, 2))
    with pytest.raises(ValueError, match="at most 8"):
        m.forward(torch.zeros(9, 128, device="cuda").bfloat16(), torch.zeros(9, 4, device="cuda"))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T", [1, 7, 300])
@pytest.mark.parametrize("align,capacity", [(0, 0), (16, 40)])
def test_serving_layer(fmt, T, align, capacity):
    """Against the fp64 layer on the values of the 4-bit weights, tokens and Act."""
    from mixture_experts_grouped_router_gb300 import layer, lowbit
    cfg = moe_synth.MoEConfig("serve", T=T, d=160, f=224, E=5, k=2, align=align,
                              capacity=capacity)
    inp = moe_synth.make_inputs(cfg, seed=T)
    x, wi, wo = (moe_synth.bits_to_f64(inp[n]) for n in ("x", "wi", "wo"))
    gx, ga = (0.0078125, 0.0009765625) if fmt == "nv" else (1.0, 1.0)
    t = lambda v: torch.tensor([v], dtype=torch.float32, device="cuda")  # noqa: E731
    w = lowbit.Fp4Experts.from_weights(fmt, dev_bf16(inp["wi"]), dev_bf16(inp["wo"]), t(gx), t(ga))
    m = lowbit.Fp4Layer(w, layer.LayerShape(512, cfg.d, cfg.f, cfg.E, cfg.k, align=align,
                                            capacity=capacity))
    out = m.forward(dev_bf16(inp["x"]), torch.from_numpy(inp["logits"]).cuda())
    assert int(m.bufs.dev_status.item()) == 0
    gi = f64(w.wi_scale) if fmt == "nv" else np.ones(cfg.E)
    go = f64(w.wo_scale) if fmt == "nv" else np.ones(cfg.E)
    fw = moe_ref.forward(x, inp["logits"], wi, wo, cfg.k, 0, 1, align, capacity)
    lay = fw["layout"]
    off, s2f = lay["group_offsets"], np.asarray(lay["sorted_to_flat"])
    want = np.zeros((T, cfg.d))
    for e in range(cfg.E):
        for r in range(off[e], off[e + 1]):
            if s2f[r] < 0:
                continue
            xq = R.fp4_quantize(x[s2f[r] // cfg.k][None], fmt, gx)[2]
            a = R.swiglu(xq @ R.fp4_quantize(wi[e].T, fmt, gi[e])[2].T)
            y = R.fp4_quantize(a, fmt, ga)[2] @ R.fp4_quantize(wo[e].T, fmt, go[e])[2].T
            want[s2f[r] // cfg.k] += fw["topk_w"].reshape(-1)[s2f[r]] * y[0]
    got = f64(out)
    assert got.shape == want.shape
    assert np.linalg.norm(got - want) <= 1e-2 * np.linalg.norm(want)


@pytest.mark.parametrize("T", [1, 700])
def test_serving_and_checkpoint_kernels_in_a_graph(T):
    """Captured once and replayed on other inputs in the same buffers: bit for bit what the
    calls give (routing, quantisation with the linked gather at T = 700, both products)."""
    from mixture_experts_grouped_router_gb300 import layer, lowbit
    d, f, E, k = 6400, 128, 6, 4
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    t = lambda v: torch.tensor([v], dtype=torch.float32, device="cuda")  # noqa: E731
    w = lowbit.Fp4Experts.from_weights("nv", (rnd(E, d, 2 * f) / 80).bfloat16(),
                                       (rnd(E, f, d) / 11).bfloat16(), t(0.0078125), t(0.0078125))
    m = lowbit.Fp4Layer(w, layer.LayerShape(T, d, f, E, k))
    x, logits = rnd(T, d).bfloat16(), rnd(T, E)
    q = torch.empty(T, d, dtype=torch.int8, device="cuda")
    s = torch.empty(T, d // 32, dtype=torch.bfloat16, device="cuda")

    def work():
        lowbit.act8_quantize(x, q, s)
        return m.forward(x, logits)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        work()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = work()
    for _ in range(3):
        x.copy_(rnd(T, d))
        logits.copy_(rnd(T, E))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), q.clone(), s.clone()
        out.zero_()
        work()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, q, s)))
    assert int(m.bufs.dev_status.item()) == 0


def test_example_trains_and_serves():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    try:
        import lowbit_experts
        losses, served, one = lowbit_experts.main(["--steps", "8"])
    finally:
        sys.path.pop(0)
    assert all(np.isfinite(losses)) and losses[-1] < 0.9 * losses[0]
    # what was learned survives 4 bits; a token's row does not depend on the batch
    # around it beyond bf16 and tie flips
    assert served < 0.5 * losses[0] and one < 2e-2


def test_example_runs_as_a_command():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "lowbit_experts.py"),
                        "--steps", "2", "--layers", "1", "--fmt", "mx"], capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0 and "serving in 4 bits" in r.stdout, r.stdout + r.stderr
