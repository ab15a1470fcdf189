"""A stack of MoE layers trained with 8-bit saved activations, then served from
4-bit experts: `python examples/lowbit_experts.py [--layers 3] [--steps 20]`.

Training: the layers share one workspace.  After each layer's forward its saved
state leaves the workspace as 8-bit codes (Checkpoint8), and the backward reads the
codes.  The model learns to reproduce a fixed random target.  Serving: the trained
weights are quantised to 4 bits (NVFP4 or MXFP4), and the same prompt runs through
Fp4Layer, then its tokens one at a time, as a decoder would.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixture_experts_grouped_router_gb300 import layer, lowbit  # noqa: E402


def forward(bufs, x, gates, weights, checkpoints=None):
    """x + MoE(x) for every layer; the layers' states in `checkpoints`."""
    inputs = []
    for n, (gate, (wi, wo)) in enumerate(zip(gates, weights)):
        inputs.append(x)
        out = layer.forward(bufs, x, x.float() @ gate, wi, wo)
        if checkpoints is not None:
            checkpoints[n].save(bufs)
        x = x + out
    return x, inputs


def step(w, g, lr):
    """w moves by lr times its own size along the gradient."""
    g = g.float().view(w.shape)
    w -= (lr * w.float().norm() / g.norm().clamp(min=1e-30) * g).to(w.dtype)


def train_step(bufs, checkpoints, x, target, gates, weights, lr):
    y, inputs = forward(bufs, x, gates, weights, checkpoints)
    err = (y - target).float()
    dy = (2.0 / err.numel() * err).bfloat16() * 1024.0  # loss scale
    for n in reversed(range(len(weights))):
        wi, wo = weights[n]
        dx, dwi, dwo, _ = checkpoints[n].backward(bufs, dy, wi, wo)
        d_gate = inputs[n].float().t() @ bufs.d_logits
        dy = dy + dx + (bufs.d_logits @ gates[n].t()).bfloat16()
        for w, g in ((wi, dwi), (wo, dwo), (gates[n], d_gate)):
            step(w, g, lr)
    return float(err.square().mean())


def serve(x, gates, served):
    for gate, moe in zip(gates, served):
        x = x + moe.forward(x, x.float() @ gate)
    return x


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--layers", type=int, default=3)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--lr", type=float, default=0.02)
    ap.add_argument("--fmt", choices=("nv", "mx"), default="nv")
    a = ap.parse_args(argv)
    d, f, E, k = 256, 512, 8, 2
    torch.manual_seed(0)
    dev = "cuda"
    shape = layer.LayerShape(a.tokens, d, f, E, k)
    x = torch.randn(a.tokens, d, device=dev).bfloat16()
    target = torch.randn(a.tokens, d, device=dev).bfloat16()
    gates = [0.02 * torch.randn(d, E, device=dev) for _ in range(a.layers)]
    weights = [((torch.randn(E, d, 2 * f, device=dev) * d ** -0.5).bfloat16(),
                (torch.randn(E, f, d, device=dev) * f ** -0.5).bfloat16())
               for _ in range(a.layers)]
    bufs = layer.MoEBuffers(shape)
    checkpoints = [lowbit.Checkpoint8(bufs) for _ in range(a.layers)]
    saved = sum(t.numel() * t.element_size() for t in (bufs.xs, bufs.h, bufs.act, bufs.y))
    losses = [train_step(bufs, checkpoints, x, target, gates, weights, lr=a.lr)
              for _ in range(a.steps)]
    print("training: mean square error %.4f -> %.4f; %.2f MB saved a layer (bf16: %.2f MB)"
          % (losses[0], losses[-1], checkpoints[0].nbytes() / 1e6, saved / 1e6))
    want, _ = forward(bufs, x, gates, weights)
    want = want.float()

    served = []
    for wi, wo in weights:
        t = (torch.tensor([6.0 / 2688.0], device=dev) if a.fmt == "nv" else None)
        served.append(lowbit.Fp4Layer(lowbit.Fp4Experts.from_weights(a.fmt, wi, wo, t, t), shape))
    prompt = serve(x, gates, served).float()
    one = torch.cat([serve(x[i:i + 1], gates, served).float() for i in range(min(8, a.tokens))])
    rel = lambda p, q: float((p - q).norm() / q.norm())  # noqa: E731
    mse = float((prompt - target.float()).square().mean())
    print("serving in 4 bits: mean square error %.4f, %.4f off the bf16 model; single tokens "
          "%.4f off the prompt" % (mse, rel(prompt, want), rel(one, prompt[:one.shape[0]])))
    return losses, mse, rel(one, prompt[:one.shape[0]])


if __name__ == "__main__":
    main()
