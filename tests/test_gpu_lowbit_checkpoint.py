"""What 8-bit checkpoints refuse: buffers of another layer, and a forward that their backward
has overwritten."""
import dataclasses

import pytest
import torch

import moe_synth
from gpu_helpers import dev_bf16, layer_shape

pytestmark = pytest.mark.gpu


def one():
    from mixture_experts_grouped_router_gb300 import layer, lowbit
    cfg = moe_synth.scaled(moe_synth.CONFIGS["tiny"], T=96, E=4, k=2)
    inp = moe_synth.make_inputs(cfg, seed=1)
    b = layer.MoEBuffers(layer_shape(cfg, False))
    x, wi, wo, dout = (dev_bf16(inp[n]) for n in ("x", "wi", "wo", "dout"))
    return layer, lowbit, b, x, torch.from_numpy(inp["logits"]).cuda(), wi, wo, dout


def test_a_forward_that_the_backward_has_overwritten():
    layer, lowbit, b, x, logits, wi, wo, dout = one()
    from mixture_experts_grouped_router_gb300 import _lib as L
    ck = lowbit.Checkpoint8(b)
    layer.forward(b, x, logits, wi, wo)
    want = layer.backward(b, dout, wi, wo)[0].clone()
    ck.save(b)
    layer.forward(b, -x, -logits, wi, wo)
    ck.backward(b, dout, wi, wo)
    with pytest.raises(L.MoEError, match="null"):
        layer.backward(b, dout, wi, wo)
    with pytest.raises(ValueError, match="before a forward"):
        ck.save(b)
    layer.forward(b, x, logits, wi, wo)  # and the buffers go on
    assert torch.equal(layer.backward(b, dout, wi, wo)[0], want)
    torch.cuda.synchronize()
    assert int(b.dev_status.item()) == 0


def test_buffers_of_another_layer():
    layer, lowbit, b, x, logits, wi, wo, dout = one()
    ck = lowbit.Checkpoint8(b)
    layer.forward(b, x, logits, wi, wo)
    ck.save(b)
    for other in (dataclasses.replace(b.s, renorm=0 if b.s.renorm else 1),
                  dataclasses.replace(b.s, T=b.s.T // 2)):
        o = layer.MoEBuffers(other)
        o.logits = logits
        with pytest.raises(ValueError, match="for buffers of"):
            ck.save(o)
        with pytest.raises(ValueError, match="for buffers of"):
            ck.backward(o, dout, wi, wo)
    ck.backward(layer.MoEBuffers(dataclasses.replace(b.s)), dout, wi, wo)  # a like one
    torch.cuda.synchronize()
