"""Every gradient of the example block against the same block in float64 with autograd: the chain
through both norms, the residual branch, the layer, the router product and the embedding."""
import math

import pytest
import torch

from examples import train_moe_block as B
from routing_dispatch_grouped_gb300 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _block_gradients(w, ids, target, k, topk):
    """Gradients by name, in float64, of the weights that the kernels read; `topk` fixes the
    experts, as the layer's own backward pass does."""
    p = {n: w[n].double().requires_grad_() for n in w.names}
    d, E, I = p["table"].shape[1], p["router"].shape[1], p["down"].shape[1]
    ids, topk = ids.long(), topk.long()
    h = p["table"][ids] * math.sqrt(d)
    x = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-5) * p["norm1"]
    logits = x @ p["router"]
    score = torch.exp(logits - logits.detach().amax(1, keepdim=True)).gather(1, topk)
    score = score / score.sum(1, keepdim=True)
    out = 0
    for e in range(E):
        gate, up = (x @ p["gate_up"][e]).split(I, 1)
        y = (gate / (1 + torch.exp(-gate)) * up) @ p["down"][e]
        out = out + y * (score * (topk == e)).sum(1, keepdim=True)
    s = h + out
    c = s - s.mean(1, keepdim=True)
    y = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * p["norm2"] + p["bias2"]
    (y - target.double()).square().mean().backward()
    return {n: t.grad for n, t in p.items()}


@pytest.mark.parametrize("T,V,d,E,I,k", [(64, 40, 128, 4, 128, 2), (300, 90, 256, 8, 64, 3)])
def test_every_gradient_of_the_block(T, V, d, E, I, k):
    w = B.make_weights(V, d, E, I, 32)
    ids = (torch.arange(T, device=DEV, dtype=torch.int32) * 7) % V
    target = torch.randn(T, d, device=DEV, generator=torch.Generator(DEV).manual_seed(3))
    # norms that are not the identity
    for name, size in (("norm1", 0.3), ("norm2", 0.3), ("bias2", 0.2)):
        noise = torch.randn(d, device=DEV, generator=torch.Generator(DEV).manual_seed(5))
        w[name].add_(size * noise)
    grads = {}
    w.step = lambda g, t, lr: grads.update(g)           # gradients only, no update
    B.train_step(w, ids, target, k, 1, 0.0)
    h = moe.moe_embed(ids, w["table"], math.sqrt(d))
    x = moe.moe_norm(h, w["norm1"], rms=True)[0]
    topk = moe.moe_route_hidden(x, w["router"], k)[0]
    ref = _block_gradients(w, ids, target, k, topk)
    assert set(grads) == set(ref)
    for name, r in ref.items():
        # about ten roundings to bf16 on the way there and back, 2^-9 of a value each: 2e-2 if all
        # fell to one side, and half as much again for what the norms and the softmax make of them
        err = (grads[name].double() - r).norm() / r.norm()
        assert err <= 3e-2, (name, float(err))
