"""The stack of MoE blocks of examples/moe_block.py, trained and served, against 64-bit formulas and autograd.

Tolerances: the layer's own parity limits on each tensor, 5e-3 for activations and 1e-2 for weight gradients, taken
twice over: each of the two blocks adds its rounding to what passes through it."""
import os
import sys

import pytest
import torch

from routing_grouped_expert_router_gb300 import binding as mb
from routing_grouped_expert_router_gb300 import build as mbuild
from tests.helpers import rel_l2

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def stack():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mbuild.build()
    mb.load()
    import moe_block
    return moe_block.Stack(blocks=2, h=256, f=192, E=4, k=2, seed=3, alpha=1.0, beta=0.5)


def rms(v, eps):
    return torch.sqrt((v * v).mean(-1, keepdim=True) + eps)


def stack64(s, r, weights, routes):
    """The stack in 64 bits, with the experts of `routes` (the kernels' own choices)."""
    n = s.norm
    for w, idx in zip(weights, routes):
        u = r / rms(r, n["eps"]) * w["w_pre"]
        gates = torch.softmax(torch.gather(u @ w["Wg"], 1, idx), -1)
        y = 0
        for e in range(s.E):
            g = (gates * (idx == e)).sum(-1, keepdim=True)
            a = u @ w["W1"][e]
            y = y + g * ((a * torch.sigmoid(a) * (u @ w["W3"][e])) @ w["W2"][e])
        r = n["alpha"] * r + n["beta"] * w["gate"] * (y / rms(y, n["eps"]) * w["w_post"])
    return r


def routes_of(s, d, kept):
    from tests.gpu_runner import saved_tensor
    return [saved_tensor(d, c["saved"], "topk_idx").long() for c in kept]


def test_forward_and_backward(stack):
    s = stack
    r0 = torch.randn(300, s.h, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    dr = torch.randn(300, s.h, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    out, ctx = s.forward(r0)
    grad, grads = s.backward(ctx, dr)
    torch.cuda.synchronize()
    leaf = r0.double().requires_grad_(True)
    weights = [{n: w.double().requires_grad_(True) for n, w in b.items()} for b in s.blocks]
    ref = stack64(s, leaf, weights, routes_of(s, ctx[0], ctx[2]))
    assert rel_l2(out.cpu(), ref.detach().cpu()) <= 2 * 5e-3
    names = ("Wg", "W1", "W3", "W2", "w_pre", "w_post", "gate")
    want = torch.autograd.grad(ref, [leaf] + [w[n] for w in weights for n in names], dr.double())
    assert rel_l2(grad.cpu(), want[0].cpu()) <= 2 * 5e-3
    for i, (b, n) in enumerate((b, n) for b in grads for n in names):
        assert rel_l2(b[n].cpu(), want[1 + i].cpu()) <= 2 * 1e-2, n


@pytest.mark.parametrize("T", [1, 7, 64])
def test_decode_agrees_with_the_forward(stack, T):
    s = stack
    r0 = torch.randn(T, s.h, device="cuda", generator=torch.Generator("cuda").manual_seed(6))
    want, _ = s.forward(r0)
    buf = s.decoder(T)
    r = r0.clone()
    s.decode(buf, r)
    torch.cuda.synchronize()
    assert mb.moe_read_device_status(buf["ws"]) == mb.MOE_OK
    assert rel_l2(r.cpu(), want.cpu()) <= 2 * 5e-3


def test_decode_step_in_a_graph(stack):
    s = stack
    r0 = torch.randn(5, s.h, device="cuda", generator=torch.Generator("cuda").manual_seed(7))
    buf, r = s.decoder(5), r0.clone()
    s.decode(buf, r)
    torch.cuda.synchronize()
    want = r.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.decode(buf, r)
    r.copy_(r0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(r, want)
