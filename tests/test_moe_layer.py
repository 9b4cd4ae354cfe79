"""The example layer (router, dispatch, experts' products, combine and their gradients together) against autograd in 64
bits with the layer's own choice of experts.

Tolerance: every tensor between two calls is rounded to bf16, half a step of 2^-8 of each value.  The forward chain has
five such roundings (pre is kept apart), the backward one six more; roundings are independent and the sums run over
hundreds of them, so each adds at most 2^-8 to the relative error of the norm: 12 * 2^-8 for gradients, 6 * 2^-8 for
the output.  The router's gradients go through d_weights, sums of rounded y and d_out, and are differences of such sums
(the softmax's), which may cancel: 2^-2 of their norm.
"""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
H = 2.0 ** -8


def example():
    spec = importlib.util.spec_from_file_location(
        "moe_layer", os.path.join(ROOT, "combine_ep_layout_07_amd", "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(layer, x, d_out, d_balance):
    """Output, balance loss and gradients in 64 bits, choice held."""
    idx = layer.route.topk_idx.reshape(x.shape[0], -1).cpu()
    leaves = [t.cpu().double().requires_grad_(True) for t in (x, layer.router, layer.w_up, layer.w_down)]
    x64, router, up, down = leaves
    s = torch.softmax(x64 @ router.t(), 1)
    w = s.gather(1, idx)
    w = w / w.sum(1, keepdim=True)
    E, K = router.shape[0], idx.shape[1]
    out = x64
    for e in range(E):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        p = x64[t] @ up[e].t()
        n = p.shape[1] // 2
        y = (torch.nn.functional.silu(p[:, :n]) * p[:, n:]) @ down[e].t()
        out = out.index_add(0, t, w[t, k][:, None] * y)
    f = torch.bincount(idx.reshape(-1), minlength=E).double() * E / (K * x.shape[0])
    loss = (f * s.mean(0)).sum()
    ((out * d_out.cpu().double()).sum() + loss * d_balance.cpu().double()[0]).backward()
    return out.detach(), loss.detach(), [t.grad for t in leaves]


def off(got, want):
    return ((got.cpu().double() - want).norm() / want.norm()).item()


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hidden,inner,experts,topk,ranks", [
    (1, 256, 128, 8, 2, 2), (37, 264, 136, 12, 3, 4), (300, 512, 256, 16, 4, 4), (1024, 256, 384, 4, 2, 1)])
def test_layer_against_autograd(tokens, hidden, inner, experts, topk, ranks):
    print(f"[moe layer] T={tokens} H={hidden} I={inner} E={experts} K={topk}", flush=True)
    layer = example().MoELayer(tokens, hidden, inner, experts, topk, ranks, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    d_out = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    d_bal = torch.tensor([0.5 * tokens], device="cuda")
    out, loss = layer.forward(x)
    d_x = layer.backward(d_out, d_bal)
    torch.cuda.synchronize()
    w_out, w_loss, (gx, gr, gu, gd) = reference(layer, x, d_out, d_bal)
    assert off(out, w_out) <= 6 * H and abs(loss.item() - w_loss.item()) <= 1e-5 * w_loss.item()
    assert off(d_x, gx) <= 12 * H and off(layer.g_up, gu) <= 12 * H and off(layer.g_down, gd) <= 12 * H
    assert off(layer.g_router, gr) <= 0.25


@pytest.mark.gpu
def test_layer_learns():
    m = example()
    layer = m.MoELayer(512, 256, 128, 8, 2)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((512, 256), generator=g, device="cuda").bfloat16()
    target = torch.roll(x, 1, 1).float()
    losses = []
    for _ in range(12):
        out, _ = layer.forward(x)
        err = out.float() - target
        layer.backward((err * (2 / 512)).bfloat16(), torch.full((1,), 0.01, device="cuda"))
        layer.step(0.05)
        losses.append(err.square().sum(1).mean().item())
    assert losses[-1] < 0.98 * losses[0] and all(b < a * 1.01 for a, b in zip(losses, losses[1:]))
