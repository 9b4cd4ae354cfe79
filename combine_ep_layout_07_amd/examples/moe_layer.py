"""A mixture-of-experts layer on one GPU from libep's calls, forward, backward and a few training steps.

    python combine_ep_layout_07_amd/examples/moe_layer.py [--tokens 2048] [--steps 20]

Forward: router -> layout and dispatch (expand layout: one row per token and chosen expert) -> the experts' gated up
product -> their down product -> combine, with the token itself added as the combine's bias.
Backward: the same calls' gradients in reverse; the dispatch copies a token to its rows, so its gradient is a combine
with weights of one.
"""
import argparse
import os
import sys
import time

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.dirname(os.path.abspath(__file__)))))
import combine_ep_layout_07_amd.ep as ep  # noqa: E402


class MoELayer:
    def __init__(self, tokens, hidden, inner, experts, topk, ranks=1, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        b16 = dict(dtype=torch.bfloat16, device=device)
        rows = tokens * topk
        self.route_cfg = ep.make_route_config(1, tokens, experts, topk)
        self.cfg = ep.make_config(1, tokens, hidden, topk, experts, ranks, tokens, expand=True)
        self.up_cfg = ep.make_expert_config(experts, rows, hidden, inner, activation="swiglu")
        self.down_cfg = ep.make_expert_config(experts, rows, inner, hidden)
        # Parameters and their gradients.
        self.router = torch.randn((experts, hidden), generator=g, device=device) * hidden ** -0.5
        self.w_up = (torch.randn((experts, 2 * inner, hidden), generator=g, device=device) * hidden ** -0.5).bfloat16()
        self.w_down = (torch.randn((experts, hidden, inner), generator=g, device=device) * inner ** -0.5).bfloat16()
        self.g_up, self.g_down = torch.empty_like(self.w_up), torch.empty_like(self.w_down)
        self.g_router = torch.empty_like(self.router)
        # Handles, receive buffers and activations, kept between steps.
        self.route, self.layout = ep.alloc_route(self.route_cfg, balance=True), ep.alloc_layout(self.cfg)
        self.recv = ep.alloc_recv(self.cfg)
        self.rows = self.recv.recv_x.view(torch.bfloat16)
        self.pre, self.mid = torch.empty((rows, 2 * inner), **b16), torch.empty((rows, inner), **b16)
        self.y, self.out = torch.empty((rows, hidden), **b16), torch.empty((tokens, hidden), **b16)
        self.d_y, self.d_mid = torch.empty_like(self.y), torch.empty_like(self.mid)
        self.d_rows, self.d_x = torch.empty_like(self.y), torch.empty_like(self.out)
        self.d_weights = torch.empty((1, tokens, topk), device=device)
        self.ones = torch.ones((1, tokens, topk), device=device)
        self.up_scratch, self.down_scratch = ep.alloc_expert_backward(self.up_cfg), ep.alloc_expert_backward(self.down_cfg)

    def forward(self, x):
        """out [tokens][hidden] and the balance loss [1] of bf16 tokens."""
        self.x = x
        self.logits = x.float() @ self.router.t()
        r, base = self.route, self.layout.expert_base
        ep.ep_route(self.route_cfg, self.logits, r)
        ep.ep_layout_dispatch(self.cfg, x, None, r.topk_idx, r.topk_weights, self.layout, self.recv)
        ep.ep_expert_mm(self.up_cfg, base, self.rows, self.w_up, self.mid, pre=self.pre)
        ep.ep_expert_mm(self.down_cfg, base, self.mid, self.w_down, self.y)
        ep.ep_combine_bias(self.cfg, self.layout, r.topk_idx, r.topk_weights, self.y, x, None, self.out)
        return self.out, r.balance_loss

    def backward(self, d_out, d_balance):
        """Gradient of the tokens; those of the parameters go to g_router, g_up and g_down."""
        r, base = self.route, self.layout.expert_base
        ep.ep_combine_backward(self.cfg, self.layout, r.topk_idx, r.topk_weights, self.y, d_out, self.d_y, self.d_weights)
        ep.ep_expert_mm_backward(self.down_cfg, base, self.mid, self.w_down, self.d_y, self.down_scratch,
                                 d_x=self.d_mid, d_w=self.g_down)
        ep.ep_expert_mm_backward(self.up_cfg, base, self.rows, self.w_up, self.d_mid, self.up_scratch, pre=self.pre,
                                 d_x=self.d_rows, d_w=self.g_up)
        ep.ep_combine_bias(self.cfg, self.layout, r.topk_idx, self.ones, self.d_rows, d_out, None, self.d_x)
        d_logits = torch.empty_like(self.logits)
        ep.ep_route_backward(self.route_cfg, self.logits, r, self.d_weights, d_balance, d_logits)
        torch.mm(d_logits.t(), self.x.float(), out=self.g_router)
        return (self.d_x.float() + d_logits @ self.router).bfloat16()

    def step(self, rate):
        self.router -= rate * self.g_router
        for w, g in ((self.w_up, self.g_up), (self.w_down, self.g_down)):
            w.sub_(rate * g)


def main():
    p = argparse.ArgumentParser()
    for name, value in (("tokens", 2048), ("hidden", 1024), ("inner", 512), ("experts", 16), ("topk", 4), ("steps", 20)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    layer = MoELayer(a.tokens, a.hidden, a.inner, a.experts, a.topk)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((a.tokens, a.hidden), generator=g, device="cuda").bfloat16()
    target = torch.roll(x, 1, 1).float()
    balance = torch.full((1,), 0.01, device="cuda")
    for i in range(a.steps):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        out, aux = layer.forward(x)
        err = out.float() - target
        layer.backward((err * (2 / a.tokens)).bfloat16(), balance)
        layer.step(0.05)
        torch.cuda.synchronize()
        print(f"step {i:3d}  loss {err.square().sum(1).mean().item():9.3f}  balance {aux.item():.4f}  "
              f"{(time.perf_counter() - t0) * 1e3:.2f} ms", flush=True)


if __name__ == "__main__":
    main()
