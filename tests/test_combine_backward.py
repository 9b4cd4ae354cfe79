"""ep_combine_backward against 64-bit sums, and its refusals.

Tolerances: d_y is one fp32 product (the weights of a shared row summed in fp32 before) rounded to bf16: half a bf16
step, 2^-8 of the value, and K + 1 fp32 roundings.  d_weights is an fp32 sum of H exact-to-fp32 products: at most
(H / 64 + 16) additions in a chain, each off by 2^-24 of the sum of magnitudes.
"""
import ctypes

import numpy as np
import pytest
import torch

import combine_ep_layout_07_amd.ep as ep

U = 2.0 ** -24


def test_refusals():
    bad = ep.EP_ERR_INVALID_ARG
    cfg = ep.make_config(1, 16, 64, 2, 8, 4, 16)
    L = ep.EpLayoutT()

    def call(c, l, *p):
        return ep._lib.ep_combine_backward(ctypes.byref(c), ctypes.byref(l) if l is not None else None, *p, None)
    assert call(cfg, L, *[None] * 6) == bad and call(cfg, None, *[None] * 6) == bad
    assert call(ep.make_config(1, 16, 64, 2, 8, 4, 8), L, *[None] * 6) == ep.EP_ERR_CAPACITY
    if torch.cuda.is_available():
        return  # fake addresses below
    fake = 0x10000
    L = ep.EpLayoutT(*[fake + 256 * i for i in range(10)])
    ok = [fake, fake, fake, fake, fake, fake]  # topk_idx, topk_weights, y, d_out, d_y, d_weights
    for i, off in ((0, 4), (1, 2), (2, 8), (3, 8), (4, 8), (5, 2)):
        p = list(ok)
        p[i] = fake + off
        assert call(cfg, L, *p) == bad, i
        if i != 4 and i != 5:
            p[i] = None
            assert call(cfg, L, *p) == bad, i
    assert call(cfg, L, fake, fake, fake, fake, None, None) == bad


def test_binding_refuses():
    cfg = ep.make_config(1, 4, 64, 2, 8, 4, 4)
    idx, w = torch.zeros((1, 4, 2), dtype=torch.int64), torch.zeros((1, 4, 2))
    h = torch.zeros((8, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="d_out must have 2-byte elements"):
        ep.ep_combine_backward(cfg, None, idx, w, h, h.float(), h, w)
    with pytest.raises(ValueError, match="float32"):
        ep.ep_combine_backward(cfg, None, idx, w, h, h, h, w.double())


def rows_of(cfg, L, idx, n_out):
    """Receive row of every lane (-1 masked) from the layout's tables."""
    S, T, K = idx.shape
    if cfg.expand:
        return L.expand_pos.cpu().numpy()
    slot, base, psum = (t.cpu().numpy() for t in (L.dst_slot, L.recv_base, L.recv_psum))
    El, n_up = cfg.num_experts // cfg.num_ranks, S // n_out
    row = np.full(idx.shape, -1, np.int64)
    for s in range(S):
        rb = s // n_up if n_out > 1 else s
        for t in range(T):
            of_rank = {}
            for k in range(K):
                if not 0 <= idx[s, t, k] < cfg.num_experts:
                    continue
                d = idx[s, t, k] // El
                if slot[s, t, k] >= 0:
                    of_rank[d] = base[d] + psum[d, s] + slot[s, t, k] - rb * cfg.num_max_tokens_per_rank
                row[s, t, k] = of_rank[d]
    return row


CASES = [  # S, T, H, K, E, R, expand, A, n_out
    (1, 1, 8, 1, 4, 4, False, 1, 1), (1, 1, 7168, 8, 256, 16, True, 1, 1), (2, 33, 520, 6, 48, 8, False, 1, 1),
    (3, 21, 1288, 6, 64, 8, True, 1, 1), (2, 40, 512, 4, 32, 8, True, 16, 1), (4, 17, 2056, 8, 64, 16, False, 1, 2),
    (1, 29, 136, 32, 64, 64, False, 1, 1), (1, 13, 4104, 32, 64, 4, True, 3, 1), (1, 50, 504, 9, 18, 2, False, 1, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("S,T,H,K,E,R,expand,A,n_out", CASES)
def test_combine_backward(S, T, H, K, E, R, expand, A, n_out):
    print(f"[combine_backward] S={S} T={T} H={H} K={K} E={E} R={R} expand={expand} A={A}", flush=True)
    rng = np.random.default_rng(S * 1000 + T)
    idx = np.stack([rng.permutation(E)[:K] for _ in range(S * T)]).reshape(S, T, K).astype(np.int64)
    idx[rng.uniform(size=idx.shape) < 0.2] = -1
    if T > 2:
        idx[0, 1] = -1  # a token without a lane
        idx[0, 2, 0] = E + 3  # an id out of range is masked too
    w = rng.standard_normal(idx.shape).astype(np.float32)
    cfg = ep.make_config(S, T, H, K, E, R, T + 3, expand=expand, alignment=A, num_scaleout_ranks=n_out)
    L = ep.alloc_layout(cfg)
    ti, tw = torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda()
    ep.ep_layout(cfg, ti, L)
    rows = int(ep.ep_query_sizes(cfg).recv_rows)
    g = torch.Generator().manual_seed(3)
    y = torch.randn((rows, H), generator=g).bfloat16()
    d = torch.randn((S * T, H), generator=g).bfloat16()
    row = rows_of(cfg, L, idx, n_out).reshape(S * T, K)
    valid = ((idx >= 0) & (idx < E)).reshape(S * T, K)
    dy, dw = torch.full((rows, H), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((S, T, K), 9.0, device="cuda")
    yd, dd = y.cuda(), d.cuda()
    ep.ep_combine_backward(cfg, L, ti, tw, yd, dd, dy, dw)
    torch.cuda.synchronize()
    y64, d64, w64 = y.double().numpy(), d.double().numpy(), w.reshape(S * T, K).astype(np.float64)
    weight, wmag, token = np.zeros(rows), np.zeros(rows), np.full(rows, -1)
    want, mag = np.zeros((S * T, K)), np.zeros((S * T, K))
    for t in range(S * T):
        for k in range(K):
            if valid[t, k]:
                r = row[t, k]
                weight[r] += w64[t, k]
                wmag[r] += abs(w64[t, k])
                token[r] = t
                want[t, k] = (y64[r] * d64[t]).sum()
                mag[t, k] = np.abs(y64[r] * d64[t]).sum()
    got = dw.cpu().numpy().reshape(S * T, K)
    assert (np.abs(got - want) <= (H / 64 + 16) * U * mag).all()
    assert (got[~valid] == 0).all()
    gy = dy.double().cpu().numpy()
    used = token >= 0
    ref = weight[used, None] * d64[token[used]]
    tol = 2.0 ** -8 * np.abs(ref) + (K + 1) * U * wmag[used, None] * np.abs(d64[token[used]]) * (1 + 2.0 ** -8)
    assert (np.abs(gy[used] - ref) <= tol).all()
    pad = np.zeros(rows, bool)
    if expand:
        base, tpe = L.expert_base.cpu().numpy(), L.tokens_per_expert.cpu().numpy().sum(0)
        for e in range(E):
            pad[base[e] + tpe[e]:base[e + 1]] = True
    assert (gy[pad] == 0).all() and (gy[~used & ~pad] == 3.0).all()
    # each gradient alone, without the other's inputs
    dy2, dw2 = torch.full_like(dy, 3.0), torch.empty_like(dw)
    ep.ep_combine_backward(cfg, L, ti, tw, None, dd, dy2, None)
    ep.ep_combine_backward(cfg, L, ti, None, yd, dd, None, dw2)
    assert torch.equal(dy2, dy) and torch.equal(dw2, dw)


@pytest.mark.gpu
def test_gradient_against_differences():
    """The combine is linear in y and in the weights: exact directional differences of its 64-bit form."""
    S, T, H, K, E, R = 1, 20, 264, 4, 16, 4
    rng = np.random.default_rng(1)
    idx = torch.from_numpy(np.stack([rng.permutation(E)[:K] for _ in range(T)]).reshape(S, T, K).astype(np.int64)).cuda()
    cfg = ep.make_config(S, T, H, K, E, R, T, expand=True)
    L = ep.alloc_layout(cfg)
    ep.ep_layout(cfg, idx, L)
    w = torch.rand((S, T, K), device="cuda")
    y, d = torch.randn((T * K, H), device="cuda").bfloat16(), torch.randn((T, H), device="cuda").bfloat16()
    dy, dw = torch.empty_like(y), torch.empty_like(w)
    ep.ep_combine_backward(cfg, L, idx, w, y, d, dy, dw)
    row = L.expand_pos.long().reshape(T, K)

    def objective(w, y):
        return ((w.reshape(T, K, 1) * y[row]).sum(1) * d.double()).sum()
    gw, gy = torch.randn_like(w).double(), torch.randn_like(y).double()
    want = objective(w.double() + gw, y.double() + gy) - objective(w.double(), y.double()) - objective(gw, gy)
    have = (dw.double() * gw).sum() + (dy.double() * gy).sum()
    size = (dw.double() * gw).abs().sum() + (dy.double() * gy).abs().sum()
    assert (have - want).abs() <= (2.0 ** -8 + 64 * U) * size


@pytest.mark.gpu
def test_no_tokens():
    cfg = ep.make_config(2, 0, 64, 2, 8, 4, 0)
    L = ep.alloc_layout(cfg)
    z = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    i, w = torch.zeros((2, 0, 2), dtype=torch.int64, device="cuda"), torch.zeros((2, 0, 2), device="cuda")
    ep.ep_layout(cfg, i, L)
    ep.ep_combine_backward(cfg, L, i, w, z, z, z, w)
    torch.cuda.synchronize()
