"""The router (ep_route, ep_route_backward) against a plain 64-bit implementation, and its refusals.

Tolerances, from the 32-bit arithmetic (u = 2^-24, the largest relative rounding): a score exp(l - max) carries the
rounding of its argument, at most 2 * max|l| * u, and a few u of the exponential, the sum and the division; with
|l| <= 24 that is below 64 u.  Gradients are sums of such terms, so their error is below 64 u times the sum of the
terms' magnitudes, plus half a step of bf16 (2^-8 of the value) where the logits are bf16.
"""
import ctypes

import numpy as np
import pytest
import torch

import combine_ep_layout_07_amd.ep as ep

U = 2.0 ** -24
REL = 64 * U


def call(cfg, r=None, logits=None, bias=None, mask=None):
    return ep._lib.ep_route(ctypes.byref(cfg), logits, bias, mask, ctypes.byref(r) if r else None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(S=0), ep.EP_ERR_INVALID_ARG), (dict(T=-1), ep.EP_ERR_INVALID_ARG), (dict(E=0), ep.EP_ERR_INVALID_ARG),
    (dict(K=0), ep.EP_ERR_INVALID_ARG), (dict(K=9, E=8), ep.EP_ERR_INVALID_ARG),
    (dict(scale=float("nan")), ep.EP_ERR_INVALID_ARG), (dict(scale=float("inf")), ep.EP_ERR_INVALID_ARG),
    (dict(E=1025), ep.EP_ERR_UNSUPPORTED), (dict(K=33), ep.EP_ERR_UNSUPPORTED), (dict(S=65536), ep.EP_ERR_UNSUPPORTED),
    (dict(T=2 ** 30 + 1, K=1), ep.EP_ERR_UNSUPPORTED), (dict(S=2, T=2 ** 30, K=1), ep.EP_ERR_UNSUPPORTED),
    (dict(T=2 ** 30, K=1), ep.EP_OK), (dict(K=32, E=1024), ep.EP_OK),
])
def test_configuration_codes(kw, code):
    base = dict(S=1, T=16, E=64, K=4, scale=1.0)
    base.update(kw)
    cfg = ep.make_route_config(**base)
    sz = ep.EpRouteSizes()
    assert ep._lib.ep_query_route_sizes(ctypes.byref(cfg), ctypes.byref(sz)) == code
    if code != ep.EP_OK:
        assert call(cfg) == code
        with pytest.raises(ep.EpError):
            ep.alloc_route(cfg)


def test_configuration_enums():
    for field, value in (("logits_dtype", ep.EP_DTYPE_FP8_E4M3FN), ("logits_dtype", 3), ("scoring", 2), ("scoring", -1)):
        cfg = ep.make_route_config(1, 4, 8, 2)
        setattr(cfg, field, value)
        assert call(cfg) == ep.EP_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        ep.make_route_config(1, 4, 8, 2, dtype="fp16")
    with pytest.raises(ValueError):
        ep.make_route_config(1, 4, 8, 2, scoring="relu")
    sz = ep.ep_query_route_sizes(ep.make_route_config(3, 100, 24, 4))
    assert (sz.topk_idx, sz.topk_weights) == (3 * 100 * 4 * 8, 3 * 100 * 4 * 4)
    assert (sz.tokens_per_expert, sz.tokens_valid, sz.balance_loss) == (3 * 24 * 4, 12, 12)


@pytest.mark.skipif(torch.cuda.is_available(), reason="passes fake device addresses; host-only check")
def test_pointer_codes():
    cfg = ep.make_route_config(1, 4, 8, 2)
    fake = 0x10000
    bad = ep.EP_ERR_INVALID_ARG
    r = ep.EpRouteT(fake, fake + 256)
    assert call(cfg, None, fake) == bad and call(cfg, r, None) == bad and call(cfg, r, fake + 2) == bad
    assert call(cfg, ep.EpRouteT(None, fake), fake) == bad and call(cfg, ep.EpRouteT(fake, None), fake) == bad
    assert call(cfg, ep.EpRouteT(fake + 4, fake), fake) == bad      # topk_idx not 8-byte aligned
    assert call(cfg, r, fake, bias=fake + 2) == bad
    for i in range(2, 6):  # the balance loss's buffers: all or none
        r = ep.EpRouteT(*[fake + 256 * j for j in range(6)])
        setattr(r, ep.EpRouteT._fields_[i][0], None)
        assert call(cfg, r, fake) == bad
    r = ep.EpRouteT(fake, fake + 256)

    def back(dw, dl, out, logits=fake):
        return ep._lib.ep_route_backward(ctypes.byref(cfg), logits, None, ctypes.byref(r), dw, dl, out, None)
    assert back(None, None, fake) == bad and back(fake, None, None) == bad and back(fake, None, fake + 2) == bad
    assert back(None, fake, fake) == bad  # the loss's gradient needs the counts
    assert back(fake, None, fake, None) == bad


def test_binding_refuses():
    cfg = ep.make_route_config(1, 4, 8, 2)
    x = torch.zeros((1, 4, 8))
    with pytest.raises(ValueError, match="logits must be"):
        ep.ep_route(cfg, x.bfloat16(), None)
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_route(cfg, x, None)
    with pytest.raises(ValueError, match="bias must be float32"):
        ep.ep_route(cfg, x, None, bias=torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError, match="must be float32"):
        ep.ep_route_backward(cfg, x, None, torch.zeros((1, 4, 2), dtype=torch.float64), None, x)


# ------------------------------------------------------------------------------------------------- the 64-bit formulas

def plain(logits, K, scoring, scale, bias=None, mask=None, low=None):
    """Everything of one source set [S][T][E] in 64 bits, choice included."""
    l = logits.astype(np.float64)
    S, T, E = l.shape
    ok = l > low
    if mask is not None:
        ok &= (mask != 0)[:, :, None]
    l = np.where(ok, np.minimum(l, -low), 0.0)
    if scoring == "softmax":
        e = np.where(ok, np.exp(l - np.where(ok, l, -np.inf).max(2, initial=-np.inf, keepdims=True, where=ok)), 0.0)
        s = e / np.maximum(e.sum(2, keepdims=True), 1e-30)
    else:
        s = np.where(ok, 1 / (1 + np.exp(-np.clip(l, -700, 700))), 0.0)
    rest = 1 / (1 + np.exp(np.clip(l, -700, 700)))  # 1 - s of the sigmoid, which 1 - s itself loses where s is near 1
    key = np.where(ok, l if bias is None else s + bias.astype(np.float64), -np.inf)
    idx = np.argsort(-key, axis=2, kind="stable")[:, :, :K]
    there = np.take_along_axis(key, idx, 2) > -np.inf
    sk = np.where(there, np.take_along_axis(s, idx, 2), 0.0)
    D = sk.sum(2, keepdims=True) + 1e-20
    p = s if scoring == "softmax" else s / (s.sum(2, keepdims=True) + 1e-20)
    count = np.zeros((S, E), np.int64)
    for a in range(S):
        np.add.at(count[a], idx[a][there[a]], 1)
    valid = ok.any(2).sum(1)
    v = np.maximum(valid, 1).astype(np.float64)
    share = count * E / (K * v[:, None])
    loss = (share * p.sum(1) / v[:, None]).sum(1)
    return dict(ok=ok, s=s, rest=rest, p=p, idx=np.where(there, idx, -1), there=there, sk=sk, D=D, w=scale * sk / D, count=count,
                valid=valid, loss=loss, share=share, v=v, key=key)


def plain_grad(f, scoring, scale, dw, dl):
    """(gradient, sum of its terms' magnitudes)."""
    def one(dw, dl, sign):
        s, p, there = f["s"], f["p"], f["there"]
        dk = np.where(there, scale * (dw + sign * (dw * f["sk"] / f["D"]).sum(2, keepdims=True)) / f["D"], 0.0)
        u = np.zeros_like(s)
        np.put_along_axis(u, np.where(there, f["idx"], 0), 0.0, 2)
        for k in range(dk.shape[2]):
            i = np.maximum(f["idx"][:, :, k:k + 1], 0)
            np.put_along_axis(u, i, np.take_along_axis(u, i, 2) + dk[:, :, k:k + 1], 2)
        a = (dl / f["v"])[:, None] * f["share"]
        a = a[:, None, :]
        if scoring == "softmax":
            u = u + a
            g = s * (u + sign * (u * s).sum(2, keepdims=True))
        else:
            u = u + (a + sign * (a * p).sum(2, keepdims=True)) / (s.sum(2, keepdims=True) + 1e-20)
            g = u * s * f["rest"]
        return np.where(f["ok"], g, 0.0)
    return one(dw, dl, -1.0), one(np.abs(dw), np.abs(dl), 1.0)


def make(S, T, E, dtype, seed, spread=1.5):
    rng = np.random.default_rng(seed)
    l = (spread * rng.standard_normal((S, T, E)) + 0.4 * rng.standard_normal((1, 1, E))).astype(np.float32)
    return torch.from_numpy(l).to(torch.bfloat16 if dtype == "bf16" else torch.float32), rng


def low_of(dtype):
    return float(torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).min)


def within(err, tol):
    bad = ~(err <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside; worst {(err / tol)[bad].max():.3g} of the tolerance"


def check(S, T, E, K, dtype, scoring, bias=None, mask=None, logits=None, seed=0, scale=2.5, rel=REL, rel_grad=REL,
          floor=0.0, floor_grad=1e-37):
    base, rng = make(S, T, E, dtype, seed)
    if logits is None:
        logits = base
    print(f"[route] S={S} T={T} E={E} K={K} {dtype} {scoring} bias={bias is not None} mask={mask is not None}", flush=True)
    f = plain(logits.float().numpy(), K, scoring, scale, bias, mask, low_of(dtype))
    cfg = ep.make_route_config(S, T, E, K, dtype, scoring, scale)
    r = ep.alloc_route(cfg, balance=True)
    x = logits.cuda()
    b = None if bias is None else torch.from_numpy(bias).cuda()
    m = None if mask is None else torch.from_numpy(mask).cuda()
    ep.ep_route(cfg, x, r, bias=b, token_mask=m)
    dw, dl = rng.standard_normal((S, T, K)).astype(np.float32), rng.uniform(0.5, 1.5, S).astype(np.float32)
    out = torch.full_like(x, 7.0)
    ep.ep_route_backward(cfg, x, r, torch.from_numpy(dw).cuda(), torch.from_numpy(dl).cuda(), out, token_mask=m)
    torch.cuda.synchronize()
    assert (r.topk_idx.cpu().numpy() == f["idx"]).all()
    assert (np.abs(r.topk_weights.cpu().numpy() - f["w"]) <= rel * np.abs(f["w"]) + floor).all()
    assert (r.tokens_per_expert.cpu().numpy() == f["count"]).all()
    assert (r.tokens_valid.cpu().numpy() == f["valid"]).all()
    assert (np.abs(r.balance_loss.cpu().numpy() - f["loss"]) <= rel * f["loss"]).all()
    g, mag = plain_grad(f, scoring, scale, dw.astype(np.float64), dl.astype(np.float64))
    half = 2.0 ** -8 if dtype == "bf16" else 0.0
    got = out.float().cpu().numpy()
    err = np.abs(got - g)
    within(err, rel_grad * mag + half * np.abs(g) + floor_grad)
    # each gradient alone, and the forward without a balance loss
    r2 = ep.alloc_route(cfg)
    ep.ep_route(cfg, x, r2, bias=b, token_mask=m)
    assert torch.equal(r2.topk_idx, r.topk_idx) and torch.equal(r2.topk_weights, r.topk_weights)
    for use_w in (True, False):
        ep.ep_route_backward(cfg, x, r, torch.from_numpy(dw).cuda() if use_w else None,
                             None if use_w else torch.from_numpy(dl).cuda(), out, token_mask=m)
        g, mag = plain_grad(f, scoring, scale, dw.astype(np.float64) * use_w, dl.astype(np.float64) * (not use_w))
        err = np.abs(out.float().cpu().numpy() - g)
        within(err, rel_grad * mag + half * np.abs(g) + floor_grad)
    return f, got


SHAPES = [(1, 1, 8, 1), (1, 1, 256, 8), (1, 3, 31, 31), (3, 67, 64, 6), (2, 130, 65, 4), (1, 257, 100, 8),
          (5, 19, 160, 6), (2, 300, 384, 11), (1, 40, 512, 8), (1, 33, 1024, 32), (2, 9, 1000, 8), (17, 5, 128, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("S,T,E,K", SHAPES)
def test_route(S, T, E, K, dtype, scoring):
    rng = np.random.default_rng(5)
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
    mask = (rng.uniform(size=(S, T)) < 0.8).astype(np.uint8)
    check(S, T, E, K, dtype, scoring, seed=1)
    check(S, T, E, K, dtype, scoring, bias, mask, seed=2)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_masked_and_special_logits(dtype, scoring):
    """Lowest values, -inf and NaN are masked, also a whole row; +inf is the type's largest value; fewer valid experts
    than K leave lanes of -1."""
    S, T, E, K = 2, 12, 40, 6
    x, _ = make(S, T, E, dtype, 3)
    x[0, 0] = float("-inf")
    x[0, 1] = low_of(dtype)
    x[0, 2] = float("nan")
    x[0, 3, 4:] = float("-inf")
    x[0, 4, ::2] = float("nan")
    x[0, 5, 1:] = low_of(dtype)
    x[1, 0, 7] = float("inf")
    x[1, 1, 3:] = float("nan")
    bias = np.linspace(-0.1, 0.1, E).astype(np.float32)
    for b in (None, bias):
        f, got = check(S, T, E, K, dtype, scoring, b, logits=x, seed=4)
        assert (f["valid"] == [T - 3, T]).all() and np.isfinite(got).all() and (got[0, :3] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(scoring):
    x = torch.zeros((1, 5, 192))
    x[0, 1, 100:] = 1.0
    x[0, 2] = torch.arange(192) % 3
    x[0, 3] = 60.0  # saturated scores: equal in 64 bits
    x[0, 3, ::2] = 80.0
    for bias in (None, np.zeros(192, np.float32), np.full(192, 1e6, np.float32)):
        check(1, 5, 192, 8, "fp32", scoring, bias, logits=x, seed=6)


@pytest.mark.gpu
def test_choice_with_a_bias_is_settled_in_64_bits():
    """Keys that differ far below a 32-bit step are told apart, and experts without a usable bias left out."""
    rng = np.random.default_rng(7)
    E, T = 64, 200
    x = torch.from_numpy((1e-4 * rng.standard_normal((1, T, E))).astype(np.float32))
    f = plain(x.numpy(), 8, "sigmoid", 1.0, np.zeros(E, np.float32), None, low_of("fp32"))
    key = np.sort(f["key"], axis=2)[:, :, ::-1]
    assert (np.diff(key[:, :, :9], axis=2) > -2.0 ** -26).any()  # some neighbours are closer than 32 bits tell
    check(1, T, E, 8, "fp32", "sigmoid", np.full(E, 3.0, np.float32), logits=x, seed=8)
    bias = np.zeros(E, np.float32)
    bias[5], bias[6] = np.nan, -np.inf
    cfg = ep.make_route_config(1, T, E, E, "fp32", "sigmoid")
    with pytest.raises(ep.EpError):
        ep.alloc_route(cfg)
    cfg = ep.make_route_config(1, T, 32, 32, "fp32", "sigmoid")
    r = ep.alloc_route(cfg)
    ep.ep_route(cfg, x[:, :, :32].contiguous().cuda(), r, bias=torch.from_numpy(bias[:32]).cuda())
    idx = r.topk_idx.cpu().numpy()
    assert (idx[:, :, 30:] == -1).all() and not np.isin(idx, (5, 6)).any()


@pytest.mark.gpu
def test_no_tokens_and_unaligned_rows():
    cfg = ep.make_route_config(2, 0, 16, 2)
    r = ep.alloc_route(cfg, balance=True)
    x = torch.zeros((2, 0, 16), device="cuda")
    ep.ep_route(cfg, x, r)
    ep.ep_route_backward(cfg, x, r, torch.zeros((2, 0, 2), device="cuda"), None, x)
    assert r.tokens_per_expert.eq(0).all() and r.tokens_valid.eq(0).all() and r.balance_loss.eq(0).all()
    # logits that begin one element off a 16-byte line
    for dtype in (torch.float32, torch.bfloat16):
        cfg = ep.make_route_config(1, 9, 64, 4, "bf16" if dtype == torch.bfloat16 else "fp32")
        flat = torch.randn(9 * 64 + 1, device="cuda").to(dtype)
        a, b = ep.alloc_route(cfg), ep.alloc_route(cfg)
        ep.ep_route(cfg, flat[1:], a)
        ep.ep_route(cfg, flat[1:].clone(), b)
        assert torch.equal(a.topk_idx, b.topk_idx) and torch.equal(a.topk_weights, b.topk_weights)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_gradient_against_differences(scoring):
    """Along random directions, with choice and counts held: central differences of the 64-bit objective.  Step
    h = 1e-4: the third-order term is below h^2 * |d|^3, relative 1e-6; the kernel's own error is tested above."""
    S, T, E, K, scale = 2, 40, 48, 4, 2.5
    x, rng = make(S, T, E, "fp32", 11)
    dw, dl = rng.standard_normal((S, T, K)), rng.uniform(0.5, 1.5, S) * T
    f = plain(x.numpy(), K, scoring, scale, low=low_of("fp32"))

    def objective(l):
        if scoring == "softmax":
            s = np.exp(l) / np.exp(l).sum(2, keepdims=True)
            p = s
        else:
            s = 1 / (1 + np.exp(-l))
            p = s / s.sum(2, keepdims=True)
        sk = np.take_along_axis(s, f["idx"], 2)
        w = scale * sk / sk.sum(2, keepdims=True)
        return (w * dw).sum() + (dl * (f["share"] * p.sum(1) / f["v"][:, None]).sum(1)).sum()
    cfg = ep.make_route_config(S, T, E, K, "fp32", scoring, scale)
    r = ep.alloc_route(cfg, balance=True)
    ep.ep_route(cfg, x.cuda(), r)
    out = torch.empty((S, T, E), device="cuda")
    ep.ep_route_backward(cfg, x.cuda(), r, torch.from_numpy(dw.astype(np.float32)).cuda(),
                         torch.from_numpy(dl.astype(np.float32)).cuda(), out)
    g = out.double().cpu().numpy()
    for _ in range(5):
        d = rng.standard_normal(g.shape)
        h = 1e-4
        want = (objective(x.numpy() + h * d) - objective(x.numpy() - h * d)) / (2 * h)
        assert abs((g * d).sum() - want) <= 1e-5 * np.abs(g * d).sum() + 1e-9


@pytest.mark.gpu
def test_route_repeats_and_replays():
    """Bitwise the same on every call, on a side stream and in a replayed graph."""
    cfg = ep.make_route_config(3, 501, 96, 6, "bf16", "sigmoid", 2.5)
    x, _ = make(3, 501, 96, "bf16", 13)
    x = x.cuda()
    r = ep.alloc_route(cfg, balance=True)
    dw, dl, out = torch.randn((3, 501, 6), device="cuda"), torch.ones(3, device="cuda"), torch.empty_like(x)

    def step():
        ep.ep_route(cfg, x, r)
        ep.ep_route_backward(cfg, x, r, dw, dl, out)

    def values():
        torch.cuda.synchronize()
        return [t.clone() for t in (r.topk_idx, r.topk_weights, r.tokens_per_expert, r.tokens_valid, r.balance_loss, out)]
    step()
    want = values()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    assert all(torch.equal(a, b) for a, b in zip(values(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        for t in (r.topk_idx, r.tokens_per_expert, out):
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(values(), want))
        step()
        assert all(torch.equal(a, b) for a, b in zip(values(), want))


# ------------------------------------------------------------------------------- many tokens: several tokens per wave

MANY = [(1, 8193, 8, 2), (3, 2731, 31, 4), (1, 8192, 64, 6), (2, 4111, 100, 8), (1, 9000, 160, 11), (5, 1639, 192, 1),
        (1, 8201, 256, 8), (1, 8192, 256, 15), (1, 8200, 260, 31), (2, 4100, 384, 6), (1, 8195, 512, 8), (1, 8192, 512, 32),
        (1, 8192, 600, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("S,T,E,K", MANY)
def test_many_tokens(S, T, E, K, dtype, scoring):
    rng = np.random.default_rng(S * 131 + T + E)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    mask = (rng.uniform(size=(S, T)) < 0.9).astype(np.uint8)
    check(S, T, E, K, dtype, scoring, seed=3)
    check(S, T, E, K, dtype, scoring, bias, mask, seed=4)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("S,T,E,K", [(1, 1025, 48, 4), (3, 683, 100, 6), (1, 1500, 256, 8), (2, 600, 512, 11), (1, 1100, 700, 32),
                                     (1, 2048, 64, 6), (2, 1031, 33, 15)])
def test_between_few_and_many_tokens(S, T, E, K, dtype, scoring):
    """A token per wave in large workgroups; several tokens per wave for few experts."""
    rng = np.random.default_rng(S * 17 + T + E)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    mask = (rng.uniform(size=(S, T)) < 0.9).astype(np.uint8)
    check(S, T, E, K, dtype, scoring, seed=5)
    check(S, T, E, K, dtype, scoring, bias, mask, seed=6)


@pytest.mark.gpu
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_many_tokens_with_near_ties(scoring, biased):
    """Keys that agree in their upper bits, in whole rows and at the border of the choice: whole keys decide."""
    T, E, K = 8400, 256, 8
    rng = np.random.default_rng(5)
    x = 1.0 + rng.integers(0, 40, size=(1, T, E)).astype(np.float32) * np.float32(2.0 ** -23)
    x[0, ::3] = rng.integers(0, 6, size=(2800, E)) * 0.25  # equal values: the lowest index
    bias = (rng.integers(-3, 4, size=E) * 2.0 ** -22).astype(np.float32) if biased else None
    check(1, T, E, K, "fp32", scoring, bias, logits=torch.from_numpy(x), seed=9)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_many_tokens_masked_and_special(dtype, scoring):
    S, T, E, K = 2, 4200, 130, 6
    x, rng = make(S, T, E, dtype, 13)
    x[0, 0:4200:7] = float("-inf")
    x[0, 1:4200:7] = low_of(dtype)
    x[0, 2:4200:7] = float("nan")
    x[0, 3:4200:7, 4:] = float("-inf")
    x[0, 4:4200:7, ::2] = float("nan")
    x[1, 5:4200:7, 7] = float("inf")
    x[1, 6:4200:7] *= 4.0
    bias = np.linspace(-0.1, 0.1, E).astype(np.float32)
    mask = (rng.uniform(size=(S, T)) < 0.5).astype(np.uint8)
    for b, m in ((None, None), (bias, None), (bias, mask)):
        f, got = check(S, T, E, K, dtype, scoring, b, m, logits=x, seed=14)
        assert np.isfinite(got).all()


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [600, 4200])
def test_long_logits(T, dtype, scoring):
    """Logits to some hundreds beside masked and special rows, with one and with several tokens per wave.

    A score's error is (2 * max|l| + 16) u, which is 64 u at |l| <= 24; a term of the gradient has at most four factors
    with that error (s, a score in a sum, s_k and 1 / D).  A score below the smallest normal value, 2^-126, may become
    0.  The chosen scores' sum D is above 1/2 here, so that moves a weight by at most 2.5 * 2^-126 * 2 < 2^-123, and a
    gradient, whose factors beside s are below 2.5 * 4.5 * 2 * 2 < 64, by at most 2^-120.
    """
    S, E, K = 2, 130, 6
    x, rng = make(S, T, E, dtype, 13)
    x[0, 0:T:7] = float("-inf")
    x[0, 1:T:7] = low_of(dtype)
    x[0, 2:T:7] = float("nan")
    x[0, 3:T:7, 4:] = float("-inf")
    x[0, 4:T:7, ::2] = float("nan")
    x[1, 5:T:7, 7] = float("inf")
    x[1, 6:T:7] *= 40.0
    top = float(x[1, 6:T:7].abs().max())
    assert 200 < top < 1000
    rel = (2 * top + 16) * U
    bias = np.linspace(-0.1, 0.1, E).astype(np.float32)
    mask = (rng.uniform(size=(S, T)) < 0.5).astype(np.uint8)
    for b, m in ((None, None), (bias, None), (bias, mask)):
        f, got = check(S, T, E, K, dtype, scoring, b, m, logits=x, seed=14, rel=rel, rel_grad=4 * rel, floor=2.0 ** -123,
                       floor_grad=2.0 ** -120)
        assert (f["D"][1, 6::7][f["there"][1, 6::7].any(1)] > 0.5).all()
        assert np.isfinite(got).all()


@pytest.mark.gpu
def test_many_tokens_on_unaligned_rows():
    for dtype in (torch.float32, torch.bfloat16):
        cfg = ep.make_route_config(1, 8200, 64, 4, "bf16" if dtype == torch.bfloat16 else "fp32")
        flat = torch.randn(8200 * 64 + 1, device="cuda").to(dtype)
        a, b = ep.alloc_route(cfg, balance=True), ep.alloc_route(cfg, balance=True)
        dw, dl = torch.randn((1, 8200, 4), device="cuda"), torch.ones(1, device="cuda")
        ep.ep_route(cfg, flat[1:], a)
        ep.ep_route(cfg, flat[1:].clone(), b)
        assert torch.equal(a.topk_idx, b.topk_idx) and torch.equal(a.topk_weights, b.topk_weights)
        assert torch.equal(a.balance_loss, b.balance_loss)
        ga, gb = torch.zeros_like(flat), torch.zeros_like(flat)
        ep.ep_route_backward(cfg, flat[1:], a, dw, dl, ga[1:])
        ep.ep_route_backward(cfg, flat[1:].clone(), b, dw, dl, gb)
        assert torch.equal(ga[1:], gb[:-1])


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,E", [(33, 64), (2050, 64), (500, 300), (8200, 300)])
def test_both_zeros_are_one_value(T, E, dtype, scoring):
    """-0 and +0 tie, with one and with several tokens per wave: the lowest index is chosen, whichever zero it holds."""
    rng = np.random.default_rng(T + E)
    x = torch.from_numpy(rng.choice(np.float32([0.0, -0.0, -1.0, 1.0]), size=(1, T, E), p=(0.4, 0.4, 0.19, 0.01)))
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    check(1, T, E, 8, dtype, scoring, logits=x, seed=15)
    x[:] = -1.0  # no other tie among the best
    x[:, :, 2], x[:, :, 5] = -0.0, 0.0
    check(1, T, E, 1, dtype, scoring, logits=x, seed=15)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [1, 3])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [64, 300])
def test_many_tokens_with_near_ties_around_a_bins_end(E, scoring, K):
    """Two experts of different scores and biases, whose keys lie within rounding of each other around 1.25, the end of
    a bin of 256 and of 512 steps of 2^-23, one of them the K-th, and an expert of a lower index well below both in the
    lower bin."""
    T, step = 8200, 2.0 ** -23
    rng = np.random.default_rng(E + K)
    l = np.full(E, -3.0)
    l[20:20 + K - 1] = 2.0  # clear winners
    near = [5, 9, 12]
    l[near] = 0.0, -0.7, 0.3
    s = 1 / (1 + np.exp(-l)) if scoring == "sigmoid" else np.exp(l) / np.exp(l).sum()
    bias = np.zeros(E, np.float32)
    bias[near] = 1.25 - s[near]
    bias[20:20 + K - 1] = 1.25
    # The scores that make the keys, steps above 1.25 with the biases as rounded, and their logits.
    want = 1.25 + np.stack([rng.uniform(lo, hi, T) for lo, hi in ((-200, -60), (-1, 1), (-1, 1))], 1) * step - bias[near]
    rest = np.exp(np.delete(l, near)).sum() / (1 - want.sum(1, keepdims=True))
    x = np.tile(l.astype(np.float32), (1, T, 1))
    x[0][:, near] = np.log(want / (1 - want)) if scoring == "sigmoid" else np.log(want * rest)
    check(1, T, E, K, "fp32", scoring, bias, logits=torch.from_numpy(x), seed=16)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,K", [(5, 1024, 1), (8200, 256, 2)])
def test_choice_where_the_softmax_sum_rounds_one_way(T, E, K):
    """The softmax sum 1 + n t, t just below half a step of 1, rounds to 1 in 32 bits when every addition meets one more
    t, n of them being as many as the additions after the lane that holds the 1.  The expert with bias 1 - n 2^-24 and
    score t is the better one by 2^-24, and behind by (n - 1) 2^-24 in 32 bits."""
    x = torch.full((1, T, E), float("-inf"))
    if E == 1024:  # 16 experts a lane, summed by a scan towards the last lane
        best, other, small = 1008, 0, list(range(1009, 1024)) + [16 * l for l in (62, 61, 59, 55, 47, 0)]
    else:          # 16 experts a lane of 16 lanes, folded by halves
        best, other, small = 0, 16, list(range(1, 16)) + [16 * l for l in (8, 4, 2, 1)]
    x[0, :, small] = float(np.log(U * (1 - 2.0 ** -9)))
    x[0, :, best] = 0.0
    bias = np.zeros(E, np.float32)
    bias[other] = 1 - len(small) * U
    f = plain(x.numpy(), K, "softmax", 1.0, bias, None, low_of("fp32"))
    assert (f["idx"][0, :, 0] == other).all()
    check(1, T, E, K, "fp32", "softmax", bias, logits=x, seed=17)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("S,T,E", [(256, 65536, 13), (128, 16384, 595)])
def test_balance_loss_of_long_sources(S, T, E, scoring):
    """Equal logits: every p is 1 / E and rounds the same way, so that a chain of 32-bit additions drifts.  All tokens
    choose expert 0, f_0 = E, and the loss is 1."""
    cfg = ep.make_route_config(S, T, E, 1, "bf16", scoring)
    r = ep.alloc_route(cfg, balance=True)
    ep.ep_route(cfg, torch.zeros((S, T, E), dtype=torch.bfloat16, device="cuda"), r)
    assert (r.topk_idx == 0).all() and (r.tokens_per_expert[:, 0] == T).all()
    assert ((r.balance_loss.double() - 1).abs() <= REL).all()


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [600, 8200])
def test_weights_of_long_logits_to_their_last_bits(T, scoring):
    """One logit near 80 beside others near 0: l - max loses bits of l in 32 bits.  A score's error does not grow with the
    logits: exp to 4 u, the division and the product with it 2 u, the sum over K of them K u more, the scale u."""
    S, E, K = 1, 200, 6
    rng = np.random.default_rng(T)
    x = rng.uniform(-1, 1, size=(S, T, E)).astype(np.float32)
    if scoring == "sigmoid":
        x -= 40.0
    top = rng.integers(0, E, size=T)
    x[0, np.arange(T), top] += np.float32(80.0)
    f = plain(x, K, scoring, 2.5, None, None, low_of("fp32"))
    cfg = ep.make_route_config(S, T, E, K, "fp32", scoring, 2.5)
    r = ep.alloc_route(cfg)
    ep.ep_route(cfg, torch.from_numpy(x).cuda(), r)
    w = r.topk_weights.cpu().numpy()
    assert (r.topk_idx.cpu().numpy() == f["idx"]).all()
    within(np.abs(w - f["w"]), 24 * U * f["w"])
