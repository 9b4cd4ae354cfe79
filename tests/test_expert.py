"""The experts' products (ep_expert_mm, ep_expert_mm_backward) against plain 64-bit products, and their refusals.

Tolerances.  A product of two bf16 (or e4m3) values is exact in fp32; a sum of k of them is off by at most 2 k u of the
sum of magnitudes (u = 2^-24, a matrix unit's step rounds once or truncates: 2u).  fp8 adds the scales' product and one
multiply-add per 128 elements: 4 u.  The activations are Lipschitz with a constant below 1.13 and computed to 16 u of
their terms; out and pre are rounded to bf16 once: half a step, 2^-8 of the value.  The backward pass rounds d to bf16
before its products: 2^-8 of every term in the worst case, and, since these roundings are independent, no more than
2^-8 of the result's norm beside the result's own 2^-8.
"""
import ctypes

import numpy as np
import pytest
import torch

import combine_ep_layout_07_amd.ep as ep

U = 2.0 ** -24
H = 2.0 ** -8
BAD, UNSUP = ep.EP_ERR_INVALID_ARG, ep.EP_ERR_UNSUPPORTED


# ------------------------------------------------------------------------------------------------------------ refusals

@pytest.mark.parametrize("kw,code", [
    (dict(E=0), BAD), (dict(rows=-1), BAD), (dict(I=0), BAD), (dict(N=0), BAD), (dict(E=1025), UNSUP),
    (dict(I=12), UNSUP), (dict(N=12), UNSUP), (dict(I=262152), UNSUP), (dict(N=262152), UNSUP),
    (dict(rows=2 ** 31), UNSUP), (dict(I=64, dtype="fp8"), UNSUP), (dict(I=128, N=8, dtype="fp8"), ep.EP_OK),
    (dict(E=1024, I=262144, N=262144, rows=2 ** 31 - 1), ep.EP_OK), (dict(rows=0), ep.EP_OK),
])
def test_configuration_codes(kw, code):
    base = dict(E=4, rows=10, I=64, N=32)
    base.update(kw)
    cfg = ep.make_expert_config(**base)
    sz = ep.EpExpertSizes()
    assert ep._lib.ep_query_expert_sizes(ctypes.byref(cfg), ctypes.byref(sz)) == code
    if code != ep.EP_OK:
        assert ep._lib.ep_expert_mm(ctypes.byref(cfg), *[None] * 10) == code
        assert ep._lib.ep_expert_mm_backward(ctypes.byref(cfg), *[None] * 10) == code
        with pytest.raises(ep.EpError):
            ep.alloc_expert_backward(cfg)


def test_configuration_fields():
    for field, value in (("x_dtype", ep.EP_DTYPE_FP32), ("activation", 5), ("activation", -1), ("reserved", 1)):
        cfg = ep.make_expert_config(4, 10, 64, 32)
        setattr(cfg, field, value)
        assert ep._lib.ep_query_expert_sizes(ctypes.byref(cfg), ctypes.byref(ep.EpExpertSizes())) == BAD
    for kw in (dict(dtype="fp32"), dict(activation="tanh")):
        with pytest.raises(ValueError):
            ep.make_expert_config(4, 10, 64, 32, **kw)
    assert ep._lib.ep_query_expert_sizes(None, None) == BAD
    sz = ep.ep_query_expert_sizes(ep.make_expert_config(3, 10, 256, 136, dtype="fp8", activation="swiglu"))
    assert (sz.x, sz.x_sf, sz.w, sz.w_sf) == (2560, 80, 3 * 272 * 256, 3 * 3 * 2 * 4)
    assert (sz.bias, sz.out, sz.pre, sz.backward_scratch) == (3 * 272 * 4, 2720, 5440, 0)


@pytest.mark.skipif(torch.cuda.is_available(), reason="passes fake device addresses; host-only check")
def test_pointer_codes():
    f = 0x10000
    cfg = ep.make_expert_config(4, 10, 64, 32, activation="silu")

    def mm(c, *p):
        return ep._lib.ep_expert_mm(ctypes.byref(c), *p, None)
    ok = [f, f, None, f, None, f, f, f, f]  # base, x, x_sf, w, w_sf, bias, residual, out, pre
    for i, off in ((0, 2), (1, 8), (3, 8), (5, 8), (6, 8), (7, 8), (8, 8)):
        p = list(ok)
        p[i] = f + off
        assert mm(cfg, *p) == BAD, i
        p[i] = None
        if i in (0, 1, 3, 7):
            assert mm(cfg, *p) == BAD, i
    for i in (2, 4):  # scales with bf16 rows
        p = list(ok)
        p[i] = f
        assert mm(cfg, *p) == BAD
    fp8 = ep.make_expert_config(4, 10, 128, 32, dtype="fp8")
    for sf in ((None, f), (f, None), (f + 2, f), (f, f + 2)):
        assert mm(fp8, f, f, sf[0], f, sf[1], None, None, f, None) == BAD

    def back(c, *p):
        return ep._lib.ep_expert_mm_backward(ctypes.byref(c), *p, None)
    ok = [f] * 9  # base, x, w, pre, d_out, d_x, d_w, d_bias, scratch
    for i in range(9):
        p = list(ok)
        p[i] = f + 2
        assert back(cfg, *p) == BAD, i
        p[i] = None
        if i in (0, 1, 2, 3, 4, 8):
            assert back(cfg, *p) == BAD, i
    assert back(cfg, f, f, f, f, f, None, None, None, f) == BAD
    assert back(fp8, *ok) == UNSUP


def test_binding_refuses():
    cfg = ep.make_expert_config(2, 4, 64, 32)
    b, x, w = torch.zeros(3, dtype=torch.int32), torch.zeros((4, 64)).bfloat16(), torch.zeros((2, 32, 64)).bfloat16()
    o = torch.zeros((4, 32)).bfloat16()
    with pytest.raises(ValueError, match="expert_base must be int32"):
        ep.ep_expert_mm(cfg, b.long(), x, w, o)
    with pytest.raises(ValueError, match="x must have 2-byte"):
        ep.ep_expert_mm(cfg, b, x.float(), w, o)
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_expert_mm(cfg, b, x, w, o)
    with pytest.raises(ValueError, match="d_out must have 2-byte"):
        ep.ep_expert_mm_backward(cfg, b, x, w, o.float(), o)


# ------------------------------------------------------------------------------------------------- the 64-bit formulas

def phi(v):
    return 0.5 * torch.special.erfc(-v / np.sqrt(2.0))


def act64(act, p, N):
    if act == "none":
        return p
    if act == "relu":
        return p.clamp(min=0)
    if act == "gelu":
        return p * phi(p)
    if act == "silu":
        return p * torch.sigmoid(p)
    return p[:, :N] * torch.sigmoid(p[:, :N]) * p[:, N:]


def slope64(act, p, d, N):
    if act == "none":
        return d
    if act == "relu":
        return torch.where(p > 0, d, 0.0)
    if act == "gelu":
        return d * (phi(p) + p * torch.exp(-0.5 * p * p) / np.sqrt(2 * np.pi))
    g = p if act == "silu" else p[:, :N]
    s = torch.sigmoid(g)
    slope = s * (1 + g * (1 - s))
    return d * slope if act == "silu" else torch.cat([d * p[:, N:] * slope, d * g * s], 1)


def cols_of(N, act):
    return 2 * N if act == "swiglu" else N


def make(counts, I, N, act, seed, first=0, spare=3):
    """Rows in the experts' segments, `first` rows before them and `spare` after."""
    g = torch.Generator().manual_seed(seed)
    E, Nw = len(counts), cols_of(N, act)
    base = first + np.concatenate([[0], np.cumsum(counts)])
    rows = int(base[-1]) + spare
    x = torch.randn((rows, I), generator=g).bfloat16()
    w = (torch.randn((E, Nw, I), generator=g) * I ** -0.5).bfloat16()
    return base, rows, x, w, g


def product64(base, x, w, bias):
    """pre of the grouped rows in 64 bits, and the sums of magnitudes."""
    pre, mag = [], []
    for e in range(len(base) - 1):
        a, we = x[base[e]:base[e + 1]].double(), w[e].double()
        p, m = a @ we.T, a.abs() @ we.abs().T
        if bias is not None:
            p, m = p + bias[e].double(), m + bias[e].double().abs()
        pre.append(p)
        mag.append(m)
    return torch.cat(pre), torch.cat(mag)


def out_error(act, p, mag, k, N):
    """Bound on the error of act(pre) before its rounding."""
    e = 2 * k * U * mag
    if act != "swiglu":
        return 1.13 * e + 16 * U * p.abs()
    g, u, eg, eu = p[:, :N], p[:, N:], e[:, :N], e[:, N:]
    return 1.13 * eg * (u.abs() + eu) + (g.abs() + eg) * eu + 16 * U * (g * u).abs()


def dev(t):
    return None if t is None else t.cuda()


COUNTS = {
    "one": [1], "few": [1, 0, 3, 2], "holes": [0, 0, 17, 0, 64, 65, 1, 0], "mid": [40, 33, 70, 16, 15, 31],
    "large": [300, 0, 513, 129, 257], "skew": [700, 3, 0, 1, 90], "many": [k % 7 for k in range(130)], "empty": [0, 0],
}
FORWARD = [  # counts, I, N, act, bias, residual, pre
    ("one", 8, 8, "none", False, False, False), ("one", 7168, 72, "swiglu", True, True, True),
    ("few", 72, 24, "gelu", True, False, True), ("few", 2048, 264, "none", True, True, False),
    ("holes", 136, 40, "silu", False, True, True), ("holes", 520, 136, "swiglu", True, True, True),
    ("mid", 1000, 248, "relu", True, True, False), ("mid", 512, 392, "swiglu", False, False, False),
    ("large", 200, 296, "gelu", True, True, True), ("large", 1160, 520, "swiglu", True, False, True),
    ("skew", 264, 264, "none", False, True, True), ("many", 264, 136, "swiglu", True, False, True),
    ("empty", 64, 64, "silu", True, True, True), ("large", 64, 8, "none", False, False, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("counts,I,N,act,bias,residual,pre", FORWARD)
def test_forward(counts, I, N, act, bias, residual, pre):
    print(f"[expert_mm] {counts} I={I} N={N} {act}", flush=True)
    c = COUNTS[counts]
    base, rows, x, w, g = make(c, I, N, act, 5, first=2)
    E, Nw = len(c), cols_of(N, act)
    b = torch.randn((E, Nw), generator=g) if bias else None
    res = torch.randn((rows, N), generator=g).bfloat16() if residual else None
    out = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    kept = torch.full((rows, Nw), 7.0, dtype=torch.bfloat16, device="cuda") if pre else None
    cfg = ep.make_expert_config(E, rows, I, N, activation=act)
    bd = torch.tensor(base, dtype=torch.int32).cuda()
    ep.ep_expert_mm(cfg, bd, dev(x), dev(w), out, bias=dev(b), residual=dev(res), pre=kept)
    torch.cuda.synchronize()
    check_forward(base, out, kept, *product64(base, x, w, b), I, N, act, res)


def check_forward(base, out, kept, p, mag, k, N, act, res):
    lo, hi = base[0], base[-1]
    got = out.cpu().double()
    assert (got[:lo] == 7).all() and (got[hi:] == 7).all()
    want, err = act64(act, p, N), out_error(act, p, mag, k, N)
    if res is not None:
        want = want + res[lo:hi].double()
        err = err + U * want.abs()
    assert (torch.abs(got[lo:hi] - want) <= H * want.abs() + err * (1 + H)).all()
    if kept is not None:
        got = kept.cpu().double()
        assert (got[:lo] == 7).all() and (got[hi:] == 7).all()
        assert (torch.abs(got[lo:hi] - p) <= H * p.abs() + 2 * k * U * mag * (1 + H)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("counts,I,N,act,bias", [
    ("one", 128, 8, "none", False), ("few", 7168, 200, "swiglu", True), ("holes", 256, 136, "silu", True),
    ("mid", 640, 128, "swiglu", False), ("large", 384, 264, "gelu", True), ("large", 896, 192, "swiglu", False),
    ("many", 128, 72, "none", True)])
def test_forward_fp8(counts, I, N, act, bias):
    print(f"[expert_mm fp8] {counts} I={I} N={N} {act}", flush=True)
    c = COUNTS[counts]
    base, rows, x, w, g = make(c, I, N, act, 6)
    E, Nw = len(c), cols_of(N, act)
    x8, w8 = x.to(torch.float8_e4m3fn), (w.float() * I ** 0.5).to(torch.float8_e4m3fn)
    xs = torch.exp(torch.randn((rows, I // 128), generator=g))
    ws = torch.exp(torch.randn((E, -(-Nw // 128), I // 128), generator=g)) * I ** -0.5
    b = torch.randn((E, Nw), generator=g) if bias else None
    out = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    kept = torch.full((rows, Nw), 7.0, dtype=torch.bfloat16, device="cuda")
    cfg = ep.make_expert_config(E, rows, I, N, dtype="fp8", activation=act)
    ep.ep_expert_mm(cfg, torch.tensor(base, dtype=torch.int32).cuda(), x8.cuda(), w8.cuda(), out, x_sf=xs.cuda(),
                    w_sf=ws.cuda(), bias=dev(b), pre=kept)
    torch.cuda.synchronize()
    x64 = x8.double() * xs.double().repeat_interleave(128, 1)
    w64 = w8.double() * ws.double().repeat_interleave(128, 2).repeat_interleave(128, 1)[:, :Nw]
    check_forward(base, out, kept, *product64(base, x64, w64, b), I + 4, N, act, None)


BACKWARD = [  # counts, I, N, act, bias
    ("one", 8, 8, "none", True), ("few", 72, 24, "gelu", True), ("holes", 136, 40, "silu", True),
    ("holes", 520, 136, "swiglu", True), ("mid", 1000, 248, "relu", False), ("mid", 264, 392, "swiglu", True),
    ("large", 200, 296, "gelu", True), ("large", 520, 264, "swiglu", False), ("skew", 264, 520, "none", True),
    ("many", 264, 136, "swiglu", True), ("empty", 64, 64, "silu", True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("counts,I,N,act,bias", BACKWARD)
def test_backward(counts, I, N, act, bias):
    print(f"[expert_mm_backward] {counts} I={I} N={N} {act}", flush=True)
    c = COUNTS[counts]
    base, rows, x, w, g = make(c, I, N, act, 7, first=1)
    E, Nw = len(c), cols_of(N, act)
    pre = torch.randn((rows, Nw), generator=g).bfloat16() if act != "none" else None
    d_out = torch.randn((rows, N), generator=g).bfloat16()
    # Rows outside the segments hold what must not reach any sum.
    for t in (x, d_out) + ((pre,) if pre is not None else ()):
        t[:base[0]] = float("nan")
        t[base[-1]:] = float("inf")
    cfg = ep.make_expert_config(E, rows, I, N, activation=act)
    bd = torch.tensor(base, dtype=torch.int32).cuda()
    dx = torch.full((rows, I), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((E, Nw, I), 7.0, dtype=torch.bfloat16, device="cuda")
    db = torch.full((E, Nw), 7.0, device="cuda") if bias else None
    scratch = ep.alloc_expert_backward(cfg)
    args = (cfg, bd, dev(x), dev(w), dev(d_out), scratch)
    ep.ep_expert_mm_backward(*args, pre=dev(pre), d_x=dx, d_w=dw, d_bias=db)
    torch.cuda.synchronize()
    gx, gw = dx.cpu().double(), dw.cpu().double()
    assert (gx[:base[0]] == 7).all() and (gx[base[-1]:] == 7).all()
    n2 = [0.0, 0.0, 0.0, 0.0]
    for e in range(E):
        s = slice(int(base[e]), int(base[e + 1]))
        n = s.stop - s.start
        d = slope64(act, None if pre is None else pre[s].double(), d_out[s].double(), N)
        d_err = 16 * U * terms64(act, None if pre is None else pre[s].double(), d_out[s].double(), N)
        dmag = d.abs() * (1 + H) + d_err
        want, mag = d @ w[e].double(), dmag @ w[e].double().abs()
        assert (torch.abs(gx[s] - want) <= H * want.abs() + (1 + H) * (H + 2 * Nw * U) * mag + (1 + H) * d_err @ w[e].double().abs()).all()
        n2[0], n2[1] = n2[0] + ((gx[s] - want) ** 2).sum(), n2[1] + (want ** 2).sum()
        want, mag = d.T @ x[s].double(), dmag.T @ x[s].double().abs()
        assert (torch.abs(gw[e] - want) <= H * want.abs() + (1 + H) * (H + 2 * n * U) * mag + (1 + H) * d_err.T @ x[s].double().abs()).all()
        n2[2], n2[3] = n2[2] + ((gw[e] - want) ** 2).sum(), n2[3] + (want ** 2).sum()
        if bias:
            assert (torch.abs(db[e].cpu().double() - d.sum(0)) <= ((n + 16) * U * dmag + d_err).sum(0)).all()
    assert n2[0] <= (2 * H) ** 2 * n2[1] and n2[2] <= (2 * H) ** 2 * n2[3]
    # each gradient alone, without what it does not need
    dx2, dw2 = torch.full_like(dx, 7.0), torch.empty_like(dw)
    ep.ep_expert_mm_backward(cfg, bd, None, args[3], args[4], scratch, pre=dev(pre), d_x=dx2)
    ep.ep_expert_mm_backward(*args, pre=dev(pre), d_w=dw2)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)
    if bias:
        db2 = torch.empty_like(db)
        ep.ep_expert_mm_backward(cfg, bd, None, args[3], args[4], scratch, pre=dev(pre), d_bias=db2)
        assert torch.equal(db2, db)


def terms64(act, p, d, N):
    """Sums of the magnitudes of the terms of act'(pre) d."""
    if act in ("none", "relu"):
        return torch.zeros_like(d)
    if act != "swiglu":
        return d.abs() * (1 + p.abs())
    return torch.cat([d.abs() * p[:, N:].abs() * (1 + p[:, :N].abs()), d.abs() * p[:, :N].abs()], 1)


# Sizes at which the tiles of 256 x 256 and of 128 x 128 are the cheapest; 64-bit products on the GPU.
LARGE = [([3001, 0, 1999], 2056, 1032, "swiglu"), ([1500, 2500], 520, 1032, "gelu"), ([1500, 2500], 1032, 520, "silu")]


@pytest.mark.gpu
@pytest.mark.parametrize("counts,I,N,act", LARGE)
def test_large(counts, I, N, act):
    print(f"[expert_mm large] {counts} I={I} N={N} {act}", flush=True)
    base, rows, x, w, g = make(counts, I, N, act, 21, first=3)
    E, Nw = len(counts), cols_of(N, act)
    b = torch.randn((E, Nw), generator=g)
    res = torch.randn((rows, N), generator=g).bfloat16()
    d = torch.randn((rows, N), generator=g).bfloat16()
    for t in (x, d):  # rows outside the segments
        t[:base[0]] = float("nan")
        t[base[-1]:] = float("inf")
    xd, wd, bd, dd = x.cuda(), w.cuda(), b.cuda(), d.cuda()
    bt = torch.tensor(base, dtype=torch.int32).cuda()
    cfg = ep.make_expert_config(E, rows, I, N, activation=act)
    out = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    pre = torch.full((rows, Nw), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_mm(cfg, bt, xd, wd, out, bias=bd, residual=res.cuda(), pre=pre)
    p, mag = (t.cpu() for t in product64(base, xd, wd, bd))
    check_forward(base, out, pre, p, mag, I, N, act, res)
    dx, dw, db = torch.full_like(xd, 7.0), torch.full_like(wd, 7.0), torch.empty((E, Nw), device="cuda")
    ep.ep_expert_mm_backward(cfg, bt, xd, wd, dd, ep.alloc_expert_backward(cfg), pre=pre, d_x=dx, d_w=dw, d_bias=db)
    assert (dx[:base[0]] == 7).all() and (dx[base[-1]:] == 7).all()
    for e in range(E):
        s = slice(int(base[e]), int(base[e + 1]))
        n, pe, de = s.stop - s.start, pre[s].double(), dd[s].double()
        grad = slope64(act, pe, de, N)
        err = 16 * U * terms64(act, pe, de, N)
        m = grad.abs() * (1 + H) + err
        want, bound = grad @ wd[e].double(), (H + 2 * Nw * U) * (m @ wd[e].double().abs()) + err @ wd[e].double().abs()
        assert (torch.abs(dx[s].double() - want) <= H * want.abs() + (1 + H) * bound).all()
        assert n == 0 or (dx[s].double() - want).norm() <= 2 * H * want.norm()
        xe = x[s].cuda().double()
        want, bound = grad.T @ xe, (H + 2 * n * U) * (m.T @ xe.abs()) + err.T @ xe.abs()
        assert (torch.abs(dw[e].double() - want) <= H * want.abs() + (1 + H) * bound).all()
        assert n == 0 or (dw[e].double() - want).norm() <= 2 * H * want.norm()
        assert (torch.abs(db[e].double() - grad.sum(0)) <= ((n + 16) * U * m + err).sum(0)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("counts,I,N,act", [([3001, 0, 1999], 768, 1032, "swiglu"), ([3001, 0, 1999], 2432, 1040, "none"),
                                            ([1500, 2500], 1024, 1032, "silu"), ([700, 1800], 1152, 520, "swiglu")])
def test_large_fp8(counts, I, N, act):
    print(f"[expert_mm large fp8] {counts} I={I} N={N} {act}", flush=True)
    base, rows, x, w, g = make(counts, I, N, act, 22, first=1)
    E, Nw = len(counts), cols_of(N, act)
    x8, w8 = x.to(torch.float8_e4m3fn), (w.float() * I ** 0.5).to(torch.float8_e4m3fn)
    xs = torch.exp(torch.randn((rows, I // 128), generator=g))
    ws = torch.exp(torch.randn((E, -(-Nw // 128), I // 128), generator=g)) * I ** -0.5
    out = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    kept = torch.full((rows, Nw), 7.0, dtype=torch.bfloat16, device="cuda")
    cfg = ep.make_expert_config(E, rows, I, N, dtype="fp8", activation=act)
    ep.ep_expert_mm(cfg, torch.tensor(base, dtype=torch.int32).cuda(), x8.cuda(), w8.cuda(), out, x_sf=xs.cuda(),
                    w_sf=ws.cuda(), pre=kept)
    x64 = x8.double() * xs.double().repeat_interleave(128, 1)
    w64 = w8.double() * ws.double().repeat_interleave(128, 2).repeat_interleave(128, 1)[:, :Nw]
    p, mag = (t.cpu() for t in product64(base, x64.cuda(), w64.cuda(), None))
    check_forward(base, out, kept, p, mag, I + 4, N, act, None)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "gelu", "silu", "swiglu"])
def test_gradient_against_differences(act):
    """Central differences of the 64-bit objective sum(out * d) along a random direction; the step's own error is of
    the order step^2 of the third derivative's terms, below 1e-6 of the sum of magnitudes."""
    c, I, N = [5, 0, 40, 19], 72, 56
    base, rows, x, w, g = make(c, I, N, act, 8, spare=0)
    E, Nw = len(c), cols_of(N, act)
    b = torch.randn((E, Nw), generator=g)
    d = torch.randn((rows, N), generator=g).bfloat16()
    vx, vw, vb = (torch.randn(t.shape, generator=g).double() for t in (x, w, b))

    def objective(x, w, b):
        return (act64(act, product64(base, x, w, b)[0], N) * d.double()).sum()
    h = 1e-4
    want = (objective(x.double() + h * vx, w.double() + h * vw, b.double() + h * vb) -
            objective(x.double() - h * vx, w.double() - h * vw, b.double() - h * vb)) / (2 * h)
    cfg = ep.make_expert_config(E, rows, I, N, activation=act)
    bd = torch.tensor(base, dtype=torch.int32).cuda()
    out = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    pre = torch.empty((rows, Nw), dtype=torch.bfloat16, device="cuda")
    xd, wd = x.cuda(), w.cuda()
    ep.ep_expert_mm(cfg, bd, xd, wd, out, bias=b.cuda(), pre=pre)
    dx, dw, db = torch.empty_like(xd), torch.empty_like(wd), torch.empty((E, Nw), device="cuda")
    ep.ep_expert_mm_backward(cfg, bd, xd, wd, d.cuda(), ep.alloc_expert_backward(cfg), pre=pre, d_x=dx, d_w=dw, d_bias=db)
    terms = torch.cat([(a.cpu().double() * v).reshape(-1) for a, v in ((dx, vx), (dw, vw), (db, vb))])
    # Roundings: pre and d to bf16 and the gradients, each 2^-8 of its terms.
    assert (terms.sum() - want).abs() <= 3 * H * terms.abs().sum()


@pytest.mark.gpu
def test_special_values_stay_in_their_rows():
    """NaN and infinities of one row, or of one expert's weights, reach that row or expert only."""
    c, I, N = [20, 300, 5], 264, 136
    base, rows, x, w, g = make(c, I, N, "none", 9, spare=0)
    cfg = ep.make_expert_config(3, rows, I, N)
    bd = torch.tensor(base, dtype=torch.int32).cuda()
    clean, out = (torch.empty((rows, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ep.ep_expert_mm(cfg, bd, x.cuda(), w.cuda(), clean)
    x2, w2 = x.clone(), w.clone()
    x2[7, 100] = float("nan")
    x2[200, 3] = float("inf")
    w2[2, 50, 260] = float("nan")
    ep.ep_expert_mm(cfg, bd, x2.cuda(), w2.cuda(), out)
    keep = torch.ones((rows, N), dtype=torch.bool)
    keep[7] = keep[200] = False
    keep[320:, 50] = False
    assert torch.equal(out.cpu()[keep], clean.cpu()[keep])
    assert out.cpu()[7].isnan().all() and not out.cpu()[200].isfinite().any() and out.cpu()[320:, 50].isnan().all()
    # the gradient of the weights: a row's NaN reaches its own expert only
    d = torch.randn((rows, N), generator=g).bfloat16()
    dw = torch.empty((3, N, I), dtype=torch.bfloat16, device="cuda")
    dw2 = torch.empty_like(dw)
    s = ep.alloc_expert_backward(cfg)
    ep.ep_expert_mm_backward(cfg, bd, x.cuda(), w.cuda(), d.cuda(), s, d_w=dw)
    ep.ep_expert_mm_backward(cfg, bd, x2.cuda(), w.cuda(), d.cuda(), s, d_w=dw2)
    same = torch.ones((3, N, I), dtype=torch.bool)
    same[0, :, 100] = same[1, :, 3] = False
    assert torch.equal(dw.cpu()[same], dw2.cpu()[same]) and dw2.cpu()[0, :, 100].isnan().all()


@pytest.mark.gpu
def test_table_outside_the_rows():
    """Entries below zero and past the rows are taken as the nearest row."""
    I, N, rows = 64, 72, 50
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn((rows, I), generator=g).bfloat16().cuda(), torch.randn((3, N, I), generator=g).bfloat16().cuda()
    cfg = ep.make_expert_config(3, rows, I, N)
    outs = []
    for base in ([-5, 20, 30, 99], [0, 20, 30, 50]):
        out = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
        dw = torch.empty((3, N, I), dtype=torch.bfloat16, device="cuda")
        bd = torch.tensor(base, dtype=torch.int32).cuda()
        ep.ep_expert_mm(cfg, bd, x, w, out)
        ep.ep_expert_mm_backward(cfg, bd, x, w, out, ep.alloc_expert_backward(cfg), d_w=dw)
        outs.append((out, dw))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.gpu
def test_stream_and_graph():
    """On a stream of its own, and replayed from a graph with eager work between; all bitwise alike."""
    c, I, N, act = [33, 0, 140, 7], 200, 104, "swiglu"
    base, rows, x, w, g = make(c, I, N, act, 11, spare=0)
    cfg = ep.make_expert_config(len(c), rows, I, N, activation=act)
    bd, xd, wd = torch.tensor(base, dtype=torch.int32).cuda(), x.cuda(), w.cuda()
    d = torch.randn((rows, N), generator=g).bfloat16().cuda()
    scratch = ep.alloc_expert_backward(cfg)

    def buffers():
        e = dict(dtype=torch.bfloat16, device="cuda")
        return [torch.empty((rows, N), **e), torch.empty((rows, 2 * N), **e), torch.empty((rows, I), **e),
                torch.empty((len(c), 2 * N, I), **e), torch.empty((len(c), 2 * N), device="cuda")]

    def step(b):
        ep.ep_expert_mm(cfg, bd, xd, wd, b[0], pre=b[1])
        ep.ep_expert_mm_backward(cfg, bd, xd, wd, d, scratch, pre=b[1], d_x=b[2], d_w=b[3], d_bias=b[4])
    first, other, kept = buffers(), buffers(), buffers()
    step(first)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step(other)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(kept)
    for _ in range(4):
        for t in kept:
            t.fill_(3.0)
        graph.replay()
        step(other)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(first, kept)) and all(torch.equal(p, q) for p, q in zip(first, other))


@pytest.mark.gpu
def test_residual_in_place():
    c, I, N = [10, 200], 136, 72
    base, rows, x, w, g = make(c, I, N, "silu", 12, spare=0)
    cfg = ep.make_expert_config(2, rows, I, N, activation="silu")
    bd, xd, wd = torch.tensor(base, dtype=torch.int32).cuda(), x.cuda(), w.cuda()
    r = torch.randn((rows, N), generator=g).bfloat16().cuda()
    out = torch.empty_like(r)
    ep.ep_expert_mm(cfg, bd, xd, wd, out, residual=r)
    ep.ep_expert_mm(cfg, bd, xd, wd, r, residual=r)
    assert torch.equal(out, r)


@pytest.mark.gpu
def test_no_rows():
    cfg = ep.make_expert_config(2, 0, 64, 32, activation="gelu")
    z = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((2, 32, 64), dtype=torch.bfloat16, device="cuda")
    o = torch.zeros((0, 32), dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(3, dtype=torch.int32, device="cuda")
    dw, db = torch.ones_like(w), torch.ones((2, 32), device="cuda")
    ep.ep_expert_mm(cfg, b, z, w, o)
    ep.ep_expert_mm_backward(cfg, b, z, w, o, ep.alloc_expert_backward(cfg), pre=o, d_x=z, d_w=dw, d_bias=db)
    assert (dw == 0).all() and (db == 0).all()


@pytest.mark.gpu
def test_gelu_in_its_tail():
    """v Phi(v) and its slope to a few u of their own size, down to where Phi leaves the normal numbers.

    exp(-v^2 / 2) has the roundings of v^2, of its product with a constant and of that constant, each u of an exponent
    v^2 / 2: 1.5 v^2 u; everything else (the tail's polynomial, the reciprocal, exp2, a few products) is below 24 u."""
    v = torch.linspace(-13.0, 13.0, 417).bfloat16()
    n = len(v)
    x = torch.zeros((n, 8)).bfloat16()
    x[:, 0] = v
    w = torch.zeros((1, 8, 8)).bfloat16()
    w[:, :, 0] = 1.0
    v64 = v.double()
    tol = (1.5 * v64 * v64 + 24) * U
    cfg = ep.make_expert_config(1, n, 8, 8, activation="gelu")
    out = torch.empty((n, 8), dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_mm(cfg, torch.tensor([0, n], dtype=torch.int32).cuda(), x.cuda(), w.cuda(), out)
    want = v64 * phi(v64)
    assert ((out.cpu().double()[:, 0] - want).abs() <= (H + tol * (1 + H)) * want.abs()).all()
    # one row per expert: d_bias is the slope itself
    cfg = ep.make_expert_config(n, n, 8, 8, activation="gelu")
    base = torch.arange(n + 1, dtype=torch.int32).cuda()
    pre, one = v[:, None].expand(n, 8).contiguous().cuda(), torch.ones((n, 8), dtype=torch.bfloat16, device="cuda")
    db = torch.empty((n, 8), device="cuda")
    ep.ep_expert_mm_backward(cfg, base, None, torch.zeros((n, 8, 8), dtype=torch.bfloat16, device="cuda"), one,
                             ep.alloc_expert_backward(cfg), pre=pre, d_bias=db)
    bell = v64 * torch.exp(-0.5 * v64 * v64) / np.sqrt(2 * np.pi)
    want, mag = phi(v64) + bell, phi(v64) + bell.abs()
    assert ((db.cpu().double()[:, 0] - want).abs() <= tol * mag).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "swiglu"])
def test_silu_in_its_tail(act):
    """v / (1 + exp(-v)) where exp(v) is below the normal numbers but the product is not, or hardly.  exp(v) has the
    roundings of an exponent |v| (2 |v| u) and two of half a step of 2^-149, which v multiplies."""
    v = torch.arange(-91.5, -80.0, 0.5).bfloat16()
    n = len(v)
    x = torch.zeros((n, 8)).bfloat16()
    x[:, 0], x[:, 1] = v, 1.0
    w = torch.zeros((1, cols_of(8, act), 8)).bfloat16()
    w[:, :8, 0] = 1.0
    w[:, 8:, 1] = 1.0
    cfg = ep.make_expert_config(1, n, 8, 8, activation=act)
    out = torch.empty((n, 8), dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_mm(cfg, torch.tensor([0, n], dtype=torch.int32).cuda(), x.cuda(), w.cuda(), out)
    v64 = v.double()
    want = v64 * torch.exp(v64)
    assert (want.abs() >= 2.0 ** -126).all()
    tol = (H + (2 * v64.abs() + 16) * U * (1 + H)) * want.abs() + v64.abs() * 2.0 ** -149 * (1 + H)
    assert ((out.cpu().double()[:, 0] - want).abs() <= tol).all()


@pytest.mark.gpu
def test_no_rows_and_their_gradient_alone():
    cfg = ep.make_expert_config(2, 0, 64, 32, activation="gelu")
    z = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((2, 32, 64), dtype=torch.bfloat16, device="cuda")
    o = torch.zeros((0, 32), dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(3, dtype=torch.int32, device="cuda")
    ep.ep_expert_mm_backward(cfg, b, None, w, o, ep.alloc_expert_backward(cfg), pre=o, d_x=z)


def test_no_gradient_wanted():
    """Refused with rows; without any, an empty d_x has no address, and there is nothing to do."""
    f = 0x10000
    for rows, code in ((10, BAD), (0, ep.EP_OK)):
        cfg = ep.make_expert_config(2, rows, 64, 32)
        assert ep._lib.ep_expert_mm_backward(ctypes.byref(cfg), f, f, f, None, f, None, None, None, f, None) == code


@pytest.mark.gpu
def test_table_that_decreases_stays_inside():
    """Every second of 1024 experts claims all of 80 million rows: their tiles together pass 2^31, and the sums of the
    experts past the partial sums that there are read nothing."""
    E, rows, N = 1024, 80_000_000, 8
    cfg = ep.make_expert_config(E, rows, 8, N)
    base = torch.tensor([0, rows] * (E // 2) + [0], dtype=torch.int32).cuda()
    d_out = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
    d_out[rows - 1] = 1.0
    db = torch.full((E, N), 7.0, device="cuda")
    w = torch.zeros((E, N, 8), dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_mm_backward(cfg, base, None, w, d_out, ep.alloc_expert_backward(cfg), d_bias=db)
    torch.cuda.synchronize()
    assert (db[0] == 1).all() and (db[1:] == 0).all()


# Sizes whose tiles (forward, d_x, d_w) those above leave out: ungated tiles of 256 x 256 with a tail of k, each
# gradient in wide tiles beside the other in smaller ones, 128 x 128 tiles over more experts than lanes, and fp8 over
# more steps than two of the scales' buffers hold.
TILES = [([1500, 2500], 2440, 2056, "silu", (256, 256, 256)), ([2001, 0, 2000], 2432, 2056, "none", (256, 256, 128)),
         ([800, 700], 2432, 2056, "relu", (64, 64, 256)),
         ([k * 37 % 190 for k in range(70)], 1032, 520, "gelu", (128, 128, 128))]
TILES_FP8 = [([1500, 2500], 2432, 2056, "none", 256), ([2001, 0, 2000], 2176, 1160, "swiglu", 256),
             ([1500, 2500], 2304, 520, "swiglu", 128), ([800, 700], 2432, 2056, "silu", 64)]


def test_tiles_of_the_large_tests():
    """The sizes tested take the tiles they are there for."""
    def tiles(counts, I, N, act, dtype="bf16"):
        t = ep.ep_query_expert_tiles(ep.make_expert_config(len(counts), sum(counts) + 5, I, N, dtype, act))
        return t.forward, t.d_x, t.d_w
    assert [tiles(*t) for t in LARGE] == [(256, 256, 256), (128, 64, 128), (64, 128, 128)]
    for t in TILES:
        assert tiles(*t[:4]) == t[4]
    for t in TILES_FP8:
        assert tiles(*t[:4], dtype="fp8") == (t[4], 0, 0)
    assert tiles([1, 0, 3, 2], 7168, 200, "swiglu", "fp8") == (32, 0, 0)
    none = ep.ep_query_expert_tiles(ep.make_expert_config(4, 0, 64, 32))
    assert (none.forward, none.d_x, none.d_w) == (0, 0, 0)
    with pytest.raises(ep.EpError):
        ep.ep_query_expert_tiles(ep.make_expert_config(4, 10, 64, 12))
    cfg = ep.make_expert_config(4, 10, 64, 32)
    assert ep._lib.ep_query_expert_tiles(ctypes.byref(cfg), None) == BAD


@pytest.mark.gpu
@pytest.mark.parametrize("counts,I,N,act,tiles", TILES)
def test_large_in_the_other_tiles(counts, I, N, act, tiles):
    test_large(counts, I, N, act)


@pytest.mark.gpu
@pytest.mark.parametrize("counts,I,N,act,tiles", TILES_FP8)
def test_large_fp8_in_the_other_tiles(counts, I, N, act, tiles):
    test_large_fp8(counts, I, N, act)


@pytest.mark.gpu
@pytest.mark.parametrize("counts,I,N,act", [t[:4] for t in TILES] + LARGE[:1])
def test_large_gradients_alone(counts, I, N, act):
    """Either gradient of the rows or the weights without the other, bitwise as with it."""
    print(f"[expert_mm_backward alone] {len(counts)} experts I={I} N={N} {act}", flush=True)
    base, rows, x, w, g = make(counts, I, N, act, 23)
    pre = torch.randn((rows, cols_of(N, act)), generator=g).bfloat16().cuda()
    d = torch.randn((rows, N), generator=g).bfloat16().cuda()
    x, w, bt = x.cuda(), w.cuda(), torch.tensor(base, dtype=torch.int32).cuda()
    cfg = ep.make_expert_config(len(counts), rows, I, N, activation=act)
    scratch = ep.alloc_expert_backward(cfg)
    dx, dw = torch.full_like(x, 7.0), torch.full_like(w, 7.0)
    dx2, dw2 = torch.full_like(x, 7.0), torch.full_like(w, 7.0)
    ep.ep_expert_mm_backward(cfg, bt, x, w, d, scratch, pre=pre, d_x=dx, d_w=dw)
    ep.ep_expert_mm_backward(cfg, bt, None, w, d, scratch, pre=pre, d_x=dx2)
    ep.ep_expert_mm_backward(cfg, bt, x, w, d, scratch, pre=pre, d_w=dw2)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.gpu
@pytest.mark.parametrize("alignment", [1, 16])
def test_fp8_rows_of_the_dispatch(alignment):
    """fp8 tokens of two sources, dispatched, multiplied with the scales that the dispatch delivers, and combined."""
    S, T, I, N, K, E, R = 2, 61, 384, 200, 3, 8, 4
    g = torch.Generator().manual_seed(31)
    x8 = torch.randn((S, T, I), generator=g).to(torch.float8_e4m3fn)
    sf = torch.exp(torch.randn((S, T, I // 128), generator=g))
    idx = torch.rand((S, T, E), generator=g).topk(K, 2).indices
    idx[torch.rand((S, T, K), generator=g) < 0.1] = -1
    weights = torch.rand((S, T, K), generator=g)
    w8 = torch.randn((E, 2 * N, I), generator=g).to(torch.float8_e4m3fn)
    ws = torch.exp(torch.randn((E, -(-2 * N // 128), I // 128), generator=g)) * I ** -0.5
    cfg = ep.make_config(S, T, I, K, E, R, T, dtype="fp8", expand=True, alignment=alignment)
    L, recv = ep.alloc_layout(cfg), ep.alloc_recv(cfg)
    recv.recv_x.fill_(0x7f)  # NaN in every row that nothing writes
    recv.recv_sf.fill_(float("nan"))
    idx_d, weights_d = idx.cuda(), weights.cuda()
    ep.ep_layout_dispatch(cfg, x8.cuda(), sf.cuda(), idx_d, weights_d, L, recv)
    rows = recv.rows
    out = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    kept = torch.full((rows, 2 * N), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_mm(ep.make_expert_config(E, rows, I, N, dtype="fp8", activation="swiglu"), L.expert_base, recv.recv_x,
                    w8.cuda(), out, x_sf=recv.recv_sf, w_sf=ws.cuda(), pre=kept)
    tokens = torch.empty((S, T, N), dtype=torch.bfloat16, device="cuda")
    ep.ep_combine(ep.make_config(S, T, N, K, E, R, T, expand=True, alignment=alignment), L, idx_d, weights_d, out, tokens)
    torch.cuda.synchronize()
    base, pos = L.expert_base.cpu().numpy(), L.expand_pos.cpu()
    assert base[-1] % alignment == 0 and base[-1] <= rows
    x64 = torch.zeros((rows, I), dtype=torch.float64)  # padding rows stay zero
    for k in range(K):
        there = idx[:, :, k] >= 0
        x64[pos[:, :, k][there].long()] = (x8.double() * sf.double().repeat_interleave(128, 2))[there]
    w64 = w8.double() * ws.double().repeat_interleave(128, 2).repeat_interleave(128, 1)[:, :2 * N]
    check_forward(base, out, kept, *product64(base, x64, w64, None), I + 4, N, "swiglu", None)
    y = torch.where((idx >= 0)[..., None], out.cpu().double()[pos.clamp(min=0).long()], 0.0) * weights.double()[..., None]
    assert ((tokens.cpu().double() - y.sum(2)).abs() <= H * y.sum(2).abs() + (1 + H) * 2 * K * U * y.abs().sum(2)).all()
