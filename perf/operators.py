"""Cases of the operators around the expert-parallel exchange: the router with its balance loss, the experts' products,
and the backward pass of the combine.

Every case is measured through ``run``.  With ``own`` false it computes the operator with elementary torch operations in
32 bits (64 where a border or a long sum needs it), rounded once at the end; with ``own`` true it calls the library.
``exact`` gives the same outputs from the definitions in 64 bits, written apart from the plain form.

Operators (n = S*T tokens, E experts, K lanes per token):

route        scores of [n][E] logits, the K best experts, their weights; for training also the counts per expert, the
             balance loss of each source and the gradient of the logits.
product      rows grouped by expert times their expert's weights, with bias, activation and residual.
product_back its gradients: rows, weights and bias, from the saved pre-activation.
combine_back gradients of the weighted sum over a token's expert rows: the rows and the weights.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


def listed():
    return [
        # One token of a serving loop: sigmoid scores, a selection bias, no loss.  Latency is all there is.
        dict(name="route one token", op="route", S=1, T=1, E=256, K=8, dtype="fp32", scoring="sigmoid", bias=True,
             mask=False, train=False),
        # The router of a 4096-token micro-batch over 256 experts: softmax, balance loss, gradient.
        dict(name="route train 4096", op="route", S=1, T=4096, E=256, K=8, dtype="fp32", scoring="softmax", bias=False,
             mask=False, train=True),
        # Several sequences of odd length with padded tokens, bf16 logits, sigmoid scores and a selection bias.
        dict(name="route train ragged", op="route", S=5, T=2731, E=160, K=6, dtype="bf16", scoring="sigmoid", bias=True,
             mask=True, train=True),
        # One token through a gated first product of 32 local experts: eight experts' weights are read for one row each.
        dict(name="product one token", op="product", T=1, E=32, K=8, I=7168, N=2048, act="swiglu", dtype="bf16",
             bias=False, residual=False, pre=False, skew=False),
        # A decode batch through the second product, with its bias and the residual rows.
        dict(name="product decode", op="product", T=64, E=32, K=8, I=2048, N=7168, act="none", dtype="bf16", bias=True,
             residual=True, pre=False, skew=False),
        # A prompt's rows on one rank's 16 experts, gated: the largest forward product.
        dict(name="product prompt", op="product", T=4096, E=16, K=8, I=7168, N=2048, act="swiglu", dtype="bf16",
             bias=False, residual=False, pre=False, skew=False),
        # The same layer fed by fp8 dispatch: e4m3 rows and weights with their scales.
        dict(name="product prompt fp8", op="product", T=4096, E=16, K=4, I=7168, N=2048, act="swiglu", dtype="fp8",
             bias=False, residual=False, pre=False, skew=False),
        # Unbalanced routing, odd sizes, a training forward that keeps the pre-activation.
        dict(name="product ragged", op="product", T=1999, E=24, K=3, I=1160, N=1416, act="gelu", dtype="bf16", bias=True,
             residual=True, pre=True, skew=True),
        # The backward pass of a gated first product on one rank's experts.
        dict(name="product back", op="product_back", T=2048, E=16, K=8, I=4096, N=1024, act="swiglu", bias=False,
             skew=False),
        # Unbalanced and odd: few rows for some experts, none for others.
        dict(name="product back ragged", op="product_back", T=777, E=24, K=3, I=1160, N=1416, act="silu", bias=True,
             skew=True),
        # The combine's gradients for a training micro-batch, per-expert rows.
        dict(name="combine back 4096", op="combine_back", S=1, T=4096, H=7168, E=256, K=8, R=16, expand=True,
             masked=False),
        # Small, several sources, compact rows shared by lanes of one rank, masked lanes.
        dict(name="combine back compact", op="combine_back", S=3, T=211, H=1288, E=64, K=6, R=8, expand=False,
             masked=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "route", "product", "product", "product_back", "combine_back"))
    if op == "route":
        S, E = rng.choice((1, 1, 2, 3, 7, 16)), rng.choice((8, 31, 64, 100, 128, 160, 256, 384, 512))
        return dict(op=op, S=S, T=_log(rng, 1, 16384 // S), E=E, K=min(E, rng.choice((1, 2, 4, 6, 8, 11))),
                    dtype=rng.choice(("fp32", "bf16")), scoring=rng.choice(("softmax", "sigmoid")),
                    bias=rng.random() < 0.5, mask=rng.random() < 0.5, train=rng.random() < 0.7)
    if op in ("product", "product_back"):
        E = rng.choice((1, 4, 7, 16, 24, 32, 48))
        fp8 = op == "product" and rng.random() < 0.25
        act = rng.choice(("none", "relu", "gelu", "silu", "swiglu"))
        step = 128 if fp8 else 8
        I, N = step * _log(rng, 1 if fp8 else 16, 4096 // step), step * _log(rng, 1 if fp8 else 16, 2048 // step)
        K = min(E, rng.choice((1, 2, 4, 8)))
        case = dict(op=op, T=_log(rng, 1, 16384 // K), E=E, K=K, I=I, N=N, act=act)
        if op == "product":
            case.update(dtype="fp8" if fp8 else "bf16", residual=rng.random() < 0.4, pre=rng.random() < 0.3)
        return dict(case, bias=rng.random() < 0.5, skew=rng.random() < 0.4)
    S, R = rng.choice((1, 1, 2, 5)), rng.choice((4, 8, 16))
    return dict(op=op, S=S, T=_log(rng, 1, 4096 // S), H=8 * _log(rng, 8, 896), E=R * rng.choice((4, 8, 16)),
                K=rng.choice((1, 2, 4, 8)), R=R, expand=rng.random() < 0.6, masked=rng.random() < 0.5)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _uniform(g, lo, hi, *shape):
    return torch.rand(shape, generator=g, device=DEV, dtype=torch.float32) * (hi - lo) + lo


def _bf16(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _wide(case):
    """Weight rows per expert: the gate's and the up projection's for the gated activation."""
    return 2 * case["N"] if case["act"] == "swiglu" else case["N"]


def prepare(case, seed):
    g = _gen(seed)
    return {"route": _prepare_route, "product": _prepare_product, "product_back": _prepare_product,
            "combine_back": _prepare_combine}[case["op"]](case, g)


def _prepare_route(c, g):
    n, E, K = c["S"] * c["T"], c["E"], c["K"]
    # A trained router: most logits near each other, some experts more popular than others.
    logits = 1.3 * _normal(g, n, E) + 0.4 * _normal(g, 1, E)
    st = dict(case=c, logits=logits.to(torch.bfloat16) if c["dtype"] == "bf16" else logits)
    st["bias"] = 0.05 * _normal(g, E) if c["bias"] else None
    st["mask"] = (_uniform(g, 0, 1, n) < 0.9).to(torch.uint8) if c["mask"] else None
    if c["train"]:
        st["d_weights"] = _normal(g, n, K)
        st["d_loss"] = _uniform(g, 0.5, 1.5, c["S"]) * 0.01 * n
        st["d_logits"] = torch.zeros_like(st["logits"])
    return st


def _counts(c, g):
    """Rows per expert of T tokens with K distinct experts each."""
    keys = -torch.log(-torch.log(torch.rand((c["T"], c["E"]), generator=g, device=DEV).clamp(1e-7, 1 - 1e-7)))
    if c["skew"]:
        keys = keys - 1.2 * torch.log(torch.arange(1, c["E"] + 1, device=DEV, dtype=torch.float32))
    return torch.bincount(keys.topk(c["K"], dim=1).indices.reshape(-1), minlength=c["E"]).tolist()


def _prepare_product(c, g):
    E, I, N, Nw = c["E"], c["I"], c["N"], _wide(c)
    counts = _counts(c, g)
    rows = sum(counts)
    base = np.concatenate([[0], np.cumsum(counts)])
    st = dict(case=c, rows=rows, counts=counts, expert_base=torch.tensor(base, dtype=torch.int32, device=DEV))
    # The plan a program without grouped products keeps: the experts with rows, their rows side by side.
    active = [e for e in range(E) if counts[e]]
    cap = max(counts)
    st["active"] = torch.tensor(active, device=DEV)
    lo, hi = torch.tensor(base[:-1], device=DEV)[st["active"]], torch.tensor(base[1:], device=DEV)[st["active"]]
    at = lo[:, None] + torch.arange(cap, device=DEV)[None, :]
    st["inside"] = at < hi[:, None]
    st["at"] = torch.minimum(at, hi[:, None] - 1)
    st["of_row"] = torch.repeat_interleave(torch.arange(E, device=DEV), torch.tensor(counts, device=DEV))
    slot = torch.zeros(E, dtype=torch.int64, device=DEV)
    slot[st["active"]] = torch.arange(len(active), device=DEV)
    st["place"] = slot[st["of_row"]] * cap + torch.arange(rows, device=DEV) - torch.tensor(base, device=DEV)[st["of_row"]]
    if c.get("dtype") == "fp8":
        st["x"] = _normal(g, rows, I).to(torch.float8_e4m3fn)
        st["x_sf"] = _uniform(g, 0.5, 2.0, rows, I // 128)
        st["w"] = torch.stack([_normal(g, Nw, I).to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(E)]).view(torch.float8_e4m3fn)
        st["w_sf"] = _uniform(g, 0.5, 1.5, E, -(-Nw // 128), I // 128) / math.sqrt(I)
    else:
        st["x"], st["x_sf"], st["w_sf"] = _bf16(g, rows, I), None, None
        st["w"] = _bf16(g, E, Nw, I).mul_(1 / math.sqrt(I))
    st["bias"] = 0.1 * _normal(g, E, Nw) if c["bias"] else None
    if c["op"] == "product":
        st["residual"] = _bf16(g, rows, N) if c["residual"] else None
        st["out"] = torch.zeros((rows, N), dtype=torch.bfloat16, device=DEV)
        st["pre"] = torch.zeros((rows, Nw), dtype=torch.bfloat16, device=DEV) if c["pre"] else None
    else:
        st["pre"] = _bf16(g, rows, Nw) if c["act"] != "none" else None
        st["d_out"] = _bf16(g, rows, N)
        st["d_x"] = torch.zeros((rows, I), dtype=torch.bfloat16, device=DEV)
        st["d_w"] = torch.zeros((E, Nw, I), dtype=torch.bfloat16, device=DEV)
        st["d_bias"] = torch.zeros((E, Nw), device=DEV) if c["bias"] else None
    return st


def _prepare_combine(c, g):
    S, T, H, E, K, R = (c[k] for k in ("S", "T", "H", "E", "K", "R"))
    n = S * T
    idx = torch.rand((n, E), generator=g, device=DEV).topk(K, dim=1).indices
    if c["masked"]:
        idx = torch.where(_uniform(g, 0, 1, n, K) < 0.15, -1, idx)
    valid = idx >= 0
    rows = n * K if c["expand"] else n * min(K, R)
    if c["expand"]:  # one row per valid lane, by expert, then token, then lane
        order = torch.where(valid, idx, E).reshape(-1).argsort(stable=True)
        row = torch.empty(n * K, dtype=torch.int64, device=DEV)
        row[order] = torch.arange(n * K, device=DEV)
        row = row.reshape(n, K)
    else:  # one row per token and rank, by rank, then token
        rank = idx.clamp(min=0) // (E // R)
        there = torch.zeros((n, R), dtype=torch.int64, device=DEV)
        there.scatter_reduce_(1, rank, valid.long(), "amax")
        flat = there.t().reshape(-1).cumsum(0) - 1
        row = flat.reshape(R, n).t().gather(1, rank)
    st = dict(case=c, topk_idx=idx.reshape(S, T, K).contiguous(), valid=valid, row=torch.where(valid, row, 0), rows=rows)
    st["topk_weights"] = torch.softmax(_normal(g, S, T, K), -1)
    st["y"], st["d_out"] = _bf16(g, rows, H), _bf16(g, n, H)
    st["d_y"] = torch.zeros((rows, H), dtype=torch.bfloat16, device=DEV)
    st["d_weights"] = torch.zeros((S, T, K), device=DEV)
    return st


def run(state):
    return {"route": _run_route, "product": _run_product, "product_back": _run_product_back,
            "combine_back": _run_combine}[state["case"]["op"]](state)


# --------------------------------------------------------------------------------------------------------- the router

def _scores(logits, mask, scoring, kind):
    """(valid, logits with masked ones at -inf, scores) in the floating type `kind`."""
    info = torch.finfo(logits.dtype)
    valid = logits.to(kind) > info.min
    if mask is not None:
        valid = valid & (mask != 0)[:, None]
    l = torch.where(valid, logits.to(kind).clamp(max=info.max), -torch.inf)
    if scoring == "sigmoid":
        return valid, l, torch.where(valid, torch.sigmoid(l), 0.0)
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(torch.isfinite(top), top, 0.0))
    return valid, l, e / e.sum(1, keepdim=True).clamp(min=1e-30)


def _run_route(st):
    c = st["case"]
    if own:
        import combine_ep_layout_07_amd.ep as ep
        if "kept" not in st:
            cfg = ep.make_route_config(c["S"], c["T"], c["E"], c["K"], dtype=c["dtype"], scoring=c["scoring"], scale=2.5)
            st["kept"] = cfg, ep.alloc_route(cfg, balance=c["train"])
        cfg, r = st["kept"]
        ep.ep_route(cfg, st["logits"], r, bias=st["bias"], token_mask=st["mask"])
        out = dict(topk_idx=r.topk_idx, topk_weights=r.topk_weights)
        if c["train"]:
            ep.ep_route_backward(cfg, st["logits"], r, st["d_weights"], st["d_loss"], st["d_logits"], token_mask=st["mask"])
            out.update(counts=r.tokens_per_expert, tokens=r.tokens_valid, loss=r.balance_loss, d_logits=st["d_logits"])
        return out
    S, T, E, K, scale = c["S"], c["T"], c["E"], c["K"], 2.5
    valid, l, s = _scores(st["logits"], st["mask"], c["scoring"], torch.float32)
    key = l
    if st["bias"] is not None:  # in 64 bits: the border between the last chosen expert and the next
        key = _scores(st["logits"], st["mask"], c["scoring"], torch.float64)[2] + st["bias"].double()
        key = torch.where(valid, key, -torch.inf)
    best = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :K]
    chosen = valid.gather(1, best)
    sk = torch.where(chosen, s.gather(1, best), 0.0)
    D = sk.sum(1, keepdim=True) + 1e-20
    out = dict(topk_idx=torch.where(chosen, best, -1).reshape(S, T, K), topk_weights=(scale * sk / D).reshape(S, T, K))
    if not c["train"]:
        return out
    there = torch.zeros_like(s).scatter_(1, best, chosen.float())
    counts = there.reshape(S, T, E).sum(1)
    tokens = valid.any(1).reshape(S, T).sum(1)
    all_s = s.sum(1, keepdim=True)
    phat = s if c["scoring"] == "softmax" else s / (all_s + 1e-20)
    some = tokens.clamp(min=1).double()[:, None]
    mean = phat.reshape(S, T, E).double().sum(1) / some
    share = counts.double() * E / (K * some)
    loss = (share * mean).sum(1).float()
    a = (st["d_loss"].double()[:, None] * share / some).float().repeat_interleave(T, 0)
    dw = st["d_weights"]
    dk = torch.where(chosen, scale * (dw - (dw * sk / D).sum(1, keepdim=True)) / D, 0.0)
    u = torch.zeros_like(s).scatter_(1, best, dk)
    if c["scoring"] == "softmax":
        u = u + a
        dl = s * (u - (u * s).sum(1, keepdim=True))
    else:
        u = u + (a - (a * phat).sum(1, keepdim=True)) / (all_s + 1e-20)
        dl = u * s * torch.sigmoid(-l)
    dl = torch.where(valid, dl, 0.0).to(st["logits"].dtype)
    out.update(counts=counts.to(torch.int32), tokens=tokens.to(torch.int32), loss=loss, d_logits=dl)
    return out


def _exact_route(st):
    c, S, T, E, K = st["case"], *(st["case"][k] for k in ("S", "T", "E", "K"))
    raw = st["logits"]
    x = raw.double().clone().requires_grad_(True)
    open_ = raw.double() > float(torch.finfo(raw.dtype).min)
    if st["mask"] is not None:
        open_ &= st["mask"].bool().unsqueeze(1)
    gone = ~open_.any(1, keepdim=True)
    if c["scoring"] == "softmax":
        p = torch.softmax(x.masked_fill(~open_, -1e300), 1).masked_fill(~open_ | gone, 0.0)
        s = p
    else:
        s = (1 / (1 + torch.exp(-x))).masked_fill(~open_, 0.0)
        p = s / (s.sum(1, keepdim=True) + 1e-20)
    key = (raw.double() if st["bias"] is None else s.detach() + st["bias"].double()).masked_fill(~open_, -np.inf)
    order = np.argsort(-key.cpu().numpy(), axis=1, kind="stable")[:, :K]
    best = torch.from_numpy(np.ascontiguousarray(order)).to(raw.device)
    ok = open_.gather(1, best)
    sk = s.gather(1, best) * ok
    w = 2.5 * sk / (sk.sum(1, keepdim=True) + 1e-20)
    out = dict(topk_idx=None, topk_weights=w.detach().reshape(S, T, K))
    if c["train"]:
        f = torch.zeros_like(s).scatter_(1, best, ok.double()).reshape(S, T, E).sum(1)
        tv = open_.any(1).reshape(S, T).sum(1).clamp(min=1).double()
        loss = (p.reshape(S, T, E).sum(1) * f).sum(1) * E / (K * tv * tv)
        ((w * st["d_weights"].double()).sum() + (loss * st["d_loss"].double()).sum()).backward()
        out.update(counts=None, tokens=None, loss=loss.detach(), d_logits=x.grad)
    return out


# ------------------------------------------------------------------------------------------------ the experts' products

def _gelu(v):
    return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))


def _act(act, pre, N):
    if act == "none":
        return pre
    if act == "relu":
        return pre.clamp(min=0)
    if act == "gelu":
        return _gelu(pre)
    if act == "silu":
        return pre * torch.sigmoid(pre)
    gate, up = pre[:, :N], pre[:, N:]
    return gate * torch.sigmoid(gate) * up


def _act_back(act, pre, d, N):
    """Gradient of the pre-activation."""
    if act == "none":
        return d
    if act == "relu":
        return torch.where(pre > 0, d, 0.0)
    if act == "gelu":
        return d * (0.5 * (1 + torch.erf(pre * math.sqrt(0.5))) + pre * torch.exp(-0.5 * pre * pre) / math.sqrt(2 * math.pi))
    if act == "silu":
        sg = torch.sigmoid(pre)
        return d * sg * (1 + pre * (1 - sg))
    gate, up = pre[:, :N], pre[:, N:]
    sg = torch.sigmoid(gate)
    return torch.cat([d * up * sg * (1 + gate * (1 - sg)), d * gate * sg], 1)


def _rows32(x, sf):
    return x.float() if sf is None else x.float() * sf.repeat_interleave(128, 1)


def _weights32(st):
    """The active experts' weights in 32 bits."""
    w, a = st["w"], st["active"]
    if st["w_sf"] is None:
        return w[a].float()
    sf = st["w_sf"][a].repeat_interleave(128, 2).repeat_interleave(128, 1)[:, :w.shape[1]]
    return w.view(torch.uint8)[a].view(w.dtype).float() * sf


def _expert_config(ep, st):
    c = st["case"]
    return ep.make_expert_config(c["E"], st["rows"], c["I"], c["N"], dtype=c.get("dtype", "bf16"), activation=c["act"])


def _run_product(st):
    c = st["case"]
    if own:
        import combine_ep_layout_07_amd.ep as ep
        if "kept" not in st:
            st["kept"] = _expert_config(ep, st)
        ep.ep_expert_mm(st["kept"], st["expert_base"], st["x"], st["w"], st["out"], x_sf=st["x_sf"], w_sf=st["w_sf"],
                        bias=st["bias"], residual=st["residual"], pre=st["pre"])
        return dict(out=st["out"], pre=st["pre"])
    N = c["N"]
    pre = torch.bmm(_rows32(st["x"], st["x_sf"])[st["at"]], _weights32(st).transpose(1, 2))
    pre = pre.reshape(-1, pre.shape[2])[st["place"]]
    if st["bias"] is not None:
        pre = pre + st["bias"][st["of_row"]]
    out = _act(c["act"], pre, N)
    if st["residual"] is not None:
        out = out + st["residual"].float()
    return dict(out=out.to(torch.bfloat16), pre=pre.to(torch.bfloat16) if c["pre"] else None)


def _run_product_back(st):
    c = st["case"]
    if own:
        import combine_ep_layout_07_amd.ep as ep
        if "kept" not in st:
            cfg = _expert_config(ep, st)
            st["kept"] = cfg, ep.alloc_expert_backward(cfg)
        cfg, scratch = st["kept"]
        ep.ep_expert_mm_backward(cfg, st["expert_base"], st["x"], st["w"], st["d_out"], scratch, pre=st["pre"],
                                 d_x=st["d_x"], d_w=st["d_w"], d_bias=st["d_bias"])
        return dict(d_x=st["d_x"], d_w=st["d_w"], d_bias=st["d_bias"])
    d = _act_back(c["act"], None if st["pre"] is None else st["pre"].float(), st["d_out"].float(), c["N"])
    side = torch.where(st["inside"][:, :, None], d[st["at"]], 0.0)
    dx = torch.bmm(side, _weights32(st))
    dx = dx.reshape(-1, dx.shape[2])[st["place"]].to(torch.bfloat16)
    dw = torch.zeros_like(st["w"])
    dw[st["active"]] = torch.bmm(side.transpose(1, 2), st["x"].float()[st["at"]]).to(torch.bfloat16)
    db = None
    if st["bias"] is not None:
        db = torch.zeros_like(st["bias"])
        db[st["active"]] = side.sum(1)
    return dict(d_x=dx, d_w=dw, d_bias=db)


def _exact_product(st):
    c, N, lo = st["case"], st["case"]["N"], 0
    back = c["op"] == "product_back"
    out, pres, dx, dw, db = [], [], [], [], []
    for e, n in enumerate(st["counts"]):
        x, w = st["x"][lo:lo + n].double(), st["w"][e].double()
        if st["x_sf"] is not None:
            x = (x.reshape(n, -1, 128) * st["x_sf"][lo:lo + n, :, None].double()).reshape(n, -1)
            r = torch.arange(w.shape[0], device=w.device) // 128
            w = (w.reshape(w.shape[0], -1, 128) * st["w_sf"][e].double()[r][:, :, None]).reshape(w.shape)
        if back:
            d = st["d_out"][lo:lo + n].double()
            if st["pre"] is not None:
                p = st["pre"][lo:lo + n].double().requires_grad_(True)
                a = _exact_act(c["act"], p, N)
                (d,) = torch.autograd.grad(a, p, d)
            dx.append(d @ w)
            dw.append(d.T @ x)
            db.append(d.sum(0))
        else:
            p = x @ w.T
            if st["bias"] is not None:
                p = p + st["bias"][e].double()
            a = _exact_act(c["act"], p, N)
            out.append(a if st["residual"] is None else a + st["residual"][lo:lo + n].double())
            pres.append(p)
        lo += n
    if back:
        return dict(d_x=torch.cat(dx), d_w=torch.stack(dw), d_bias=torch.stack(db) if c["bias"] else None)
    return dict(out=torch.cat(out), pre=torch.cat(pres) if c["pre"] else None)


def _exact_act(act, p, N):
    if act == "swiglu":
        return p[:, :N] / (1 + torch.exp(-p[:, :N])) * p[:, N:]
    if act == "silu":
        return p / (1 + torch.exp(-p))
    if act == "gelu":
        return p * torch.special.ndtr(p)
    return torch.maximum(p, torch.zeros_like(p)) if act == "relu" else p


# ------------------------------------------------------------------------------------------ the combine's backward pass

def _run_combine(st):
    c = st["case"]
    S, T, H, K = c["S"], c["T"], c["H"], c["K"]
    if own:
        import combine_ep_layout_07_amd.ep as ep
        if "kept" not in st:  # the handle of the forward pass
            cfg = ep.make_config(S, T, H, K, c["E"], c["R"], T, expand=c["expand"])
            layout = ep.alloc_layout(cfg)
            ep.ep_layout(cfg, st["topk_idx"], layout)
            st["kept"] = cfg, layout
        cfg, layout = st["kept"]
        ep.ep_combine_backward(cfg, layout, st["topk_idx"], st["topk_weights"], st["y"], st["d_out"], st["d_y"],
                               st["d_weights"])
        return dict(d_y=st["d_y"], d_weights=st["d_weights"])
    row, valid = st["row"], st["valid"]
    w = torch.where(valid, st["topk_weights"].reshape(-1, K), 0.0)
    if not c["expand"]:  # lanes of one row: their weights' sum
        total = torch.zeros(st["rows"], device=w.device).index_add_(0, row.reshape(-1), w.reshape(-1))
    d = st["d_out"].float()
    dots = (st["y"][row].float() * d[:, None, :]).sum(2)
    dots = torch.where(valid, dots, 0.0).reshape(S, T, K)
    # One row each for the expand layout; for the compact one every lane of a row writes the same values.
    factor = w if c["expand"] else total[row]
    value = (factor[:, :, None] * d[:, None, :]).to(torch.bfloat16).reshape(-1, H)
    dy = torch.zeros((st["rows"] + 1, H), dtype=torch.bfloat16, device=d.device)
    dy[torch.where(valid, row, st["rows"]).reshape(-1)] = value
    return dict(d_y=dy[:-1], d_weights=dots)


def _exact_combine(st):
    c = st["case"]
    S, T, H, K = c["S"], c["T"], c["H"], c["K"]
    d, y = st["d_out"].double(), st["y"]
    dy = torch.zeros((st["rows"], H), dtype=torch.float64, device=d.device)
    dw = torch.zeros((S * T, K), dtype=torch.float64, device=d.device)
    for k in range(K):
        t = torch.nonzero(st["valid"][:, k]).squeeze(1)
        r = st["row"][t, k]
        dy.index_add_(0, r, st["topk_weights"].reshape(-1, K)[t, k].double()[:, None] * d[t])
        dw[t, k] = torch.linalg.vecdot(y[r].double(), d[t])
    return dict(d_y=dy, d_weights=dw.reshape(S, T, K))


def exact(case, seed):
    st = prepare(case, seed)
    return {"route": _exact_route, "product": _exact_product, "product_back": _exact_product,
            "combine_back": _exact_combine}[case["op"]](st)


def work(case):
    c = case
    if c["op"] == "route":
        n, E, K, el = c["S"] * c["T"], c["E"], c["K"], 2 if c["dtype"] == "bf16" else 4
        b = n * (E * el + 12 * K) + (4 * E if c["bias"] else 0) + (n if c["mask"] else 0)
        if c["train"]:
            b += n * (E * el + 4 * K) + c["S"] * (4 * E + 12)  # the gradient, the counts, the loss
        return dict(bytes=b, flops=n * E * (25 if c["train"] else 10))
    if c["op"] in ("product", "product_back"):
        rows, I, N, Nw, E = c["T"] * c["K"], c["I"], c["N"], _wide(c), c["E"]
        active = E * (1 - (1 - c["K"] / E) ** c["T"])  # experts that some token picks, with even routing
        el = 1 if c.get("dtype") == "fp8" else 2
        b = rows * I * el + active * Nw * I * el + (4 * active * Nw if c["bias"] else 0)
        if el == 1:
            b += 4 * rows * I / 128 + 4 * active * Nw * I / 16384
        if c["op"] == "product":
            b += 2 * rows * N * (2 if c["residual"] else 1) + (2 * rows * Nw if c["pre"] else 0)
            return dict(bytes=b, flops=2.0 * rows * I * Nw)
        b += 2 * rows * (N + I) + (2 * rows * Nw if c["act"] != "none" else 0) + 2.0 * E * Nw * I
        return dict(bytes=b, flops=4.0 * rows * I * Nw)
    n, K, H = c["S"] * c["T"], c["K"], c["H"]
    lanes = n * K * (0.85 if c["masked"] else 1.0)
    per = c["E"] // c["R"]
    rows = lanes if c["expand"] else n * c["R"] * (1 - (1 - lanes / n / c["E"]) ** per)
    return dict(bytes=2 * n * H + 4 * rows * H + n * K * 16, flops=4.0 * lanes * H)
