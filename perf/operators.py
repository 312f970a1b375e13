"""Operators around the MoE layer: what is measured, their plain forms and their exact values.

Three groups, five calls: the residual addition with RMSNorm and MXFP8 output ("norm") and its
backward pass ("norm_bwd"), the router's balance and z losses with per-expert counts ("loss") and
their backward pass ("loss_bwd"), and the 4-bit matrix-vector product ("linear").
"""
import math

import torch

own = False

EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token of a decode step, hidden 2048: latency is everything
        {"name": "norm 1x2048", "op": "norm", "rows": 1, "cols": 2048, "y": True},
        # a decode batch of a wide model; y also feeds the router
        {"name": "norm 64x7168", "op": "norm", "rows": 64, "cols": 7168, "y": True},
        # a prefill chunk that only feeds a W4A8 layer
        {"name": "norm 16384x4096", "op": "norm", "rows": 16384, "cols": 4096, "y": False},
        # a training micro-batch, with the gradient that arrives over the residual stream
        {"name": "norm_bwd 8192x2048", "op": "norm_bwd", "rows": 8192, "cols": 2048, "dh": True},
        # an odd number of rows, a width that is no power of two, no residual gradient
        {"name": "norm_bwd 1999x7168", "op": "norm_bwd", "rows": 1999, "cols": 7168, "dh": False},
        # expert load of one decode batch, as a server records it
        {"name": "loss 64x128", "op": "loss", "rows": 64, "experts": 128, "k": 8, "router": "softmax", "mask": False},
        # a training batch of a 256-expert layer, padded tokens masked
        {"name": "loss 131072x256", "op": "loss", "rows": 131072, "experts": 256, "k": 8, "router": "softmax", "mask": True},
        # gradients of both losses and of the top-k weights, the sqrt-softplus router
        {"name": "loss_bwd 8192x256 sp", "op": "loss_bwd", "rows": 8192, "experts": 256, "k": 8, "router": "sqrtsoftplus", "mask": True},
        # the same for many tokens over few experts, an expert count that is no multiple of 32
        {"name": "loss_bwd 100003x60", "op": "loss_bwd", "rows": 100003, "experts": 60, "k": 4, "router": "softmax", "mask": False},
        # one token through a square projection of the decode configuration
        {"name": "linear 1x2048x2048", "op": "linear", "rows": 1, "n": 2048, "cols": 2048, "format": "nvfp4", "fp32": False},
        # one token's output logits over a large vocabulary
        {"name": "linear 1x131072x4096", "op": "linear", "rows": 1, "n": 131072, "cols": 4096, "format": "nvfp4", "fp32": True},
        # a decode batch through a wide projection, MXFP4 weights, an odd number of rows and outputs
        {"name": "linear 15x18431x7168 mx", "op": "linear", "rows": 15, "n": 18431, "cols": 7168, "format": "mxfp4", "fp32": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "loss", "loss_bwd", "linear", "linear"])
    if op in ("norm", "norm_bwd"):
        cols = 32 * _log(rng, 8, 512)
        rows = min(_log(rng, 1, 20000), 64_000_000 // cols)
        if op == "norm":
            return {"op": op, "rows": rows, "cols": cols, "y": rng.random() < 0.5}
        return {"op": op, "rows": rows, "cols": cols, "dh": rng.random() < 0.5}
    if op in ("loss", "loss_bwd"):
        experts = _log(rng, 8, 1024)
        rows = min(_log(rng, 1, 130000), 33_000_000 // experts)
        return {"op": op, "rows": rows, "experts": experts, "k": rng.randint(1, min(experts, 16)),
                "router": rng.choice(["softmax", "sqrtsoftplus"]), "mask": rng.random() < 0.5}
    cols = 32 * _log(rng, 8, 512)
    n = min(_log(rng, 16, 131072), 520_000_000 // cols)
    return {"op": op, "rows": _log(rng, 1, 64), "n": n, "cols": cols,
            "format": rng.choice(["nvfp4", "mxfp4"]), "fp32": rng.random() < 0.5}


def _weights(n, cols, fmt, g):
    """Codes [n, cols/2], scales and the tensor scale of normal weights, quantised block by block."""
    dev = "cuda"
    block = 16 if fmt == "nvfp4" else 32
    codes = torch.empty(n, cols // 2, dtype=torch.uint8, device=dev)
    sf = torch.empty(n, cols // block, dtype=torch.uint8, device=dev)
    ts = torch.full((1,), 0.02 * 5.5 / (6 * 448), device=dev) if fmt == "nvfp4" else None
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=dev)
    step = max(1, (1 << 25) // cols)
    for i in range(0, n, step):
        m = min(step, n - i)
        w = torch.randn(m, cols // block, block, device=dev, generator=g) * 0.02
        top = w.abs().amax(-1, keepdim=True)
        if fmt == "nvfp4":
            s8 = (top / 6 / ts).clamp(max=448).to(torch.float8_e4m3fn)
            s = s8.float() * ts
            sf[i:i + m] = s8.view(torch.uint8).squeeze(-1)
        else:
            e = (torch.frexp(top).exponent - 1 - 2).clamp(-127, 127)
            s = torch.ldexp(torch.ones_like(top), e)
            sf[i:i + m] = (e + 127).to(torch.uint8).squeeze(-1)
        q = w / s
        c = torch.bucketize(q.abs(), edges).to(torch.uint8) + (q < 0).to(torch.uint8) * 8
        c = c.reshape(m, cols // 2, 2)
        codes[i:i + m] = c[..., 0] | (c[..., 1] << 4)
    return codes, sf, ts


def prepare(case, seed):
    dev, bf = "cuda", torch.bfloat16
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0, mean=0.0):
        return torch.randn(*shape, device=dev, generator=g) * scale + mean

    s, T = dict(case), case["rows"]
    op = case["op"]
    if op == "norm":
        # a residual stream wider than the update that is added to it, gains around one
        C = case["cols"]
        s.update(x=normal(T, C).to(bf), res=normal(T, C, scale=2.0).to(bf), gamma=normal(C, scale=0.1, mean=1.0).to(bf))
        s["out"] = {"h": torch.empty(T, C, dtype=bf, device=dev),
                    "codes": torch.empty(T, C, dtype=torch.uint8, device=dev),
                    "sf": torch.empty(T, C // 32, dtype=torch.uint8, device=dev)}
        if case["y"]:
            s["out"]["y"] = torch.empty(T, C, dtype=bf, device=dev)
    elif op == "norm_bwd":
        C = case["cols"]
        h = normal(T, C, scale=2.0).to(bf)
        s.update(h=h, rrms=torch.rsqrt(h.float().square().mean(-1) + EPS), gamma=normal(C, scale=0.1, mean=1.0).to(bf),
                 dy=normal(T, C).to(bf), dh_in=normal(T, C).to(bf) if case["dh"] else None)
        s["out"] = {"dx": torch.empty(T, C, dtype=bf, device=dev), "dgamma": torch.empty(C, device=dev)}
    elif op in ("loss", "loss_bwd"):
        E, k = case["experts"], case["k"]
        # some experts are more popular than others
        logits = normal(T, E) + 0.5 * normal(1, E)
        s.update(logits=logits, ids=logits.topk(k, dim=-1).indices.to(torch.int32))
        s["token_mask"] = (torch.rand(T, device=dev, generator=g) < 0.94) if case["mask"] else None
        if op == "loss":
            s["out"] = {"losses": torch.empty(2, device=dev), "counts": torch.empty(E, dtype=torch.int32, device=dev),
                        "tokens": torch.empty(1, dtype=torch.int32, device=dev), "probs": torch.empty(E, device=dev)}
        else:
            m = s["token_mask"] if case["mask"] else torch.ones(T, dtype=torch.bool, device=dev)
            hits = torch.zeros(E, dtype=torch.int32, device=dev)
            hits.scatter_add_(0, s["ids"].long().reshape(-1), m.to(torch.int32)[:, None].expand(T, k).reshape(-1))
            s.update(stats={"counts": hits, "tokens": m.sum().to(torch.int32).reshape(1)},
                     grad_losses=torch.tensor([0.01, 0.001], device=dev), grad_w=normal(T, k, scale=1e-5),
                     dlogits=torch.empty(T, E, device=dev))
    else:
        C = case["cols"]
        s["codes"], s["sf"], s["ts"] = _weights(case["n"], C, case["format"], g)
        s["x"] = normal(T, C).to(bf)
        s["out"] = torch.empty(T, case["n"], dtype=torch.float32 if case["fp32"] else bf, device=dev)
    return s


# ---- the framework's calls ----

def _own(s):
    import nvfp4_mixture_experts_softmax_gb300 as moe
    op = s["op"]
    if op == "norm":
        o = moe.add_rmsnorm_quantize_mx(s["x"], s["res"], s["gamma"], EPS, out=s["out"])
        return _norm_outputs(o["h"], o["codes"].view(torch.float8_e4m3fn), o["sf"].view(torch.float8_e8m0fnu), o.get("y"))
    if op == "norm_bwd":
        if "workspace" not in s:
            s["workspace"] = moe.add_rmsnorm_backward_workspace(s["rows"], s["cols"], device=s["h"].device)
        return moe.add_rmsnorm_backward(s["dy"], s["h"], s["rrms"], s["gamma"], dh=s["dh_in"], out=s["out"], workspace=s["workspace"])
    if op == "loss":
        if "workspace" not in s:
            s["workspace"] = moe.router_loss_workspace(s["rows"], s["experts"], device=s["logits"].device)
        return moe.router_loss(s["logits"], s["ids"], mask=s["token_mask"], router=s["router"], out=s["out"], workspace=s["workspace"])
    if op == "loss_bwd":
        return moe.router_loss_backward(s["logits"], s["ids"], s["stats"], s["grad_losses"], grad_topk_w=s["grad_w"], mask=s["token_mask"],
                                        router=s["router"], dlogits=s["dlogits"])
    return moe.linear_w4(s["x"], s["codes"], s["sf"], s["ts"], y=s["out"])


# ---- the plain forms: 32 bits ----

def _norm_outputs(h, codes, sf, y):
    o = {"h": h, "codes": codes, "sf": sf}
    if y is not None:
        o["y"] = y
    return o


def _plain_norm(s):
    h = (s["x"].float() + s["res"].float()).to(torch.bfloat16)
    f = h.float()
    y = f * (1.0 / torch.sqrt(f.square().mean(-1, keepdim=True) + EPS)) * s["gamma"].float()
    b = y.reshape(s["rows"], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent - 1 - 8, -127).clamp(-127, 127)
    q = torch.ldexp(b, -e).clamp(-448, 448).to(torch.float8_e4m3fn).reshape(y.shape)
    sf = (e + 127).to(torch.uint8).squeeze(-1).view(torch.float8_e8m0fnu)
    return _norm_outputs(h, q, sf, y.to(torch.bfloat16) if s["y"] else None)


def _plain_norm_bwd(s):
    h, dy, r = s["h"].float(), s["dy"].float(), s["rrms"][:, None]
    a = dy * s["gamma"].float()
    dx = r * a - h * (r * r * r) * ((a * h).sum(-1, keepdim=True) / s["cols"])
    if s["dh_in"] is not None:
        dx = dx + s["dh_in"].float()
    return {"dx": dx.to(torch.bfloat16), "dgamma": (dy * (h * r)).sum(0)}


def _scores(logits, router):
    """Unnormalised expert scores of a row, and their derivatives by the logits (sqrt-softplus)."""
    sp = torch.where(logits > 20, logits, torch.log1p(torch.exp(logits.clamp(max=20))))
    sc = torch.sqrt(sp)
    return sc, torch.sigmoid(logits) / (2 * sc)


def _softmax(l):
    top = l.amax(-1, keepdim=True)
    ex = torch.exp(l - top)
    total = ex.sum(-1, keepdim=True)
    return ex / total, (top + torch.log(total))


def _plain_loss(s):
    l, E, k = s["logits"], s["experts"], s["k"]
    m = s["token_mask"] if s["token_mask"] is not None else torch.ones(s["rows"], dtype=torch.bool, device=l.device)
    n = m.sum()
    p, lse = _softmax(l)
    if s["router"] == "sqrtsoftplus":
        sc, _ = _scores(l, s["router"])
        p = sc / sc.sum(-1, keepdim=True)
    counts = torch.zeros(E, dtype=torch.int32, device=l.device)
    counts.scatter_add_(0, s["ids"].long().reshape(-1), m.to(torch.int32)[:, None].expand(-1, k).reshape(-1))
    d = n.clamp(min=1).double()
    probs = ((p * m[:, None]).double().sum(0) / d).float()
    balance = E * (counts.double() / (d * k) * probs.double()).sum()
    z = (lse.double().square().squeeze(-1) * m).sum() / d
    return {"losses": torch.stack([balance, z]).float(), "counts": counts, "tokens": n.to(torch.int32).reshape(1), "probs": probs}


def _plain_loss_bwd(s):
    l, E, k = s["logits"], s["experts"], s["k"]
    n = s["stats"]["tokens"].float().clamp(min=1)
    f = s["stats"]["counts"].float() / (n * k)
    gb, gz = s["grad_losses"][0], s["grad_losses"][1]
    p, lse = _softmax(l)
    ids = s["ids"].long()
    gw = s["grad_w"]
    d = gz * (2.0 / n) * lse * p
    if s["router"] == "softmax":
        d = d + gb * (E / n) * p * (f - (f * p).sum(-1, keepdim=True))
        w, _ = _softmax(l.gather(1, ids))
        top = w * (gw - (gw * w).sum(-1, keepdim=True))
    else:
        sc, ds = _scores(l, s["router"])
        total = sc.sum(-1, keepdim=True)
        q = sc / total
        d = d + gb * (E / n) * (f - (f * q).sum(-1, keepdim=True)) / total * ds
        sk = sc.gather(1, ids)
        tk = sk.sum(-1, keepdim=True)
        top = (gw - (gw * (sk / tk)).sum(-1, keepdim=True)) / tk * ds.gather(1, ids)
    d = d.scatter_add(1, ids, top)
    return d if s["token_mask"] is None else d * s["token_mask"][:, None]


def _decode(codes, sf, ts, dtype):
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=codes.device)
    w = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).reshape(codes.shape[0], -1)
    block = w.shape[1] // sf.shape[1]
    if ts is not None:
        scale = sf.view(torch.float8_e4m3fn).to(dtype)
    else:
        scale = torch.ldexp(torch.ones(sf.shape, dtype=dtype, device=sf.device), sf.int() - 127)
    return (w.reshape(codes.shape[0], -1, block) * scale[..., None]).reshape(w.shape)


def _plain_linear(s):
    w = _decode(s["codes"], s["sf"], s["ts"], torch.float32)
    y = s["x"].float() @ w.t()
    if s["ts"] is not None:
        y = y * s["ts"]
    return y if s["fp32"] else y.to(torch.bfloat16)


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "loss": _plain_loss, "loss_bwd": _plain_loss_bwd,
            "linear": _plain_linear}[state["op"]](state)


def work(case):
    T, op = case["rows"], case["op"]
    if op == "norm":
        C = case["cols"]
        return {"bytes": T * C * (7 + 1 / 32 + (2 if case["y"] else 0)) + 2 * C, "flops": 8.0 * T * C}
    if op == "norm_bwd":
        C = case["cols"]
        return {"bytes": T * C * (6 + (2 if case["dh"] else 0)) + 4 * T + 6 * C, "flops": 10.0 * T * C}
    if op in ("loss", "loss_bwd"):
        E, k = case["experts"], case["k"]
        mask = T if case["mask"] else 0
        if op == "loss":
            return {"bytes": 4.0 * T * E + 4 * T * k + mask + 8 * E, "flops": 6.0 * T * E}
        return {"bytes": 8.0 * T * E + 8 * T * k + mask + 4 * E, "flops": 12.0 * T * E}
    n, C = case["n"], case["cols"]
    per = 1 / 2 + (1 / 16 if case["format"] == "nvfp4" else 1 / 32)
    return {"bytes": n * C * per + 2 * T * C + T * n * (4 if case["fp32"] else 2), "flops": 2.0 * T * n * C}


# ---- the definitions in 64 bits ----

def exact(case, seed):
    s, T = prepare(case, seed), case["rows"]
    op, f64 = case["op"], torch.float64
    if op == "norm":
        h = (s["x"].to(f64) + s["res"].to(f64)).to(torch.bfloat16).to(f64)
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["cols"] + EPS) * s["gamma"].to(f64)
        b = y.view(T, -1, 32)
        scale = torch.exp2(torch.floor(torch.log2(b.abs().amax(2, keepdim=True))) - 8)
        q = b / scale
        # E4M3 steps: 2^-9 below 2^-6, else an eighth of the power of two at or below the value
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        q = (torch.round(q / step) * step).clamp(-448, 448)
        return _norm_outputs(h, q.view(T, -1), scale.squeeze(2), y if case["y"] else None)
    if op == "norm_bwd":
        h, dy, g = s["h"].to(f64), s["dy"].to(f64), s["gamma"].to(f64)
        u = h * s["rrms"].to(f64).view(-1, 1)          # the normalised rows
        gu = dy * g
        dx = (gu - u * (gu * u).mean(1, keepdim=True)) * s["rrms"].to(f64).view(-1, 1)
        if case["dh"]:
            dx += s["dh_in"].to(f64)
        return {"dx": dx, "dgamma": torch.einsum("tc,tc->c", dy, u)}
    if op in ("loss", "loss_bwd"):
        E, k = case["experts"], case["k"]
        l = s["logits"].to(f64).requires_grad_(op == "loss_bwd")
        keep = torch.ones(T, dtype=f64, device=l.device) if s["token_mask"] is None else s["token_mask"].to(f64)
        lse = torch.logsumexp(l, 1)
        sc = torch.exp(l - lse[:, None]) if case["router"] == "softmax" else torch.nn.functional.softplus(l, threshold=1e9).sqrt()
        p = sc / sc.sum(1, keepdim=True)
        n = max(float(keep.sum()), 1.0)
        hits = torch.bincount(s["ids"].reshape(-1).long(), weights=keep.repeat_interleave(k), minlength=E)
        P = keep @ p / n
        Lb, Lz = E * torch.dot(hits / (n * k), P), torch.dot(keep, lse * lse) / n
        if op == "loss":
            return {"losses": torch.stack([Lb, Lz]), "counts": hits.to(torch.int32), "tokens": keep.sum().to(torch.int32).view(1), "probs": P}
        ws = sc.gather(1, s["ids"].long())
        ws = ws / ws.sum(1, keepdim=True)
        goal = s["grad_losses"][0].to(f64) * Lb + s["grad_losses"][1].to(f64) * Lz + (ws * s["grad_w"].to(f64) * keep[:, None]).sum()
        return torch.autograd.grad(goal, l)[0]
    y = []
    for i in range(0, case["n"], 8192):
        w = _exact_weights(s["codes"][i:i + 8192], s["sf"][i:i + 8192], case["format"])
        y.append(torch.einsum("tk,nk->tn", s["x"].to(f64), w))
    y = torch.cat(y, 1)
    return y * s["ts"].to(f64) if s["ts"] is not None else y


def _exact_weights(codes, sf, fmt):
    """Values of E2M1 codes and their block scales, from the fields of their bits."""
    c = torch.stack((codes & 15, codes >> 4), 2).flatten(1).long()
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e > 0, torch.exp2(e.double() - 1) * (1 + m / 2), m / 2) * (1 - 2 * (c >> 3).double())
    b = sf.long()
    if fmt == "nvfp4":
        e, m = b >> 3 & 15, (b & 7).double()
        scale = torch.where(e > 0, torch.exp2(e.double() - 7) * (1 + m / 8), m * 2.0 ** -9)
    else:
        scale = torch.exp2(b.double() - 127)
    return v * scale.repeat_interleave(v.shape[1] // sf.shape[1], 1)
