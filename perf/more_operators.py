"""Operators of the layer's training pass: what is measured, their plain forms and their exact values.

Three groups.  Layer norm with the residual addition before it ("norm") and its backward pass
("norm_bwd"); tokens sorted by expert and their rows laid out in that order ("dispatch"), brought back
with the router's weights ("combine"), and the gradients of the latter ("combine_bwd"; the gradient of
the former is a combine without weights); the experts' products on BF16 weights with the activation
between them ("experts"), their gradients down to the rows ("experts_bwd") and the gradients of the
weights ("experts_wgrad").
"""
import math

import torch

own = False

EPS = 1e-5
LIMIT, ALPHA = 7.0, 1.702     # of the clamped activations
ACTIVATIONS = ("swiglu", "swiglu_clamp", "relu2", "swiglu_oai")


def listed():
    return [
        # one token of a decode step, hidden 2048: latency is everything
        {"name": "norm 1x2048", "op": "norm", "rows": 1, "cols": 2048, "type": "bf16", "res": True, "beta": True},
        # a training micro-batch or prefill chunk, statistics kept for the backward pass
        {"name": "norm 16384x4096", "op": "norm", "rows": 16384, "cols": 4096, "type": "bf16", "res": True, "beta": True},
        # a training micro-batch of a wide model with the gradient of the residual stream, an odd number of rows
        {"name": "norm_bwd 8191x7168", "op": "norm_bwd", "rows": 8191, "cols": 7168, "type": "bf16", "dh": True, "beta": True},
        # a model that keeps FP32 activations, a width that is no power of two, no bias
        {"name": "norm_bwd 4100x1440 fp32", "op": "norm_bwd", "rows": 4100, "cols": 1440, "type": "fp32", "dh": False, "beta": False},
        # one token of a decode step to its eight experts
        {"name": "dispatch 1x2048", "op": "dispatch", "rows": 1, "cols": 2048, "experts": 128, "k": 8, "type": "bf16", "mask": False},
        # a training batch, padded tokens masked
        {"name": "dispatch 32768x2048", "op": "dispatch", "rows": 32768, "cols": 2048, "experts": 256, "k": 8, "type": "bf16", "mask": True},
        # a decode batch of a wide model, summed with the router's weights
        {"name": "combine 64x7168", "op": "combine", "rows": 64, "cols": 7168, "experts": 256, "k": 8, "type": "bf16", "mask": False, "weights": True},
        # gradients of the rows and of the router's weights, four experts a token, some tokens masked
        {"name": "combine_bwd 16384x4096", "op": "combine_bwd", "rows": 16384, "cols": 4096, "experts": 64, "k": 4, "type": "bf16", "mask": True},
        # a decode batch through 128 experts, four rows each: reading the weights is everything
        {"name": "experts 64 tokens", "op": "experts", "rows": 64, "cols": 2048, "inter": 768, "experts": 128, "k": 8,
         "act": "swiglu", "skew": 0.0, "mask": False, "keep": False},
        # a training batch over experts of uneven popularity, what the backward pass needs kept
        {"name": "experts 16384 tokens", "op": "experts", "rows": 16384, "cols": 4096, "inter": 1536, "experts": 64, "k": 4,
         "act": "swiglu", "skew": 1.0, "mask": False, "keep": True},
        # gradients down to the rows: many narrow experts, ragged segments of about 256 rows
        {"name": "experts_bwd 8192 tokens", "op": "experts_bwd", "rows": 8192, "cols": 2048, "inter": 512, "experts": 256, "k": 8,
         "act": "swiglu", "skew": 0.5, "mask": True},
        # gradients of all three weight matrices of 64 experts, FP32
        {"name": "experts_wgrad 16384 tokens", "op": "experts_wgrad", "rows": 16384, "cols": 4096, "inter": 1536, "experts": 64, "k": 4,
         "act": "swiglu", "skew": 1.0, "mask": False, "add": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "dispatch", "combine", "combine_bwd", "experts", "experts_bwd", "experts_wgrad"])
    if op in ("norm", "norm_bwd"):
        cols = 8 * _log(rng, 8, 2048)
        rows = min(_log(rng, 1, 20000), 29_000_000 // cols)
        c = {"op": op, "rows": rows, "cols": cols, "type": rng.choice(["bf16", "bf16", "fp32"]), "beta": rng.random() < 0.7}
        c["res" if op == "norm" else "dh"] = rng.random() < 0.6
        return c
    experts = _log(rng, 4, 512)
    k = rng.randint(1, min(experts, 10))
    if op in ("dispatch", "combine", "combine_bwd"):
        cols = 8 * _log(rng, 8, 1024)
        rows = min(_log(rng, 1, 60000), 125_000_000 // (cols * k))
        c = {"op": op, "rows": max(rows, 1), "cols": cols, "experts": experts, "k": k, "type": rng.choice(["bf16", "bf16", "fp32"]),
             "mask": rng.random() < 0.5}
        if op == "combine":
            c["weights"] = rng.random() < 0.7
        return c
    cols, inter = 32 * _log(rng, 8, 160), 32 * _log(rng, 4, 64)
    experts = max(1, min(experts, 400_000_000 // (cols * inter)))
    k = min(k, experts)
    rows = max(1, min(_log(rng, 1, 16384), 390_000_000_000 // (cols * inter * k)))
    c = {"op": op, "rows": rows, "cols": cols, "inter": inter, "experts": experts, "k": k, "act": rng.choice(ACTIVATIONS),
         "skew": round(rng.uniform(0.0, 1.5), 2), "mask": rng.random() < 0.4}
    if op == "experts":
        c["keep"] = rng.random() < 0.5
    if op == "experts_wgrad":
        c["add"] = rng.random() < 0.4
    return c


def _gated(act):
    return act != "relu2"


def prepare(case, seed):
    dev, bf = "cuda", torch.bfloat16
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0, mean=0.0, dtype=torch.float32):
        if dtype is torch.float32:
            return torch.randn(*shape, device=dev, generator=g) * scale + mean
        return torch.randn(*shape, device=dev, generator=g, dtype=bf) * scale + mean

    s, T, op, C = dict(case), case["rows"], case["op"], case["cols"]
    dt = {"bf16": bf, "fp32": torch.float32}[case.get("type", "bf16")]
    if op in ("norm", "norm_bwd"):
        # a residual stream wider than the update that is added to it, with a mean of its own
        s["gamma"] = normal(C, scale=0.1, mean=1.0).to(dt)
        s["beta_v"] = normal(C, scale=0.1).to(dt) if case["beta"] else None
        if op == "norm":
            s["x"] = normal(T, C).to(dt)
            s["res_v"] = normal(T, C, scale=2.0, mean=0.3).to(dt) if case["res"] else None
            s["out"] = {"y": torch.empty(T, C, dtype=dt, device=dev), "mean": torch.empty(T, device=dev), "rstd": torch.empty(T, device=dev)}
            if case["res"]:
                s["out"]["h"] = torch.empty(T, C, dtype=dt, device=dev)
        else:
            h = normal(T, C, scale=2.0, mean=0.3).to(dt)
            f = h.double()
            s.update(h=h, mean=f.mean(-1).float(), rstd=torch.rsqrt(f.var(-1, unbiased=False) + EPS).float(),
                     dy=normal(T, C).to(dt), dh_in=normal(T, C).to(dt) if case["dh"] else None)
            s["out"] = {"dx": torch.empty(T, C, dtype=dt, device=dev), "dgamma": torch.empty(C, device=dev)}
            if case["beta"]:
                s["out"]["dbeta"] = torch.empty(C, device=dev)
        return s

    E, k = case["experts"], case["k"]
    R = T * k
    # some experts are more popular than others
    logits = normal(T, E) + case.get("skew", 0.5) * normal(1, E)
    top = logits.topk(k, dim=-1)
    ids = top.indices.to(torch.int32)
    mask = (torch.rand(T, device=dev, generator=g) < 0.94) if case["mask"] else None
    s.update(ids=ids, token_mask=mask)
    if op == "dispatch":
        s["x"] = normal(T, C).to(dt)
        # rows behind the last expert's stay as they were
        s["out"] = torch.zeros(R, C, dtype=dt, device=dev)
        s["plan_out"] = {"counts": torch.empty(E, dtype=torch.int32, device=dev), "offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
                         "perm_src": torch.empty(R, dtype=torch.int32, device=dev), "inv": torch.empty(R, dtype=torch.int32, device=dev)}
        return s
    plan = _plain_sort(ids, E, mask)
    s["plan"] = plan
    if op in ("combine", "combine_bwd"):
        s["rows_in"] = normal(R, C).to(dt)
        s["w"] = torch.softmax(top.values, -1) if case.get("weights", True) else None
        if op == "combine":
            s["out"] = torch.empty(T, C, dtype=dt, device=dev)
        else:
            s["dy"] = normal(T, C).to(dt)
            s["out"] = {"drows": torch.zeros(R, C, dtype=dt, device=dev), "dtopk_w": torch.empty(T, k, device=dev)}
        return s

    I, act = case["inter"], case["act"]
    s["bounds"] = plan["offsets"].tolist()
    if op != "experts_wgrad":
        s["w_gate"] = normal(E, I, C, scale=0.02, dtype=bf) if _gated(act) else None
        s["w_up"] = normal(E, I, C, scale=0.02, dtype=bf)
        s["w_down"] = normal(E, C, I, scale=0.02, dtype=bf)
    rows_like = lambda n: torch.zeros(R, n, dtype=bf, device=dev)  # noqa: E731
    if op == "experts":
        s["x"] = normal(R, C, dtype=bf)
        s["out"] = {"out": rows_like(C)}
        if case["keep"]:
            s["out"].update(u=rows_like(I), h=rows_like(I))
            if _gated(act):
                s["out"]["g"] = rows_like(I)
        return s
    s["dout"] = normal(R, C, scale=0.01, dtype=bf)
    if op == "experts_bwd":
        s["saved"] = {"u": normal(R, I, dtype=bf)}
        if _gated(act):
            s["saved"]["g"] = normal(R, I, dtype=bf)
        s["out"] = {"drows": rows_like(C), "du": rows_like(I)}
        if _gated(act):
            s["out"]["dg"] = rows_like(I)
        return s
    s["x"] = normal(R, C, dtype=bf)
    s["saved"] = {"h": normal(R, I, scale=0.5, dtype=bf)}
    s["grads"] = {"du": normal(R, I, scale=0.01, dtype=bf)}
    if _gated(act):
        s["grads"]["dg"] = normal(R, I, scale=0.01, dtype=bf)
    shapes = {"w_gate": (E, I, C), "w_up": (E, I, C), "w_down": (E, C, I)}
    if not _gated(act):
        del shapes["w_gate"]
    s["out"] = {n: torch.zeros(*d, device=dev) for n, d in shapes.items()}
    if case["add"]:
        # the sums of earlier micro-batches; copied into the accumulator before each pass
        s["before"] = {n: normal(*d, scale=0.1) for n, d in shapes.items()}
    return s


# ---- the framework's calls ----

def _own(s):
    import nvfp4_mixture_experts_softmax_gb300 as moe
    op = s["op"]
    if op == "norm":
        return moe.add_layernorm(s["x"], s["res_v"], s["gamma"], s["beta_v"], EPS, out=s["out"])
    if op == "norm_bwd":
        if "workspace" not in s:
            s["workspace"] = moe.add_layernorm_backward_workspace(s["rows"], s["cols"], device=s["h"].device)
        return moe.add_layernorm_backward(s["dy"], s["h"], s["mean"], s["rstd"], s["gamma"], dh=s["dh_in"], out=s["out"],
                                          workspace=s["workspace"])
    if op == "dispatch":
        if "workspace" not in s:
            s["workspace"] = moe.sort_tokens_workspace(s["rows"], s["experts"], s["k"], device=s["x"].device)
        plan = moe.sort_tokens(s["ids"], s["experts"], mask=s["token_mask"], out=s["plan_out"], workspace=s["workspace"])
        return dict(plan, rows=moe.permute_tokens(s["x"], plan, out=s["out"]))
    if op == "combine":
        if s["w"] is None:
            return moe.permute_tokens_backward(s["rows_in"], s["plan"], s["rows"], out=s["out"])
        return moe.combine_tokens(s["rows_in"], s["plan"], s["w"], out=s["out"])
    if op == "combine_bwd":
        return moe.combine_tokens_backward(s["dy"], s["rows_in"], s["plan"], s["w"], out=s["out"])
    if "workspace" not in s:
        s["workspace"] = moe.experts_workspace(s["rows"] * s["k"], s["inter"], device=s["ids"].device)
    if op == "experts_wgrad":
        if s["add"]:
            for n, t in s["before"].items():
                s["out"][n].copy_(t)
        return moe.experts_weight_grad(s["x"], s["dout"], s["saved"], s["grads"], s["plan"], accumulate=s["add"], out=s["out"],
                                       workspace=s["workspace"])
    how = {"activation": "swiglu" if s["act"] == "swiglu_clamp" else s["act"], "out": s["out"], "workspace": s["workspace"]}
    if s["act"] in ("swiglu_clamp", "swiglu_oai"):
        how.update(swiglu_limit=LIMIT, swiglu_alpha=ALPHA)
    weights = s["w_gate"], s["w_up"], s["w_down"]
    if op == "experts":
        return moe.experts_forward(s["x"], s["plan"], *weights, **how)
    return moe.experts_backward(s["dout"], s["saved"], s["plan"], *weights, **how)


# ---- the plain forms: 32 bits ----

def _plain_norm(s):
    h = s["x"].float()
    if s["res_v"] is not None:
        h = (h + s["res_v"].float()).to(s["x"].dtype).float()
    mean = h.mean(-1, keepdim=True)
    d = h - mean
    rstd = 1.0 / torch.sqrt(d.square().mean(-1, keepdim=True) + EPS)
    y = d * rstd * s["gamma"].float()
    if s["beta_v"] is not None:
        y = y + s["beta_v"].float()
    o = {"y": y.to(s["x"].dtype), "mean": mean.squeeze(-1), "rstd": rstd.squeeze(-1)}
    if s["res_v"] is not None:
        o["h"] = h.to(s["x"].dtype)
    return o


def _plain_norm_bwd(s):
    dy, r = s["dy"].float(), s["rstd"][:, None]
    xh = (s["h"].float() - s["mean"][:, None]) * r
    a = dy * s["gamma"].float()
    dx = r * (a - a.mean(-1, keepdim=True) - xh * (a * xh).mean(-1, keepdim=True))
    if s["dh_in"] is not None:
        dx = dx + s["dh_in"].float()
    o = {"dx": dx.to(s["dy"].dtype), "dgamma": (dy * xh).sum(0)}
    if s["beta"]:
        o["dbeta"] = dy.sum(0)
    return o


def _plain_sort(ids, E, mask):
    """Assignments t * k + j in the order of their experts, masked tokens' left out."""
    T, k = ids.shape
    e = ids.long()
    if mask is not None:
        e = torch.where(mask[:, None], e, E)
    e = e.reshape(-1)
    order = torch.sort(e, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, e, torch.ones_like(e))[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    place = torch.arange(T * k, device=ids.device)
    kept = place < offsets[-1]
    inv = torch.empty_like(e)
    inv[order] = torch.where(kept, place, -1)
    perm = torch.where(kept, order // k, -1)
    i32 = lambda t: t.to(torch.int32)  # noqa: E731
    return {"counts": i32(counts), "offsets": i32(offsets), "perm_src": i32(perm), "inv": i32(inv)}


def _plain_dispatch(s):
    plan = _plain_sort(s["ids"], s["experts"], s["token_mask"])
    src = plan["perm_src"].long()
    rows = torch.where((src >= 0)[:, None], s["x"][src.clamp(min=0)], torch.zeros((), dtype=s["x"].dtype, device=src.device))
    return dict(plan, rows=rows)


def _gathered(s):
    """The rows of each token's assignments [T, k, cols] in 32 bits, zeros where there is none."""
    inv = s["plan"]["inv"].long().reshape(s["rows"], s["k"])
    got = s["rows_in"][inv.clamp(min=0)].float()
    return torch.where((inv >= 0)[..., None], got, 0.0), inv


def _plain_combine(s):
    got, _ = _gathered(s)
    if s["w"] is not None:
        got = got * s["w"][..., None]
    return got.sum(1).to(s["rows_in"].dtype)


def _plain_combine_bwd(s):
    got, inv = _gathered(s)
    dy = s["dy"].float()[:, None, :]
    dw = (got * dy).sum(-1)
    drows = torch.zeros_like(s["rows_in"])
    keep = inv >= 0
    drows[inv[keep]] = (s["w"][..., None] * dy).to(drows.dtype)[keep]
    return {"drows": drows, "dtopk_w": dw}


def _activation(g, u, act):
    if act == "relu2":
        return torch.clamp(u, min=0).square()
    if act != "swiglu":
        g, u = torch.clamp(g, max=LIMIT), torch.clamp(u, -LIMIT, LIMIT)
    if act == "swiglu_oai":
        return (u + 1) * g / (1 + torch.exp(-ALPHA * g))
    return g / (1 + torch.exp(-g)) * u


def _activation_grad(g, u, act):
    """Derivatives of the activation by g and u."""
    if act == "relu2":
        return None, 2 * torch.clamp(u, min=0)
    gc, uc, a, one = g, u, 1.0, 0.0
    if act != "swiglu":
        gc, uc = torch.clamp(g, max=LIMIT), torch.clamp(u, -LIMIT, LIMIT)
    if act == "swiglu_oai":
        a, one = ALPHA, 1.0
    sg = 1 / (1 + torch.exp(-a * gc))
    fg, fu = (uc + one) * sg * (1 + a * gc * (1 - sg)), gc * sg
    if act != "swiglu":
        fg, fu = fg * (g <= LIMIT), fu * (u.abs() <= LIMIT)
    return fg, fu


def _segments(s):
    return [(e, a, b) for e, (a, b) in enumerate(zip(s["bounds"][:-1], s["bounds"][1:])) if b > a]


def _plain_experts(s):
    bf = torch.bfloat16
    o = {n: torch.zeros_like(t) for n, t in s["out"].items()}
    for e, a, b in _segments(s):
        x = s["x"][a:b].float()
        g = x @ s["w_gate"][e].float().t() if s["w_gate"] is not None else None
        u = x @ s["w_up"][e].float().t()
        h = _activation(g, u, s["act"]).to(bf)     # the down projection reads BF16
        o["out"][a:b] = (h.float() @ s["w_down"][e].float().t()).to(bf)
        for n, t in (("g", g), ("u", u), ("h", h)):
            if n in o:
                o[n][a:b] = t.to(bf)
    return o


def _plain_experts_bwd(s):
    bf = torch.bfloat16
    o = {n: torch.zeros_like(t) for n, t in s["out"].items()}
    for e, a, b in _segments(s):
        dh = s["dout"][a:b].float() @ s["w_down"][e].float()
        g = s["saved"]["g"][a:b].float() if "g" in s["saved"] else None
        fg, fu = _activation_grad(g, s["saved"]["u"][a:b].float(), s["act"])
        du = (dh * fu).to(bf)                      # the products below read BF16
        dx = du.float() @ s["w_up"][e].float()
        o["du"][a:b] = du
        if fg is not None:
            dg = (dh * fg).to(bf)
            dx = dx + dg.float() @ s["w_gate"][e].float()
            o["dg"][a:b] = dg
        o["drows"][a:b] = dx.to(bf)
    return o


def _plain_experts_wgrad(s):
    o = {n: t.clone() if s["add"] else torch.zeros_like(t) for n, t in (s["before"] if s["add"] else s["out"]).items()}
    for e, a, b in _segments(s):
        x = s["x"][a:b].float()
        o["w_up"][e] += s["grads"]["du"][a:b].float().t() @ x
        if "w_gate" in o:
            o["w_gate"][e] += s["grads"]["dg"][a:b].float().t() @ x
        o["w_down"][e] += s["dout"][a:b].float().t() @ s["saved"]["h"][a:b].float()
    return o


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "dispatch": _plain_dispatch, "combine": _plain_combine,
            "combine_bwd": _plain_combine_bwd, "experts": _plain_experts, "experts_bwd": _plain_experts_bwd,
            "experts_wgrad": _plain_experts_wgrad}[state["op"]](state)


def work(case):
    T, C, op = case["rows"], case["cols"], case["op"]
    b = 4 if case.get("type") == "fp32" else 2
    if op == "norm":
        return {"bytes": T * C * b * (4 if case["res"] else 2) + 8 * T + 2 * C * b, "flops": 9.0 * T * C}
    if op == "norm_bwd":
        return {"bytes": T * C * b * (4 if case["dh"] else 3) + 8 * T + C * (b + 8), "flops": 14.0 * T * C}
    E, k = case["experts"], case["k"]
    live = 0.94 if case["mask"] else 1.0           # the share of the tokens that are not masked
    R = T * k * live
    if op == "dispatch":
        return {"bytes": live * T * C * b + R * C * b + 12.0 * T * k + 8 * E, "flops": 0.0}
    if op == "combine":
        return {"bytes": R * C * b + T * C * b + 4 * T * k + (4 * R if case["weights"] else 0), "flops": 2.0 * R * C}
    if op == "combine_bwd":
        return {"bytes": 2 * R * C * b + live * T * C * b + 12.0 * T * k, "flops": 3.0 * R * C}
    I, n = case["inter"], 3 if _gated(case["act"]) else 2
    used = E * (1 - (1 - k / E) ** (T * live))     # experts that get a row, of E equally popular ones
    flops = 2.0 * R * C * I * n
    if op == "experts":
        return {"bytes": used * n * C * I * 2 + R * C * 4 + (R * I * 2 * n if case["keep"] else 0), "flops": flops}
    if op == "experts_bwd":
        return {"bytes": used * n * C * I * 2 + R * C * 4 + R * I * 4 * (n - 1), "flops": flops}
    return {"bytes": E * n * C * I * (12 if case["add"] else 4) + R * C * 4 + R * I * 2 * n, "flops": flops}


# ---- the definitions in 64 bits ----

def exact(case, seed):
    s, T, op, f64 = prepare(case, seed), case["rows"], case["op"], torch.float64
    if op == "norm":
        h = s["x"].to(f64)
        if case["res"]:
            h = (h + s["res_v"].to(f64)).to(s["x"].dtype).to(f64)     # the residual stream's own type
        var, mu = torch.var_mean(h, 1, correction=0)
        y = (h - mu[:, None]) / torch.sqrt(var + EPS)[:, None] * s["gamma"].to(f64)
        if case["beta"]:
            y += s["beta_v"].to(f64)
        o = {"y": y, "mean": mu, "rstd": (var + EPS) ** -0.5}
        if case["res"]:
            o["h"] = h
        return o
    if op == "norm_bwd":
        # the statistics are inputs, and the gradients are those of the norm that has them
        C, dy = case["cols"], s["dy"].to(f64)
        n = (s["h"].to(f64) - s["mean"].to(f64).view(-1, 1)) * s["rstd"].to(f64).view(-1, 1)
        gy = dy * s["gamma"].to(f64)
        dx = (gy * C - gy.sum(1, keepdim=True) - n * torch.einsum("tc,tc->t", gy, n)[:, None]) * (s["rstd"].to(f64)[:, None] / C)
        if case["dh"]:
            dx += s["dh_in"].to(f64)
        o = {"dx": dx, "dgamma": torch.einsum("tc,tc->c", dy, n)}
        if case["beta"]:
            o["dbeta"] = torch.ones(T, dtype=f64, device=dy.device) @ dy
        return o
    k = case["k"]
    if op == "dispatch":
        E, R = case["experts"], T * k
        flat = s["ids"].reshape(-1).long()
        live = torch.ones(R, dtype=torch.bool, device=flat.device) if s["token_mask"] is None else s["token_mask"].repeat_interleave(k)
        a = live.nonzero().squeeze(1)                                     # kept assignments, in order
        a = a[torch.argsort(flat[a] * R + a)]
        i32 = torch.int32
        count = torch.bincount(flat[a], minlength=E)
        off = torch.zeros(E + 1, dtype=i32, device=flat.device)
        off[1:] = count.cumsum(0).to(i32)
        src = torch.full((R,), -1, dtype=i32, device=flat.device)
        src[:a.numel()] = (a // k).to(i32)
        inv = torch.full((R,), -1, dtype=i32, device=flat.device)
        inv[a] = torch.arange(a.numel(), dtype=i32, device=flat.device)
        rows = torch.zeros(R, case["cols"], dtype=s["x"].dtype, device=flat.device)
        rows[:a.numel()] = s["x"].index_select(0, a // k)
        return {"counts": count.to(i32), "offsets": off, "perm_src": src, "inv": inv, "rows": rows.to(f64)}
    if op in ("combine", "combine_bwd"):
        inv = s["plan"]["inv"].long().view(T, k)
        if op == "combine":
            y = torch.zeros(T, case["cols"], dtype=f64, device=inv.device)
            for j in range(k):
                t = (inv[:, j] >= 0).nonzero().squeeze(1)
                part = s["rows_in"].index_select(0, inv[t, j]).to(f64)
                y[t] += part if s["w"] is None else part * s["w"][t, j].to(f64)[:, None]
            return y
        dr, dw = torch.zeros(T * k, case["cols"], dtype=f64, device=inv.device), torch.zeros(T, k, dtype=f64, device=inv.device)
        for j in range(k):
            t = (inv[:, j] >= 0).nonzero().squeeze(1)
            p, dy = inv[t, j], s["dy"].index_select(0, t).to(f64)
            dw[t, j] = torch.einsum("tc,tc->t", s["rows_in"].index_select(0, p).to(f64), dy)
            dr[p] = dy * s["w"][t, j].to(f64)[:, None]
        return {"drows": dr, "dtopk_w": dw}

    bf, act, cuts = torch.bfloat16, case["act"], s["bounds"]
    if op == "experts_wgrad":
        o = {n: (s["before"][n].to(f64) if case["add"] else torch.zeros(t.shape, dtype=f64, device=t.device)) for n, t in s["out"].items()}
    else:
        o = {n: torch.zeros(t.shape, dtype=f64, device=t.device) for n, t in s["out"].items()}
    for e in range(case["experts"]):
        r = slice(cuts[e], cuts[e + 1])
        if cuts[e] == cuts[e + 1]:
            continue
        if op == "experts":
            x = s["x"][r].to(f64)
            u = torch.einsum("rc,ic->ri", x, s["w_up"][e].to(f64))
            g = torch.einsum("rc,ic->ri", x, s["w_gate"][e].to(f64)) if _gated(act) else None
            h = _exact_activation(g, u, act)
            o["out"][r] = torch.einsum("ri,ci->rc", h.to(bf).to(f64), s["w_down"][e].to(f64))
            for n, t in (("g", g), ("u", u), ("h", h)):
                if n in o:
                    o[n][r] = t
        elif op == "experts_bwd":
            dh = torch.einsum("rc,ci->ri", s["dout"][r].to(f64), s["w_down"][e].to(f64))
            u = s["saved"]["u"][r].to(f64).requires_grad_()
            g = s["saved"]["g"][r].to(f64).requires_grad_() if _gated(act) else None
            leaves = (g, u) if _gated(act) else (u,)
            grads = dict(zip(("dg", "du") if _gated(act) else ("du",), torch.autograd.grad(_exact_activation(g, u, act), leaves, dh)))
            for n, d in grads.items():
                o[n][r] = d
                o["drows"][r] += torch.einsum("ri,ic->rc", d.to(bf).to(f64), s["w_gate" if n == "dg" else "w_up"][e].to(f64))
        else:
            x, d = s["x"][r].to(f64), s["dout"][r].to(f64)
            o["w_up"][e] += torch.einsum("ri,rc->ic", s["grads"]["du"][r].to(f64), x)
            if "w_gate" in o:
                o["w_gate"][e] += torch.einsum("ri,rc->ic", s["grads"]["dg"][r].to(f64), x)
            o["w_down"][e] += torch.einsum("rc,ri->ci", d, s["saved"]["h"][r].to(f64))
    return o


def _exact_activation(g, u, act):
    if act == "relu2":
        return torch.relu(u) ** 2
    if act == "swiglu":
        return torch.nn.functional.silu(g) * u
    low, mid = torch.minimum(g, torch.full_like(g, LIMIT)), torch.clamp(u, min=-LIMIT, max=LIMIT)
    if act == "swiglu_clamp":
        return torch.nn.functional.silu(low) * mid
    return (mid + 1) * low * torch.sigmoid(ALPHA * low)
