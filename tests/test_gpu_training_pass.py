"""The training pass of one block, as it is used: layer norm, router, sort, experts, combine, losses, and the gradients back
through all of them to the residual stream and every weight, against 64-bit autograd of the same chain.

The chosen ids are held fixed.  Every stage rounds to BF16 (2^-9 of a value's size on average half of 2^-8): y, g, u, h, the
rows, dy and the gradients on their way; a gradient passes at most ten of them: relative L2 within 10 * 2^-9 of the
exact chain."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


class Block:
    def __init__(self, moe, T, H, E, k, I, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.n = lambda *s, scale=1.0: torch.randn(*s, device="cuda", generator=g) * scale  # noqa: E731
        n = self.n
        self.moe, self.T, self.H, self.E, self.k, self.I = moe, T, H, E, k, I
        self.x, self.res = n(T, H).to(BF16), n(T, H, scale=2.0).to(BF16)
        self.gamma, self.beta = (1 + 0.1 * n(H)).to(BF16), (0.1 * n(H)).to(BF16)
        self.wr = n(E, H, scale=H ** -0.5)
        self.wg, self.wu = n(E, I, H, scale=H ** -0.5).to(BF16), n(E, I, H, scale=H ** -0.5).to(BF16)
        self.wd = n(E, H, I, scale=I ** -0.5).to(BF16)
        self.mask = torch.arange(T, device="cuda") < T - max(1, T // 9) if T > 1 else None
        self.dout, self.gl = n(T, H, scale=0.1).to(BF16), torch.tensor([1.0, 0.1], device="cuda")

    def step(self):
        m = self.moe
        o = m.add_layernorm(self.x, self.res, self.gamma, self.beta, want_stats=True)
        lg = o["y"].float() @ self.wr.t()
        p = m.plan(lg, self.k)
        ids, w = p["topk_ids"], p["topk_w"]
        plan = m.sort_tokens(ids, self.E, mask=self.mask)
        rows = m.permute_tokens(o["y"], plan)
        f = m.experts_forward(rows, plan, self.wg, self.wu, self.wd, keep=True)
        out = m.combine_tokens(f["out"], plan, w)
        st = m.router_loss(lg, ids, mask=self.mask)
        # and back
        c = m.combine_tokens_backward(self.dout, f["out"], plan, w)
        b = m.experts_backward(c["drows"], f, plan, self.wg, self.wu, self.wd)
        dw = m.experts_weight_grad(rows, c["drows"], f, b, plan)
        dl = m.router_loss_backward(lg, ids, st, self.gl, grad_topk_w=c["dtopk_w"], mask=self.mask)
        dy = (m.permute_tokens_backward(b["drows"], plan, self.T).float() + dl @ self.wr).to(BF16)
        nb = m.add_layernorm_backward(dy, o["h"], o["mean"], o["rstd"], self.gamma, dh=self.dout)
        return dict(out=out, ids=ids, losses=st["losses"], counts=st["counts"], dwr=dl.t() @ o["y"].float(), **nb, **dw), o["h"], plan


def exact(blk, h, ids, counts):
    leaves = [t.double().requires_grad_() for t in (h, blk.gamma, blk.beta, blk.wr, blk.wg, blk.wu, blk.wd)]
    hd, ga, be, wr, wg, wu, wd = leaves
    m = blk.mask.double() if blk.mask is not None else torch.ones(blk.T, device="cuda", dtype=torch.float64)
    mu = hd.mean(-1, keepdim=True)
    y = (hd - mu) / torch.sqrt((hd - mu).square().mean(-1, keepdim=True) + 1e-5) * ga + be
    lg = y @ wr.t()
    w = torch.softmax(lg.gather(1, ids.long()), -1)
    out = torch.zeros_like(y)
    for e in range(blk.E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if blk.mask is not None:
            t, j = t[blk.mask[t]], j[blk.mask[t]]
        if t.numel():
            g, u = y[t] @ wg[e].t(), y[t] @ wu[e].t()
            out = out.index_add(0, t, (torch.nn.functional.silu(g) * u) @ wd[e].t() * w[t, j][:, None])
    n, f = m.sum(), counts.double()
    p = torch.softmax(lg, -1)
    loss = torch.stack([blk.E * (f / (n * blk.k) * (p * m[:, None]).sum(0) / n).sum(), ((torch.logsumexp(lg, -1) ** 2) * m).sum() / n])
    goal = ((out + hd) * blk.dout.double()).sum() + (loss * blk.gl.double()).sum()
    grads = torch.autograd.grad(goal, leaves)
    return dict(zip(("dx", "dgamma", "dbeta", "dwr", "w_gate", "w_up", "w_down"), grads), out=out.detach(), losses=loss.detach())


@pytest.mark.parametrize("T,H,E,k,I", [(1, 64, 4, 2, 32), (90, 256, 12, 4, 96), (700, 288, 6, 2, 544)])
def test_training_step(moe, T, H, E, k, I):
    blk = Block(moe, T, H, E, k, I)
    got, h, plan = blk.step()
    if blk.mask is not None:
        assert int(plan["offsets"][-1]) == int(blk.mask.sum()) * k and not got["out"][~blk.mask].any()
    want = exact(blk, h, got["ids"], got["counts"])
    for name, ref in want.items():
        rel = float((got[name].double() - ref).norm() / (ref.norm() + 1e-30))
        assert rel <= 10 * 2.0 ** -9, (name, rel)


def test_captured_step(moe):
    """The whole step as one graph, replayed on other inputs (and another routing)."""
    blk = Block(moe, 200, 256, 16, 4, 160, seed=2)
    blk.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rec, _, rplan = blk.step()
    blk.x.copy_(blk.n(200, 256))
    blk.wr.copy_(blk.n(16, 256, scale=1 / 16))
    g.replay()
    got, _, plan = blk.step()
    torch.cuda.synchronize()
    assert torch.equal(rplan["inv"], plan["inv"])
    assert all(torch.equal(rec[k], got[k]) for k in got)


def test_gradients_of_two_micro_batches(moe):
    """accumulate adds the second batch's gradients to the first's."""
    blk = Block(moe, 120, 128, 6, 2, 64, seed=3)
    first, _, _ = blk.step()
    kept = {k: first[k].clone() for k in ("w_gate", "w_up", "w_down")}
    blk.x.copy_(blk.n(120, 128))
    second, _, _ = blk.step()
    m = blk.moe
    o = m.add_layernorm(blk.x, blk.res, blk.gamma, blk.beta)
    p = m.plan(o["y"].float() @ blk.wr.t(), 2)
    plan = m.sort_tokens(p["topk_ids"], 6, mask=blk.mask)
    rows = m.permute_tokens(o["y"], plan)
    f = m.experts_forward(rows, plan, blk.wg, blk.wu, blk.wd, keep=True)
    c = m.combine_tokens_backward(blk.dout, f["out"], plan, p["topk_w"])
    b = m.experts_backward(c["drows"], f, plan, blk.wg, blk.wu, blk.wd)
    acc = {k: v.clone() for k, v in kept.items()}
    m.experts_weight_grad(rows, c["drows"], f, b, plan, accumulate=True, out=acc)
    for k in acc:     # at most 1024 rows an expert: one chain, one addition
        assert torch.equal(acc[k], kept[k] + second[k])
