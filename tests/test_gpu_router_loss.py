"""Router losses, per-expert counts and the gradient of the logits against the formulas in 64 bits.

Counts and tokens are integers: equal.  Probabilities of one token: exp and its argument (|l - max|
<= 40 here: 2^-24 * 40 absolute), a sum of at most 32 + 5 additions, a division: < 128 * 2^-24
relative; their mean over T tokens adds at most T roundings: (T + 128) * 2^-24.  The losses are
sums of those.  Gradients: each of the three terms (balance, z, top-k) carries at most ~256
roundings of quantities bounded by the term's own magnitudes: 2^-16 of their sum."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
G_REL = 2.0 ** -16
ROUTERS = ("softmax", "sqrtsoftplus")


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


def scores(l, router):
    if router == "softmax":
        return torch.exp(l - torch.logsumexp(l, -1, keepdim=True))
    return torch.sqrt(torch.nn.functional.softplus(l, threshold=1e9))


def make(T, E, k, seed=0, masked=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = torch.randn(T, E, device="cuda", generator=g) * 2 + torch.randn(1, E, device="cuda", generator=g)
    ids = torch.rand(T, E, device="cuda", generator=g).topk(k, -1).indices.int()
    gw = torch.randn(T, k, device="cuda", generator=g)
    mask = (torch.rand(T, device="cuda", generator=g) < 0.7) if masked else None
    return l, ids, gw, mask


def forward_reference(l, ids, mask, router):
    T, E = l.shape
    k = ids.shape[1]
    keep = (torch.ones(T, device="cuda", dtype=torch.bool) if mask is None else mask.bool()) & (l > -float("inf")).any(-1)
    ld, idk = l.double()[keep], ids.long()[keep]
    n = int(keep.sum())
    s = scores(ld, router)
    p = s / s.sum(-1, keepdim=True)
    counts = torch.bincount(idk.reshape(-1), minlength=E)
    P = p.sum(0) / max(n, 1)
    lse = torch.logsumexp(ld, -1)
    bal = E * (counts.double() / max(n * k, 1) * P).sum()
    return bal, (lse ** 2).sum() / max(n, 1), counts, n, P


CASES = [(1, 8, 2), (1, 1, 1), (5, 7, 3), (64, 128, 8), (333, 256, 8), (77, 60, 4), (50, 64, 6), (9, 1024, 32),
         (130, 33, 5), (41, 510, 9), (2049, 16, 2), (20, 1021, 7), (31, 32, 32), (5000, 96, 4)]


@pytest.mark.parametrize("T,E,k", CASES)
@pytest.mark.parametrize("router", ROUTERS)
@pytest.mark.parametrize("masked", [False, True])
def test_losses_and_counts(moe, T, E, k, router, masked):
    l, ids, _, mask = make(T, E, k, T + E, masked)
    ws = moe.router_loss_workspace(T, E)
    o = moe.router_loss(l, ids, mask=mask, router=router, workspace=ws)
    bal, z, counts, n, P = forward_reference(l, ids, mask, router)
    assert moe.last_device_status(ws) == 0
    assert torch.equal(o["counts"].long(), counts) and int(o["tokens"]) == n
    tol = (T + 128) * U
    assert bool(((o["probs"].double() - P).abs() <= tol * P + 1e-30).all())
    assert abs(float(o["losses"][0]) - float(bal)) <= tol * abs(float(bal)) + 1e-30
    assert abs(float(o["losses"][1]) - float(z)) <= tol * 4 * abs(float(z)) + 1e-12
    again = moe.router_loss(l, ids, mask=mask, router=router)
    assert all(torch.equal(again[x], o[x]) for x in o)


def gradient_reference(l, ids, gw, mask, router, gl):
    """Gradient by autograd in 64 bits, and the sum of the magnitudes of its terms."""
    T, E = l.shape
    k = ids.shape[1]
    keep = (torch.ones(T, device="cuda", dtype=torch.bool) if mask is None else mask.bool())
    _, _, counts, n, _ = forward_reference(l, ids, mask, router)
    n = max(n, 1)
    ld = l.double().requires_grad_()
    s = scores(ld, router)
    p = s / s.sum(-1, keepdim=True)
    f = counts.double() / (n * k)
    lse = torch.logsumexp(ld, -1)
    kd = keep.double()
    sk = s.gather(1, ids.long())
    w = sk / sk.sum(-1, keepdim=True)
    terms = []
    for v in (gl[0] * E * (f * (p * kd[:, None]).sum(0) / n).sum(), gl[1] * (lse ** 2 * kd).sum() / n,
              (w * gw.double() * kd[:, None]).sum()):
        terms.append(torch.autograd.grad(v, ld, retain_graph=True)[0])
    # magnitudes before the subtractions inside a term; ds/dl <= s for either router's scores
    pd, sm = p.detach(), scores(l.double(), "softmax")
    size = abs(gl[0]) * E / n * pd * (f + (f * pd).sum(-1, keepdim=True)) + terms[1].abs()
    wt = w.detach() * (gw.double().abs() + (gw.double().abs() * w.detach()).sum(-1, keepdim=True))
    size = size.scatter_add(1, ids.long(), wt)
    return sum(terms), size * kd[:, None] + sm * 1e-30


@pytest.mark.parametrize("T,E,k", CASES)
@pytest.mark.parametrize("router", ROUTERS)
def test_gradient(moe, T, E, k, router):
    l, ids, gw, mask = make(T, E, k, T * 2 + E, masked=T > 4)
    stats = moe.router_loss(l, ids, mask=mask, router=router)
    gl = [0.7, -0.3]
    glt = torch.tensor(gl, device="cuda")
    got = moe.router_loss_backward(l, ids, stats, glt, grad_topk_w=gw, mask=mask, router=router)
    want, size = gradient_reference(l, ids, gw, mask, router, gl)
    assert bool(((got.double() - want).abs() <= G_REL * size + 1e-30).all()), float(((got.double() - want).abs() / (size + 1e-30)).max())
    if mask is not None:
        assert not got[~mask].any()
    # the parts alone, and the same bits again
    a = moe.router_loss_backward(l, ids, stats, glt, mask=mask, router=router)
    b = moe.router_loss_backward(l, ids, stats, grad_topk_w=gw, mask=mask, router=router)
    assert bool(((a.double() + b.double() - want).abs() <= G_REL * size + 1e-30).all())
    assert torch.equal(got, moe.router_loss_backward(l, ids, stats, glt, grad_topk_w=gw, mask=mask, router=router))


@pytest.mark.parametrize("router", ROUTERS)
def test_gradient_against_differences(moe, router):
    """Along random directions, against central differences of the losses in 64 bits (the counts
    held fixed)."""
    l, ids, gw, mask = make(12, 20, 3, 5, masked=True)
    stats = moe.router_loss(l, ids, mask=mask, router=router)
    gl = [0.9, 0.2]
    d = moe.router_loss_backward(l, ids, stats, torch.tensor(gl, device="cuda"), grad_topk_w=gw, mask=mask, router=router)
    f, n = stats["counts"].double() / (int(stats["tokens"]) * 3), int(stats["tokens"])

    def goal(x):
        s = scores(x, router)
        p = s / s.sum(-1, keepdim=True)
        sk = s.gather(1, ids.long())
        w = sk / sk.sum(-1, keepdim=True)
        m = mask.double()
        return float(gl[0] * 20 * (f * (p * m[:, None]).sum(0) / n).sum() + gl[1] * (torch.logsumexp(x, -1) ** 2 * m).sum() / n
                     + (w * gw.double() * m[:, None]).sum())

    rng = torch.Generator(device="cuda").manual_seed(3)
    for _ in range(4):
        v = torch.randn(12, 20, device="cuda", generator=rng, dtype=torch.float64)
        num = (goal(l.double() + 1e-4 * v) - goal(l.double() - 1e-4 * v)) / 2e-4
        assert abs(num - float((d.double() * v).sum())) <= 1e-5 * float((d.double() * v).abs().sum()) + 1e-6


@pytest.mark.parametrize("router", ROUTERS)
def test_extreme_logits(moe, router):
    """Experts masked with -infinity or the type's lowest value, far apart logits, rows with
    nothing left, and NaN in rows that do not count."""
    l, ids, gw, _ = make(8, 40, 4, 11)
    ids[:] = torch.arange(4, device="cuda", dtype=torch.int32)
    l[0, 4:] = -float("inf")
    l[1, 6:] = torch.finfo(torch.float32).min
    l[2] = -float("inf")
    l[3, 5] = 80.0
    l[4] = -60.0 + l[4]
    l[5] = float("nan")
    l[6, 7] = float("inf")
    mask = torch.tensor([1, 1, 1, 1, 1, 0, 0, 1], device="cuda", dtype=torch.uint8)
    o = moe.router_loss(l, ids, mask=mask, router=router)
    assert int(o["tokens"]) == 5
    use = torch.tensor([0, 1, 3, 4, 7], device="cuda")
    bal, z, counts, n, P = forward_reference(l[use], ids[use], None, router)
    assert torch.equal(o["counts"].long(), counts)
    assert bool(((o["probs"].double() - P).abs() <= 256 * U * P + 1e-30).all())
    assert abs(float(o["losses"][0] - bal)) <= 256 * U * float(bal) and abs(float(o["losses"][1] - z)) <= 256 * U * float(z)
    d = moe.router_loss_backward(l, ids, o, torch.tensor([1.0, 1.0], device="cuda"), grad_topk_w=gw, mask=mask, router=router)
    assert bool(d.isfinite().all()) and not d[2].any() and not d[5].any() and not d[6].any()
    assert not d[0, 4:].any()
    # without the mask the NaN row reaches the losses and its own gradient row only
    o2 = moe.router_loss(l, ids, router=router)
    assert bool(o2["losses"].isnan().all())
    d2 = moe.router_loss_backward(l, ids, o, torch.tensor([1.0, 1.0], device="cuda"), grad_topk_w=gw, router=router)
    assert bool(d2[5].isnan().any()) and torch.equal(d2[[0, 1, 2, 3, 4, 7]], d[[0, 1, 2, 3, 4, 7]])


def test_nothing_counts(moe):
    l, ids, gw, _ = make(6, 12, 3, 12)
    mask = torch.zeros(6, dtype=torch.bool, device="cuda")
    o = moe.router_loss(l, ids, mask=mask)
    assert not o["losses"].any() and not o["counts"].any() and not o["probs"].any() and int(o["tokens"]) == 0
    assert not moe.router_loss_backward(l, ids, o, torch.ones(2, device="cuda"), grad_topk_w=gw, mask=mask).any()
    o = moe.router_loss(l[:0], ids[:0])
    assert not o["losses"].any() and not o["counts"].any() and int(o["tokens"]) == 0
    assert moe.router_loss_backward(l[:0], ids[:0], o, torch.ones(2, device="cuda")).shape == (0, 12)


@pytest.mark.parametrize("E", [24, 40, 200, 1000])
def test_ids_outside_and_twice(moe, E):
    l, ids, gw, _ = make(70, E, 4, 13)
    ids[3, 1], ids[9, 0] = -1, E
    ids[5, 2] = ids[5, 0]
    ids[6] = ids[6, 0].clone()
    ws = moe.router_loss_workspace(70, E)
    o = moe.router_loss(l, ids, workspace=ws)
    assert moe.last_device_status(ws) == -1
    ok = (ids >= 0) & (ids < E)
    assert torch.equal(o["counts"].long(), torch.bincount(ids[ok].long(), minlength=E))
    d = moe.router_loss_backward(l, ids, o, grad_topk_w=gw)
    ld = l.double()
    want = torch.zeros_like(ld)
    for t in range(70):
        i = ids[t][ok[t]].long()
        w = torch.softmax(ld[t, i], 0)
        g = gw[t][ok[t]].double()
        want[t].index_add_(0, i, w * (g - (g * w).sum()))
    assert float((d.double() - want).abs().max()) <= G_REL * 4 * float(gw.abs().max())
    assert torch.equal(d, moe.router_loss_backward(l, ids, o, grad_topk_w=gw))
    moe.router_loss(l, ids.clamp(0, E - 1), workspace=ws)
    assert moe.last_device_status(ws) == 0


def test_unaligned_rows_side_stream_and_graph(moe):
    l, ids, gw, mask = make(100, 64, 4, 14, masked=True)
    flat = torch.empty(100 * 64 + 1, device="cuda")
    shifted = flat[1:].reshape(100, 64)
    shifted.copy_(l)
    o = moe.router_loss(l, ids, mask=mask)
    p = moe.router_loss(shifted, ids, mask=mask)
    assert torch.equal(o["counts"], p["counts"])
    assert float((o["losses"] - p["losses"]).abs().max()) <= 256 * U * float(o["losses"].max())
    gl = torch.ones(2, device="cuda")
    d = moe.router_loss_backward(l, ids, o, gl, grad_topk_w=gw, mask=mask)
    d2 = moe.router_loss_backward(shifted, ids, o, gl, grad_topk_w=gw, mask=mask)
    assert float((d - d2).abs().max()) <= G_REL * float(gw.abs().max())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q = moe.router_loss(l, ids, mask=mask, stream=s)
    s.synchronize()
    assert all(torch.equal(q[x], o[x]) for x in o)
    out, ws, dl = {x: torch.empty_like(v) for x, v in o.items()}, moe.router_loss_workspace(100, 64), torch.empty_like(l)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.router_loss(l, ids, mask=mask, out=out, workspace=ws)
        moe.router_loss_backward(l, ids, out, gl, grad_topk_w=gw, mask=mask, dlogits=dl)
    l2 = make(100, 64, 4, 15)[0]
    l.copy_(l2)
    graph.replay()
    want = moe.router_loss(l, ids, mask=mask)
    dw = moe.router_loss_backward(l, ids, want, gl, grad_topk_w=gw, mask=mask)
    torch.cuda.synchronize()
    assert all(torch.equal(out[x], want[x]) for x in want) and torch.equal(dl, dw)


def test_refusals(moe):
    l, ids, gw, _ = make(6, 12, 3)
    with pytest.raises(ValueError, match="logits"):
        moe.router_loss(l.bfloat16(), ids)
    with pytest.raises(ValueError, match="topk_ids"):
        moe.router_loss(l, ids.long())
    with pytest.raises(ValueError, match="topk_ids"):
        moe.router_loss(l, ids[:3])
    with pytest.raises(ValueError, match="mask"):
        moe.router_loss(l, ids, mask=torch.ones(6, device="cuda"))
    with pytest.raises(ValueError, match="unknown router"):
        moe.router_loss(l, ids, router="sigmoid")
    with pytest.raises(ValueError, match="grad_losses"):
        moe.router_loss_backward(l, ids, moe.router_loss(l, ids), torch.ones(3, device="cuda"))
    with pytest.raises(RuntimeError, match="WORKSPACE_TOO_SMALL"):
        moe.router_loss(l, ids, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    wide = torch.zeros(1, 1025, device="cuda")
    with pytest.raises(RuntimeError, match="UNSUPPORTED_SHAPE"):
        moe.router_loss(wide, ids[:1], workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
