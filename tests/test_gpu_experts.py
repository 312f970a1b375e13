"""The experts' products and their gradients, each stage against 64 bits on the stage's own BF16 inputs.

Bounds.  A product of K terms is K / 16 + 4 additions in the tensor cores, which truncate: 2^-22 of the terms' magnitudes
each.  g, u, out, drows: then half a BF16 step (2^-8 relative).  h: the activation's slope by g is at most 1.1 (|u| + 1),
by u at most |g| + 2 |u| (of any of the four), and its own evaluation errs by 2^-18 of (|u| + 1) (|g| + 1).
dg, du: the products' errors times the derivatives, plus the derivatives' own 2^-18, then half a step.  The weights'
gradients: a chain of at most 64 such additions, then one FP32 addition (2^-24 of the sum's size) a chain."""
import pytest
import torch

pytestmark = pytest.mark.gpu

HALF, STEP, U = 2.0 ** -8, 2.0 ** -22, 2.0 ** -24
LIMIT, ALPHA = 1.5, 1.702
ACTS = {"swiglu": dict(), "clamp": dict(swiglu_limit=LIMIT), "relu2": dict(activation="relu2"),
        "oai": dict(activation="swiglu_oai", swiglu_limit=LIMIT, swiglu_alpha=ALPHA)}
# rows of each expert; tiles end and begin at 32, 64, 128 and 256 rows, chains at 1024
SEGMENTS = {"one": [1], "ends": [0, 1, 0], "ragged": [31, 32, 33, 63, 64, 65, 0, 127, 128, 129, 255, 256, 257, 1],
            "long": [1100, 0, 2049, 3], "many": [3, 0, 0, 5, 1, 0, 2] * 40}
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


def act64(g, u, name):
    if name == "relu2":
        return torch.relu(u) ** 2
    if name != "swiglu":
        g, u = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
    if name == "oai":
        return (u + 1) * g * torch.sigmoid(ALPHA * g)
    return g * torch.sigmoid(g) * u


class Case:
    def __init__(self, segs, H, I, act, extra=5, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed + H + I + len(segs))
        n = lambda *s, scale=1.0: (torch.randn(*s, device="cuda", generator=gen) * scale).to(BF16)  # noqa: E731
        self.act, self.kw, E = act, ACTS[act], len(segs)
        off = torch.tensor([0] + segs).cumsum(0)
        self.off, self.R = off.tolist(), int(off[-1]) + extra
        self.plan = {"offsets": off.to(torch.int32).cuda()}
        self.x, self.dout = n(self.R, H), n(self.R, H, scale=0.1)
        s = 1.5 / H ** 0.5
        self.wg = n(E, I, H, scale=s) if act != "relu2" else None
        self.wu, self.wd = n(E, I, H, scale=s), n(E, H, I, scale=1 / I ** 0.5)
        self.x[self.off[-1]:], self.dout[self.off[-1]:] = float("nan"), float("inf")     # not to be used
        self.H, self.I, self.E = H, I, E

    def out(self, *names):
        width = {"out": self.H, "drows": self.H}
        return {m: torch.full((self.R, width.get(m, self.I)), 7.0, device="cuda", dtype=BF16) for m in names if self.wg is not None or m not in ("g", "dg")}

    def forward(self, moe, **kw):
        return moe.experts_forward(self.x, self.plan, self.wg, self.wu, self.wd, **self.kw, **kw)

    def backward(self, moe, saved, **kw):
        return moe.experts_backward(self.dout, saved, self.plan, self.wg, self.wu, self.wd, **self.kw, **kw)

    def segments(self):
        return [(e, slice(a, b)) for e, (a, b) in enumerate(zip(self.off[:-1], self.off[1:])) if b > a]


def product(a, b):
    """a [r, K] @ b [K, n] in 64 bits, and the bound of its accumulation."""
    a, b = a.double(), b.double()
    return a @ b, (a.shape[1] / 16 + 4) * STEP * (a.abs() @ b.abs())


def close(got, want, err, what):
    bad = (got.double() - want).abs() - err - HALF * (want.abs() + err)
    assert bool((bad <= 1e-38).all()), (what, float(bad.max()))


@pytest.mark.parametrize("segs", SEGMENTS)
@pytest.mark.parametrize("H,I", [(32, 32), (96, 160), (288, 544), (1024, 256)])
@pytest.mark.parametrize("act", ACTS)
def test_stages(moe, segs, H, I, act):
    c = Case(SEGMENTS[segs], H, I, act)
    ws = moe.experts_workspace(c.R, I)
    o = c.forward(moe, out=c.out("out", "g", "u", "h"), workspace=ws)
    assert moe.last_device_status(ws) == 0
    b = c.backward(moe, o, out=c.out("drows", "dg", "du"), workspace=ws)
    w = moe.experts_weight_grad(c.x, c.dout, o, b, c.plan, workspace=ws)
    assert moe.last_device_status(ws) == 0 and set(w) == ({"w_up", "w_down"} if act == "relu2" else {"w_gate", "w_up", "w_down"})
    for t in (*o.values(), *b.values()):          # rows behind the last expert's: as they were
        assert bool((t[c.off[-1]:] == 7).all())
    for e, r in c.segments():
        u, eu = product(c.x[r], c.wu[e].t())
        close(o["u"][r], u, eu, "u")
        g, eg = (u * 0, eu * 0) if c.wg is None else product(c.x[r], c.wg[e].t())
        if c.wg is not None:
            close(o["g"][r], g, eg, "g")
        own = 2.0 ** -18 * (u.abs() + 1) * (g.abs() + 1)
        close(o["h"][r], act64(g, u, act), 1.1 * (u.abs() + 1) * eg + (g.abs() + 2 * u.abs() + eu) * eu + own, "h")
        close(o["out"][r], *product(o["h"][r], c.wd[e].t()), "out")
        # backward, from the stored g and u
        dh, edh = product(c.dout[r], c.wd[e])
        u = o["u"][r].double().requires_grad_()
        g = o["g"][r].double().requires_grad_() if c.wg is not None else torch.zeros_like(u).requires_grad_()
        fg, fu = torch.autograd.grad(act64(g, u, act).sum(), (g, u), allow_unused=True)
        own = 2.0 ** -18 * (u.abs() + 1) * (g.abs() + 1) * dh.abs()
        close(b["du"][r], dh * fu, edh * fu.abs() + own, "du")
        dx, edx = product(b["du"][r], c.wu[e])
        if c.wg is not None:
            close(b["dg"][r], dh * fg, edh * fg.abs() + own, "dg")
            more, emore = product(b["dg"][r], c.wg[e])
            dx, edx = dx + more, edx + emore + STEP * I / 16 * (b["dg"][r].double().abs() @ c.wg[e].double().abs())
        close(b["drows"][r], dx, 2 * edx, "drows")
    have = dict(c.segments())
    for name, left, right in (("w_gate", b.get("dg"), c.x), ("w_up", b["du"], c.x), ("w_down", c.dout, o["h"])):
        if name not in w:
            continue
        for e in range(c.E):
            if e not in have:
                assert not w[name][e].any()
                continue
            l, rt = left[have[e]].double(), right[have[e]].double()
            size, rows = l.abs().t() @ rt.abs(), l.shape[0]
            bound = ((min(rows, 1024) / 16 + 4) * STEP + (rows / 1024 + 1) * U) * size
            assert bool(((w[name][e].double() - l.t() @ rt).abs() <= bound + 1e-38).all()), (name, e)


@pytest.mark.parametrize("act", ["swiglu", "relu2"])
def test_without_keeping(moe, act):
    c = Case([40, 0, 300], 160, 96, act)
    want = c.forward(moe, keep=True)
    got = c.forward(moe)
    n = c.off[-1]
    assert set(got) == {"out"} and torch.equal(got["out"][:n], want["out"][:n])
    assert set(want) == ({"out", "u", "h"} if act == "relu2" else {"out", "g", "u", "h"})
    some = c.forward(moe, out=c.out("out", "h"))
    assert torch.equal(some["out"][:n], want["out"][:n]) and torch.equal(some["h"][:n], want["h"][:n])


@pytest.mark.parametrize("act", ["swiglu", "relu2"])
def test_accumulate(moe, act):
    c = Case([70, 0, 1500], 160, 288, act)
    o = c.forward(moe, keep=True)
    b = c.backward(moe, o)
    once = moe.experts_weight_grad(c.x, c.dout, o, b, c.plan)
    before = {k: torch.randn(v.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) for k, v in once.items()}
    out = {k: v.clone() for k, v in before.items()}
    got = moe.experts_weight_grad(c.x, c.dout, o, b, c.plan, accumulate=True, out=out)
    for k in once:
        assert got[k] is out[k] and torch.equal(got[k][1], before[k][1])             # the expert without rows
        size = once[k].double().abs() + before[k].double().abs()
        # three additions here against two there, of partial sums that may be a few times the result
        left, right = {"w_up": (b["du"], c.x), "w_gate": (b.get("dg"), c.x), "w_down": (c.dout, o["h"])}[k]
        for e, r in c.segments():
            terms = left[r].double().abs().t() @ right[r].double().abs()
            assert bool(((got[k][e].double() - once[k][e].double() - before[k][e].double()).abs() <= 4 * U * (size[e] + terms)).all())


def test_no_rows(moe):
    c = Case([0, 0], 64, 96, "swiglu", extra=0)
    for R in (0, 3):                                     # no rows at all, or none that an expert owns
        c.R, c.x, c.dout = R, torch.full((R, 64), float("nan"), device="cuda", dtype=BF16), torch.ones(R, 64, device="cuda", dtype=BF16)
        o = c.forward(moe, out=c.out("out", "g", "u", "h"))
        b = c.backward(moe, o, out=c.out("drows", "dg", "du"))
        assert all(bool((t == 7).all()) for t in (*o.values(), *b.values()))
        keep = {n: torch.full((2, *s), 3.0, device="cuda") for n, s in (("w_gate", (96, 64)), ("w_up", (96, 64)), ("w_down", (64, 96)))}
        w = moe.experts_weight_grad(c.x, c.dout, o, b, c.plan, accumulate=True, out=keep)
        assert all(bool((t == 3).all()) for t in w.values())
        w = moe.experts_weight_grad(c.x, c.dout, o, b, c.plan, out=keep)
        assert all(bool((t == 0).all()) for t in w.values())


def test_nonfinite_rows_stay_alone(moe):
    c = Case([100, 37, 200], 96, 160, "swiglu")
    o, n = c.forward(moe, keep=True), c.off[-1]
    b = c.backward(moe, o)
    w = moe.experts_weight_grad(c.x, c.dout, o, b, c.plan)
    c.x[120, 5], c.dout[121, 7] = float("nan"), float("inf")
    o2 = c.forward(moe, keep=True)
    b2 = c.backward(moe, o2)
    w2 = moe.experts_weight_grad(c.x, c.dout, o2, b2, c.plan)
    good = [r for r in range(n) if r not in (120, 121)]
    assert all(torch.equal(o2[k][good], o[k][good]) for k in o) and bool(o2["out"][120].isnan().all())
    assert all(torch.equal(b2[k][good], b[k][good]) for k in b) and not bool(b2["drows"][121].isfinite().any())
    for k in w:      # row 120 and 121 belong to expert 1
        assert torch.equal(w2[k][[0, 2]], w[k][[0, 2]]) and not bool(w2[k][1].isfinite().all())


@pytest.mark.parametrize("bad", [[0, 10, 5, 20], [0, 10, 20, 400], [-1, 5, 6, 7], [0, 2 ** 31 - 1, 3, 4], [30, 20, 10, 0]])
def test_bad_offsets(moe, bad):
    """Offsets that do not ascend within the rows: reported, nothing computed."""
    c = Case([10, 10, 10], 64, 64, "swiglu")
    c.plan = {"offsets": torch.tensor(bad, dtype=torch.int32, device="cuda")}
    ws = moe.experts_workspace(c.R, 64)
    o = c.forward(moe, out=c.out("out", "g", "u", "h"), workspace=ws)
    assert moe.last_device_status(ws) == -1 and all(bool((t == 7).all()) for t in o.values())
    b = c.backward(moe, o, out=c.out("drows", "dg", "du"), workspace=ws)
    assert moe.last_device_status(ws) == -1 and all(bool((t == 7).all()) for t in b.values())
    keep = {n: torch.full((3, 64, 64), 3.0, device="cuda") for n in ("w_gate", "w_up", "w_down")}
    moe.experts_weight_grad(c.x, c.dout, o, b, c.plan, out=keep, workspace=ws)
    assert moe.last_device_status(ws) == -1 and all(bool((t == 3).all()) for t in keep.values())
    c.plan = {"offsets": torch.tensor([0, 10, 20, 30], dtype=torch.int32, device="cuda")}
    c.forward(moe, out=c.out("out", "g", "u", "h"), workspace=ws)
    assert moe.last_device_status(ws) == 0


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(moe, act):
    """Central differences of the 64-bit formula (h unrounded) along random directions.  The kernels' gradients carry the
    BF16 roundings of g, u, h, dg, du and drows: each moves a term of the sums by half a step, independently, so that a
    sum of n terms of size s is off by about sqrt(n) s 2^-9; bound: 8 such deviations.  The clamped activations have kinks,
    which a difference of step 1e-6 almost never crosses; but the backward pass clamps the stored g and u, and those that
    round across the limit (2^-8 of the density at each limit: about 30 of 15744 here, 4% of the root of the sum of squares,
    above the 3% of the bound) have the derivative of the other side: such an element (r, i) changes the sum by its whole
    dh act' times the direction's part in g or u, which is added to the bound for the elements counted."""
    c = Case([90, 33], 96, 128, act, extra=0, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen, dtype=torch.float64)  # noqa: E731
    o = c.forward(moe, keep=True)
    b = c.backward(moe, o)
    w = moe.experts_weight_grad(c.x, c.dout, o, b, c.plan)

    def loss(x, wg, wu, wd):
        t = 0.0
        for e, r in c.segments():
            g = x[r] @ wg[e].t() if wg is not None else None
            t = t + (act64(g, x[r] @ wu[e].t(), act) @ wd[e].t() * c.dout[r].double()).sum()
        return t

    base = [t.double() if t is not None else None for t in (c.x, c.wg, c.wu, c.wd)]
    for i, grad in enumerate((b["drows"], w.get("w_gate"), w["w_up"], w["w_down"])):
        if grad is None:
            continue
        d, h = n(*grad.shape), 1e-6
        lo, hi = list(base), list(base)
        lo[i], hi[i] = base[i] - h * d, base[i] + h * d
        want = float((loss(*hi) - loss(*lo)) / (2 * h))
        terms, crossed = grad.double() * d, 0.0
        for e, r in c.segments() if c.act in ("clamp", "oai") else []:
            x, dh = base[0][r], (c.dout[r].double() @ base[3][e]).abs()
            for j, name in ((1, "g"), (2, "u")):
                part = d[r] @ base[j][e].t() if i == 0 else x @ d[e].t() if i == j else None
                if part is None:
                    continue
                at, stored = x @ base[j][e].t(), o[name][r].double()
                over = (lambda t: t > LIMIT) if name == "g" else (lambda t: t.abs() > LIMIT)
                slope = 1.1 * (LIMIT + 1) if name == "g" else o["g"][r].double().abs()
                crossed += float((dh * slope * part.abs())[over(at) != over(stored)].sum())
        assert abs(float(terms.sum()) - want) <= 8 * 2.0 ** -8 * float(terms.square().sum().sqrt()) + crossed + 1e-6, (act, i)


def test_same_bits_graph_and_streams(moe):
    c = Case([300, 20, 0, 700], 256, 160, "swiglu")
    side = torch.cuda.Stream()

    def step(stream=None):
        o = c.forward(moe, keep=True, stream=stream)
        b = c.backward(moe, o, stream=stream)
        return o, b, moe.experts_weight_grad(c.x, c.dout, o, b, c.plan, stream=stream)

    n = c.off[-1]
    same = lambda p, q: all(torch.equal(p[i][k][:n], q[i][k][:n]) for i in range(2) for k in p[i]) and all(torch.equal(p[2][k], q[2][k]) for k in p[2])  # noqa: E731
    first = step()
    side.wait_stream(torch.cuda.current_stream())
    assert same(first, step())
    on_side = step(side)
    here = step()
    torch.cuda.synchronize()
    assert same(first, on_side) and same(first, here)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rec = step()
    c.x[:n] = torch.randn(n, 256, device="cuda").to(BF16)
    c.plan["offsets"].copy_(torch.tensor([0, 1, 600, 601, n], dtype=torch.int32))      # other segments in the replay
    g.replay()
    torch.cuda.synchronize()
    assert same(rec, step()) and not same(rec, first)


def test_refusals(moe):
    c = Case([10, 10], 64, 96, "swiglu")
    ok = dict(rows=c.x, plan=c.plan, w_gate=c.wg, w_up=c.wu, w_down=c.wd)
    for bad in (dict(rows=c.x.float()), dict(rows=c.x[:, :48].contiguous()), dict(w_gate=None), dict(w_down=c.wu), dict(w_up=c.wu[0]),
                dict(plan={"offsets": c.plan["offsets"][:2]}), dict(plan={}), dict(activation="gelu"), dict(activation="swiglu_oai"),
                dict(rows=c.x[:, ::2])):
        with pytest.raises(ValueError):
            moe.experts_forward(**{**ok, **bad})
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        moe.experts_forward(**ok, workspace=moe.experts_workspace(0, 96))
    with pytest.raises(RuntimeError, match="INVALID_ARG"):       # a limit below zero
        moe.experts_forward(**ok, swiglu_limit=-1.0)
    o = moe.experts_forward(**ok, keep=True)
    b = moe.experts_backward(c.dout, o, c.plan, c.wg, c.wu, c.wd)
    with pytest.raises(ValueError, match="accumulate"):
        moe.experts_weight_grad(c.x, c.dout, o, b, c.plan, accumulate=True)
    with pytest.raises(ValueError):
        moe.experts_weight_grad(c.x, c.dout[:4], o, b, c.plan)
