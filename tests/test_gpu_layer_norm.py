"""Residual addition + layer norm and its backward pass against the formulas in 64 bits.

Bounds, u = 2^-24.  h: one FP32 addition rounded to its type, bit-exact.  The mean is a chain of at most 32
additions a thread and two 5-step trees (44 u of the row's largest |h| with its scaling); h - m and the products
with 1/sigma, gamma and the addition of beta round once each; the variance is a sum of non-negative terms (45 u
relative, plus the square of the mean's error, 2^-37 of h^2), halved by the root: 2^-18 relative in all.  The output's
rounding: half a step, 2^-8 relative in BF16, u in FP32.
Backward: n = (h - m) r with given m and r has two roundings; the row means 46 u of their terms' magnitudes;
the sums over rows (rows + 8) u of theirs."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
SIZES = [(1, 8), (1, 2048), (3, 72), (7, 4064), (64, 7168), (5, 16384), (300, 1024), (2, 4104), (2, 8200), (700, 256), (1000, 8200)]


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


def normal(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, device="cuda", generator=g)


def check_forward(o, x, res, gamma, beta, eps):
    h = (x.float() + res.float()).to(x.dtype) if res is not None else x
    if res is not None:
        assert torch.equal(o["h"], h)
    else:
        assert "h" not in o
    d = h.double()
    m = d.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((d - m).square().mean(-1, keepdim=True) + eps)
    n = (d - m) * r
    b = beta.double() if beta is not None else torch.zeros_like(gamma).double()
    y = n * gamma.double() + b
    top = d.abs().amax(-1, keepdim=True)
    off = 46 * U * top                                              # of the mean
    rel = 2.0 ** -18 + (off * r).square()
    assert bool(((o["mean"].double() - m.squeeze(-1)).abs() <= off.squeeze(-1)).all())
    assert bool(((o["rstd"].double() / r.squeeze(-1) - 1).abs() <= rel.squeeze(-1)).all())
    own = (off * r + rel * n.abs()) * gamma.double().abs() + 2 * U * (y.abs() + b.abs())
    assert bool(((o["y"].double() - y).abs() <= own + HALF[x.dtype] * (y.abs() + own) + 1e-45).all())


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual,bias", [(True, True), (False, False)])
def test_forward(moe, rows, cols, dtype, residual, bias):
    n = normal(rows + cols)
    x, gamma = n(rows, cols).to(dtype), (1 + 0.1 * n(cols)).to(dtype)
    res = (2 * n(rows, cols) + 0.5).to(dtype) if residual else None
    beta = n(cols).to(dtype) if bias else None
    o = moe.add_layernorm(x, res, gamma, beta, 1e-5, want_stats=True)
    check_forward(o, x, res, gamma, beta, 1e-5)
    only = moe.add_layernorm(x, res, gamma, beta, 1e-5)
    assert torch.equal(only["y"], o["y"]) and "mean" not in only


def test_mean_far_from_zero(moe):
    """Rows whose spread is a hundredth of their mean, constant rows and rows of tiny values."""
    n = normal(5)
    x = 100 + n(40, 1000)
    x[3], x[4], x[5] = 7.5, 0.0, n(1000) * 1e-18
    gamma, beta = 1 + 0.1 * n(1000), n(1000)
    o = moe.add_layernorm(x, None, gamma, beta, 1e-6, want_stats=True)
    keep = [i for i in range(40) if i != 3]
    check_forward({k: v[keep] for k, v in o.items()}, x[keep], None, gamma, beta, 1e-6)
    assert float((o["y"][3] - beta).abs().max()) <= 1000 * 46 * U * 7.5 * 2       # (h - m) / sqrt(eps)


def test_nonfinite_rows_stay_alone(moe):
    n = normal(6)
    x, gamma = n(6, 264).bfloat16(), (1 + 0.1 * n(264)).bfloat16()
    clean = moe.add_layernorm(x, None, gamma, want_stats=True)
    x[1, 40], x[3, 7], x[4, 0] = float("nan"), float("inf"), -float("inf")
    o = moe.add_layernorm(x, None, gamma, want_stats=True)
    for r in (1, 3, 4):
        assert bool(o["y"][r].isnan().all())
    assert torch.equal(o["y"][[0, 2, 5]], clean["y"][[0, 2, 5]])


def reference_backward(dy, h, mean, rstd, gamma, dh):
    d, r = dy.double(), rstd.double()[:, None]
    n = (h.double() - mean.double()[:, None]) * r
    a = d * gamma.double()
    ma, mn = a.mean(-1, keepdim=True), (a * n).mean(-1, keepdim=True)
    dx = r * (a - ma - n * mn)
    size = r * (8 * U * (a.abs() + ma.abs() + (n * mn).abs()) + 48 * U * (a.abs().mean(-1, keepdim=True) + n.abs() * (a * n).abs().mean(-1, keepdim=True)))
    if dh is not None:
        dx = dx + dh.double()
        size = size + 2 * U * dh.double().abs()
    return dx, size, (d * n).sum(0), (d * n).abs().sum(0), d.sum(0), d.abs().sum(0)


@pytest.mark.parametrize("rows,cols", SIZES + [(2500, 64), (700, 5120), (620, 16384)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("with_dh,bias", [(True, True), (False, False)])
def test_backward(moe, rows, cols, dtype, with_dh, bias):
    n = normal(rows * 3 + cols)
    h, dy, gamma = (2 * n(rows, cols) + 0.5).to(dtype), n(rows, cols).to(dtype), (1 + 0.1 * n(cols)).to(dtype)
    dh = n(rows, cols).to(dtype) if with_dh else None
    st = moe.add_layernorm(h, None, gamma, want_stats=True)
    out = None if bias else {"dx": torch.empty_like(dy), "dgamma": torch.empty(cols, device="cuda")}
    o = moe.add_layernorm_backward(dy, h, st["mean"], st["rstd"], gamma, dh=dh, out=out)
    dx, size, dg, dg_size, db, db_size = reference_backward(dy, h, st["mean"], st["rstd"], gamma, dh)
    err = (o["dx"].double() - dx).abs()
    assert bool((err <= size + HALF[dtype] * (dx.abs() + size) + 1e-45).all()), float((err - size).max())
    assert bool(((o["dgamma"].double() - dg).abs() <= (rows + 8) * U * dg_size).all())
    if bias:
        assert bool(((o["dbeta"].double() - db).abs() <= (rows + 8) * U * db_size).all())
    again = moe.add_layernorm_backward(dy, h, st["mean"], st["rstd"], gamma, dh=dh)
    assert torch.equal(again["dx"], o["dx"]) and torch.equal(again["dgamma"], o["dgamma"])


def test_gradient_against_differences(moe):
    """FP32: the directional derivative of sum(c * y) against a central difference of the operator itself.
    Step 1/64: third derivatives leave about 1e-4 of the sum's terms, the FP32 outputs 64 * 2^-23."""
    n = normal(8)
    x, gamma, beta, c, dirx, dirg = n(50, 200), 1 + 0.2 * n(200), n(200), n(50, 200), n(50, 200), n(200)
    st = moe.add_layernorm(x, None, gamma, beta, want_stats=True)
    b = moe.add_layernorm_backward(c, x, st["mean"], st["rstd"], gamma)
    f = lambda t: (moe.add_layernorm(x + t * dirx, None, gamma + t * dirg, beta + t)["y"].double() * c).sum()  # noqa: E731
    e = 1.0 / 64
    want = float((f(e) - f(-e)) / (2 * e))
    got = float((b["dx"].double() * dirx).sum() + (b["dgamma"].double() * dirg).sum() + b["dbeta"].double().sum())
    assert abs(got - want) <= 2e-3 * float(c.abs().sum() ** 0.5) * 14, (got, want)


def test_in_place(moe):
    n = normal(9)
    x, res, gamma, dy, dh = n(33, 2080).bfloat16(), n(33, 2080).bfloat16(), n(2080).bfloat16(), n(33, 2080).bfloat16(), n(33, 2080).bfloat16()
    want = moe.add_layernorm(x, res, gamma, want_stats=True)
    for place in (0, 1):
        a, b = x.clone(), res.clone()
        out = {"h": (a, b)[place], "y": torch.empty_like(x)}
        moe.add_layernorm(a, b, gamma, out=out)
        assert torch.equal(out["h"], want["h"]) and torch.equal(out["y"], want["y"])
    args = want["h"], want["mean"], want["rstd"], gamma
    back = moe.add_layernorm_backward(dy, *args, dh=dh)
    for place in (0, 1):
        a, b = dy.clone(), dh.clone()
        out = {"dx": (a, b)[place], "dgamma": torch.empty(2080, device="cuda"), "dbeta": torch.empty(2080, device="cuda")}
        moe.add_layernorm_backward(a, *args, dh=b, out=out)
        assert all(torch.equal(out[k], back[k]) for k in back)


def test_no_rows_and_refusals(moe):
    gamma = torch.ones(64, device="cuda").bfloat16()
    empty = torch.empty(0, 64, device="cuda").bfloat16()
    o = moe.add_layernorm(empty, empty, gamma, want_stats=True)
    assert o["y"].shape == (0, 64) and o["mean"].shape == (0,)
    b = moe.add_layernorm_backward(empty, empty, o["mean"], o["rstd"], gamma)
    assert not b["dgamma"].any() and not b["dbeta"].any()
    x = torch.zeros(4, 64, device="cuda").bfloat16()
    for bad in (dict(x=x[:, ::2]), dict(x=x.half()), dict(gamma=gamma.float()), dict(residual=x[:2]), dict(beta=gamma[:32]), dict(x=x[:, :60].contiguous())):
        with pytest.raises(ValueError):
            moe.add_layernorm(**{**dict(x=x, residual=None, gamma=gamma), **bad})


def test_graph_and_stream(moe):
    n = normal(10)
    x, res, gamma, dy = n(300, 1032).bfloat16(), n(300, 1032).bfloat16(), n(1032).bfloat16(), n(300, 1032).bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step(stream=None):
        o = moe.add_layernorm(x, res, gamma, want_stats=True, stream=stream)
        return o, moe.add_layernorm_backward(dy, o["h"], o["mean"], o["rstd"], gamma, stream=stream)

    o2, b2 = step(side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        og, bg = step()
    x.copy_(n(300, 1032))
    g.replay()
    o, b = step()
    torch.cuda.synchronize()
    assert torch.equal(og["y"], o["y"]) and all(torch.equal(bg[k], b[k]) for k in b)
    assert not torch.equal(o2["y"], o["y"])
