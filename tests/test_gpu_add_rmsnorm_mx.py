"""Residual addition + RMSNorm + MXFP8 and its backward pass against the formulas in 64 bits.

Bounds.  h is one FP32 addition rounded to BF16: bit-exact.  r: the sum of squares is a chain of
at most 32 fused additions per thread, then two 5-step trees (42 * 2^-24 relative, every term
non-negative), halved by the square root, plus four roundings: < 2^-19.  y: r, two products
(< 2^-18), then half a BF16 step (2^-8 relative).  Codes: the quotient y / 2^s is exact, so a code
is off by half an E4M3 step of the quotient (2^-4 relative, 2^-10 below 2^-6) plus y's own 2^-18;
the scale byte can differ only where max|y| lies within 2^-18 of a power of two.
Backward: dx is a sum of three FP32 terms whose own errors stay below 2^-18 of their magnitudes
(the row mean: a chain of 32 + trees of Cauchy-bounded terms), rounded to BF16 (2^-8); dgamma is a
sum of `rows` products in some fixed order: (rows + 8) * 2^-24 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

R_REL, Y_REL = 2.0 ** -19, 2.0 ** -18
BF16_HALF, E4M3_HALF = 2.0 ** -8, 2.0 ** -4


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


def make(rows, cols, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return ((n(rows, cols) * scale).bfloat16(), (n(rows, cols) * 2 * scale).bfloat16(),
            (1 + 0.1 * n(cols)).bfloat16())


def decode_scale(sf):
    return torch.exp2(sf.double() - 127)


def check_codes(codes, sf, y):
    """codes / sf against the exact y (64 bits)."""
    b = y.reshape(y.shape[0], -1, 32)
    top = b.abs().amax(-1)
    want = torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=1e-300))) - 8 + 127, 0.0)
    want = want.clamp(0, 254)
    near = (torch.log2(top.clamp(min=1e-300)) - torch.round(torch.log2(top.clamp(min=1e-300)))).abs() < 2.0 ** -17
    same = sf.double() == want
    assert bool((same | near).all())
    s = decode_scale(sf)[..., None]
    q = codes.view(torch.float8_e4m3fn).double().reshape(b.shape)
    target = (b / s).clamp(-448, 448)
    err = (q - target).abs()
    bound = (E4M3_HALF * target.abs()).clamp(min=2.0 ** -10) * (1 + 2.0 ** -10) + Y_REL * target.abs() + 1e-300
    assert bool((err <= bound).all()), float((err - bound).max())


def reference(x, res, gamma, eps):
    h = (x.float() + res.float()).bfloat16() if res is not None else x
    hd = h.double()
    r = 1 / torch.sqrt((hd * hd).mean(-1) + eps)
    return h, r, hd * r[:, None] * gamma.double()


@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 2048), (3, 96), (7, 4064), (64, 7168), (5, 16384),
                                       (300, 1024), (2, 4096), (2, 4128), (2, 8192), (2, 8224)])
@pytest.mark.parametrize("residual", [True, False])
def test_forward(moe, rows, cols, residual):
    x, res, gamma = make(rows, cols, rows + cols)
    if not residual:
        res = None
    o = moe.add_rmsnorm_quantize_mx(x, res, gamma, 1e-5, want_y=True, want_rrms=True)
    h, r, y = reference(x, res, gamma, 1e-5)
    if residual:
        assert torch.equal(o["h"], h)
    else:
        assert "h" not in o
    assert float(((o["rrms"].double() - r).abs() / r).max()) <= R_REL
    err = (o["y"].double() - y).abs()
    assert bool((err <= (BF16_HALF + Y_REL) * y.abs() + 1e-40).all())
    check_codes(o["codes"], o["sf"], y)
    # without y, and y alone, give the same bits
    only = moe.add_rmsnorm_quantize_mx(x, res, gamma, 1e-5)
    assert torch.equal(only["codes"], o["codes"]) and torch.equal(only["sf"], o["sf"])
    alone = moe.add_rmsnorm_quantize_mx(x, res, gamma, 1e-5, want_y=True, quantize=False)
    assert torch.equal(alone["y"], o["y"]) and "codes" not in alone


def test_wide_range_and_zero_rows(moe):
    x, res, gamma = make(64, 512, 3)
    x *= torch.exp2(torch.randint(-60, 20, (64, 1), device="cuda").float()).bfloat16()
    res *= 0
    x[5], x[9, 32:64] = 0, 0
    gamma[64:96] = 0
    o = moe.add_rmsnorm_quantize_mx(x, res, gamma, 1e-30, want_y=True)
    _, _, y = reference(x, res, gamma, 1e-30)
    check_codes(o["codes"], o["sf"], y)
    assert not o["codes"][5].any() and not o["sf"][5].any()
    assert not o["sf"][9, 1].any() and not o["sf"][:, 2].any()


def test_nonfinite_blocks(moe):
    x, res, gamma = make(6, 256, 4)
    x[1, 40] = float("nan")
    x[3, 7] = float("inf")
    res[4, 9] = -3e38
    x[4, 9] = -3e38          # the sum overflows to -infinity
    gamma2 = gamma.clone()
    gamma2[200] = float("inf")
    o = moe.add_rmsnorm_quantize_mx(x, res, gamma, 1e-5, want_y=True)
    clean = moe.add_rmsnorm_quantize_mx(x[[0, 2, 5]], res[[0, 2, 5]], gamma, 1e-5)
    assert torch.equal(o["codes"][[0, 2, 5]], clean["codes"])     # other rows are untouched
    assert bool((o["sf"][1] == 255).all()) and bool(((o["codes"][1] & 0x7F) == 0x7F).all())
    assert bool(o["y"][1].isnan().all())
    for row, blk in ((3, 0), (4, 0)):   # r = 0: the infinite element is NaN, the others are zero
        assert int(o["sf"][row, blk]) == 255 and bool((o["codes"][row, :32] == 0x7F).all())
        assert not o["codes"][row, 32:].bitwise_and(0x7F).any() and not o["sf"][row, 1:].any()
    g = moe.add_rmsnorm_quantize_mx(x[:1], res[:1], gamma2, 1e-5)
    assert int(g["sf"][0, 6]) == 255 and int(g["sf"][0, 5]) != 255


def test_in_place_and_out(moe):
    x, res, gamma = make(33, 2080, 5)
    want = moe.add_rmsnorm_quantize_mx(x, res, gamma, want_y=True, want_rrms=True)
    for inplace in ("residual", "x"):
        x2, r2 = x.clone(), res.clone()
        out = {k: torch.full_like(v, 7) for k, v in want.items()}
        out["h"] = r2 if inplace == "residual" else x2
        got = moe.add_rmsnorm_quantize_mx(x2, r2, gamma, out=out)
        assert got is out and all(torch.equal(got[k], want[k]) for k in want)


def test_zero_rows_on_a_side_stream_and_in_a_graph(moe):
    e = moe.add_rmsnorm_quantize_mx(*make(0, 64)[:2], make(1, 64)[2])
    assert e["h"].shape == (0, 64) and e["sf"].shape == (0, 2)
    x, res, gamma = make(17, 320, 6)
    want = moe.add_rmsnorm_quantize_mx(x, res, gamma)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = moe.add_rmsnorm_quantize_mx(x, res, gamma, stream=s)
    s.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    out = {k: torch.empty_like(v) for k, v in want.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.add_rmsnorm_quantize_mx(x, res, gamma, out=out)
    x.copy_(make(17, 320, 7)[0])
    graph.replay()
    want = moe.add_rmsnorm_quantize_mx(x, res, gamma)
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], want[k]) for k in want)


def backward_reference(dy, h, r, gamma, dh):
    dy, h, r, gamma = dy.double(), h.double(), r.double()[:, None], gamma.double()
    a = gamma * dy
    m = (a * h).mean(-1, keepdim=True)
    dx = r * a - h * r ** 3 * m
    size = (r * a).abs() + h.abs() * r ** 3 * (a * h).abs().mean(-1, keepdim=True)
    if dh is not None:
        dx, size = dx + dh.double(), size + dh.double().abs()
    t = dy * h * r
    return dx, size, t.sum(0), t.abs().sum(0)


@pytest.mark.parametrize("rows,cols,with_dh", [(1, 32, True), (1, 2048, False), (5, 96, True), (611, 1024, True),
                                               (1999, 352, False), (3, 16384, True), (40, 7168, False),
                                               (700, 4128, True)])
def test_backward(moe, rows, cols, with_dh):
    h, dy, gamma = make(rows, cols, rows * 3 + cols)
    dh = make(rows, cols, 9)[0] if with_dh else None
    r = moe.add_rmsnorm_quantize_mx(h, None, gamma, want_rrms=True)["rrms"]
    o = moe.add_rmsnorm_backward(dy, h, r, gamma, dh=dh)
    dx, size, dg, dgsize = backward_reference(dy, h, r, gamma, dh)
    assert bool(((o["dx"].double() - dx).abs() <= BF16_HALF * dx.abs() + Y_REL * size).all())
    assert bool(((o["dgamma"].double() - dg).abs() <= (rows + 8) * 2.0 ** -24 * dgsize).all())
    # again, the same bits; in place over dy and over dh
    again = moe.add_rmsnorm_backward(dy, h, r, gamma, dh=dh)
    assert torch.equal(again["dx"], o["dx"]) and torch.equal(again["dgamma"], o["dgamma"])
    for buf in ("dy", "dh") if with_dh else ("dy",):
        dy2, dh2 = dy.clone(), None if dh is None else dh.clone()
        got = moe.add_rmsnorm_backward(dy2, h, r, gamma, dh=dh2,
                                       out={"dx": dy2 if buf == "dy" else dh2, "dgamma": torch.empty_like(o["dgamma"])})
        assert torch.equal(got["dx"], o["dx"]) and torch.equal(got["dgamma"], o["dgamma"])


def test_backward_against_differences(moe):
    """The kernel's gradients along random directions against central differences of the forward
    formula in 64 bits (their own error is of the order step^2, 1e-8)."""
    rows, cols, eps = 6, 160, 1e-5
    h, dy, gamma = make(rows, cols, 21)
    r = moe.add_rmsnorm_quantize_mx(h, None, gamma, eps, want_rrms=True)["rrms"]
    o = moe.add_rmsnorm_backward(dy, h, r, gamma)

    def goal(hd, gd):
        return float((dy.double() * hd / torch.sqrt((hd * hd).mean(-1, keepdim=True) + eps) * gd).sum())

    rng = torch.Generator(device="cuda").manual_seed(3)
    step = 1e-4
    for _ in range(4):
        v = torch.randn(rows, cols, device="cuda", generator=rng, dtype=torch.float64)
        u = torch.randn(cols, device="cuda", generator=rng, dtype=torch.float64)
        hd, gd = h.double(), gamma.double()
        num = (goal(hd + step * v, gd) - goal(hd - step * v, gd)) / (2 * step)
        assert abs(num - float((o["dx"].double() * v).sum())) <= BF16_HALF * float((o["dx"].double() * v).abs().sum()) + 1e-5
        num = (goal(hd, gd + step * u) - goal(hd, gd - step * u)) / (2 * step)
        assert abs(num - float((o["dgamma"].double() * u).sum())) <= 1e-5 * float((o["dgamma"].double() * u).abs().sum()) + 1e-5


def test_backward_no_rows_and_graph(moe):
    z = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    o = moe.add_rmsnorm_backward(z, z, torch.zeros(0, device="cuda"), g,
                                 out={"dx": z.clone(), "dgamma": torch.full((64,), 5.0, device="cuda")})
    assert not o["dgamma"].any()
    h, dy, gamma = make(700, 256, 31)
    r = moe.add_rmsnorm_quantize_mx(h, None, gamma, want_rrms=True)["rrms"]
    out = {"dx": torch.empty_like(h), "dgamma": torch.empty(256, device="cuda")}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.add_rmsnorm_backward(dy, h, r, gamma, out=out)
    dy.copy_(make(700, 256, 32)[1])
    graph.replay()
    want = moe.add_rmsnorm_backward(dy, h, r, gamma)
    torch.cuda.synchronize()
    assert torch.equal(out["dx"], want["dx"]) and torch.equal(out["dgamma"], want["dgamma"])


def test_refusals(moe):
    x, res, gamma = make(4, 64)
    with pytest.raises(ValueError, match="contiguous"):
        moe.add_rmsnorm_quantize_mx(x.t().contiguous().t(), res, gamma)
    with pytest.raises(ValueError, match="residual"):
        moe.add_rmsnorm_quantize_mx(x, res.float(), gamma)
    with pytest.raises(ValueError, match="gamma"):
        moe.add_rmsnorm_quantize_mx(x, res, gamma[:32])
    with pytest.raises(ValueError, match="CUDA"):
        moe.add_rmsnorm_quantize_mx(x.cpu(), res, gamma)
    with pytest.raises(ValueError, match="multiple of 32"):
        moe.add_rmsnorm_quantize_mx(x[:, :40].contiguous(), None, gamma[:40])
    with pytest.raises(RuntimeError, match="INVALID_ARG"):      # nothing to write
        moe.add_rmsnorm_quantize_mx(x, None, gamma, quantize=False)
    with pytest.raises(RuntimeError, match="INVALID_ARG"):      # a residual without h
        moe.add_rmsnorm_quantize_mx(x, res, gamma, out={"y": torch.empty_like(x)})
    flat = torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(RuntimeError, match="INVALID_ARG"):      # not on a 16-byte boundary
        moe.add_rmsnorm_quantize_mx(flat[1:].reshape(4, 64), None, gamma)
    wide = torch.zeros(1, 16416, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(RuntimeError, match="UNSUPPORTED_SHAPE"):
        moe.add_rmsnorm_quantize_mx(wide, None, wide[0])
    with pytest.raises(RuntimeError, match="WORKSPACE_TOO_SMALL"):
        moe.add_rmsnorm_backward(x, x, torch.ones(4, device="cuda"), gamma,
                                 workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
