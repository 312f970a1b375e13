"""The training pass's operators beyond 2^32 elements of a tensor, and at their widest: offsets past 32 bits, the last rows
compared.  Bounds as in the operators' own tests (2^-8: half a BF16 step)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, HALF, STEP, U = torch.bfloat16, 2.0 ** -8, 2.0 ** -22, 2.0 ** -24


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 120 * 2 ** 30:
        pytest.skip("needs 120 GB of device memory")
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def test_layer_norm(moe):
    rows, cols = 300_000, 16384                     # 4.9e9 elements
    x = torch.empty(rows, cols, dtype=BF16, device="cuda")
    for i in range(0, rows, 10_000):
        x[i:i + 10_000] = torch.randn(10_000, cols, device="cuda").to(BF16)
    gamma, beta = torch.randn(cols, device="cuda").to(BF16), torch.randn(cols, device="cuda").to(BF16)
    o = moe.add_layernorm(x, None, gamma, beta, want_stats=True)
    for r in (0, rows // 2, rows - 1):
        d = x[r].double()
        n = (d - d.mean()) / torch.sqrt(d.var(unbiased=False) + 1e-5)
        y = n * gamma.double() + beta.double()
        assert bool(((o["y"][r].double() - y).abs() <= HALF * y.abs() + 2.0 ** -17 * ((n * gamma.double()).abs() + beta.double().abs() + 1)).all())
    b = moe.add_layernorm_backward(o["y"], x, o["mean"], o["rstd"], gamma, out={"dx": o["y"], "dgamma": torch.empty(cols, device="cuda")})
    assert bool(b["dx"][-3:].isfinite().all()) and bool(b["dx"][-1].any()) and bool(b["dgamma"].isfinite().all())


def test_tokens(moe):
    T, k, cols = 75_000, 8, 8192                    # rows: 4.9e9 elements
    ids = torch.randint(0, 32, (T, k), device="cuda", dtype=torch.int32)
    plan = moe.sort_tokens(ids, 32)
    x = torch.randn(T, cols, device="cuda").to(BF16)
    rows = moe.permute_tokens(x, plan)
    src = plan["perm_src"].long()
    for p in (0, T * k // 2, T * k - 1):
        assert torch.equal(rows[p], x[src[p]])
    w = torch.rand(T, k, device="cuda")
    y = moe.combine_tokens(rows, plan, w)
    want = x.double() * w.double().sum(1, keepdim=True)
    assert bool(((y.double() - want).abs() <= (HALF + 16 * U) * want.abs() * 1.01).all())
    b = moe.combine_tokens_backward(x, rows, plan, w, out={"drows": rows, "dtopk_w": torch.empty_like(w)})
    p = T * k - 1
    a = int((plan["inv"] == p).nonzero())
    assert torch.equal(b["drows"][p], (x[a // k].float() * w.reshape(-1)[a]).to(BF16))
    sq = x.double().square().sum(1, keepdim=True)
    assert bool(((b["dtopk_w"].double() - sq).abs() <= 300 * U * sq).all())


def test_experts_rows(moe):
    R, H, I, E = 600_000, 8192, 32, 2               # rows and out: 4.9e9 elements
    x = torch.randn(R, H, device="cuda", dtype=BF16)
    wg, wu, wd = (torch.randn(E, I, H, device="cuda", dtype=BF16) * 0.02 for _ in range(3))
    wd = wd.transpose(1, 2).contiguous()
    plan = {"offsets": torch.tensor([0, 299_999, R], dtype=torch.int32, device="cuda")}
    o = moe.experts_forward(x, plan, wg, wu, wd, keep=True)
    b = moe.experts_backward(x, o, plan, wg, wu, wd)
    w = moe.experts_weight_grad(x, x, o, b, plan)
    for e, r in ((0, 0), (0, 299_998), (1, 299_999), (1, R - 1)):
        d = x[r].double()
        g, u = wg[e].double() @ d, wu[e].double() @ d
        assert bool(((o["g"][r].double() - g).abs() <= HALF * g.abs() + 520 * STEP * (wg[e].double().abs() @ d.abs())).all())
        h = o["h"][r].double()
        assert bool(((h - torch.nn.functional.silu(g) * u).abs() <= 2.0 ** -7 * (g.abs() + 1) * (u.abs() + 1)).all())
        out = wd[e].double() @ h
        assert bool(((o["out"][r].double() - out).abs() <= HALF * out.abs() + 8 * STEP * (wd[e].double().abs() @ h.abs()) + 1e-30).all())
        dx = b["dg"][r].double() @ wg[e].double() + b["du"][r].double() @ wu[e].double()
        size = b["dg"][r].double().abs() @ wg[e].double().abs() + b["du"][r].double().abs() @ wu[e].double().abs()
        assert bool(((b["drows"][r].double() - dx).abs() <= HALF * dx.abs() + 16 * STEP * size + 1e-30).all())
    want, size = torch.zeros(I, H, dtype=torch.float64, device="cuda"), torch.zeros(I, H, dtype=torch.float64, device="cuda")
    for i in range(299_999, R, 20_000):
        s = slice(i, min(i + 20_000, R))
        want += b["du"][s].double().t() @ x[s].double()
        size += b["du"][s].double().abs().t() @ x[s].double().abs()
    assert bool(((w["w_up"][1].double() - want).abs() <= (36 * STEP + (300_001 / 512 + 1) * U) * size).all())


def test_experts_weights(moe):
    E, H, I = 1024, 2080, 2080                      # a gradient of 4.4e9 elements; the last expert has the rows
    R = 70
    x, h, d, du = (torch.randn(R, 2080, device="cuda", dtype=BF16) for _ in range(4))
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = R
    w = moe.experts_weight_grad(x, d, {"h": h}, {"du": du}, {"offsets": off})
    for name, l, r in (("w_up", du, x), ("w_down", d, h)):
        want, size = l.double().t() @ r.double(), l.double().abs().t() @ r.double().abs()
        assert bool(((w[name][E - 1].double() - want).abs() <= 10 * STEP * size).all())
        assert not w[name][E - 2].any() and not w[name][0].any()


@pytest.mark.parametrize("H,I", [(65536, 32), (32, 65536), (16384, 96)])
def test_experts_widest(moe, H, I):
    x, wg, wu = (torch.randn(*s, device="cuda", dtype=BF16) * 0.05 for s in ((3, H), (2, I, H), (2, I, H)))
    wd = torch.randn(2, H, I, device="cuda", dtype=BF16) * 0.05
    plan = {"offsets": torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")}
    o = moe.experts_forward(x, plan, wg, wu, wd, keep=True)
    b = moe.experts_backward(x, o, plan, wg, wu, wd)
    w = moe.experts_weight_grad(x, x, o, b, plan)
    for e, s in ((0, slice(0, 1)), (1, slice(1, 3))):
        h = o["h"][s].double()
        out, size = h @ wd[e].double().t(), h.abs() @ wd[e].double().abs().t()
        assert bool(((o["out"][s].double() - out).abs() <= HALF * out.abs() + (I / 16 + 8) * STEP * size + 1e-30).all())
        u, size = x[s].double() @ wu[e].double().t(), x[s].double().abs() @ wu[e].double().abs().t()
        assert bool(((o["u"][s].double() - u).abs() <= HALF * u.abs() + (H / 16 + 8) * STEP * size).all())
        dx = b["dg"][s].double() @ wg[e].double() + b["du"][s].double() @ wu[e].double()
        size = b["dg"][s].double().abs() @ wg[e].double().abs() + b["du"][s].double().abs() @ wu[e].double().abs()
        assert bool(((b["drows"][s].double() - dx).abs() <= HALF * dx.abs() + (I / 8 + 16) * STEP * size + 1e-30).all())
        want = b["dg"][s].double().t() @ x[s].double()
        assert bool(((w["w_gate"][e].double() - want).abs() <= 8 * STEP * (b["dg"][s].double().abs().t() @ x[s].double().abs())).all())
