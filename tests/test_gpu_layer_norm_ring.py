"""Layer norm at sizes whose rows come through the ring in shared memory (more rows than are on the SMs at once), one size for
each layout: vectors a lane, warps a row, rows a block, slots; and both forward kernels in place."""
import pytest
import torch

from test_gpu_layer_norm import HALF, U, check_forward, normal, reference_backward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("rows,cols", [(5, 1032), (64, 8200), (7, 16384),                                        # a row a block
                                       (20011, 256), (9001, 1024), (3001, 4096), (2003, 5120), (2003, 8192), (1300, 16384)])   # the ring
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place(moe, rows, cols, dtype):
    """h in the buffer of x or of the residual, of which later rows are read ahead: the bits of a call with a buffer of its own."""
    n = normal(rows + 2 * cols)
    x, res, gamma = n(rows, cols).to(dtype), n(rows, cols).to(dtype), n(cols).to(dtype)
    want = moe.add_layernorm(x, res, gamma, want_stats=True)
    check_forward(want, x, res, gamma, None, 1e-5)
    for place in (0, 1):
        a, b = x.clone(), res.clone()
        out = {"h": (a, b)[place], "y": torch.full_like(x, float("nan"))}
        moe.add_layernorm(a, b, gamma, out=out)
        assert torch.equal(out["h"], want["h"]) and torch.equal(out["y"], want["y"])


@pytest.mark.parametrize("rows,cols", [(40, 24), (300, 1000), (300, 7168), (40, 12296), (20000, 264), (9000, 1000), (2003, 5120), (1300, 12296)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_constant_rows(moe, rows, cols, dtype):
    """Rows of one value of 8 significant bits: at most 16384 of them add up within FP32's 24 bits, in any order, so their mean is
    the value itself and y is beta, however large the value is against eps."""
    beta = normal(cols)(cols).to(dtype)
    c = (torch.randint(129, 256, (rows, 1), device="cuda", generator=torch.Generator(device="cuda").manual_seed(cols)).float()
         * torch.tensor([1.0, -0.25, 512.0], device="cuda").repeat(rows)[:rows, None])
    x = c.to(dtype).expand(rows, cols).contiguous()
    o = moe.add_layernorm(x, None, torch.ones(cols, device="cuda").to(dtype), beta, 1e-12, want_stats=True)
    assert torch.equal(o["mean"], c[:, 0])
    assert torch.equal(o["y"], beta.expand(rows, cols))


# vectors a lane, warps a row, rows a block: 1/1/16, 2/1/16, 2/2/8 (one lane in the last warp), 2/2/8, 2/3/5, 2/8/2, 3/7/2, 2/14/1,
# 2/16/1, 4/16/1 (FP32: one slot)
RING = [(20011, 256), (15000, 408), (12000, 520), (9001, 1024), (7000, 1288), (3001, 4096), (2003, 5120), (2003, 7168), (2003, 8192), (1300, 16384)]


@pytest.mark.parametrize("rows,cols", RING)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [True, False])
def test_forward(moe, rows, cols, dtype, residual):
    n = normal(rows + cols)
    x, gamma, beta = n(rows, cols).to(dtype), (1 + 0.1 * n(cols)).to(dtype), n(cols).to(dtype)
    res = (2 * n(rows, cols) + 0.5).to(dtype) if residual else None
    o = {"y": torch.full_like(x, float("nan")), "mean": torch.full((rows,), float("nan"), device="cuda"), "rstd": torch.full((rows,), float("nan"), device="cuda")}
    if residual:
        o["h"] = torch.full_like(x, float("nan"))
    check_forward(moe.add_layernorm(x, res, gamma, beta, 1e-5, out=o), x, res, gamma, beta, 1e-5)


@pytest.mark.parametrize("rows,cols", RING)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("with_dh", [True, False])
def test_backward(moe, rows, cols, dtype, with_dh):
    """Many rows a group, so that every slot is filled again, and several groups a block; statistics from 64 bits."""
    n = normal(rows * 3 + cols)
    h, dy, gamma = (2 * n(rows, cols) + 0.5).to(dtype), n(rows, cols).to(dtype), (1 + 0.1 * n(cols)).to(dtype)
    dh = n(rows, cols).to(dtype) if with_dh else None
    var, mean = torch.var_mean(h.double(), 1, correction=0)
    mean, rstd = mean.float(), (var + 1e-5).rsqrt().float()
    out = {"dx": torch.full_like(dy, float("nan")), "dgamma": torch.full((cols,), float("nan"), device="cuda"), "dbeta": torch.full((cols,), float("nan"), device="cuda")}
    o = moe.add_layernorm_backward(dy, h, mean, rstd, gamma, dh=dh, out=out)
    dx, size, dg, dg_size, db, db_size = reference_backward(dy, h, mean, rstd, gamma, dh)
    assert bool(((o["dx"].double() - dx).abs() <= size + HALF[dtype] * (dx.abs() + size) + 1e-45).all())
    assert bool(((o["dgamma"].double() - dg).abs() <= (rows + 8) * U * dg_size).all())
    assert bool(((o["dbeta"].double() - db).abs() <= (rows + 8) * U * db_size).all())
    a, b = dy.clone(), h.clone()
    again = moe.add_layernorm_backward(a, b, mean, rstd, gamma, dh=dh, out={"dx": a, "dgamma": torch.empty_like(dg, dtype=torch.float32)})
    assert torch.equal(again["dx"], o["dx"]) and torch.equal(again["dgamma"], o["dgamma"])      # dx over dy
    if with_dh:
        b = dh.clone()
        again = moe.add_layernorm_backward(dy, h, mean, rstd, gamma, dh=b, out={"dx": b, "dgamma": torch.empty_like(dg, dtype=torch.float32)})
        assert torch.equal(again["dx"], o["dx"])                                               # dx over dh


def test_graph_and_two_streams(moe):
    """The ring's kernels captured and replayed over other inputs, and two calls at a time."""
    n = normal(11)
    rows, cols = 9001, 1024
    x, res, dy, gamma = n(rows, cols).bfloat16(), n(rows, cols).bfloat16(), n(rows, cols).bfloat16(), n(cols).bfloat16()

    def step(stream=None):
        o = moe.add_layernorm(x, res, gamma, want_stats=True, stream=stream)
        return {**o, **moe.add_layernorm_backward(dy, o["h"], o["mean"], o["rstd"], gamma, dh=x, stream=stream)}

    first, side = step(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pairs = [(step(side), step()) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a[k], first[k]) and torch.equal(b[k], first[k]) for a, b in pairs for k in first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rec = step()
    x.copy_(n(rows, cols))
    g.replay()
    torch.cuda.synchronize()
    got = step()
    assert all(torch.equal(rec[k], got[k]) for k in got) and not torch.equal(rec["y"], first["y"])


def test_beyond_32_bits(moe):
    """4.9e9 elements: the gradient's first, middle and last rows and the sums over all rows."""
    if torch.cuda.mem_get_info()[0] < 60 * 2 ** 30:
        pytest.skip("needs 60 GB of device memory")
    rows, cols, part = 300_000, 16384, 5000
    n = normal(12)
    h, dy = (torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    for i in range(0, rows, part):
        h[i:i + part], dy[i:i + part] = n(part, cols).bfloat16(), n(part, cols).bfloat16()
        var, mu = torch.var_mean(h[i:i + part].double(), 1, correction=0)
        mean[i:i + part], rstd[i:i + part] = mu.float(), (var + 1e-5).rsqrt().float()
    gamma = (1 + 0.1 * n(cols)).bfloat16()
    out = {"dx": torch.full_like(dy, float("nan")), "dgamma": torch.empty(cols, device="cuda"), "dbeta": torch.empty(cols, device="cuda")}
    o = moe.add_layernorm_backward(dy, h, mean, rstd, gamma, out=out)
    total = [torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(4)]
    for i in range(0, rows, part):
        s = slice(i, i + part)
        dx, size, *sums = reference_backward(dy[s], h[s], mean[s], rstd[s], gamma, None)
        total = [t + u for t, u in zip(total, sums)]
        assert bool(((o["dx"][s].double() - dx).abs() <= size + HALF[torch.bfloat16] * (dx.abs() + size) + 1e-45).all()), i
    dg, dg_size, db, db_size = total
    # a block adds some 2000 rows one after another, then 152 blocks are joined
    assert bool(((o["dgamma"].double() - dg).abs() <= 2200 * U * dg_size).all())
    assert bool(((o["dbeta"].double() - db).abs() <= 2200 * U * db_size).all())
    del h, dy, out, o
    torch.cuda.empty_cache()
