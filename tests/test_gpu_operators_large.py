"""The operators around the layer at sizes where their blocks work through several rows: rows read
ahead, several row groups a block, losses joined by a cluster with several experts a lane.

References, magnitudes and bounds are those of test_gpu_add_rmsnorm_mx.py and
test_gpu_router_loss.py; their derivations hold for any number of rows."""
import pytest
import torch

from test_gpu_add_rmsnorm_mx import BF16_HALF, R_REL, Y_REL, backward_reference, check_codes, make as make_rows, reference
from test_gpu_router_loss import G_REL, ROUTERS, U, forward_reference, gradient_reference, make as make_logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


# (more than two rows an SM take row groups; above that, more rows than groups on the GPU)
ROWS = [(20000, 256), (9001, 96), (5000, 1024), (4099, 4128), (2500, 7168), (2000, 16384)]


@pytest.mark.parametrize("rows,cols", ROWS)
def test_norm_of_many_rows(moe, rows, cols):
    x, res, gamma = make_rows(rows, cols, rows + cols)
    o = moe.add_rmsnorm_quantize_mx(x, res, gamma, 1e-5, want_y=True, want_rrms=True)
    h, r, y = reference(x, res, gamma, 1e-5)
    assert torch.equal(o["h"], h)
    assert float(((o["rrms"].double() - r).abs() / r).max()) <= R_REL
    assert bool(((o["y"].double() - y).abs() <= (BF16_HALF + Y_REL) * y.abs() + 1e-40).all())
    check_codes(o["codes"], o["sf"], y)
    # in place over either input, and without a residual
    for inplace in ("residual", "x"):
        x2, r2 = x.clone(), res.clone()
        out = {k: torch.full_like(v, 7) for k, v in o.items()}
        out["h"] = r2 if inplace == "residual" else x2
        moe.add_rmsnorm_quantize_mx(x2, r2, gamma, 1e-5, out=out)
        assert all(torch.equal(out[k], o[k]) for k in o)
    again = moe.add_rmsnorm_quantize_mx(h, None, gamma, 1e-5, want_y=True, want_rrms=True)
    assert all(torch.equal(again[k], o[k]) for k in again)


@pytest.mark.parametrize("rows,cols", [(20000, 512), (9001, 96), (5000, 2048), (2001, 7168), (1000, 16384), (3000, 8224)])
@pytest.mark.parametrize("with_dh", [True, False])
def test_norm_backward_of_many_rows(moe, rows, cols, with_dh):
    h, dy, gamma = make_rows(rows, cols, rows * 3 + cols)
    dh = make_rows(rows, cols, 9)[0] if with_dh else None
    r = moe.add_rmsnorm_quantize_mx(h, None, gamma, want_rrms=True)["rrms"]
    o = moe.add_rmsnorm_backward(dy, h, r, gamma, dh=dh)
    dx, size, dg, dgsize = backward_reference(dy, h, r, gamma, dh)
    assert bool(((o["dx"].double() - dx).abs() <= BF16_HALF * dx.abs() + Y_REL * size).all())
    assert bool(((o["dgamma"].double() - dg).abs() <= (rows + 8) * 2.0 ** -24 * dgsize).all())
    for buf in ("dy", "dh") if with_dh else ("dy",):
        dy2, dh2 = dy.clone(), None if dh is None else dh.clone()
        got = moe.add_rmsnorm_backward(dy2, h, r, gamma, dh=dh2,
                                       out={"dx": dy2 if buf == "dy" else dh2, "dgamma": torch.empty_like(o["dgamma"])})
        assert torch.equal(got["dx"], o["dx"]) and torch.equal(got["dgamma"], o["dgamma"])


TOKENS = [(60000, 60, 4), (30000, 31, 6), (40000, 128, 8), (20000, 256, 8), (9000, 510, 9), (5000, 1021, 16), (5000, 1024, 32),
          (2000, 300, 8), (2000, 600, 3), (2000, 1000, 8), (3001, 720, 5)]


@pytest.mark.parametrize("T,E,k", TOKENS)
@pytest.mark.parametrize("router", ROUTERS)
@pytest.mark.parametrize("masked", [False, True])
def test_losses_and_gradient_of_many_tokens(moe, T, E, k, router, masked):
    l, ids, gw, mask = make_logits(T, E, k, T + E, masked)
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
    gl = [0.7, -0.3]
    got = moe.router_loss_backward(l, ids, o, torch.tensor(gl, device="cuda"), grad_topk_w=gw, mask=mask, router=router)
    want, size = gradient_reference(l, ids, gw, mask, router, gl)
    assert bool(((got.double() - want).abs() <= G_REL * size + 1e-30).all())
    if masked:
        assert not got[~mask].any()


def _room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip("not enough memory")


def test_norm_beyond_2_32_elements(moe):
    """The last rows of 4.3 G elements, as a call of their own gives them."""
    _room(80)
    rows, cols = 263000, 16384
    x, res = (torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    xs, rs, gamma = make_rows(400, cols, 1)
    x[-400:], res[-400:] = xs, rs
    want = moe.add_rmsnorm_quantize_mx(xs, rs, gamma, want_y=True, want_rrms=True)
    o = moe.add_rmsnorm_quantize_mx(x, res, gamma, out={"h": x, "codes": torch.empty(rows, cols, dtype=torch.uint8, device="cuda"),
                                                        "sf": torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda"),
                                                        "rrms": torch.empty(rows, device="cuda")})
    assert all(torch.equal(o[k][-400:], want[k]) for k in o) and not o["codes"][:1000].any()
    del o["codes"], res
    dy = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    dy[-400:] = rs
    g = moe.add_rmsnorm_backward(dy, x, o["rrms"], gamma, out={"dx": dy, "dgamma": torch.empty(cols, device="cuda")})
    dx, size, dg, dgsize = backward_reference(rs, want["h"], want["rrms"], gamma, None)
    assert bool(((g["dx"][-400:].double() - dx).abs() <= BF16_HALF * dx.abs() + Y_REL * size).all()) and not g["dx"][:1000].any()
    assert bool(((g["dgamma"].double() - dg).abs() <= (rows + 8) * 2.0 ** -24 * dgsize).all())


@pytest.mark.parametrize("router", ROUTERS)
def test_losses_beyond_2_32_elements(moe, router):
    """4.3 G logits: sums over all tokens against the same token counted often, gradients of the last
    tokens against a call of their own."""
    _room(60)
    T, E, k = 4200000, 1024, 4
    l1, ids1, _, _ = make_logits(100, E, k, 3)
    l = torch.empty(T, E, device="cuda")
    l.view(T // 100, 100, E).copy_(l1.expand(T // 100, 100, E))
    ids = ids1.repeat(T // 100, 1)
    o = moe.router_loss(l, ids, router=router)
    bal, z, counts, n, P = forward_reference(l1, ids1, None, router)
    assert torch.equal(o["counts"].long(), counts * (T // 100)) and int(o["tokens"]) == T
    # a warp's chain over T / (152 * 16) tokens, then sums over warps and blocks, each in FP32
    tol = (T / (152 * 16) + 16 + 152 + 128) * U
    assert bool(((o["probs"].double() - P).abs() <= tol * P).all())
    assert abs(float(o["losses"][0]) - float(bal)) <= tol * float(bal) and abs(float(o["losses"][1]) - float(z)) <= 4 * tol * float(z)
    gl, gw = torch.tensor([0.7, -0.3], device="cuda"), torch.randn(T, k, device="cuda")
    d = moe.router_loss_backward(l, ids, o, gl, grad_topk_w=gw, router=router)
    few = moe.router_loss_backward(l[-500:].clone(), ids[-500:].clone(), o, gl, grad_topk_w=gw[-500:].clone(), router=router)
    assert torch.equal(d[-500:], few)
