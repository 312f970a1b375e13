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
