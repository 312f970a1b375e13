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
