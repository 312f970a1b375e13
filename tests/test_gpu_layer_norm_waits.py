"""Layer norm when the waits for its own copies run out: each of its numbers is right or NaN, nothing is left under way, and the
next call is right.

A copy of the kernels is built whose waits give up after 0, 1500 or 4000 ns instead of a second, without the poll that sleeps
up to a millisecond before the first look at the clock; everything else in it is the library's."""
import ctypes
import subprocess

import pytest
import torch

from test_gpu_layer_norm import HALF, normal, reference_backward

pytestmark = pytest.mark.gpu

CALLS = ("moe_add_layernorm", "moe_add_layernorm_backward")
SMS = """
namespace nvfp4moe {
int num_sms() {
  int n = 0;
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, 0);
  return n;
}
}
"""


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


@pytest.fixture(scope="module", params=[0, 1500, 4000])
def impatient(moe, request, tmp_path_factory):
    """The library's calls, those of the layer norm with a limit of request.param ns."""
    from nvfp4_mixture_experts_softmax_gb300 import _build
    with open(_build.CSRC + "/layer_norm.cu") as f:
        src = f.read()
    start, end = src.index("__device__ __noinline__ bool wait_on"), src.index("struct Ring {")
    wait = src[start:end]
    assert wait.count("mbar_try_wait(") == 1 and wait.count("> kCopyLimitNs") == 1
    wait = wait.replace("mbar_try_wait(", "mbar_test_wait(").replace("> kCopyLimitNs", f">= {request.param}ull")
    rest = src[end:]
    assert rest.count("return mbar_try_wait(") == 1
    src = src[:start] + wait + rest.replace("return mbar_try_wait(", "return mbar_test_wait(") + SMS
    where = tmp_path_factory.mktemp("waits")
    (where / "layer_norm.cu").write_text(src)
    subprocess.run([_build._nvcc(), *_build.ARCH, *_build.FLAGS, "-shared", "-o", str(where / "waits.so"), str(where / "layer_norm.cu")],
                   check=True, capture_output=True, timeout=300)
    short, full = ctypes.CDLL(str(where / "waits.so")), moe.lib()

    class Calls:
        def __getattr__(self, name):
            f = getattr(full, name)
            if name in CALLS:
                g = getattr(short, name)
                g.restype, g.argtypes = f.restype, f.argtypes
                return g
            return f

    return Calls(), request.param


def right_or_nan(got, want, err):
    """The share of NaN in got; the rest is within err of want."""
    lost = got.isnan()
    assert bool((lost | ((got.double() - want).abs() <= err)).all()), float(((got.double() - want).abs() - err)[~lost].max())
    return float(lost.float().mean())


@pytest.mark.parametrize("rows,cols", [(20011, 256), (9001, 1024), (3001, 4096), (2003, 5120), (2003, 8192), (1300, 16384)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_right_or_nan(moe, impatient, monkeypatch, rows, cols, dtype):
    n = normal(rows + 5 * cols)
    x, res, dy, dh = (n(rows, cols).to(dtype) for _ in range(4))
    gamma, beta = (1 + 0.1 * n(cols)).to(dtype), n(cols).to(dtype)
    new = lambda: ({"h": torch.zeros_like(x), "y": torch.zeros_like(x), "mean": torch.zeros(rows, device="cuda"), "rstd": torch.zeros(rows, device="cuda")},  # noqa: E731
                   {"dx": torch.zeros_like(x), "dgamma": torch.zeros(cols, device="cuda"), "dbeta": torch.zeros(cols, device="cuda")})
    want, back = new()
    moe.add_layernorm(x, res, gamma, beta, out=want)
    args = dy, want["h"], want["mean"], want["rstd"], gamma
    moe.add_layernorm_backward(*args, dh=dh, out=back)
    calls, limit = impatient
    lost = 0.0
    with monkeypatch.context() as m:
        m.setattr(moe, "lib", lambda: calls)
        for _ in range(3):
            o, b = new()
            moe.add_layernorm(x, res, gamma, beta, out=o)
            moe.add_layernorm_backward(*args, dh=dh, out=b)
            torch.cuda.synchronize()
            for got, ref in ((o, want), (b, back)):
                lost += sum(right_or_nan(got[k], ref[k].double(), 0.0) for k in got)
    if limit == 0 and cols == 16384:
        assert lost > 0           # a row takes longer than a poll
    again, behind = new()
    moe.add_layernorm(x, res, gamma, beta, out=again)
    moe.add_layernorm_backward(*args, dh=dh, out=behind)
    assert all(torch.equal(again[k], want[k]) for k in again) and all(torch.equal(behind[k], back[k]) for k in behind)
    dx, size, dg, dg_size, _, _ = reference_backward(*args, dh)
    assert bool(((back["dx"].double() - dx).abs() <= size + HALF[dtype] * (dx.abs() + size)).all())
    assert bool(((back["dgamma"].double() - dg).abs() <= (rows + 8) * 2.0 ** -24 * dg_size).all())
