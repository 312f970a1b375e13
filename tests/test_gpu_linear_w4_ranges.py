"""The 4-bit matrix-vector product where scales or elements of x lie far apart: the same results
whatever the number of rows, which decides the kernel.

Equality throughout: x and the codes are small whole numbers or halves and the scales that meet in
one sum span two binades, so every product and partial sum is a multiple of one power of two below
2^24 of it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
ROWS = [1, 3, 8, 9, 12, 16, 17, 40]
# one block and many, clusters that split K, rows longer than shared memory
SHAPES = [(40, 64), (300, 2048), (129, 7168), (33, 32768)]


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


def decode(codes, sf, ts=None):
    t = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device="cuda")
    v = t[torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1).long()]
    s = sf.view(torch.float8_e4m3fn).double() * ts.double() if ts is not None else torch.exp2(sf.double() - 127)
    return v * s.repeat_interleave(v.shape[1] // sf.shape[1], 1)


def whole(shape, top, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, device="cuda", generator=g).bfloat16()


def mx_weights(N, K, seed):
    """Codes, and scales of 1/2, 1 and 2."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), device="cuda", generator=g, dtype=torch.uint8)
    return codes, torch.randint(126, 129, (N, K // 32), device="cuda", generator=g).to(torch.uint8), g


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("T", ROWS)
def test_mxfp4_zero_blocks_of_any_scale(moe, T, N, K):
    """A block of zeros (of either sign) may carry any scale: it takes no part."""
    codes, sf, g = mx_weights(N, K, N + K)
    bytes_of = torch.tensor([0, 1, 90, 103, 141, 165, 200, 254], device="cuda", dtype=torch.uint8)
    zero = torch.rand(N, K // 32, device="cuda", generator=g) < 0.3
    zero[N // 2] = True                                   # a row of nothing else
    sf = torch.where(zero, bytes_of[torch.randint(0, 8, zero.shape, device="cuda", generator=g)], sf)
    signs = torch.randint(0, 4, codes.shape, device="cuda", generator=g)
    empty = ((signs & 1) * 0x08 + (signs >> 1) * 0x80).to(torch.uint8)
    codes = torch.where(zero.repeat_interleave(16, 1), empty, codes)
    x = whole((T, K), 1, K)                               # 24 units of 1/4 a term at most: 32768 of them below 2^24
    want = x.double() @ decode(codes, sf).t()
    assert torch.equal(moe.linear_w4(x, codes, sf, out_dtype=torch.float32).double(), want)


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("T", ROWS)
def test_mxfp4_scales_far_apart(moe, T, N, K):
    """Blocks of 2^-100, 2^-60, 1 and 2^90 in one row; each row of x meets one of these classes only."""
    codes, sf, g = mx_weights(N, K, N + K + 1)
    blocks = torch.arange(K // 32, device="cuda") % 4
    sf = (sf.int() + torch.tensor([-100, -60, 0, 90], device="cuda")[blocks]).to(torch.uint8)
    x = whole((T, K), 1, K)
    x *= (torch.arange(T, device="cuda")[:, None] % 4 == blocks.repeat_interleave(32))
    want = x.double() @ decode(codes, sf).t()
    assert torch.equal(moe.linear_w4(x, codes, sf, out_dtype=torch.float32).double(), want)
    # one odd block in a matrix of ordinary ones
    codes, sf, _ = mx_weights(N, K, N + K + 2)
    sf[N // 3, K // 64] = 20
    x = whole((T, K), 1, K + 1)
    x[:, K // 64 * 32:K // 64 * 32 + 32] *= (torch.arange(T, device="cuda")[:, None] % 2 == 0)
    x[::2] = 0
    x[::2, K // 64 * 32:K // 64 * 32 + 32] = 1
    want = x.double() @ decode(codes, sf).t()
    y = moe.linear_w4(x, codes, sf, out_dtype=torch.float32).double()
    assert torch.equal(y[1::2], want[1::2])               # ordinary blocks only
    assert torch.equal(y[::2, N // 3], want[::2, N // 3])   # the odd one only


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("T", ROWS)
def test_elements_of_x_far_apart(moe, T, N, K, fmt):
    """Each row of x has columns of two magnitudes; each row of weights is zero at one of the two, so
    that the small elements stand alone in half of the outputs."""
    codes, sf, g = mx_weights(N, K, N + K + 3)
    ts = None
    if fmt == "nvfp4":
        sf = torch.exp2(torch.randint(0, 3, (N, K // 16), device="cuda", generator=g).float()).to(torch.float8_e4m3fn).view(torch.uint8)
        ts = torch.tensor([0.25], device="cuda")
    small = torch.rand(K // 2, device="cuda", generator=g).repeat_interleave(2) < 0.5        # columns
    drop = small[None, ::2] == (torch.arange(N, device="cuda")[:, None] % 2 == 0)            # code bytes
    codes = torch.where(drop, 0, codes).to(torch.uint8)
    x = whole((T, K), 1, K + 5).double()
    large_e = torch.tensor([0.0, -6, 60, -90, 3, 20, 120, 0], device="cuda", dtype=torch.float64)
    small_e = torch.tensor([0.0, -26, -20, -130, -40, -13, 70, 0], device="cuda", dtype=torch.float64)
    for first in range(8 if T == 1 else 1):                # which pairs meet in one call
        row = (torch.arange(T, device="cuda") + first) % 8
        xs = (x * torch.exp2(torch.where(small, small_e[row][:, None], large_e[row][:, None]))).bfloat16()
        w = decode(codes, sf, ts)
        want = (xs.double() @ w.t()).float()
        # a partial sum is bounded only by the sum of the magnitudes: where that is beyond FP32 (some
        # sums of 2^120), a partial sum may be infinite although the whole one is not
        inside = xs.double().abs() @ w.abs().t() < torch.finfo(torch.float32).max
        y = moe.linear_w4(xs, codes, sf, ts, out_dtype=torch.float32)
        assert bool(((y == want) | ~inside).all()), first
        y = moe.linear_w4(xs, codes, sf, ts)
        assert bool(((y == want.bfloat16()) | ~inside).all()), first


@pytest.mark.parametrize("T", [1, 8, 12, 20])
def test_one_outlier_whose_weight_is_zero(moe, T):
    """The outlier decides the power of two of its row, and then has no part in the sums."""
    codes, sf, _ = mx_weights(64, 512, 5)
    codes[:, 100] = 0
    ordinary = whole((T, 512), 3, 6)
    for outlier, rest in ((-6, -26), (9, -30), (10, 0), (30, -5), (-60, -133)):
        x = (ordinary.double() * 2.0 ** rest).bfloat16()
        x[:, 200] = 2.0 ** outlier
        want = (x.double() @ decode(codes, sf).t()).float()
        assert torch.equal(moe.linear_w4(x, codes, sf, out_dtype=torch.float32), want), (outlier, rest)


@pytest.mark.parametrize("T", [1, 8, 12])
def test_nonfinite_x_beside_a_wide_row(moe, T):
    """NaN and infinity stay in their row of y where the product takes BF16."""
    codes, sf, _ = mx_weights(64, 512, 7)
    nv = torch.full((64, 32), 0x38, dtype=torch.uint8, device="cuda")     # ones
    x = whole((T + 2, 512), 2, 8)[:T + 2].contiguous()
    x = x[:T]
    x[0, ::2] *= 2.0 ** -50
    for args in ((codes, sf), (codes, nv, torch.ones(1, device="cuda"))):
        clean = moe.linear_w4(x, *args, out_dtype=torch.float32)
        for v in (float("nan"), float("inf")):
            bad = x.clone()
            bad[T - 1, 17] = v
            y = moe.linear_w4(bad, *args, out_dtype=torch.float32)
            assert torch.equal(y[:T - 1], clean[:T - 1]) and not bool(y[T - 1].isfinite().any())
