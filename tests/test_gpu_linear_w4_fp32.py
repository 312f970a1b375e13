"""FP32 output of the 4-bit matrix-vector product over long rows.

Products are exact.  A tensor core's addition truncates: it loses less than 2^-23 of the partial sum.
With terms of one sign the partial sums of a chain of n additions grow to the chain's sum S, so the chain
loses less than the sum of 2^-23 S i / n, about n / 2 * 2^-23 S.  Chains are at most 256 additions long,
and their sums meet in at most 64 rounded additions of 2^-24 each: (128 + 32) * 2^-23 of the sum of
magnitudes, whatever the signs.  (One chain over all of K = 16384 loses half of its bound of 512 * 2^-23,
3e-5.)"""
import pytest
import torch

from test_gpu_linear_w4 import decode, random_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


# one tile whose K a cluster splits, in one and in several parts; a tile for each of half the SMs; several
# tiles a block; parts that are not equal, rows that are no multiple of 128
SHAPES = [(300, 45088), (70, 90112), (19713, 16384), (40961, 7168), (19713, 5152), (39999, 4320)]


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [1, 5, 8, 12, 16, 17, 33, 64])
def test_error_of_long_sums(moe, T, N, K, fmt):
    codes, sf, ts = random_weights(N, K, fmt, False, T + N + K)
    codes &= 0x77                                          # all of one sign: the largest sums
    if fmt == "nvfp4":
        sf = sf % 16 + 0x30
        ts.fill_(1.0)
    else:
        sf = sf % 4 + 125
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(T, K, device="cuda", generator=g).abs().bfloat16()
    y = moe.linear_w4(x, codes, sf, ts, out_dtype=torch.float32).double()
    signs = torch.randint(0, 2, (T, K), device="cuda", generator=g) * 2 - 1
    z = moe.linear_w4((x * signs).bfloat16(), codes, sf, ts, out_dtype=torch.float32).double()
    for i in range(0, N, 4096):
        w = decode(codes[i:i + 4096], sf[i:i + 4096], ts).t()
        size = x.double() @ w
        assert bool(((y[:, i:i + 4096] - size).abs() <= 160 * 2.0 ** -23 * size).all())
        assert bool(((z[:, i:i + 4096] - (x * signs).double() @ w).abs() <= 160 * 2.0 ** -23 * size).all())


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [12, 17, 64])
def test_exact_sums_of_parts(moe, T, N, K, fmt):
    """Whole numbers, equality: |x| <= 1 and half of x zero keeps every sum below 2^24 units."""
    codes, sf, ts = random_weights(N, K, fmt, True, T + N + K)
    g = torch.Generator(device="cuda").manual_seed(K)
    x = (torch.rand(T, K, device="cuda", generator=g) < 0.1).bfloat16()
    buf = torch.full((T + 2, N), 7.0, device="cuda")
    y = moe.linear_w4(x, codes, sf, ts, y=buf[1:T + 1])
    for i in range(0, N, 4096):
        assert torch.equal(y[:, i:i + 4096].double(), x.double() @ decode(codes[i:i + 4096], sf[i:i + 4096], ts).t())
    assert bool((buf[0] == 7).all()) and bool((buf[T + 1] == 7).all())
    assert torch.equal(moe.linear_w4(x, codes, sf, ts, out_dtype=torch.float32), y)
    bad = x.clone()
    bad[T - 1, K - 1] = float("nan")
    y2 = moe.linear_w4(bad, codes, sf, ts, out_dtype=torch.float32)
    assert torch.equal(y2[:T - 1], y[:T - 1]) and bool(y2[T - 1].isnan().all())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [1, 7, 12, 17, 64])
def test_exact_longest_rows(moe, T, fmt):
    """K = 2^20: ordinary x, and a row whose elements lie too far apart for F16 (the product in BF16)."""
    N, K = 37, 1 << 20
    codes, sf, ts = random_weights(N, K, fmt, True, T)
    g = torch.Generator(device="cuda").manual_seed(K)
    x = (torch.rand(T, K, device="cuda", generator=g) < 0.1).bfloat16()
    w = decode(codes, sf, ts).t()
    for dtype in (torch.float32, torch.bfloat16):
        want = (x.double() @ w).to(torch.float32).to(dtype)
        assert torch.equal(moe.linear_w4(x, codes, sf, ts, out_dtype=dtype), want)
    x[0] *= 2.0 ** -60
    x[0, 5:K:2] = 0
    x[0, 4] = 1.0
    codes[:, 2] &= 0xF0                                    # the weight of column 4: zero
    want = (x.double() @ decode(codes, sf, ts).t()).float()
    assert torch.equal(moe.linear_w4(x, codes, sf, ts, out_dtype=torch.float32), want)


@pytest.mark.parametrize("T,N,K", [(64, 300, 45088), (64, 19713, 7168), (24, 19713, 7168), (12, 2048, 16384)])
def test_parts_captured_and_on_two_streams(moe, T, N, K):
    """Calls that follow one another, in a graph, and beside another stream's: exact each time."""
    codes, sf, ts = random_weights(N, K, "nvfp4", True, 3)
    w = decode(codes, sf, ts).float()

    def rows(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return (torch.rand(T, K, device="cuda", generator=g) < 0.1).bfloat16()

    def exact(y, x):
        return torch.equal(y.double(), torch.cat([x.double() @ p.double().t() for p in w.split(4096)], 1))

    x, other, side = rows(0), rows(1), torch.cuda.Stream()
    moe.linear_w4(x, codes, sf, ts, out_dtype=torch.float32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = [moe.linear_w4(x, codes, sf, ts, out_dtype=torch.float32) for _ in range(3)]
    for seed in (2, 3):
        x.copy_(rows(seed))
        graph.replay()
        assert all(exact(t, x) for t in y)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = [moe.linear_w4(other, codes, sf, ts, out_dtype=torch.float32) for _ in range(12)]
    a = [moe.linear_w4(x, codes, sf, ts, out_dtype=torch.float32) for _ in range(12)]
    torch.cuda.synchronize()
    assert exact(a[0], x) and exact(b[0], other)
    assert all(torch.equal(t, a[0]) for t in a) and all(torch.equal(t, b[0]) for t in b)
