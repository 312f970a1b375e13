"""The 4-bit matrix-vector product against decoded weights in 64 bits.

Two kinds of check.  With whole-number x (|x| <= 4) and power-of-two block scales every product
is a multiple of 1/2 of a bounded size and every partial sum is exact in FP32, so the result is
exact whatever the order: equality, which no wrong index survives.  With normal data: the products
are exact, and the sum of K terms runs through at most K / 128 + 8 FP32 accumulations of
tensor-core dot products, each within 2^-21 of the sum of magnitudes: (K / 128 + 16) * 2^-21 of
sum |x w|, plus half a BF16 step for BF16 output."""
import pytest
import torch

pytestmark = pytest.mark.gpu

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


def decode(codes, sf, ts):
    t = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device="cuda")
    v = t[torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1).long()]
    s = sf.view(torch.float8_e4m3fn).double() * ts.double() if ts is not None else torch.exp2(sf.double() - 127)
    return v * s.repeat_interleave(v.shape[1] // sf.shape[1], 1)


def random_weights(N, K, fmt, exact, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), device="cuda", generator=g, dtype=torch.uint8)
    if fmt == "nvfp4":
        if exact:    # 1, 2 or 4
            sf = torch.exp2(torch.randint(0, 3, (N, K // 16), device="cuda", generator=g).float()).to(torch.float8_e4m3fn).view(torch.uint8)
            ts = torch.tensor([0.5], device="cuda")
        else:        # any positive finite scale, subnormal ones too
            sf = torch.randint(0, 0x7F, (N, K // 16), device="cuda", generator=g, dtype=torch.uint8)
            ts = torch.tensor([3.7e-5], device="cuda")
        return codes, sf, ts
    lo, hi = (126, 129) if exact else (100, 140)
    return codes, torch.randint(lo, hi, (N, K // 32), device="cuda", generator=g).to(torch.uint8), None


SHAPES = [(1, 1, 32), (1, 16, 128), (3, 17, 96), (8, 2048, 2048), (9, 40, 4064), (16, 129, 1024), (17, 33, 160), (32, 100, 2080),
          (33, 15, 224), (64, 257, 7168), (64, 16, 32), (1, 511, 16384), (2, 1000, 992), (7, 4097, 512), (63, 31, 1056), (5, 3, 65536)]


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_exact(moe, T, N, K, fmt, dtype):
    codes, sf, ts = random_weights(N, K, fmt, True, T + N + K)
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randint(-4, 5, (T, K), device="cuda", generator=g).bfloat16()
    buf = torch.full((T + 2, N), 7.0, dtype=dtype, device="cuda")
    y = moe.linear_w4(x, codes, sf, ts, y=buf[1:T + 1])
    want = (x.double() @ decode(codes, sf, ts).t()).float().to(dtype)
    assert torch.equal(y, want)
    assert bool((buf[0] == 7).all()) and bool((buf[T + 1] == 7).all())
    assert torch.equal(moe.linear_w4(x, codes, sf, ts, out_dtype=dtype), want)


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_normal_data(moe, T, N, K, fmt):
    codes, sf, ts = random_weights(N, K, fmt, False, T + N + K)
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(T, K, device="cuda", generator=g).bfloat16()
    w = decode(codes, sf, ts)
    want, size = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    tol = (K / 128 + 16) * 2.0 ** -21 * size
    y = moe.linear_w4(x, codes, sf, ts, out_dtype=torch.float32)
    assert bool(((y.double() - want).abs() <= tol).all())
    b = moe.linear_w4(x, codes, sf, ts)
    assert torch.equal(b, y.bfloat16())
    # a token's result does not depend on the other tokens of the same launch size class
    one = moe.linear_w4(x[:1].contiguous(), codes, sf, ts, out_dtype=torch.float32)
    assert bool(((one.double() - want[:1]).abs() <= tol[:1]).all())


def test_quantised_matrix_and_every_code(moe):
    """quantize_act of a BF16 matrix is the weight format; then every code with every scale."""
    g = torch.Generator(device="cuda").manual_seed(5)
    W = (torch.randn(96, 512, device="cuda", generator=g) * 0.02).bfloat16()
    codes, sf, ts = moe.quantize_act(W)
    x = torch.randn(4, 512, device="cuda", generator=g).bfloat16()
    y = moe.linear_w4(x, codes, sf, ts, out_dtype=torch.float32)
    want = x.double() @ decode(codes, sf, ts).t()
    assert float((y.double() - want).norm() / want.norm()) <= 2.0 ** -20
    assert float((y.double() - x.double() @ W.double().t()).norm() / want.norm()) < 0.2
    # one-hot x reads single weights: bit-exact in FP32 for every finite scale byte of both signs
    sfb = torch.tensor([b for b in range(256) if (b & 0x7F) != 0x7F], device="cuda", dtype=torch.uint8)
    N = sfb.numel()
    codes = (torch.arange(8, device="cuda") * 2 + (torch.arange(8, device="cuda") * 2 + 1) * 16).to(torch.uint8).repeat(N, 2)
    sf = sfb[:, None].repeat(1, 2).contiguous()
    one = torch.tensor([1.0], device="cuda")
    y = moe.linear_w4(torch.eye(32, device="cuda").bfloat16(), codes, sf, one, out_dtype=torch.float32)
    assert torch.equal(y.t().double(), decode(codes, sf, one))
    # every E8M0 scale: the products are exact down to BF16's smallest subnormal
    b = torch.arange(0, 253, device="cuda", dtype=torch.uint8)
    codes = codes[:1].repeat(253, 1)
    y = moe.linear_w4(torch.eye(32, device="cuda").bfloat16(), codes, b[:, None].contiguous(), out_dtype=torch.float32)
    assert torch.equal(y.t().double(), decode(codes, b[:, None], None))


LONG = [(64, 100, 16384), (8, 70, 16384), (12, 33, 32768), (33, 40, 20000 // 32 * 32), (1, 20, 131072)]


@pytest.mark.parametrize("T,N,K", LONG)
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_exact_rows_longer_than_shared_memory(moe, T, N, K, fmt):
    """|x| <= 1 keeps the whole-number sums of K terms exact: at most 24 K in units of 1/2 (NVFP4)
    or 12 K in units of 1/4, below 2^24 up to K = 131072 / 1 with half of x zero."""
    codes, sf, ts = random_weights(N, K, fmt, True, T + N + K)
    g = torch.Generator(device="cuda").manual_seed(K)
    x = (torch.rand(T, K, device="cuda", generator=g) < 0.1).bfloat16()
    y = moe.linear_w4(x, codes, sf, ts, out_dtype=torch.float32)
    assert torch.equal(y.double(), x.double() @ decode(codes, sf, ts).t())


@pytest.mark.parametrize("T,N,K", [(1, 50, 512), (8, 33, 4096), (16, 40, 7168), (30, 70, 2048), (64, 40, 16384)])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_rows_of_any_magnitude(moe, T, N, K, fmt):
    """Rows of x far from one, with outliers, of zeros, and MXFP4 rows whose scales span more than
    F16.  Elements of x are at worst rounded to 2^-24 of their row's largest (half of 2^-30 where
    that is at least 2^-6), scales below 2^-36 of a row's largest are zero."""
    codes, sf, ts = random_weights(N, K, fmt, False, T + N + K)
    g = torch.Generator(device="cuda").manual_seed(K)
    if fmt == "mxfp4":
        rows = torch.randint(0, 4, (N, 1), device="cuda", generator=g)
        spread = torch.randint(0, 60, (N, K // 32), device="cuda", generator=g)
        base = torch.tensor([110, 20, 180, 64], device="cuda")[rows]
        sf = torch.where(rows == 0, base + spread % 8, base + spread).to(torch.uint8)
    x = torch.randn(T, K, device="cuda", generator=g)
    e = torch.tensor([0, 30, -60, 12, -14, 0, -100, 3], device="cuda")[torch.arange(T, device="cuda") % 8].double()
    x = (x.double() * torch.exp2(e)[:, None]).float().bfloat16()
    x[T // 2, 7] = 2.0 ** 20 * x[T // 2].abs().max()
    if T > 3:
        x[3] = 0
    w = decode(codes, sf, ts)
    want, size = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    top = x.double().abs().amax(1, keepdim=True)
    tol = (K / 128 + 16) * 2.0 ** -21 * size + 2.0 ** -24 * top * w.abs().sum(1)
    if fmt == "mxfp4":
        tol = tol + x.double().abs().sum(1, keepdim=True) * 6 * 2.0 ** -36 * torch.exp2(sf.double().amax(1) - 127)
    y = moe.linear_w4(x, codes, sf, ts, out_dtype=torch.float32).double()
    # FP32 sums: a partial sum is bounded only by the sum of the magnitudes, so where that is beyond
    # FP32's 3.4e38 a partial sum may be infinite although the whole one is not
    over = size + tol > 3e38
    under = 2.0 ** -140                        # FP32's own smallest steps
    assert bool((((y - want).abs() <= tol + under) | over).all())


@pytest.mark.parametrize("T", [1, 12, 40])
def test_nonfinite(moe, T):
    codes, sf, ts = random_weights(40, 256, "nvfp4", False, 7)
    x = torch.randn(T, 256, device="cuda").bfloat16()
    clean = moe.linear_w4(x, codes, sf, ts)
    sf2 = sf.clone()
    sf2[5, 3] = 0x7F                      # NaN scale: its row alone
    y = moe.linear_w4(x, codes, sf2, ts)
    rest = [n for n in range(40) if n != 5]
    assert bool(y[:, 5].isnan().all()) and torch.equal(y[:, rest], clean[:, rest])
    mx = random_weights(40, 256, "mxfp4", False, 8)
    s2 = mx[1].clone()
    s2[9, 1] = 255
    y = moe.linear_w4(x, mx[0], s2)
    assert bool(y[:, 9].isnan().all()) and bool(y[:, rest[:8]].isfinite().all())
    x2 = x.clone()
    x2[T - 1, 17] = float("nan")          # NaN in one token: that token alone
    y = moe.linear_w4(x2, codes, sf, ts)
    assert bool(y[T - 1].isnan().all()) and torch.equal(y[:T - 1], clean[:T - 1])


# N and K around the splits of the kernel for many rows: tiles of 256 weight rows, blocks of a cluster
# that split K in steps of 128 (one of them with nothing left), scales that are not loaded in one piece
MANY = [(9, 1, 32), (10, 255, 1184), (16, 257, 2048), (17, 300, 2144), (24, 256, 2176), (31, 520, 96), (33, 2000, 1056),
        (40, 2049, 4096), (48, 3841, 2080), (49, 9217, 512), (64, 10001, 640), (63, 19457, 288), (20, 40000, 160),
        (17, 120001, 32), (64, 99999, 224), (33, 79900, 416)]   # several tiles a block, fewer steps than warp groups


@pytest.mark.parametrize("T,N,K", MANY)
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_exact_many_rows(moe, T, N, K, fmt):
    """|x| <= 2: terms of at most 96 units of 1/4, whole sums of up to 4096 of them below 2^24."""
    codes, sf, ts = random_weights(N, K, fmt, True, T + N + K)
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randint(-2, 3, (T, K), device="cuda", generator=g).bfloat16()
    want = (x.double() @ decode(codes, sf, ts).t()).float()
    buf = torch.full((T + 2, N), 7.0, device="cuda")
    assert torch.equal(moe.linear_w4(x, codes, sf, ts, y=buf[1:T + 1]), want)
    assert bool((buf[0] == 7).all()) and bool((buf[T + 1] == 7).all())
    # scales that start two bytes into an allocation
    off = torch.empty(sf.numel() + 2, dtype=torch.uint8, device="cuda")[2:].view(sf.shape)
    off.copy_(sf)
    assert torch.equal(moe.linear_w4(x, codes, off, ts, out_dtype=torch.float32), want)


@pytest.mark.parametrize("T", [12, 50])
def test_many_rows_captured_and_on_two_streams(moe, T):
    """Calls that follow one another on a stream, in a graph, and beside another stream's."""
    codes, sf, ts = random_weights(1024, 1024, "nvfp4", True, 3)
    ts.fill_(2.0 ** -6)
    w = decode(codes, sf, ts)
    x = torch.randint(-1, 2, (T, 1024), device="cuda").bfloat16()

    def chain(x):
        return moe.linear_w4(moe.linear_w4(x, codes, sf, ts), codes, sf, ts, out_dtype=torch.float32)

    def formula(x):
        mid = (x.double() @ w.t()).float().bfloat16().double()
        return mid @ w.t(), mid.abs() @ w.abs().t()

    def close(y, x):
        want, size = formula(x)   # the first product is exact; K / 128 + 16 roundings as above
        return bool(((y.double() - want).abs() <= (1024 / 128 + 16) * 2.0 ** -21 * size).all())

    chain(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = chain(x)
    for seed in range(3):
        x.copy_(torch.randint(-1, 2, (T, 1024), device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)))
        graph.replay()
        assert close(y, x)
    side, other = torch.cuda.Stream(), torch.randint(-1, 2, (T, 1024), device="cuda").bfloat16()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = [chain(other) for _ in range(20)]
    a = [chain(x) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(close(t, x) for t in a) and all(close(t, other) for t in b)
    assert all(torch.equal(t, a[0]) for t in a) and all(torch.equal(t, b[0]) for t in b)


def test_large_offsets(moe):
    """More than 2^32 bytes of codes: the last rows."""
    N, K = 70000, 131072
    if torch.cuda.mem_get_info()[0] < (12 << 30):
        pytest.skip("not enough memory")
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    sf = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    codes[-3:] = 0x22                     # ones
    x = torch.ones(2, K, dtype=torch.bfloat16, device="cuda")
    y = moe.linear_w4(x, codes, sf, out_dtype=torch.float32)
    assert bool((y[:, -3:] == K).all()) and not y[:, :-3].any()


def test_threads_with_different_sizes(moe):
    """Two host threads whose launches of one kernel need different shared memory."""
    import threading
    sizes = [[(8, 64, 13312), (8, 64, 4096)], [(16, 64, 6656), (16, 64, 4480)], [(64, 512, 4096), (20, 512, 4096)]]
    work = {s: random_weights(s[1], s[2], "nvfp4", True, 1) for pair in sizes for s in pair}
    x = {s: torch.ones(s[0], s[2], device="cuda").bfloat16() for s in work}
    want = {s: moe.linear_w4(x[s], *work[s]) for s in work}
    for pair in sizes:
        wrong = []

        def run(s):
            try:
                with torch.cuda.stream(torch.cuda.Stream()):
                    out = [moe.linear_w4(x[s], *work[s]) for _ in range(300)]
                    torch.cuda.current_stream().synchronize()
                wrong.extend(1 for o in out if not torch.equal(o, want[s]))
            except Exception as error:
                wrong.append(error)

        torch.cuda.synchronize()
        threads = [threading.Thread(target=run, args=(s,)) for s in pair]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not wrong


def test_large_offsets_many_rows(moe):
    N, K = 70000, 131072
    if torch.cuda.mem_get_info()[0] < (12 << 30):
        pytest.skip("not enough memory")
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    sf = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    codes[-3:] = 0x22                     # ones
    x = torch.ones(17, K, dtype=torch.bfloat16, device="cuda")
    y = moe.linear_w4(x, codes, sf, out_dtype=torch.float32)
    assert bool((y[:, -3:] == K).all()) and not y[:, :-3].any()


def test_empty_stream_and_graph(moe):
    codes, sf, ts = random_weights(48, 512, "nvfp4", False, 9)
    x = torch.randn(3, 512, device="cuda").bfloat16()
    assert moe.linear_w4(x[:0], codes, sf, ts).shape == (0, 48)
    assert moe.linear_w4(x, codes[:0], sf[:0], ts).shape == (3, 0)
    want = moe.linear_w4(x, codes, sf, ts)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = moe.linear_w4(x, codes, sf, ts, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    y = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.linear_w4(x, codes, sf, ts, y=y)
    x.copy_(torch.randn(3, 512, device="cuda"))
    graph.replay()
    want = moe.linear_w4(x, codes, sf, ts)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_refusals(moe):
    codes, sf, ts = random_weights(48, 512, "nvfp4", False, 9)
    x = torch.randn(3, 512, device="cuda").bfloat16()
    with pytest.raises(ValueError, match="x must"):
        moe.linear_w4(x.float(), codes, sf, ts)
    with pytest.raises(ValueError, match="codes"):
        moe.linear_w4(x, codes[:, :128].contiguous(), sf, ts)
    with pytest.raises(ValueError, match="sf"):
        moe.linear_w4(x, codes, sf)                 # NVFP4 scales without a tensor scale
    with pytest.raises(ValueError, match="x must"):
        moe.linear_w4(x[:, ::2], codes[:, ::2], sf[:, ::2], ts)
    with pytest.raises(ValueError, match="output"):
        moe.linear_w4(x, codes, sf, ts, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="multiple of 32"):
        moe.linear_w4(x[:, :40].contiguous(), codes, sf, ts)
    with pytest.raises(RuntimeError, match="UNSUPPORTED_SHAPE"):
        moe.linear_w4(x[:1].repeat(65, 1), codes, sf, ts)
    flat = torch.zeros(3 * 512 + 1, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        moe.linear_w4(flat[1:].reshape(3, 512), codes, sf, ts)
