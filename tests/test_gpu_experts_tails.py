"""The weights' gradients at the ends of segments: what is behind a segment's last row takes no part, whatever it holds and
however the segments follow one another.

Bounds as in the experts' own tests: a chain of at most 44 additions in the tensor cores, which truncate (2^-22 of the
terms' magnitudes each), then one FP32 addition (2^-24) a chain."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, STEP, U = torch.bfloat16, 2.0 ** -22, 2.0 ** -24


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("H,I", [(256, 256), (512, 160), (96, 480)])
def test_neighbours_stay_out(moe, H, I):
    """Segments of 1 to 130 rows, every other one of huge rows: a row of a neighbour in a sum, from either half of either
    operand, would be 2^60 times what the sum may be off by.  The same bits in each of twenty passes over a busy GPU."""
    g = torch.Generator(device="cuda").manual_seed(H + I)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    lens = torch.randint(1, 131, (300,), generator=torch.Generator().manual_seed(7))
    lens[::29] = 64
    off = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)])
    R = int(off[-1])
    big = torch.repeat_interleave(torch.tensor([1.0, 2.0 ** 40]).repeat(150), lens).cuda()[:, None]
    x, dout, h, dg, du = ((n(R + 70, w)).to(BF16) for w in (H, H, I, I, I))
    for t in (x, dout, h, dg, du):
        t[:R] *= big.to(BF16)
        t[R:] = float("nan")                     # behind the last segment
    plan = {"offsets": off.to(torch.int32).cuda()}
    ws = moe.experts_workspace(0, I)
    first = moe.experts_weight_grad(x, dout, {"h": h}, {"dg": dg, "du": du}, plan, workspace=ws)
    assert moe.last_device_status(ws) == 0
    for name, left, right in (("w_gate", dg, x), ("w_up", du, x), ("w_down", dout, h)):
        for e in range(0, 300, 2):
            a, b = (t[off[e]:off[e + 1]].double() for t in (left, right))
            bound = (12 * STEP + 2 * U) * (a.abs().t() @ b.abs())          # three blocks: twelve additions
            assert bool(((first[name][e].double() - a.t() @ b).abs() <= bound + 1e-38).all()), (name, e)
    for _ in range(20):
        again = moe.experts_weight_grad(x, dout, {"h": h}, {"dg": dg, "du": du}, plan, workspace=ws)
        assert all(torch.equal(again[k].view(torch.int32), first[k].view(torch.int32)) for k in first)


def test_one_long_ragged_segment(moe):
    """One expert of 6e8 + 37 narrow rows, 2.5 s of products: no wait of the kernel lasts that long, as none spans more than
    a block or a chain.  Whole numbers in a few rows: the sums are exact."""
    if torch.cuda.mem_get_info()[0] < 60 * 2 ** 30:
        pytest.skip("needs 60 GB of device memory")
    R = 600_000_037
    x = torch.zeros(R, 32, dtype=BF16, device="cuda")
    at = torch.tensor([0, 63, 64, 2 ** 28 + 5, R // 2, R - 38, R - 37, R - 36, R - 1], device="cuda")
    x[at] = torch.randint(-8, 9, (len(at), 32), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).to(BF16)
    some = x[at].double()
    plan = {"offsets": torch.tensor([0, R], dtype=torch.int32, device="cuda")}
    ws = moe.experts_workspace(0, 32)
    w = moe.experts_weight_grad(x, x, {"h": x}, {"du": x}, plan, workspace=ws)
    assert moe.last_device_status(ws) == 0
    for name in ("w_up", "w_down"):
        assert torch.equal(w[name][0].double(), some.t() @ some)
    del x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("lens", [[1], [63, 65], [5, 1, 2], [0, 0, 17, 0, 700]])
def test_first_and_last_rows_of_the_tensors(moe, lens):
    """Segments whose last block is also the first rows, or the last ones, of the tensors."""
    g = torch.Generator(device="cuda").manual_seed(sum(lens))
    off = torch.tensor([0] + lens).cumsum(0)
    R = int(off[-1])
    x, d, h, du = (torch.randn(R, w, device="cuda", generator=g).to(BF16) for w in (160, 160, 96, 96))
    w = moe.experts_weight_grad(x, d, {"h": h}, {"du": du}, {"offsets": off.to(torch.int32).cuda()})
    for name, left, right in (("w_up", du, x), ("w_down", d, h)):
        for e in range(len(lens)):
            a, b = (t[off[e]:off[e + 1]].double() for t in (left, right))
            bound = (44 * STEP + 2 * U) * (a.abs().t() @ b.abs())
            assert bool(((w[name][e].double() - a.t() @ b).abs() <= bound).all()), (name, e)


@pytest.mark.parametrize("H,I", [(96, 160), (256, 512)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_chains(moe, H, I, accumulate):
    """Segments at the edges of one, two and more chains: eleven blocks of 64 rows are one chain, twelve are two."""
    lens = [704, 705, 703, 64, 1216, 1217, 0, 2049, 5000]
    g = torch.Generator(device="cuda").manual_seed(H)
    off = torch.tensor([0] + lens).cumsum(0)
    R = int(off[-1])
    x, d, h, dg, du = (torch.randn(R, w, device="cuda", generator=g).to(BF16) for w in (H, H, I, I, I))
    before = {k: torch.randn(len(lens), *s, device="cuda", generator=g) for k, s in (("w_gate", (I, H)), ("w_up", (I, H)), ("w_down", (H, I)))}
    out = {k: v.clone() for k, v in before.items()}
    w = moe.experts_weight_grad(x, d, {"h": h}, {"dg": dg, "du": du}, {"offsets": off.to(torch.int32).cuda()}, accumulate=accumulate, out=out)
    for name, left, right in (("w_gate", dg, x), ("w_up", du, x), ("w_down", d, h)):
        for e, rows in enumerate(lens):
            a, b = (t[off[e]:off[e + 1]].double() for t in (left, right))
            old = before[name][e].double() if accumulate else torch.zeros((), dtype=torch.float64, device="cuda")
            chains = (((rows + 63) // 64) + 4) // 8
            size = a.abs().t() @ b.abs()
            bound = (44 * STEP + (chains + 1) * U) * size + U * old.abs()
            assert bool(((w[name][e].double() - a.t() @ b - old).abs() <= bound).all()), (name, e)


def test_tensors_that_fill_their_memory(moe):
    """Every tensor is a whole number of the allocator's 2 MB blocks, so that it begins and ends with them: segments of a few
    rows at its beginning and its end, tiles that are mostly zeros, all three passes."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    R, H, I, lens = 8192, 1024, 1024, [3, 130, 0, 1, 700, 5000, 2351, 5, 2]
    assert sum(lens) == R
    E = len(lens)
    g = torch.Generator(device="cuda").manual_seed(31)
    n = lambda *s, scale=1.0: (torch.randn(*s, device="cuda", generator=g, dtype=BF16) * scale)  # noqa: E731
    x, dout = n(R, H), n(R, H, scale=0.1)
    wg, wu, wd = n(E, I, H, scale=0.03), n(E, I, H, scale=0.03), n(E, H, I, scale=0.03)
    off = torch.tensor([0] + lens).cumsum(0)
    plan = {"offsets": off.to(torch.int32).cuda()}
    ws = moe.experts_workspace(R, I)
    torch.cuda.empty_cache()
    o = moe.experts_forward(x, plan, wg, wu, wd, keep=True, workspace=ws)
    b = moe.experts_backward(dout, o, plan, wg, wu, wd, workspace=ws)
    w = moe.experts_weight_grad(x, dout, o, b, plan, workspace=ws)
    assert moe.last_device_status(ws) == 0
    half = 2.0 ** -8
    for e, rows in enumerate(lens):
        r = slice(int(off[e]), int(off[e + 1]))
        for got, left, right in ((o["u"], x, wu[e].t()), (o["g"], x, wg[e].t()), (o["out"], o["h"], wd[e].t())):
            want, size = left[r].double() @ right.double(), left[r].double().abs() @ right.double().abs()
            assert bool(((got[r].double() - want).abs() <= half * want.abs() + (1024 / 16 + 4) * STEP * size * (1 + half)).all()), e
        dx = b["dg"][r].double() @ wg[e].double() + b["du"][r].double() @ wu[e].double()
        size = b["dg"][r].double().abs() @ wg[e].double().abs() + b["du"][r].double().abs() @ wu[e].double().abs()
        assert bool(((b["drows"][r].double() - dx).abs() <= half * dx.abs() + (2048 / 16 + 4) * STEP * size * (1 + half)).all()), e
        for name, left, right in (("w_gate", b["dg"], x), ("w_up", b["du"], x), ("w_down", dout, o["h"])):
            want, size = left[r].double().t() @ right[r].double(), left[r].double().abs().t() @ right[r].double().abs()
            assert bool(((w[name][e].double() - want).abs() <= (44 * STEP + (rows / 512 + 2) * U) * size).all()), (name, e)
