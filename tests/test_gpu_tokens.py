"""Tokens sorted by expert and back: the plan exactly, sums against 64 bits.

Bounds, u = 2^-24: a combined element is a chain of k fused additions (k + 1 roundings of at most the terms'
magnitudes), then half a step of its type (2^-8 relative in BF16); drows is one product rounded twice; dtopk_w a chain of
cols / 32 + 8 terms a lane and a 5-step tree."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def reference(ids, E, mask=None):
    """The plan by a stable sort on the host."""
    e = ids.cpu().long().reshape(-1)
    live = (e >= 0) & (e < E)
    if mask is not None:
        live &= mask.cpu().bool().repeat_interleave(ids.shape[1])
    a = live.nonzero().squeeze(1)
    a = a[torch.sort(e[a], stable=True).indices]
    counts = torch.bincount(e[a], minlength=E)
    perm, inv = torch.full((e.numel(),), -1), torch.full((e.numel(),), -1)
    perm[:a.numel()] = a // ids.shape[1]
    inv[a] = torch.arange(a.numel())
    want = {"counts": counts, "offsets": torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]), "perm_src": perm, "inv": inv}
    return {n: t.to(torch.int32) for n, t in want.items()}


def same(plan, want):
    return all(torch.equal(plan[n].cpu(), want[n]) for n in want)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (5, 3, 2), (64, 128, 8), (512, 1024, 8), (513, 7, 8), (4096, 1, 1), (4097, 1024, 1),
                                   (1000, 60, 32), (20000, 256, 8), (33333, 1021, 3)])
@pytest.mark.parametrize("masked", [False, True])
def test_sort(moe, T, E, k, masked):
    ids = torch.randint(0, E, (T, k), device="cuda", generator=gen(T + E), dtype=torch.int32)    # ids may repeat in a token
    mask = torch.rand(T, device="cuda", generator=gen(1)) < 0.7 if masked else None
    ws = moe.sort_tokens_workspace(T, E, k)
    plan = moe.sort_tokens(ids, E, mask=mask, workspace=ws)
    assert same(plan, reference(ids, E, mask)) and moe.last_device_status(ws) == 0
    if masked:
        assert same(moe.sort_tokens(ids, E, mask=mask.to(torch.uint8) * 3, workspace=ws), reference(ids, E, mask))


@pytest.mark.parametrize("T", [40, 3000])
def test_left_out_and_bad_ids(moe, T):
    ids = torch.randint(-1, 16, (T, 4), device="cuda", generator=gen(3), dtype=torch.int32)
    ws = moe.sort_tokens_workspace(T, 16, 4)
    assert same(moe.sort_tokens(ids, 16, workspace=ws), reference(ids, 16)) and moe.last_device_status(ws) == 0
    bad = ids.clone()
    bad[T // 2, 1], bad[T - 1, 3], bad[0, 0] = 16, -2 ** 31, 2 ** 31 - 1
    assert same(moe.sort_tokens(bad, 16, workspace=ws), reference(bad, 16)) and moe.last_device_status(ws) == -1
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[[T // 2, T - 1, 0]] = False                 # a masked token's ids are not read
    assert same(moe.sort_tokens(bad, 16, mask=mask, workspace=ws), reference(bad, 16, mask)) and moe.last_device_status(ws) == 0
    none = moe.sort_tokens(bad, 16, mask=mask & False, workspace=ws)
    assert not none["counts"].any() and not none["offsets"].any() and bool((none["inv"] == -1).all() and (none["perm_src"] == -1).all())


def test_sort_equals_the_router_plan(moe):
    for T, E, k in ((7, 16, 4), (900, 64, 8)):
        p = moe.plan(torch.randn(T, E, device="cuda", generator=gen(4)), k)
        s = moe.sort_tokens(p["topk_ids"], E)
        assert all(torch.equal(s[n], p[n]) for n in s)


def test_no_tokens(moe):
    plan = moe.sort_tokens(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 9)
    assert not plan["counts"].any() and not plan["offsets"].any() and plan["inv"].numel() == 0
    x = torch.empty(0, 64, device="cuda")
    assert moe.permute_tokens(x, plan).shape == (0, 64)
    assert moe.combine_tokens(x, plan, torch.empty(0, 4, device="cuda")).shape == (0, 64)
    assert moe.permute_tokens_backward(x, plan, 0).shape == (0, 64)
    b = moe.combine_tokens_backward(x, x, plan, torch.empty(0, 4, device="cuda"))
    assert b["drows"].shape == (0, 64) and b["dtopk_w"].shape == (0, 4)


CASES = [(1, 8, 1, 1), (1, 2048, 128, 8), (3, 72, 5, 5), (64, 7168, 256, 8), (700, 520, 64, 3), (33, 64, 40, 32), (9, 16392, 4, 2)]


def setup(moe, T, cols, E, k, dtype, mask=True):
    g = gen(T + cols)
    ids = torch.rand(T, E, device="cuda", generator=g).topk(k, -1).indices.to(torch.int32)
    plan = moe.sort_tokens(ids, E, mask=torch.rand(T, device="cuda", generator=g) < 0.8 if mask else None)
    x = torch.randn(T, cols, device="cuda", generator=g).to(dtype)
    rows = torch.randn(T * k, cols, device="cuda", generator=g).to(dtype)
    rows[int(plan["offsets"][-1]):] = float("nan")          # rows behind the last expert's are not read
    return plan, x, rows, torch.rand(T, k, device="cuda", generator=g)


def gathered(rows, plan, T, k):
    inv = plan["inv"].long().reshape(T, k)
    return torch.where((inv >= 0)[..., None], rows.double()[inv.clamp(min=0)], 0.0), inv


@pytest.mark.parametrize("T,cols,E,k", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_there_and_back(moe, T, cols, E, k, dtype):
    plan, x, rows, w = setup(moe, T, cols, E, k, dtype)
    n = int(plan["offsets"][-1])
    out = torch.full((T * k, cols), 7.0, device="cuda", dtype=dtype)
    got = moe.permute_tokens(x, plan, out=out)
    assert torch.equal(got[:n], x[plan["perm_src"][:n].long()]) and bool((got[n:] == 7).all())
    back = moe.permute_tokens_backward(rows, plan, T)
    y = moe.combine_tokens(rows, plan, w)
    r, inv = gathered(rows, plan, T, k)
    for have, terms in ((back, r), (y, r * w.double()[..., None])):
        want, size = terms.sum(1), terms.abs().sum(1)
        err = (have.double() - want).abs()
        assert bool((err <= (k + 1) * U * size + HALF[dtype] * (want.abs() + (k + 1) * U * size)).all())
    assert not y[(inv < 0).all(1)].any()
    out = {"drows": torch.full_like(rows, 7.0), "dtopk_w": torch.full_like(w, 7.0)}
    b = moe.combine_tokens_backward(x, rows, plan, w, out=out)
    keep = inv >= 0
    want = (w.double()[..., None] * x.double()[:, None, :])[keep]
    assert bool(((b["drows"][inv[keep]].double() - want).abs() <= (HALF[dtype] + 2 * U) * want.abs()).all())
    assert bool((b["drows"][n:] == 7).all())
    prod = r * x.double()[:, None, :]
    assert bool(((b["dtopk_w"].double() - prod.sum(-1)).abs() <= (cols / 32 + 16) * U * prod.abs().sum(-1)).all())
    own = rows.clone()
    b2 = moe.combine_tokens_backward(x, own, plan, w, out={"drows": own, "dtopk_w": torch.empty_like(w)})
    assert torch.equal(b2["drows"][:n], b["drows"][:n]) and torch.equal(b2["dtopk_w"], b["dtopk_w"])


@pytest.mark.parametrize("dtype,cols", [(torch.uint8, 48), (torch.float16, 40), (torch.float32, 4), (torch.float64, 6)])
def test_permute_any_type(moe, dtype, cols):
    ids = torch.randint(0, 6, (50, 3), device="cuda", generator=gen(6), dtype=torch.int32)
    plan = moe.sort_tokens(ids, 6)
    x = torch.randint(0, 200, (50, cols), device="cuda", generator=gen(7)).to(dtype)
    assert torch.equal(moe.permute_tokens(x, plan), x[plan["perm_src"].long()])


def test_nonfinite_weights_and_rows(moe):
    """What stands in dropped assignments is not read; NaN and infinities stay in their token."""
    T, E, k = 20, 8, 2
    ids = torch.stack([torch.arange(T, device="cuda") % E, (torch.arange(T, device="cuda") + 1) % E], 1).to(torch.int32)
    ids[3] = -1
    ids[5, 1] = -1
    plan = moe.sort_tokens(ids, E)
    rows, w = torch.randn(T * k, 64, device="cuda", generator=gen(8)), torch.rand(T, k, device="cuda", generator=gen(9))
    want = moe.combine_tokens(rows, plan, w)
    w2, rows2 = w.clone(), rows.clone()
    w2[3], w2[5, 1] = float("nan"), float("inf")
    rows2[plan["inv"][2 * 7].item(), 3] = float("inf")
    got = moe.combine_tokens(rows2, plan, w2)
    same_rows = [t for t in range(T) if t != 7]
    assert torch.equal(got[same_rows], want[same_rows]) and not got[3].any()
    assert bool(got[7, 3].isinf()) and torch.equal(got[7, 4:], want[7, 4:])


def test_inverse_out_of_range(moe):
    """A plan of more rows than there are (a truncated buffer): entries outside stand for no row."""
    plan, x, rows, w = setup(moe, 60, 128, 8, 2, torch.float32, mask=False)
    short = rows[:100]
    r, inv = gathered(rows, plan, 60, 2)
    keep = inv < 100
    want = (r * (w.double() * keep)[..., None]).sum(1)
    assert bool(((moe.combine_tokens(short, plan, w).double() - want).abs() <= 4 * U * (r * w.double()[..., None]).abs().sum(1)).all())
    out = moe.permute_tokens(x, plan, out=torch.zeros(100, 128, device="cuda"))
    assert torch.equal(out, x[plan["perm_src"][:100].long()])
    b = moe.combine_tokens_backward(x, short, plan, w)
    assert not b["dtopk_w"][~keep].any() and bool(b["dtopk_w"][keep].any())


def test_gradients_against_differences(moe):
    """FP32: sum(c * combine(rows, w)) is linear in each argument: a central difference is its derivative but for the
    outputs' rounding, (k + 2) u of the terms over the step."""
    T, k, cols = 50, 3, 72
    plan, x, rows, w = setup(moe, T, cols, 16, k, torch.float32, mask=False)
    c, dr, dw = x, torch.randn(T * k, cols, device="cuda", generator=gen(11)), torch.randn(T, k, device="cuda", generator=gen(12))
    b = moe.combine_tokens_backward(c, rows, plan, w)
    f = lambda r, v: (moe.combine_tokens(r, plan, v).double() * c).sum()  # noqa: E731
    size = float((gathered(rows.abs() + dr.abs(), plan, T, k)[0] * (w + dw.abs()).double()[..., None] * c.double().abs()[:, None]).sum())
    for got, lo, hi in (((b["drows"].double() * dr).sum(), (rows - dr, w), (rows + dr, w)), ((b["dtopk_w"].double() * dw).sum(), (rows, w - dw), (rows, w + dw))):
        assert abs(float(got - (f(*hi) - f(*lo)) / 2)) <= 8 * U * size
    back = moe.permute_tokens_backward(dr, plan, T)
    assert abs(float((back.double() * x).sum() - (moe.permute_tokens(x, plan).double() * dr).sum())) <= 8 * U * float((x.abs().sum() * 8 * k))


def test_refusals(moe):
    plan, x, rows, w = setup(moe, 8, 64, 4, 2, torch.bfloat16)
    ids = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    for call in (lambda: moe.sort_tokens(ids.long(), 4), lambda: moe.sort_tokens(ids[:, :1].expand(8, 2), 4),
                 lambda: moe.sort_tokens(ids, 4, mask=torch.ones(7, dtype=torch.bool, device="cuda")),
                 lambda: moe.permute_tokens(x[:, ::2], plan), lambda: moe.permute_tokens(x[:3].contiguous(), plan),
                 lambda: moe.combine_tokens(rows.half(), plan, w), lambda: moe.combine_tokens(rows, plan, w[:, :1].contiguous()),
                 lambda: moe.combine_tokens(rows, plan, w.bfloat16()), lambda: moe.combine_tokens_backward(x.float(), rows, plan, w),
                 lambda: moe.combine_tokens(rows[:, :60].contiguous(), plan, w)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        moe.permute_tokens(x[:, :4].contiguous(), plan)             # rows of 8 bytes
    with pytest.raises(RuntimeError, match="SHAPE"):
        moe.sort_tokens(ids, 1025)


def test_graph_and_streams(moe):
    plan, x, rows, w = setup(moe, 900, 256, 16, 8, torch.bfloat16, mask=False)
    ids = torch.randint(0, 16, (900, 8), device="cuda", generator=gen(13), dtype=torch.int32)
    ws = [moe.sort_tokens_workspace(900, 16, 8) for _ in range(2)]

    def step(i, stream=None):
        p = moe.sort_tokens(ids, 16, workspace=ws[i], stream=stream)
        r = moe.permute_tokens(x, p, stream=stream)
        return p, r, moe.combine_tokens(r, p, w, stream=stream), moe.combine_tokens_backward(x, r, p, w, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both = [step(0), step(1, side)]
    torch.cuda.synchronize()
    assert torch.equal(both[0][2], both[1][2]) and torch.equal(both[0][3]["drows"], both[1][3]["drows"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pg, rg, yg, bg = step(0)
    ids.copy_(torch.randint(0, 16, (900, 8), device="cuda", generator=gen(14), dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    p, r, y, b = step(1)
    assert all(torch.equal(pg[n], p[n]) for n in p) and torch.equal(yg, y) and torch.equal(bg["dtopk_w"], b["dtopk_w"])
