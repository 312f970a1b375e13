"""Tokens to their experts and back at the ends of the range: as many tokens as the calls take, rows that are read and
written in the same place."""
import pytest
import torch

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


def test_most_tokens(moe):
    """2^31 - 1 tokens of 16 bytes with one expert each, three of which have a row."""
    if torch.cuda.mem_get_info()[0] < 60 * 2 ** 30:
        pytest.skip("needs 60 GB of device memory")
    T = 2 ** 31 - 1
    at = torch.tensor([0, 2 ** 30 + 1, T - 1], device="cuda")
    inv = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    inv[at] = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    plan = {"inv": inv}
    x = torch.empty(T, 16, dtype=torch.uint8, device="cuda")
    x[at] = torch.arange(48, dtype=torch.uint8, device="cuda").reshape(3, 16)
    rows = moe.permute_tokens(x, plan, out=torch.zeros(3, 16, dtype=torch.uint8, device="cuda"))
    assert torch.equal(rows, x[at[[1, 2, 0]]])
    del x
    torch.cuda.empty_cache()
    r = torch.arange(1.0, 25.0, device="cuda").reshape(3, 8).bfloat16()
    y = moe.permute_tokens_backward(r, plan, T)
    assert torch.equal(y[at], r[[2, 0, 1]])
    y[at] = 0
    for i in range(0, T, 2 ** 28):
        assert not y[i:i + 2 ** 28].view(torch.int32).any()
    del y, inv, plan
    torch.cuda.empty_cache()


def test_sort_of_most_tokens(moe):
    """2^31 - 1 tokens, the experts 0, 1 and 2 in turn: the ranks past 2^31 / 1024 chunks."""
    if torch.cuda.mem_get_info()[0] < 80 * 2 ** 30:
        pytest.skip("needs 80 GB of device memory")
    T = 2 ** 31 - 1                                   # 3 * 715827882 + 1
    ids = torch.empty(T, 1, dtype=torch.int32, device="cuda")
    for i in range(0, T, 2 ** 28):
        n = min(2 ** 28, T - i)
        ids[i:i + n, 0] = torch.arange(i, i + n, device="cuda") % 3
    plan = moe.sort_tokens(ids, 3)
    each = T // 3
    assert plan["counts"].tolist() == [each + 1, each, each] and plan["offsets"].tolist() == [0, each + 1, 2 * each + 1, T]
    a = torch.tensor([0, 1, 2, 1023, 1024, 2 ** 30 + 7, T - 3, T - 2, T - 1], device="cuda")
    p = plan["inv"][a].long()
    assert torch.equal(p, plan["offsets"].long()[a % 3] + a // 3) and torch.equal(plan["perm_src"][p].long(), a)
    del ids, plan
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,cols,k", [(1, 8, 1), (3000, 1032, 1), (2500, 4096, 4), (700, 16392, 2)])
def test_gradients_over_the_rows(moe, dtype, T, cols, k):
    """drows in the buffer of rows: the bits of a call with a buffer of its own, at sizes with many rows an SM."""
    g = torch.Generator(device="cuda").manual_seed(T + cols)
    ids = torch.rand(T, 16, device="cuda", generator=g).topk(k, -1).indices.to(torch.int32)
    plan = moe.sort_tokens(ids, 16, mask=torch.arange(T, device="cuda") % 7 != 3)
    n = int(plan["offsets"][-1])
    dy, rows = (torch.randn(r, cols, device="cuda", generator=g).to(dtype) for r in (T, T * k))
    rows[n:] = float("nan")
    w = torch.rand(T, k, device="cuda", generator=g)
    want = moe.combine_tokens_backward(dy, rows, plan, w)
    for _ in range(3):
        own = rows.clone()
        got = moe.combine_tokens_backward(dy, own, plan, w, out={"drows": own, "dtopk_w": torch.empty_like(w)})
        assert torch.equal(got["drows"][:n], want["drows"][:n]) and torch.equal(got["dtopk_w"], want["dtopk_w"])
        assert bool(own[n:].isnan().all())
    inv = plan["inv"].long().reshape(T, k)
    keep = inv >= 0
    exact = (w.double()[..., None] * dy.double()[:, None])[keep]
    assert bool(((got["drows"][inv[keep]].double() - exact).abs() <= (HALF[dtype] + 2.0 ** -23) * exact.abs()).all())
