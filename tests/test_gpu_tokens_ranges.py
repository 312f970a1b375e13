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
