"""Tokens that the mask takes out of the router losses: nothing of them reaches the results, whatever
stands in their logits, ids and weight gradients, in every lane layout and in the rounds that read
ahead.  (Their memory is not read either: the loads depend on the mask, a round ahead.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


# experts: the six lane layouts, with and without 16-byte loads; tokens: one round, several rounds a
# warp in both kernels
@pytest.mark.parametrize("E,k", [(31, 3), (32, 32), (60, 4), (127, 5), (256, 8), (510, 9), (1000, 32)])
@pytest.mark.parametrize("T", [7, 60000])
@pytest.mark.parametrize("router", ["softmax", "sqrtsoftplus"])
def test_masked_tokens_have_no_part(moe, T, E, k, router):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    l = torch.randn(T, E, device="cuda", generator=g) * 2
    ids = torch.randint(0, E, (T, k), device="cuda", generator=g, dtype=torch.int32)
    gw = torch.randn(T, k, device="cuda", generator=g)
    mask = torch.rand(T, device="cuda", generator=g) < 0.5
    mask[0], mask[-1] = True, False
    gl = torch.tensor([0.7, -0.3], device="cuda")

    def both(l, ids, gw):
        ws = moe.router_loss_workspace(T, E)
        o = moe.router_loss(l, ids, mask=mask, router=router, workspace=ws)
        assert moe.last_device_status(ws) == 0
        return o, moe.router_loss_backward(l, ids, o, gl, grad_topk_w=gw, mask=mask, router=router)

    o, d = both(l, ids, gw)
    assert not d[~mask].any() and bool(d.isfinite().all())
    kept = ids[mask].long().reshape(-1)
    assert torch.equal(o["counts"].long(), torch.bincount(kept, minlength=E)) and int(o["tokens"]) == int(mask.sum())
    for bad in (float("nan"), float("inf"), -float("inf")):
        l2, ids2, gw2 = l.clone(), ids.clone(), gw.clone()
        l2[~mask], ids2[~mask], gw2[~mask] = bad, 0x7FFFFFFF if bad > 0 else -0x80000000, bad
        o2, d2 = both(l2, ids2, gw2)
        assert all(torch.equal(o2[x], o[x]) for x in o) and torch.equal(d2, d)
        ids2[~mask] = ids[~mask]
        assert torch.equal(both(l2, ids2, gw2)[1], d)
