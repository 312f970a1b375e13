"""Argument checks of the operators around the layer: rejected on the host, before any device work,
with or without a GPU."""
import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    from nvfp4_mixture_experts_softmax_gb300 import _build
    _build.build()
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


P = 4096   # a non-null, aligned address that no rejected call reads


def norm(moe, x=P, res=P, gamma=P, eps=1e-6, rows=4, cols=64, h=P, codes=P, sf=P, y=None, rrms=None):
    return moe.lib().moe_add_rmsnorm_quantize_mx(x, res, gamma, eps, rows, cols, h, codes, sf, y, rrms, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), 0), (dict(rows=0, x=None, gamma=None), 0), (dict(rows=-1), -1), (dict(cols=0), -1), (dict(cols=48), -1),
    (dict(cols=16416), -2), (dict(rows=1 << 31), -2), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(eps=float("inf")), -1), (dict(x=None), -1), (dict(gamma=None), -1), (dict(h=None), -1), (dict(res=None), -1),
    (dict(codes=None), -1), (dict(sf=None), -1), (dict(codes=None, sf=None), -1), (dict(x=P + 8), -1), (dict(res=P + 2), -1),
    (dict(h=P + 8), -1), (dict(y=P + 8), -1), (dict(codes=P + 4), -1), (dict(gamma=P + 2), -1), (dict(rrms=P + 2), -1)])
def test_norm_rejections(moe, kw, want):
    assert norm(moe, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), -1), (dict(cols=40), -1), (dict(cols=16416), -2), (dict(ws=None), -3), (dict(n=100), -3), (dict(ws=P + 8), -1),
    (dict(dy=None), -1), (dict(h=None), -1), (dict(rrms=None), -1), (dict(gamma=None), -1), (dict(dx=None), -1),
    (dict(dgamma=None), -1), (dict(dh=P + 8), -1), (dict(dx=P + 8), -1), (dict(rrms=P + 1), -1), (dict(dgamma=P + 2), -1)])
def test_norm_backward_rejections(moe, kw, want):
    a = dict(dy=P, dh=None, h=P, rrms=P, gamma=P, rows=4, cols=64, dx=P, dgamma=P, ws=P, n=1 << 24)
    a.update(kw)
    assert moe.lib().moe_add_rmsnorm_backward(a["dy"], a["dh"], a["h"], a["rrms"], a["gamma"], a["rows"], a["cols"], a["dx"],
                                              a["dgamma"], a["ws"], a["n"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), -1), (dict(E=0), -1), (dict(k=0), -1), (dict(k=9), -1), (dict(E=1025, k=8), -2), (dict(E=64, k=33), -2),
    (dict(T=1 << 30, k=2), -2), (dict(flags=2), -1), (dict(losses=None), -1), (dict(counts=None), -1), (dict(tokens=None), -1), (dict(probs=None), -1),
    (dict(ws=None), -3), (dict(n=64), -3), (dict(ws=P + 16), -1), (dict(logits=None), -1), (dict(ids=None), -1),
    (dict(logits=P + 2), -1), (dict(ids=P + 2), -1), (dict(losses=P + 1), -1)])
def test_loss_rejections(moe, kw, want):
    a = dict(logits=P, ids=P, mask=None, T=4, E=8, k=2, flags=0, losses=P, counts=P, tokens=P, probs=P, ws=P, n=1 << 24)
    a.update(kw)
    assert moe.lib().moe_router_loss(a["logits"], a["ids"], a["mask"], a["T"], a["E"], a["k"], a["flags"], a["losses"],
                                     a["counts"], a["tokens"], a["probs"], a["ws"], a["n"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), 0), (dict(T=-1), -1), (dict(k=9), -1), (dict(E=1025), -2), (dict(T=1 << 30, k=2), -2), (dict(flags=4), -1),
    (dict(logits=None), -1),
    (dict(counts=None), -1), (dict(tokens=None), -1), (dict(dl=None), -1), (dict(ids=None, gw=P), -1), (dict(gw=P + 2), -1),
    (dict(gl=P + 1), -1), (dict(dl=P + 2), -1)])
def test_loss_backward_rejections(moe, kw, want):
    a = dict(logits=P, ids=P, T=4, E=8, k=2, flags=0, counts=P, tokens=P, gl=None, gw=None, dl=P)
    a.update(kw)
    assert moe.lib().moe_router_loss_backward(a["logits"], a["ids"], None, a["T"], a["E"], a["k"], a["flags"], a["counts"],
                                              a["tokens"], a["gl"], a["gw"], a["dl"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), 0), (dict(N=0), 0), (dict(T=-1), -1), (dict(N=-1), -1), (dict(K=0), -1), (dict(K=48), -2), (dict(T=65), -2),
    (dict(K=(1 << 20) + 32), -2), (dict(N=(1 << 30) + 1), -2), (dict(flags=4), -1), (dict(x=None), -1), (dict(codes=None), -1),
    (dict(sf=None), -1), (dict(y=None), -1), (dict(ts=None), -1), (dict(flags=1), -1), (dict(x=P + 8), -1), (dict(codes=P + 8), -1),
    (dict(sf=P + 1), -1), (dict(ts=P + 2), -1), (dict(y=P + 1), -1), (dict(flags=2, y=P + 2), -1)])
def test_linear_rejections(moe, kw, want):
    a = dict(x=P, codes=P, sf=P, ts=P, T=4, N=8, K=64, flags=0, y=P)
    a.update(kw)
    assert moe.lib().moe_linear_w4(a["x"], a["codes"], a["sf"], a["ts"], a["T"], a["N"], a["K"], a["flags"], a["y"], None) == want


def test_workspace_sizes(moe):
    L = moe.lib()
    assert L.moe_add_rmsnorm_backward_workspace_size(-1, 64) == 0
    assert L.moe_add_rmsnorm_backward_workspace_size(1, 64) >= 4 * 64
    assert L.moe_router_loss_workspace_size(-1, 8) == 0
    assert L.moe_router_loss_workspace_size(1000, 64) >= L.moe_router_loss_workspace_size(10, 64) >= 256


def test_python_checks_without_a_device(moe):
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    for call in (lambda: moe.add_rmsnorm_quantize_mx(x, x, x[0]), lambda: moe.add_rmsnorm_backward(x, x, x[:, 0].float(), x[0]),
                 lambda: moe.router_loss(x.float(), torch.zeros(2, 2, dtype=torch.int32)), lambda: moe.linear_w4(x, x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
