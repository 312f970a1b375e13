"""Argument checks of the training pass's operators (layer norm, tokens to their experts and back, the
experts): rejected on the host, before any device work, with or without a GPU; and their Python signatures."""
import inspect

import pytest
import torch

OPS = {"add_layernorm": ("x", "residual", "gamma"), "add_layernorm_backward": ("dy", "h", "mean", "rstd", "gamma"),
       "sort_tokens": ("topk_ids", "num_experts"), "permute_tokens": ("x", "plan"),
       "permute_tokens_backward": ("drows", "plan", "num_tokens"), "combine_tokens": ("rows", "plan", "topk_w"),
       "combine_tokens_backward": ("dy", "rows", "plan", "topk_w"),
       "experts_forward": ("rows", "plan", "w_gate", "w_up", "w_down"),
       "experts_backward": ("dout", "saved", "plan", "w_gate", "w_up", "w_down"),
       "experts_weight_grad": ("rows", "dout", "saved", "grads", "plan")}


@pytest.fixture(scope="module")
def moe():
    from nvfp4_mixture_experts_softmax_gb300 import _build
    _build.build()
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


P = 4096   # a non-null, aligned address that no rejected call reads


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), 0), (dict(rows=-1), -1), (dict(cols=0), -1), (dict(cols=20), -1), (dict(cols=16392), -2), (dict(rows=1 << 31), -2),
    (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(flags=2), -1), (dict(x=None), -1),
    (dict(gamma=None), -1), (dict(y=None), -1), (dict(h=None), -1), (dict(res=None), -1), (dict(x=P + 8), -1), (dict(res=P + 8), -1),
    (dict(beta=P + 4), -1), (dict(y=P + 8), -1), (dict(mean=P + 2), -1), (dict(rstd=P + 1), -1)])
def test_layernorm(moe, kw, want):
    a = dict(x=P, res=P, gamma=P, beta=None, eps=1e-5, rows=4, cols=64, flags=0, h=P, y=P, mean=None, rstd=None)
    a.update(kw)
    assert moe.lib().moe_add_layernorm(a["x"], a["res"], a["gamma"], a["beta"], a["eps"], a["rows"], a["cols"], a["flags"], a["h"], a["y"],
                                       a["mean"], a["rstd"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), -1), (dict(cols=12), -1), (dict(cols=16392), -2), (dict(flags=4), -1), (dict(ws=None), -3), (dict(n=100), -3),
    (dict(ws=P + 8), -1), (dict(dy=None), -1), (dict(h=None), -1), (dict(mean=None), -1), (dict(rstd=None), -1), (dict(gamma=None), -1),
    (dict(dx=None), -1), (dict(dgamma=None), -1), (dict(dh=P + 8), -1), (dict(dx=P + 8), -1), (dict(dbeta=P + 2), -1),
    (dict(h=P, dx=P), -1)])
def test_layernorm_backward(moe, kw, want):
    a = dict(dy=P, dh=None, h=2 * P, mean=P, rstd=P, gamma=P, rows=4, cols=64, flags=0, dx=P, dgamma=P, dbeta=P, ws=P, n=1 << 24)
    a.update(kw)
    assert moe.lib().moe_add_layernorm_backward(a["dy"], a["dh"], a["h"], a["mean"], a["rstd"], a["gamma"], a["rows"], a["cols"], a["flags"],
                                                a["dx"], a["dgamma"], a["dbeta"], a["ws"], a["n"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), -1), (dict(E=0), -1), (dict(k=0), -1), (dict(E=1025), -2), (dict(k=33), -2), (dict(T=1 << 30, k=2), -2), (dict(ws=None), -3),
    (dict(n=64), -3), (dict(ws=P + 16), -1), (dict(ids=None), -1), (dict(counts=None), -1), (dict(offsets=None), -1), (dict(perm=None), -1),
    (dict(inv=None), -1), (dict(ids=P + 2), -1), (dict(inv=P + 1), -1)])
def test_sort(moe, kw, want):
    a = dict(ids=P, T=4, E=8, k=2, counts=P, offsets=P, perm=P, inv=P, ws=P, n=1 << 24)
    a.update(kw)
    assert moe.lib().moe_sort_tokens(a["ids"], None, a["T"], a["E"], a["k"], a["counts"], a["offsets"], a["perm"], a["inv"], a["ws"], a["n"],
                                     None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), 0), (dict(R=0), 0), (dict(T=-1), -1), (dict(k=0), -1), (dict(k=33), -2), (dict(T=1 << 30, k=2), -2), (dict(rb=24), -1),
    (dict(rb=0), -1), (dict(rb=(1 << 20) + 16), -2), (dict(R=-1), -1), (dict(R=1 << 31), -2), (dict(x=None), -1), (dict(inv=None), -1),
    (dict(rows=None), -1), (dict(x=P + 8), -1), (dict(rows=P + 8), -1), (dict(inv=P + 2), -1)])
def test_permute(moe, kw, want):
    a = dict(x=P, inv=P, T=4, k=2, rb=64, R=8, rows=2 * P)
    a.update(kw)
    assert moe.lib().moe_permute_rows(a["x"], a["inv"], a["T"], a["k"], a["rb"], a["R"], a["rows"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), 0), (dict(T=-1), -1), (dict(k=0), -1), (dict(k=33), -2), (dict(cols=0), -1), (dict(cols=12), -1), (dict(cols=-8), -1),
    (dict(cols=1 << 40), -2), (dict(flags=2), -1), (dict(flags=1, cols=6), -1), (dict(R=-1), -1), (dict(rows=None), -1), (dict(inv=None), -1),
    (dict(y=None), -1), (dict(rows=P + 8), -1), (dict(y=P + 8), -1), (dict(w=P + 2), -1)])
def test_combine(moe, kw, want):
    a = dict(rows=P, inv=P, w=P, T=4, k=2, cols=64, R=8, flags=0, y=2 * P)
    a.update(kw)
    assert moe.lib().moe_combine_rows(a["rows"], a["inv"], a["w"], a["T"], a["k"], a["cols"], a["R"], a["flags"], a["y"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), 0), (dict(T=-1), -1), (dict(k=33), -2), (dict(cols=12), -1), (dict(flags=2), -1), (dict(R=-1), -1), (dict(dy=None), -1),
    (dict(rows=None), -1), (dict(inv=None), -1), (dict(w=None), -1), (dict(drows=None), -1), (dict(dw=None), -1), (dict(dy=P + 8), -1),
    (dict(drows=P + 8), -1), (dict(dw=P + 2), -1)])
def test_combine_backward(moe, kw, want):
    a = dict(dy=P, rows=P, inv=P, w=P, T=4, k=2, cols=64, R=8, flags=0, drows=P, dw=P)
    a.update(kw)
    assert moe.lib().moe_combine_rows_backward(a["dy"], a["rows"], a["inv"], a["w"], a["T"], a["k"], a["cols"], a["R"], a["flags"],
                                               a["drows"], a["dw"], None) == want


SHAPES = [(dict(R=-1), -1), (dict(E=0), -1), (dict(E=1025), -2), (dict(H=48), -1), (dict(I=0), -1), (dict(H=65568), -2), (dict(R=1 << 31), -2),
          (dict(ws=None), -3), (dict(n=128), -3), (dict(ws=P + 16), -1), (dict(off=None), -1), (dict(off=P + 2), -1)]
ACTS = [(dict(flags=1), -1), (dict(flags=2 | 4), -1), (dict(flags=16), -1), (dict(flags=2, L=-1.0), -1), (dict(flags=2, L=float("nan")), -1),
        (dict(flags=8, L=7.0, alpha=float("inf")), -1)]


@pytest.mark.parametrize("kw,want", SHAPES + ACTS + [
    (dict(x=None), -1), (dict(wg=None), -1), (dict(wu=None), -1), (dict(wd=None), -1), (dict(out=None), -1), (dict(g=None), -1),
    (dict(u=None), -1), (dict(h=None, n=300), -3), (dict(flags=4), -1), (dict(x=P + 8), -1), (dict(wd=P + 8), -1), (dict(out=P + 16), -1),
    (dict(h=P + 16), -1), (dict(g=P + 16), -1)])
def test_experts_forward(moe, kw, want):
    a = dict(x=P, off=P, R=8, E=4, H=64, I=64, wg=P, wu=P, wd=P, flags=0, L=0.0, alpha=0.0, g=P, u=P, h=P, out=P, ws=P, n=1 << 20)
    a.update(kw)
    assert moe.lib().moe_experts_forward(a["x"], a["off"], a["R"], a["E"], a["H"], a["I"], a["wg"], a["wu"], a["wd"], a["flags"], a["L"],
                                         a["alpha"], a["g"], a["u"], a["h"], a["out"], a["ws"], a["n"], None) == want


@pytest.mark.parametrize("kw,want", SHAPES + ACTS + [
    (dict(d=None), -1), (dict(wg=None), -1), (dict(wu=None), -1), (dict(wd=None), -1), (dict(g=None), -1), (dict(u=None), -1),
    (dict(dg=None), -1), (dict(du=None), -1), (dict(dx=None), -1), (dict(flags=4), -1), (dict(d=P + 8), -1), (dict(dx=P + 16), -1)])
def test_experts_backward(moe, kw, want):
    a = dict(d=P, off=P, R=8, E=4, H=64, I=64, wg=P, wu=P, wd=P, flags=0, L=0.0, alpha=0.0, g=P, u=P, dg=P, du=P, dx=P, ws=P, n=1 << 20)
    a.update(kw)
    assert moe.lib().moe_experts_backward(a["d"], a["off"], a["R"], a["E"], a["H"], a["I"], a["wg"], a["wu"], a["wd"], a["flags"], a["L"],
                                          a["alpha"], a["g"], a["u"], a["dg"], a["du"], a["dx"], a["ws"], a["n"], None) == want


@pytest.mark.parametrize("kw,want", SHAPES + [
    (dict(flags=1), -1), (dict(flags=512), -1), (dict(x=None), -1), (dict(d=None), -1), (dict(h=None), -1), (dict(dg=None), -1),
    (dict(du=None), -1), (dict(wg=None), -1), (dict(wu=None), -1), (dict(wd=None), -1), (dict(flags=4), -1), (dict(flags=4, wg=None), -1),
    (dict(x=P + 8), -1), (dict(wd=P + 16), -1)])
def test_experts_weight_grad(moe, kw, want):
    a = dict(x=P, d=P, h=P, dg=P, du=P, off=P, R=8, E=4, H=64, I=64, flags=0, wg=P, wu=P, wd=P, ws=P, n=1 << 20)
    a.update(kw)
    assert moe.lib().moe_experts_weight_grad(a["x"], a["d"], a["h"], a["dg"], a["du"], a["off"], a["R"], a["E"], a["H"], a["I"], a["flags"],
                                             a["wg"], a["wu"], a["wd"], a["ws"], a["n"], None) == want


def test_workspace_sizes(moe):
    L = moe.lib()
    assert L.moe_experts_workspace_size(-1, 64) == 0 and L.moe_experts_workspace_size(0, 64) == 256
    assert L.moe_experts_workspace_size(1 << 20, 4096) == 256 + (1 << 33)        # beyond 32 bits
    assert L.moe_sort_tokens_workspace_size(4, 2000, 2) == 0 and L.moe_add_layernorm_backward_workspace_size(4, 20000) == 0


@pytest.mark.parametrize("name", OPS)
def test_signatures(moe, name):
    params = inspect.signature(getattr(moe, name)).parameters
    assert tuple(n for n, p in params.items() if p.default is p.empty) == OPS[name]
    assert params["stream"].kind is inspect.Parameter.KEYWORD_ONLY and params["stream"].default is None


@pytest.mark.parametrize("name", OPS)
def test_by_name_without_a_device(moe, name):
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        getattr(moe, name)(**{n: x for n in OPS[name]})
    with pytest.raises(ValueError, match="required"):
        getattr(moe, name)(**{n: x for n in OPS[name][1:]})


def test_in_place_moves_are_refused(moe):
    """Rows cannot be laid out, or summed, into the buffer that they are read from."""
    L = moe.lib()
    assert L.moe_permute_rows(P, P, 4, 2, 64, 8, P, None) == -1
    assert L.moe_combine_rows(P, P, P, 4, 2, 64, 8, 0, P, None) == -1
