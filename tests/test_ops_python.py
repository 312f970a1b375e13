"""The Python functions of the operators around the layer take their arguments by the names that
their signatures and documentation give."""
import inspect

import pytest
import torch

OPS = {"add_rmsnorm_quantize_mx": ("x", "residual", "gamma"), "add_rmsnorm_backward": ("dy", "h", "rrms", "gamma"),
       "router_loss": ("logits", "topk_ids"), "router_loss_backward": ("logits", "topk_ids", "stats"),
       "linear_w4": ("x", "codes", "sf")}


@pytest.fixture(scope="module")
def moe():
    from nvfp4_mixture_experts_softmax_gb300 import _build
    _build.build()
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("name", OPS)
def test_signatures(moe, name):
    params = inspect.signature(getattr(moe, name)).parameters
    required = [n for n, p in params.items() if p.default is p.empty]
    assert tuple(required) == OPS[name]
    assert params["stream"].kind is inspect.Parameter.KEYWORD_ONLY and params["stream"].default is None


@pytest.mark.parametrize("name", OPS)
def test_by_name_without_a_device(moe, name):
    """A call by name gets as far as the check of the device; without the first tensor it says so."""
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        getattr(moe, name)(**{n: x for n in OPS[name]})
    with pytest.raises(ValueError, match="required"):
        getattr(moe, name)(**{n: x for n in OPS[name][1:]})


@pytest.mark.gpu
def test_by_name(moe):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, res, gamma, side = n(5, 64).bfloat16(), n(5, 64).bfloat16(), n(64).bfloat16(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = moe.add_rmsnorm_quantize_mx(x, res, gamma, want_rrms=True)
    b = moe.add_rmsnorm_quantize_mx(gamma=gamma, residual=res, x=x, want_rrms=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a[k], b[k]) for k in a)
    a2 = moe.add_rmsnorm_backward(x, a["h"], a["rrms"], gamma)
    b2 = moe.add_rmsnorm_backward(dy=x, h=a["h"], rrms=a["rrms"], gamma=gamma)
    assert all(torch.equal(a2[k], b2[k]) for k in a2)
    lg, ids = n(5, 8), torch.arange(10, device="cuda", dtype=torch.int32).reshape(5, 2) % 8
    sa, sb = moe.router_loss(lg, ids), moe.router_loss(logits=lg, topk_ids=ids)
    assert all(torch.equal(sa[k], sb[k]) for k in sa)
    gl = torch.ones(2, device="cuda")
    assert torch.equal(moe.router_loss_backward(lg, ids, sa, gl), moe.router_loss_backward(logits=lg, topk_ids=ids, stats=sa, grad_losses=gl))
    w = moe.quantize_act(n(48, 64).bfloat16())
    assert torch.equal(moe.linear_w4(x, *w), moe.linear_w4(x=x, codes=w[0], sf=w[1], ts=w[2]))


def test_backward_over_h_is_refused(moe):
    """dx may take the place of dy or dh; h is still read after the first rows of dx are written."""
    P = 4096   # an address that no rejected call reads
    call = moe.lib().moe_add_rmsnorm_backward
    assert call(P, None, 2 * P, P, P, 4, 64, 2 * P, P, P, 1 << 24, None) == -1
