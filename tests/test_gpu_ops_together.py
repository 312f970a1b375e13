"""The operators around the layer run as they are used.

Decode: 4-bit output projection -> residual addition + RMSNorm + MXFP8 -> FP32 router logits ->
W4A8 layer on the codes (moe_run_quantized) -> expert load of the batch.  Training: norm -> logits
-> plan -> losses -> gradients back to the residual stream.

The W4A8 layer on MXFP8 input equals the layer on the decoded BF16 values: those quantise to the
same values again (the largest element of a block keeps its power of two, every element is
representable), so only the order of the FP32 reduction of the output may differ: relative L2
2^-9 + 1e-4, a BF16 rounding apart."""
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_mixture_experts_softmax_gb300 as m
    m.lib()
    return m


def mx_decode(codes, sf):
    s = torch.exp2(sf.double() - 127).repeat_interleave(32, 1)
    return (codes.view(torch.float8_e4m3fn).double() * s).bfloat16()


def layer(moe, cs, T, shared=0):
    wg, wu, wd = synth.gen_all_experts(cs, device="cuda")
    cfg = moe.make_config(cs.experts, cs.hidden, cs.inter, cs.top_k, shared_inter=shared, max_tokens=T, precision="w4a8")
    return cfg, moe.quantize_weights(cfg, wg, wu, wd, shared=synth.gen_shared(cs, device="cuda") if shared else None)


def close(a, b):
    a, b = a.double(), b.double()
    return float((a - b).norm() / b.norm()) <= 2.0 ** -9 + 1e-4


@pytest.mark.parametrize("T,H,I,shared", [(1, 512, 256, 0), (20, 512, 256, 256), (64, 288, 160, 0), (300, 512, 256, 256), (300, 288, 160, 160)])
def test_w4a8_layer_on_mxfp8_input(moe, T, H, I, shared):
    cs = synth.custom_config("mxin", T, H, 16, 4, I, shared_inter=shared, config_id=180)
    cfg, wbuf = layer(moe, cs, T, shared)
    x, lg = synth.gen_x(cs, T, device="cuda"), synth.gen_logits(cs, T, device="cuda")
    o = moe.add_rmsnorm_quantize_mx(x, None, torch.ones(H, device="cuda").bfloat16(), 1e-6)
    ws = torch.empty(moe.workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    y, dbg = moe.run(cfg, wbuf, None, lg, workspace=ws, quantized=(o["codes"], o["sf"], None), debug=True)
    assert moe.last_device_status(ws) == 0
    assert torch.equal(dbg["xq"], o["codes"]) and torch.equal(dbg["xsf"], o["sf"])
    want, wdbg = moe.run(cfg, wbuf, mx_decode(o["codes"], o["sf"]), lg, workspace=ws, debug=True)
    assert torch.equal(dbg["hq"], wdbg["hq"]) and torch.equal(dbg["hsf"], wdbg["hsf"])
    assert close(y, want)
    bad = o["sf"].clone()
    bad[T - 1, 2] = 255
    moe.run(cfg, wbuf, None, lg, workspace=ws, quantized=(o["codes"], bad, None))
    assert moe.last_device_status(ws) == -6
    with pytest.raises(RuntimeError, match="INVALID_ARG"):       # MXFP8 has no tensor scale
        moe.run(cfg, wbuf, None, lg, workspace=ws, quantized=(o["codes"], o["sf"], torch.ones(1, device="cuda")))


@pytest.mark.parametrize("T", [1, 8, 64])
def test_decode_step(moe, T):
    H, E, k = 512, 16, 4
    cs = synth.custom_config("block", T, H, E, k, 256, config_id=181)
    cfg, wbuf = layer(moe, cs, T)
    g = torch.Generator(device="cuda").manual_seed(T)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    wo, wr = moe.quantize_act((n(H, 768) * 0.03).bfloat16()), moe.quantize_act((n(E, H) * 0.1).bfloat16())
    attn, res, gamma = n(T, 768).bfloat16(), n(T, H).bfloat16(), (1 + 0.1 * n(H)).bfloat16()
    ws = torch.empty(moe.workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    lws = moe.router_loss_workspace(T, E)

    def step(res):
        a = moe.linear_w4(attn, *wo)
        o = moe.add_rmsnorm_quantize_mx(a, res, gamma, want_y=True)
        lg = moe.linear_w4(o["y"], *wr, out_dtype=torch.float32)
        y, d = moe.run(cfg, wbuf, None, lg, workspace=ws, quantized=(o["codes"], o["sf"], None), debug=True)
        return a, o, lg, y, d, moe.router_loss(lg, d["topk_ids"], workspace=lws)

    a, o, lg, y, d, st = step(res)
    assert moe.last_device_status(ws) == 0 and moe.last_device_status(lws) == 0
    assert torch.equal(o["h"], (a.float() + res.float()).bfloat16())
    assert torch.equal(d["topk_ids"], moe.plan(lg, k)["topk_ids"])
    assert torch.equal(st["counts"], d["counts"]) and int(st["tokens"]) == T
    assert close(y, moe.run(cfg, wbuf, mx_decode(o["codes"], o["sf"]), lg, workspace=ws))
    # the whole step as one graph, replayed on another residual
    g1 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        ga, go, glg, gy, gd, gst = step(res)
    res.copy_(n(T, H))
    g1.replay()
    a, o, lg, y, d, st = step(res)
    torch.cuda.synchronize()
    assert torch.equal(go["codes"], o["codes"]) and torch.equal(glg, lg) and torch.equal(gst["counts"], st["counts"])
    assert torch.equal(gst["losses"], st["losses"]) and close(gy, y)


def test_training_step(moe):
    """The gradient of the losses with respect to the residual stream through the norm and the
    router matrix, against 64-bit autograd of the same chain (ids and counts held fixed).  The
    gradient of y is rounded to BF16 before the norm's backward pass, and dx after it: 2^-8 each,
    and y itself enters the router in BF16 (another 2^-8 of the gradient's size)."""
    T, H, E, k = 90, 256, 24, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, res, gamma, wr = n(T, H).bfloat16(), n(T, H).bfloat16(), (1 + 0.1 * n(H)).bfloat16(), n(E, H) * 0.1
    mask = torch.arange(T, device="cuda") < 80
    gl, gw = torch.tensor([1.0, 0.1], device="cuda"), n(T, k) * 0.01
    o = moe.add_rmsnorm_quantize_mx(x, res, gamma, want_y=True, want_rrms=True, quantize=False)
    lg = o["y"].float() @ wr.t()
    ids = moe.plan(lg, k)["topk_ids"]
    st = moe.router_loss(lg, ids, mask=mask)
    dl = moe.router_loss_backward(lg, ids, st, gl, grad_topk_w=gw, mask=mask)
    dy = (dl @ wr).bfloat16()
    back = moe.add_rmsnorm_backward(dy, o["h"], o["rrms"], gamma)

    h, gd = o["h"].double().requires_grad_(), gamma.double().requires_grad_()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * gd
    l = y @ wr.double().t()
    p, m = torch.softmax(l, -1), mask.double()
    f = st["counts"].double() / (80 * k)
    w = torch.softmax(l.gather(1, ids.long()), -1)
    goal = (E * (f * (p * m[:, None]).sum(0) / 80).sum() + 0.1 * (torch.logsumexp(l, -1) ** 2 * m).sum() / 80
            + (w * gw.double() * m[:, None]).sum())
    dh, dg = torch.autograd.grad(goal, (h, gd))
    assert float((back["dx"].double() - dh).norm() / dh.norm()) <= 4 * 2.0 ** -8
    assert float((back["dgamma"].double() - dg).norm() / dg.norm()) <= 4 * 2.0 ** -8
    assert not back["dx"][80:].any()
