"""Fused NVFP4 Mixture-of-Experts layer for GB300 (sm_103a): Python binding.

Thin ctypes marshalling over the C ABI in ``include/nvfp4_moe.h``; every step of the layer runs
in the library's CUDA kernels.  PyTorch only provides device memory and the current stream.  The
library must have been built (``__graft_entry__.build()``); there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes as C
import functools
import inspect
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnvfp4moe.so")
_lib = None

MOE_OK = 0
STATUS = {0: "MOE_OK", -1: "MOE_ERR_INVALID_ARG", -2: "MOE_ERR_UNSUPPORTED_SHAPE",
          -3: "MOE_ERR_WORKSPACE_TOO_SMALL", -4: "MOE_ERR_CUDA", -5: "MOE_ERR_DEVICE_TIMEOUT",
          -6: "MOE_ERR_NONFINITE", -7: "MOE_ERR_UNIMPLEMENTED"}

EXPORTED = ["moe_status_string", "moe_config_check", "moe_weights_size", "moe_quantize_weights",
            "moe_weights_export", "moe_act_workspace_size", "moe_quantize_act",
            "moe_plan_workspace_size", "moe_plan", "moe_workspace_size", "moe_run",
            "moe_last_device_status", "moe_plan_static", "moe_run_kernel_count",
            "moe_set_router_bias", "moe_rmsnorm_workspace_size", "moe_rmsnorm_quantize_act",
            "moe_run_quantized", "moe_add_rmsnorm_quantize_mx",
            "moe_add_rmsnorm_backward_workspace_size", "moe_add_rmsnorm_backward",
            "moe_router_loss_workspace_size", "moe_router_loss", "moe_router_loss_backward",
            "moe_linear_w4", "moe_add_layernorm", "moe_add_layernorm_backward_workspace_size",
            "moe_add_layernorm_backward", "moe_sort_tokens_workspace_size", "moe_sort_tokens",
            "moe_permute_rows", "moe_combine_rows", "moe_combine_rows_backward",
            "moe_experts_workspace_size", "moe_experts_forward", "moe_experts_backward",
            "moe_experts_weight_grad"]


class MoeConfig(C.Structure):
    _fields_ = [("num_experts", C.c_int32), ("hidden", C.c_int32), ("inter", C.c_int32),
                ("top_k", C.c_int32), ("shared_inter", C.c_int32), ("h_tensor_scale", C.c_float),
                ("max_tokens", C.c_int32), ("flags", C.c_uint32), ("swiglu_limit", C.c_float),
                ("swiglu_alpha", C.c_float)]

    def __repr__(self):
        return (f"MoeConfig(E={self.num_experts}, H={self.hidden}, I={self.inter}, k={self.top_k}, "
                f"shared_inter={self.shared_inter}, ts_h={self.h_tensor_scale}, "
                f"max_tokens={self.max_tokens})")


# Stages between the library's stage events.  Small batches run the quantiser, router and plan
# as one fused kernel: its time is reported under "act_quant" and "router_plan" is then empty.
STAGES = ("act_quant", "router_plan", "gemm1_swiglu", "gemm2_combine", "bf16_out")
N_STAGE_EVENTS = len(STAGES) + 1


class MoeDebug(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("topk_ids", "topk_w", "counts", "offsets", "perm_src",
                                          "inv", "xq", "xsf", "ts_a", "hq", "hsf",
                                          "stage_events")] + [("inject", C.c_uint32),
                                                              ("hb", C.c_void_p)]


MOE_INJECT_NO_PLAN_FLAG = 1


def lib():
    """The loaded CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it first (python -c 'import "
                               "__graft_entry__ as g; g.build()')")
        L = C.CDLL(LIB_PATH)
        vp, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
        u32, f32 = C.c_uint32, C.c_float
        cfgp = C.POINTER(MoeConfig)
        sig = {
            "moe_status_string": (C.c_char_p, [C.c_int]),
            "moe_config_check": (C.c_int, [cfgp]),
            "moe_weights_size": (sz, [cfgp]),
            "moe_quantize_weights": (C.c_int, [cfgp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "moe_weights_export": (C.c_int, [cfgp, vp, i32, i32, vp, vp, vp, vp]),
            "moe_act_workspace_size": (sz, [i64, i64]),
            "moe_quantize_act": (C.c_int, [vp, i64, i64, vp, vp, vp, vp, sz, vp]),
            "moe_plan_workspace_size": (sz, [i32, i32, i32]),
            "moe_plan": (C.c_int, [vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "moe_workspace_size": (sz, [cfgp, i32]),
            "moe_run": (C.c_int, [cfgp, vp, vp, vp, i32, i32, vp, vp, sz, vp, C.POINTER(MoeDebug)]),
            "moe_run_quantized": (C.c_int, [cfgp, vp, vp, vp, vp, vp, i32, i32, vp, vp, sz, vp,
                                            C.POINTER(MoeDebug)]),
            "moe_last_device_status": (C.c_int, [vp, C.POINTER(C.c_int32)]),
            "moe_plan_static": (C.c_int, [vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]),
            "moe_run_kernel_count": (C.c_int, [cfgp, i32]),
            "moe_set_router_bias": (C.c_int, [cfgp, vp, vp, vp]),
            "moe_rmsnorm_workspace_size": (sz, [i64]),
            "moe_rmsnorm_quantize_act": (C.c_int, [vp, vp, C.c_float, i64, i64, vp, vp, vp, vp, vp, sz,
                                                   vp]),
            "moe_add_rmsnorm_quantize_mx": (C.c_int, [vp, vp, vp, f32, i64, i64, vp, vp, vp, vp,
                                                      vp, vp]),
            "moe_add_rmsnorm_backward_workspace_size": (sz, [i64, i64]),
            "moe_add_rmsnorm_backward": (C.c_int, [vp, vp, vp, vp, vp, i64, i64, vp, vp, vp, sz,
                                                   vp]),
            "moe_router_loss_workspace_size": (sz, [i32, i32]),
            "moe_router_loss": (C.c_int, [vp, vp, vp, i32, i32, i32, u32, vp, vp, vp, vp, vp, sz,
                                          vp]),
            "moe_router_loss_backward": (C.c_int, [vp, vp, vp, i32, i32, i32, u32, vp, vp, vp, vp,
                                                   vp, vp]),
            "moe_linear_w4": (C.c_int, [vp, vp, vp, vp, i32, i64, i64, u32, vp, vp]),
            "moe_add_layernorm": (C.c_int, [vp, vp, vp, vp, f32, i64, i64, u32, vp, vp, vp, vp, vp]),
            "moe_add_layernorm_backward_workspace_size": (sz, [i64, i64]),
            "moe_add_layernorm_backward": (C.c_int, [vp, vp, vp, vp, vp, vp, i64, i64, u32, vp, vp, vp,
                                                     vp, sz, vp]),
            "moe_sort_tokens_workspace_size": (sz, [i32, i32, i32]),
            "moe_sort_tokens": (C.c_int, [vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]),
            "moe_permute_rows": (C.c_int, [vp, vp, i32, i32, i64, i64, vp, vp]),
            "moe_combine_rows": (C.c_int, [vp, vp, vp, i32, i32, i64, i64, u32, vp, vp]),
            "moe_combine_rows_backward": (C.c_int, [vp, vp, vp, vp, i32, i32, i64, i64, u32, vp, vp,
                                                    vp]),
            "moe_experts_workspace_size": (sz, [i64, i64]),
            "moe_experts_forward": (C.c_int, [vp, vp, i64, i32, i64, i64, vp, vp, vp, u32, f32, f32,
                                              vp, vp, vp, vp, vp, sz, vp]),
            "moe_experts_backward": (C.c_int, [vp, vp, i64, i32, i64, i64, vp, vp, vp, u32, f32, f32,
                                               vp, vp, vp, vp, vp, vp, sz, vp]),
            "moe_experts_weight_grad": (C.c_int, [vp, vp, vp, vp, vp, vp, i64, i32, i64, i64, u32, vp,
                                                  vp, vp, vp, sz, vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def status_string(st: int) -> str:
    return lib().moe_status_string(st).decode()


def _check(st: int, what: str):
    if st != MOE_OK:
        raise RuntimeError(f"{what} failed: {STATUS.get(st, st)} ({status_string(st)})")


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


FLAG_ROUTER_SQRTSOFTPLUS = 1
FLAG_SWIGLU_CLAMP = 2
FLAG_ACT_RELU2 = 4
FLAG_ACT_SWIGLU_OAI = 8
FLAG_ACT_BF16 = 16
FLAG_ACT_MXFP8 = 32
ACTIVATIONS = ("swiglu", "relu2", "swiglu_oai")


def _activation_flag(activation, swiglu_limit):
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    if activation == "swiglu_oai" and swiglu_limit is None:
        raise ValueError("swiglu_oai needs swiglu_limit")
    if activation == "relu2":
        return FLAG_ACT_RELU2
    if activation == "swiglu_oai":
        return FLAG_ACT_SWIGLU_OAI
    return FLAG_SWIGLU_CLAMP if swiglu_limit is not None else 0


def make_config(num_experts, hidden, inter, top_k, shared_inter=0, h_tensor_scale=1.0,
                max_tokens=0, router="softmax", swiglu_limit=None, activation="swiglu",
                swiglu_alpha=1.702, precision="nvfp4") -> MoeConfig:
    """router: "softmax" (top-k of the logits, softmax over the k) or "sqrtsoftplus" (scores
    sqrt(softplus(logit)), selection on score + the bias set by set_router_bias, weights the
    normalised unbiased scores).  activation: "swiglu" (silu(g)*u, or with swiglu_limit L
    silu(min(g, L)) * clamp(u, -L, L)), "relu2" (non-gated experts, max(u, 0)^2) or "swiglu_oai"
    ((clamp(u, -L, L) + 1) * g' * sigmoid(alpha * g'), g' = min(g, L); needs swiglu_limit).
    precision: "nvfp4" (activations and h quantised to NVFP4), "w4a16" (BF16 activations as
    they are, weights decoded to BF16 in the GEMMs, h rounded to BF16) or "w4a8" (MXFP4 weights,
    MXFP8 activations and h)."""
    if router not in ("softmax", "sqrtsoftplus"):
        raise ValueError(f"unknown router {router!r}")
    flags = FLAG_ROUTER_SQRTSOFTPLUS if router == "sqrtsoftplus" else 0
    flags |= _activation_flag(activation, swiglu_limit)
    if precision == "w4a16":
        flags |= FLAG_ACT_BF16
    elif precision == "w4a8":
        flags |= FLAG_ACT_MXFP8
    elif precision != "nvfp4":
        raise ValueError(f"unknown precision {precision!r}")
    return MoeConfig(num_experts, hidden, inter, top_k, shared_inter, h_tensor_scale, max_tokens,
                     flags, 0.0 if swiglu_limit is None else float(swiglu_limit),
                     float(swiglu_alpha))


def config_check(cfg: MoeConfig) -> int:
    return lib().moe_config_check(C.byref(cfg))


def weights_size(cfg: MoeConfig) -> int:
    return int(lib().moe_weights_size(C.byref(cfg)))


def quantize_weights(cfg: MoeConfig, w_gate, w_up, w_down, shared=None, wbuf=None, stream=None):
    """BF16 expert weights -> packed NVFP4 weight buffer (a uint8 CUDA tensor).  w_gate (and the
    shared expert's gate) may be None for non-gated (relu2) layers; they are not read there."""
    n = weights_size(cfg)
    if n == 0:
        _check(config_check(cfg), "moe_weights_size")
    if wbuf is None:
        wbuf = torch.empty(n, dtype=torch.uint8, device=w_up.device)
    sg, su, sd = shared if shared is not None else (None, None, None)
    _check(lib().moe_quantize_weights(C.byref(cfg), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                      _ptr(sg), _ptr(su), _ptr(sd), _ptr(wbuf), wbuf.numel(),
                                      _stream(stream)), "moe_quantize_weights")
    return wbuf


def set_router_bias(cfg: MoeConfig, wbuf: torch.Tensor, bias: torch.Tensor) -> None:
    """Stores the sqrt-softplus router's per-expert selection bias (FP32 [E]) in wbuf."""
    bias = bias.to(device=wbuf.device, dtype=torch.float32).contiguous()
    if bias.numel() != cfg.num_experts:
        raise ValueError("bias must have num_experts entries")
    _check(lib().moe_set_router_bias(C.byref(cfg), _ptr(wbuf), _ptr(bias), _stream()),
           "moe_set_router_bias")
    torch.cuda.current_stream().synchronize()


def weights_export(cfg: MoeConfig, wbuf, expert: int, matrix: int, stream=None):
    """Canonical (codes [N,K/2], sf [N,K/16] E4M3 - or [N,K/32] E8M0 for a W4A8 layer's MXFP4
    weights - and ts [1]) of one expert matrix (-1 = shared)."""
    Iw = cfg.shared_inter if expert == -1 else cfg.inter   # this expert's intermediate size
    N, K = (Iw, cfg.hidden) if matrix < 2 else (cfg.hidden, Iw)
    dev = wbuf.device
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device=dev)
    sf = torch.empty(N, K // (32 if cfg.flags & FLAG_ACT_MXFP8 else 16), dtype=torch.uint8,
                     device=dev)
    ts = torch.empty(1, dtype=torch.float32, device=dev)
    _check(lib().moe_weights_export(C.byref(cfg), _ptr(wbuf), expert, matrix, _ptr(codes), _ptr(sf),
                                    _ptr(ts), _stream(stream)), "moe_weights_export")
    return codes, sf, ts


def quantize_act(x, workspace=None, stream=None):
    """x [rows, cols] BF16 -> (codes [rows, cols/2], sf [rows, cols/16], ts [1]) on the device."""
    rows, cols = x.shape
    dev = x.device
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=dev)
    sf = torch.empty(rows, cols // 16, dtype=torch.uint8, device=dev)
    ts = torch.empty(1, dtype=torch.float32, device=dev)
    nws = int(lib().moe_act_workspace_size(rows, cols))
    if workspace is None:
        workspace = torch.empty(nws, dtype=torch.uint8, device=dev)
    _check(lib().moe_quantize_act(_ptr(x), rows, cols, _ptr(codes), _ptr(sf), _ptr(ts),
                                  _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_quantize_act")
    return codes, sf, ts


def rmsnorm_quantize_act(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6,
                         workspace=None, stream=None, want_rrms: bool = False):
    """RMSNorm of BF16 x [rows, cols] by BF16 gamma [cols], then NVFP4 (codes, sf, ts) on the
    device (+ each row's 1/rms when want_rrms); a non-finite result is reported through the
    device status (last_device_status), not raised here."""
    rows, cols = x.shape
    dev = x.device
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=dev)
    sf = torch.empty(rows, cols // 16, dtype=torch.uint8, device=dev)
    ts = torch.empty(1, dtype=torch.float32, device=dev)
    rr = torch.empty(rows, dtype=torch.float32, device=dev) if want_rrms else None
    if workspace is None:
        workspace = torch.empty(lib().moe_rmsnorm_workspace_size(rows), dtype=torch.uint8,
                                device=dev)
    _check(lib().moe_rmsnorm_quantize_act(_ptr(x), _ptr(gamma), float(eps), rows, cols,
                                          _ptr(codes), _ptr(sf), _ptr(ts),
                                          _ptr(rr) if rr is not None else None, _ptr(workspace),
                                          workspace.numel(), _stream(stream)),
           "moe_rmsnorm_quantize_act")
    return (codes, sf, ts, rr) if want_rrms else (codes, sf, ts)


def plan(logits, k: int, workspace=None, stream=None):
    """Router top-k + permutation plan for logits [T, E] FP32 (dict of device tensors)."""
    T, E = logits.shape
    dev = logits.device
    out = dict(topk_ids=torch.empty(T, k, dtype=torch.int32, device=dev),
               topk_w=torch.empty(T, k, dtype=torch.float32, device=dev),
               counts=torch.empty(E, dtype=torch.int32, device=dev),
               offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
               perm_src=torch.empty(T * k, dtype=torch.int32, device=dev),
               inv=torch.empty(T * k, dtype=torch.int32, device=dev))
    nws = int(lib().moe_plan_workspace_size(T, E, k))
    if workspace is None:
        workspace = torch.empty(max(nws, 256), dtype=torch.uint8, device=dev)
    _check(lib().moe_plan(_ptr(logits), T, E, k, _ptr(out["topk_ids"]), _ptr(out["topk_w"]),
                          _ptr(out["counts"]), _ptr(out["offsets"]), _ptr(out["perm_src"]),
                          _ptr(out["inv"]), _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_plan")
    return out


def plan_static(logits, k: int, out=None, stream=None):
    """moe_plan through moe_plan_static: no workspace argument, for callers that cannot
    allocate device memory (the library's static per-device scratch is used; calls on several
    streams at once race).  ``out`` may pass preallocated output tensors."""
    T, E = logits.shape
    dev = logits.device
    if out is None:
        out = dict(topk_ids=torch.empty(T, k, dtype=torch.int32, device=dev),
                   topk_w=torch.empty(T, k, dtype=torch.float32, device=dev),
                   counts=torch.empty(E, dtype=torch.int32, device=dev),
                   offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                   perm_src=torch.empty(T * k, dtype=torch.int32, device=dev),
                   inv=torch.empty(T * k, dtype=torch.int32, device=dev))
    _check(lib().moe_plan_static(_ptr(logits), T, E, k, _ptr(out["topk_ids"]), _ptr(out["topk_w"]),
                                 _ptr(out["counts"]), _ptr(out["offsets"]), _ptr(out["perm_src"]),
                                 _ptr(out["inv"]), _stream(stream)), "moe_plan_static")
    return out


def workspace_size(cfg: MoeConfig, T: int) -> int:
    return int(lib().moe_workspace_size(C.byref(cfg), T))


def run_kernel_count(cfg: MoeConfig, T: int) -> int:
    """Kernels one run() at T tokens launches (host arithmetic, no device needed)."""
    n = int(lib().moe_run_kernel_count(C.byref(cfg), T))
    if n < 0:
        raise RuntimeError(f"moe_run_kernel_count: {status_string(n)}")
    return n


class StageTimer:
    """CUDA events the library records on its launch stream between the layer's stages."""

    def __init__(self):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(N_STAGE_EVENTS)]
        for e in self.events:      # torch creates the CUDA event on its first record
            e.record()
        self._handles = (C.c_void_p * N_STAGE_EVENTS)(*[e.cuda_event for e in self.events])
        self.c_debug = MoeDebug(*([None] * 11), C.cast(self._handles, C.c_void_p))

    def stage_ms(self):
        """Milliseconds of each stage of the last recorded call (synchronise first)."""
        return {n: self.events[i].elapsed_time(self.events[i + 1]) for i, n in enumerate(STAGES)}


def run(cfg: MoeConfig, wbuf, x, logits, k=None, y=None, workspace=None, debug=False, stream=None,
        timer: StageTimer = None, quantized=None, inject: int = 0):
    """The layer: y [T, H] BF16 (and, with debug=True, a dict of its intermediates).  x is the BF16
    input [T, H]; or pass x=None and quantized=(xq [T, H/2] u8, xsf [T, H/16] u8, ts_a [1] f32),
    already-NVFP4 activations (moe_run_quantized).  A W4A8 layer takes MXFP8 there: (xq [T, H] u8,
    xsf [T, H/32] u8, None), as add_rmsnorm_quantize_mx gives them."""
    if quantized is not None:
        xq, xsf, ts_a = quantized
        T, H = xq.shape[0], xq.shape[1] * (1 if cfg.flags & FLAG_ACT_MXFP8 else 2)
        dev = xq.device
    else:
        T, H = x.shape
        dev = x.device
    k = cfg.top_k if k is None else k
    if y is None:
        y = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    if workspace is None:
        workspace = torch.empty(max(workspace_size(cfg, T), 256), dtype=torch.uint8, device=dev)
    dbg = None
    dbg_c = None
    if debug:
        # h rows are as wide as the layer's widest intermediate (a shared expert of another
        # width than the routed ones: the narrower rows end in zeros)
        E, I = cfg.num_experts, max(cfg.inter, cfg.shared_inter)
        Rt = T * k + (T if cfg.shared_inter else 0)
        dbg = dict(topk_ids=torch.empty(T, k, dtype=torch.int32, device=dev),
                   topk_w=torch.empty(T, k, dtype=torch.float32, device=dev),
                   counts=torch.empty(E, dtype=torch.int32, device=dev),
                   offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                   perm_src=torch.empty(T * k, dtype=torch.int32, device=dev),
                   inv=torch.empty(T * k, dtype=torch.int32, device=dev),
                   xq=torch.empty(T, H // 2, dtype=torch.uint8, device=dev),
                   xsf=torch.empty(T, H // 16, dtype=torch.uint8, device=dev),
                   ts_a=torch.empty(1, dtype=torch.float32, device=dev),
                   hq=torch.empty(Rt, I // 2, dtype=torch.uint8, device=dev),
                   hsf=torch.empty(Rt, I // 16, dtype=torch.uint8, device=dev))
        if cfg.flags & FLAG_ACT_BF16:        # nothing is quantised; h stays BF16 (hb)
            for n in ("hq", "hsf", "xq", "xsf", "ts_a"):
                del dbg[n]
            dbg["hb"] = torch.empty(Rt, I, dtype=torch.bfloat16, device=dev)
        if cfg.flags & FLAG_ACT_MXFP8:       # MXFP8 codes + E8M0 scales of x and h, decoded h
            del dbg["ts_a"]
            dbg["xq"] = torch.empty(T, H, dtype=torch.uint8, device=dev)
            dbg["xsf"] = torch.empty(T, H // 32, dtype=torch.uint8, device=dev)
            dbg["hq"] = torch.empty(Rt, I, dtype=torch.uint8, device=dev)
            dbg["hsf"] = torch.empty(Rt, I // 32, dtype=torch.uint8, device=dev)
            dbg["hb"] = torch.empty(Rt, I, dtype=torch.bfloat16, device=dev)
        dbg_c = MoeDebug(*[dbg[n].data_ptr() if n in dbg else None
                           for n, _ in MoeDebug._fields_[:11]],
                         C.cast(timer._handles, C.c_void_p) if timer is not None else None)
        if "hb" in dbg:
            dbg_c.hb = dbg["hb"].data_ptr()
    elif timer is not None:
        dbg_c = timer.c_debug
    if inject:
        dbg_c = MoeDebug.from_buffer_copy(dbg_c) if dbg_c is not None else MoeDebug()
        dbg_c.inject = inject
    dptr = C.byref(dbg_c) if dbg_c is not None else None
    if quantized is not None:
        _check(lib().moe_run_quantized(C.byref(cfg), _ptr(wbuf), _ptr(xq), _ptr(xsf), _ptr(ts_a),
                                       _ptr(logits), T, k, _ptr(y), _ptr(workspace),
                                       workspace.numel(), _stream(stream), dptr),
               "moe_run_quantized")
    else:
        _check(lib().moe_run(C.byref(cfg), _ptr(wbuf), _ptr(x), _ptr(logits), T, k, _ptr(y),
                             _ptr(workspace), workspace.numel(), _stream(stream), dptr), "moe_run")
    return (y, dbg) if debug else y


# ---- operators around the layer ----
#
# Every function takes stream=, the torch.cuda.Stream to launch on (default: the current one).  None of
# them records anything for autograd: a backward pass is a call of its own.

# The current stream's handle of a device: torch's own accessor where it has it (0.1 us; the Stream
# object costs 1.1 us of a call's 9)
_stream_handle = getattr(torch._C, "_cuda_getCurrentRawStream",
                         lambda dev: torch.cuda.current_stream(dev).cuda_stream)
# the current device's index, CUDA being initialised (there are tensors on it): half the time of
# torch.cuda.current_device
_device_index = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _scoped(fn):
    """Calls fn(stream handle, ...) with its first tensor's device current, on `stream` (a
    torch.cuda.Stream) if that is passed, which then owns what fn allocates, or on the device's
    current stream."""
    sig = inspect.signature(fn)
    params = list(sig.parameters.values())[1:]   # without the stream handle
    name = params[0].name

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        first = args[0] if args else kw.get(name)
        if first is None:
            raise ValueError(f"{fn.__name__}: {name} is required")
        if not first.is_cuda:
            raise ValueError(f"{fn.__name__} needs CUDA tensors, got one on {first.device}")
        dev = first.get_device()
        if stream is None and dev == _device_index():
            return fn(_stream_handle(dev), *args, **kw)
        if stream is not None and stream.device != first.device:
            raise ValueError(f"{fn.__name__}: the stream is on {stream.device}, the tensors on "
                             f"{first.device}")
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            return fn(_stream_handle(dev), *args, **kw)

    call.__signature__ = sig.replace(parameters=params + [
        inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)])
    return call


def _given(t, name, dtype, shape, dev):
    """Device address of a tensor argument after its checks (None stays None); dev: the index of
    the device that it has to be on."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                     f"cuda:{dev}, got {t.dtype} {tuple(t.shape)} stride {t.stride()} on {t.device}")


def _need(t, name):
    if t is None:
        raise ValueError(f"{name} is required")
    return t


def _bytes_on(n, device):
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


_U8, _BF16, _F32, _I32 = torch.uint8, torch.bfloat16, torch.float32, torch.int32


@_scoped
def add_rmsnorm_quantize_mx(handle, x, residual, gamma, eps: float = 1e-6, want_y: bool = False,
                            want_rrms: bool = False, quantize: bool = True, out=None):
    """h = bf16(x + residual), y = RMSNorm(h) * gamma and MXFP8 of y, in one launch.

    x, residual [rows, cols] BF16 (residual None: h is x), gamma [cols] BF16.  Returns a dict of
    h (absent without a residual), codes [rows, cols] u8 (E4M3) and sf [rows, cols/32] u8 (E8M0)
    unless quantize is False, y [rows, cols] BF16 (want_y) and rrms [rows] FP32 (want_rrms).
    out: a dict of preallocated tensors that takes the place of those switches; out["h"] may be
    residual or x itself (in place).  stream: a torch.cuda.Stream to launch on."""
    if x.dim() != 2 or x.shape[1] % 32:
        raise ValueError(f"x must be [rows, cols] with cols a multiple of 32, got {tuple(x.shape)}")
    rows, cols = shape = x.shape
    dev = x.get_device()
    if out is None:
        out = {}
        if residual is not None:
            out["h"] = torch.empty_like(x)
        if quantize:
            out["codes"] = torch.empty(shape, dtype=_U8, device=dev)
            out["sf"] = torch.empty(rows, cols // 32, dtype=_U8, device=dev)
        if want_y:
            out["y"] = torch.empty_like(x)
        if want_rrms:
            out["rrms"] = torch.empty(rows, dtype=_F32, device=dev)
    get = out.get
    st = lib().moe_add_rmsnorm_quantize_mx(
        _given(x, "x", _BF16, shape, dev), _given(residual, "residual", _BF16, shape, dev),
        _given(_need(gamma, "gamma"), "gamma", _BF16, (cols,), dev), eps, rows, cols,
        _given(get("h"), "h", _BF16, shape, dev), _given(get("codes"), "codes", _U8, shape, dev),
        _given(get("sf"), "sf", _U8, (rows, cols // 32), dev),
        _given(get("y"), "y", _BF16, shape, dev), _given(get("rrms"), "rrms", _F32, (rows,), dev),
        handle)
    if st:
        _check(st, "moe_add_rmsnorm_quantize_mx")
    return out


def add_rmsnorm_backward_workspace(rows: int, cols: int, device="cuda"):
    return _bytes_on(lib().moe_add_rmsnorm_backward_workspace_size(rows, cols), device)


@_scoped
def add_rmsnorm_backward(handle, dy, h, rrms, gamma, dh=None, out=None, workspace=None):
    """Backward pass of add_rmsnorm_quantize_mx's norm, the quantisation passed straight through.

    dy, h [rows, cols] BF16, rrms [rows] FP32, gamma [cols] BF16 as in the forward pass; dh: the
    gradient that reaches h over the residual stream (BF16, or None).  Returns a dict of dx
    [rows, cols] BF16 (the gradient of x and of the residual alike; out["dx"] may be dy or dh) and
    dgamma [cols] FP32.  stream: a torch.cuda.Stream to launch on."""
    if dy.dim() != 2 or dy.shape[1] % 32:
        raise ValueError(f"dy must be [rows, cols] with cols a multiple of 32, got {tuple(dy.shape)}")
    rows, cols = shape = dy.shape
    dev = dy.get_device()
    if out is None:
        out = {"dx": torch.empty_like(dy), "dgamma": torch.empty(cols, dtype=_F32, device=dev)}
    if workspace is None:
        workspace = add_rmsnorm_backward_workspace(rows, cols, dev)
    st = lib().moe_add_rmsnorm_backward(
        _given(dy, "dy", _BF16, shape, dev), _given(dh, "dh", _BF16, shape, dev),
        _given(_need(h, "h"), "h", _BF16, shape, dev),
        _given(_need(rrms, "rrms"), "rrms", _F32, (rows,), dev),
        _given(_need(gamma, "gamma"), "gamma", _BF16, (cols,), dev), rows, cols,
        _given(out["dx"], "dx", _BF16, shape, dev),
        _given(out["dgamma"], "dgamma", _F32, (cols,), dev),
        _given(workspace, "workspace", _U8, workspace.shape, dev), workspace.numel(),
        handle)
    if st:
        _check(st, "moe_add_rmsnorm_backward")
    return out


_ROUTER_FLAGS = {"softmax": 0, "sqrtsoftplus": FLAG_ROUTER_SQRTSOFTPLUS}


def _router_flag(router):
    if router not in _ROUTER_FLAGS:
        raise ValueError(f"unknown router {router!r}")
    return _ROUTER_FLAGS[router]


def _mask_ptr(mask, T, dev):
    if mask is None:
        return None
    return _given(mask, "mask", torch.bool if mask.dtype is torch.bool else _U8, (T,), dev)


def _routing_shape(logits, topk_ids):
    if logits.dim() != 2 or _need(topk_ids, "topk_ids").dim() != 2:
        raise ValueError("logits must be [T, E] and topk_ids [T, k]")
    return logits.shape[0], logits.shape[1], topk_ids.shape[1]


def router_loss_workspace(T: int, E: int, device="cuda"):
    return _bytes_on(lib().moe_router_loss_workspace_size(T, E), device)


@_scoped
def router_loss(handle, logits, topk_ids, mask=None, router: str = "softmax", out=None, workspace=None):
    """Per-expert counts and the router's losses for logits [T, E] FP32 and topk_ids [T, k] int32
    (as plan gives them); mask [T] (bool or uint8) is 0 for padded tokens.

    Returns a dict of losses [2] FP32 (balance, z), counts [E] int32, tokens [1] int32 and probs
    [E] FP32 (mean expert probabilities); pass it to router_loss_backward.  An id outside [0, E)
    is reported in the workspace's device status (pass a workspace to read it with
    last_device_status).  stream: a torch.cuda.Stream to launch on."""
    T, E, k = _routing_shape(logits, topk_ids)
    dev = logits.get_device()
    if out is None:
        out = dict(losses=torch.empty(2, dtype=_F32, device=dev),
                   counts=torch.empty(E, dtype=_I32, device=dev),
                   tokens=torch.empty(1, dtype=_I32, device=dev),
                   probs=torch.empty(E, dtype=_F32, device=dev))
    if workspace is None:
        workspace = router_loss_workspace(T, E, dev)
    st = lib().moe_router_loss(
        _given(logits, "logits", _F32, (T, E), dev), _given(topk_ids, "topk_ids", _I32, (T, k), dev),
        _mask_ptr(mask, T, dev), T, E, k, _router_flag(router),
        _given(out["losses"], "losses", _F32, (2,), dev),
        _given(out["counts"], "counts", _I32, (E,), dev),
        _given(out["tokens"], "tokens", _I32, (1,), dev),
        _given(out["probs"], "probs", _F32, (E,), dev),
        _given(workspace, "workspace", _U8, workspace.shape, dev), workspace.numel(),
        handle)
    if st:
        _check(st, "moe_router_loss")
    return out


@_scoped
def router_loss_backward(handle, logits, topk_ids, stats, grad_losses=None, grad_topk_w=None, mask=None,
                         router: str = "softmax", dlogits=None):
    """Gradient [T, E] FP32 of the logits from grad_losses [2] FP32 (on the device; the gradients
    of the balance and z losses) and grad_topk_w [T, k] FP32 (of the top-k weights); either may be
    None.  The latter is the dtopk_w of combine_tokens_backward, or comes from the caller's own backward pass
    through the experts.  stats: what router_loss returned for the same logits, ids, mask and router.
    stream: a torch.cuda.Stream to launch on."""
    T, E, k = _routing_shape(logits, topk_ids)
    dev = logits.get_device()
    if dlogits is None:
        dlogits = torch.empty(T, E, dtype=_F32, device=dev)
    st = lib().moe_router_loss_backward(
        _given(logits, "logits", _F32, (T, E), dev), _given(topk_ids, "topk_ids", _I32, (T, k), dev),
        _mask_ptr(mask, T, dev), T, E, k, _router_flag(router),
        _given(stats["counts"], "counts", _I32, (E,), dev),
        _given(stats["tokens"], "tokens", _I32, (1,), dev),
        _given(grad_losses, "grad_losses", _F32, (2,), dev),
        _given(grad_topk_w, "grad_topk_w", _F32, (T, k), dev),
        _given(dlogits, "dlogits", _F32, (T, E), dev), handle)
    if st:
        _check(st, "moe_router_loss_backward")
    return dlogits


LINEAR_MXFP4 = 1
LINEAR_F32_OUT = 2
LINEAR_MAX_TOKENS = 64


@_scoped
def linear_w4(handle, x, codes, sf, ts=None, out_dtype=torch.bfloat16, y=None):
    """x [T, K] BF16 (T <= LINEAR_MAX_TOKENS) times a 4-bit matrix: y [T, N] in out_dtype (bfloat16 or float32).

    codes [N, K/2] u8 with sf [N, K/16] u8 (E4M3) and ts [1] FP32: NVFP4, as quantize_act(W) gives
    them; with sf [N, K/32] u8 (E8M0) and no ts: MXFP4.
    stream: a torch.cuda.Stream to launch on."""
    if x.dim() != 2 or codes.dim() != 2 or sf.dim() != 2:
        raise ValueError("x must be [T, K], codes [N, K/2] and sf [N, K/16] or [N, K/32]")
    (T, K), N, dev = x.shape, codes.shape[0], x.get_device()
    flags, block = (LINEAR_MXFP4, 32) if ts is None else (0, 16)
    if K % 32:
        raise ValueError(f"K must be a multiple of 32, got {K}")
    if y is None:
        y = torch.empty(T, N, dtype=out_dtype, device=dev)
    if y.dtype is _F32:
        flags |= LINEAR_F32_OUT
    elif y.dtype is not _BF16:
        raise ValueError(f"the output is bfloat16 or float32, not {y.dtype}")
    if ts is not None and ts.dim() == 0:
        ts = ts.reshape(1)
    st = lib().moe_linear_w4(
        _given(x, "x", _BF16, (T, K), dev), _given(codes, "codes", _U8, (N, K // 2), dev),
        _given(sf, "sf", _U8, (N, K // block), dev), _given(ts, "ts", _F32, (1,), dev), T, N, K,
        flags, _given(y, "y", y.dtype, (T, N), dev), handle)
    if st:
        _check(st, "moe_linear_w4")
    return y


# ---- the layer's training pass: layer norm, tokens to their experts and back, the experts ----

ROWS_F32 = 1
EXPERTS_ACCUMULATE = 0x100


def _row_type(t, name):
    if t.dtype is _BF16:
        return 0
    if t.dtype is _F32:
        return ROWS_F32
    raise ValueError(f"{name} must be bfloat16 or float32, not {t.dtype}")


def _matrix(t, name, multiple):
    if t.dim() != 2 or t.shape[1] % multiple or t.shape[1] == 0:
        raise ValueError(f"{name} must be [rows, cols] with cols a multiple of {multiple}, got {tuple(t.shape)}")
    return t.shape


@_scoped
def add_layernorm(handle, x, residual, gamma, beta=None, eps: float = 1e-5, want_stats: bool = False, out=None):
    """h = x + residual and y = LayerNorm(h) * gamma + beta, in one launch.

    x, residual [rows, cols] (residual None: h is x), gamma, beta [cols] (beta may be None), all
    bfloat16 or all float32, cols a multiple of 8.  Returns a dict of h (absent without a residual), y
    and, with want_stats, mean and rstd [rows] FP32, which add_layernorm_backward takes.  out: a dict
    of preallocated tensors (y and, with a residual, h) that takes the place of the switch; out["h"] may be
    residual or x itself (in place).  stream: a torch.cuda.Stream to launch on."""
    rows, cols = shape = _matrix(x, "x", 8)
    dt, dev, flags = x.dtype, x.get_device(), _row_type(x, "x")
    if out is None:
        out = {"y": torch.empty_like(x)}
        if residual is not None:
            out["h"] = torch.empty_like(x)
        if want_stats:
            out["mean"] = torch.empty(rows, dtype=_F32, device=dev)
            out["rstd"] = torch.empty(rows, dtype=_F32, device=dev)
    get, line, each = out.get, (cols,), (rows,)
    st = lib().moe_add_layernorm(
        _given(x, "x", dt, shape, dev), _given(residual, "residual", dt, shape, dev),
        _given(_need(gamma, "gamma"), "gamma", dt, line, dev), _given(beta, "beta", dt, line, dev), eps, rows,
        cols, flags, _given(get("h"), "h", dt, shape, dev), _given(_need(get("y"), "y"), "y", dt, shape, dev),
        _given(get("mean"), "mean", _F32, each, dev), _given(get("rstd"), "rstd", _F32, each, dev), handle)
    if st:
        _check(st, "moe_add_layernorm")
    return out


def add_layernorm_backward_workspace(rows: int, cols: int, device="cuda"):
    return _bytes_on(lib().moe_add_layernorm_backward_workspace_size(rows, cols), device)


@_scoped
def add_layernorm_backward(handle, dy, h, mean, rstd, gamma, dh=None, out=None, workspace=None):
    """Backward pass of add_layernorm.

    dy, h [rows, cols], gamma [cols] (types as in the forward pass), mean, rstd [rows] FP32 as the forward
    pass gives them; dh: the gradient that reaches h over the residual stream (or None).  Returns a dict
    of dx [rows, cols] (the gradient of x and of the residual alike; out["dx"] may be dy or dh), dgamma
    and dbeta [cols] FP32; an out without "dbeta" leaves that out.  stream: a torch.cuda.Stream to launch on."""
    rows, cols = shape = _matrix(dy, "dy", 8)
    dt, dev, flags = dy.dtype, dy.get_device(), _row_type(dy, "dy")
    if out is None:
        out = {"dx": torch.empty_like(dy), "dgamma": torch.empty(cols, dtype=_F32, device=dev),
               "dbeta": torch.empty(cols, dtype=_F32, device=dev)}
    if workspace is None:
        workspace = add_layernorm_backward_workspace(rows, cols, dev)
    st = lib().moe_add_layernorm_backward(
        _given(dy, "dy", dt, shape, dev), _given(dh, "dh", dt, shape, dev),
        _given(_need(h, "h"), "h", dt, shape, dev), _given(_need(mean, "mean"), "mean", _F32, (rows,), dev),
        _given(_need(rstd, "rstd"), "rstd", _F32, (rows,), dev),
        _given(_need(gamma, "gamma"), "gamma", dt, (cols,), dev), rows, cols, flags,
        _given(out["dx"], "dx", dt, shape, dev), _given(out["dgamma"], "dgamma", _F32, (cols,), dev),
        _given(out.get("dbeta"), "dbeta", _F32, (cols,), dev),
        _given(workspace, "workspace", _U8, workspace.shape, dev), workspace.numel(), handle)
    if st:
        _check(st, "moe_add_layernorm_backward")
    return out


def sort_tokens_workspace(T: int, num_experts: int, k: int, device="cuda"):
    return _bytes_on(lib().moe_sort_tokens_workspace_size(T, num_experts, k), device)


@_scoped
def sort_tokens(handle, topk_ids, num_experts: int, mask=None, out=None, workspace=None):
    """The plan of given expert ids [T, k] int32 (any router's): a dict of counts [E], offsets [E+1],
    perm_src [T*k] (row -> token) and inv [T*k] (assignment -> row), int32, as plan gives them.

    mask [T] (bool or uint8) is 0 for tokens that are left out; ids of -1 are left out too (inv -1,
    perm_src -1 from offsets[E] on).  Any other id outside [0, num_experts) is left out and reported in
    the workspace's device status (pass a workspace to read it with last_device_status).  stream: a
    torch.cuda.Stream to launch on."""
    if topk_ids.dim() != 2:
        raise ValueError(f"topk_ids must be [T, k], got {tuple(topk_ids.shape)}")
    (T, k), E, dev = topk_ids.shape, num_experts, topk_ids.get_device()
    if out is None:
        out = {n: torch.empty(m, dtype=_I32, device=dev)
               for n, m in (("counts", max(E, 0)), ("offsets", max(E, 0) + 1), ("perm_src", T * k), ("inv", T * k))}
    if workspace is None:
        workspace = sort_tokens_workspace(T, E, k, dev)
    st = lib().moe_sort_tokens(
        _given(topk_ids, "topk_ids", _I32, (T, k), dev), _mask_ptr(mask, T, dev), T, E, k,
        _given(out["counts"], "counts", _I32, (E,), dev), _given(out["offsets"], "offsets", _I32, (E + 1,), dev),
        _given(out["perm_src"], "perm_src", _I32, (T * k,), dev), _given(out["inv"], "inv", _I32, (T * k,), dev),
        _given(workspace, "workspace", _U8, workspace.shape, dev), workspace.numel(), handle)
    if st:
        _check(st, "moe_sort_tokens")
    return out


def _inverse(plan, T, dev):
    """Address of the plan's inv for T tokens, and k."""
    inv = _need(_need(plan, "plan").get("inv"), "plan['inv']")
    if T == 0:
        return None, 1
    if inv.numel() == 0 or inv.numel() % T:
        raise ValueError(f"plan['inv'] has {inv.numel()} entries, which is no multiple of the {T} tokens")
    return _given(inv, "plan['inv']", _I32, (inv.numel(),), dev), inv.numel() // T


@_scoped
def permute_tokens(handle, x, plan, out=None):
    """Rows sorted by expert: rows[inv[t*k+j]] = x[t] for x [T, cols] of any type (rows of a multiple of
    16 bytes) and a plan of plan or sort_tokens.  Returns rows [T*k, cols]; rows behind the last expert's stay
    as they were in out (uninitialised without one).  stream: a torch.cuda.Stream to launch on."""
    if x.dim() != 2:
        raise ValueError(f"x must be [T, cols], got {tuple(x.shape)}")
    (T, cols), dev = x.shape, x.get_device()
    inv, k = _inverse(plan, T, dev)
    if out is None:
        out = torch.empty(T * k, cols, dtype=x.dtype, device=dev)
    st = lib().moe_permute_rows(_given(x, "x", x.dtype, (T, cols), dev), inv, T, k, cols * x.element_size(), out.shape[0],
                                _given(out, "out", x.dtype, (out.shape[0], cols), dev), handle)
    if st:
        _check(st, "moe_permute_rows")
    return out


@_scoped
def permute_tokens_backward(handle, drows, plan, num_tokens: int, out=None):
    """Gradient [num_tokens, cols] of permute_tokens's x: the sum of each token's rows of drows (bfloat16 or
    float32), in FP32 and slot order.  stream: a torch.cuda.Stream to launch on."""
    return _combine(handle, drows, "drows", plan, None, num_tokens, out)


@_scoped
def combine_tokens(handle, rows, plan, topk_w, out=None):
    """y[t] = sum_j topk_w[t, j] * rows[inv[t*k+j]]: rows [T*k, cols] bfloat16 or float32 in expert order, topk_w
    [T, k] FP32.  Returns y [T, cols] in the type of rows; assignments that were left out add nothing.
    stream: a torch.cuda.Stream to launch on."""
    if _need(topk_w, "topk_w").dim() != 2:
        raise ValueError(f"topk_w must be [T, k], got {tuple(topk_w.shape)}")
    return _combine(handle, rows, "rows", plan, topk_w, topk_w.shape[0], out)


def _combine(handle, rows, name, plan, topk_w, T, out):
    flags = _row_type(rows, name)
    R, cols = _matrix(rows, name, 4 if flags else 8)
    dev = rows.get_device()
    inv, k = _inverse(plan, T, dev)
    if out is None:
        out = torch.empty(T, cols, dtype=rows.dtype, device=dev)
    st = lib().moe_combine_rows(_given(rows, name, rows.dtype, (R, cols), dev), inv,
                                _given(topk_w, "topk_w", _F32, (T, k), dev) if T else None, T, k, cols, R, flags,
                                _given(out, "out", rows.dtype, (T, cols), dev), handle)
    if st:
        _check(st, "moe_combine_rows")
    return out


@_scoped
def combine_tokens_backward(handle, dy, rows, plan, topk_w, out=None):
    """Backward pass of combine_tokens: from dy [T, cols] a dict of drows [T*k, cols] (in the type of rows; rows
    behind the last expert's stay as they were in out) and dtopk_w [T, k] FP32 (0 where there is no row),
    which router_loss_backward takes as grad_topk_w.  out["drows"] may be rows itself.  stream: a
    torch.cuda.Stream to launch on."""
    flags = _row_type(dy, "dy")
    T, cols = _matrix(dy, "dy", 4 if flags else 8)
    if _need(rows, "rows").dim() != 2:
        raise ValueError(f"rows must be [T*k, cols], got {tuple(rows.shape)}")
    dt, dev, R = dy.dtype, dy.get_device(), rows.shape[0]
    inv, k = _inverse(plan, T, dev)
    if out is None:
        out = {"drows": torch.empty_like(rows), "dtopk_w": torch.empty_like(_need(topk_w, "topk_w"))}
    st = lib().moe_combine_rows_backward(
        _given(dy, "dy", dt, (T, cols), dev), _given(rows, "rows", dt, (R, cols), dev), inv,
        _given(_need(topk_w, "topk_w"), "topk_w", _F32, (T, k) if T else topk_w.shape, dev), T, k, cols, R, flags,
        _given(out["drows"], "drows", dt, (R, cols), dev),
        _given(out["dtopk_w"], "dtopk_w", _F32, topk_w.shape, dev), handle)
    if st:
        _check(st, "moe_combine_rows_backward")
    return out


def experts_workspace(R: int, inter: int, device="cuda"):
    """Workspace of the three experts_* functions for up to R rows."""
    return _bytes_on(lib().moe_experts_workspace_size(R, inter), device)


def _experts_shapes(rows, name, plan, w_up, w_down):
    if rows.dim() != 2 or _need(w_up, "w_up").dim() != 3 or _need(w_down, "w_down").dim() != 3:
        raise ValueError(f"{name} must be [R, H], w_up [E, I, H] and w_down [E, H, I]")
    (R, H), (E, I) = rows.shape, w_up.shape[:2]
    if H % 32 or I % 32 or H == 0 or I == 0:
        raise ValueError(f"H and I must be multiples of 32, got {H} and {I}")
    return R, H, E, I


def _offsets(plan, E, dev):
    return _given(_need(_need(plan, "plan").get("offsets"), "plan['offsets']"), "plan['offsets']", _I32, (E + 1,), dev)


@_scoped
def experts_forward(handle, rows, plan, w_gate, w_up, w_down, activation: str = "swiglu", swiglu_limit=None,
                    swiglu_alpha: float = 1.702, keep: bool = False, out=None, workspace=None):
    """The experts on rows [R, H] BF16 sorted by expert (permute_tokens), plan["offsets"] their segments:
    out = act(rows Wg^T, rows Wu^T) Wd^T per expert.

    w_gate, w_up [E, I, H], w_down [E, H, I] BF16 (w_gate None for relu2); activation, swiglu_limit and
    swiglu_alpha as in make_config.  Returns a dict of out [R, H] and, with keep, of what the backward pass
    reads: g, u (relu2: u alone) and h [R, I].  out: a dict of preallocated tensors that takes the place of the
    switch.  Rows behind the last expert's stay as they were.  stream: a torch.cuda.Stream to launch on."""
    flags = _activation_flag(activation, swiglu_limit)
    R, H, E, I = _experts_shapes(rows, "rows", plan, w_up, w_down)
    dev, gated = rows.get_device(), activation != "relu2"
    if out is None:
        out = {"out": torch.empty_like(rows)}
        if keep:
            out.update({n: torch.empty(R, I, dtype=_BF16, device=dev) for n in (("g", "u", "h") if gated else ("u", "h"))})
    get = out.get
    if workspace is None:
        workspace = experts_workspace(0 if get("h") is not None else R, I, dev)
    st = lib().moe_experts_forward(
        _given(rows, "rows", _BF16, (R, H), dev), _offsets(plan, E, dev), R, E, H, I,
        _given(_need(w_gate, "w_gate"), "w_gate", _BF16, (E, I, H), dev) if gated else None,
        _given(w_up, "w_up", _BF16, (E, I, H), dev), _given(w_down, "w_down", _BF16, (E, H, I), dev), flags,
        0.0 if swiglu_limit is None else swiglu_limit, swiglu_alpha,
        _given(get("g"), "g", _BF16, (R, I), dev), _given(get("u"), "u", _BF16, (R, I), dev),
        _given(get("h"), "h", _BF16, (R, I), dev), _given(out["out"], "out", _BF16, (R, H), dev),
        _given(workspace, "workspace", _U8, workspace.shape, dev), workspace.numel(), handle)
    if st:
        _check(st, "moe_experts_forward")
    return out


@_scoped
def experts_backward(handle, dout, saved, plan, w_gate, w_up, w_down, activation: str = "swiglu", swiglu_limit=None,
                     swiglu_alpha: float = 1.702, out=None, workspace=None):
    """Gradients of experts_forward down to its rows, from dout [R, H] BF16 and saved, the forward pass's dict
    (g and u): a dict of drows [R, H] (for permute_tokens_backward) and dg, du [R, I] BF16, the
    gradients of g and u (relu2: du alone), which experts_weight_grad takes.  Rows behind the last
    expert's stay as they were.  stream: a torch.cuda.Stream to launch on."""
    flags = _activation_flag(activation, swiglu_limit)
    R, H, E, I = _experts_shapes(dout, "dout", plan, w_up, w_down)
    dev, gated = dout.get_device(), activation != "relu2"
    if out is None:
        out = {n: torch.empty(R, I, dtype=_BF16, device=dev) for n in (("dg", "du") if gated else ("du",))}
        out["drows"] = torch.empty_like(dout)
    if workspace is None:
        workspace = experts_workspace(0, I, dev)
    saved = _need(saved, "saved")
    st = lib().moe_experts_backward(
        _given(dout, "dout", _BF16, (R, H), dev), _offsets(plan, E, dev), R, E, H, I,
        _given(_need(w_gate, "w_gate"), "w_gate", _BF16, (E, I, H), dev) if gated else None,
        _given(w_up, "w_up", _BF16, (E, I, H), dev), _given(w_down, "w_down", _BF16, (E, H, I), dev), flags,
        0.0 if swiglu_limit is None else swiglu_limit, swiglu_alpha,
        _given(saved["g"], "g", _BF16, (R, I), dev) if gated else None, _given(saved["u"], "u", _BF16, (R, I), dev),
        _given(out["dg"], "dg", _BF16, (R, I), dev) if gated else None, _given(out["du"], "du", _BF16, (R, I), dev),
        _given(out["drows"], "drows", _BF16, (R, H), dev),
        _given(workspace, "workspace", _U8, workspace.shape, dev), workspace.numel(), handle)
    if st:
        _check(st, "moe_experts_backward")
    return out


@_scoped
def experts_weight_grad(handle, rows, dout, saved, grads, plan, accumulate: bool = False, out=None, workspace=None):
    """Gradients of the experts' weights, FP32: a dict of w_gate, w_up [E, I, H] and w_down [E, H, I].

    rows, dout [R, H] BF16: the forward pass's rows and the gradient of its out; saved: its dict (h);
    grads: experts_backward's (dg, du; without dg, as relu2 has none, there is no w_gate).  accumulate: added
    to out, the sums of earlier micro-batches, instead of taking its place.  stream: a torch.cuda.Stream to
    launch on."""
    if rows.dim() != 2 or _need(grads, "grads")["du"].dim() != 2:
        raise ValueError("rows must be [R, H] and du [R, I]")
    (R, H), I, dev = rows.shape, grads["du"].shape[1], rows.get_device()
    if H % 32 or I % 32 or H == 0 or I == 0:
        raise ValueError(f"H and I must be multiples of 32, got {H} and {I}")
    E = _need(_need(plan, "plan").get("offsets"), "plan['offsets']").numel() - 1
    gated = grads.get("dg") is not None
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out, the gradients to add to")
        out = {"w_up": torch.empty(E, I, H, dtype=_F32, device=dev), "w_down": torch.empty(E, H, I, dtype=_F32, device=dev)}
        if gated:
            out["w_gate"] = torch.empty(E, I, H, dtype=_F32, device=dev)
    if workspace is None:
        workspace = experts_workspace(0, I, dev)
    st = lib().moe_experts_weight_grad(
        _given(rows, "rows", _BF16, (R, H), dev), _given(_need(dout, "dout"), "dout", _BF16, (R, H), dev),
        _given(_need(saved, "saved")["h"], "h", _BF16, (R, I), dev),
        _given(grads["dg"], "dg", _BF16, (R, I), dev) if gated else None, _given(grads["du"], "du", _BF16, (R, I), dev),
        _offsets(plan, E, dev), R, E, H, I, (0 if gated else FLAG_ACT_RELU2) | (EXPERTS_ACCUMULATE if accumulate else 0),
        _given(out["w_gate"], "w_gate", _F32, (E, I, H), dev) if gated else None,
        _given(out["w_up"], "w_up", _F32, (E, I, H), dev), _given(out["w_down"], "w_down", _F32, (E, H, I), dev),
        _given(workspace, "workspace", _U8, workspace.shape, dev), workspace.numel(), handle)
    if st:
        _check(st, "moe_experts_weight_grad")
    return out


def last_device_status(workspace) -> int:
    st = C.c_int32(0)
    _check(lib().moe_last_device_status(_ptr(workspace), C.byref(st)), "moe_last_device_status")
    return int(st.value)


class MoeLayer:
    """Packed weights + a reusable workspace for one layer shape."""

    def __init__(self, cfg: MoeConfig, w_gate, w_up, w_down, shared=None, max_tokens=None):
        self.cfg = cfg
        self.device = w_up.device          # w_gate is None for non-gated (relu2) experts
        self.wbuf = quantize_weights(cfg, w_gate, w_up, w_down, shared)
        self._ws = None
        self._ws_T = -1
        if max_tokens:
            self._ensure_ws(max_tokens)

    def _ensure_ws(self, T):
        if self._ws is None or T > self._ws_T:
            self._ws = torch.empty(max(workspace_size(self.cfg, T), 256), dtype=torch.uint8,
                                   device=self.device)
            self._ws_T = T
        return self._ws

    def __call__(self, x, logits, y=None, debug=False):
        ws = self._ensure_ws(x.shape[0])
        return run(self.cfg, self.wbuf, x, logits, y=y, workspace=ws, debug=debug)

    def status(self) -> int:
        return last_device_status(self._ws)
