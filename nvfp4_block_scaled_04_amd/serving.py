"""Thin Python binding of the serving operators (include/nvfp4_serving.h): a
whole mixture-of-experts layer for a few tokens, and low-rank adapters of many
requests beside a shared NVFP4 projection.

As in ops.py, torch supplies device memory and the current HIP stream, every
tensor is checked before the library sees its pointer, and every step of the
computation runs in the library's kernels.  Outputs and workspaces left as None
are allocated here with torch.
"""
import ctypes

import torch

from . import ops as _ops
from .ops import BF16, BYTES, F32, I32, _check, _dev, _dims, _opt, _ptr, _stream, sf_size

EXPORTS = ("nvfp4_moe_small", "nvfp4_linear_adapters", "nvfp4_gemm_adapters")

SCORES = {"softmax": 0, "sigmoid": 1}   # nvfp4_route_score
_LOGITS = (torch.bfloat16, torch.float32)


def _load():
    lib = _ops.lib()
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    sig = {
        "nvfp4_moe_small": [vp, i64, i64, vp, i32, i64, i64, i32, i32, vp, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp,
                            i64, vp],
        "nvfp4_linear_adapters": [vp] * 10 + [i64] * 5 + [vp, i64, vp],
        "nvfp4_gemm_adapters": [vp] * 12 + [i64] * 5 + [vp, i64, vp],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    return lib


_lib = _load()


def moe_small_ws_bytes(t, top_k, h, inter):
    """NVFP4_MOE_SMALL_WS_BYTES: workspace bytes of nvfp4_moe_small."""
    return 4 * t * top_k * inter + 4096 + (4096 * 4 + 1) * ((h + 127) // 128 * 32)


def adapters_ws_bytes(m, r, split=False):
    """NVFP4_ADAPTERS_WS_BYTES: workspace bytes of the adapter calls; with split,
    also room for the partial sums of products spread over more workgroups."""
    return (m * r * 4 + 255) // 256 * 256 + (_ops.GEMM_WS_BYTES if split else 0)


def _workspace(workspace, need, dev):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    _dev(workspace, "workspace", BYTES, need, dev)
    return workspace


def nvfp4_moe_small(x, logits, w13, w13_sf, alpha13, w2, w2_sf, alpha2, top_k, score="softmax", renormalize=True,
                    out=None, topk_ids=None, topk_weights=None, workspace=None):
    """A whole mixture-of-experts layer for t <= 64 tokens.  x: [t, h] bf16;
    logits: [t, E] fp32 or bf16 (the router's); w13: [E, 2*inter, h/2] packed FP4
    (gate rows, then up rows), w2: [E, h, inter/2], with their swizzled scales and
    alpha [E] = 1 / global scale each; score: "softmax" or "sigmoid"; renormalize:
    divide a token's weights by their sum.  A logit of NaN or -inf is never
    chosen.  Returns (out [t, h] bf16, topk_ids [t, top_k] int32, -1 in slots left
    over, topk_weights [t, top_k] fp32)."""
    _dims(x, "x", 2)
    _dims(logits, "logits", 2)
    _dims(w13, "w13", 3)
    _dims(w2, "w2", 3)
    t, h = x.shape
    E = logits.shape[1]
    inter = w2.shape[2] * 2
    dev = x.device
    if score not in SCORES:
        raise ValueError(f"score must be one of {tuple(SCORES)}, got {score!r}")
    if logits.shape[0] != t:
        raise ValueError(f"logits must be [{t}, E], got {tuple(logits.shape)}")
    if w13.shape != (E, 2 * inter, h // 2) or w2.shape != (E, h, inter // 2) or h % 2:
        raise ValueError(f"w13 / w2 must be [E, 2*inter, h/2] / [E, h, inter/2] with E = {E}, h = {h}, got "
                         f"{tuple(w13.shape)} / {tuple(w2.shape)}")
    k = int(top_k)
    if out is None:
        out = torch.empty(t, h, dtype=torch.bfloat16, device=dev)
    if topk_ids is None:
        topk_ids = torch.empty(t, max(k, 0), dtype=torch.int32, device=dev)
    if topk_weights is None:
        topk_weights = torch.empty(t, max(k, 0), dtype=torch.float32, device=dev)
    workspace = _workspace(workspace, moe_small_ws_bytes(t, k, h, inter), dev)
    _dev(x, "x", BF16, t * h, dev)
    _dev(logits, "logits", _LOGITS, t * E, dev)
    _dev(w13, "w13", BYTES, E * inter * h, dev)
    _dev(w13_sf, "w13_sf", BYTES, E * sf_size(2 * inter, h), dev)
    _dev(alpha13, "alpha13", F32, E, dev)
    _dev(w2, "w2", BYTES, E * h * (inter // 2), dev)
    _dev(w2_sf, "w2_sf", BYTES, E * sf_size(h, inter), dev)
    _dev(alpha2, "alpha2", F32, E, dev)
    _dev(out, "out", BF16, t * h, dev)
    _dev(topk_ids, "topk_ids", I32, t * k, dev)
    _dev(topk_weights, "topk_weights", F32, t * k, dev)
    rc = _lib.nvfp4_moe_small(x.data_ptr(), t, h, logits.data_ptr(), 0 if logits.dtype is torch.bfloat16 else 1, E, k,
                              SCORES[score], 1 if renormalize else 0, w13.data_ptr(), w13_sf.data_ptr(),
                              alpha13.data_ptr(), w2.data_ptr(), w2_sf.data_ptr(), alpha2.data_ptr(), inter,
                              out.data_ptr(), topk_ids.data_ptr(), topk_weights.data_ptr(), workspace.data_ptr(),
                              workspace.numel(), _stream(dev))
    _check(rc, "nvfp4_moe_small")
    return out, topk_ids, topk_weights


def _adapters(x, lora_a, lora_b, adapter, scaling, bias, n):
    """Checks of the adapters' own tensors; returns (m, k, r, n_adapters)."""
    _dims(x, "x", 2)
    _dims(lora_a, "lora_a", 3)
    _dims(lora_b, "lora_b", 3)
    m, k = x.shape
    L, r = lora_a.shape[0], lora_a.shape[1]
    dev = x.device
    if lora_a.shape[2] != k or lora_b.shape != (L, n, r):
        raise ValueError(f"lora_a / lora_b must be [L, r, {k}] / [L, {n}, r], got {tuple(lora_a.shape)} / "
                         f"{tuple(lora_b.shape)}")
    _dev(x, "x", BF16, m * k, dev)
    _dev(lora_a, "lora_a", BF16, L * r * k, dev)
    _dev(lora_b, "lora_b", BF16, L * n * r, dev)
    _dev(adapter, "adapter", I32, m, dev)
    _opt(scaling, "scaling", F32, L, dev)
    _opt(bias, "bias", BF16, n, dev)
    return m, k, r, L


def nvfp4_linear_adapters(x, b, b_sf, alpha, lora_a, lora_b, adapter, scaling=None, bias=None, out=None,
                          workspace=None):
    """x: [m, k] bf16, b: [n, k/2] packed FP4 weight (alpha = 1 / its global
    scale), lora_a: [L, r, k] and lora_b: [L, n, r] bf16, adapter: [m] int32 (a
    row's adapter; outside [0, L): none), scaling: [L] fp32 or None -> out [m, n]
    bf16 = alpha * x @ dequant(b)^T + scaling * (x @ lora_a^T) @ lora_b^T (+bias).
    For decode (few rows); each row has its own adapter, in any order.  workspace:
    adapters_ws_bytes(m, r, split=True) bytes (allocated when None), or without
    split, where few workgroups then walk the whole K axis."""
    _dims(b, "b", 2)
    n = b.shape[0]
    m, k, r, L = _adapters(x, lora_a, lora_b, adapter, scaling, bias, n)
    dev = x.device
    if b.shape[1] * 2 != k:
        raise ValueError(f"b must be [n, {k // 2}] packed FP4, got {tuple(b.shape)}")
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=dev)
    workspace = _workspace(workspace, adapters_ws_bytes(m, r, workspace is None), dev)
    _dev(b, "b", BYTES, n * (k // 2), dev)
    _dev(b_sf, "b_sf", BYTES, sf_size(n, k), dev)
    _dev(alpha, "alpha", F32, 1, dev)
    _dev(out, "out", BF16, m * n, dev)
    rc = _lib.nvfp4_linear_adapters(x.data_ptr(), b.data_ptr(), b_sf.data_ptr(), alpha.data_ptr(), lora_a.data_ptr(),
                                    lora_b.data_ptr(), adapter.data_ptr(), _ptr(scaling), _ptr(bias), out.data_ptr(),
                                    m, n, k, r, L, workspace.data_ptr(), workspace.numel(), _stream(dev))
    _check(rc, "nvfp4_linear_adapters")
    return out


def nvfp4_gemm_adapters(a, b, a_sf, b_sf, alpha, x, lora_a, lora_b, adapter, scaling=None, bias=None, out=None,
                        workspace=None):
    """The same beside the block-scaled NVFP4 product, for prefill: a: [m, k/2]
    and a_sf, the quantized x, with alpha = 1 / (gs_a * gs_b); x: [m, k] bf16 for
    the adapters.  With a workspace of adapters_ws_bytes(m, r, split=True) bytes
    (as by default) the GEMM takes the split-tail schedule."""
    _dims(a, "a", 2)
    _dims(b, "b", 2)
    n = b.shape[0]
    m, k, r, L = _adapters(x, lora_a, lora_b, adapter, scaling, bias, n)
    dev = x.device
    if a.shape != (m, k // 2) or b.shape[1] * 2 != k:
        raise ValueError(f"a / b must be [{m}, {k // 2}] / [n, {k // 2}] packed FP4, got {tuple(a.shape)} / "
                         f"{tuple(b.shape)}")
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=dev)
    workspace = _workspace(workspace, adapters_ws_bytes(m, r, workspace is None), dev)
    _ops._operands(a, b, a_sf, b_sf, 1, m, n, k, dev, sf_size)
    _dev(alpha, "alpha", F32, 1, dev)
    _dev(out, "out", BF16, m * n, dev)
    rc = _lib.nvfp4_gemm_adapters(a.data_ptr(), b.data_ptr(), a_sf.data_ptr(), b_sf.data_ptr(), alpha.data_ptr(),
                                  x.data_ptr(), lora_a.data_ptr(), lora_b.data_ptr(), adapter.data_ptr(),
                                  _ptr(scaling), _ptr(bias), out.data_ptr(), m, n, k, r, L, workspace.data_ptr(),
                                  workspace.numel(), _stream(dev))
    _check(rc, "nvfp4_gemm_adapters")
    return out
