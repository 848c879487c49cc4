"""Thin Python binding of the attention operators (include/nvfp4_attention.h): rotary
positions with several axes, a paged cache of keys and values in NVFP4, attention of
single tokens over it, and attention of whole prompts.

As in ops.py, torch supplies device memory and the current HIP stream, every tensor
is checked before the library sees its pointer, and every step of the computation
runs in the library's kernels.  Outputs and workspaces left as None are allocated
here with torch.
"""
import ctypes

import torch

from . import ops as _ops
from .ops import BF16, BYTES, F32, I32, _check, _dev, _dims, _need, _opt, _ptr, _stream

EXPORTS = ("rope_axes", "nvfp4_kv_append", "nvfp4_kv_read", "nvfp4_attention_decode", "attention_prefill")

MAX_SLOTS = 1024  # NVFP4_ATTENTION_MAX_SLOTS


def _load():
    lib = _ops.lib()
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    sig = {
        "rope_axes": [vp, i64, vp, i64, i64, i64, i64, vp, vp, vp, i32, i32, vp],
        "nvfp4_kv_append": [vp, i64, vp, i64, i64, i64, i64, vp, vp, vp, vp, i64, i64, vp],
        "nvfp4_kv_read": [vp, vp, vp, i64, i64, vp, i64, i64, i64, vp, i64, vp, i64, vp],
        "nvfp4_attention_decode": [vp, i64, i64, i64, vp, vp, vp, i64, i64, i64, i64, vp, i64, vp, f32, vp, vp, vp, i64,
                                   vp],
        "attention_prefill": [vp, i64, vp, i64, vp, i64, i64, i64, i64, i64, i64, vp, vp, i64, f32, i32, vp, i64, vp, vp],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    return lib


_lib = _load()


def attention_ws_bytes(b, d):
    """NVFP4_ATTENTION_WS_BYTES: workspace bytes of nvfp4_attention_decode."""
    return (8 * b + 255) // 256 * 256 + MAX_SLOTS * 64 * ((64 if d <= 64 else 128 if d <= 128 else 256) + 2)


def _rows(x, name, device=None):
    """A bf16 tensor [t, heads, d] whose heads lie one after the other: its token stride."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError(f"{name} must be a tensor [t, heads, d], got {getattr(x, 'shape', type(x))}")
    t, heads, d = x.shape
    s0, s1, s2 = x.stride()
    if not x.is_cuda or x.dtype is not torch.bfloat16 or (device is not None and x.device != device):
        raise ValueError(f"{name} must be a bf16 tensor on {device or 'the GPU'}, got {x.dtype} on {x.device}")
    if (d > 1 and s2 != 1) or (heads > 1 and s1 != d):
        raise ValueError(f"{name} must have its heads one after the other, got strides {(s0, s1, s2)} of shape {(t, heads, d)}")
    return s0 if t > 1 else heads * d


def _out(out, name, shape, device):
    if out is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=device)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(out.shape)}")
    return out


def _call(name, dev, *args):
    """The library launches on the current device, so that has to be the tensors'."""
    if dev.index == torch.cuda.current_device():
        rc = getattr(_lib, name)(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = getattr(_lib, name)(*args, _stream(dev))
    _check(rc, name)


def rope_axes(x, positions, inv_freq, sections, interleaved=False, out=None):
    """Rotary positions with several axes.  x: [t, heads, d] bf16 (any stride from token to
    token); positions: [axes, t] int32; inv_freq: [sum(sections)] fp32; sections: the pairs of
    each axis; interleaved: pairs are (2i, 2i + 1) instead of (i, i + pairs).  Returns out (x
    itself for in place), with the elements past the pairs copied."""
    stride = _rows(x, "x")
    dev = x.device
    t, heads, d = x.shape
    axes = len(sections)
    out = _out(out, "out", x.shape, dev)
    _dev(positions, "positions", I32, axes * t, dev)
    if positions.dim() != 2 or tuple(positions.shape) != (axes, t):
        raise ValueError(f"positions must be [{axes}, {t}], got {tuple(positions.shape)}")
    _dev(inv_freq, "inv_freq", F32, sum(sections), dev)
    host = (ctypes.c_int32 * max(axes, 1))(*sections)
    _call("rope_axes", dev, x.data_ptr(), stride, out.data_ptr(), _rows(out, "out", dev), t, heads, d,
          positions.data_ptr(), inv_freq.data_ptr(), host, axes, 1 if interleaved else 0)
    return out


def _cache(kv, kv_sf, kv_gs):
    """(pages, heads, page, d) of a cache."""
    _dims(kv, "kv", 5)
    _dims(kv_sf, "kv_sf", 5)
    pages, two, heads, page, half = kv.shape
    dev = kv.device
    if two != 2 or tuple(kv_sf.shape) != (pages, 2, heads, half // 8, page):
        raise ValueError(f"kv / kv_sf must be [pages, 2, heads, page, d/2] / [pages, 2, heads, d/16, page], got "
                         f"{tuple(kv.shape)} / {tuple(kv_sf.shape)}")
    _dev(kv, "kv", BYTES, kv.numel(), dev)
    _dev(kv_sf, "kv_sf", BYTES, kv_sf.numel(), dev)
    _dev(kv_gs, "kv_gs", F32, 2, dev)
    return pages, heads, page, 2 * half


def nvfp4_kv_append(k, v, slots, kv_gs, kv, kv_sf):
    """Quantizes rows k, v [t, heads, d] bf16 into the cache's slots ([t] int32; negative: none).
    kv: [pages, 2, heads, page, d/2] bytes, kv_sf: [pages, 2, heads, d/16, page] bytes, kv_gs: [2]
    fp32 global scales of keys and values."""
    pages, heads, page, d = _cache(kv, kv_sf, kv_gs)
    dev = kv.device
    ks, vs = _rows(k, "k", dev), _rows(v, "v", dev)
    t = k.shape[0]
    if tuple(k.shape) != (t, heads, d) or tuple(v.shape) != (t, heads, d):
        raise ValueError(f"k / v must be [t, {heads}, {d}], got {tuple(k.shape)} / {tuple(v.shape)}")
    _dev(slots, "slots", I32, t, dev)
    _call("nvfp4_kv_append", dev, k.data_ptr(), ks, v.data_ptr(), vs, t, heads, d, slots.data_ptr(), kv_gs.data_ptr(),
          kv.data_ptr(), kv_sf.data_ptr(), pages, page)


def nvfp4_kv_read(slots, kv_gs, kv, kv_sf, k=None, v=None):
    """The cache's rows in slots [t] as bf16 (k, v) [t, heads, d].  Rows of negative slots are
    left as they were (zeros in tensors allocated here)."""
    pages, heads, page, d = _cache(kv, kv_sf, kv_gs)
    dev = kv.device
    _need(slots, "slots")
    t = slots.numel()
    shape = (t, heads, d)
    k = torch.zeros(shape, dtype=torch.bfloat16, device=dev) if k is None else _out(k, "k", shape, dev)
    v = torch.zeros(shape, dtype=torch.bfloat16, device=dev) if v is None else _out(v, "v", shape, dev)
    _dev(slots, "slots", I32, t, dev)
    _call("nvfp4_kv_read", dev, kv.data_ptr(), kv_sf.data_ptr(), kv_gs.data_ptr(), pages, page, slots.data_ptr(), t,
          heads, d, k.data_ptr(), _rows(k, "k", dev), v.data_ptr(), _rows(v, "v", dev))
    return k, v


def nvfp4_attention_decode(q, kv, kv_sf, kv_gs, block_table, lengths, scale=None, out=None, lse=None, workspace=None):
    """Attention of t new tokens a sequence over the cache, which holds them already.  q: [b, t,
    q_heads, d] bf16; block_table: [b, pages of a sequence] int32; lengths: [b] int32, the new
    tokens included; scale: d ** -0.5 when None; lse: None or [b, t, q_heads] fp32, written.
    Token j sees the positions below lengths - (t - 1 - j).  workspace: attention_ws_bytes(b, d)
    bytes.  Returns out [b, t, q_heads, d] bf16."""
    pages, heads, page, d = _cache(kv, kv_sf, kv_gs)
    dev = kv.device
    _dims(q, "q", 4)
    _dims(block_table, "block_table", 2)
    b, t, q_heads = q.shape[:3]
    if q.shape[3] != d or heads < 1 or q_heads % heads:
        raise ValueError(f"q must be [b, t, a multiple of {heads}, {d}], got {tuple(q.shape)}")
    if block_table.shape[0] != b:
        raise ValueError(f"block_table must be [{b}, pages], got {tuple(block_table.shape)}")
    out = _out(out, "out", q.shape, dev)
    need = attention_ws_bytes(b, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _dev(workspace, "workspace", BYTES, need, dev)
    _dev(q, "q", BF16, q.numel(), dev)
    _dev(out, "out", BF16, q.numel(), dev)
    _dev(block_table, "block_table", I32, 0, dev)
    _dev(lengths, "lengths", I32, b, dev)
    _opt(lse, "lse", F32, b * t * q_heads, dev)
    _call("nvfp4_attention_decode", dev, q.data_ptr(), b, t, q_heads, kv.data_ptr(), kv_sf.data_ptr(), kv_gs.data_ptr(),
          heads, d, pages, page, block_table.data_ptr(), block_table.shape[1], lengths.data_ptr(),
          d ** -0.5 if scale is None else scale, out.data_ptr(), _ptr(lse), workspace.data_ptr(), workspace.numel())
    return out


def attention_prefill(q, k, v, cu_q, cu_k=None, causal=True, scale=None, out=None, lse=None):
    """Attention of packed prompts.  q: [tq, q_heads, d], k, v: [tk, heads, d] bf16, any strides from
    token to token; cu_q, cu_k: [b + 1] int32, where each sequence's rows and keys start (cu_k =
    cu_q when None); causal: row r of n rows and m keys sees the keys up to r + m - n, else all;
    scale: d ** -0.5 when None; lse: None or [tq, q_heads] fp32, written.  Returns out [tq, q_heads,
    d] bf16; rows outside all sequences are left as they were (zeros in an out allocated here)."""
    qs = _rows(q, "q")
    dev = q.device
    ks, vs = _rows(k, "k", dev), _rows(v, "v", dev)
    tq, q_heads, d = q.shape
    tk, heads = k.shape[:2]
    if k.shape[2] != d or v.shape != k.shape or heads < 1 or q_heads % heads:
        raise ValueError(f"k / v must be [tk, heads, {d}] with heads a divisor of {q_heads}, got {tuple(k.shape)} / "
                         f"{tuple(v.shape)}")
    if cu_k is None:
        cu_k = cu_q
    _dims(cu_q, "cu_q", 1)
    b = cu_q.numel() - 1
    if out is None:
        out = torch.zeros(tq, q_heads, d, dtype=torch.bfloat16, device=dev)
    _out(out, "out", q.shape, dev)
    _dev(cu_q, "cu_q", I32, b + 1, dev)
    _dev(cu_k, "cu_k", I32, b + 1, dev)
    _opt(lse, "lse", F32, tq * q_heads, dev)
    _call("attention_prefill", dev, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, tq, tk, q_heads, heads, d,
          cu_q.data_ptr(), cu_k.data_ptr(), b, d ** -0.5 if scale is None else scale, 1 if causal else 0, out.data_ptr(),
          _rows(out, "out", dev), _ptr(lse))
    return out
