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
from .ops import BF16, BYTES, F32, I32, _check, _dev

EXPORTS = ("rope_axes", "nvfp4_kv_append", "nvfp4_kv_read", "nvfp4_attention_decode", "attention_prefill")

MAX_SLOTS = 2048  # NVFP4_ATTENTION_MAX_SLOTS
MAX_AXES = 4      # NVFP4_ROPE_MAX_AXES
_Sections = ctypes.c_int32 * MAX_AXES


def _load():
    lib = _ops.lib()
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    sig = {
        "rope_axes": [vp, i64, vp, i64, i64, i64, i64, vp, vp, vp, i32, i32, vp],
        "nvfp4_kv_append": [vp, i64, vp, i64, i64, i64, i64, vp, vp, vp, vp, i64, i64, vp],
        "nvfp4_kv_read": [vp, vp, vp, i64, i64, vp, i64, i64, i64, vp, i64, vp, i64, vp],
        "nvfp4_attention_decode": [vp, i64, i64, i64, i64, vp, vp, vp, i64, i64, i64, i64, vp, i64, vp, f32, vp, vp, vp, i64,
                                   vp],
        "attention_prefill": [vp, i64, vp, i64, vp, i64, i64, i64, i64, i64, i64, vp, vp, i64, f32, i32, vp, i64, vp, vp, i64, vp],
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


def attention_prefill_ws_bytes(tq, tk, q_heads, heads, b, d):
    """Workspace bytes that attention_prefill takes with these sizes: 0 where it needs none."""
    if min(tq, q_heads, heads, b) < 1 or tk // b < 1536:
        return 0
    keys = tk // b
    n = max(1, tq // b)
    tiles, packed = (n + 127) // 128 * q_heads, (n * (q_heads // heads) + 127) // 128 * heads
    most = 512 // (b * (packed if 20 * packed <= 19 * tiles else tiles))
    parts = min(keys // 256, most, 64, 66048 // (tq * q_heads)) if most >= 4 else 1
    return 0 if parts < 2 else parts * tq * q_heads * ((64 if d <= 64 else 128 if d <= 128 else 256) + 4) * 4


def _rows(x, name, i):
    """A bf16 tensor [t, heads, d] on GPU i whose heads lie one after the other: t, heads, d and its
    token stride."""
    try:
        if x.get_device() == i and x.dtype is BF16[0]:
            t, heads, d = x.shape
            s0, s1, s2 = x.stride()
            if (s2 == 1 or d == 1) and (s1 == d or heads == 1):
                return t, heads, d, s0 if t > 1 else heads * d
    except (AttributeError, ValueError, TypeError):
        pass
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError(f"{name} must be a tensor [t, heads, d], got {getattr(x, 'shape', type(x))}")
    if not x.is_cuda or x.get_device() != i or x.dtype is not BF16[0]:
        raise ValueError(f"{name} must be a bf16 tensor on GPU {i}, got {x.dtype} on {x.device}")
    raise ValueError(f"{name} must have its heads one after the other, got strides {x.stride()} of shape {tuple(x.shape)}")


def _gpu(x, name):
    """The tensor's GPU."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return x.get_device()


def _at(t, name, dtype, numel, i):
    """ops._dev by GPU index, with the common path in four calls: the tensor's pointer."""
    try:
        if t.get_device() == i and t.dtype is dtype[0] and t.is_contiguous() and t.numel() >= numel:
            return t.data_ptr()
    except AttributeError:
        pass
    return _dev(t, name, dtype, numel, torch.device("cuda", i)).data_ptr()


def _bytes(t, name, numel, i):
    try:
        if t.get_device() == i and t.element_size() == 1 and t.is_contiguous() and t.numel() >= numel:
            return t.data_ptr()
    except AttributeError:
        pass
    return _dev(t, name, BYTES, numel, torch.device("cuda", i)).data_ptr()


def _rows_as(x, name, i, shape):
    """The token stride of such a tensor of that shape."""
    t, heads, d, stride = _rows(x, name, i)
    if (t, heads, d) != shape:
        raise ValueError(f"{name} must be {shape}, got {tuple(x.shape)}")
    return stride


def _shaped(out, name, shape):
    if getattr(out, "shape", None) != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {getattr(out, 'shape', type(out))}")


_device, _stream_of = torch.cuda.current_device, torch._C._cuda_getCurrentRawStream


def _call(f, name, i, *args):
    """Calls the library with GPU i current (it launches on the current device) and its
    current stream.  (The raw handle: torch's Stream object costs 2 us a call.)"""
    if i == _device():
        rc = f(*args, _stream_of(i))
    else:
        with torch.cuda.device(i):
            rc = f(*args, _stream_of(i))
    if rc:
        _check(rc, name)


def rope_axes(x, positions, inv_freq, sections, interleaved=False, out=None):
    """Rotary positions with several axes.  x: [t, heads, d] bf16 (any stride from token to
    token); positions: [axes, t] int32; inv_freq: [sum(sections)] fp32; sections: the pairs of
    each axis; interleaved: pairs are (2i, 2i + 1) instead of (i, i + pairs).  Returns out (x
    itself for in place), with the elements past the pairs copied."""
    i = _gpu(x, "x")
    t, heads, d, stride = _rows(x, "x", i)
    axes = len(sections)
    if axes > MAX_AXES:
        raise ValueError(f"at most {MAX_AXES} axes, got {axes}")
    if out is None:
        out = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    out_stride = stride if out is x else _rows_as(out, "out", i, (t, heads, d))
    pos = _at(positions, "positions", I32, axes * t, i)
    if positions.shape != (axes, t):
        raise ValueError(f"positions must be [{axes}, {t}], got {tuple(positions.shape)}")
    _call(_lib.rope_axes, "rope_axes", i, x.data_ptr(), stride, out.data_ptr(), out_stride, t, heads, d, pos,
          _at(inv_freq, "inv_freq", F32, sum(sections), i), _Sections(*sections), axes, 1 if interleaved else 0)
    return out


def _cache(kv, kv_sf, kv_gs):
    """(GPU, pages, heads, page, d) of a cache and its pointers."""
    i = _gpu(kv, "kv")
    shape = kv.shape
    if len(shape) != 5 or shape[1] != 2:
        raise ValueError(f"kv must be [pages, 2, heads, page, d/2], got {tuple(shape)}")
    pages, _, heads, page, half = shape
    at = _bytes(kv, "kv", 0, i)
    if not isinstance(kv_sf, torch.Tensor) or kv_sf.shape != (pages, 2, heads, half // 8, page):
        raise ValueError(f"kv_sf must be [{pages}, 2, {heads}, {half // 8}, {page}] beside kv {tuple(kv.shape)}, got "
                         f"{tuple(kv_sf.shape) if isinstance(kv_sf, torch.Tensor) else type(kv_sf)}")
    return i, pages, heads, page, 2 * half, at, _bytes(kv_sf, "kv_sf", 0, i), _at(kv_gs, "kv_gs", F32, 2, i)


def nvfp4_kv_append(k, v, slots, kv_gs, kv, kv_sf):
    """Quantizes rows k, v [t, heads, d] bf16 into the cache's slots ([t] int32; negative: none).
    kv: [pages, 2, heads, page, d/2] bytes, kv_sf: [pages, 2, heads, d/16, page] bytes, kv_gs: [2]
    fp32 global scales of keys and values."""
    i, pages, heads, page, d, kv_at, sf_at, gs_at = _cache(kv, kv_sf, kv_gs)
    t, k_heads, k_d, ks = _rows(k, "k", i)
    if k_heads != heads or k_d != d:
        _shaped(k, "k", (t, heads, d))
    vs = _rows_as(v, "v", i, (t, heads, d))
    _call(_lib.nvfp4_kv_append, "nvfp4_kv_append", i, k.data_ptr(), ks, v.data_ptr(), vs, t, heads, d,
          _at(slots, "slots", I32, t, i), gs_at, kv_at, sf_at, pages, page)


def nvfp4_kv_read(slots, kv_gs, kv, kv_sf, k=None, v=None):
    """The cache's rows in slots [t] as bf16 (k, v) [t, heads, d].  Rows of negative slots are
    left as they were (zeros in tensors allocated here)."""
    i, pages, heads, page, d, kv_at, sf_at, gs_at = _cache(kv, kv_sf, kv_gs)
    slots_at = _at(slots, "slots", I32, 0, i)
    t = slots.numel()
    k = torch.zeros(t, heads, d, dtype=torch.bfloat16, device=kv.device) if k is None else k
    v = torch.zeros(t, heads, d, dtype=torch.bfloat16, device=kv.device) if v is None else v
    ks, vs = _rows_as(k, "k", i, (t, heads, d)), _rows_as(v, "v", i, (t, heads, d))
    _call(_lib.nvfp4_kv_read, "nvfp4_kv_read", i, kv_at, sf_at, gs_at, pages, page, slots_at, t, heads, d, k.data_ptr(),
          ks, v.data_ptr(), vs)
    return k, v


def nvfp4_attention_decode(q, kv, kv_sf, kv_gs, block_table, lengths, scale=None, out=None, lse=None, workspace=None):
    """Attention of t new tokens a sequence over the cache, which holds them already.  q: [b, t,
    q_heads, d] bf16 (any stride from token to token); block_table: [b, pages of a sequence] int32;
    lengths: [b] int32, the new tokens included; scale: d ** -0.5 when None; lse: None or [b, t,
    q_heads] fp32, written.  Token j sees the positions below lengths - (t - 1 - j).  workspace:
    attention_ws_bytes(b, d) bytes.  Returns out [b, t, q_heads, d] bf16."""
    i, pages, heads, page, d, kv_at, sf_at, gs_at = _cache(kv, kv_sf, kv_gs)
    if _gpu(q, "q") != i or q.dtype is not BF16[0] or q.dim() != 4 or q.shape[3] != d or heads < 1 or q.shape[2] % heads:
        raise ValueError(f"q must be bf16 [b, t, a multiple of {heads}, {d}] on GPU {i}, got {q.dtype} {tuple(q.shape)} on {q.device}")
    b, t, q_heads, _ = q.shape
    if q.is_contiguous():
        stride = q_heads * d
    else:
        s0, s1, s2, s3 = q.stride()
        stride = s1 if t > 1 else s0
        if s3 != 1 or (q_heads > 1 and s2 != d) or (t > 1 and b > 1 and s0 != t * s1):
            raise ValueError(f"q must have its heads one after the other and its tokens in even steps, got strides {q.stride()}")
        if b * t == 1:
            stride = q_heads * d
    table_at = _at(block_table, "block_table", I32, 0, i)
    if block_table.dim() != 2 or block_table.shape[0] != b:
        raise ValueError(f"block_table must be [{b}, pages], got {tuple(block_table.shape)}")
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    else:
        _shaped(out, "out", q.shape)
    need = attention_ws_bytes(b, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _call(_lib.nvfp4_attention_decode, "nvfp4_attention_decode", i, q.data_ptr(), stride, b, t, q_heads, kv_at, sf_at, gs_at, heads, d,
          pages, page, table_at, block_table.shape[1], _at(lengths, "lengths", I32, b, i), d ** -0.5 if scale is None else scale,
          _at(out, "out", BF16, 0, i), None if lse is None else _at(lse, "lse", F32, b * t * q_heads, i),
          _bytes(workspace, "workspace", need, i), workspace.numel())
    return out


def attention_prefill(q, k, v, cu_q, cu_k=None, causal=True, scale=None, out=None, lse=None, workspace=None):
    """Attention of packed prompts.  q: [tq, q_heads, d], k, v: [tk, heads, d] bf16, any strides from
    token to token; cu_q, cu_k: [b + 1] int32, where each sequence's rows and keys start (cu_k =
    cu_q when None); causal: row r of n rows and m keys sees the keys up to r + m - n, else all;
    scale: d ** -0.5 when None; lse: None or [tq, q_heads] fp32, written; workspace:
    attention_prefill_ws_bytes bytes, where few rows meet many keys.  Returns out [tq, q_heads, d]
    bf16; rows outside all sequences are left as they were (zeros in an out allocated here)."""
    i = _gpu(q, "q")
    tq, q_heads, d, qs = _rows(q, "q", i)
    tk, heads, dk, ks = _rows(k, "k", i)
    tv, v_heads, dv, vs = _rows(v, "v", i)
    if dk != d or tv != tk or v_heads != heads or dv != d or heads < 1 or q_heads % heads:
        raise ValueError(f"k / v must be [tk, heads, {d}] with heads a divisor of {q_heads}, got {tuple(k.shape)} / "
                         f"{tuple(v.shape)}")
    cu_at = _at(cu_q, "cu_q", I32, 0, i)
    b = cu_q.numel() - 1
    if out is None:
        out = torch.zeros(tq, q_heads, d, dtype=torch.bfloat16, device=q.device)
    out_stride = _rows_as(out, "out", i, (tq, q_heads, d))
    ws, need = None, attention_prefill_ws_bytes(tq, tk, q_heads, heads, b, d)
    if need:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        ws, need = _bytes(workspace, "workspace", need, i), workspace.numel()
    _call(_lib.attention_prefill, "attention_prefill", i, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, tq, tk, q_heads,
          heads, d, cu_at, cu_at if cu_k is None else _at(cu_k, "cu_k", I32, b + 1, i), b, d ** -0.5 if scale is None else scale,
          1 if causal else 0, out.data_ptr(), out_stride, None if lse is None else _at(lse, "lse", F32, tq * q_heads, i),
          ws, need)
    return out
