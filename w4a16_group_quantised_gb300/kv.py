"""ctypes binding of the paged 8-bit key/value cache (argument marshalling only).

Every function has the name of the C entry point it calls and the semantics
include/w4a16.h states; tensors' data pointers and the current CUDA stream are
handed over unchanged.  Scratch is allocated per call on that stream unless
the caller passes a workspace.

A cache is a KVCache of four tensors.  Its codes are [n_pages, n_kv_heads,
page_size, head_dim] in that order of dimensions, int8 or float8_e4m3fn, with
any strides that keep head_dim contiguous (a permuted [n_pages, page_size,
n_kv_heads, head_dim] tensor is as good); its scales are float32 [n_pages,
n_kv_heads].
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

from .binding import _check, _dtype_code, _p, _stream_ptr, load_library

KV_INT8, KV_E4M3 = 0, 1


class KVCache(NamedTuple):
    """Codes and scales of a paged cache (see the module's docstring)."""
    k: "torch.Tensor"         # noqa: F821
    v: "torch.Tensor"         # noqa: F821
    k_scale: "torch.Tensor"   # noqa: F821
    v_scale: "torch.Tensor"   # noqa: F821


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("page_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong), ("token_stride", ctypes.c_longlong), ("kv_dtype", ctypes.c_int)]


class _Batch(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("q_starts", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int), ("max_blocks", ctypes.c_int), ("n_tokens", ctypes.c_int)]


def _tensor(name, t, dtype=None, dim=None, contiguous=True):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor, got device {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must be {dim}-D, got {list(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _one_device(*tensors):
    devs = {t.device for t in tensors if t is not None}
    if len(devs) > 1:
        raise ValueError(f"operands are on different devices: {sorted(map(str, devs))}")


def _cache(c):
    """The cache as the C struct; TypeError / ValueError for what it cannot be."""
    import torch
    if not isinstance(c, KVCache):
        raise TypeError(f"cache must be a KVCache, got {type(c).__name__}")
    k, v = _tensor("cache.k", c.k, dim=4, contiguous=False), _tensor("cache.v", c.v, dim=4, contiguous=False)
    if k.dtype == torch.int8:
        kind = KV_INT8
    elif k.dtype == torch.float8_e4m3fn:
        kind = KV_E4M3
    else:
        raise TypeError(f"cache.k must be int8 or float8_e4m3fn, got {k.dtype}")
    if v.dtype != k.dtype or v.shape != k.shape or v.stride() != k.stride():
        raise ValueError("cache.k and cache.v must have the same dtype, shape and strides")
    n_pages, heads, page_size, head_dim = k.shape
    sp, sh, st, sd = k.stride()
    if sd != 1:
        raise ValueError("the codes' last dimension must be contiguous")
    for name, t in (("cache.k_scale", c.k_scale), ("cache.v_scale", c.v_scale)):
        _tensor(name, t, torch.float32, 2)
        if t.shape[0] != n_pages or t.shape[1] != heads:
            raise ValueError(f"{name} must be [{n_pages}, {heads}], got {list(t.shape)}")
    _one_device(k, v, c.k_scale, c.v_scale)
    return _Cache(k.data_ptr(), v.data_ptr(), c.k_scale.data_ptr(), c.v_scale.data_ptr(), n_pages, page_size, heads,
                  head_dim, sp, sh, st, kind)


def _table(block_table, kv_lens):
    import torch
    _tensor("block_table", block_table, torch.int32, 2)
    _tensor("kv_lens", kv_lens, torch.int32, 1)
    if block_table.shape[0] != kv_lens.shape[0]:
        raise ValueError(f"block_table has {block_table.shape[0]} rows, kv_lens {kv_lens.shape[0]}")
    _one_device(block_table, kv_lens)


def _batch(block_table, kv_lens, q_starts, n_tokens, device):
    import torch
    _table(block_table, kv_lens)
    _tensor("q_starts", q_starts, torch.int32, 1)
    n = kv_lens.shape[0]
    if q_starts.shape[0] != n + 1:
        raise ValueError(f"q_starts must be [n_seqs + 1] = [{n + 1}], got {list(q_starts.shape)}")
    if block_table.device != device or q_starts.device != device:
        raise ValueError("block_table, kv_lens and q_starts must be on the cache's device")
    return _Batch(block_table.data_ptr(), kv_lens.data_ptr(), q_starts.data_ptr(), n, block_table.shape[1], n_tokens)


def _rows(name, t, heads, head_dim, device):
    """Row stride of a [tokens, heads, head_dim] tensor whose rows are dense."""
    _tensor(name, t, dim=3, contiguous=False)
    if t.shape[1] != heads or t.shape[2] != head_dim:
        raise ValueError(f"{name} must be [n_tokens, {heads}, {head_dim}], got {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on the cache's device")
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != head_dim):
        raise ValueError(f"each row of {name} must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), heads * head_dim)


def _scratch(workspace, need, device, stream):
    import torch
    if workspace is None:
        workspace = torch.empty(max(16, need), dtype=torch.uint8, device=device)
        if stream is not None:
            workspace.record_stream(stream)
    else:
        _tensor("workspace", workspace)
        if workspace.device != device:
            raise ValueError("workspace must be on the cache's device")
    return workspace, workspace.numel() * workspace.element_size()


def w4a16_kv_append(cache, k_new, v_new, block_table, kv_lens, q_starts, stream=None):
    """Quantise k_new, v_new [n_tokens, n_kv_heads, head_dim] (fp16/bf16, rows
    may be strided views) into the cache as each sequence's newest tokens:
    positions kv_lens[b] - (q_starts[b+1] - q_starts[b]) .. kv_lens[b] - 1."""
    c = _cache(cache)
    dev = cache.k.device
    sk = _rows("k_new", k_new, c.n_kv_heads, c.head_dim, dev)
    sv = _rows("v_new", v_new, c.n_kv_heads, c.head_dim, dev)
    if v_new.dtype != k_new.dtype or v_new.shape != k_new.shape:
        raise ValueError("k_new and v_new must have the same dtype and shape")
    dt = _dtype_code(k_new)
    b = _batch(block_table, kv_lens, q_starts, k_new.shape[0], dev)
    _check("w4a16_kv_append", load_library().w4a16_kv_append(
        ctypes.byref(c), _p(k_new), sk, _p(v_new), sv, ctypes.byref(b), dt, _stream_ptr(stream)))


def w4a16_kv_read(cache, block_table, kv_lens, q_starts, n_tokens: int, dtype, k_out=None, v_out=None, stream=None):
    """The newest q_starts[b+1] - q_starts[b] cached tokens of each sequence as
    values of `dtype`: (k, v), each [n_tokens, n_kv_heads, head_dim]."""
    import torch
    c = _cache(cache)
    dev = cache.k.device
    shape = (n_tokens, c.n_kv_heads, c.head_dim)
    outs = []
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=dev)
        else:
            _tensor(name, t, dtype, 3)
            if tuple(t.shape) != shape or t.device != dev:
                raise ValueError(f"{name} must be {list(shape)} on the cache's device")
        outs.append(t)
    b = _batch(block_table, kv_lens, q_starts, n_tokens, dev)
    _check("w4a16_kv_read", load_library().w4a16_kv_read(
        ctypes.byref(c), ctypes.byref(b), _p(outs[0]), _p(outs[1]), _dtype_code(outs[0]), _stream_ptr(stream)))
    return outs[0], outs[1]


def w4a16_kv_attention(q, cache, block_table, kv_lens, q_starts, max_q_len: int, scale=None, window: int = 0,
                       sinks: int = 0, out=None, lse=None, workspace=None, stream=None):
    """Causal attention of q [n_tokens, n_heads, head_dim] over the cache, with
    an optional sliding window (0: none) and sink tokens; out [n_tokens,
    n_heads, head_dim].  scale defaults to head_dim ** -0.5; lse, if given, is
    float32 [n_tokens, n_heads] and receives the log-sum-exp of each row."""
    import torch
    c = _cache(cache)
    dev = cache.k.device
    _tensor("q", q, dim=3, contiguous=False)
    T, H = q.shape[0], q.shape[1]
    sq = _rows("q", q, H, c.head_dim, dev)
    dt = _dtype_code(q)
    if out is None:
        out = torch.empty((T, H, c.head_dim), dtype=q.dtype, device=dev)
    else:
        _tensor("out", out, q.dtype, 3)
        if out.shape != q.shape or out.device != dev:
            raise ValueError(f"out must be {list(q.shape)} on the cache's device")
    if lse is not None:
        _tensor("lse", lse, torch.float32, 2)
        if lse.shape[0] != T or lse.shape[1] != H or lse.device != dev:
            raise ValueError(f"lse must be [{T}, {H}] on the cache's device")
    b = _batch(block_table, kv_lens, q_starts, T, dev)
    lib = load_library()
    need = ctypes.c_longlong(0)
    _check("w4a16_kv_attention_workspace", lib.w4a16_kv_attention_workspace(
        H, c.n_kv_heads, c.head_dim, b.n_seqs, T, ctypes.byref(need)))
    ws, size = _scratch(workspace, need.value, dev, stream)
    _check("w4a16_kv_attention", lib.w4a16_kv_attention(
        _p(q), sq, H, ctypes.byref(c), ctypes.byref(b), max_q_len, c.head_dim ** -0.5 if scale is None else scale,
        window, sinks, _p(out), _p(lse), dt, _p(ws), size, _stream_ptr(stream)))
    return out


def w4a16_kv_attention_workspace(n_heads: int, n_kv_heads: int, head_dim: int, n_seqs: int, n_tokens: int) -> int:
    """Bytes of workspace that w4a16_kv_attention needs for these sizes, whatever the lengths."""
    need = ctypes.c_longlong(0)
    _check("w4a16_kv_attention_workspace", load_library().w4a16_kv_attention_workspace(
        n_heads, n_kv_heads, head_dim, n_seqs, n_tokens, ctypes.byref(need)))
    return need.value


def _ids(name, t, device):
    import torch
    _tensor(name, t, torch.int32, 1)
    if t.device != device:
        raise ValueError(f"{name} must be on the cache's device")
    return t.shape[0]


def _refcount(refcount, device, n_pages=None):
    import torch
    _tensor("refcount", refcount, torch.int32, 1)
    if refcount.device != device:
        raise ValueError("refcount must be on the cache's device")
    if n_pages is not None and refcount.shape[0] != n_pages:
        raise ValueError(f"refcount must be [n_pages] = [{n_pages}], got {list(refcount.shape)}")


def w4a16_kv_copy_pages(cache, src, dst, stream=None):
    """Pages src[i] (codes and scales) copied to pages dst[i]; pairs with a negative id are skipped."""
    c = _cache(cache)
    n = _ids("src", src, cache.k.device)
    if _ids("dst", dst, cache.k.device) != n:
        raise ValueError("src and dst must have the same length")
    _check("w4a16_kv_copy_pages", load_library().w4a16_kv_copy_pages(
        ctypes.byref(c), _p(src), _p(dst), n, _stream_ptr(stream)))


def w4a16_kv_pool_workspace(n_pages: int) -> int:
    """Bytes of workspace that w4a16_kv_fork and w4a16_kv_compact need."""
    need = ctypes.c_longlong(0)
    _check("w4a16_kv_pool_workspace", load_library().w4a16_kv_pool_workspace(n_pages, ctypes.byref(need)))
    return need.value


def w4a16_kv_fork(cache, block_table, kv_lens, refcount, parents, children, workspace=None, stream=None):
    """Rows children[i] of the table continue rows parents[i]: full pages are
    shared, a partly filled last page is copied into the lowest free page."""
    c = _cache(cache)
    dev = cache.k.device
    _table(block_table, kv_lens)
    _one_device(cache.k, block_table)
    _refcount(refcount, dev, c.n_pages)
    n = _ids("parents", parents, dev)
    if _ids("children", children, dev) != n:
        raise ValueError("parents and children must have the same length")
    ws, size = _scratch(workspace, w4a16_kv_pool_workspace(c.n_pages), dev, stream)
    _check("w4a16_kv_fork", load_library().w4a16_kv_fork(
        ctypes.byref(c), _p(block_table), _p(kv_lens), block_table.shape[0], block_table.shape[1], _p(refcount),
        _p(parents), _p(children), n, _p(ws), size, _stream_ptr(stream)))


def w4a16_kv_free(block_table, kv_lens, refcount, seqs, stream=None):
    """Rows seqs[i] give up their pages: counts go down, entries become -1, lengths 0."""
    _table(block_table, kv_lens)
    _refcount(refcount, block_table.device)
    n = _ids("seqs", seqs, block_table.device)
    _check("w4a16_kv_free", load_library().w4a16_kv_free(
        _p(block_table), _p(kv_lens), block_table.shape[0], block_table.shape[1], _p(refcount), refcount.shape[0],
        _p(seqs), n, _stream_ptr(stream)))


def w4a16_kv_trim(block_table, kv_lens, refcount, page_size: int, window: int, sinks: int = 0, stream=None):
    """Every row gives up the pages that no later token sees with this window and these sinks."""
    _table(block_table, kv_lens)
    _refcount(refcount, block_table.device)
    _check("w4a16_kv_trim", load_library().w4a16_kv_trim(
        _p(block_table), _p(kv_lens), block_table.shape[0], block_table.shape[1], _p(refcount), refcount.shape[0],
        page_size, window, sinks, _stream_ptr(stream)))


def w4a16_kv_compact(cache, block_table, refcount, n_live=None, workspace=None, stream=None):
    """The m pages in use move to pages 0..m-1; table entries and counts
    follow.  n_live, if given, is an int32 [1] tensor that receives m."""
    import torch
    c = _cache(cache)
    dev = cache.k.device
    _tensor("block_table", block_table, torch.int32, 2)
    _one_device(cache.k, block_table)
    _refcount(refcount, dev, c.n_pages)
    if n_live is not None:
        _tensor("n_live", n_live, torch.int32, 1)
        if n_live.shape[0] != 1 or n_live.device != dev:
            raise ValueError("n_live must be [1] on the cache's device")
    ws, size = _scratch(workspace, w4a16_kv_pool_workspace(c.n_pages), dev, stream)
    _check("w4a16_kv_compact", load_library().w4a16_kv_compact(
        ctypes.byref(c), _p(block_table), block_table.shape[0], block_table.shape[1], _p(refcount), _p(n_live),
        _p(ws), size, _stream_ptr(stream)))
