"""ctypes binding of the paged 8-bit key/value cache (argument marshalling only).

Every function has the name of the C entry point it calls and the semantics
include/w4a16.h states; tensors' data pointers and the current CUDA stream are
handed over unchanged.  Scratch is allocated per call on that stream unless
the caller passes a workspace.  The tensors have to be on the current device.
With `stream`, the work runs there, and a result that is allocated here is
that stream's memory, safe to use on the current stream once that has waited
for it; the tensors passed in are the caller's to keep.

A cache is a KVCache of four tensors.  Its codes are [n_pages, n_kv_heads,
page_size, head_dim] in that order of dimensions, int8 or float8_e4m3fn, with
any strides that keep head_dim contiguous (a permuted [n_pages, page_size,
n_kv_heads, head_dim] tensor is as good); its scales are float32 [n_pages,
n_kv_heads].
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple

import torch

from .binding import W4A16_BF16, W4A16_F16, _check, _dtype_code, load_library

KV_INT8, KV_E4M3 = 0, 1


class KVCache(NamedTuple):
    """Codes and scales of a paged cache (see the module's docstring)."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


# w4a16_kv_cache_t and w4a16_kv_batch_t, in native layout
_CACHE = struct.Struct("@PPPPiiiiqqqi4x")
_BATCH = struct.Struct("@PPPiii4x")


def _refuse(name, t, dtype, dim, device):
    """Why `t` is not a contiguous tensor of this dtype and dimension on this CUDA device (None: any)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor, got device {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must be {dim}-D, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"operands are on different devices: {name} on {t.device}, others on cuda:{device}")


def _ints(name, t, dim, device):
    """An int32 tensor's address, checked; `device` is a CUDA device's index."""
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.dim() == dim and t.get_device() == device >= 0
            and t.is_contiguous()):
        _refuse(name, t, torch.int32, dim, device)
    return t.data_ptr()


def _device_of(name, t):
    if not isinstance(t, torch.Tensor) or t.get_device() < 0:
        _refuse(name, t, None, None, None)
    return t.get_device()


def _current(device):
    """`device`, which has to be the current one: the library launches there."""
    if torch._C._cuda_getDevice() != device:
        raise ValueError(f"the tensors are on cuda:{device}, the current device is cuda:{torch._C._cuda_getDevice()}: "
                         f"call under torch.cuda.device({device})")
    return device


def _cache(c):
    """(the cache as the C struct's bytes, device index, pages, heads, page size, head dim)"""
    if not isinstance(c, KVCache):
        raise TypeError(f"cache must be a KVCache, got {type(c).__name__}")
    k, v, ks, vs = c
    device = _current(_device_of("cache.k", k))
    kind = KV_INT8 if k.dtype is torch.int8 else KV_E4M3
    if kind == KV_E4M3 and k.dtype is not torch.float8_e4m3fn:
        raise TypeError(f"cache.k must be int8 or float8_e4m3fn, got {k.dtype}")
    if k.dim() != 4:
        raise ValueError(f"cache.k must be 4-D, got {list(k.shape)}")
    if _device_of("cache.v", v) != device:
        raise ValueError(f"operands are on different devices: {k.device}, {v.device}")
    shape, stride, v_stride = k.shape, k.stride(), v.stride()
    n_pages, heads, page_size, head_dim = shape
    if n_pages == 1 or heads == 1:             # strides of one element say nothing
        stride, v_stride = (tuple(x if n > 1 else 0 for n, x in zip(shape, y)) for y in (stride, v_stride))
    if v.dtype is not k.dtype or v.shape != shape or v_stride != stride:
        raise ValueError("cache.k and cache.v must have the same dtype, shape and strides")
    sp, sh, st, sd = stride
    if sd != 1:
        raise ValueError("the codes' last dimension must be contiguous")
    for name, t in (("cache.k_scale", ks), ("cache.v_scale", vs)):
        if not (isinstance(t, torch.Tensor) and t.dtype is torch.float32 and t.get_device() == device
                and t.dim() == 2 and t.is_contiguous()):
            _refuse(name, t, torch.float32, 2, device)
        if t.shape != (n_pages, heads):
            raise ValueError(f"{name} must be [{n_pages}, {heads}], got {list(t.shape)}")
    return (_CACHE.pack(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), n_pages, page_size, heads, head_dim,
                        sp, sh, st, kind), device, n_pages, heads, page_size, head_dim)


def _table(block_table, kv_lens, device):
    """(table's address, lengths' address, rows, width)"""
    table, lens = _ints("block_table", block_table, 2, device), _ints("kv_lens", kv_lens, 1, device)
    rows, width = block_table.shape
    if kv_lens.shape[0] != rows:
        raise ValueError(f"block_table has {rows} rows, kv_lens {kv_lens.shape[0]}")
    return table, lens, rows, width


def _batch(block_table, kv_lens, q_starts, n_tokens, device):
    """(the batch as the C struct's bytes, sequences)"""
    table, lens, n, width = _table(block_table, kv_lens, device)
    starts = _ints("q_starts", q_starts, 1, device)
    if q_starts.shape[0] != n + 1:
        raise ValueError(f"q_starts must be [n_seqs + 1] = [{n + 1}], got {list(q_starts.shape)}")
    return _BATCH.pack(table, lens, starts, n, width, n_tokens), n


def _rows(name, t, heads, head_dim, device):
    """Row stride of a [tokens, heads, head_dim] tensor whose rows are dense."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device or t.dim() != 3:
        if _device_of(name, t) != device:
            raise ValueError(f"{name} must be on the cache's device")
        raise ValueError(f"{name} must be 3-D, got {list(t.shape)}")
    n, h, d = t.shape
    if h != heads or d != head_dim:
        raise ValueError(f"{name} must be [n_tokens, {heads}, {head_dim}], got {list(t.shape)}")
    row, head, one = t.stride()
    if one != 1 or (heads > 1 and head != head_dim):
        raise ValueError(f"each row of {name} must be contiguous")
    return row if n > 1 else heads * head_dim


def _act(t):
    return W4A16_BF16 if t.dtype is torch.bfloat16 else W4A16_F16 if t.dtype is torch.float16 else _dtype_code(t)


@functools.lru_cache(maxsize=None)
def _device(index):
    # an index in a call's place costs torch more than the object: 1.8 us an allocation
    return torch.device("cuda", index)


def _on(stream, shape, dtype, device):
    """A result that work on `stream` writes: that stream's memory, so that what used it before is done, and held back
    after its end for the current stream, where the caller goes on."""
    here = torch.cuda.current_stream(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, _device(device))
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=_device(device))
    if stream != here:
        t.record_stream(here)
    return t


def _output(name, t, shape, dtype, device, stream):
    if t is None:
        if stream is not None:
            return _on(stream, shape, dtype, device)
        return torch.empty(shape, dtype=dtype, device=_device(device))
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device and t.is_contiguous()
            and t.dim() == len(shape)):
        _refuse(name, t, dtype, len(shape), device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t


class _Block:
    """Scratch of a stream from torch's allocator, given back with the object (2 us less than a tensor)."""
    __slots__ = ("at",)

    def __init__(self, size, stream):
        self.at = 0
        self.at = torch._C._cuda_cudaCachingAllocator_raw_alloc(size, stream)

    def __del__(self):
        if self.at:
            torch._C._cuda_cudaCachingAllocator_raw_delete(self.at)


def _scratch(workspace, need, device, handle):
    """(what holds the scratch, its address, its bytes): the caller's tensor, or from torch's allocator."""
    if workspace is None:
        block = _Block(need, handle)
        return block, block.at, need
    if not (isinstance(workspace, torch.Tensor) and workspace.get_device() == device and workspace.is_contiguous()):
        _refuse("workspace", workspace, None, None, device)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _stream(stream, device):
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def w4a16_kv_append(cache, k_new, v_new, block_table, kv_lens, q_starts, stream=None):
    """Quantise k_new, v_new [n_tokens, n_kv_heads, head_dim] (fp16/bf16, rows
    may be strided views) into the cache as each sequence's newest tokens:
    positions kv_lens[b] - (q_starts[b+1] - q_starts[b]) .. kv_lens[b] - 1."""
    c, dev, _, heads, _, dim = _cache(cache)
    sk, sv = _rows("k_new", k_new, heads, dim, dev), _rows("v_new", v_new, heads, dim, dev)
    if v_new.dtype is not k_new.dtype or v_new.shape != k_new.shape:
        raise ValueError("k_new and v_new must have the same dtype and shape")
    b, _ = _batch(block_table, kv_lens, q_starts, k_new.shape[0], dev)
    _check("w4a16_kv_append", load_library().w4a16_kv_append(
        c, k_new.data_ptr(), sk, v_new.data_ptr(), sv, b, _act(k_new), _stream(stream, dev)))


def w4a16_kv_read(cache, block_table, kv_lens, q_starts, n_tokens: int, dtype, k_out=None, v_out=None, stream=None):
    """The newest q_starts[b+1] - q_starts[b] cached tokens of each sequence as
    values of `dtype`: (k, v), each [n_tokens, n_kv_heads, head_dim]."""
    c, dev, _, heads, _, dim = _cache(cache)
    k_out = _output("k_out", k_out, (n_tokens, heads, dim), dtype, dev, stream)
    v_out = _output("v_out", v_out, (n_tokens, heads, dim), dtype, dev, stream)
    b, _ = _batch(block_table, kv_lens, q_starts, n_tokens, dev)
    _check("w4a16_kv_read", load_library().w4a16_kv_read(
        c, b, k_out.data_ptr(), v_out.data_ptr(), _act(k_out), _stream(stream, dev)))
    return k_out, v_out


def w4a16_kv_attention(q, cache, block_table, kv_lens, q_starts, max_q_len: int, scale=None, window: int = 0,
                       sinks: int = 0, out=None, lse=None, workspace=None, stream=None):
    """Causal attention of q [n_tokens, n_heads, head_dim] over the cache, with
    an optional sliding window (0: none) and sink tokens; out [n_tokens,
    n_heads, head_dim].  scale defaults to head_dim ** -0.5; lse, if given, is
    float32 [n_tokens, n_heads] and receives the log-sum-exp of each row."""
    c, dev, _, kv_heads, _, dim = _cache(cache)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        _refuse("q", q, None, 3, dev)
    T, H, _ = q.shape
    sq, dt = _rows("q", q, H, dim, dev), _act(q)
    out = _output("out", out, (T, H, dim), q.dtype, dev, stream)
    if lse is not None:
        _output("lse", lse, (T, H), torch.float32, dev, stream)
    b, n = _batch(block_table, kv_lens, q_starts, T, dev)
    handle = _stream(stream, dev)
    ws, at, size = _scratch(workspace, _attention_workspace(dev, H, kv_heads, dim, n, T), dev, handle)
    _check("w4a16_kv_attention", load_library().w4a16_kv_attention(
        q.data_ptr(), sq, H, c, b, max_q_len, dim ** -0.5 if scale is None else scale, window, sinks, out.data_ptr(),
        None if lse is None else lse.data_ptr(), dt, at, size, handle))
    return out


@functools.lru_cache(maxsize=1024)
def _attention_workspace(device, n_heads, n_kv_heads, head_dim, n_seqs, n_tokens):
    # a function of the device's size and these numbers alone
    return max(16, w4a16_kv_attention_workspace(n_heads, n_kv_heads, head_dim, n_seqs, n_tokens))


def w4a16_kv_attention_workspace(n_heads: int, n_kv_heads: int, head_dim: int, n_seqs: int, n_tokens: int) -> int:
    """Bytes of workspace that w4a16_kv_attention needs for these sizes, whatever the lengths."""
    need = ctypes.c_longlong(0)
    _check("w4a16_kv_attention_workspace", load_library().w4a16_kv_attention_workspace(
        n_heads, n_kv_heads, head_dim, n_seqs, n_tokens, ctypes.byref(need)))
    return need.value


def w4a16_kv_attention_shared(q, cache, block_table, kv_lens, q_starts, max_q_len: int, group_starts, prefix_lens, scale=None,
                              out=None, lse=None, workspace=None, stream=None):
    """w4a16_kv_attention, without a window, of a batch whose sequences
    [group_starts[g], group_starts[g + 1]) have their first prefix_lens[g]
    positions in the same pages: these are read once for all of a group."""
    c, dev, _, kv_heads, _, dim = _cache(cache)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        _refuse("q", q, None, 3, dev)
    T, H, _ = q.shape
    sq, dt = _rows("q", q, H, dim, dev), _act(q)
    out = _output("out", out, (T, H, dim), q.dtype, dev, stream)
    if lse is not None:
        _output("lse", lse, (T, H), torch.float32, dev, stream)
    b, n = _batch(block_table, kv_lens, q_starts, T, dev)
    starts, prefix = _ints("group_starts", group_starts, 1, dev), _ints("prefix_lens", prefix_lens, 1, dev)
    groups = prefix_lens.shape[0]
    if group_starts.shape[0] != groups + 1:
        raise ValueError(f"group_starts must be [n_groups + 1] = [{groups + 1}], got {list(group_starts.shape)}")
    handle = _stream(stream, dev)
    ws, at, size = _scratch(workspace, _shared_workspace(dev, H, kv_heads, dim, n, groups, T), dev, handle)
    _check("w4a16_kv_attention_shared", load_library().w4a16_kv_attention_shared(
        q.data_ptr(), sq, H, c, b, max_q_len, starts, prefix, groups, dim ** -0.5 if scale is None else scale, out.data_ptr(),
        None if lse is None else lse.data_ptr(), dt, at, size, handle))
    return out


@functools.lru_cache(maxsize=1024)
def _shared_workspace(device, n_heads, n_kv_heads, head_dim, n_seqs, n_groups, n_tokens):
    return max(16, w4a16_kv_attention_shared_workspace(n_heads, n_kv_heads, head_dim, n_seqs, n_groups, n_tokens))


def w4a16_kv_attention_shared_workspace(n_heads: int, n_kv_heads: int, head_dim: int, n_seqs: int, n_groups: int,
                                        n_tokens: int) -> int:
    """Bytes of workspace that w4a16_kv_attention_shared needs for these sizes, whatever the lengths."""
    need = ctypes.c_longlong(0)
    _check("w4a16_kv_attention_shared_workspace", load_library().w4a16_kv_attention_shared_workspace(
        n_heads, n_kv_heads, head_dim, n_seqs, n_groups, n_tokens, ctypes.byref(need)))
    return need.value


def _counts(refcount, device, n_pages=None):
    at = _ints("refcount", refcount, 1, device)
    if n_pages is not None and refcount.shape[0] != n_pages:
        raise ValueError(f"refcount must be [n_pages] = [{n_pages}], got {list(refcount.shape)}")
    return at


def w4a16_kv_copy_pages(cache, src, dst, stream=None):
    """Pages src[i] (codes and scales) copied to pages dst[i]; pairs with a negative id are skipped."""
    c, dev = _cache(cache)[:2]
    a, b = _ints("src", src, 1, dev), _ints("dst", dst, 1, dev)
    if src.shape[0] != dst.shape[0]:
        raise ValueError("src and dst must have the same length")
    _check("w4a16_kv_copy_pages", load_library().w4a16_kv_copy_pages(c, a, b, src.shape[0], _stream(stream, dev)))


@functools.lru_cache(maxsize=64)
def w4a16_kv_pool_workspace(n_pages: int) -> int:
    """Bytes of workspace that w4a16_kv_fork and w4a16_kv_compact need."""
    need = ctypes.c_longlong(0)
    _check("w4a16_kv_pool_workspace", load_library().w4a16_kv_pool_workspace(n_pages, ctypes.byref(need)))
    return need.value


def w4a16_kv_fork(cache, block_table, kv_lens, refcount, parents, children, workspace=None, stream=None):
    """Rows children[i] of the table continue rows parents[i]: full pages are
    shared, a partly filled last page is copied into the lowest free page."""
    c, dev, pages = _cache(cache)[:3]
    table, lens, rows, width = _table(block_table, kv_lens, dev)
    counts = _counts(refcount, dev, pages)
    a, b = _ints("parents", parents, 1, dev), _ints("children", children, 1, dev)
    if parents.shape[0] != children.shape[0]:
        raise ValueError("parents and children must have the same length")
    handle = _stream(stream, dev)
    ws, at, size = _scratch(workspace, w4a16_kv_pool_workspace(pages), dev, handle)
    _check("w4a16_kv_fork", load_library().w4a16_kv_fork(
        c, table, lens, rows, width, counts, a, b, parents.shape[0], at, size, handle))


@functools.lru_cache(maxsize=256)
def w4a16_kv_grow_workspace(n_pages: int, n_seqs: int) -> int:
    """Bytes of workspace that w4a16_kv_grow needs."""
    need = ctypes.c_longlong(0)
    _check("w4a16_kv_grow_workspace", load_library().w4a16_kv_grow_workspace(n_pages, n_seqs, ctypes.byref(need)))
    return need.value


def w4a16_kv_grow(cache, block_table, kv_lens, refcount, new_lens, n_tokens: int, q_starts=None, positions=None, slots=None,
                  workspace=None, stream=None):
    """Room for new_lens[b] more tokens of every row: pages from the free ones,
    a last page that other rows name too copied.  kv_lens grows with them.
    Returns (q_starts int32 [rows + 1], positions int32 [n_tokens], slots int64
    [n_tokens]): the rows of the step's token tensors, where each token is in
    its sequence and in the pool; -1 past the last token."""
    c, dev, pages = _cache(cache)[:3]
    table, lens, rows, width = _table(block_table, kv_lens, dev)
    counts, new = _counts(refcount, dev, pages), _ints("new_lens", new_lens, 1, dev)
    if new_lens.shape[0] != rows:
        raise ValueError(f"block_table has {rows} rows, new_lens {new_lens.shape[0]}")
    q_starts = _output("q_starts", q_starts, (rows + 1,), torch.int32, dev, stream)
    positions = _output("positions", positions, (n_tokens,), torch.int32, dev, stream)
    slots = _output("slots", slots, (n_tokens,), torch.int64, dev, stream)
    handle = _stream(stream, dev)
    ws, at, size = _scratch(workspace, w4a16_kv_grow_workspace(pages, rows), dev, handle)
    _check("w4a16_kv_grow", load_library().w4a16_kv_grow(
        c, table, lens, rows, width, counts, new, n_tokens, q_starts.data_ptr(), positions.data_ptr(), slots.data_ptr(), at,
        size, handle))
    return q_starts, positions, slots


def w4a16_kv_reorder(block_table, kv_lens, refcount, src, dst=None, stream=None):
    """Rows dst[i] (or i) become what rows src[i] were, none where src[i] is
    negative; pages' counts follow, nothing is copied."""
    dev = _current(_device_of("block_table", block_table))
    table, lens, rows, width = _table(block_table, kv_lens, dev)
    counts, a = _counts(refcount, dev), _ints("src", src, 1, dev)
    b = None if dst is None else _ints("dst", dst, 1, dev)
    if dst is not None and dst.shape[0] != src.shape[0]:
        raise ValueError("src and dst must have the same length")
    _check("w4a16_kv_reorder", load_library().w4a16_kv_reorder(
        table, lens, rows, width, counts, refcount.shape[0], b, a, src.shape[0], _stream(stream, dev)))


def w4a16_kv_free(block_table, kv_lens, refcount, seqs, stream=None):
    """Rows seqs[i] give up their pages: counts go down, entries become -1, lengths 0."""
    dev = _current(_device_of("block_table", block_table))
    table, lens, rows, width = _table(block_table, kv_lens, dev)
    counts, ids = _counts(refcount, dev), _ints("seqs", seqs, 1, dev)
    _check("w4a16_kv_free", load_library().w4a16_kv_free(
        table, lens, rows, width, counts, refcount.shape[0], ids, seqs.shape[0], _stream(stream, dev)))


def w4a16_kv_trim(block_table, kv_lens, refcount, page_size: int, window: int, sinks: int = 0, stream=None):
    """Every row gives up the pages that no later token sees with this window and these sinks."""
    dev = _current(_device_of("block_table", block_table))
    table, lens, rows, width = _table(block_table, kv_lens, dev)
    counts = _counts(refcount, dev)
    _check("w4a16_kv_trim", load_library().w4a16_kv_trim(
        table, lens, rows, width, counts, refcount.shape[0], page_size, window, sinks, _stream(stream, dev)))


def w4a16_kv_compact(cache, block_table, refcount, n_live=None, workspace=None, stream=None):
    """The m pages in use move to pages 0..m-1; table entries and counts
    follow.  n_live, if given, is an int32 [1] tensor that receives m."""
    c, dev, pages = _cache(cache)[:3]
    table = _ints("block_table", block_table, 2, dev)
    rows, width = block_table.shape
    counts = _counts(refcount, dev, pages)
    live = None if n_live is None else _ints("n_live", n_live, 1, dev)
    if n_live is not None and n_live.shape[0] != 1:
        raise ValueError(f"n_live must be [1], got {list(n_live.shape)}")
    handle = _stream(stream, dev)
    ws, at, size = _scratch(workspace, w4a16_kv_pool_workspace(pages), dev, handle)
    _check("w4a16_kv_compact", load_library().w4a16_kv_compact(
        c, table, rows, width, counts, live, at, size, handle))
