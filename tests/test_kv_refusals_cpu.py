"""What the paged-cache entry points refuse on the host, before any device is
touched, and what the binding refuses before the C call."""
import ctypes

import pytest
import torch

NULL, OK = None, 0x1000                # addresses are never dereferenced: validation fails first
ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_DTYPE, ERR_ARG = -1, -2, -4, -5, -9


class Cache(ctypes.Structure):         # w4a16_kv_cache_t
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("page_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong), ("token_stride", ctypes.c_longlong), ("kv_dtype", ctypes.c_int)]


class Batch(ctypes.Structure):         # w4a16_kv_batch_t
    _fields_ = [("block_table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("q_starts", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int), ("max_blocks", ctypes.c_int), ("n_tokens", ctypes.c_int)]


@pytest.fixture(scope="module")
def lib():
    from w4a16_group_quantised_gb300 import build
    build.build()
    import w4a16_group_quantised_gb300 as w
    return w.load_library()


def cache(**kw):
    f = dict(k=OK, v=OK, k_scale=OK, v_scale=OK, n_pages=8, page_size=16, n_kv_heads=2, head_dim=128,
             page_stride=4096, head_stride=2048, token_stride=128, kv_dtype=0)
    f.update(kw)
    return ctypes.byref(Cache(**f))


def batch(**kw):
    f = dict(block_table=OK, kv_lens=OK, q_starts=OK, n_seqs=2, max_blocks=4, n_tokens=3)
    f.update(kw)
    return ctypes.byref(Batch(**f))


def append(lib, c=None, b=None, k=OK, ks=256, v=OK, vs=256, dt=0):
    return lib.w4a16_kv_append(c or cache(), k, ks, v, vs, b or batch(), dt, None)


def read(lib, c=None, b=None, k=OK, v=OK, dt=0):
    return lib.w4a16_kv_read(c or cache(), b or batch(), k, v, dt, None)


def attend(lib, c=None, b=None, q=OK, qs=1024, heads=8, most=1, scale=0.1, window=0, sinks=0, out=OK, lse=None, dt=0,
           ws=OK, size=1 << 40):
    return lib.w4a16_kv_attention(q, qs, heads, c or cache(), b or batch(), most, scale, window, sinks, out, lse, dt, ws,
                                  size, None)


@pytest.mark.parametrize("call", [append, read, attend])
def test_cache_and_batch(lib, call):
    assert call(lib, c=cache(kv_dtype=2)) == ERR_DTYPE
    assert call(lib, dt=2) == ERR_DTYPE
    for bad in (dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(head_dim=96), dict(head_dim=256),
                dict(n_pages=0), dict(n_kv_heads=0), dict(token_stride=64), dict(head_stride=112), dict(page_stride=-16),
                dict(page_stride=64)):
        assert call(lib, c=cache(**bad)) == ERR_SHAPE, bad
    for bad in (dict(k=NULL), dict(v=NULL), dict(k_scale=NULL), dict(v_scale=NULL)):
        assert call(lib, c=cache(**bad)) == ERR_NULL, bad
    for bad in (dict(k=OK + 8), dict(v=OK + 1), dict(k_scale=OK + 2), dict(token_stride=136), dict(head_stride=2052),
                dict(page_stride=4104)):
        assert call(lib, c=cache(**bad)) == ERR_ALIGN, bad
    for bad in (dict(n_seqs=-1), dict(max_blocks=0), dict(max_blocks=1 << 28), dict(n_tokens=-1), dict(n_seqs=0)):
        assert call(lib, b=batch(**bad)) == ERR_SHAPE, bad
    for bad in (dict(block_table=NULL), dict(kv_lens=NULL), dict(q_starts=NULL)):
        assert call(lib, b=batch(**bad)) == ERR_NULL, bad
    for bad in (dict(block_table=OK + 2), dict(kv_lens=OK + 1), dict(q_starts=OK + 3)):
        assert call(lib, b=batch(**bad)) == ERR_ALIGN, bad
    # no tokens: a no-op that needs no device
    assert call(lib, b=batch(n_tokens=0)) == 0
    assert call(lib, b=batch(n_tokens=0, n_seqs=0, block_table=NULL, kv_lens=NULL, q_starts=NULL)) == 0


def test_append(lib):
    assert append(lib, k=NULL) == ERR_NULL and append(lib, v=NULL) == ERR_NULL
    assert append(lib, k=OK + 8) == ERR_ALIGN and append(lib, v=OK + 2) == ERR_ALIGN
    assert append(lib, ks=260) == ERR_ALIGN and append(lib, vs=248) == ERR_SHAPE


def test_read(lib):
    assert read(lib, k=NULL) == ERR_NULL and read(lib, v=NULL) == ERR_NULL
    assert read(lib, k=OK + 8) == ERR_ALIGN and read(lib, v=OK + 4) == ERR_ALIGN


def test_attention(lib):
    assert attend(lib, q=NULL) == ERR_NULL and attend(lib, out=NULL) == ERR_NULL
    assert attend(lib, q=OK + 8) == ERR_ALIGN and attend(lib, out=OK + 4) == ERR_ALIGN
    assert attend(lib, lse=OK + 2) == ERR_ALIGN
    assert attend(lib, qs=1020) == ERR_SHAPE and attend(lib, qs=1028) == ERR_ALIGN
    for heads in (0, -8, 7, 2 * 129):
        assert attend(lib, heads=heads, qs=1 << 20) == ERR_SHAPE
    assert attend(lib, window=-1) == ERR_ARG and attend(lib, sinks=-1) == ERR_ARG and attend(lib, most=-1) == ERR_ARG
    assert attend(lib, scale=float("nan")) == ERR_ARG


def test_workspaces(lib):
    n = ctypes.c_longlong()
    assert lib.w4a16_kv_attention_workspace(8, 2, 128, 4, 4, None) == ERR_NULL
    for bad in ((7, 2, 128, 4, 4), (8, 0, 128, 4, 4), (8, 2, 96, 4, 4), (8, 2, 128, -1, 4), (8, 2, 128, 4, -1)):
        assert lib.w4a16_kv_attention_workspace(*bad, ctypes.byref(n)) == ERR_SHAPE
    assert lib.w4a16_kv_pool_workspace(8, None) == ERR_NULL
    assert lib.w4a16_kv_pool_workspace(0, ctypes.byref(n)) == ERR_SHAPE
    assert lib.w4a16_kv_pool_workspace(5000, ctypes.byref(n)) == 0 and n.value >= 3 * 4 * 5000


def test_copy_pages(lib):
    f = lib.w4a16_kv_copy_pages
    assert f(cache(), OK, OK, -1, None) == ERR_SHAPE and f(cache(), OK, OK, 1 << 30, None) == ERR_SHAPE
    assert f(cache(), NULL, OK, 1, None) == ERR_NULL and f(cache(), OK, NULL, 1, None) == ERR_NULL
    assert f(cache(), OK + 1, OK, 1, None) == ERR_ALIGN
    assert f(cache(page_size=24), OK, OK, 1, None) == ERR_SHAPE
    assert f(cache(), NULL, NULL, 0, None) == 0


def test_fork(lib):
    def f(c=None, table=OK, lens=OK, n_seqs=4, blocks=4, ref=OK, par=OK, chi=OK, n=2, ws=OK, size=1 << 20):
        return lib.w4a16_kv_fork(c or cache(), table, lens, n_seqs, blocks, ref, par, chi, n, ws, size, None)
    assert f(n=5) == ERR_SHAPE and f(n=-1) == ERR_SHAPE and f(blocks=0) == ERR_SHAPE
    for bad in (dict(table=NULL), dict(lens=NULL), dict(ref=NULL), dict(par=NULL), dict(chi=NULL), dict(ws=NULL)):
        assert f(**bad) == ERR_NULL, bad
    for bad in (dict(table=OK + 2), dict(ref=OK + 1), dict(chi=OK + 2), dict(ws=OK + 8)):
        assert f(**bad) == ERR_ALIGN, bad
    assert f(size=64) == ERR_ARG
    assert f(n=0) == 0


def test_free_trim_compact(lib):
    free, trim, comp = lib.w4a16_kv_free, lib.w4a16_kv_trim, lib.w4a16_kv_compact
    assert free(OK, OK, 2, 4, OK, 8, OK, 3, None) == ERR_SHAPE
    assert free(OK, OK, 2, 4, OK, 0, OK, 1, None) == ERR_SHAPE
    assert free(NULL, OK, 2, 4, OK, 8, OK, 1, None) == ERR_NULL
    assert free(OK, OK, 2, 4, NULL, 8, OK, 1, None) == ERR_NULL
    assert free(OK, OK, 2, 4, OK, 8, OK + 1, 1, None) == ERR_ALIGN
    assert free(OK, OK, 2, 4, OK, 8, NULL, 0, None) == 0
    assert trim(OK, OK, 2, 4, OK, 8, 17, 4, 0, None) == ERR_SHAPE
    assert trim(OK, OK, 2, 4, OK, 8, 16, -4, 0, None) == ERR_ARG
    assert trim(OK, OK, 2, 4, OK, 8, 16, 4, -1, None) == ERR_ARG
    assert trim(OK, OK, 2, 4, NULL, 8, 16, 4, 0, None) == ERR_NULL
    assert trim(OK, OK, 2, 4, OK, 8, 16, 0, 0, None) == 0
    assert comp(cache(), NULL, 2, 4, OK, None, OK, 1 << 20, None) == ERR_NULL
    assert comp(cache(), OK, 2, 4, NULL, None, OK, 1 << 20, None) == ERR_NULL
    assert comp(cache(), OK, 2, 4, OK, None, OK, 8, None) == ERR_ARG
    assert comp(cache(), OK, 2, 4, OK, OK + 2, OK, 1 << 20, None) == ERR_ALIGN
    assert comp(cache(), OK, -2, 4, OK, None, OK, 1 << 20, None) == ERR_SHAPE


def test_binding_refuses_before_the_call():
    import w4a16_group_quantised_gb300 as w
    k = torch.zeros((4, 2, 16, 128), dtype=torch.int8)
    c = w.KVCache(k, k, torch.zeros(4, 2), torch.zeros(4, 2))
    ints = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros((1, 4, 128), dtype=torch.float16)
    with pytest.raises(TypeError):
        w.w4a16_kv_attention(q, (k, k), ints, ints, ints, 1)
    with pytest.raises(ValueError, match="CUDA"):
        w.w4a16_kv_attention(q, c, ints, ints, ints, 1)
    with pytest.raises(ValueError, match="CUDA"):
        w.w4a16_kv_append(c, q, q, ints, ints, ints)
    with pytest.raises(TypeError):
        w.w4a16_kv_free([0], ints, ints, ints)


def test_binding_packs_the_structs_as_c_lays_them_out():
    from w4a16_group_quantised_gb300 import kv
    assert kv._CACHE.size == ctypes.sizeof(Cache) and kv._BATCH.size == ctypes.sizeof(Batch)
    raw = Cache.from_buffer_copy(kv._CACHE.pack(1, 2, 3, 4, 5, 6, 7, 8, 1 << 40, 10, 11, 1))
    assert [getattr(raw, f[0]) for f in Cache._fields_] == [1, 2, 3, 4, 5, 6, 7, 8, 1 << 40, 10, 11, 1]
    raw = Batch.from_buffer_copy(kv._BATCH.pack(1, 2, 3, 4, 5, 6))
    assert [getattr(raw, f[0]) for f in Batch._fields_] == [1, 2, 3, 4, 5, 6]
