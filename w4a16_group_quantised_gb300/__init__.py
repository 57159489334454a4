"""GB300-native W4A16 group-quantised linear layer.

y = x . dequant(W)^T with x fp16/bf16 [M, K], W 4-bit packed 8 per int32 along
K as [N, K/8], per-group scales [N, K/G] (G in {32, 64, 128}), symmetric
(bias 8) or asymmetric weights (zero points packed 8 per int32 along N as
[N/8, K/G]), fp32 accumulation.

Beside it, for whole decoder layers: a paged key/value cache in 8 bits (kv.py:
append, attention with an optional window and sinks, page operators).

The compute path is the C-ABI shared library ``libw4a16.so`` built from
``csrc/`` (hand-written CUDA for sm_103a); ``binding`` marshals torch tensors
into it.  Nothing here falls back to a CPU or PyTorch implementation: if the
library is missing the calls raise.
"""
from .binding import (  # noqa: F401
    EPI_NONE,
    EPI_SILU_MUL,
    W4A16Error,
    library_path,
    load_library,
    w4a16_clear_device_error,
    w4a16_debug_decode_trace,
    w4a16_debug_set_config,
    w4a16_dequant_debug,
    w4a16_gemm,
    w4a16_dequantize,
    w4a16_gemm_cached,
    w4a16_gemm_chain,
    w4a16_gemm_dense,
    w4a16_gemm_decode_noalloc,
    w4a16_gemm_fused,
    w4a16_gemm_host,
    w4a16_gemm_host_async,
    w4a16_last_device_error,
    w4a16_moe_gemm,
    w4a16_pack,
    w4a16_pack_zeros,
    w4a16_select_path,
)

_KV = ("KVCache", "w4a16_kv_append", "w4a16_kv_attention", "w4a16_kv_attention_workspace", "w4a16_kv_compact",
       "w4a16_kv_copy_pages", "w4a16_kv_fork", "w4a16_kv_free", "w4a16_kv_pool_workspace", "w4a16_kv_read",
       "w4a16_kv_trim")


def __getattr__(name):
    # kv.py imports torch: on first use, so that building the library does not
    if name in _KV:
        from . import kv
        for n in _KV:
            globals()[n] = getattr(kv, n)
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def __dir__():
    return sorted(list(globals()) + list(_KV))
