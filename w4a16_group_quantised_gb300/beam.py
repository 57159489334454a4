"""ctypes binding of beam search's selection (argument marshalling only).

w4a16_beam_select has the semantics include/w4a16.h states.  As in kv.py: the
tensors have to be on the current device, scratch and results are the current
stream's, or with `stream` that stream's, safe to use on the current one once
that has waited for it.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from .binding import W4A16_BF16, W4A16_F16, _check, load_library
from .kv import _current, _device_of, _output, _refuse, _scratch, _stream

W4A16_F32 = 2
_LOGITS = {torch.float16: W4A16_F16, torch.bfloat16: W4A16_BF16, torch.float32: W4A16_F32}


@functools.lru_cache(maxsize=256)
def _workspace(device, n_groups, width, vocab, n_out):
    need = ctypes.c_longlong(0)
    _check("w4a16_beam_select_workspace", load_library().w4a16_beam_select_workspace(
        n_groups, width, vocab, n_out, ctypes.byref(need)))
    return max(16, need.value)


def w4a16_beam_select_workspace(n_groups: int, width: int, vocab: int, n_out: int) -> int:
    """Bytes of workspace that w4a16_beam_select needs on the current device."""
    return _workspace(torch.cuda.current_device(), n_groups, width, vocab, n_out)


def w4a16_beam_select(logits, scores, width: int, n_out: int, finished=None, end_token: int = -1, out_scores=None,
                      out_rows=None, out_tokens=None, out_finished=None, workspace=None, stream=None):
    """The n_out best continuations of each request over its `width` beams and
    the vocabulary: logits [requests * width, vocab] (fp16, bf16 or fp32; rows
    may be strided), scores float32 [requests * width], finished bool
    [requests * width] or None.  Returns (scores float32, rows int32, tokens
    int32, finished bool), each [requests, n_out]."""
    dev = _current(_device_of("logits", logits))
    kind = _LOGITS.get(logits.dtype)
    if kind is None:
        raise TypeError(f"logits must be float16, bfloat16 or float32, got {logits.dtype}")
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError(f"logits must be 2-D with contiguous rows, got {list(logits.shape)}, strides {logits.stride()}")
    beams, vocab = logits.shape
    if width < 1 or beams % width != 0:
        raise ValueError(f"logits must be [requests * width, vocab] with width {width}, got {list(logits.shape)}")
    for name, t, dtype in (("scores", scores, torch.float32), ("finished", finished, torch.bool)):
        if t is None and name == "finished":
            continue
        if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.dim() == 1
                and t.is_contiguous()):
            _refuse(name, t, dtype, 1, dev)
        if t.shape[0] != beams:
            raise ValueError(f"{name} must be [{beams}], got {list(t.shape)}")
    requests, shape = beams // width, (beams // width, n_out)
    need = _workspace(dev, requests, width, vocab, n_out)           # checks the sizes
    out_scores = _output("out_scores", out_scores, shape, torch.float32, dev, stream)
    out_rows = _output("out_rows", out_rows, shape, torch.int32, dev, stream)
    out_tokens = _output("out_tokens", out_tokens, shape, torch.int32, dev, stream)
    out_finished = _output("out_finished", out_finished, shape, torch.bool, dev, stream)
    handle = _stream(stream, dev)
    ws, at, size = _scratch(workspace, need, dev, handle)
    _check("w4a16_beam_select", load_library().w4a16_beam_select(
        logits.data_ptr(), logits.stride(0) if beams > 1 else vocab, kind, scores.data_ptr(),
        None if finished is None else finished.data_ptr(), requests, width, vocab, end_token, n_out, out_scores.data_ptr(),
        out_rows.data_ptr(), out_tokens.data_ptr(), out_finished.data_ptr(), at, size, handle))
    return out_scores, out_rows, out_tokens, out_finished
