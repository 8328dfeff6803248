"""Python binding of sampling under each request's own settings (``include/sdv_sample.h``).

Argument marshalling and checks only; the work runs in the library's kernels.

Typical use, the rows of a verify step whose requests have settings of their own::

    sample(logits, status, probs=p, temperature=t, top_k=k, top_p=tp, min_p=mp, row_request=owner)
    engine.accept(p, batch, result)                      # p as the target's probabilities

and next tokens without drafts, or a draft model's proposals with their distributions::

    sample(logits, status, uniforms=u, tokens=x, probs=q, temperature=t, top_p=tp)
"""
from __future__ import annotations

import ctypes

import torch

from . import SdvError
from ._abi import SdvSampleRows, load_library

__all__ = ["sample"]

INT_MAX = 2 ** 31 - 1


def sample(logits, status, *, uniforms=None, tokens=None, probs=None, temperature=None, top_k=None, top_p=None, min_p=None,
           row_request=None, stream=None, lib=None):
    """Filter each row of logits [rows, vocab] (bf16 or fp32, rows strided) under its request's settings.

    tokens [rows] int32 gets a token drawn with uniforms [rows] fp32, probs [rows, vocab] fp32 (rows strided) the
    distribution that it is drawn from; one of them or both, in memory of their own (probs over logits is refused).
    temperature, top_p, min_p fp32 and top_k int32 [requests] are device tensors, None for 1, 1, 0 and 0 (off);
    row_request [rows] int32 says which request's a row takes (None: row r is request r; negative: the row's outputs are
    left as they are).  lib: a load_library() other than libsdv.so.
    """
    index = logits.get_device()
    dtype = logits.dtype
    if logits.dim() != 2 or dtype is not torch.float32 and dtype is not torch.bfloat16 or index < 0:
        raise ValueError(f"logits: {dtype} {tuple(logits.shape)} on {logits.device}, bf16 or fp32 [rows, vocab] on a GPU is wanted")
    if torch._C._cuda_getDevice() != index:
        raise ValueError(f"logits: on {logits.device}, the current device is {torch.cuda.current_device()}")
    rows, vocab = logits.shape
    if rows == 0:
        return
    if tokens is None and probs is None:
        raise ValueError("tokens, probs: one of them is wanted")
    if tokens is not None and uniforms is None:
        raise ValueError("uniforms: drawing tokens takes them")
    step, one = logits.stride()
    if one != 1 and vocab > 1:
        raise ValueError(f"logits: strides {(step, one)}: a row must be contiguous")
    if status.dtype is not torch.int32 or status.get_device() != index:
        raise ValueError(f"status: {status.dtype} on {status.device}, int32 on {logits.device} is wanted")
    requests = None
    for t in (temperature, top_k, top_p, min_p):
        if t is not None:
            requests = t.shape[0] if t.dim() == 1 else -1
            break
    f32, i32 = torch.float32, torch.int32
    tp = None if temperature is None else _vector(temperature, "temperature", f32, requests, index)
    kp = None if top_k is None else _vector(top_k, "top_k", i32, requests, index)
    pp = None if top_p is None else _vector(top_p, "top_p", f32, requests, index)
    mp = None if min_p is None else _vector(min_p, "min_p", f32, requests, index)
    rp = None if row_request is None else _vector(row_request, "row_request", i32, rows, index)
    if rows > INT_MAX or vocab > INT_MAX:
        raise ValueError(f"logits: {tuple(logits.shape)}, sizes below 2^31 are wanted")
    if requests is None:
        requests = rows if rp is None else INT_MAX          # no setting is looked up
    if rp is None and requests < rows:
        raise ValueError(f"settings of {requests} requests for {rows} rows: row_request says which a row takes")
    if requests > INT_MAX:
        requests = INT_MAX      # (what row_request can name)
    up = None if uniforms is None else _vector(uniforms, "uniforms", f32, rows, index)
    xp = None if tokens is None else _vector(tokens, "tokens", i32, rows, index)
    op = None
    wide = 0
    if probs is not None:
        if probs.dtype is not f32 or probs.get_device() != index or probs.dim() != 2 or tuple(probs.shape) != (rows, vocab):
            raise ValueError(f"probs: {probs.dtype} {tuple(probs.shape)} on {probs.device}, fp32 {(rows, vocab)} on {logits.device} is wanted")
        wide, one = probs.stride()
        if vocab > 1 and one != 1 or rows > 1 and wide < vocab:
            raise ValueError(f"probs: strides {(wide, one)}: a row must be contiguous, and rows apart")
        op = probs.data_ptr()
        if rows == 1:
            wide = vocab
    r = SdvSampleRows(logits.data_ptr(), 1 if dtype is f32 else 0, step if rows > 1 else vocab, rows, vocab, requests, rp, tp, kp, pp, mp, up,
                      xp, op, wide)
    if lib is None:
        lib = load_library()
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    rc = lib.sdv_sample(ctypes.byref(r), status.data_ptr(), raw)
    if rc:
        extra = f" (cuda error {lib.sdv_last_cuda_error()})" if rc == 4 else ""
        raise SdvError(rc, "sdv_sample" + extra)


def _vector(t, name, dtype, n, index):
    """The address of a contiguous [n] tensor on the GPU `index`."""
    if t.dtype is dtype and t.dim() == 1 and t.shape[0] == n and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device} (contiguous: {t.is_contiguous()}), contiguous {dtype} [{n}] on "
                     f"cuda:{index} is wanted")
