"""Python binding of low-rank adapters beside a shared projection (``include/sdv_adapter.h``).

Argument marshalling and checks only; the work runs in the library's kernels.

Typical use, a projection whose requests have adapters of their own::

    adapters = Adapters(a, b, scales, max_rows=8192, max_slots=64)    # a [count, rank, K], b [count, N, rank] bf16
    engine.linear(0, x, y)                                            # shared by all rows
    adapters.apply(x, y, y, row_offsets, ids, status)                 # request b's rows add adapter ids[b]
"""
from __future__ import annotations

import ctypes

import torch

from . import SdvError
from ._abi import SDV_OK, SdvAdapterConfig, SdvAdapterRows, load_library
from .cache import _c_int

__all__ = ["Adapters"]

BOTH = (torch.bfloat16, torch.float32)
INT_MAX = 2 ** 31 - 1


class Adapters:
    """The adapters of one projection, for batches of up to max_rows rows of max_slots (at most 1024) requests.

    a [count, rank, K], b [count, N, rank] bf16 and scales [count] fp32 are contiguous, on one GPU, the current one, and stay
    the caller's: their contents may be exchanged between calls.  Calls may overlap.
    """

    def __init__(self, a, b, scales, max_rows: int, max_slots: int, lib_path: str | None = None):
        self.lib = load_library(lib_path) if lib_path else load_library()
        self._index = a.get_device()
        for t, name, dtype, dim in ((a, "a", torch.bfloat16, 3), (b, "b", torch.bfloat16, 3), (scales, "scales", torch.float32, 1)):
            if t.dtype is not dtype or t.dim() != dim or t.get_device() != self._index or self._index < 0 or not t.is_contiguous():
                raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device} (contiguous: {t.is_contiguous()}), contiguous "
                                 f"{dtype} of {dim} dimensions on one GPU is wanted")
        count, rank, k = a.shape
        n = b.shape[1]
        if tuple(b.shape) != (count, n, rank) or scales.shape[0] != count:
            raise ValueError(f"a {tuple(a.shape)}, b {tuple(b.shape)}, scales {tuple(scales.shape)}: [count, rank, K], [count, N, rank] "
                             "and [count] are wanted")
        if torch.cuda.current_device() != self._index:
            raise ValueError(f"a: on {a.device}, the current device is {torch.cuda.current_device()}")
        self.tensors = (a, b, scales)
        self.device = a.device
        self.k, self.n = k, n
        self.max_rows, self.max_slots = _c_int(max_rows), _c_int(max_slots)
        self.cfg = SdvAdapterConfig(_c_int(k), _c_int(n), _c_int(rank), _c_int(count), a.data_ptr(), b.data_ptr(), scales.data_ptr())
        h = ctypes.c_void_p()
        self._check(self.lib.sdv_adapters_create(ctypes.byref(self.cfg), self.max_rows, self.max_slots, ctypes.byref(h)),
                    "sdv_adapters_create")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None):
            self.lib.sdv_adapters_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, rc, what):
        if rc != SDV_OK:
            extra = f" (cuda error {self.lib.sdv_last_cuda_error()})" if rc == 4 else ""
            raise SdvError(rc, what + extra)

    def _rows(self, t, name, rows, width, dtypes):
        """The row stride of a [rows, width] tensor whose rows are contiguous."""
        n, st = t.shape, t.stride()
        if len(n) == 2 and t.dtype in dtypes and t.get_device() == self._index and n[0] == rows and n[1] == width and st[1] == 1:
            return st[0] if rows > 1 else width
        raise ValueError(f"{name}: {t.dtype} {tuple(n)} with strides {tuple(st)} on {t.device}, one of {dtypes} [{rows}, {width}] with "
                         f"contiguous rows on {self.device} is wanted")

    def apply(self, x, base, out, row_offsets, adapter_ids, status, stream=None):
        """out = base + scale (x A^T) B^T for the rows of each request under its adapter: x [T, K], base and out [T, N], bf16
        or fp32 (base and out alike), rows strided; out may be base, and shares no memory with it or x otherwise.
        row_offsets [B + 1] and adapter_ids [B] int32, an id below 0 being no adapter."""
        T = x.shape[0]
        xs = self._rows(x, "x", T, self.k, BOTH)
        bs, os_ = self._rows(base, "base", T, self.n, BOTH), self._rows(out, "out", T, self.n, (base.dtype,))
        B = adapter_ids.shape[0] if adapter_ids.dim() == 1 else -1
        for t, name, n in ((row_offsets, "row_offsets", B + 1), (adapter_ids, "adapter_ids", B)):
            if t.dtype is not torch.int32 or t.dim() != 1 or t.shape[0] != n or t.get_device() != self._index or not t.is_contiguous():
                raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device} (contiguous: {t.is_contiguous()}), contiguous int32 "
                                 f"[{'B + 1' if name == 'row_offsets' else 'B'}] on {self.device} is wanted")
        if status.dtype is not torch.int32 or status.get_device() != self._index:
            raise ValueError(f"status: {status.dtype} on {status.device}, int32 on {self.device} is wanted")
        raw = torch._C._cuda_getCurrentRawStream(self._index) if stream is None else stream.cuda_stream
        if T > INT_MAX or B > INT_MAX:
            raise ValueError(f"x: {tuple(x.shape)}, adapter_ids: {tuple(adapter_ids.shape)}, sizes below 2^31 are wanted")
        r = SdvAdapterRows(B, T, row_offsets.data_ptr(), adapter_ids.data_ptr(), x.data_ptr(), 1 if x.dtype is torch.float32 else 0, xs,
                           base.data_ptr(), out.data_ptr(), 1 if base.dtype is torch.float32 else 0, bs, os_)
        rc = self.lib.sdv_adapters_apply(self.handle, ctypes.byref(r), status.data_ptr(), raw)
        if rc:
            self._check(rc, "sdv_adapters_apply")
