"""Python binding of the paged cache's operators (``include/sdv_cache.h``).

Argument marshalling and checks only; the work runs in the library's kernels.

Typical use, a chunk of new tokens through one layer::

    cache = PagedCache(dict(n_q=32, n_kv=8, head_dim=128, cache_format="e4m3", rope_theta=1e6),
                       max_rows=8192, max_slots=64)
    pool, scales = cache.new_pool(pages)
    chunk = cache.chunk(rows=T, max_q=longest, row_offsets=offsets, kv_lens=lens, page_table=table,
                        kv_pool=pool, kv_scales=scales)
    cache.append(chunk, k, v, status, q=q, q_out=q_rot)      # rotate, round, store
    cache.attention(chunk, q_rot, out, status)               # over everything cached
    cache.read(chunk, k_back, v_back, status)                # what the cache holds now

A chunk keeps the addresses of its tensors; their contents (offsets, lengths,
tables, pages) may change between calls, so one chunk serves a captured graph
or a loop of steps, and every cache of the same key heads, head size and format.
"""
from __future__ import annotations

import ctypes

import torch

from . import SdvError, _ptr, _stream
from ._abi import (SDV_CACHE_BF16, SDV_CACHE_E4M3, SDV_OK, SdvAppendRows, SdvCacheConfig, SdvCacheTables, SdvChunk,
                   load_library)

__all__ = ["PagedCache", "Chunk", "Tables"]

BF16, BOTH = (torch.bfloat16,), (torch.bfloat16, torch.float32)
FORMATS = {"bf16": SDV_CACHE_BF16, "e4m3": SDV_CACHE_E4M3}


def _c_int(x) -> int:
    """x for a 32-bit field, which ctypes would wrap: the largest there is, or -1, beyond its ends."""
    return max(-1, min(int(x), 2 ** 31 - 1))


class Chunk:
    """A ragged chunk's description (sdv_chunk), the tensors that it points to and the geometry of their pages."""

    def __init__(self, struct: SdvChunk, tensors: tuple, geometry: tuple):
        self.struct = struct
        self.geometry = geometry
        self.ref = ctypes.byref(struct)
        self.rows = struct.T
        self.tensors = tensors


class PagedCache:
    """Operators over a paged cache of one geometry, with their workspace.

    cfg: n_q, n_kv, head_dim, page_size (16), cache_format ("bf16" or "e4m3"),
    rope_theta (0 or absent: append does not rotate).  The workspace is
    allocated here through torch, on the current device; calls of one
    PagedCache must not overlap in time.  It may be let go while its calls are
    still running, on whichever stream; a captured graph needs it as long as it is replayed.
    """

    def __init__(self, cfg: dict, max_rows: int, max_slots: int, lib_path: str | None = None):
        self.lib = load_library(lib_path) if lib_path else load_library()
        fmt = cfg.get("cache_format", "bf16")
        if fmt not in FORMATS:
            raise ValueError(f"cache_format {fmt!r}: one of {sorted(FORMATS)}")
        c = SdvCacheConfig(_c_int(cfg["n_q"]), _c_int(cfg["n_kv"]), _c_int(cfg["head_dim"]), _c_int(cfg.get("page_size", 16)),
                           FORMATS[fmt], float(cfg.get("rope_theta", 0.0)))
        self.max_rows, self.max_slots = _c_int(max_rows), _c_int(max_slots)
        nbytes = self.lib.sdv_cache_workspace_size(ctypes.byref(c), self.max_rows, self.max_slots)
        if nbytes == 0:
            raise SdvError(1, "sdv_cache_workspace_size rejected the configuration")
        self._setup(c, fmt, torch.empty(int(nbytes), dtype=torch.uint8, device="cuda"))
        self._streams.add(torch._C._cuda_getCurrentRawStream(self._index))
        h = ctypes.c_void_p()
        self._check(self.lib.sdv_cache_create(ctypes.byref(self.cfg), _ptr(self.workspace), ctypes.c_size_t(nbytes),
                                              self.max_rows, self.max_slots, _stream(None), ctypes.byref(h)),
                    "sdv_cache_create")
        self.handle = h

    def _setup(self, cfg: SdvCacheConfig, fmt: str, workspace):
        self.cfg, self.format, self.workspace = cfg, fmt, workspace
        self.device = workspace.device
        self._index = workspace.get_device()
        self._n_q, self._n_kv, self._d = cfg.n_q, cfg.n_kv, cfg.head_dim
        self._geometry = (cfg.n_kv, cfg.head_dim, fmt, self._index)
        self._streams = set()  # whose work the workspace's memory is known to wait for

    def close(self):
        if getattr(self, "handle", None):
            self.lib.sdv_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- marshalling -------------------------------------------------------

    def _check(self, rc, what):
        if rc != SDV_OK:
            extra = f" (cuda error {self.lib.sdv_last_cuda_error()})" if rc == 4 else ""
            raise SdvError(rc, what + extra)

    def _want(self, t, name, dtype, shape=None):
        if t.dtype != dtype:
            raise ValueError(f"{name}: {t.dtype}, {dtype} is wanted")
        if t.device != self.device:
            raise ValueError(f"{name}: on {t.device}, the cache's operators run on {self.device}")
        if shape is not None and (tuple(t.shape) != tuple(shape) or not t.is_contiguous()):
            raise ValueError(f"{name}: shape {tuple(t.shape)} (contiguous: {t.is_contiguous()}), contiguous {tuple(shape)} is wanted")

    def _rows(self, t, name, heads, rows, dtypes):
        """The row stride of a [>= rows, heads, head_dim] tensor whose heads are contiguous."""
        d = self._d
        n, st = t.shape, t.stride()
        if len(n) == 3 and t.dtype in dtypes and t.get_device() == self._index and n[0] >= rows and n[1] == heads \
                and n[2] == d and st[2] == 1 and (st[1] == d or heads == 1):
            return st[0] if n[0] > 1 else heads * d
        if t.dtype not in dtypes:
            raise ValueError(f"{name}: {t.dtype}, one of {dtypes} is wanted")
        if t.get_device() != self._index:
            raise ValueError(f"{name}: on {t.device}, the cache's operators run on {self.device}")
        if len(n) != 3 or n[0] < rows or n[1] != heads or n[2] != d:
            raise ValueError(f"{name}: shape {tuple(n)}, [{rows}, {heads}, {d}] is wanted")
        raise ValueError(f"{name}: strides {tuple(st)}: a row's heads must be contiguous")

    def _mine(self, chunk):
        """The chunk's rows; its pages must be laid out as this cache's."""
        if chunk.geometry != self._geometry:
            raise ValueError(f"chunk: of a cache with (n_kv, head_dim, format, device) {chunk.geometry}, "
                             f"{self._geometry} is wanted")
        return chunk.rows

    def _enqueue(self, status, stream):
        """The status word's address and the stream's handle (the current stream's by default)."""
        if status.dtype is not torch.int32 or status.get_device() != self._index:
            raise ValueError(f"status: {status.dtype} on {status.device}, int32 on {self.device} is wanted")
        return status.data_ptr(), torch._C._cuda_getCurrentRawStream(self._index) if stream is None else stream.cuda_stream

    def new_pool(self, pages: int):
        """(kv_pool, kv_scales) of a cache of `pages` pages; kv_scales is None for bf16."""
        shape = (int(pages), self.cfg.n_kv, 2, self.cfg.page_size, self.cfg.head_dim)
        if self.format == "bf16":
            return torch.zeros(shape, dtype=torch.bfloat16, device=self.device), None
        return (torch.zeros(shape, dtype=torch.uint8, device=self.device),
                torch.full(shape[:-1], 127, dtype=torch.uint8, device=self.device))

    def chunk(self, rows: int, max_q: int, row_offsets, kv_lens, page_table, kv_pool, kv_scales=None,
              window: int = 0) -> Chunk:
        """Describe a ragged chunk (sdv_chunk): `rows` rows of at most `max_q` per sequence."""
        B = int(kv_lens.shape[0])
        self._want(kv_lens, "kv_lens", torch.int32, (B,))
        self._want(row_offsets, "row_offsets", torch.int32, (B + 1,))
        self._want(page_table, "page_table", torch.int32, (B, page_table.shape[-1]))
        c = self.cfg
        pool_shape = (kv_pool.shape[0], c.n_kv, 2, c.page_size, c.head_dim)
        self._want(kv_pool, "kv_pool", torch.bfloat16 if self.format == "bf16" else torch.uint8, pool_shape)
        if self.format == "e4m3":
            if kv_scales is None:
                raise ValueError("kv_scales: an e4m3 cache has them")
            self._want(kv_scales, "kv_scales", torch.uint8, pool_shape[:-1])
        elif kv_scales is not None:
            raise ValueError("kv_scales: a bf16 cache has none")
        s = SdvChunk(B, _c_int(rows), _c_int(max_q), row_offsets.data_ptr(), kv_lens.data_ptr(), kv_pool.data_ptr(),
                     kv_scales.data_ptr() if kv_scales is not None else None, _c_int(kv_pool.shape[0]),
                     page_table.data_ptr(), _c_int(page_table.shape[1]), _c_int(window))
        return Chunk(s, (row_offsets, kv_lens, page_table, kv_pool, kv_scales), self._geometry)

    # -- entry points ------------------------------------------------------

    def append(self, chunk: Chunk, k, v, status, q=None, q_out=None, stream=None):
        """Store the chunk's k, v [T, n_kv, head_dim] (bf16 or fp32, rows strided), rotated where the cache
        rotates; with q [T, n_q, head_dim] also its rotation in bf16 into q_out."""
        n_kv, T, x = self._n_kv, self._mine(chunk), k.dtype
        io = (x,)
        ks, vs = self._rows(k, "k", n_kv, T, BOTH), self._rows(v, "v", n_kv, T, io)
        qp = op = None
        qs = os_ = 0
        if q is not None and q_out is not None:
            qs, qp = self._rows(q, "q", self._n_q, T, io), q.data_ptr()
            os_, op = self._rows(q_out, "q_out", self._n_q, T, BF16), q_out.data_ptr()
        elif q is not None or q_out is not None:
            raise ValueError("q and q_out come together")
        r = SdvAppendRows(k.data_ptr(), v.data_ptr(), qp, ks, vs, qs, 1 if x is torch.float32 else 0, op, os_)
        st, raw = self._enqueue(status, stream)
        rc = self.lib.sdv_cache_append(self.handle, chunk.ref, ctypes.byref(r), st, raw)
        if rc:
            self._check(rc, "sdv_cache_append")

    def attention(self, chunk: Chunk, q, out, status, stream=None):
        """Attention of q [T, n_q, head_dim] bf16 over the cached positions each row sees, into out."""
        n_q, T = self._n_q, self._mine(chunk)
        qs, os_ = self._rows(q, "q", n_q, T, BF16), self._rows(out, "out", n_q, T, BF16)
        st, raw = self._enqueue(status, stream)
        if raw not in self._streams:
            # the allocator hands the workspace on only when this stream's work has ended
            self.workspace.record_stream(torch.cuda.current_stream(self.device) if stream is None else stream)
            self._streams.add(raw)
        rc = self.lib.sdv_cache_attention(self.handle, chunk.ref, q.data_ptr(), qs, out.data_ptr(), os_, st, raw)
        if rc:
            self._check(rc, "sdv_cache_attention")

    def read(self, chunk: Chunk, k_out, v_out, status, stream=None):
        """Read the chunk's positions back into k_out, v_out [T, n_kv, head_dim] (bf16 or fp32; either may be None)."""
        n_kv, T = self._n_kv, self._mine(chunk)
        first = k_out if k_out is not None else v_out
        if first is None:
            raise ValueError("k_out, v_out: one of them is wanted")
        kp = vp = None
        ks = vs = 0
        if k_out is not None:
            ks, kp = self._rows(k_out, "k_out", n_kv, T, BOTH), k_out.data_ptr()
        if v_out is not None:
            vs, vp = self._rows(v_out, "v_out", n_kv, T, BOTH if k_out is None else (k_out.dtype,)), v_out.data_ptr()
        st, raw = self._enqueue(status, stream)
        rc = self.lib.sdv_cache_read(self.handle, chunk.ref, kp, ks, vp, vs, 1 if first.dtype is torch.float32 else 0, st, raw)
        if rc:
            self._check(rc, "sdv_cache_read")


class Tables:
    """The page tables of up to max_slots requests, their free stack, and a step's rows (sdv_cache_plan).

    Tensors, all int32 on the current device but slots (int64): page_table [max_slots, max_pages_per_seq], page_counts
    [max_slots], free_pages [num_pages] and num_free [1] are the state, at first every page free; row_offsets
    [max_slots + 1], row_request, positions, slots [max_rows] and last_rows [max_slots] describe the step that was
    planned last.  They keep their addresses, so that a chunk made of them serves every step, captured ones too; in a step
    of fewer requests than max_slots the others have no rows (last_rows -1).
    """

    def __init__(self, max_slots: int, max_rows: int, max_pages_per_seq: int, num_pages: int, lib_path: str | None = None):
        self.lib = load_library(lib_path) if lib_path else load_library()
        self.max_slots, self.max_rows = _c_int(max_slots), _c_int(max_rows)
        self.max_pages_per_seq, self.num_pages = _c_int(max_pages_per_seq), _c_int(num_pages)
        if not 0 < self.max_slots <= 1024 or self.max_rows < 0 or self.max_pages_per_seq <= 0 or self.num_pages <= 0:
            raise ValueError(f"max_slots {max_slots}, max_rows {max_rows}, max_pages_per_seq {max_pages_per_seq}, num_pages "
                             f"{num_pages}: 1 to 1024 slots and positive sizes are wanted")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.page_table = torch.full((self.max_slots, self.max_pages_per_seq), -1, **i32)
        self.page_counts = torch.zeros(self.max_slots, **i32)
        self.free_pages = torch.arange(self.num_pages - 1, -1, -1, **i32)
        self.num_free = torch.full((1,), self.num_pages, **i32)
        self.row_offsets = torch.zeros(self.max_slots + 1, **i32)
        self.row_request = torch.full((self.max_rows,), -1, **i32)
        self.positions = torch.full((self.max_rows,), -1, **i32)
        self.slots = torch.full((self.max_rows,), -1, dtype=torch.int64, device="cuda")
        self.last_rows = torch.full((self.max_slots,), -1, **i32)
        self.device = self.page_table.device
        self._index = self.page_table.get_device()
        self._structs = {}  # by the number of requests

    def _struct(self, B):
        s = SdvCacheTables(B, self.max_rows, None, None, self.page_table.data_ptr(), self.max_pages_per_seq,
                           self.page_counts.data_ptr(), self.free_pages.data_ptr(), self.num_pages, self.num_free.data_ptr(),
                           self.row_offsets.data_ptr(), self.row_request.data_ptr(), self.positions.data_ptr(),
                           self.last_rows.data_ptr(), self.slots.data_ptr(), self.max_slots)
        self._structs[B] = s, ctypes.byref(s)
        return self._structs[B]

    def plan(self, new_rows, lens, status, stream=None):
        """Plan a step of the first B requests: new_rows and lens [B] int32, the rows that each brings and its positions
        with them.  Requests behind the B keep their pages; end one by a length of 0."""
        for t, name in ((new_rows, "new_rows"), (lens, "lens")):
            if t.dtype is not torch.int32 or t.get_device() != self._index or t.dim() != 1 or not t.is_contiguous():
                raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device} (contiguous: {t.is_contiguous()}), "
                                 f"contiguous int32 [B] on {self.device} is wanted")
        B = lens.shape[0]
        if not 0 < B <= self.max_slots or new_rows.shape[0] != B:
            raise ValueError(f"new_rows {tuple(new_rows.shape)}, lens {tuple(lens.shape)}: one of each for 1 to "
                             f"{self.max_slots} requests is wanted")
        if status.dtype is not torch.int32 or status.get_device() != self._index:
            raise ValueError(f"status: {status.dtype} on {status.device}, int32 on {self.device} is wanted")
        if torch._C._cuda_getDevice() != self._index:
            raise ValueError(f"the current device is {torch.cuda.current_device()}, the tables are on {self.device}")
        s, ref = self._structs.get(B) or self._struct(B)
        s.new_rows, s.lens = new_rows.data_ptr(), lens.data_ptr()
        raw = torch._C._cuda_getCurrentRawStream(self._index) if stream is None else stream.cuda_stream
        rc = self.lib.sdv_cache_plan(ref, status.data_ptr(), raw)
        if rc:
            extra = f" (cuda error {self.lib.sdv_last_cuda_error()})" if rc == 4 else ""
            raise SdvError(rc, "sdv_cache_plan" + extra)
