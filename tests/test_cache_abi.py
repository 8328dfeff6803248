"""The paged cache's C ABI on the CPU: struct layouts and refusals before any CUDA call."""
import ctypes
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROBE = r"""
#include <stdio.h>
#include <stddef.h>
#include "sdv_cache.h"
#define F(T, f) printf(#T "." #f " %zu\n", offsetof(T, f));
int main(void) {
  printf("sdv_cache_config %zu\nsdv_chunk %zu\nsdv_append_rows %zu\n", sizeof(sdv_cache_config), sizeof(sdv_chunk),
         sizeof(sdv_append_rows));
  F(sdv_cache_config, rope_theta) F(sdv_chunk, row_offsets) F(sdv_chunk, num_pool_pages) F(sdv_chunk, page_table)
  F(sdv_chunk, window) F(sdv_append_rows, k_stride) F(sdv_append_rows, x_format) F(sdv_append_rows, q_out_stride)
  return 0;
}
"""


def test_layout(tmp_path):
    from speculative_decoding_verify_ragged_gb300 import _abi
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text(PROBE)
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    vals = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                        check=True).stdout.splitlines())
    names = dict(sdv_cache_config=_abi.SdvCacheConfig, sdv_chunk=_abi.SdvChunk, sdv_append_rows=_abi.SdvAppendRows)
    for key, want in vals.items():
        cls, _, field = key.partition(".")
        got = getattr(names[cls], field).offset if field else ctypes.sizeof(names[cls])
        assert got == int(want), key


def test_refusals_without_a_device():
    from speculative_decoding_verify_ragged_gb300 import _abi
    lib = _abi.load_library()
    bad, none = _abi.SDV_ERR_INVALID_ARG, ctypes.c_void_p()
    cfg = lambda *a: _abi.SdvCacheConfig(*a)  # noqa: E731
    good = (32, 8, 128, 16, 0, 1e6)
    for i, v in ((0, 0), (0, 33), (1, 0), (3, 32), (4, 2), (4, -1), (5, 0.5), (5, -1.0), (5, float("inf")), (5, float("nan"))):
        c = cfg(*[v if j == i else x for j, x in enumerate(good)])
        assert lib.sdv_cache_workspace_size(ctypes.byref(c), 8, 2) == 0
        assert lib.sdv_cache_create(ctypes.byref(c), ctypes.c_void_p(256), 1 << 30, 8, 2, None, ctypes.byref(none)) == bad
    c = cfg(32, 8, 96, 16, 0, 0.0)
    assert lib.sdv_cache_workspace_size(ctypes.byref(c), 8, 2) == 0
    assert lib.sdv_cache_create(ctypes.byref(c), ctypes.c_void_p(256), 1 << 30, 8, 2, None,
                                ctypes.byref(none)) == _abi.SDV_ERR_UNSUPPORTED
    c = cfg(*good)
    assert lib.sdv_cache_workspace_size(ctypes.byref(c), 0, 2) == 0
    assert lib.sdv_cache_workspace_size(ctypes.byref(c), 8, 1025) == 0
    assert lib.sdv_cache_create(ctypes.byref(c), ctypes.c_void_p(256), 1 << 30, 8, 1025, None,
                                ctypes.byref(none)) == _abi.SDV_ERR_CAPACITY
    assert lib.sdv_cache_create(ctypes.byref(c), ctypes.c_void_p(8), 1 << 30, 8, 2, None, ctypes.byref(none)) == bad
    assert lib.sdv_cache_create(None, ctypes.c_void_p(256), 1 << 30, 8, 2, None, ctypes.byref(none)) == bad
    assert lib.sdv_cache_create(ctypes.byref(c), ctypes.c_void_p(256), 1 << 30, 8, 2, None, None) == bad
    chunk, rows = _abi.SdvChunk(), _abi.SdvAppendRows()
    assert lib.sdv_cache_append(None, ctypes.byref(chunk), ctypes.byref(rows), None, None) == bad
    assert lib.sdv_cache_attention(None, ctypes.byref(chunk), None, 0, None, 0, None, None) == bad
    assert lib.sdv_cache_read(None, ctypes.byref(chunk), None, 0, None, 0, 0, None, None) == bad
    lib.sdv_cache_destroy(None)
