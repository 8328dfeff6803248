"""Rows of an input and of an output that share memory: the host's check against sets of bytes, and sampling's refusal."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROBE = r"""
#include <cstdio>
#include <set>
#include "rows.h"
int main() {
  int wrong = 0, shared = 0, apart = 0;
  for (int rows = 1; rows <= 4; ++rows)
    for (int pa = 1; pa <= 6; ++pa)
      for (int na = 1; na <= pa; ++na)
        for (int pb = 1; pb <= 6; ++pb)
          for (int nb = 1; nb <= pb; ++nb)
            for (int at = -30; at <= 30; ++at) {
              std::set<int> bytes;
              for (int r = 0; r < rows; ++r)
                for (int i = 0; i < na; ++i) bytes.insert(r * pa + i);
              bool want = false;
              for (int r = 0; r < rows; ++r)
                for (int i = 0; i < nb; ++i) want |= bytes.count(at + r * pb + i) > 0;
              const bool got = sdv::rows_share(reinterpret_cast<void*>(4096), pa, na, reinterpret_cast<void*>(4096 + at), pb, nb, rows);
              // of unlike pitches a shared byte is always found, and a range that lies apart never is one
              const bool meet = at < (rows - 1) * pa + na && -at < (rows - 1) * pb + nb;
              wrong += pa == pb || rows == 1 ? got != want : (want && !got) || (got && !meet);
              (want ? shared : apart) += 1;
            }
  std::printf("%d %d %d\n", wrong, shared, apart);
  return 0;
}
"""


def test_rows_share_is_what_sets_of_bytes_say(tmp_path):
    src, exe = tmp_path / "probe.cpp", tmp_path / "probe"
    src.write_text(PROBE)
    csrc = os.path.join(ROOT, "speculative_decoding_verify_ragged_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", csrc, str(src), "-o", str(exe)], check=True)
    wrong, shared, apart = map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split())
    assert wrong == 0 and shared > 1000 and apart > 1000


@pytest.mark.parametrize("io,logits,stride,probs,probs_stride", [
    (1, 4096, 64, 4096, 64),                    # in place
    (0, 4096, 64, 4096, 64), (0, 4096, 128, 4096, 64),
    (1, 4096, 64, 4096 + 4 * 63, 64),           # a row's end
    (1, 4096 + 4 * 200, 64, 4096, 64),          # the last row of one, the first of the other
    (1, 4096, 100, 4096 + 4 * 60, 100),         # columns of one buffer that meet
    (1, 4096, 64, 4096 + 4 * 4, 128)])
def test_sampling_refuses_probs_over_logits(io, logits, stride, probs, probs_stride):
    """The first reading of a row writes zeros to probs; a row that is read again would be computed from them."""
    from speculative_decoding_verify_ragged_gb300 import _abi
    lib = _abi.load_library()
    r = _abi.SdvSampleRows(logits, io, stride, 4, 64, 4, None, None, None, None, None, 1 << 20, 1 << 21, probs, probs_stride)
    assert lib.sdv_sample(ctypes.byref(r), ctypes.c_void_p(1 << 22), None) == _abi.SDV_ERR_INVALID_ARG
