// Host checks of rows that a call reads and writes.
#pragma once
#include <cstdint>

namespace sdv {

// Whether `rows` rows of a and as many of b, each `bytes` long and `pitch` >= bytes apart, share memory.  Exact for one pitch (columns
// of one buffer); rows of unlike pitches count as shared where their address ranges meet.
inline bool rows_share(const void* a, long long a_pitch, long long a_bytes, const void* b, long long b_pitch, long long b_bytes,
                       long long rows) {
  const long long apart = static_cast<long long>(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  if (apart >= (rows - 1) * a_pitch + a_bytes || -apart >= (rows - 1) * b_pitch + b_bytes) return false;
  if (rows == 1 || a_pitch != b_pitch) return true;
  const long long column = (apart % a_pitch + a_pitch) % a_pitch;  // of b in a's rows
  return column < a_bytes || column + b_bytes > a_pitch;
}

}  // namespace sdv
