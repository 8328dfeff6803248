// Shared by the kernels over a ragged chunk of the paged cache (include/sdv_cache.h):
// the chunk's description on the device, its validation, and the 8-bit
// format's conversions.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "../../include/sdv_cache.h"
#include "common.cuh"
#include "internal.h"

namespace sdv {

constexpr int kPage = 16;
constexpr int kMaxChunkSlots = 1024;  // sequences of a chunk (their offsets and lengths sit in shared memory)
constexpr int kScaleMin = -15, kScaleMax = 7;  // exponents of the 8-bit cache's scales
constexpr float kCodeMax = 448.f;              // largest e4m3 value

struct ChunkParams {
  int B = 0, T = 0, max_q = 0, window = 0;
  const int* row_offsets = nullptr;
  const int* kv_lens = nullptr;
  uint8_t* pool = nullptr;
  uint8_t* scales = nullptr;
  const int* page_table = nullptr;
  int pool_pages = 0, max_pages = 0;
  int n_q = 0, n_kv = 0;
  int* status = nullptr;
};

// Sequence b of the chunk: rows [off, off + n), positions pos0 + i.
struct SeqRows {
  int off, n, len, pos0;
};

// Copy offsets [B + 1] and lengths [B] to shared memory and check them.  Every
// block of a launch reads the same words and comes to the same verdict, so a
// bad chunk stops all of them before any output.  `dead`: the status word was
// set already; another block may set it meanwhile, so the block's threads agree
// on what they saw.  Ends with a barrier.
__device__ __forceinline__ bool load_chunk(const ChunkParams& p, int* s_off, int* s_len, bool& dead) {
  int bad = 0;
  const int status = read_status(p.status);
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    const int o = p.row_offsets[b], e = p.row_offsets[b + 1], len = p.kv_lens[b];
    s_off[b] = o;
    if (b == p.B - 1) s_off[p.B] = e;
    s_len[b] = len;
    if (o < 0 || e < o || e > p.T || e - o > p.max_q || (b == 0 && o != 0) || len < 0) bad |= 1;
    if (len > (long long)p.max_pages * kPage) bad |= 2;
  }
  const bool b1 = __syncthreads_or(bad & 1), b2 = __syncthreads_or(bad & 2);
  dead = __syncthreads_or(status != 0);
  if ((b1 || b2) && threadIdx.x == 0) set_status(p.status, b1 ? SDV_ERR_BAD_INPUT : SDV_ERR_PAGE_RANGE);
  return !b1 && !b2;
}

__device__ __forceinline__ SeqRows seq_rows(const int* s_off, const int* s_len, int b) {
  const int o = s_off[b], n = s_off[b + 1] - o, len = s_len[b];
  return SeqRows{o, n, len, len - n};
}

// The sequence that owns row r (r < s_off[B]): the last b with s_off[b] <= r.
__device__ __forceinline__ int row_sequence(const int* s_off, int B, int r) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_off[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Cache loads are used once by this SM: kept out of L1.
__device__ __forceinline__ uint4 load16(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load8(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// Two e4m3 codes (low byte first) as fp16, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(x)));
  return r;
}

// 2^(byte - 127) as fp32, for bytes 1 .. 254 (the cache holds 112 .. 134).
__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float((byte & 0xFFu) << 23); }

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 2^x on the special-function unit; results below 2^-126 are 0.
__device__ __forceinline__ float fast_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct AppendParams {
  ChunkParams c;
  const void *k = nullptr, *v = nullptr, *q = nullptr;
  long long k_stride = 0, v_stride = 0, q_stride = 0;
  void* q_out = nullptr;
  long long q_out_stride = 0;
  int rope = 0;
};
// Per rotary pair j the angle's share of a turn per position, theta^(-2j/d) / (2 pi) as a 64-bit fraction.
struct RopeTurns {
  unsigned long long f[64];
};
cudaError_t launch_cache_append(int head_dim, int cache_format, int x_format, const AppendParams& p,
                                const RopeTurns& turns, int sms, cudaStream_t stream);

struct ReadParams {
  ChunkParams c;
  void *k = nullptr, *v = nullptr;
  long long k_stride = 0, v_stride = 0;
};
cudaError_t launch_cache_read(int head_dim, int cache_format, int out_format, const ReadParams& p, int sms,
                              cudaStream_t stream);

struct ChunkAttnParams {
  ChunkParams c;
  const __nv_bfloat16* q = nullptr;
  __nv_bfloat16* out = nullptr;
  long long q_stride = 0, out_stride = 0;
  float* part = nullptr;     // partial results of cut items, two per block of the launch
  int* counters = nullptr;   // arrivals at them, zero between launches
  int4* cuts = nullptr;      // tcgen05: [2 * blocks] the item of many parts that begins in each run
  int small_rows = 0;        // packed rows up to which a sequence is the mma.sync kernel's
  float scale_log2 = 0.f;    // log2(e) / sqrt(head_dim)
};
// Sequences of many rows on tcgen05, one block per SM (chunk_attention_tc.cu).
size_t chunk_attn_tc_part_floats(int head_dim, int grid);
cudaError_t setup_chunk_attn_tc(int head_dim, int cache_format);
cudaError_t launch_chunk_attn_tc(int head_dim, int cache_format, const CUtensorMap& map, const ChunkAttnParams& p, int grid,
                                 cudaStream_t stream);
// Sequences of few rows on mma.sync, in items of 8 (eight) or 16 packed rows
// (chunk_attention.cu); chunk_attn_grid_max: blocks of a launch at most.
constexpr int kItemRows = 16;
int chunk_attn_grid_max(int sms);
size_t chunk_attn_part_floats(int head_dim, int sms);
// Once per device before the first launch.
cudaError_t setup_chunk_attn(int head_dim, int cache_format);
cudaError_t launch_chunk_attn(int head_dim, int cache_format, bool eight, const ChunkAttnParams& p, int sms, cudaStream_t stream);

}  // namespace sdv
