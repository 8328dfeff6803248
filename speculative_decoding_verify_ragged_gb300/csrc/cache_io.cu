// Writing a chunk of new tokens into the paged cache and reading positions back.
#include "chunk.cuh"

namespace sdv {
namespace {

constexpr int IO_THREADS = 256;
constexpr int READ_BLOCKS = 8;  // blocks per SM (3, 4, 6 and 8: 45.9, 44.0, 44.4 and 42.6 us for 32749 bf16 rows)

// 8 or 4 consecutive elements as fp32, in one 16-byte load.
__device__ __forceinline__ void load_elements(const float* p, float (&x)[4]) {
  const float4 w = *reinterpret_cast<const float4*>(p);
  x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
}
__device__ __forceinline__ void load_elements(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float(ws[j] << 16);
    x[2 * j + 1] = __uint_as_float(ws[j] & 0xFFFF0000u);
  }
}

template <int N>
__device__ __forceinline__ void store_bf16(__nv_bfloat16* p, const float (&x)[N]) {
  uint32_t w[N / 2];
#pragma unroll
  for (int j = 0; j < N / 2; ++j) w[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
  if constexpr (N == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

template <int N>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&x)[N], float inv) {
  uint32_t w[N / 4];
#pragma unroll
  for (int j = 0; j < N / 4; ++j) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * j] * inv, x[4 * j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * j + 2] * inv, x[4 * j + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    w[j] = lo | (hi << 16);
  }
  if constexpr (N == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(p) = w[0];
}

// Smallest e in [kScaleMin, kScaleMax] with amax <= 448 * 2^e: with amax = m 2^x
// and m in [1, 2), 448 = 1.75 * 2^8 makes it x - 8 where m <= 1.75, else x - 7.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int x = static_cast<int>(b >> 23) - 127;
  return min(max(x - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0), kScaleMin), kScaleMax);
}

// Where row r of the chunk lives: its position (below 0: nowhere) and that
// position's page (-1: a bad page id, reported here).
__device__ __forceinline__ int2 row_place(const ChunkParams& c, const int* s_off, const int* s_len, int r) {
  const int b = row_sequence(s_off, c.B, r);
  const int pos = s_len[b] - s_off[b + 1] + r;
  if (pos < 0) return make_int2(pos, -1);
  int page = c.page_table[(long long)b * c.max_pages + pos / kPage];
  if (page < 0 || page >= c.pool_pages) {
    set_status(c.status, SDV_ERR_PAGE_RANGE);
    page = -1;
  }
  return make_int2(pos, page);
}

// A block takes `per` rows of the chunk at a time; a few lanes take one head of
// a row, each with the elements that the rotation pairs in both halves, so that
// rotation and row maximum stay in registers and every input is read once, in 16-byte
// loads, several heads' at a time.  The next rows' places, cosines and sines are
// made while these rows' data travels: one barrier a round.
//
// Angles: position * theta^(-2j/d) in turns is a product of integers modulo 2^64
// (RopeTurns), so far positions lose nothing; the quarter turns are taken off
// as integers before the rest is rounded to fp32.
//
// Bound by the input's bytes.  8192 rows of 48 heads of 128, fp32 to e4m3 and
// queries to bf16 (285 MB): 48.1 us, 5.9 TB/s.  3635 rows of 16 heads, bf16 (30 MB): 9.6 us, 3.1 TB/s: 909 blocks of
// one round each, of which 456 are resident, so two waves of waits, checks and loads.
template <int D, int FMT, typename T>
__global__ void __launch_bounds__(IO_THREADS)
    cache_append_kernel(const AppendParams p, const __grid_constant__ RopeTurns turns, int per) {
  extern __shared__ int s_meta[];
  constexpr int PAIRS = D / 2, ROWS = IO_THREADS / PAIRS;  // rows a round at most
  constexpr int N = 16 / sizeof(T), LANES = PAIRS / N, GROUPS = IO_THREADS / LANES;
  constexpr int AHEAD = sizeof(T) == 4 ? 4 : 2;            // heads a group has on their way
  __shared__ float2 s_cs[2][ROWS][PAIRS];
  __shared__ int2 s_place[2][ROWS];
  griddep_launch_dependents();
  griddep_wait();
  bool dead;
  int* s_off = s_meta;
  int* s_len = s_meta + p.c.B + 1;
  if (!load_chunk(p.c, s_off, s_len, dead) || dead) return;
  const int rows = s_off[p.c.B];
  const int n_kv = p.c.n_kv, heads = 2 * n_kv + (p.q_out ? p.c.n_q : 0);
  const int tid = threadIdx.x, group = tid / LANES, lane = tid % LANES;
  const unsigned long long turn = turns.f[tid % PAIRS];
  const unsigned mask = LANES == 32 ? 0xFFFFFFFFu : ((1u << LANES) - 1) << ((tid & 31) / LANES * LANES);
  auto prepare = [&](int r0, int buf) {
    const int k = tid / PAIRS;
    if (p.rope && k < per && r0 + k < rows) {
      const int b = row_sequence(s_off, p.c.B, r0 + k);
      const int pos = s_len[b] - s_off[b + 1] + r0 + k;  // (of a row below 0 nothing is used)
      const uint32_t t = static_cast<uint32_t>((turn * static_cast<unsigned long long>(max(pos, 0))) >> 32);
      const uint32_t quarter = (t + (1u << 29)) >> 30;
      const float x = static_cast<float>(static_cast<int>(t - (quarter << 30))) * 0x1p-31f;  // half turns, |x| <= 1/4
      float s, c;
      sincospif(x, &s, &c);
      const float sw = (quarter & 1) ? s : c;  // cos of the whole angle up to sign
      const float tw = (quarter & 1) ? c : s;
      s_cs[buf][k][tid % PAIRS] = make_float2(((quarter + 1) & 2) ? -sw : sw, (quarter & 2) ? -tw : tw);
    }
    if (tid < per && r0 + tid < rows) s_place[buf][tid] = row_place(p.c, s_off, s_len, r0 + tid);
  };
  const int step = gridDim.x * per;
  int buf = 0;
  if (blockIdx.x * per < rows) prepare(blockIdx.x * per, 0);
  __syncthreads();
  for (int r0 = blockIdx.x * per; r0 < rows; r0 += step, buf ^= 1) {
    const int items = min(per, rows - r0) * heads;
    bool made = false;
    for (int i0 = blockIdx.y * GROUPS + group; i0 < items || !made; i0 += AHEAD * GROUPS * gridDim.y) {
      float lo[AHEAD][N], hi[AHEAD][N];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int i = i0 + u * GROUPS * gridDim.y;
        if (i < items) {
          const int k = i / heads, h = i - k * heads, which = h < n_kv ? 0 : h < 2 * n_kv ? 1 : 2;  // key, value, query
          const T* src = reinterpret_cast<const T*>(which == 0 ? p.k : which == 1 ? p.v : p.q) +
                         (long long)(r0 + k) * (which == 0 ? p.k_stride : which == 1 ? p.v_stride : p.q_stride) +
                         (h - which * n_kv) * D + lane * N;
          load_elements(src, lo[u]);
          load_elements(src + PAIRS, hi[u]);
        }
      }
      if (!made) {
        made = true;
        if (r0 + step < rows) prepare(r0 + step, buf ^ 1);
      }
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int i = i0 + u * GROUPS * gridDim.y;
        if (i >= items) continue;
        const int k = i / heads, h = i - k * heads, which = h < n_kv ? 0 : h < 2 * n_kv ? 1 : 2, hh = h - which * n_kv;
        const int2 at = s_place[buf][k];
        if (at.x < 0) continue;
        if (p.rope && which != 1) {
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const float2 cs = s_cs[buf][k][lane * N + j];
            const float a = lo[u][j], c = hi[u][j];
            lo[u][j] = a * cs.x - c * cs.y;
            hi[u][j] = c * cs.x + a * cs.y;
          }
        }
        if (which == 2) {
          __nv_bfloat16* dst =
              reinterpret_cast<__nv_bfloat16*>(p.q_out) + (long long)(r0 + k) * p.q_out_stride + hh * D + lane * N;
          store_bf16(dst, lo[u]);
          store_bf16(dst + PAIRS, hi[u]);
          continue;
        }
        if (at.y < 0) continue;
        const long long place = (((long long)at.y * n_kv + hh) * 2 + which) * kPage + at.x % kPage;
        if constexpr (FMT == SDV_CACHE_BF16) {
          __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.c.pool) + place * D + lane * N;
          store_bf16(dst, lo[u]);
          store_bf16(dst + PAIRS, hi[u]);
        } else {
          float m = 0.f;  // fmaxf drops NaNs
#pragma unroll
          for (int j = 0; j < N; ++j) m = fmaxf(m, fmaxf(fabsf(lo[u][j]), fabsf(hi[u][j])));
#pragma unroll
          for (int o = LANES / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, o));
          const int e = scale_exponent(m);
          const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e
          uint8_t* dst = p.c.pool + place * D + lane * N;
          store_codes(dst, lo[u], inv);
          store_codes(dst + PAIRS, hi[u], inv);
          if (lane == 0) p.c.scales[place] = static_cast<uint8_t>(e + 127);
        }
      }
    }
    __syncthreads();
  }
}

// A warp takes a row (of few rows several take one), a lane 16 bytes of codes or
// 16-bit values of one of its heads, eight at a time; the next row's place is found meanwhile.  Bound by
// the bytes: 32749 positions of 8 heads of 128, bf16 (268 MB), 42.8 us, 6.3 TB/s; e4m3 to bf16 (202 MB) 41.9 us,
// 4.8 TB/s; to fp32, bf16 (402 MB) 77.3 us, 5.2 TB/s, e4m3 (336 MB) 84.6 us, 4.0 TB/s.
template <int D, int FMT, int OUT>
__global__ void __launch_bounds__(IO_THREADS) cache_read_kernel(const ReadParams p, int split) {
  extern __shared__ int s_meta[];
  constexpr int PER = FMT == SDV_CACHE_BF16 ? 8 : 16;  // elements a lane takes
  constexpr int LANES = D / PER, AHEAD = 8;
  griddep_launch_dependents();
  griddep_wait();
  bool dead;
  int* s_off = s_meta;
  int* s_len = s_meta + p.c.B + 1;
  if (!load_chunk(p.c, s_off, s_len, dead) || dead) return;
  // the heads asked for: keys, values or both
  const int n_kv = p.c.n_kv, first = p.k ? 0 : n_kv, pieces = ((p.v ? 2 * n_kv : n_kv) - first) * LANES;
  const int rows = s_off[p.c.B], wid = blockIdx.x * (IO_THREADS / kWarp) + (threadIdx.x >> 5);
  const int lane = (threadIdx.x & 31) + wid % split * kWarp, lanes = split * kWarp;  // of the row's
  const int warps = gridDim.x * (IO_THREADS / kWarp) / split;
  int r = wid / split;
  int2 next = r < rows ? row_place(p.c, s_off, s_len, r) : make_int2(-1, -1);
  for (; r < rows; r += warps) {
    const int2 at = next;
    const bool there = at.y >= 0;
    if (at.x >= 0 && !there) {  // a bad page id: reported, nothing written
      if (r + warps < rows) next = row_place(p.c, s_off, s_len, r + warps);
      continue;
    }
    const long long base = ((long long)(there ? at.y : 0) * n_kv * 2) * kPage + at.x % kPage;  // + (2 h + which) * 16
    for (int j0 = lane; j0 < pieces || j0 == lane; j0 += AHEAD * lanes) {
      uint4 w[AHEAD];
      float s[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int j = j0 + u * lanes, hw = first + j / LANES, which = hw >= n_kv, h = hw - which * n_kv;
        w[u] = make_uint4(0u, 0u, 0u, 0u);
        s[u] = 0.f;
        if (there && j < pieces) {
          const long long place = base + (2 * h + which) * kPage;
          w[u] = *reinterpret_cast<const uint4*>(p.c.pool + (place * D + j % LANES * PER) * (FMT == SDV_CACHE_BF16 ? 2 : 1));
          if constexpr (FMT == SDV_CACHE_E4M3) s[u] = scale_value(p.c.scales[place]);
        }
      }
      if (j0 == lane && r + warps < rows) next = row_place(p.c, s_off, s_len, r + warps);
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int j = j0 + u * lanes, hw = first + j / LANES, which = hw >= n_kv, h = hw - which * n_kv;
        if (j >= pieces) continue;
        const uint32_t ws[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        const long long to = (long long)r * (which ? p.v_stride : p.k_stride) + h * D + j % LANES * PER;
        void* out = which ? p.v : p.k;
        if constexpr (FMT == SDV_CACHE_BF16 && OUT == 0) {
          *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(out) + to) = w[u];
        } else {
          float x[PER];
          if constexpr (FMT == SDV_CACHE_BF16) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[2 * e] = __uint_as_float(ws[e] << 16);
              x[2 * e + 1] = __uint_as_float(ws[e] & 0xFFFF0000u);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t h2 = e4m3x2_to_f16x2(ws[e >> 1] >> (16 * (e & 1)));
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
              x[2 * e] = f.x * s[u];
              x[2 * e + 1] = f.y * s[u];
            }
          }
          if constexpr (OUT == 0) {
            uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(out) + to);
#pragma unroll
            for (int e = 0; e < PER; e += 8)
              dst[e / 8] = make_uint4(pack_bf16x2(x[e], x[e + 1]), pack_bf16x2(x[e + 2], x[e + 3]),
                                      pack_bf16x2(x[e + 4], x[e + 5]), pack_bf16x2(x[e + 6], x[e + 7]));
          } else {
            float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + to);
#pragma unroll
            for (int e = 0; e < PER; e += 4) dst[e / 4] = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
          }
        }
      }
    }
  }
}

size_t meta_bytes(int B) { return static_cast<size_t>(2 * B + 1) * sizeof(int); }

// Rows a block takes at a time: as many as leave every SM several blocks.
int rows_at_a_time(int T, int most, int blocks) {
  int per = 1;
  while (per < most && (T + 2 * per - 1) / (2 * per) >= blocks) per *= 2;
  return per;
}

template <int D, int FMT, typename T>
cudaError_t append_launch(const AppendParams& p, const RopeTurns& turns, int sms, cudaStream_t stream) {
  constexpr int GROUPS = IO_THREADS / (D / 2 / (16 / static_cast<int>(sizeof(T))));
  const int heads = 2 * p.c.n_kv + (p.q_out ? p.c.n_q : 0), passes = (heads + GROUPS - 1) / GROUPS;
  const int per = rows_at_a_time(p.c.T, IO_THREADS / (D / 2), sms * 4);
  // few rows: the heads of a row are spread over blocks as well
  const int y = (long long)p.c.T * passes <= sms * 4 ? passes : 1;
  const int want = (p.c.T + per - 1) / per, x = want < sms * 8 ? want : sms * 8;
  return launch_pdl(cache_append_kernel<D, FMT, T>, dim3(x, y), dim3(IO_THREADS), meta_bytes(p.c.B), stream, p, turns, per);
}

template <int D, int FMT, int OUT>
cudaError_t read_launch(const ReadParams& p, int sms, cudaStream_t stream) {
  constexpr int WARPS = IO_THREADS / kWarp;
  int split = 1;  // a divisor of the warps of a block
  while (split < WARPS && (long long)p.c.T * split < sms * WARPS * 2) split *= 2;
  const long long want = ((long long)p.c.T * split + WARPS - 1) / WARPS;
  const int grid = want < sms * READ_BLOCKS ? static_cast<int>(want) : sms * READ_BLOCKS;
  return launch_pdl(cache_read_kernel<D, FMT, OUT>, dim3(grid), dim3(IO_THREADS), meta_bytes(p.c.B), stream, p, split);
}

}  // namespace

cudaError_t launch_cache_append(int head_dim, int cache_format, int x_format, const AppendParams& p,
                                const RopeTurns& turns, int sms, cudaStream_t stream) {
#define SDV_APPEND(D)                                                                                            \
  return cache_format == SDV_CACHE_BF16                                                                          \
             ? (x_format ? append_launch<D, SDV_CACHE_BF16, float>(p, turns, sms, stream)                       \
                         : append_launch<D, SDV_CACHE_BF16, __nv_bfloat16>(p, turns, sms, stream))              \
             : (x_format ? append_launch<D, SDV_CACHE_E4M3, float>(p, turns, sms, stream)                       \
                         : append_launch<D, SDV_CACHE_E4M3, __nv_bfloat16>(p, turns, sms, stream))
  if (head_dim == 64) SDV_APPEND(64);
  SDV_APPEND(128);
#undef SDV_APPEND
}

cudaError_t launch_cache_read(int head_dim, int cache_format, int out_format, const ReadParams& p, int sms,
                              cudaStream_t stream) {
#define SDV_READ(D)                                                                                     \
  return cache_format == SDV_CACHE_BF16 ? (out_format ? read_launch<D, SDV_CACHE_BF16, 1>(p, sms, stream) \
                                                      : read_launch<D, SDV_CACHE_BF16, 0>(p, sms, stream)) \
                                        : (out_format ? read_launch<D, SDV_CACHE_E4M3, 1>(p, sms, stream) \
                                                      : read_launch<D, SDV_CACHE_E4M3, 0>(p, sms, stream))
  if (head_dim == 64) SDV_READ(64);
  SDV_READ(128);
#undef SDV_READ
}

}  // namespace sdv
