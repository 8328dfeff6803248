// Writing a chunk of new tokens into the paged cache and reading positions back.
#include "chunk.cuh"

namespace sdv {
namespace {

constexpr int IO_THREADS = 256;

// 4 consecutive elements as fp32.
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xFFFF0000u));
}

__device__ __forceinline__ float max_abs(float m, const float4& a) {  // fmaxf drops NaNs
  return fmaxf(fmaxf(fmaxf(m, fabsf(a.x)), fmaxf(fabsf(a.y), fabsf(a.z))), fabsf(a.w));
}

// Smallest e in [kScaleMin, kScaleMax] with amax <= 448 * 2^e: with amax = m 2^x
// and m in [1, 2), 448 = 1.75 * 2^8 makes it x - 8 where m <= 1.75, else x - 7.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int x = static_cast<int>(b >> 23) - 127;
  return min(max(x - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0), kScaleMin), kScaleMax);
}

__device__ __forceinline__ uint32_t codes4(const float4& a, float inv) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a.x * inv, a.y * inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(a.z * inv, a.w * inv), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// One block takes rows of the chunk in turn; D / 8 lanes take one head of the
// row, each lane 4 elements of its lower half and the 4 that the rotation pairs
// them with in its upper half, so the rotation and the row maximum stay in
// registers and every input is read once.
//
// Angles: position * theta^(-2j/d) in turns is a product of integers modulo 2^64
// (RopeTurns), so far positions lose nothing; the quarter turns are taken off
// as integers before the rest is rounded to fp32.  Each row's cosines and
// sines are computed once for all its heads.
template <int D, int FMT, typename T>
__global__ void __launch_bounds__(IO_THREADS)
    cache_append_kernel(const AppendParams p, const __grid_constant__ RopeTurns turns) {
  extern __shared__ int s_meta[];
  __shared__ float2 s_cs[2][D / 2];
  constexpr int LANES = D / 8;
  constexpr int GROUPS = IO_THREADS / LANES;
  griddep_launch_dependents();
  griddep_wait();
  if (read_status(p.c.status) != 0) return;
  int* s_off = s_meta;
  int* s_len = s_meta + p.c.B + 1;
  if (!load_chunk(p.c, s_off, s_len)) return;
  const int rows = s_off[p.c.B];
  const int n_kv = p.c.n_kv, heads = 2 * n_kv + (p.q_out ? p.c.n_q : 0);
  const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES;
  const unsigned long long turn = turns.f[threadIdx.x % (D / 2)];
  const unsigned mask = LANES == 16 ? 0xFFFFu << (threadIdx.x & 16) : 0xFFu << (threadIdx.x & 24);
  int buf = 0;
  for (int r = blockIdx.x; r < rows; r += gridDim.x) {
    const int b = row_sequence(s_off, p.c.B, r);
    const int pos = s_len[b] - s_off[b + 1] + r;
    if (pos < 0) continue;  // the same for the whole block
    if (p.rope) {
      if (threadIdx.x < D / 2) {
        const uint32_t t = static_cast<uint32_t>((turn * static_cast<unsigned long long>(pos)) >> 32);
        const uint32_t quarter = (t + (1u << 29)) >> 30;
        const float x = static_cast<float>(static_cast<int>(t - (quarter << 30))) * 0x1p-31f;  // half turns, |x| <= 1/4
        float s, c;
        sincospif(x, &s, &c);
        const float sw = (quarter & 1) ? s : c;  // cos of the whole angle up to sign
        const float tw = (quarter & 1) ? c : s;
        s_cs[buf][threadIdx.x] = make_float2(((quarter + 1) & 2) ? -sw : sw, (quarter & 2) ? -tw : tw);
      }
      __syncthreads();
    }
    int page = -1;
    for (int h = blockIdx.y * GROUPS + group; h < heads; h += GROUPS * gridDim.y) {
      const int which = h < n_kv ? 0 : h < 2 * n_kv ? 1 : 2;  // key, value, query
      const int hh = h - which * n_kv;
      const T* src = reinterpret_cast<const T*>(which == 0 ? p.k : which == 1 ? p.v : p.q) +
                     (long long)r * (which == 0 ? p.k_stride : which == 1 ? p.v_stride : p.q_stride) + hh * D + lane * 4;
      float4 lo = load4(src), hi = load4(src + D / 2);
      if (p.rope && which != 1) {
        float* l = &lo.x;
        float* u = &hi.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 cs = s_cs[buf][lane * 4 + j];
          const float a = l[j], c = u[j];
          l[j] = a * cs.x - c * cs.y;
          u[j] = c * cs.x + a * cs.y;
        }
      }
      if (which == 2) {
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.q_out) + (long long)r * p.q_out_stride + hh * D + lane * 4;
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(lo.x, lo.y), pack_bf16x2(lo.z, lo.w));
        *reinterpret_cast<uint2*>(dst + D / 2) = make_uint2(pack_bf16x2(hi.x, hi.y), pack_bf16x2(hi.z, hi.w));
        continue;
      }
      if (page < 0) {
        page = p.c.page_table[(long long)b * p.c.max_pages + pos / kPage];
        if (page < 0 || page >= p.c.pool_pages) {
          set_status(p.c.status, SDV_ERR_PAGE_RANGE);
          page = -1;
        }
      }
      const long long place = (((long long)page * n_kv + hh) * 2 + which) * kPage + pos % kPage;
      if constexpr (FMT == SDV_CACHE_BF16) {
        if (page < 0) continue;
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.c.pool) + place * D + lane * 4;
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(lo.x, lo.y), pack_bf16x2(lo.z, lo.w));
        *reinterpret_cast<uint2*>(dst + D / 2) = make_uint2(pack_bf16x2(hi.x, hi.y), pack_bf16x2(hi.z, hi.w));
      } else {
        float m = max_abs(max_abs(0.f, lo), hi);
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, o));
        const int e = scale_exponent(m);
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e
        if (page < 0) continue;
        uint8_t* dst = p.c.pool + place * D + lane * 4;
        *reinterpret_cast<uint32_t*>(dst) = codes4(lo, inv);
        *reinterpret_cast<uint32_t*>(dst + D / 2) = codes4(hi, inv);
        if (lane == 0) p.c.scales[place] = static_cast<uint8_t>(e + 127);
      }
    }
    buf ^= 1;
  }
}

// Each group of lanes copies one (row, head, key or value): 16 bytes of codes
// or 16-bit values a lane.
template <int D, int FMT, int OUT>
__global__ void __launch_bounds__(IO_THREADS) cache_read_kernel(const ReadParams p) {
  extern __shared__ int s_meta[];
  constexpr int PER = FMT == SDV_CACHE_BF16 ? 8 : 16;  // elements a lane takes
  constexpr int LANES = D / PER;
  griddep_launch_dependents();
  griddep_wait();
  if (read_status(p.c.status) != 0) return;
  int* s_off = s_meta;
  int* s_len = s_meta + p.c.B + 1;
  if (!load_chunk(p.c, s_off, s_len)) return;
  const int n_kv = p.c.n_kv;
  const long long total = (long long)s_off[p.c.B] * n_kv * 2;
  const int lane = threadIdx.x % LANES;
  const long long step = (long long)gridDim.x * (IO_THREADS / LANES);
  for (long long i = (long long)blockIdx.x * (IO_THREADS / LANES) + threadIdx.x / LANES; i < total; i += step) {
    const int r = static_cast<int>(i / (2 * n_kv)), hw = static_cast<int>(i - (long long)r * 2 * n_kv);
    const int which = hw >= n_kv, h = hw - which * n_kv;
    void* base = which ? p.v : p.k;
    if (!base) continue;
    const int b = row_sequence(s_off, p.c.B, r);
    const int pos = s_len[b] - s_off[b + 1] + r;
    float x[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) x[j] = 0.f;
    if (pos >= 0) {
      const int page = p.c.page_table[(long long)b * p.c.max_pages + pos / kPage];
      if (page < 0 || page >= p.c.pool_pages) {
        set_status(p.c.status, SDV_ERR_PAGE_RANGE);
        continue;
      }
      const long long place = (((long long)page * n_kv + h) * 2 + which) * kPage + pos % kPage;
      if constexpr (FMT == SDV_CACHE_BF16) {
        const uint4 w = *reinterpret_cast<const uint4*>(p.c.pool + (place * D + lane * PER) * 2);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[2 * j] = __uint_as_float(ws[j] << 16);
          x[2 * j + 1] = __uint_as_float(ws[j] & 0xFFFF0000u);
        }
      } else {
        const uint4 w = *reinterpret_cast<const uint4*>(p.c.pool + place * D + lane * PER);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        const float s = scale_value(p.c.scales[place]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t h2 = e4m3x2_to_f16x2(ws[j >> 1] >> (16 * (j & 1)));
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
          x[2 * j] = f.x * s;
          x[2 * j + 1] = f.y * s;
        }
      }
    }
    const long long at = (long long)r * (which ? p.v_stride : p.k_stride) + h * D + lane * PER;
    if constexpr (OUT == 0) {
      uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(base) + at);
#pragma unroll
      for (int j = 0; j < PER; j += 8)
        dst[j / 8] = make_uint4(pack_bf16x2(x[j], x[j + 1]), pack_bf16x2(x[j + 2], x[j + 3]), pack_bf16x2(x[j + 4], x[j + 5]),
                                pack_bf16x2(x[j + 6], x[j + 7]));
    } else {
      float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + at);
#pragma unroll
      for (int j = 0; j < PER; j += 4) dst[j / 4] = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
    }
  }
}

size_t meta_bytes(int B) { return static_cast<size_t>(2 * B + 1) * sizeof(int); }

template <int D, int FMT, typename T>
cudaError_t append_launch(const AppendParams& p, const RopeTurns& turns, int sms, cudaStream_t stream) {
  constexpr int GROUPS = IO_THREADS / (D / 8);
  const int heads = 2 * p.c.n_kv + (p.q_out ? p.c.n_q : 0), passes = (heads + GROUPS - 1) / GROUPS;
  // few rows: the heads of a row are spread over blocks as well
  const int y = (long long)p.c.T * passes <= sms * 8 ? passes : 1;
  const int x = p.c.T < sms * 8 ? p.c.T : sms * 8;
  return launch_pdl(cache_append_kernel<D, FMT, T>, dim3(x, y), dim3(IO_THREADS), meta_bytes(p.c.B), stream, p, turns);
}

template <int D, int FMT, int OUT>
cudaError_t read_launch(const ReadParams& p, int sms, cudaStream_t stream) {
  constexpr int PER = FMT == SDV_CACHE_BF16 ? 8 : 16;
  const long long groups = (long long)p.c.T * p.c.n_kv * 2 * (D / PER);
  const long long want = (groups + IO_THREADS - 1) / IO_THREADS;
  const int grid = want < sms * 8 ? static_cast<int>(want) : sms * 8;
  return launch_pdl(cache_read_kernel<D, FMT, OUT>, dim3(grid), dim3(IO_THREADS), meta_bytes(p.c.B), stream, p);
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
