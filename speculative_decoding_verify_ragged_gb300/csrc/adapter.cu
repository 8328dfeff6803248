// Low-rank adapters of many requests beside a shared projection (include/sdv_adapter.h).
//
// One kernel, a cluster of blocks to an item of up to 32 or 64 rows of one request.  First v = scale * x A^T,
// the blocks sharing k: mma.sync with the ranks as the M side and eight rows as the N side, so
// that one row a request wastes the least.  A and x come by asynchronous copies in slabs of k, as many on
// their way as fit; a warp takes 16 rows and, as there are more warps, some of a slab's steps.
// The contraction is a sum, so its index may be permuted alike on both sides: a thread takes eight neighbouring k of a
// row of A and of x in one 16-byte load each.  The parts meet in shared memory, each block adding up its share of the
// values and all of them reading the sums.
//
// Then v B^T is added to base, the blocks sharing the features: features as the M side, numbered so that a thread
// ends with four neighbouring features of a row and eight lanes with a 128-byte line.  A warp holds its 32
// features' B in registers for all of the item's rows, the next ones' on its way; base comes by asynchronous copies, each
// thread's own, several tiles ahead and the first while v is still being made.
//
// v enters the second product as bf16 values that add up to it, three of them (2^-27)
// for an fp32 out, two (2^-18) for a bf16 one: what a rank value lost would be an error common to a whole row (of an fp32
// out 1.2e-6 with two).  Three serve fp32 x.  Both products are exact in fp32 but for their sums.
//
// Bound by the bytes in principle: A and B of the adapters in use, x, base and out.  Four prompts of 2015 rows, 4096 by 4096, rank 64
// (86 MB; a copy of base to out alone takes 17 us from cold): 39 us, of which v takes 18 -- slabs of x and A 8, the cluster's two
// meetings and the sums 9 -- and the rest the second product at the pace of base and out.  64 rows of as many adapters, rank 16,
// 4096 by 6144 (25 MB): 12 us, waits one after another (offsets, slabs 3, sums 2, B and base 2.5).  Before, two kernels with v in memory
// between them took 49 and 15 us.
#include <cooperative_groups.h>

#include <new>

#include "../../include/sdv_adapter.h"
#include "chunk.cuh"
#include "rows.h"

namespace cg = cooperative_groups;

namespace sdv {
namespace {

constexpr int AD_THREADS = 256, AD_WARPS = AD_THREADS / kWarp;
constexpr int MAX_RANK = 128, MAX_CLUSTER = 8;

struct AdapterParams {
  sdv_adapter_rows r;
  int k, n, rank, count;
  const __nv_bfloat16 *a, *b;
  const float* scales;
  int item_rows;  // 32 or 64
  int* status;
};

// The batch's rows in items of up to item_rows rows of one request, numbered over the requests: first those of requests of more than a
// tile, then the others', which take a fraction of their time and fill what the long ones leave.
struct Items {
  int* off;    // [B + 1] row offsets
  int* first;  // [B + 1] first item of each long request
  int* brief;  // [B + 1] that of each other one, counted from 0
  int* id;     // [B]
};
constexpr int kItemInts = 4 * kMaxChunkSlots + 3;

// Offsets, adapters and items to shared memory, checked; every block comes to the same verdict, as nothing here writes what they
// read.  Requests without an adapter have items only if `all`.  Ends with a barrier.
__device__ __forceinline__ bool load_items(const AdapterParams& p, const Items& it, bool all, long long* s_warp) {
  int bad = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long base = 0;  // long items in steps of 2^11, others in ones
  for (int b0 = 0; b0 < p.r.B; b0 += AD_THREADS) {
    const int b = b0 + threadIdx.x;
    long long items = 0;
    if (b < p.r.B) {
      const int o = p.r.row_offsets[b], e = p.r.row_offsets[b + 1], id = p.r.adapter_ids[b];
      it.off[b] = o;
      if (b == p.r.B - 1) it.off[p.r.B] = e;
      it.id[b] = id;
      if (o < 0 || e < o || e > p.r.T || (b == 0 && o != 0) || id >= p.count) bad = 1;
      else if (all || id >= 0) items = e - o > 8 ? ((0LL + e - o + p.item_rows - 1) / p.item_rows) << 11 : e > o ? 1 : 0;
    }
    long long incl = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    long long before = base, total = base;
    for (int w = 0; w < AD_WARPS; ++w) {
      if (w < warp) before += s_warp[w];
      total += s_warp[w];
    }
    before += incl - items;
    if (b < p.r.B) it.first[b] = static_cast<int>(before >> 11), it.brief[b] = static_cast<int>(before & 2047);
    base = total;
    __syncthreads();
  }
  if (threadIdx.x == 0) it.first[p.r.B] = static_cast<int>(base >> 11), it.brief[p.r.B] = static_cast<int>(base & 2047);
  const bool found = __syncthreads_or(bad);
  if (found && threadIdx.x == 0) set_status(p.status, SDV_ERR_BAD_INPUT);
  return !found;
}

// The last request whose first item, in `first`, is i or before.
__device__ __forceinline__ int item_request(const int* first, int B, int i) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// x as the sum of P bf16 (within 2^-9P of it), pairs packed.  All but the last stop at bf16's largest value: what lies between it and
// fp32's keeps its rest, and an infinity stays one in the sum (an infinite first part would leave inf - inf to the others).
template <int P>
__device__ __forceinline__ void split(float x0, float x1, uint32_t (&w)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (i < P - 1) asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x1), "f"(x0));
    else w[i] = pack_bf16x2(x0, x1);
    x0 -= __uint_as_float(w[i] << 16);
    x1 -= __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void copy16(void* to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(there ? 16 : 0) : "memory");
}

// Shared memory of a block, two to an SM.  First slabs of k: rows of A, then rows of x.  Then, in their place: the block's part of v, the sums of its
// share of the values, v's planes of bf16 pairs, and base on its way.
// Rows of A and x lie end to end, of every other row the 64-byte halves of each line swapped (of fp32 x the 16-byte
// pieces), so that the four neighbouring lanes of two rows, who read together, meet no bank twice.
template <int MT, bool XF, bool YF>
struct Layout {
  static constexpr int SPACE = 96 * 1024;
  static constexpr int ROWS = MT == 8 ? 32 : 64;  // of an item at most
  static constexpr int K = MT == 1 && !XF ? 256 : MT <= 4 ? 128 : 64;
  static constexpr int XB = XF ? 4 : 2, X_PLANES = XF ? 3 : 1, V_PLANES = YF ? 3 : 2;
  static constexpr int A_PITCH = K * 2, X_PITCH = K * XB, A_BYTES = MT * 16 * A_PITCH;
  static constexpr int A_SWAP = 4, X_SWAP = XF ? 1 : 4;  // of a 16-byte piece's number, in odd rows
  static_assert(2 * (A_BYTES + ROWS * X_PITCH) <= SPACE, "two slabs at least");
  static constexpr int R = MT * 16, PITCH = MT == 1 ? 8 : R / 2 + 8, PLANE = ROWS * PITCH;  // pairs; a row starts 8 banks on
  static constexpr int SUMS = ROWS * R * 4, PLANES = SUMS + SUMS / 2;  // (a cluster is two blocks at least)
  static constexpr int PARTS = AD_WARPS * 16 * R * 4;                  // of v, one of each warp's rows
  static constexpr int RING = PLANES + V_PLANES * PLANE * 4 > PARTS ? PLANES + V_PLANES * PLANE * 4 : PARTS;
  static constexpr int QUAD = 4 * (YF ? 4 : 2), STEP = 2 * AD_THREADS * QUAD;  // bytes of a thread's four values, and of a step's
  static constexpr int STEPS = (SPACE - RING) / STEP < 8 ? (SPACE - RING) / STEP : 8;
  static_assert(STEPS >= 2, "a step ahead at least");
};

// Four neighbouring values of a row of base, on their way through shared memory, and of out.
template <bool YF>
__device__ __forceinline__ void quad_copy(uint32_t to, const uint8_t* from) {
  if constexpr (YF) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
template <bool YF>
__device__ __forceinline__ void quad_add_store(const uint8_t* base, uint8_t* out, float d0, float d1, float d2, float d3) {
  if constexpr (YF) {
    const float4 w = *reinterpret_cast<const float4*>(base);
    *reinterpret_cast<float4*>(out) = make_float4(w.x + d0, w.y + d1, w.z + d2, w.w + d3);
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(base);
    uint2 o;
    o.x = pack_bf16x2(__uint_as_float(w.x << 16) + d0, __uint_as_float(w.x & 0xFFFF0000u) + d1);
    o.y = pack_bf16x2(__uint_as_float(w.y << 16) + d2, __uint_as_float(w.y & 0xFFFF0000u) + d3);
    *reinterpret_cast<uint2*>(out) = o;
  }
}

constexpr int GROUP = 32;  // features a warp takes at a time

template <int N>
__device__ __forceinline__ void wait_copies() {  // all but the newest N groups
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// MT: rank in sixteens (and the A side's tiles).  XF, YF: fp32 x, fp32 base and out.
template <int MT, bool XF, bool YF>
__global__ void __launch_bounds__(AD_THREADS, 2) adapter_kernel(const AdapterParams p) {
  using L = Layout<MT, XF, YF>;
  constexpr int R = L::R;
  constexpr bool EARLY = MT <= 4;  // registers for the next features' B
  extern __shared__ __align__(16) uint8_t s_space[];
  __shared__ int s_items[kItemInts];
  __shared__ long long s_warp[AD_WARPS];
  __shared__ int s_dead;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), blocks = cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  griddep_launch_dependents();
  griddep_wait();
  const Items it{s_items, s_items + kMaxChunkSlots + 1, s_items + 2 * kMaxChunkSlots + 2, s_items + 3 * kMaxChunkSlots + 3};
  if (tid == 0 && rank == 0) s_dead = read_status(p.status);
  if (!load_items(p, it, p.r.out != p.r.base, s_warp)) return;
  // the word may be set meanwhile by a call on another stream: the cluster's blocks go by the first one's view, which they look at
  // when they next meet
  cluster.barrier_arrive();
  bool met = false;
  auto dead = [&] {
    if (met) return false;
    met = true;
    cluster.barrier_wait();
    return *cluster.map_shared_rank(&s_dead, 0) != 0;
  };
  float* const part = reinterpret_cast<float*>(s_space);                // [rows][R], this block's share of k
  float* const sums = reinterpret_cast<float*>(s_space + L::SUMS);      // its share of the values, over all blocks
  uint32_t* const planes = reinterpret_cast<uint32_t*>(s_space + L::PLANES);
  constexpr int YB = L::QUAD / 4;
  uint8_t* const ring = s_space + L::RING + tid * L::QUAD;
  const uint32_t ring_at = smem_u32(ring);
  const long long base_row = p.r.base_stride * YB, out_row = p.r.out_stride * YB;  // bytes
  const int long_items = it.first[p.r.B], items = long_items + it.brief[p.r.B], clusters = gridDim.x / blocks;
  // the cluster's warps side by side along the features: what they read and write at a time lies together
  const int groups = (p.n + GROUP - 1) / GROUP, g_begin = rank * AD_WARPS + warp, g_stride = blocks * AD_WARPS;
  const int k_share = ((p.k + blocks - 1) / blocks + 31) / 32 * 32, k_begin = rank * k_share, k_end = min(p.k, k_begin + k_share);
  const int slabs = k_end > k_begin ? (k_end - k_begin + L::K - 1) / L::K : 0;
  for (int item = blockIdx.x / blocks; item < items; item += clusters) {
    const bool is_long = item < long_items;
    const int b = is_long ? item_request(it.first, p.r.B, item) : item_request(it.brief, p.r.B, item - long_items);
    const int row0 = it.off[b] + (is_long ? item - it.first[b] : 0) * p.item_rows, rows = min(p.item_rows, it.off[b + 1] - row0);
    const int id = it.id[b], tiles = (rows + 7) >> 3;
    // this thread's values: rows q * 2 and q * 2 + 1 of a tile, features g * 4 .. of a group
    const uint8_t* const base_at = static_cast<const uint8_t*>(p.r.base) + (row0 + q * 2) * base_row + g * 4 * YB;
    uint8_t* const out_at = static_cast<uint8_t*>(p.r.out) + (row0 + q * 2) * out_row + g * 4 * YB;
    int ask_grp = g_begin, ask_t = 0, ask_slot = 0;
    auto ask_base = [&] {
      if (ask_grp < groups) {
        const uint8_t* from = base_at + ask_t * 8 * base_row + ask_grp * (GROUP * YB);
        const uint32_t to = ring_at + ask_slot * L::STEP;
        const int left = ask_grp * GROUP + g * 4 < p.n ? rows - ask_t * 8 - q * 2 : 0;
        if (left > 0) quad_copy<YF>(to, from);
        if (left > 1) quad_copy<YF>(to + AD_THREADS * L::QUAD, from + base_row);
        if (++ask_t == tiles) ask_t = 0, ask_grp += g_stride;
        if (++ask_slot == L::STEPS) ask_slot = 0;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    uint2 fb[MT][4], next[EARLY ? MT : 1][4];
    auto ask_b = [&](auto& w, int grp) {
      const int f = grp * GROUP + g * 4;
      const __nv_bfloat16* at = p.b + ((long long)id * p.n + f) * p.rank;
#pragma unroll
      for (int d = 0; d < MT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = d * 16 + q * 4;
          w[d][e] = id >= 0 && grp < groups && f < p.n && j < p.rank ? __ldg(reinterpret_cast<const uint2*>(at + e * p.rank + j)) : make_uint2(0, 0);
        }
    };
    if (id >= 0) {
      const __nv_bfloat16* a = p.a + (long long)id * p.rank * p.k;
      const uint8_t* x = static_cast<const uint8_t*>(p.r.x) + (long long)row0 * p.r.x_stride * L::XB;
      const int bytes = L::A_BYTES + tiles * 8 * L::X_PITCH, stages = min(8, L::SPACE / bytes);
      // one group of copies to a slab, empty past the last
      auto ask = [&](int n) {
        if (n < slabs) {
          uint8_t* to = s_space + (n % stages) * bytes;
          const int k0 = k_begin + n * L::K;
          constexpr int AC = L::K / 8, XC = L::K * L::XB / 16;  // 16-byte pieces of a row
          for (int i = tid; i < R * AC; i += AD_THREADS) {
            const int j = i / AC, c = i - j * AC, k = k0 + c * 8;
            const bool in = j < p.rank && k < k_end;
            copy16(to + j * L::A_PITCH + (c ^ (j & 1) * L::A_SWAP) * 16, in ? a + (long long)j * p.k + k : a, in);
          }
          to += L::A_BYTES;
          for (int i = tid; i < tiles * 8 * XC; i += AD_THREADS) {
            const int r = i / XC, c = i - r * XC, k = k0 + c * (16 / L::XB);
            const bool in = r < rows && k < k_end;
            copy16(to + r * L::X_PITCH + (c ^ (r & 1) * L::X_SWAP) * 16, in ? x + ((long long)r * p.r.x_stride + k) * L::XB : x, in);
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      // warps to pairs of tiles, up to four, and to a slab's steps
      const int pairs = tiles > 4 ? 4 : tiles > 2 ? 2 : 1, pair = warp & (pairs - 1), share = warp / pairs, shares = AD_WARPS / pairs;
      float acc[2][MT][4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[t][m][e] = 0.f;
      for (int n = 0; n < stages - 1; ++n) ask(n);
      for (int n = 0; n < slabs; ++n) {
        switch (stages) {  // this slab's group: stages - 2 may be on their way behind it
          case 2: wait_copies<0>(); break;
          case 3: wait_copies<1>(); break;
          case 4: wait_copies<2>(); break;
          case 5: wait_copies<3>(); break;
          case 6: wait_copies<4>(); break;
          case 7: wait_copies<5>(); break;
          default: wait_copies<6>(); break;
        }
        __syncthreads();
        ask(n + stages - 1);
        const uint8_t* sa = s_space + (n % stages) * bytes;
        const int odd = g & 1;  // (of rows of A and of x)
        // a slab's products by themselves: the MMAs cut where they add, so chains are kept short (with 10^4 terms of fp32 x an fp32 out
        // was up to 1.3e-6 off), and slabs add up rounded
        float add[2][MT][4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) add[t][m][e] = 0.f;
        for (int step = share; step < L::K / 32; step += shares) {
          uint32_t fx[2][L::X_PLANES][4];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (pair * 2 + t >= tiles) break;
            const uint8_t* sx = sa + L::A_BYTES + ((pair * 2 + t) * 8 + g) * L::X_PITCH;
            if constexpr (XF) {
              const int c = step * 8 + q * 2;
              const float4 lo = *reinterpret_cast<const float4*>(sx + (c ^ odd) * 16), hi = *reinterpret_cast<const float4*>(sx + ((c + 1) ^ odd) * 16);
              const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t w[L::X_PLANES];
                split<L::X_PLANES>(f[2 * e], f[2 * e + 1], w);
#pragma unroll
                for (int i = 0; i < L::X_PLANES; ++i) fx[t][i][e] = w[i];
              }
            } else {
              const uint4 w = *reinterpret_cast<const uint4*>(sx + ((step * 4 + q) ^ odd * L::X_SWAP) * 16);
              fx[t][0][0] = w.x, fx[t][0][1] = w.y, fx[t][0][2] = w.z, fx[t][0][3] = w.w;
            }
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const int c = ((step * 4 + q) ^ odd * L::A_SWAP) * 16;
            const uint4 f0 = *reinterpret_cast<const uint4*>(sa + (m * 16 + g) * L::A_PITCH + c);
            const uint4 f1 = *reinterpret_cast<const uint4*>(sa + (m * 16 + 8 + g) * L::A_PITCH + c);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (pair * 2 + t >= tiles) break;
#pragma unroll
              for (int i = L::X_PLANES - 1; i >= 0; --i) {
                mma_bf16(add[t][m], {f0.x, f1.x, f0.y, f1.y}, fx[t][i][0], fx[t][i][1]);
                mma_bf16(add[t][m], {f0.z, f1.z, f0.w, f1.w}, fx[t][i][2], fx[t][i][3]);
              }
            }
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[t][m][e] += add[t][m][e];
      }
      wait_copies<0>();
      __syncthreads();  // the slabs have been read
      // the shares' parts, [share][row][R], then their sum in place of the first.  Ranks behind the adapter's are 0 whatever x is (an
      // infinity times their zeros is not)
      const int stride = tiles * 8 * R;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int tile = pair * 2 + t;
        if (tile >= tiles) break;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            part[share * stride + (tile * 8 + q * 2 + (e & 1)) * R + m * 16 + g + (e >> 1) * 8] = m * 16 + (e >> 1) * 8 < p.rank ? acc[t][m][e] : 0.f;
      }
      __syncthreads();
      constexpr int OWN = L::ROWS * R / AD_THREADS;
      float own[OWN];
#pragma unroll
      for (int c = 0; c < OWN; ++c) {
        const int i = c * AD_THREADS + tid;
        own[c] = 0.f;
        if (i < stride)
          for (int w = 0; w < shares; ++w) own[c] += part[w * stride + i];
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < OWN; ++c)
        if (c * AD_THREADS + tid < stride) part[c * AD_THREADS + tid] = own[c];
      if (dead()) {
        wait_copies<0>();
        cluster.sync();  // (the first block's word has been read)
        return;
      }
      cluster.sync();
      const float scale = p.scales[id];
      auto put = [&](int i, float2 v) {  // pair i of the values, to the planes
        const int r = i / (R / 2), j = i - r * (R / 2);
        uint32_t w[L::V_PLANES];
        split<L::V_PLANES>(v.x, v.y, w);
#pragma unroll
        for (int e = 0; e < L::V_PLANES; ++e) planes[e * L::PLANE + r * L::PITCH + j] = w[e];
      };
      if (stride <= 2 * AD_THREADS) {
        // few values: every block adds up all of them
        for (int i = tid; i < stride / 2; i += AD_THREADS) {
          float2 v = make_float2(0.f, 0.f), x[MAX_CLUSTER];  // (all asked for before the first is used)
#pragma unroll
          for (int o = 0; o < MAX_CLUSTER; ++o)
            x[o] = o < blocks ? reinterpret_cast<const float2*>(cluster.map_shared_rank(part, o))[i] : make_float2(0.f, 0.f);
#pragma unroll
          for (int o = 0; o < MAX_CLUSTER; ++o) v.x += x[o].x, v.y += x[o].y;
          put(i, make_float2(scale * v.x, scale * v.y));
        }
      } else {
        // each block adds up its share (stride: 128 or more a tile; blocks 2, 4 or 8) and reads the others'
        const int chunk = stride / blocks;
        for (int i = tid; i < chunk / 4; i += AD_THREADS) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f), x[MAX_CLUSTER];
#pragma unroll
          for (int o = 0; o < MAX_CLUSTER; ++o)
            x[o] = o < blocks ? reinterpret_cast<const float4*>(cluster.map_shared_rank(part, o) + rank * chunk)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int o = 0; o < MAX_CLUSTER; ++o) v.x += x[o].x, v.y += x[o].y, v.z += x[o].z, v.w += x[o].w;
          reinterpret_cast<float4*>(sums)[i] = make_float4(scale * v.x, scale * v.y, scale * v.z, scale * v.w);
        }
        cluster.sync();
        constexpr int MINE = (L::ROWS * R / 4 + AD_THREADS - 1) / AD_THREADS;
        float4 v[MINE];
#pragma unroll
        for (int c = 0; c < MINE; ++c) {
          const int i = c * AD_THREADS + tid, o = min(4 * i / chunk, blocks - 1);
          v[c] = i < stride / 4 ? reinterpret_cast<const float4*>(cluster.map_shared_rank(sums, o))[i - o * (chunk / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int c = 0; c < MINE; ++c) {
          const int i = c * AD_THREADS + tid;
          if (i < stride / 4) {
            put(2 * i, make_float2(v[c].x, v[c].y));
            put(2 * i + 1, make_float2(v[c].z, v[c].w));
          }
        }
      }
      cluster.barrier_arrive();  // this block has read the others' values; it waits for them to have read its own at the item's end
#pragma unroll
      for (int n = 0; n < L::STEPS - 1; ++n) ask_base();
      if constexpr (EARLY) ask_b(next, g_begin);
      __syncthreads();
    } else {
      if (dead()) {
        cluster.sync();
        return;
      }
#pragma unroll
      for (int n = 0; n < L::STEPS - 1; ++n) ask_base();
    }
    int slot = 0;
    const uint32_t* const at_planes = planes + g * L::PITCH + q * 2;
    for (int grp = g_begin; grp < groups; grp += g_stride) {
      if constexpr (EARLY) {
#pragma unroll
        for (int d = 0; d < MT; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) fb[d][e] = next[d][e];
        ask_b(next, grp + g_stride);
      } else {
        ask_b(fb, grp);
      }
      uint8_t* to = out_at + grp * (GROUP * YB);
      int left = grp * GROUP + g * 4 < p.n ? rows - q * 2 : 0;  // of this thread's rows
      const uint32_t* v = at_planes;
      for (int t = 0; t < tiles; ++t, to += 8 * out_row, left -= 8, v += 8 * L::PITCH) {
        ask_base();
        // (a plane's products apart: shorter chains)
        float acc[L::V_PLANES][2][4];
#pragma unroll
        for (int i = 0; i < L::V_PLANES; ++i)
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][m][e] = 0.f;
        if (id >= 0) {
#pragma unroll
          for (int d = 0; d < MT; ++d)
#pragma unroll
            for (int i = L::V_PLANES - 1; i >= 0; --i) {
              const uint2 x = *reinterpret_cast<const uint2*>(v + i * L::PLANE + d * 8);
              mma_bf16(acc[i][0], {fb[d][0].x, fb[d][1].x, fb[d][0].y, fb[d][1].y}, x.x, x.y);
              mma_bf16(acc[i][1], {fb[d][2].x, fb[d][3].x, fb[d][2].y, fb[d][3].y}, x.x, x.y);
            }
        }
#pragma unroll
        for (int i = L::V_PLANES - 1; i > 0; --i)
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i - 1][m][e] += acc[i][m][e];
        wait_copies<L::STEPS - 1>();
        const uint8_t* from = ring + slot * L::STEP;
        if (left > 0) quad_add_store<YF>(from, to, acc[0][0][0], acc[0][0][2], acc[0][1][0], acc[0][1][2]);
        if (left > 1) quad_add_store<YF>(from + AD_THREADS * L::QUAD, to + out_row, acc[0][0][1], acc[0][0][3], acc[0][1][1], acc[0][1][3]);
        if (++slot == L::STEPS) slot = 0;
      }
    }
    wait_copies<0>();
    if (id >= 0) cluster.barrier_wait();
    __syncthreads();  // planes and base have been read
  }
  if (!met) cluster.barrier_wait();
  cluster.sync();  // (the first block's word has been read)
}

}  // namespace
}  // namespace sdv

using namespace sdv;

struct sdv_adapters {
  sdv_adapter_config cfg;
  int device, sms, max_rows, max_slots;
};

namespace {

bool config_ok(const sdv_adapter_config* c) {
  return c && c->k > 0 && c->n > 0 && c->rank > 0 && c->count > 0 && c->k % 8 == 0 && c->n % 8 == 0 && c->rank % 8 == 0 &&
         c->rank <= MAX_RANK && c->k <= (1 << 24) && c->n <= (1 << 24);
}

int sms_of(int dev) {
  int n = 0;
  return cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? n : 0;
}
bool aligned(const void* p, int to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

template <int MT, bool XF, bool YF>
cudaError_t start(AdapterParams p, int sms, cudaStream_t stream) {
  using L = Layout<MT, XF, YF>;
  p.item_rows = L::ROWS == 64 && p.r.T >= 128LL * p.r.B ? 64 : 32;
  // items at most; a cluster as large as lets two in three of them run at once, two blocks to an SM: an item's time is mostly
  // waits, and many are short ones
  const long long items = (0LL + p.r.T + p.item_rows - 1) / p.item_rows + (p.r.B < p.r.T ? p.r.B : p.r.T) - 1;
  int cluster = MAX_CLUSTER;
  while (cluster > 2 && items * cluster > 3 * sms) cluster /= 2;
  const int most = 2 * sms / cluster * 4, clusters = static_cast<int>(items < most ? items : most);
  return launch_pdl_cluster(adapter_kernel<MT, XF, YF>, cluster, dim3(clusters * cluster), dim3(AD_THREADS), L::SPACE, stream, p);
}
template <int MT>
cudaError_t start(const AdapterParams& p, int sms, cudaStream_t stream) {
  return p.r.x_format ? (p.r.y_format ? start<MT, true, true>(p, sms, stream) : start<MT, true, false>(p, sms, stream))
                      : (p.r.y_format ? start<MT, false, true>(p, sms, stream) : start<MT, false, false>(p, sms, stream));
}
// The size of shared memory that the kernels of a rank may take, once per device.
template <int MT>
cudaError_t setup() {
  const auto allow = [](const void* kernel, int bytes) { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); };
  cudaError_t e = allow(reinterpret_cast<const void*>(adapter_kernel<MT, false, false>), Layout<MT, false, false>::SPACE);
  if (e == cudaSuccess) e = allow(reinterpret_cast<const void*>(adapter_kernel<MT, false, true>), Layout<MT, false, true>::SPACE);
  if (e == cudaSuccess) e = allow(reinterpret_cast<const void*>(adapter_kernel<MT, true, false>), Layout<MT, true, false>::SPACE);
  if (e == cudaSuccess) e = allow(reinterpret_cast<const void*>(adapter_kernel<MT, true, true>), Layout<MT, true, true>::SPACE);
  return e;
}

}  // namespace

extern "C" sdv_status sdv_adapters_create(const sdv_adapter_config* cfg, int max_rows, int max_slots, sdv_adapters** out) {
  if (!out) return SDV_ERR_INVALID_ARG;
  *out = nullptr;
  if (!config_ok(cfg) || !cfg->a || !cfg->b || !cfg->scales || !aligned(cfg->a, 16) || !aligned(cfg->b, 16) ||
      !aligned(cfg->scales, 4) || max_rows <= 0 || max_slots <= 0)
    return SDV_ERR_INVALID_ARG;
  if (max_slots > kMaxChunkSlots) return SDV_ERR_CAPACITY;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  const int sms = sms_of(dev);
  const int mt = (cfg->rank + 15) / 16;
  e = mt <= 1 ? setup<1>() : mt <= 2 ? setup<2>() : mt <= 4 ? setup<4>() : setup<8>();
  if (e != cudaSuccess) return cuda_fail(e);
  sdv_adapters* h = new (std::nothrow) sdv_adapters;
  if (!h) return SDV_ERR_INTERNAL;
  *h = sdv_adapters{*cfg, dev, sms, max_rows, max_slots};
  *out = h;
  return SDV_OK;
}

extern "C" void sdv_adapters_destroy(sdv_adapters* h) { delete h; }

extern "C" sdv_status sdv_adapters_apply(sdv_adapters* h, const sdv_adapter_rows* r, int* status, void* stream) {
  if (!h || !r || !status) return SDV_ERR_INVALID_ARG;
  if (r->B <= 0 || r->T < 0 || (r->x_format != 0 && r->x_format != 1) || (r->y_format != 0 && r->y_format != 1))
    return SDV_ERR_INVALID_ARG;
  if (!r->row_offsets || !r->adapter_ids) return SDV_ERR_INVALID_ARG;
  if (r->B > h->max_slots || r->T > h->max_rows) return SDV_ERR_CAPACITY;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != h->device) return SDV_ERR_INVALID_ARG;
  if (r->T == 0) return SDV_OK;  // no rows: their pointers may be null
  const int xb = r->x_format ? 4 : 2, yb = r->y_format ? 4 : 2;
  if (!r->x || !r->base || !r->out || !aligned(r->x, 16) || !aligned(r->base, 16) || !aligned(r->out, 16)) return SDV_ERR_INVALID_ARG;
  if (r->x_stride < h->cfg.k || r->base_stride < h->cfg.n || r->out_stride < h->cfg.n || (r->x_stride * xb) % 16 ||
      (r->base_stride * yb) % 16 || (r->out_stride * yb) % 16)
    return SDV_ERR_INVALID_ARG;
  if (r->out == r->base && r->out_stride != r->base_stride) return SDV_ERR_INVALID_ARG;
  // base is read ahead of what is written, x by other blocks than write
  const long long out_pitch = r->out_stride * yb, out_bytes = 1LL * h->cfg.n * yb;
  if ((r->out != r->base && rows_share(r->out, out_pitch, out_bytes, r->base, r->base_stride * yb, out_bytes, r->T)) ||
      rows_share(r->out, out_pitch, out_bytes, r->x, r->x_stride * xb, 1LL * h->cfg.k * xb, r->T))
    return SDV_ERR_INVALID_ARG;
  AdapterParams p;
  p.r = *r;
  p.k = h->cfg.k;
  p.n = h->cfg.n;
  p.rank = h->cfg.rank;
  p.count = h->cfg.count;
  p.a = static_cast<const __nv_bfloat16*>(h->cfg.a);
  p.b = static_cast<const __nv_bfloat16*>(h->cfg.b);
  p.scales = h->cfg.scales;
  p.status = status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int mt = (p.rank + 15) / 16;
  const cudaError_t e = mt <= 1 ? start<1>(p, h->sms, s) : mt <= 2 ? start<2>(p, h->sms, s) : mt <= 4 ? start<4>(p, h->sms, s) : start<8>(p, h->sms, s);
  return e == cudaSuccess ? SDV_OK : cuda_fail(e);
}
