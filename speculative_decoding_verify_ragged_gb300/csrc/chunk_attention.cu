// Attention of a ragged chunk over the paged cache, for few query rows per
// sequence (mma.sync): softmax(q k^T / sqrt(d)) v with a running maximum and sum.
//
// An item is 8 or 16 packed query rows -- the n_q / n_kv heads of consecutive
// tokens -- of one (sequence, key head) against its visible pages.  The items'
// pages are laid end to end and cut into equal runs, one per block, so a single
// long sequence and a batch of unlike ones load the GPU alike; an item cut
// between blocks is joined by the last of them to arrive, in block order, so
// equal inputs give equal bits.
//
// Within a block the four warps take pages in turn, straight from global memory
// to registers.  Scores and output are computed transposed (16 keys, or 16
// columns, by 8 rows), so that 8 rows fill the MMA.  The sum over d of a
// score may run in any order, so a lane takes 16 contiguous bytes of a key
// wherever the MMA wants its k index, and queries are laid out to match; the
// columns of the output are likewise assigned so that a lane's V loads are 16
// contiguous bytes of four keys.  No value is staged in shared memory.  e4m3 codes
// become fp16 exactly; a key's scale multiplies its scores, a value's its weight.
//
// Bound by the cache's bytes where there are enough of them (32 query and 8 key
// heads of 128): 64 sequences of 1000 to 9000 tokens, one row each, bf16 1.33 GB
// in 208 us (0.94 of the copy peak), e4m3 670 MB in 122 us (0.81; the conversions and
// three blocks per SM hold it there); 128 sequences of 2048 tokens, 4 rows each, bf16
// 182 us (0.88), e4m3 158 us (0.52: 237 registers leave two blocks per SM, a page on its way each warp).  Small batches are a chain of latencies: 1 sequence of 517
// tokens 9.1 us, of which the kernel's own 4.8.
#include "chunk.cuh"

namespace sdv {
namespace {

constexpr int CA_WARPS = 4;
constexpr int CA_THREADS = CA_WARPS * kWarp;
constexpr float kNoMax = -1e30f;  // the maximum before the first visible key
constexpr int kFewItems = 4;      // blocks per item from which the items are cut by themselves (2, 3, 4: 18 sequences 33.4, 33.5, 32.6 us)
constexpr int kMinPages = 4;      // pages a block takes at least: one per warp (4, 8, 16: 11.5, 11.8, 13.3 us for one sequence of 517)
// e4m3: a weight enters fp16 times its value's scale, 2^(s + e), and the bound m is one of s + e: the largest
// stands at 2^15, so weights keep fp16's half step of 2^-11 down to 2^-29 of the largest, whatever e is.  A page whose
// own largest lies more than 24 binades down moves the bound there (sum and output scale up; they are fp32),
// so that one key far above the rest takes nothing from the pages behind it.  A bound is moved down by 48 binades at
// most, and no more once the sum is past 2^50 (sums stay below 2^101, outputs below 2^117): what is lost
// then is below 2^-50 of the sum.
constexpr float kTopWeight = 15.f, kDeepest = 24.f, kSumMost = 0x1p50f, kDropMost = 48.f;

constexpr int part_floats(int D) { return kItemRows * (D + 2); }

template <int D, int FMT>
struct Frag {
  static constexpr bool kCodes = FMT == SDV_CACHE_E4M3;
  static constexpr int KSTEPS = D / 16;
  static constexpr int ROW_BYTES = kCodes ? D : 2 * D;
  static constexpr int KCH = ROW_BYTES / 64;                    // 16-byte chunks of a key row per lane (4 lanes a row)
  static constexpr int VW = ROW_BYTES / 8 / 4;                  // words of a value row per lane (8 lanes a row)
  static constexpr int MT = D / 16;                             // 16-row tiles of the transposed output
  uint32_t k[2][KCH * 4];  // keys g and g + 8
  uint32_t v[4][VW];       // keys 2t, 2t + 1, 2t + 8, 2t + 9
  uint32_t sc[2];          // e4m3: scale bytes of keys g and g + 8: K's low byte, V's above
};

// The output column of (lane group g of 8, tile j), its neighbour following in
// the tile's rows g + 8: the V words of a lane are contiguous.
template <int D, int FMT>
__device__ __forceinline__ int out_col(int g, int j) {
  if constexpr (FMT == SDV_CACHE_E4M3) return g * (D / 8) + 2 * j;
  return ((j >> 2) * 8 + g) * 8 + 2 * (j & 3);
}

// Transpose of an 8 x 8 matrix of 16-bit values, one row of pairs per four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int D, int FMT>
__device__ __forceinline__ void load_page(Frag<D, FMT>& f, const ChunkParams& c, int page, int h, int g, int t) {
  using F = Frag<D, FMT>;
  const long long head = ((long long)page * c.n_kv + h) * 2 * kPage;
  const uint8_t* kp = c.pool + head * F::ROW_BYTES;
  const uint8_t* vp = kp + kPage * F::ROW_BYTES;
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int i = 0; i < F::KCH; ++i) {
      const uint4 w = load16(reinterpret_cast<const uint4*>(kp + (g + 8 * r) * F::ROW_BYTES + (i * 4 + t) * 16));
      f.k[r][4 * i] = w.x, f.k[r][4 * i + 1] = w.y, f.k[r][4 * i + 2] = w.z, f.k[r][4 * i + 3] = w.w;
    }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint8_t* row = vp + (2 * t + (r & 1) + 8 * (r >> 1)) * F::ROW_BYTES;
    if constexpr (F::VW == 2) {
      const uint2 w = load8(reinterpret_cast<const uint2*>(row + g * 8));
      f.v[r][0] = w.x, f.v[r][1] = w.y;
    } else {
#pragma unroll
      for (int i = 0; i < F::VW / 4; ++i) {
        const uint4 w = load16(reinterpret_cast<const uint4*>(row + (i * 8 + g) * 16));
        f.v[r][4 * i] = w.x, f.v[r][4 * i + 1] = w.y, f.v[r][4 * i + 2] = w.z, f.v[r][4 * i + 3] = w.w;
      }
    }
  }
  if constexpr (F::kCodes) {
    const uint8_t* s = c.scales + head;
#pragma unroll
    for (int r = 0; r < 2; ++r) f.sc[r] = static_cast<uint32_t>(s[g + 8 * r]) | static_cast<uint32_t>(s[kPage + g + 8 * r]) << 8;
  }
}

// What the end of an item needs: out of the registers of the pages' loop.
struct ItemEnd {
  int off, head, row0, rows, first, last, units;
};
struct Plan {
  long long per, run;  // pages of a piece; units of a block
  bool pieces;
};

// Blocks per SM: what the registers allow (held: two pages, the output, the
// queries).  e4m3, 8 rows: 2, 3 and 4 blocks 149, 122 and 125 us for 64 sequences;
// bf16, 8 rows: 2 and 3 blocks 209 and 228 us; 16 rows: 1 and 2 blocks 270 and 181 us.
// Heads of 64, bf16, 8 rows: 3, 4 and 5 blocks 124, 118 and 140 us; 16 rows: 2, 3 and 4 135, 110 and 123; e4m3, 8 rows:
// 87, 73 and 67; 16 rows: 172, 123 and 110 (one more of each would serve it; 5 want a larger workspace).
template <int D, int FMT, int NT>
constexpr int per_sm() {
  return D == 64 ? (NT == 1 ? 4 : 3) : FMT == SDV_CACHE_E4M3 ? (NT == 1 ? 3 : 2) : 2;
}

template <int D, int FMT, int NT>
__global__ void __launch_bounds__(CA_THREADS, per_sm<D, FMT, NT>()) chunk_attn_kernel(const ChunkAttnParams p) {
  using F = Frag<D, FMT>;
  constexpr int ROWS = 8 * NT;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  float* s_o = reinterpret_cast<float*>(smem_raw);                     // [warps][16][D]
  float* s_ml = s_o + CA_WARPS * ROWS * D;                             // [warps][2][16]
  long long* s_base = reinterpret_cast<long long*>(s_ml + CA_WARPS * 2 * ROWS);  // [B + 1] first unit of each sequence
  int* s_off = reinterpret_cast<int*>(s_base + p.c.B + 1);
  int* s_len = s_off + p.c.B + 1;
  __shared__ long long s_scan[CA_WARPS], s_items[CA_WARPS];
  __shared__ Plan s_plan;
  __shared__ ItemEnd s_end;
  __shared__ int s_last;

  griddep_launch_dependents();
  griddep_wait();
  const int B = p.c.B, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int group = p.c.n_q / p.c.n_kv, window = p.c.window;
  // a call that has failed already writes nothing, but still takes its part in
  // the counting below, so that the counters end at zero whichever block saw it
  bool dead;
  if (!load_chunk(p.c, s_off, s_len, dead)) return;

  // pages of each of a sequence's items (those that any of its rows sees), first page
  auto seq_of = [&](int b) {
    SeqRows s = seq_rows(s_off, s_len, b);
    if (s.n * group > p.small_rows) s.n = 0;  // the tcgen05 kernel's
    return s;
  };
  auto seq_pages = [&](const SeqRows& s, int& lo) {
    lo = window > 0 ? max(0, s.pos0 - window + 1) / kPage : 0;
    return s.n > 0 ? max(1, (s.len + kPage - 1) / kPage - lo) : 0;
  };
  auto seq_tiles = [&](const SeqRows& s) { return (int)(((long long)s.n * group + ROWS - 1) / ROWS); };
  // Units: pages, cut into equal runs over the blocks; a block that holds the end of
  // one item and the beginning of another pays both items' latencies in turn.
  // With few items they are cut by themselves instead, into pieces of `per_cta`
  // pages, one a block (the sum over items of ceil(pages / per) is at most the
  // blocks then), and a unit is a piece: 1 sequence of 517 tokens 11.4 -> 9.1 us.
  const int per_thread = (B + CA_THREADS - 1) / CA_THREADS, b_lo = min(B, tid * per_thread), b_hi = min(B, b_lo + per_thread);
  long long pages = 0, items = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const SeqRows s = seq_of(b);
    int lo;
    const long long n = (long long)seq_tiles(s) * p.c.n_kv;
    pages += seq_pages(s, lo) * n;
    items += n;
  }
  pages = warp_sum_u64(pages);
  items = warp_sum_u64(items);
  if (lane == 0) {
    s_scan[warp] = pages;
    s_items[warp] = items;
  }
  __syncthreads();
  pages = items = 0;
#pragma unroll
  for (int w = 0; w < CA_WARPS; ++w) {
    pages += s_scan[w];
    items += s_items[w];
  }
  const bool pieces = items * kFewItems <= gridDim.x;
  const long long blocks = pieces ? gridDim.x - items : gridDim.x;
  const long long per_cta = max((long long)kMinPages, (pages + blocks - 1) / blocks);
  {
    long long sum = 0;
    for (int b = b_lo; b < b_hi; ++b) {
      const SeqRows s = seq_of(b);
      int lo;
      const int u = seq_pages(s, lo);
      s_base[b] = sum;
      sum += (pieces ? (u + per_cta - 1) / per_cta : u) * seq_tiles(s) * p.c.n_kv;
    }
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    __syncthreads();  // the totals have been read
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    long long add = inc - sum;
    for (int w = 0; w < warp; ++w) add += s_scan[w];
    for (int b = b_lo; b < b_hi; ++b) s_base[b] += add;
    if (tid == CA_THREADS - 1) s_base[B] = add + sum;
    if (tid == 0) s_plan = Plan{per_cta, pieces ? 1 : per_cta, pieces};
    __syncthreads();
  }

  for (long long u = blockIdx.x * s_plan.run;;) {
    // (the plan is read anew for each item: held across the pages it spilled; the bf16 kernel of 16 rows still spills 36 bytes)
    const bool pieces = s_plan.pieces;
    const long long units = s_base[B], per_cta = s_plan.per, run = s_plan.run, u_end = min(units, (blockIdx.x + 1) * run);
    if (u >= u_end) break;
    int b = 0;
    {
      int lo = 0, hi = B - 1;  // the last b with s_base[b] <= u (empty sequences share their successor's base)
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_base[mid] <= u) lo = mid;
        else hi = mid - 1;
      }
      b = lo;
    }
    const SeqRows sq = seq_of(b);
    int lo_page;
    const int n_pages = seq_pages(sq, lo_page), tiles = seq_tiles(sq);
    // within the sequence: key head, then tile, then page (in 32 bits where they fit, as nearly always)
    const long long in_seq = u - s_base[b];
    const int item_units = pieces ? static_cast<int>((n_pages + per_cta - 1) / per_cta) : n_pages;
    const long long item = units < 0x7FFFFFFF ? static_cast<unsigned>(in_seq) / static_cast<unsigned>(item_units) : in_seq / item_units;
    const int at_unit = static_cast<int>(in_seq - item * item_units), page0 = pieces ? static_cast<int>(at_unit * per_cta) : at_unit;
    const int h = units < 0x7FFFFFFF ? static_cast<unsigned>(item) / static_cast<unsigned>(tiles) : static_cast<int>(item / tiles);
    const int row0 = static_cast<int>(item - (long long)h * tiles) * ROWS;
    const int n_here = static_cast<int>(min(pieces ? per_cta : u_end - u, (long long)(n_pages - page0)));
    const int n_rows = static_cast<int>(min((long long)ROWS, (long long)sq.n * group - row0));
    if (tid == 0) {
      // with the blocks that hold pages of this item
      const long long u0 = s_base[b] + item * item_units, u1 = u0 + item_units - 1;
      const bool small = units < 0x7FFFFFFF;
      s_end = ItemEnd{sq.off, h * group, row0, n_rows,
                      small ? static_cast<int>(static_cast<unsigned>(u0) / static_cast<unsigned>(run)) : static_cast<int>(u0 / run),
                      small ? static_cast<int>(static_cast<unsigned>(u1) / static_cast<unsigned>(run)) : static_cast<int>(u1 / run),
                      pieces ? 1 : n_here};
    }
    const int pmin = sq.pos0 + row0 / group, pmax = sq.pos0 + (row0 + n_rows - 1) / group;
    // pages of this run that a row of the item sees
    const int first = max(lo_page + page0, window > 0 ? max(0, pmin - window + 1) / kPage : 0);
    const int last = min(lo_page + page0 + n_here, pmax < 0 ? 0 : pmax / kPage + 1);

    const int pg0 = first + warp;
    const int mine = dead || pg0 >= last ? 0 : (last - pg0 + CA_WARPS - 1) / CA_WARPS;  // this warp's pages
    int ids = 0;
    Frag<D, FMT> nxt, cur;
    auto page_id = [&](int i) {  // the warp's i-th page; the lanes fetch 32 ids at a time
      if ((i & 31) == 0) {
        ids = -1;
        if (i + lane < mine) {
          ids = p.c.page_table[(long long)b * p.c.max_pages + pg0 + (i + lane) * CA_WARPS];
          if (ids < 0 || ids >= p.c.pool_pages) {
            set_status(p.c.status, SDV_ERR_PAGE_RANGE);
            ids = 0;  // some page of the pool: the call's outputs hold nothing meaningful
          }
        }
      }
      return __shfl_sync(0xffffffffu, ids, i & 31);
    };
    if (mine > 0) load_page(nxt, p.c, page_id(0), h, g, t);

    // queries: row g of each 8, laid out like the keys; the rows whose scores
    // this lane holds are 2 t and 2 t + 1 of each 8
    uint32_t qf[NT][F::KSTEPS][2];
    int pos[NT][2];
    float cz[NT][2];
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      const int row = row0 + g + 8 * r;
      const bool in = g + 8 * r < n_rows;
      const __nv_bfloat16* src =
          p.q + (in ? (long long)(sq.off + row / group) * p.q_stride + (long long)(h * group + row % group) * D : 0);
      float scale = p.scale_log2;
      if constexpr (F::kCodes) {
        // fp16 with the row's largest magnitude in [1/2, 1): what falls below
        // 2^-25 of it is lost, far under the products' own rounding
        uint2 w[F::KSTEPS];
        float a = 0.f;
#pragma unroll
        for (int ks = 0; ks < F::KSTEPS; ++ks) {
          w[ks] = in ? *reinterpret_cast<const uint2*>(src + (ks >> 2) * 64 + t * 16 + (ks & 3) * 4) : make_uint2(0u, 0u);
          a = fmaxf(a, fmaxf(fmaxf(fabsf(__uint_as_float(w[ks].x << 16)), fabsf(__uint_as_float(w[ks].x & 0xFFFF0000u))),
                             fmaxf(fabsf(__uint_as_float(w[ks].y << 16)), fabsf(__uint_as_float(w[ks].y & 0xFFFF0000u)))));
        }
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
        const int e = min(max(static_cast<int>(__float_as_uint(a) >> 23) - 126, -100), 100);
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        scale *= __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
        for (int ks = 0; ks < F::KSTEPS; ++ks) {
          const __half2 x = __floats2half2_rn(__uint_as_float(w[ks].x << 16) * inv, __uint_as_float(w[ks].x & 0xFFFF0000u) * inv);
          const __half2 y = __floats2half2_rn(__uint_as_float(w[ks].y << 16) * inv, __uint_as_float(w[ks].y & 0xFFFF0000u) * inv);
          qf[r][ks][0] = *reinterpret_cast<const uint32_t*>(&x);
          qf[r][ks][1] = *reinterpret_cast<const uint32_t*>(&y);
        }
      } else {
#pragma unroll
        for (int i = 0; i < F::KCH; ++i) {
          const uint4 w = in ? *reinterpret_cast<const uint4*>(src + (i * 4 + t) * 8) : make_uint4(0u, 0u, 0u, 0u);
          qf[r][2 * i][0] = w.x, qf[r][2 * i][1] = w.y, qf[r][2 * i + 1][0] = w.z, qf[r][2 * i + 1][1] = w.w;
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int rr = 2 * t + x + 8 * r;
        pos[r][x] = rr < n_rows ? sq.pos0 + (row0 + rr) / group : -1;
        cz[r][x] = __shfl_sync(0xffffffffu, scale, (2 * t + x) * 4);
      }
    }

    // the output transposed: o[r][j] holds columns out_col(g, j) and the next of rows 2 t and 2 t + 1
    float o[NT][F::MT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int r = 0; r < NT; ++r) {
#pragma unroll
      for (int j = 0; j < F::MT; ++j) o[r][j][0] = o[r][j][1] = o[r][j][2] = o[r][j][3] = 0.f;
      m[r][0] = m[r][1] = kNoMax;
      l[r][0] = l[r][1] = 0.f;
    }

    for (int i = 0; i < mine; ++i) {
      cur = nxt;
      if (i + 1 < mine) load_page(nxt, p.c, page_id(i + 1), h, g, t);
      const int key0 = (pg0 + i * CA_WARPS) * kPage;
      // scores transposed: s[r][2 y + x] is key key0 + g + 8 y, row 2 t + x of 8-row tile r
      float s[NT][4];
#pragma unroll
      for (int r = 0; r < NT; ++r) s[r][0] = s[r][1] = s[r][2] = s[r][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < F::KSTEPS; ++ks) {
        uint32_t a[4];
        if constexpr (F::kCodes) {
          a[0] = e4m3x2_to_f16x2(cur.k[0][ks] & 0xFFFFu), a[1] = e4m3x2_to_f16x2(cur.k[1][ks] & 0xFFFFu);
          a[2] = e4m3x2_to_f16x2(cur.k[0][ks] >> 16), a[3] = e4m3x2_to_f16x2(cur.k[1][ks] >> 16);
#pragma unroll
          for (int r = 0; r < NT; ++r) mma_f16(s[r], a, qf[r][ks][0], qf[r][ks][1]);
        } else {
          a[0] = cur.k[0][2 * ks], a[1] = cur.k[1][2 * ks], a[2] = cur.k[0][2 * ks + 1], a[3] = cur.k[1][2 * ks + 1];
#pragma unroll
          for (int r = 0; r < NT; ++r) mma_bf16(s[r], a, qf[r][ks][0], qf[r][ks][1]);
        }
      }
      // base-2 logits; e4m3: plus the exponent e of the value's scale, and 2^-e for the sum
      float un[2] = {1.f, 1.f};
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        if constexpr (F::kCodes) {
          const uint32_t vb = cur.sc[y] >> 8;
          const float ksc = scale_value(cur.sc[y]), ve = __uint_as_float(0x4B000000u | vb) - 8388735.f;  // 2^23 + byte, less 2^23 + 127
          un[y] = scale_value(254u - vb);
#pragma unroll
          for (int r = 0; r < NT; ++r) {
            s[r][2 * y] = fmaf(s[r][2 * y], cz[r][0] * ksc, ve);
            s[r][2 * y + 1] = fmaf(s[r][2 * y + 1], cz[r][1] * ksc, ve);
          }
        } else {
#pragma unroll
          for (int r = 0; r < NT; ++r) {
            s[r][2 * y] *= cz[r][0];
            s[r][2 * y + 1] *= cz[r][1];
          }
        }
      }
      const bool full = key0 + kPage - 1 <= pmin && (window <= 0 || key0 > pmax - window);
      if (!full) {
        // keys that no row of the item sees may hold anything: their weight is
        // 0 and their values are taken as 0
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int key = key0 + g + 8 * y;
          if (key > pmax || (window > 0 && key <= pmin - window)) un[y] = 0.f;
#pragma unroll
          for (int r = 0; r < NT; ++r)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (key > pos[r][x] || (window > 0 && key <= pos[r][x] - window)) s[r][2 * y + x] = -INFINITY;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int key = key0 + 2 * t + (r & 1) + 8 * (r >> 1);
          if (key > pmax || (window > 0 && key <= pmin - window))
#pragma unroll
            for (int w = 0; w < F::VW; ++w) cur.v[r][w] = 0u;
        }
      }
      bool move = false;
#pragma unroll
      for (int r = 0; r < NT; ++r)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float top = fmaxf(s[r][x], s[r][2 + x]);
          if constexpr (F::kCodes) {
            const float a = top - m[r][x];
            move |= a > kTopWeight || (a < kTopWeight - kDeepest && top > kNoMax);
          } else {
            move |= top > m[r][x];
          }
        }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int r = 0; r < NT; ++r)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float top = fmaxf(s[r][x], s[r][2 + x]);
            if constexpr (!F::kCodes) top = fmaxf(top, m[r][x]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            if constexpr (F::kCodes) {
              // the page's largest decides; every lane of the row comes to the same bound
              float most = l[r][x];
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
              const bool seen = top > kNoMax;
              top -= kTopWeight;
              const float old = m[r][x];
              if (!(top > old)) top = seen && top < old - kDeepest && most <= kSumMost ? fmaxf(top, old - kDropMost) : old;
            }
            const float f = fast_ex2(m[r][x] - top);
            m[r][x] = top;
            l[r][x] *= f;
#pragma unroll
            for (int j = 0; j < F::MT; ++j) o[r][j][x] *= f, o[r][j][2 + x] *= f;
          }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int r = 0; r < NT; ++r)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float a = fast_ex2(s[r][2 * y] - m[r][0]), b2 = fast_ex2(s[r][2 * y + 1] - m[r][1]);
          uint32_t w;
          if constexpr (F::kCodes) {
            l[r][0] = fmaf(a, un[y], l[r][0]);
            l[r][1] = fmaf(b2, un[y], l[r][1]);
            const __half2 hw = __floats2half2_rn(a, b2);
            w = *reinterpret_cast<const uint32_t*>(&hw);
          } else {
            l[r][0] += a;
            l[r][1] += b2;
            w = pack_bf16x2(a, b2);
          }
          pb[r][y] = transpose8(w);
        }
#pragma unroll
      for (int w = 0; w < F::VW; ++w) {
        uint32_t a[4];
        if constexpr (F::kCodes) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t lo = __byte_perm(cur.v[0][w], cur.v[1][w], y ? 0x7362 : 0x5140);
            const uint32_t hi = __byte_perm(cur.v[2][w], cur.v[3][w], y ? 0x7362 : 0x5140);
            a[0] = e4m3x2_to_f16x2(lo & 0xFFFFu), a[1] = e4m3x2_to_f16x2(lo >> 16);
            a[2] = e4m3x2_to_f16x2(hi & 0xFFFFu), a[3] = e4m3x2_to_f16x2(hi >> 16);
#pragma unroll
            for (int r = 0; r < NT; ++r) mma_f16(o[r][2 * w + y], a, pb[r][0], pb[r][1]);
          }
        } else {
          a[0] = __byte_perm(cur.v[0][w], cur.v[1][w], 0x5410), a[1] = __byte_perm(cur.v[0][w], cur.v[1][w], 0x7632);
          a[2] = __byte_perm(cur.v[2][w], cur.v[3][w], 0x5410), a[3] = __byte_perm(cur.v[2][w], cur.v[3][w], 0x7632);
#pragma unroll
          for (int r = 0; r < NT; ++r) mma_bf16(o[r][w], a, pb[r][0], pb[r][1]);
        }
      }
    }

    // the warps' parts into shared memory, then joined
#pragma unroll
    for (int r = 0; r < NT; ++r)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int row = 8 * r + 2 * t + x;
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[r][x] += __shfl_xor_sync(0xffffffffu, l[r][x], d);
        if (g == 0) {
          s_ml[warp * 2 * ROWS + row] = m[r][x];
          s_ml[warp * 2 * ROWS + ROWS + row] = l[r][x];
        }
#pragma unroll
        for (int j = 0; j < F::MT; ++j)
          *reinterpret_cast<float2*>(s_o + (warp * ROWS + row) * D + out_col<D, FMT>(g, j)) =
              make_float2(o[r][j][x], o[r][j][2 + x]);
      }
    __syncthreads();
    constexpr int TPR = CA_THREADS / ROWS, PER = D / TPR;  // threads a row, columns a thread
    const int row = tid / TPR, c0 = (tid % TPR) * PER;
    float acc[PER], M = kNoMax, L = 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j) acc[j] = 0.f;
#pragma unroll
    for (int w = 0; w < CA_WARPS; ++w) M = fmaxf(M, s_ml[w * 2 * ROWS + row]);
#pragma unroll
    for (int w = 0; w < CA_WARPS; ++w) {
      const float a = fast_ex2(s_ml[w * 2 * ROWS + row] - M);
      L += a * s_ml[w * 2 * ROWS + ROWS + row];
#pragma unroll
      for (int j = 0; j < PER; ++j) acc[j] += a * s_o[(w * ROWS + row) * D + c0 + j];
    }
    const ItemEnd e = s_end;
    const int c_first = e.first, c_last = e.last;
    bool write = row < e.rows && !dead;
    if (c_first != c_last) {
      // a block has at most two cut items: one begun before its run (slot 0)
      // and one that goes on behind it (slot 1)
      constexpr int PF = part_floats(D);
      float* mine_part = p.part + (2LL * blockIdx.x + (c_first == (int)blockIdx.x)) * PF;
#pragma unroll
      for (int j = 0; j < PER; j += 4)
        *reinterpret_cast<float4*>(mine_part + row * D + c0 + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
      if (tid % TPR == 0) {
        mine_part[kItemRows * D + row] = M;
        mine_part[kItemRows * (D + 1) + row] = L;
      }
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        s_last = atomicAdd(p.counters + c_first, 1) == c_last - c_first;
        if (s_last) p.counters[c_first] = 0;
        __threadfence();
      }
      __syncthreads();
      write = write && s_last;
      if (s_last) {
        M = kNoMax;
#pragma unroll 8
        for (int cta = c_first; cta <= c_last; ++cta)
          M = fmaxf(M, __ldcg(p.part + (2LL * cta + (cta == c_first)) * PF + kItemRows * D + row));
        L = 0.f;
#pragma unroll
        for (int j = 0; j < PER; ++j) acc[j] = 0.f;
#pragma unroll 4
        for (int cta = c_first; cta <= c_last; ++cta) {
          const float* src = p.part + (2LL * cta + (cta == c_first)) * PF;
          const float a = fast_ex2(__ldcg(src + kItemRows * D + row) - M);
          L += a * __ldcg(src + kItemRows * (D + 1) + row);
#pragma unroll
          for (int j = 0; j < PER; j += 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(src + row * D + c0 + j));
            acc[j] += a * x.x, acc[j + 1] += a * x.y, acc[j + 2] += a * x.z, acc[j + 3] += a * x.w;
          }
        }
      }
    }
    if (write) {
      const float inv = L == 0.f ? 0.f : 1.f / L;  // a row that sees nothing gives 0
      const int rr = e.row0 + row;
      __nv_bfloat16* dst = p.out + (long long)(e.off + rr / group) * p.out_stride + (long long)(e.head + rr % group) * D + c0;
#pragma unroll
      for (int j = 0; j < PER; j += 4)
        *reinterpret_cast<uint2*>(dst + j) =
            make_uint2(pack_bf16x2(acc[j] * inv, acc[j + 1] * inv), pack_bf16x2(acc[j + 2] * inv, acc[j + 3] * inv));
    }
    __syncthreads();
    u += e.units;
  }
}

size_t smem_bytes(int D, int rows, int B) {
  return (CA_WARPS * rows * D + CA_WARPS * 2 * rows) * sizeof(float) + (B + 1) * sizeof(long long) + (2 * B + 1) * sizeof(int);
}

template <int D, int FMT, int NT>
cudaError_t launch_one(const ChunkAttnParams& p, int sms, cudaStream_t stream) {
  return launch_pdl(chunk_attn_kernel<D, FMT, NT>, dim3(sms * per_sm<D, FMT, NT>()), dim3(CA_THREADS), smem_bytes(D, 8 * NT, p.c.B), stream, p);
}

template <int D, int FMT>
cudaError_t setup_one() {
  const cudaError_t e = cudaFuncSetAttribute(chunk_attn_kernel<D, FMT, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem_bytes(D, 8, kMaxChunkSlots)));
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(chunk_attn_kernel<D, FMT, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(smem_bytes(D, 16, kMaxChunkSlots)));
}

}  // namespace

int chunk_attn_grid_max(int sms) { return 4 * sms; }
size_t chunk_attn_part_floats(int head_dim, int sms) { return static_cast<size_t>(2) * chunk_attn_grid_max(sms) * part_floats(head_dim); }

cudaError_t setup_chunk_attn(int head_dim, int cache_format) {
  if (head_dim == 64)
    return cache_format == SDV_CACHE_BF16 ? setup_one<64, SDV_CACHE_BF16>() : setup_one<64, SDV_CACHE_E4M3>();
  return cache_format == SDV_CACHE_BF16 ? setup_one<128, SDV_CACHE_BF16>() : setup_one<128, SDV_CACHE_E4M3>();
}

cudaError_t launch_chunk_attn(int head_dim, int cache_format, bool eight, const ChunkAttnParams& p, int sms, cudaStream_t stream) {
#define SDV_CHUNK(D, F) return eight ? launch_one<D, F, 1>(p, sms, stream) : launch_one<D, F, 2>(p, sms, stream)
  if (head_dim == 64) {
    if (cache_format == SDV_CACHE_BF16) SDV_CHUNK(64, SDV_CACHE_BF16);
    SDV_CHUNK(64, SDV_CACHE_E4M3);
  }
  if (cache_format == SDV_CACHE_BF16) SDV_CHUNK(128, SDV_CACHE_BF16);
  SDV_CHUNK(128, SDV_CACHE_E4M3);
#undef SDV_CHUNK
}

}  // namespace sdv
