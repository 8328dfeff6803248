// Sampling under temperature, top-k, top-p and min-p (include/sdv_sample.h).
//
// What stays of a row is always the beginning of it in the order (logit
// descending, index ascending), so a row's work is to find the last token that
// stays -- its logit and, among equals, its index -- and then the token that
// the uniform falls on.
//
// Weights.  Both answers hang on sums over the whole row next to a border, and a
// token more or less in a tail of 10^5 moves every border behind it: with fp32
// exponentials (2^-22) a row in some ten thousands would come out differently from its
// definition.  So w = exp((z - max) / T) is made as an integer in steps of 2^-42 and
// within 2^-34 of its value: t = (max - z) log2(e) / T is carried as an
// unevaluated sum of two floats, its multiple of 2^-10 looked up (2^-j/1024, a table
// of 1024 made from the series of exp) and the rest, below 2^-11, taken by a
// quadratic.  Below 2^-13 the special-function unit's 2^-22, for the same t, is within 2^-33 of the largest.  Sums of integers
// are exact and have no order: any split over threads, blocks and passes gives the same answer.
//
// What can stay is nearly always a few hundred tokens of 10^5, so a row is read once and what may stay is
// kept: a block samples the beginning of each warp's run (64 maxima of 128 or 256 neighbours; one of their lower order
// statistics has about 1 % of the row above it, whatever the row's distribution), and each warp keeps what reaches that in a
// list of its own, in the order of the row.  Where top-p needs the whole row's sum, the rest goes into it through the
// special-function unit, with a bound of its error; the answer counts if it is the same at both ends of that bound.  Where the lists
// do not hold the answer (a flat row, no setting at all, ends of the bound that differ) the same functions read the row
// again beside the lists, and every weight is exact.
//
// Those functions: count (top-k) or add up (top-p) what lies up to levels of t (32 over the lists, 6 over memory); the first level at which the bound
// is reached is usually passed by a few dozen tokens, which are gathered in the first block and ranked one against another by
// value and by index, and the row is done.  Of more, those between that level and the one before go into a
// histogram by t, the tokens of the bin that the bound falls into are ranked, and a last pass adds up what stays
// by warp; the warp that holds the drawn point walks its run of indices.  A bin of too many (tied logits) is cut by further
// histograms over the logits' bits until one value is left, of which the first few by index stay.
//
// A cluster of up to 8 blocks takes a row where rows are few; two blocks share an SM.
//
// Bound by the row's bytes where rows are many, by waits one after another (settings, first loads, the sample, meetings, the
// list) where they are few: 512 rows of 151936 fp32 values under top-p (311 MB) 99 us, 3.1 TB/s: while it reads, a
// block keeps pace with memory, but some 8 us of waits a block lie beside 25 us of reading, and 512 blocks are 1.7 of what
// runs at once; greedy 69 us, top-k 83, no setting (two readings, every weight) 224; one row 9 to 20 us.
#include <atomic>

#include <cooperative_groups.h>

#include "../../include/sdv_sample.h"
#include "common.cuh"
#include "internal.h"
#include "rows.h"

namespace cg = cooperative_groups;

namespace sdv {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / kWarp;
constexpr int kBins = 1024;       // of a histogram
constexpr int kList = 512;        // tokens that are ranked in the first block: each by a thread of its own at most
constexpr int kFew = 96;          // up to which that is done one against another, else by sorting
constexpr int kLevels = 32;       // of t at most
constexpr int kSteps = 1024;      // table entries a binade
constexpr int kFraction = 42;     // weights in steps of 2^-42, the largest 2^42
constexpr float kFine = 13.f;     // t from which the special-function unit serves in sums
constexpr float kLast = 19.f;     // t of the last level of a row that is not kept
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2eLow = 1.9259629911e-8f;  // log2(e) less its fp32 value
constexpr int kKeep = 512;        // tokens that a warp keeps
constexpr float kMasked = -3.3e38f;  // below it lie the types' lowest values: masks, not kept unless all is
constexpr int kBatch = 8;         // 4-byte words that a lane reads at a time, the next batch on its way meanwhile
constexpr int kGroup = 4;         // of which are looked at together
constexpr int kSamples = 2 * kBatch / kGroup * kWarps;  // maxima of a warp's groups
constexpr int kMaxCluster = 8;
using u64 = unsigned long long;
using u32 = unsigned int;

// 2^-(j / 1024) as an integer in steps of 2^-42 and as fp32.
struct __align__(16) PowerTable {
  u64 fixed[kSteps];
  float value[kSteps];
};
constexpr double power(double x) {  // 2^-x for x in [0, 1) by the series of exp
  const double y = -x * 0.693147180559945309417232121458;
  double sum = 1.0, term = 1.0;
  for (int n = 1; n < 24; ++n) {
    term *= y / n;
    sum += term;
  }
  return sum;
}
constexpr PowerTable make_table() {
  PowerTable t{};
  for (int j = 0; j < kSteps; ++j) {
    const double v = power(j / static_cast<double>(kSteps));
    t.fixed[j] = static_cast<u64>(v * 4398046511104.0 + 0.5);
    t.value[j] = static_cast<float>(v);
  }
  return t;
}
__device__ const PowerTable c_powers = make_table();

struct SampleParams {
  sdv_sample_rows r;
  int* status;
  int steps;      // words of a lane
  int keep_all;   // a warp's run fits its list
};

// A cut: what comes before (value, index) stays, that token included.
struct Cut {
  float z;
  int index;
};

// What a block shares; the first block's is read by the others.
struct __align__(16) Shared {
  u32 count[kBins], lo[kBins], hi[kBins];
  PowerTable powers;  // (copied in 16-byte pieces)
  float list_z[kList];
  int list_i[kList];
  u64 list_w[kList];
  u64 warp_sum[kWarps], part_sum[kWarps];
  u32 warp_count[kWarps];
  float sample[kSamples];
  float warp_max[kWarps], warp_rest[kWarps];
  // this block's tokens and their sum at each level (last: beyond), and the whole row's up to it (last: all)
  u32 level_count[kLevels], level_lo[kLevels + 1], level_hi[kLevels + 1];
  u32 all_count[kLevels];
  u64 all_mass[kLevels + 1];
  float block_max, block_rest, block_ref, threshold;
  int over;  // a list was too short
  u64 block_sum;
  int listed;
  // the first block's findings
  int bin;
  u32 bin_count, base_count;
  u64 base_mass, found_mass;
  Cut cut;
  int place, state, sure;
  u32 low, high;  // the candidates' order, of each block
  float c, c_low, floor_z;
  double below_top;  // T ln(min_p)
};

// fp32 bits in the order of their values; both zeros alike.
__device__ __forceinline__ u32 order_of(float z) {
  const u32 b = __float_as_uint(z + 0.f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(u32 o) { return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu)); }

// A row's weights.  What decides which weight, level or bin a token has is written in steps that round by themselves (no product is taken
// into the sum after it): lost() is what those roundings took off, and every pass has to give a token the same number.
struct Weights {
  float top, c, c_low;  // maximum, log2(e) / T in two parts
  const PowerTable* powers;

  __device__ __forceinline__ float t_of(float z) const { return z == top ? 0.f : __fmul_rn(__fsub_rn(top, z), c); }
  // what the three roundings on the way to t took off
  __device__ __forceinline__ float lost(float z, float t) const {
    const float d = __fsub_rn(top, z);
    const bool swap = fabsf(z) > fabsf(top);
    const float big = swap ? -z : top, small = swap ? top : -z;
    const float rest = __fsub_rn(small, __fsub_rn(d, big));
    return fmaf(rest, c, fmaf(d, c_low, fmaf(d, c, -t)));
  }
  __device__ __forceinline__ u64 fine(float z, float t) const {
    const float shifted = __fadd_rn(t, 12288.f);  // floats about 12288 come in steps of 2^-10
    const int i = __float_as_int(shifted) - __float_as_int(12288.f);
    const float x = __fadd_rn(__fsub_rn(t, __fsub_rn(shifted, 12288.f)), lost(z, t));  // within 2^-11
    const int j = i & (kSteps - 1);
    // 2^-x - 1 = -x ln 2 + (x ln 2)^2 / 2 - ..., the next term below 2^-37
    const float q = __fmul_rn(x, fmaf(x, 0.2402265069591007f, -kLn2));
    const int n = i >> 10;
    const u64 v = powers->fixed[j] + static_cast<long long>(__float2int_rn(__fmul_rn(powers->value[j], __fmul_rn(q, 4398046511104.f))));
    return n == 0 ? v : (v + (1ull << (n - 1))) >> n;
  }
  // 2^-t in fp32 by the special-function unit (2^-22), `behind` being what t lost
  static __device__ __forceinline__ float rough(float t, float behind, float scale) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(-t));
    return __fmul_rn(y, fmaf(behind, -kLn2 * scale, scale));
  }
  // t from 13 on, below 2^29.  Of what t lost, all but the difference's rounding is put right: that is t 2^-24 at most, with the rest 2^-33 of
  // the largest weight at t = 13 and less beyond (all of it put right: rows without a setting 225 -> 240 us)
  __device__ __forceinline__ u32 coarse(float z, float t) const {
    const float d = __fsub_rn(top, z);
    return __float2uint_rn(rough(t, fmaf(d, c_low, fmaf(d, c, -t)), 4398046511104.f));
  }
  __device__ __forceinline__ u64 operator()(float z) const {
    const float t = t_of(z);
    if (!(t < 44.f)) return 0;  // below half a step; -inf
    if (t < kFine) return z == top ? 1ull << kFraction : fine(z, t);
    return coarse(z, t);
  }
  // w / 2^42 in fp32, also where the steps of 2^-42 are too coarse for it
  __device__ __forceinline__ float share(float z) const {
    const float t = t_of(z);
    if (z == top) return 1.f;
    if (t < kFine) return static_cast<float>(fine(z, t)) * 0x1p-42f;
    return t < 126.f ? rough(t, lost(z, t), 1.f) : 0.f;  // (at t = 126 the difference alone would be 2^-17.6 of it)
  }
};

template <typename T>
struct Word;
template <>
struct Word<float> {
  static constexpr int N = 1;
  __device__ static void unpack(u32 w, float (&z)[1]) { z[0] = __uint_as_float(w); }
  __device__ static u32 none() { return 0xFF800000u; }
};
template <>
struct Word<__nv_bfloat16> {
  static constexpr int N = 2;
  __device__ static void unpack(u32 w, float (&z)[2]) { z[0] = __uint_as_float(w << 16), z[1] = __uint_as_float(w & 0xFFFF0000u); }
  __device__ static u32 none() { return 0xFF80FF80u; }
};

// A run of a row in memory, in words of 4 bytes: a warp reads 32 neighbouring words at a time, so that its lanes and its loads are
// in the row's order.  Word v holds elements v * N - shift ..; those outside [0, V) read as -inf.
template <typename T>
struct Slice {
  static constexpr int N = Word<T>::N;
  const T* row;
  int shift, V, first, last;  // words [first, last)
  int lane;

  __device__ __forceinline__ u32 load(int v) const {
    if (v >= last) return Word<T>::none();
    const int i = v * N - shift;
    if (N == 1 || (i >= 0 && i + N <= V)) {
      u32 w;
      asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(w) : "l"(row + i));
      return w;
    }
    u32 w = 0;  // (16-bit values, one of them outside)
    for (int j = 0; j < N; ++j)
      w |= (i + j >= 0 && i + j < V ? static_cast<u32>(reinterpret_cast<const unsigned short*>(row)[i + j]) : 0xFF80u) << (16 * j);
    return w;
  }
  // f(index, value) of every element, and of some past the run's end with -inf
  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {
    constexpr int AHEAD = 8;
    for (int v1 = first; v1 < last; v1 += 32 * AHEAD) {
      const int v0 = v1 + lane;
      u32 w[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) w[u] = load(v0 + 32 * u);
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        float z[N];
        Word<T>::unpack(w[u], z);
#pragma unroll
        for (int j = 0; j < N; ++j) f((v0 + 32 * u) * N - shift + j, z[j]);
      }
    }
  }
  // the run in rounds, a lane's N elements of round c in the order of the row
  __device__ __forceinline__ int rounds() const { return (last - first + 31) / 32; }
  __device__ __forceinline__ void round(int c, float (&z)[N], int (&i)[N]) const {
    const int v = first + 32 * c + lane;
    Word<T>::unpack(load(v), z);
#pragma unroll
    for (int j = 0; j < N; ++j) i[j] = v * N - shift + j;
  }
};

// What a warp kept of its run, in the order of the row.
struct Kept {
  static constexpr int N = 1;
  static constexpr bool LONG = false;
  static constexpr int LEVELS = 32;  // counted in shared memory
  static constexpr float SPAN = 80.f;  // of the levels, in the first one's width
  const float2* list;  // (value, index's bits)
  int n, lane;

  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {
    for (int e = lane; e < n; e += 32) {
      const float2 x = list[e];
      f(__float_as_int(x.y), x.x);
    }
  }
  template <typename P, typename F>
  __device__ __forceinline__ void each_of(P&& wanted, F&& f) const {
    each([&](int i, float z) {
      if (wanted(i, z)) f(i, z);
    });
  }
  __device__ __forceinline__ int rounds() const { return (n + 31) / 32; }
  __device__ __forceinline__ void round(int c, float (&z)[1], int (&i)[1]) const {
    const int e = 32 * c + lane;
    const float2 x = e < n ? list[e] : make_float2(-INFINITY, 0.f);
    z[0] = x.x, i[0] = __float_as_int(x.y);
  }
};

// A warp's whole run: what it kept from its list, where weights are dear, and the rest from memory.
template <typename T>
struct Both {
  static constexpr bool LONG = true;
  static constexpr int LEVELS = 6;  // counted in registers
  static constexpr float SPAN = 6.f;
  Slice<T> slice;
  Kept kept;
  float threshold;  // of the list; NaN if there is none
  int per_warp, words, first_run;  // words of a run and of the row; the block's first run

  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {
    slice.each([&](int i, float z) {
      if (!(z >= threshold)) f(i, z);
    });
    kept.each(f);
  }
  // f of the wanted ones
  template <typename P, typename F>
  __device__ __forceinline__ void each_of(P&& wanted, F&& f) const {
    each([&](int i, float z) {
      if (wanted(i, z)) f(i, z);
    });
  }
  // part `k` of `parts` of warp `warp`'s run
  __device__ __forceinline__ Slice<T> part(int warp, int k, int parts) const {
    Slice<T> s = slice;
    const int first = min(words, (first_run + warp) * per_warp), last = min(words, first + per_warp);
    const int each = ((per_warp + parts * 32 - 1) / (parts * 32)) * 32;
    s.first = min(last, first + k * each);
    s.last = min(last, s.first + each);
    return s;
  }
};

// p * s for p in [0, 1] and s < 2^63, rounded up or down, exact (p = m 2^-e with m < 2^24).
__device__ __forceinline__ u64 product_of(float p, u64 s, bool up) {
  if (p <= 0.f) return 0;
  const u32 b = __float_as_uint(p);
  const u64 m = (b & 0x7FFFFFu) | ((b >> 23) ? 0x800000u : 0u);
  const int e = 150 - static_cast<int>(max(b >> 23, 1u));  // p = m 2^-e, e >= 23
  const u64 hi = __umul64hi(m, s), lo = m * s;             // below 2^87
  if (e >= 128) return up && (hi | lo) ? 1 : 0;
  u64 q, rest;
  if (e >= 64) {
    q = e == 64 ? hi : hi >> (e - 64);
    rest = lo | (e == 64 ? 0 : hi & ((1ull << (e - 64)) - 1));
  } else {
    q = (hi << (64 - e)) | (lo >> e);
    rest = lo & ((1ull << e) - 1);
  }
  return q + (up && rest ? 1 : 0);
}

// p[i] += w on a 64-bit sum in two words of shared memory
__device__ __forceinline__ void add_mass(u32* lo, u32* hi, u64 w) {
  const u32 l = static_cast<u32>(w), old = atomicAdd(lo, l);
  const u32 h = static_cast<u32>(w >> 32) + (old + l < old ? 1u : 0u);
  if (h) atomicAdd(hi, h);
}

// max of two, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// a warp's sum of values below 2^54, in two halves
__device__ __forceinline__ u64 warp_add(u64 v) {
  const u32 lo = __reduce_add_sync(0xFFFFFFFFu, static_cast<u32>(v) & 0x7FFFFFFu);
  const u32 hi = __reduce_add_sync(0xFFFFFFFFu, static_cast<u32>(v >> 27));
  return (static_cast<u64>(hi) << 27) + lo;
}

// The row's finder of cuts and places; every thread of every block of the cluster calls its functions.
template <typename Source>
struct Row {
  cg::cluster_group cluster;
  Shared& s;
  Shared* lead;  // the first block's
  Source run;
  Weights w;
  int rank, blocks;
  float inv;  // levels per t, of the first ones

  static constexpr int LEVELS = Source::LEVELS;

  // t in levels.  Of 32 the last 16 are four times as wide: a bound falls near the largest weights or far off.
  __device__ __forceinline__ float scaled(float t) const {
    const float x = __fmul_rn(t, inv);
    return Source::LONG || x < 16.f ? x : fmaf(x, 0.25f, 12.f);
  }
  // 0 .. LEVELS - 1, LEVELS beyond the last level (-inf too)
  __device__ __forceinline__ int level_at(float t) const {
    const float x = scaled(t);
    return x < static_cast<float>(LEVELS) ? static_cast<int>(x) : LEVELS;
  }

  __device__ __forceinline__ int tid() const { return threadIdx.x; }
  __device__ __forceinline__ bool first_thread() const { return rank == 0 && threadIdx.x == 0; }

  __device__ void clear_bins() {
    for (int i = tid(); i < kBins; i += kThreads) s.count[i] = s.lo[i] = s.hi[i] = 0;
  }
  __device__ void clear_levels() {
    if (tid() <= kLevels) {
      if (tid() < kLevels) s.level_count[tid()] = 0;
      s.level_lo[tid()] = s.level_hi[tid()] = 0;
    }
  }

  __device__ __forceinline__ void put(int bin, u64 weight) {
    atomicAdd(&s.count[bin], 1u);
    if (weight) add_mass(&s.lo[bin], &s.hi[bin], weight);
  }

  // The number of the row's tokens up to each level, and (mass) their sums and everything's, in
  // every block's all_* when it returns.  level_* were cleared before.
  template <bool MASS>
  __device__ void levels() {
    const int lane = tid() & 31;
    if constexpr (LEVELS == kLevels) {
      run.each([&](int, float z) {
        const int level = level_at(w.t_of(z));
        if (level < LEVELS) atomicAdd(&s.level_count[level], 1u);
        if (MASS) add_mass(&s.level_lo[level], &s.level_hi[level], w(z));
      });
    } else {
      u64 sum[MASS ? LEVELS + 1 : 1] = {};
      u64 many = 0;  // 10 bits each
      auto add = [&](int, float z) {
        const int level = level_at(w.t_of(z));
        if (level < LEVELS) many += 1ull << (10 * level);
        if (MASS) {
          const u64 x = w(z);
          if (level == LEVELS) {
            sum[MASS ? LEVELS : 0] += x;
          } else {
#pragma unroll
            for (int l = 0; l < (MASS ? LEVELS : 1); ++l)
              if (l == level) sum[l] += x;
          }
        }
      };
      if constexpr (MASS) run.each_of([&](int, float z) { return w.t_of(z) < 44.f; }, add);
      else run.each(add);
#pragma unroll
      for (int l = 0; l <= LEVELS; ++l) {
        const u32 count = l < LEVELS ? __reduce_add_sync(0xFFFFFFFFu, static_cast<u32>(many >> (10 * l)) & 1023u) : 0;
        if (lane == 0 && count) atomicAdd(&s.level_count[l], count);
        if (MASS) {
          const u64 mass = warp_add(sum[MASS ? l : 0]);
          if (lane == 0 && mass) add_mass(&s.level_lo[l], &s.level_hi[l], mass);
        }
      }
    }
    cluster.sync();
    // each block adds all blocks' up
    if (tid() < kWarp) {
      // (every block's words asked for before the first is used: each is a trip through the cluster)
      u32 c8[kMaxCluster], lo8[kMaxCluster], hi8[kMaxCluster];
#pragma unroll
      for (int b = 0; b < kMaxCluster; ++b) {
        const Shared* o = cluster.map_shared_rank(&s, b < blocks ? b : 0);
        const bool there = b < blocks && lane < LEVELS;
        c8[b] = there ? o->level_count[lane] : 0;
        lo8[b] = there ? o->level_lo[lane] : 0;
        hi8[b] = there ? o->level_hi[lane] : 0;
      }
      const Shared* mine = cluster.map_shared_rank(&s, lane < blocks ? lane : 0);
      const u64 beyond = warp_sum_u64(lane < blocks ? (static_cast<u64>(mine->level_hi[LEVELS]) << 32) + mine->level_lo[LEVELS] : 0);
      u32 c = 0;
      u64 m = 0;
#pragma unroll
      for (int b = 0; b < kMaxCluster; ++b) c += c8[b], m += (static_cast<u64>(hi8[b]) << 32) + lo8[b];
#pragma unroll
      for (int o = 1; o < LEVELS; o <<= 1) {
        const u32 y = __shfl_up_sync(0xFFFFFFFFu, c, o);
        const u64 x = __shfl_up_sync(0xFFFFFFFFu, m, o);
        if (lane >= o) c += y, m += x;
      }
      if (lane < LEVELS) s.all_count[lane] = c, s.all_mass[lane] = m;
      if (lane == LEVELS - 1) s.all_mass[LEVELS] = m + beyond;
    }
    __syncthreads();
  }
  // the first level at which the bound is reached, LEVELS if none
  __device__ int level_of(bool by_count, u64 target) const {
    const int lane = tid() & 31;
    const bool there = lane < LEVELS && (by_count ? s.all_count[min(lane, LEVELS - 1)] : s.all_mass[min(lane, LEVELS - 1)]) >= target;
    const u32 votes = __ballot_sync(0xFFFFFFFFu, there);
    return votes ? __ffs(votes) - 1 : LEVELS;
  }

  // First block: the first bin (of all blocks' histograms together, bins in falling order of logits) at which the
  // count (by_count) or the sum, with what lies before it, reaches `target`; -1 if none does.  Its count and what
  // lies before it (base_*) go to the block's findings.
  __device__ void cross(bool by_count, u64 target, u32 base_count, u64 base_mass) {
    if (rank != 0) return;
    constexpr int PER = kBins / kThreads;
    u32 c[PER];
    u64 m[PER];
    u32 sum_c = 0;
    u64 sum_m = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = tid() * PER + j;
      u32 c8[kMaxCluster], lo8[kMaxCluster], hi8[kMaxCluster];
#pragma unroll
      for (int b = 0; b < kMaxCluster; ++b) {
        const Shared* o = cluster.map_shared_rank(&s, b < blocks ? b : 0);
        c8[b] = b < blocks ? o->count[i] : 0;
        lo8[b] = b < blocks ? o->lo[i] : 0;
        hi8[b] = b < blocks ? o->hi[i] : 0;
      }
      c[j] = 0, m[j] = 0;
#pragma unroll
      for (int b = 0; b < kMaxCluster; ++b) c[j] += c8[b], m[j] += (static_cast<u64>(hi8[b]) << 32) + lo8[b];
      sum_c += c[j], sum_m += m[j];
    }
    const int lane = tid() & 31, warp = tid() >> 5;
    u32 run_c = sum_c;
    u64 run_m = sum_m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u32 y = __shfl_up_sync(0xFFFFFFFFu, run_c, o);
      const u64 x = __shfl_up_sync(0xFFFFFFFFu, run_m, o);
      if (lane >= o) run_c += y, run_m += x;
    }
    if (lane == 31) s.warp_count[warp] = run_c, s.warp_sum[warp] = run_m;
    if (tid() == 0) s.bin = -1, s.listed = 0;
    __syncthreads();
    u32 before_c = base_count + run_c - sum_c;
    u64 before_m = base_mass + run_m - sum_m;
    for (int k = 0; k < warp; ++k) before_c += s.warp_count[k], before_m += s.warp_sum[k];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const u64 before = by_count ? before_c : before_m, own = by_count ? c[j] : m[j];
      if (before < target && target <= before + own) {
        s.bin = tid() * PER + j;
        s.bin_count = c[j];
        s.base_count = before_c, s.base_mass = before_m;
      }
      before_c += c[j], before_m += m[j];
    }
  }

  // The index of the token at which the running sum by index of the wanted ones' weight(z) first exceeds the target that
  // target_of(total) names; -1 if none.
  template <typename P, typename F, typename G>
  __device__ int locate(P&& wanted, F&& weight, G&& target_of) {
    const int lane = tid() & 31, warp = tid() >> 5;
    u64 mine = 0;
    run.each_of(wanted, [&](int, float z) { mine += weight(z); });
    auto f = [&](float z, int i) -> u64 { return wanted(i, z) ? weight(z) : 0; };
    mine = warp_sum_u64(mine);
    if (lane == 0) s.warp_sum[warp] = mine;
    if (tid() == 0) s.place = -1;
    __syncthreads();
    const u64 all = lane < kWarps ? s.warp_sum[lane] : 0;
    u64 incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += y;
    }
    if (tid() == 31) s.block_sum = incl;
    cluster.sync();
    const u64 theirs = lane < blocks ? *cluster.map_shared_rank(&s.block_sum, lane) : 0;  // (a lane to a block)
    const u64 total = warp_sum_u64(theirs);
    u64 before = warp_sum_u64(lane < rank ? theirs : 0);
    const u64 target = target_of(total);
    // the warp that lane's sum reaches past the target first, and what lies before it
    const auto pick = [&](u64 upto, u64 own) {
      const u32 past = __ballot_sync(0xFFFFFFFFu, lane < kWarps && target < before + upto);
      const int k = __ffs(past) - 1;
      before += __shfl_sync(0xFFFFFFFFu, upto - own, k);
      return k;
    };
    if (before <= target && target < before + s.block_sum) {  // (the whole block)
      const int owner = pick(incl, all);
      if constexpr (Source::LONG) {
        // the block's warps share the owner's run
        const auto part = run.part(owner, warp, kWarps);
        u64 sum = 0;
        part.each([&](int i, float z) { sum += f(z, i); });
        sum = warp_sum_u64(sum);
        if (lane == 0) s.part_sum[warp] = sum;
        __syncthreads();
        const u64 own = lane < kWarps ? s.part_sum[lane] : 0;
        u64 upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
          if (lane >= o) upto += y;
        }
        if (warp == pick(upto, own)) walk(part, f, target, before);
      } else if (warp == owner) {
        walk(run, f, target, before);
      }
    }
    cluster.sync();
    return lead->place;
  }

  // The token of a run at which the running sum, `before` at its start, passes the target, to the first block's `place`.
  template <typename R, typename F>
  __device__ __forceinline__ void walk(const R& part, F&& f, u64 target, u64 before) {
    const int lane = tid() & 31;
    for (int c = 0; c < part.rounds(); ++c) {
      float z[R::N];
      int i[R::N];
      part.round(c, z, i);
      u64 own = 0, x[R::N];
#pragma unroll
      for (int j = 0; j < R::N; ++j) own += x[j] = f(z[j], i[j]);
      u64 upto = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += y;
      }
      const u64 step = __shfl_sync(0xFFFFFFFFu, upto, 31);
      if (target < before + step) {
        u64 at = before + upto - own;
#pragma unroll
        for (int j = 0; j < R::N; ++j) {
          if (at <= target && target < at + x[j]) lead->place = i[j];
          at += x[j];
        }
        break;
      }
      before += step;
    }
  }

  // Gathers the tokens that `candidate` names, at most kList, in the first block's list.
  template <typename F>
  __device__ void gather(F&& candidate) {
    run.each_of([&](int, float z) { return candidate(z); }, [&](int i, float z) {
      const int at = atomicAdd(&lead->listed, 1);
      if (at < kList) {
        lead->list_z[at] = z;
        lead->list_i[at] = i;
        lead->list_w[at] = w(z);
      }
    });
    cluster.sync();
  }

  // First block: f(a listed token's place in the list, how many of the list come before it, their sum) for each of the n
  // listed tokens; a few neighbouring threads share a token's comparisons.
  template <typename B, typename F>
  __device__ __forceinline__ void each_listed(int n, B&& before, F&& f) {
    int log = 5;
    while (n << log > kThreads) --log;
    const int parts = 1 << log, k = tid() >> log, part = tid() & (parts - 1);
    if ((tid() & ~31) >> log >= n) return;  // (the whole warp)
    const int own = min(k, n - 1);
    const float z = s.list_z[own];
    const int i = s.list_i[own];
    u32 c = 0;
    u64 m = 0;
#pragma unroll 4
    for (int j = part; j < n; j += parts)
      if (before(s.list_z[j], s.list_i[j], z, i)) c += 1, m += s.list_w[j];
    for (int o = 1; o < parts; o <<= 1) {
      c += __shfl_xor_sync(0xFFFFFFFFu, c, o);
      m += __shfl_xor_sync(0xFFFFFFFFu, m, o);
    }
    if (k < n && part == 0) f(k, c, m);
  }
  static __device__ __forceinline__ bool ahead(float x, int j, float z, int i) { return x > z || (x == z && j < i); }

  // First block: f(a listed token's place in the list, how many of the list come before it in order, their sum) for each of the n.
  template <typename F>
  __device__ __forceinline__ void each_ranked(int n, F&& f) {
    if (n <= kFew) {
      each_listed(n, ahead, f);
      return;
    }
    // bitonic, the largest first, in the place of the histogram; equal logits by index
    u64* key = reinterpret_cast<u64*>(s.count);
    static_assert(sizeof(s.count) >= kList * sizeof(u64) && kList <= kThreads, "a key for each listed token");
    const int k = tid(), size = 1 << (32 - __clz(n - 1));
    if (k < size) key[k] = k < n ? static_cast<u64>(order_of(s.list_z[k])) << 32 | (0xFFFFFFFFu - s.list_i[k]) : 0;
    for (int half = 1; half < size; half *= 2)
      for (int apart = half; apart > 0; apart /= 2) {
        __syncthreads();
        const int i = 2 * k - (k & (apart - 1)), j = i + apart;
        if (j < size) {
          const u64 x = key[i], y = key[j];
          if ((x < y) == ((i & (2 * half)) == 0)) key[i] = y, key[j] = x;
        }
      }
    __syncthreads();
    u64 own = 0;
    if (k < n) {
      const u64 x = key[k];
      s.list_z[k] = value_of(static_cast<u32>(x >> 32)), s.list_i[k] = 0xFFFFFFFFu - static_cast<u32>(x);
      s.list_w[k] = own = w(s.list_z[k]);
    }
    const int lane = k & 31, warp = k >> 5;
    u64 upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) s.part_sum[warp] = upto;
    __syncthreads();
    u64 before = upto - own;
    for (int o = 0; o < warp; ++o) before += s.part_sum[o];
    if (k < n) f(k, static_cast<u32>(k), before);
  }

  // First block: the cut and the sum of what stays from the list, which holds every token that may stay, and of few tokens also
  // the one drawn.  The sum's bound is known to lie from mass_bound to mass_high: `sure` says whether the cut is the same for all of them.
  __device__ void finish(int n, bool by_k, u32 top_k, u64 mass_bound, u64 mass_high, float top_p, float floor_z, float uniform) {
    u32 c = 0;
    u64 before = 0;
    int mine = -1;
    each_ranked(n, [&](int k, u32 count, u64 m) {
      mine = k, c = count, before = m;
      if (by_k && count == top_k - 1) s.found_mass = m + s.list_w[k];
    });
    __syncthreads();
    if (by_k) mass_bound = mass_high = top_p < 1.f ? max(product_of(top_p, s.found_mass, true), 1ull) : ~0ull;
    bool stays = false, doubt = false;
    if (mine >= 0) {
      const bool above = s.list_z[mine] >= floor_z;
      stays = before < mass_bound && (!by_k || c < top_k) && above;
      doubt = before >= mass_bound && before < mass_high && above;
    }
    const u32 left = __syncthreads_count(stays);
    const bool doubts = __syncthreads_or(doubt);
    if (tid() == 0) s.sure = !doubts, s.place = -1;
    if (stays && c == left - 1) {
      s.cut = Cut{s.list_z[mine], s.list_i[mine]};
      s.found_mass = before + s.list_w[mine];
    }
    if (n > kFew) return;
    __syncthreads();
    const Cut cut = s.cut;
    const u64 target = product_of(uniform, s.found_mass, false);
    each_listed(
        n, [&](float x, int j, float, int i) { return j < i && (x > cut.z || (x == cut.z && j <= cut.index)); },
        [&](int k, u32, u64 m) {
          const float z = s.list_z[k];
          const int i = s.list_i[k];
          if ((z > cut.z || (z == cut.z && i <= cut.index)) && m <= target && target < m + s.list_w[k]) s.place = i;
        });
  }

  // The cut after the shortest beginning of the row whose count or sum reaches `target`, from the levels with their sums.
  // Leaves the sum up to it in lead->found_mass.  False: the row ends before.
  __device__ bool find(bool by_count, u64 target, Cut& cut) {
    const int level = level_of(by_count, target);
    u32 base_count = level == 0 ? 0 : s.all_count[level - 1];
    u64 base_mass = level == 0 ? 0 : s.all_mass[level - 1];
    u32 count = level < LEVELS ? s.all_count[level] - base_count : kList + 1;
    int bin = -1;                        // once the histogram by t has named it
    u32 low = 0, high = 0xFFFFFFFFu;     // the candidates' order, once narrowed
    auto bin_of = [&](float t) { return min(max(static_cast<int>(__fmul_rn(__fsub_rn(scaled(t), static_cast<float>(level)), static_cast<float>(kBins))), 0), kBins - 1); };
    auto candidate = [&](float z) {
      const float t = w.t_of(z);
      if (level_at(t) != level || !(z > -INFINITY) || (bin >= 0 && bin_of(t) != bin)) return false;
      const u32 o = order_of(z);
      return o >= low && o <= high;
    };
    auto narrow = [&] {  // to the bin that the bound falls into
      cluster.sync();
      cross(by_count, target, base_count, base_mass);
      cluster.sync();
      count = lead->bin_count;
      base_count = lead->base_count;
      base_mass = lead->base_mass;
      return lead->bin;
    };
    if (first_thread()) s.listed = 0;
    if (count > kList && level < LEVELS) {
      clear_bins();
      __syncthreads();
      run.each_of([&](int, float z) { return level_at(w.t_of(z)) == level; }, [&](int, float z) { put(bin_of(w.t_of(z)), w(z)); });
      bin = narrow();
    }
    if (count > kList) {
      // the range of the candidates' bits
      u32 lo = 0xFFFFFFFFu, hi = 0;
      run.each([&](int, float z) {
        if (candidate(z)) {
          const u32 o = order_of(z);
          lo = min(lo, o), hi = max(hi, o);
        }
      });
      lo = __reduce_min_sync(0xFFFFFFFFu, lo);
      hi = __reduce_max_sync(0xFFFFFFFFu, hi);
      if (tid() == 0) s.low = 0xFFFFFFFFu, s.high = 0;
      __syncthreads();
      if ((tid() & 31) == 0) atomicMin(&s.low, lo), atomicMax(&s.high, hi);
      cluster.sync();
      const int lane = tid() & 31;
      low = __reduce_min_sync(0xFFFFFFFFu, lane < blocks ? *cluster.map_shared_rank(&s.low, lane) : 0xFFFFFFFFu);
      high = __reduce_max_sync(0xFFFFFFFFu, lane < blocks ? *cluster.map_shared_rank(&s.high, lane) : 0);
      if (low > high) return false;  // none: the row has ended
      do {
        const int shift = max(0, 32 - static_cast<int>(__clz(high - low)) - 10);
        clear_bins();
        __syncthreads();
        run.each_of([&](int, float z) { return candidate(z); }, [&](int, float z) { put((high - order_of(z)) >> shift, w(z)); });
        const int digit = narrow();
        if (digit < 0) return false;
        const u32 upper = high - (static_cast<u32>(digit) << shift), width = (1u << shift) - 1;
        low = upper - low > width ? upper - width : low;
        high = upper;
      } while (count > kList && low != high);
      if (count > kList) {
        // one value, more than can be ranked: the first few by index
        const float z = value_of(high);
        const u64 each = w(z);
        const u64 left = by_count ? target - base_count : (target - base_mass + each - 1) / each;
        cut.z = z;
        cut.index = locate([&](int, float x) { return x == z; }, [](float) { return 1ull; }, [&](u64) { return left - 1; });
        if (first_thread()) s.found_mass = base_mass + left * each;
        cluster.sync();
        return true;
      }
    }
    cluster.sync();  // `listed` is 0, findings have been read
    gather(candidate);
    if (rank == 0) {
      each_ranked(min(s.listed, kList), [&](int k, u32 c, u64 m) {
        const u64 own = s.list_w[k], before = by_count ? base_count + c : base_mass + m;
        if (before < target && target <= before + (by_count ? 1 : own)) {
          s.cut = Cut{s.list_z[k], s.list_i[k]};
          s.found_mass = base_mass + m + own;
        }
      });
    }
    cluster.sync();
    cut = lead->cut;
    return true;
  }
};

// A request's settings.
struct Settings {
  float temperature, top_p, min_p, uniform;
  int top_k;
  bool by_k, by_p;
};

// What a row comes to.
struct Answer {
  Cut cut{-INFINITY, -1};    // everything above -inf stays
  float floor_z = -INFINITY;  // min-p: logits from here up stay
  u64 mass = 0;
  int token = -1;
  __device__ __forceinline__ bool stays(float z, int i) const {
    return z >= floor_z && (z > cut.z || (z == cut.z && i <= cut.index));
  }
};

// The row's answer from what `row` holds: every token (whole) or those with t below SPAN / inv.  `rest`: the sum of what it does not
// hold, in steps of 2^-42, and `off` how far that may be off.  False: it cannot be told from them.
template <typename Source>
__device__ bool answer(Row<Source>& row, const Settings& g, bool whole, u64 rest, u64 off, Answer& a) {
  Shared& s = row.s;
  const Weights& w = row.w;
  const bool first_block = row.rank == 0;
  if (g.temperature == 0.f) {
    int first = 0x7FFFFFFF;
    row.run.each([&](int i, float z) {
      if (z == w.top) first = min(first, i);
    });
    first = __reduce_min_sync(0xFFFFFFFFu, first);
    if (row.tid() % kWarp == 0 && first != 0x7FFFFFFF) atomicMin(&row.lead->place, first);
    row.cluster.sync();
    a.token = row.lead->place;
    a.cut = Cut{w.top, a.token};
    return true;
  }
  constexpr int LEVELS = Row<Source>::LEVELS;
  if (g.by_k || g.by_p) {
    u64 target = g.top_k, high;
    const bool many = g.by_k && g.top_k > kList;  // past the list: sums are wanted too
    if (g.by_k && !many) {
      row.template levels<false>();
      high = target;
    } else if (many) {
      row.template levels<true>();
      high = target;
    } else {
      row.template levels<true>();
      const u64 sum = s.all_mass[LEVELS] + rest;
      target = max(product_of(g.top_p, sum - min(off, rest), true), 1ull);
      high = max(product_of(g.top_p, sum + off, true), 1ull);
    }
    const int level = row.level_of(g.by_k, target);
    if (level == LEVELS && !whole) return false;
    if (level < LEVELS && s.all_count[level] <= kList) {
      row.gather([&](float z) { return row.level_at(w.t_of(z)) <= level; });
      const int n = s.all_count[level];
      if (first_block) row.finish(n, g.by_k, g.top_k, target, high, g.top_p, a.floor_z, g.uniform);
      row.cluster.sync();
      a.cut = row.lead->cut;
      a.mass = row.lead->found_mass;
      a.token = row.lead->place;
      // (a token in doubt that is not listed: the bound's upper end lies beyond the list)
      if (!row.lead->sure || (!g.by_k && high > s.all_mass[level])) return false;
      if (n <= kFew) return true;
      row.cluster.sync();  // findings have been read
      a.token = row.locate([&](int i, float z) { return a.stays(z, i); }, [&](float z) { return w(z); },
                           [&](u64 total) { return product_of(g.uniform, total, false); });
      return true;
    }
    if (g.by_k) {
      if (!many) {
        row.cluster.sync();  // every block's counts have been read
        row.clear_levels();
        __syncthreads();
        row.template levels<true>();
      }
      u64 total = s.all_mass[LEVELS];
      if (row.find(true, target, a.cut)) total = row.lead->found_mass;
      if (g.by_p) {
        row.cluster.sync();  // found_mass and the bins have been read
        row.find(false, max(product_of(g.top_p, total, true), 1ull), a.cut);
      }
    } else {
      row.find(false, target, a.cut);
      if (row.lead->found_mass < high) return false;
    }
    row.cluster.sync();  // findings have been read
  }
  u64& mass = a.mass;
  a.token = row.locate([&](int i, float z) { return a.stays(z, i); }, [&](float z) { return w(z); },
                       [&](u64 total) {
                         mass = total;
                         return product_of(g.uniform, total, false);
                       });
  return true;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p) {
  extern __shared__ float2 s_kept[];  // [kWarps][kKeep]
  __shared__ Shared s;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster.block_rank(), blocks = cluster.num_blocks();
  const int r = blockIdx.x / blocks;
  constexpr int N = Word<T>::N;
  griddep_launch_dependents();
  griddep_wait();
  const T* row = static_cast<const T*>(p.r.logits) + r * p.r.stride;
  const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 3) / sizeof(T));
  const int words = (p.r.vocab + shift + N - 1) / N, per_warp = p.steps * 32;
  Slice<T> slice;
  slice.row = row;
  slice.shift = shift;
  slice.V = p.r.vocab;
  slice.first = min(words, (rank * kWarps + warp) * per_warp);
  slice.last = min(words, slice.first + per_warp);
  slice.lane = lane;
  u32 now[kBatch], next[kBatch];
  auto ask = [&](u32 (&w)[kBatch], int v0) {
    if (N == 1 && v0 + 32 * kBatch <= slice.last) {
      const T* at = row + v0 + lane;
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(w[u]) : "l"(at + 32 * u));
    } else if (v0 * N - shift >= 0 && (v0 + 32 * kBatch) * N - shift <= p.r.vocab && v0 + 32 * kBatch <= slice.last) {
      const T* at = row + (v0 + lane) * N - shift;
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(w[u]) : "l"(at + 32 * N * u));
    } else {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) w[u] = slice.load(v0 + 32 * u + lane);
    }
  };
  ask(now, slice.first);
  ask(next, slice.first + 32 * kBatch);

  // the table, wanted when the row has been read
  for (int i = tid; i < static_cast<int>(sizeof(PowerTable) / 16); i += kThreads)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(reinterpret_cast<uint4*>(&s.powers) + i)),
                 "l"(reinterpret_cast<const uint4*>(&c_powers) + i)
                 : "memory");
  // (every block of the cluster reads the same words, so all of them leave here together)
  const int request = p.r.row_request ? p.r.row_request[r] : r;
  if (request < 0 || request >= p.r.requests) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (request >= 0 && rank == 0 && tid == 0) set_status(p.status, SDV_ERR_BAD_INPUT);
    return;
  }
  Settings g;
  g.temperature = p.r.temperature ? p.r.temperature[request] : 1.f;
  g.top_k = p.r.top_k ? p.r.top_k[request] : 0;
  g.top_p = p.r.top_p ? p.r.top_p[request] : 1.f;
  g.min_p = p.r.min_p ? p.r.min_p[request] : 0.f;
  g.uniform = p.r.tokens ? p.r.uniforms[r] : 0.f;
  bool bad = !(g.temperature == 0.f || (g.temperature >= 1e-30f && g.temperature <= 1e30f)) || g.top_k < 0 ||
             !(g.top_p > 0.f && g.top_p <= 1.f) || !(g.min_p >= 0.f && g.min_p <= 1.f) || !(g.uniform >= 0.f && g.uniform < 1.f);
  g.by_k = g.top_k > 0 && g.top_k < p.r.vocab, g.by_p = g.top_p < 1.f;
  if (tid == 0) {
    // log2(e) / T in two parts, the second from the first's exact remainder
    s.c = g.temperature > 0.f ? kLog2e / g.temperature : 0.f;
    s.c_low = g.temperature > 0.f ? (fmaf(-s.c, g.temperature, kLog2e) + kLog2eLow) / g.temperature : 0.f;
    s.listed = 0;
    s.over = 0;
    s.threshold = p.keep_all ? -INFINITY : kMasked;
    s.block_ref = 0.f;
    s.place = 0x7FFFFFFF;
    s.state = read_status(p.status);
  }
  // (64-bit arithmetic is slow here: one thread's, while the first loads are on their way)
  if (tid == kWarp && g.min_p > 0.f && g.temperature > 0.f)
    s.below_top = static_cast<double>(g.temperature) * log(static_cast<double>(g.min_p));

  // what a token has to reach to be kept
  if (!p.keep_all) {
#pragma unroll
    for (int k = 0; k < kSamples / kWarps; ++k) {
      float m = -INFINITY;
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        const int at = k * kGroup + u;
        float z[N];
        Word<T>::unpack(at < kBatch ? now[at] : next[at - kBatch], z);
#pragma unroll
        for (int j = 0; j < N; ++j) m = fmaxf(m, z[j]);
      }
      const int most = __reduce_max_sync(0xFFFFFFFFu, static_cast<int>(order_of(m) ^ 0x80000000u));
      if (lane == 0) s.sample[warp * (kSamples / kWarps) + k] = value_of(static_cast<u32>(most) ^ 0x80000000u);
    }
  }
  __syncthreads();
  if (!p.keep_all) {
    // a share x of the row is above the maximum of m neighbours with e^(-x m) of the maxima below it.  Kept are about a thousand
    // tokens, with top-k some times what it names, the largest alone at temperature 0
    const float most = static_cast<float>(kWarps * kKeep / 2) / (p.steps * kThreads * N);  // half of what the lists hold
    const float want = g.by_k ? fmaxf(fminf(6.f * g.top_k, 2.f * g.top_k + 1000.f), 384.f) : fmaxf(1000.f, 0.005f * p.r.vocab);
    constexpr int PARTS = kThreads / kSamples;  // threads to a sample, neighbours in a warp
    const int k = tid / PARTS;
    const float m = s.sample[k], c = s.c;
    float most_of = -INFINITY;
#pragma unroll
    for (int j = 0; j < kSamples / PARTS; ++j) most_of = fmaxf(most_of, s.sample[j * PARTS + tid % PARTS]);
#pragma unroll
    for (int o = 1; o < PARTS; o <<= 1) most_of = fmaxf(most_of, __shfl_xor_sync(0xFFFFFFFFu, most_of, o));
    // neighbours that are all masked, by -inf or by the type's lowest value, say nothing of what may stay
    auto counts = [&](float x) { return x > kMasked && (x == most_of || (most_of - x) * c < 100.f); };
    int there = 0, below = 0;
#pragma unroll
    for (int j = 0; j < kSamples / PARTS; ++j) {
      const int at = j * PARTS + tid % PARTS;
      const float x = s.sample[at];
      there += counts(x);
      below += counts(x) && (x < m || (x == m && at < k));
    }
#pragma unroll
    for (int o = 1; o < PARTS; o <<= 1) {
      there += __shfl_xor_sync(0xFFFFFFFFu, there, o);
      below += __shfl_xor_sync(0xFFFFFFFFu, below, o);
    }
    // (of the part that is not masked)
    const float share = g.temperature == 0.f ? 0.f : fminf(want * kSamples / (static_cast<float>(p.r.vocab) * max(there, 1)), most);
    const int nth = min(static_cast<int>(there * __expf(-share * (32 * kGroup * N))), there - 1);
    if (counts(m) && below == nth) s.threshold = m;
    if (tid == 0 && most_of > kMasked) s.block_ref = most_of;
    __syncthreads();
  }
  const float threshold = fmaxf(s.threshold, -3.402823466e38f), ref = s.block_ref, c = s.c;
  const bool sums = g.by_p && !g.by_k && !p.keep_all;

  // the row, once: its maximum (NaN if there is one), what is kept and the sum of what is not
  float top = -INFINITY, rest[4] = {0.f, 0.f, 0.f, 0.f};
  float2* list = s_kept + warp * kKeep;
  const u32 below = (1u << lane) - 1;
  int n = 0;
  bool over = false;
  float* out = p.r.probs && s.state == 0 ? p.r.probs + r * p.r.probs_stride : nullptr;
  const bool wide = N == 2 && (reinterpret_cast<uintptr_t>(out - shift) & 7) == 0;  // a word's two values at once
  for (int v0 = slice.first; v0 < slice.last; v0 += 32 * kBatch) {
#pragma unroll
    for (int u0 = 0; u0 < kBatch; u0 += kGroup) {
      float z[kGroup][N], most = -INFINITY;
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        Word<T>::unpack(now[u0 + u], z[u]);
#pragma unroll
        for (int j = 0; j < N; ++j) most = max_nan(most, z[u][j]);
      }
      top = max_nan(top, most);
      if (sums) {
#pragma unroll
        for (int u = 0; u < kGroup; ++u)
#pragma unroll
          for (int j = 0; j < N; ++j) {
            float y;
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((z[u][j] - ref) * c));
            rest[u] += z[u][j] < threshold ? y : 0.f;
          }
      }
      if (!__any_sync(0xFFFFFFFFu, most >= threshold)) continue;
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        u32 votes[N], any = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) any |= votes[j] = __ballot_sync(0xFFFFFFFFu, z[u][j] >= threshold);
        if (!any) continue;
        const int i = (v0 + 32 * (u0 + u) + lane) * N - shift;
        int at = n, all = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) at += __popc(votes[j] & below), all += __popc(votes[j]);
        if (n + all <= kKeep) {
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (z[u][j] >= threshold) list[at++] = make_float2(z[u][j], __int_as_float(i + j));
          n += all;
        } else {
          over = true;
        }
      }
    }
    if (out) {  // zeros; what stays is written over them
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int v = v0 + 32 * u + lane, i = v * N - shift;
        if (v >= slice.last) break;
        if (wide && i >= 0 && i + N <= p.r.vocab) {
          *reinterpret_cast<float2*>(out + i) = make_float2(0.f, 0.f);
        } else {
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (N == 1 || (i + j >= 0 && i + j < p.r.vocab)) out[i + j] = 0.f;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) now[u] = next[u];
    ask(next, v0 + 2 * 32 * kBatch);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const float mine = warp_sum((rest[0] + rest[1]) + (rest[2] + rest[3]));
  if (lane == 0) {
    s.warp_max[warp] = top, s.warp_rest[warp] = mine;
    if (over) s.over = 1;
  }
  Row<Kept> kept{cluster, s, cluster.map_shared_rank(&s, 0), Kept{list, n, lane}, {}, rank, blocks, 0.f};
  kept.clear_levels();
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  if (warp == 0) {
    top = s.warp_max[lane % kWarps];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float all = warp_sum(lane < kWarps ? s.warp_rest[lane] : 0.f);
    if (lane == 0) s.block_max = top, s.block_rest = all;
  }
  cluster.sync();
  const Shared* theirs = cluster.map_shared_rank(&s, lane < blocks ? lane : 0);  // (a lane to a block)
  top = theirs->block_max;
  float from = theirs->threshold;  // kept: every token of the row from here up
  over = __any_sync(0xFFFFFFFFu, theirs->over != 0);
#pragma unroll
  for (int o = kMaxCluster / 2; o > 0; o >>= 1) {
    top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    from = fmaxf(from, __shfl_xor_sync(0xFFFFFFFFu, from, o));
  }
  top = __shfl_sync(0xFFFFFFFFu, top, 0);
  from = __shfl_sync(0xFFFFFFFFu, from, 0);
  // a word that was set before the call or by another row of it: the first block's view counts for all
  if (kept.lead->state != 0) {
    cluster.sync();  // (the first block's shared memory has been read)
    return;
  }
  bad |= !(top > -INFINITY);

  Answer a;
  Weights w;
  w.top = top;
  w.powers = &s.powers;
  w.c = c;
  w.c_low = s.c_low;
  if (!bad) {
    if (g.min_p > 0.f && g.temperature > 0.f) {
      // w >= min_p: z >= max + T ln(min_p), the first fp32 value of them
      if (tid == 0) s.floor_z = g.min_p == 1.f ? top : __double2float_ru(static_cast<double>(top) + s.below_top);
      __syncthreads();
      a.floor_z = s.floor_z;
    }
    bool told = false;
    const bool whole = from == -INFINITY;
    // levels end with what is kept; beyond t = 44 weights are 0
    const float t_from = fminf(w.t_of(from), 64.f);
    if (!over && (whole || (g.temperature == 0.f && top >= from) || (g.temperature > 0.f && t_from > 0.f && (g.by_k || g.by_p || a.floor_z >= from)))) {
      kept.w = w;
      kept.inv = t_from > 0.f ? __fdiv_ru(Kept::SPAN, t_from) : 0.f;
      float others = 0.f;
      if (sums) others = warp_sum(lane < blocks && theirs->block_rest > 0.f ? theirs->block_rest * exp2f((theirs->block_ref - top) * c) : 0.f);
      // in steps of 2^-42.  Its error, up to t = 32: of t a difference, a product, the quotient log2(e) / T (2^-24 each) and log2(e) itself
      // (2^-26), alike for the scale to `top`, 1.7 * 2^-23 of t in all, so 2^-17.7 of a term; 2^-22 of each exponential; 2^-16 of a
      // thread's sums of up to 250 terms; and 2^-19.4 of the weights that it stands for: below 2^-15 together.  Beyond t = 32 2^20 tokens add up to 2^-12 of the largest weight at
      // most, with errors of 2^-16: 2^-28.  What the sum stands for has each token rounded to a step, half of one away at most.
      const u64 sum = static_cast<u64>(others * 4398046511104.f);
      const u64 off = (sum >> 15) + (1 << 14) + p.r.vocab / 2;
      told = answer(kept, g, whole, sum, sums ? off : 0, a);
    }
    if (!told) {
      cluster.sync();  // findings and sums have been read
      kept.clear_levels();
      if (tid == 0) s.listed = 0;
      cluster.sync();
      if (over) kept.run.n = 0;
      const Both<T> both{slice, kept.run, over ? NAN : threshold, per_warp, words, rank * kWarps};
      Row<Both<T>> full{cluster, s, kept.lead, both, w, rank, blocks, Both<T>::SPAN / kLast};
      a.cut = Cut{-INFINITY, -1};
      answer(full, g, true, 0, 0, a);
      if (out) {
        const float inv = 4398046511104.f / static_cast<float>(a.mass);
        const int end = min(p.r.vocab, slice.last * N - shift);  // (a round's lanes may lie past the run)
        both.each([&](int i, float z) {
          if (i >= 0 && i < end) out[i] = !a.stays(z, i) ? 0.f : g.temperature == 0.f ? 1.f : w.share(z) * inv;
        });
      }
    } else if (out) {
      const float inv = 4398046511104.f / static_cast<float>(a.mass);
      kept.run.each([&](int i, float z) {
        if (a.stays(z, i)) out[i] = g.temperature == 0.f ? 1.f : w.share(z) * inv;
      });
    }
  }
  if (rank == 0 && tid == 0) {
    if (bad) set_status(p.status, SDV_ERR_BAD_INPUT);
    if (p.r.tokens) p.r.tokens[r] = a.token;
  }
  cluster.sync();  // the first block's shared memory is read until here
}

template <typename T>
cudaError_t launch(const sdv_sample_rows& rows, int* status, int device, int sms, cudaStream_t stream) {
  constexpr int N = Word<T>::N;
  const int words = rows.vocab / N + 2;  // at most, wherever the row begins
  // more blocks to a row while they are few for the SMs, and runs of at most 1000 values a thread.  A block costs some 8 us beside its run;
  // two run on an SM, so pairs may be a little more than run at once (11 / 4 to an SM), fours as many (2) and eights half of that, as
  // clusters of 8 leave SMs unfilled.  The three limits stand between these measured points; nothing was measured nearer to them, and
  // rows that row_request turns off count as rows.  Rows x values (fp32): us with 1, 2, 4 and 8 blocks
  //   512 x 151936, top-p       107  128 174 310      64 x 151936, mixed settings  81  51  41  62
  //   200 x 50000, distributions 173 64 112 167     40 x 20011, no setting       25  21  15  21
  int blocks = 1;
  auto steps = [&](int b) { return (words + b * kThreads - 1) / (b * kThreads); };
  auto fit = [&](int b) { return static_cast<long long>(rows.rows) * b <= (b == 2 ? sms * 11 / 4 : b == 4 ? sms * 2 : sms); };
  while (blocks < kMaxCluster && ((steps(blocks) > 4 && fit(2 * blocks)) || steps(blocks) * N > 1000)) blocks *= 2;
  SampleParams p{rows, status, steps(blocks), steps(blocks) * 32 * N <= kKeep};
  constexpr int smem = kWarps * kKeep * sizeof(float2);
  // the kernel's leave to take so much shared memory, once per device
  static std::atomic<unsigned long long> allowed{0};
  const unsigned long long bit = device < 64 ? 1ull << device : 0;
  if (!bit || !(allowed.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  const cudaError_t e = launch_pdl_cluster(sample_kernel<T>, blocks, dim3(rows.rows * blocks), dim3(kThreads), smem, stream, p);
  if (e != cudaSuccess) allowed.fetch_and(~bit, std::memory_order_relaxed);  // (a reset device has forgotten it)
  return e;
}

}  // namespace
}  // namespace sdv

using namespace sdv;

extern "C" sdv_status sdv_sample(const sdv_sample_rows* r, int* status, void* stream) {
  if (!r || !status) return SDV_ERR_INVALID_ARG;
  if (r->rows < 0 || r->vocab <= 0 || r->requests < 0 || (r->x_format != 0 && r->x_format != 1)) return SDV_ERR_INVALID_ARG;
  if (!r->row_request && r->requests < r->rows) return SDV_ERR_INVALID_ARG;
  if (r->rows > (1 << 20)) return SDV_ERR_CAPACITY;
  if (r->vocab > (1 << 20)) return SDV_ERR_UNSUPPORTED;
  if (r->rows == 0) return SDV_OK;  // no rows: their pointers may be null
  const int bytes = r->x_format ? 4 : 2;
  if (!r->logits || r->stride < r->vocab || (reinterpret_cast<uintptr_t>(r->logits) & (bytes - 1))) return SDV_ERR_INVALID_ARG;
  if (!r->tokens && !r->probs) return SDV_ERR_INVALID_ARG;
  if (r->tokens && !r->uniforms) return SDV_ERR_INVALID_ARG;
  if (r->probs && (r->probs_stride < r->vocab || (reinterpret_cast<uintptr_t>(r->probs) & 3))) return SDV_ERR_INVALID_ARG;
  // (zeros are written while the row is read, and a row may be read again)
  if (r->probs && rows_share(r->logits, r->stride * bytes, 1LL * r->vocab * bytes, r->probs, r->probs_stride * 4, 4LL * r->vocab, r->rows))
    return SDV_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = r->x_format ? launch<float>(*r, status, dev, sms, static_cast<cudaStream_t>(stream))
                    : launch<__nv_bfloat16>(*r, status, dev, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SDV_OK : cuda_fail(e);
}
