// Attention of a ragged chunk over the paged cache on the 5th-generation tensor
// cores, for sequences of more than 16 packed rows (prompts, pieces of them, many drafts).
//
// An item is two tiles of 128 packed query rows (row = token, head of the group)
// of one (sequence, key head) against the blocks of 128 keys that they see.  The
// items' blocks are laid end to end, weighed by what they cost, and cut into
// equal runs, one per SM; the parts of an item cut between SMs are joined in the
// runs' order, so equal inputs give equal bits.  Per step of 64 keys and tile t
//   S_t = Q_t K^T  (M = 128 rows, N = 64 keys),  O_t += P_t V  (P_t from TMEM):
// one thread issues each tile's products, S of the next step before this step's
// softmax is waited for, into the other of two buffers; a thread of the softmax
// holds one row, reads its scores from TMEM once and writes the weights over
// them in 16 bits (bf16 with a bf16 cache, fp16 with codes: half a step of each
// weight is the one rounding between the scores and the output's own; fp16's small
// weights: kAbove).  The running maximum is a bound, set by the first step and moved only
// when a step's weights add up to more than kMost, or with codes to too little (then the step is taken
// again and O is rescaled in TMEM): their sum, which is needed anyway, stands in for a maximum.
//
// TMEM: two buffers of S_t for each tile (64 columns, P over the first 32), O_0, O_1.
// Shared memory: Q tiles and a ring of K and V blocks, rows of 128 bytes,
// 128-byte swizzle.  A bf16 cache is loaded by TMA, a page's 64-wide half a copy,
// by two warps; e4m3 codes go through four warps' registers and land as fp16, scales
// applied, exact.  Values of keys that an item's rows cannot see are zeroed in
// shared memory, so that nothing behind a sequence's end is ever multiplied.
//
// What bounds it, 32 query and 8 key heads of 128, bf16: 2048 new tokens over 32749
// take 725 to 750 us back to back (1450 TFLOP/s, 0.76 of the burst peak, 0.85 of the sustained one: the power
// limit holds it there; a few calls after a pause take 667).  A block of two tiles takes 2780 cycles: its
// products 2560 (N = 64 scores wait for shared memory: 48 cycles each in place
// of 32, measured), the rest is the round from a step's weights to the scores
// after next.  Scores of 128 keys at once into one buffer, their weights in
// halves, the tiles taking turns, were slower (903 us: the softmax waits for each round).  One
// issuing thread for both tiles under `lane == 0` issued at 70 cycles a product (1001 us).
// With codes the same work takes 758 us, and 64 sequences of 16 rows 248 us against
// 229 in bf16: a step of two tiles takes 1600 cycles in place of 1390, for the four
// converting warps share the issue slots and the instruction cache with the softmax (without its
// exponentials a step takes as long).  What helped is less code and fewer instructions:
// the next codes are asked for only when the last are published (64 x 16 rows 260 -> 249 us),
// stores that need no swap (280 -> 260), short loops at an item's ends (315 -> 283),
// no spilled register (a few in the conversion cost 50 us).  What did not: eight converting
// warps, codes by bulk copies through shared memory, blocks of 64 keys.
#include "chunk.cuh"
#include "tcgen05.cuh"

namespace sdv {
namespace {

using namespace tc;

constexpr int BM = 128;              // query rows of a tile
constexpr int BK = 128;              // keys of a block
constexpr int BPAGES = BK / kPage;
constexpr int SK = 64;               // keys of a step: half a block
constexpr int HALF = BM * 128;       // 64 columns of 128 rows: 16 KB
constexpr float kNoMax = -1e30f;     // the bound before the first visible key, in base-2 logits
// A row's weights of one step may add up to this before its bound moves: each
// then fits fp16, and no maximum is taken in the steps between.
constexpr float kMost = 16384.f, kMostCodes = 60000.f;
// Codes: the weights are fp16, of 2^-14 at least in its normal range, so the bound is set
// kAbove binades below a step's largest logit, and a step whose weights add up to less than kLeast
// (64 equal ones: 2^-14 each) moves it down, sum and output scaling up (they are fp32): one key far above the
// rest takes nothing from the steps behind it, and of its own step what lies 2^-18 below it keeps fewer bits.
// A bound moves down by kDropMost binades at most, and no more once the sum is past kSumMost (sums stay
// below 2^101, outputs below 2^117): what is lost then is below 2^-50 of the sum.  bf16 weights have fp32's
// range and need none of it.  (kAbove 2, 4, 6, 8: six pieces of prompts 95.4, 94.4, 94.4, 96.4 us, 91.2 without
// moves down; 2048 tokens over 8200 195.0, 195.0, 195.4, 199.4 us, 194.5 without.)
constexpr float kAbove = 4.f, kLeast = 0x1p-8f, kSumMost = 0x1p50f, kDropMost = 48.f;
// An item of up to this many parts more than one is joined by its last block, one of more by chunk_join_kernel
// (2, 4, 6: 64 sequences x 8 rows over codes, heads of 64, 165, 171, 186 us, of 128 235, 236, 237; 4096 new
// tokens, bf16, heads of 128, 119, 120, 121).
constexpr int kJoinHere = 4;

constexpr int MMA_WARP = 8, TMA_WARP = 10, CONV_WARP = 12;  // MMA_WARP + t issues tile t's products, TMA_WARP + 1 copies V

template <int D, int FMT>
struct Cfg {
  static constexpr bool kCodes = FMT == SDV_CACHE_E4M3;
  static constexpr int THREADS = kCodes ? 512 : 384;
  static constexpr int HALVES = D / 64;
  static constexpr int SLOT = HALVES * HALF;          // K or V of one block
  static constexpr int NS = D == 128 ? 5 : 8;
  static constexpr int OFF_Q = NS * SLOT;
  static constexpr int OFF_BAR = OFF_Q + 2 * SLOT;
  static constexpr int NBAR = 2 * NS + 2 * 7 + 2;     // full, empty; s, p (two each), q, v, o of each tile; tail, done
  static constexpr int SMEM = 1024 + OFF_BAR + NBAR * 8 + 64;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static constexpr int FULL_COUNT = kCodes ? 4 : 1;
  // registers a thread: softmax, products and copies, conversion (launched with
  // 65536 / THREADS, rounded down to a multiple of 8: 168, or 128)
  static constexpr int R_SOFT = kCodes ? 168 : 192, R_ISSUE = kCodes ? 64 : 120, R_CONV = 112;
  static_assert(2 * R_SOFT + R_ISSUE + (kCodes ? R_CONV : 0) <= (kCodes ? 4 * 128 : 3 * 168), "register shares");
  static constexpr int T_O = 2 * BK;                  // TMEM columns of O_0
};

// Shared-memory descriptors (128-byte swizzle, version 1) as two words: the low
// one holds the address and is all that changes from product to product, so
// the issuing thread adds a constant to it and nothing else.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // 1024 bytes between 8-row groups
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }                        // K-major
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr) { return (saddr >> 4) | (static_cast<uint32_t>(HALF >> 4) << 16); }  // V rows, MN-major: 16 KB between 64-column halves

// fp32 accumulate; bf16 operands, or fp16 (format 0)
__host__ __device__ constexpr uint32_t idesc(bool f16, int N, bool b_mn) {
  return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(BM >> 4) << 24);
}

// D (+)= A B, both from shared memory; acc 0 starts D anew.
template <uint32_t ID>
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t acc) {
  asm volatile(
      "{\n"
      " .reg .pred p;\n"
      " .reg .b64 a, b;\n"
      " mov.b64 a, {%1, %3};\n"
      " mov.b64 b, {%2, %3};\n"
      " setp.ne.b32 p, %5, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n"
      "}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "n"(kDescHi), "r"(ID), "r"(acc));
}
// The same with A from TMEM.
template <uint32_t ID>
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t acc) {
  asm volatile(
      "{\n"
      " .reg .pred p;\n"
      " .reg .b64 b;\n"
      " mov.b64 b, {%2, %3};\n"
      " setp.ne.b32 p, %5, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n"
      "}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "n"(kDescHi), "r"(ID), "r"(acc));
}

// One lane of the warp, known as such to the compiler: what it issues takes its operands
// from uniform registers (8 products of 64 columns cost 37 cycles each to issue, 70 under lane == 0).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n"
      " .reg .pred p;\n"
      " elect.sync _|p, 0xffffffff;\n"
      " selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(r));
  return r != 0;
}

// mbar_wait with the clock read only after the barrier has been asked for a while.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t addr = smem_u32(bar);
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(addr, parity)) return true;
  return mbar_wait(bar, parity);
}

// 16 bytes into shared memory, or 16 zeros (bytes = 0: src is not read).
__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Registers per thread of this warpgroup (the shares of all add up to the launch's).
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

#define R8(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7])
#define W8(v, o) "+r"(v[o]), "+r"(v[o + 1]), "+r"(v[o + 2]), "+r"(v[o + 3]), "+r"(v[o + 4]), "+r"(v[o + 5]), "+r"(v[o + 6]), "+r"(v[o + 7])
#define I8(v, o) "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7])

// 32 lanes x 32 columns; the registers hold the values only after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
      "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : R8(r, 0), R8(r, 8), R8(r, 16), R8(r, 24)
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : W8(r, 0), W8(r, 8), W8(r, 16), W8(r, 24)::"memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
      "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      I8(r, 0), I8(r, 8), I8(r, 16), I8(r, 24)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 lanes in one instruction.
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unf2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The blocks of 256 packed rows of a sequence, and what each of its tiles sees.
struct Item {
  int row0, rows;       // packed rows
  int klo, khi;         // keys that a row sees (khi = 0: none)
  int page_lo, blocks;  // first page; blocks of BK keys (one at least)
};
__device__ __forceinline__ Item make_item(const SeqRows& s, int group, int window, int qt) {
  Item it;
  it.row0 = qt * 2 * BM;
  it.rows = min(2 * BM, s.n * group - it.row0);
  const int pmin = s.pos0 + it.row0 / group, pmax = s.pos0 + (it.row0 + it.rows - 1) / group;
  it.khi = max(0, pmax + 1);
  it.klo = min(it.khi, window > 0 ? max(0, pmin - window + 1) : 0);
  it.page_lo = it.klo / kPage;
  it.blocks = max(1, (it.khi - it.page_lo * kPage + BK - 1) / BK);
  return it;
}
// The item's steps [s0, s1) that tile t needs, and its rows' range of positions.
struct Tile {
  int rows, pmin, pmax, s0, s1;
};
__device__ __forceinline__ Tile make_tile(const SeqRows& s, const Item& it, int group, int window, int t) {
  Tile x;
  x.rows = min(BM, it.rows - t * BM);
  x.s0 = x.s1 = 0;
  x.pmin = x.pmax = -1;
  if (x.rows <= 0) return x;
  const int r0 = it.row0 + t * BM;
  x.pmin = s.pos0 + r0 / group;
  x.pmax = s.pos0 + (r0 + x.rows - 1) / group;
  const int hi = x.pmax + 1, lo = window > 0 ? max(0, x.pmin - window + 1) : 0;
  if (hi <= lo || hi <= 0) return x;
  x.s0 = (lo - it.page_lo * kPage) / SK;
  x.s1 = (hi - it.page_lo * kPage + SK - 1) / SK;
  return x;
}

// What a block of the item costs, and an item before its first block (query,
// first scores, output), in eighths of a block of two tiles: a block
// of one tile takes 2450 cycles against 2750 (bf16, heads of 128; measured there and used for all).
// Items at 1.5, 3 and 4.5 blocks, us: 4096 new tokens bf16 134, 120, 122, heads of 64 104, 99, 101, codes 159, 139, 138;
// six pieces of prompts bf16 106, 103, 103, codes 120, 119, 115.  Blocks of one tile at 8 in place of 7: within 2 %
// either way, but six pieces over codes 119 -> 115.
// (With items free the SMs with the short ones ended last: 4096 new tokens 193 us.)
__device__ __forceinline__ int weight(const Item& it) { return it.rows > BM ? 8 : 7; }
constexpr int kItemCost = 24;
__device__ __forceinline__ int units_of(const Item& it) { return kItemCost + it.blocks * weight(it); }

// A part of a run: blocks [b0, b1) of an item of (sequence b, key head h) whose first unit is u0.
struct Part {
  SeqRows s;
  Item it;
  int b, h, qt, b0, b1;
  long long u0;
};
// An item whose output is to be taken from TMEM: its rows, the runs [first, last] that hold a
// part of it, and whether this one had steps.
struct Held {
  int off, h, row0, rows, first, last, went;
};
struct Place {
  int b, h, qt, blk;
  long long u0;
};

// Where run `cta` leaves its part of tile t of the item that begins in run
// c_first: a run has two at most, of an item begun before it and of one that goes on behind it.
__device__ __forceinline__ float* part_slot(float* part, int D, int cta, int c_first, int t) {
  return part + ((2LL * cta + (cta == c_first)) * 2 + t) * ((long long)BM * (D + 2));
}

template <int D, int FMT>
__global__ void __launch_bounds__(Cfg<D, FMT>::THREADS, 1)
    chunk_attn_tc_kernel(const __grid_constant__ CUtensorMap tmKV, const ChunkAttnParams p) {
  using C = Cfg<D, FMT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::NS;
  uint64_t* s_full = empty + C::NS;  // [tile][buffer] a step's scores are in TMEM
  uint64_t* p_full = s_full + 4;     // [tile][buffer] its weights are, and O may be added to
  uint64_t* q_full = p_full + 4;     // [tile]
  uint64_t* v_done = q_full + 2;     // [tile] a step's second product is in O
  uint64_t* o_full = v_done + 2;     // [tile] the item's last one is
  uint64_t* tail = o_full + 2;       // copies of a block whose end is zeroed before use
  uint64_t* done = tail + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  __shared__ long long s_scan[2];  // units of a run; of the launch
  __shared__ Place s_start;
  // the softmax warps' place in the run, and the item whose output is still in
  // TMEM: out of the registers of their inner loop
  __shared__ Part s_part[8];
  __shared__ Held s_held[8];
  __shared__ int s_flag[2][2];     // [tile][turn] whether the others' parts of an item are all there

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&full[i], C::FULL_COUNT);
      mbar_init(&empty[i], 2);  // both tiles' products have read it
    }
    for (int t = 0; t < 2; ++t) {
      for (int n = 0; n < 2; ++n) {
        mbar_init(&s_full[2 * t + n], 1);
        mbar_init(&p_full[2 * t + n], 4);
      }
      mbar_init(&q_full[t], 4);
      mbar_init(&v_done[t], 1);
      mbar_init(&o_full[t], 1);
    }
    mbar_init(tail, 1);
    mbar_init(done, 2);
    fence_barrier_init();
  }
  if (warp == MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  griddep_launch_dependents();  // (only now that this block has its TMEM)
  griddep_wait();

  const int B = p.c.B, group = p.c.n_q / p.c.n_kv, window = p.c.window, n_kv = p.c.n_kv;
  auto seq_of = [&](int b) {
    const int o = p.c.row_offsets[b], e = p.c.row_offsets[b + 1], len = p.c.kv_lens[b];
    SeqRows s{o, e - o, len, len - (e - o)};
    if (s.n * group <= p.small_rows) s.n = 0;  // the other kernel's
    return s;
  };
  auto items_of = [&](const SeqRows& s) { return (int)(((long long)s.n * group + 2 * BM - 1) / (2 * BM)); };

  // ---- the chunk's check and this block's run of units ----
  bool good, dead0;
  {
    int bad = 0;
    const int status0 = read_status(p.c.status);
    for (int b = tid; b < B; b += blockDim.x) {
      const int o = p.c.row_offsets[b], e = p.c.row_offsets[b + 1], len = p.c.kv_lens[b];
      if (o < 0 || e < o || e > p.c.T || e - o > p.c.max_q || (b == 0 && o != 0) || len < 0) bad |= 1;
      if (len > (long long)p.c.max_pages * kPage) bad |= 2;
    }
    const bool b1 = __syncthreads_or(bad & 1), b2 = __syncthreads_or(bad & 2);
    dead0 = __syncthreads_or(status0 != 0);  // one verdict for the block
    if ((b1 || b2) && tid == 0) set_status(p.c.status, b1 ? SDV_ERR_BAD_INPUT : SDV_ERR_PAGE_RANGE);
    good = !b1 && !b2;
    if (tid == 0) p.cuts[2 * blockIdx.x].x = -1;  // no item begins here and goes on, so far
  }
  long long u_begin = 0, u_end = 0, per_cta = 1;
  if (good) {
    // units (items and blocks by what they cost) of one key head of each sequence, a warp a sequence, into the ring (not in use yet)
    long long* s_units = reinterpret_cast<long long*>(smem);  // [B]
    for (int b = warp; b < B; b += blockDim.x / kWarp) {
      const SeqRows s = seq_of(b);
      long long sum = 0;
      for (int qt = lane; qt < items_of(s); qt += kWarp) {
        sum += units_of(make_item(s, group, window, qt));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) s_units[b] = sum;
    }
    __syncthreads();
    if (warp == 0) {
      // total, then the sequence, key head, item and block of the run's first unit
      long long total = 0;
      for (int b0 = 0; b0 < B; b0 += kWarp) {
        long long v = b0 + lane < B ? s_units[b0 + lane] * n_kv : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        total += v;
      }
      const long long per = max(8LL, (total + gridDim.x - 1) / gridDim.x);  // eight: a block begins in every run that an item spans
      const long long u = (long long)blockIdx.x * per;
      if (u < total) {
        long long base = 0;
        int b = -1;
        for (int b0 = 0; b0 < B && b < 0; b0 += kWarp) {
          const long long v = b0 + lane < B ? s_units[b0 + lane] * n_kv : 0;
          long long inc = v;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const long long w = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += w;
          }
          const unsigned hit = __ballot_sync(0xffffffffu, base + inc > u);
          if (hit) {
            const int l = __ffs(hit) - 1;
            b = b0 + l;
            base += __shfl_sync(0xffffffffu, inc - v, l);
          } else {
            base += __shfl_sync(0xffffffffu, inc, 31);
          }
        }
        const SeqRows s = seq_of(b);
        const long long per_head = s_units[b];
        const int h = static_cast<int>((u - base) / per_head);
        long long rest = (u - base) - h * per_head;
        int qt = -1;
        for (int q0 = 0; qt < 0; q0 += kWarp) {
          const long long v = q0 + lane < items_of(s) ? units_of(make_item(s, group, window, q0 + lane)) : 0;
          long long inc = v;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const long long w = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += w;
          }
          const unsigned hit = __ballot_sync(0xffffffffu, inc > rest);
          if (hit) {
            const int l = __ffs(hit) - 1;
            qt = q0 + l;
            rest -= __shfl_sync(0xffffffffu, inc - v, l);
          } else {
            rest -= __shfl_sync(0xffffffffu, inc, 31);
          }
        }
        if (lane == 0) {
          // the first block that begins at the run's first unit or behind it
          const int w = weight(make_item(s, group, window, qt));
          s_start = Place{b, h, qt, static_cast<int>((max(0LL, rest - kItemCost) + w - 1) / w), u - rest};
        }
      }
      if (lane == 0) {
        s_scan[0] = per;
        s_scan[1] = total;
      }
    }
    fence_proxy_async_smem();  // the ring's next writers are copies
    __syncthreads();
    per_cta = s_scan[0];
    u_begin = (long long)blockIdx.x * per_cta;
    u_end = min(s_scan[1], u_begin + per_cta);
  }
  // the parts of the run, one after another; a block is of the run that its first unit falls in
  auto end_block = [&](const Part& x) {  // blocks of x that begin before the run's end
    const int w = weight(x.it);
    return (static_cast<int>(min((long long)x.it.blocks * w, max(0LL, u_end - x.u0 - kItemCost))) + w - 1) / w;
  };
  auto next_part = [&](Part& x) {
    {
      x.u0 += units_of(x.it);
      if (x.u0 >= u_end) return false;
      x.b0 = 0;
      if (++x.qt == items_of(x.s)) {
        x.qt = 0;
        if (++x.h == n_kv) {
          x.h = 0;
          do x.s = seq_of(++x.b);
          while (x.s.n == 0);
        }
      }
      x.it = make_item(x.s, group, window, x.qt);
      x.b1 = end_block(x);
      if (x.b1 == 0) return false;
      return true;
    }
  };
  auto first_part = [&](Part& x) {
    if (u_begin >= u_end) return false;
    const Place at = s_start;
    x.b = at.b, x.h = at.h, x.qt = at.qt, x.b0 = at.blk, x.u0 = at.u0;
    x.s = seq_of(x.b);
    x.it = make_item(x.s, group, window, x.qt);
    x.b1 = end_block(x);
    return x.b0 < x.b1 || next_part(x);
  };
  auto walk = [&](auto&& f) {
    Part x;
    for (bool more = first_part(x); more; more = next_part(x))
      if (!f(x.s, x.b, x.h, x.it, x.b0, x.b1)) return;
  };
  auto clip = [](Tile x, int b0, int b1) {  // the tile's steps within blocks [b0, b1)
    x.s0 = max(x.s0, 2 * b0);
    x.s1 = min(x.s1, 2 * b1);
    if (x.s0 >= x.s1) x.s0 = x.s1 = 0;
    return x;
  };

  // the blocks that either tile needs: their ranges meet, for a tile's rows
  // follow one another and so do the positions that they see
  auto both = [](const Tile& a, const Tile& b) {
    if (a.s0 >= a.s1) return make_int2(b.s0 >> 1, (b.s1 + 1) >> 1);
    if (b.s0 >= b.s1) return make_int2(a.s0 >> 1, (a.s1 + 1) >> 1);
    return make_int2(min(a.s0, b.s0) >> 1, (max(a.s1, b.s1) + 1) >> 1);
  };
  auto load = [&](int kv0) {
    // ---------------- loads: K and V of each block into the ring, in turn ----------------
    // bf16: one warp copies the keys (kv0 = 0), one the values; codes: four warps take both
    constexpr int EVERY = C::kCodes ? 1 : 2;
    int slot = kv0;
    uint32_t phase = 0, tail_phase = 0;
    bool dead = dead0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!dead && !bar_wait(bar, parity)) {
        set_status(p.c.status, SDV_ERR_TIMEOUT);
        dead = true;
      }
      dead = __any_sync(0xffffffffu, dead);
    };
    auto next = [&]() {
      slot += EVERY;
      if (slot >= C::NS) {
        slot -= C::NS;
        phase ^= 1;
      }
    };
    walk([&](const SeqRows& s, int b, int h, const Item& it, int b0, int b1) {
      const Tile t0 = clip(make_tile(s, it, group, window, 0), b0, b1), t1 = clip(make_tile(s, it, group, window, 1), b0, b1);
      const int2 used = both(t0, t1);
      if (used.x >= used.y || dead) return !dead;
      const int* table = p.c.page_table + (long long)b * p.c.max_pages;
      const int page0 = it.page_lo + used.x * BPAGES, pages_end = min((it.khi + kPage - 1) / kPage, it.page_lo + used.y * BPAGES);
      // the lanes hold the pages of four blocks, and fetch the next four's meanwhile
      auto fetch = [&](int jj) {
        int pg = 0;
        if (page0 + jj * BPAGES + lane < pages_end) {
          pg = table[page0 + jj * BPAGES + lane];
          if (pg < 0 || pg >= p.c.pool_pages) {
            set_status(p.c.status, SDV_ERR_PAGE_RANGE);
            pg = 0;  // some page of the pool: the call's outputs hold nothing meaningful
          }
        }
        return pg;
      };
      int ids = fetch(0), ids_next = fetch(4);
      auto seen = [&](int jj) {  // the rows [x, y) of block jj that are seen
        const int key0 = (page0 + jj * BPAGES) * kPage;
        return make_int2(max(0, it.klo - key0), min(BK, it.khi - key0));
      };
      const int n = used.y - used.x;
      if constexpr (!C::kCodes) {
        for (int jj = 0; jj < n; ++jj) {
          if (jj && (jj & 3) == 0) {
            ids = ids_next;
            ids_next = fetch(jj + 4);
          }
          const int2 rows = seen(jj);
          const int pages = (rows.y + kPage - 1) / kPage;
          // lane 2 i + half copies that half of page i's rows
          const int pgi = C::HALVES == 2 ? lane >> 1 : lane, half = C::HALVES == 2 ? lane & 1 : 0;
          const int page = __shfl_sync(0xffffffffu, ids, ((jj & 3) * BPAGES + pgi) & 31);
          wait(&empty[slot], phase ^ 1);
          if (dead) return false;
          uint8_t* dst = smem + slot * C::SLOT;
          const bool cut = kv0 == 1 && (rows.x > 0 || rows.y < BK);
          uint64_t* bar = cut ? tail : &full[slot];
          if (lane == 0) mbar_arrive_expect_tx(bar, pages * C::HALVES * 2048);
          __syncwarp();
          if (pgi < pages) tma_load_5d(dst + half * HALF + pgi * 2048, &tmKV, bar, half * 64, 0, kv0, h, page);
          if (cut) {
            // zero the values of keys that are not seen: they may be anything
            wait(tail, tail_phase);
            tail_phase ^= 1;
            for (int r = lane >> 3; r < BK; r += 4)
              if (r < rows.x || r >= rows.y)
#pragma unroll
                for (int hf = 0; hf < C::HALVES; ++hf)
                  *reinterpret_cast<uint4*>(dst + hf * HALF + r * 128 + (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[slot]);
          }
          next();
        }
      } else {
        // A warp takes two pages of the block's eight: 8 lanes (4 with 64 columns)
        // a row, 16 codes each.  K and V have registers of their own, asked for
        // again (for the next block) as soon as their products may start; a lane
        // holds the scale of one of the 32 rows.
        constexpr int LANES = D / 16, RP = kWarp / LANES, NR = kWarp / RP;  // rows a pass, passes
        const int cw = warp - CONV_WARP;
        // this lane's codes [16 ch, + 16) of row sub of a pass: 8 lanes take 64 codes of an even
        // and of an odd row, whose swizzled chunks share no bank when they are stored
        const int ch = D == 128 ? (lane & 3) | ((lane >> 1) & 4) : lane & 3, sub = D == 128 ? ((lane >> 2) & 1) | ((lane >> 3) & 2) : lane >> 2;
        const uint32_t page_bytes = static_cast<uint32_t>(n_kv) * 2 * kPage * D, page_scales = static_cast<uint32_t>(n_kv) * 2 * kPage;
        uint4 w[2][NR];
        uint32_t sc[2];
        const uint8_t* from[2];  // this lane's 16 bytes of the first row of the warp's two pages
        auto ask_rows = [&](int jj, int kv) {  // where block jj's rows are, and their scales
          const int2 rows = seen(jj);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t page = __shfl_sync(0xffffffffu, ids, ((jj & 3) * BPAGES + 2 * cw + y) & 31);
            from[y] = p.c.pool + (unsigned long long)page * page_bytes + ((h * 2 + kv) * kPage + sub) * D + ch * 16;
          }
          const uint32_t page = __shfl_sync(0xffffffffu, ids, ((jj & 3) * BPAGES + 2 * cw + (lane >> 4)) & 31);
          const int r = cw * kWarp + lane;
          sc[kv] = 127;
          if (r >= rows.x && r < rows.y) sc[kv] = p.c.scales[(unsigned long long)page * page_scales + (h * 2 + kv) * kPage + (lane & 15)];
          return rows;
        };
        auto ask = [&](int2 rows, int kv) {
          if (rows.x <= cw * kWarp && rows.y >= (cw + 1) * kWarp) {
#pragma unroll
            for (int i = 0; i < NR; ++i) w[kv][i] = load16(reinterpret_cast<const uint4*>(from[i * RP >> 4] + (i * RP & 15) * D));
          } else {
#pragma unroll
            for (int i = 0; i < NR; ++i) {
              const int r = cw * kWarp + i * RP + sub;
              w[kv][i] = make_uint4(0u, 0u, 0u, 0u);
              if (r >= rows.x && r < rows.y) w[kv][i] = load16(reinterpret_cast<const uint4*>(from[i * RP >> 4] + (i * RP & 15) * D));
            }
          }
        };
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) ask(ask_rows(0, kv), kv);
        for (int jj = 0; jj < n; ++jj) {
          if (((jj + 1) & 3) == 0) {
            ids = ids_next;
            ids_next = fetch(jj + 5);
          }
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            wait(&empty[slot], phase ^ 1);
            if (dead) return false;
            // 2^e in fp16, below its normal range for e = -15
            const uint32_t bits = sc[kv] == 112 ? 0x200u : (sc[kv] - 112) << 10;
            const uint32_t pair = bits | (bits << 16);
            uint8_t* dst = smem + slot * C::SLOT + (ch >> 2) * HALF;
            const int c0 = (ch & 3) * 2;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
              const int r = cw * kWarp + i * RP + sub;
              const uint32_t mb = __shfl_sync(0xffffffffu, pair, i * RP + sub);
              const __half2 m = *reinterpret_cast<const __half2*>(&mb);
              const uint32_t ws[4] = {w[kv][i].x, w[kv][i].y, w[kv][i].z, w[kv][i].w};
              uint32_t o[8];
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const uint32_t c2 = e4m3x2_to_f16x2(ws[x >> 1] >> (16 * (x & 1)));
                const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&c2), m);
                o[x] = *reinterpret_cast<const uint32_t*>(&y);
              }
              uint8_t* row = dst + r * 128;
              *reinterpret_cast<uint4*>(row + ((c0 ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
              *reinterpret_cast<uint4*>(row + (((c0 + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[slot]);
            if (jj + 1 < n) ask(ask_rows(jj + 1, kv), kv);
            next();
          }
        }
      }
      return true;
    });
    // (the products wait for every slot's copies, and the block for the products:
    // no copy is in flight when it ends)
  };
  auto multiply = [&](int t) {
    // ---------------- tile t's products, one thread ----------------
    // S of the next step goes out before the softmax of this one is waited for,
    // into the other of two buffers: the softmax finds its next scores ready,
    // and the tensor cores have work whichever tile is slow
    if (elect_one()) {
      constexpr uint32_t id_s = idesc(C::kCodes, SK, false), id_o = idesc(C::kCodes, D, true);
      const uint32_t d_s = tmem + t * BK, d_o = tmem + C::T_O + t * D;
      const uint32_t ring_k = desc_k(smem_u32(smem)), ring_v = desc_mn(smem_u32(smem)), q_lo = desc_k(smem_u32(smem) + C::OFF_Q + t * C::SLOT);
      int ks = 0, vs = 1;  // slots of the next K and V
      uint32_t kph = 0, vph = 0, qph = 0, n = 0;  // n: steps so far
      bool dead = dead0;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!dead && !bar_wait(bar, parity)) {
          set_status(p.c.status, SDV_ERR_TIMEOUT);
          dead = true;
        }
      };
      auto advance = [&](int& slot, uint32_t& ph) {
        umma_commit(&empty[slot]);
        slot += 2;
        if (slot >= C::NS) {
          slot -= C::NS;
          ph ^= 1;
        }
      };
      walk([&](const SeqRows& s, int, int, const Item& it, int b0, int b1) {
        const Tile t0 = clip(make_tile(s, it, group, window, 0), b0, b1), t1 = clip(make_tile(s, it, group, window, 1), b0, b1);
        const int2 used = both(t0, t1);
        const int first = t ? t1.s0 : t0.s0, last = t ? t1.s1 : t0.s1;
        int kj = used.x, vj = used.x;  // blocks whose K and V are next
        // a block that only the other tile needs is waited for all the same:
        // arriving on a slot's empty barrier a round early would count twice
        auto skip_to = [&](int j) {
          while (kj < j && !dead) {
            wait(&full[ks], kph);
            advance(ks, kph);
            ++kj;
            wait(&full[vs], vph);
            advance(vs, vph);
            ++vj;
          }
        };
        auto scores = [&](int i, uint32_t at) {
          if ((i & 1) == 0 || i == first) wait(&full[ks], kph);
          if (dead) return;
          tc_fence_after();
          const uint32_t kb = ring_k + ks * (C::SLOT >> 4) + (i & 1) * (SK * 128 >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * HALF + (k & 3) * 32) >> 4;
            umma_ss<id_s>(d_s + (at & 1) * SK, q_lo + off, kb + off, k == 0 ? 0u : 1u);
          }
          umma_commit(&s_full[2 * t + (at & 1)]);
          if ((i & 1) || i + 1 == last) {
            advance(ks, kph);
            ++kj;
          }
        };
        if (first < last) {
          skip_to(first >> 1);
          wait(&q_full[t], qph);
          qph ^= 1;
          scores(first, n);
          for (int i = first; i < last && !dead; ++i, ++n) {
            if (i + 1 < last) scores(i + 1, n + 1);
            if ((i & 1) == 0 || i == first) wait(&full[vs], vph);
            wait(&p_full[2 * t + (n & 1)], (n >> 1) & 1);
            if (dead) return false;
            tc_fence_after();
            const uint32_t vb = ring_v + vs * (C::SLOT >> 4) + (i & 1) * (SK * 128 >> 4), pb = d_s + (n & 1) * SK;
            umma_ts<id_o>(d_o, pb, vb, i == first ? 0u : 1u);
#pragma unroll
            for (int k = 1; k < SK / 16; ++k) umma_ts<id_o>(d_o, pb + k * 8, vb + k * (2048 >> 4), 1u);
            umma_commit(&v_done[t]);
            if (i + 1 == last) umma_commit(&o_full[t]);
            if ((i & 1) || i + 1 == last) {
              advance(vs, vph);
              ++vj;
            }
          }
        }
        skip_to(used.y);
        return !dead;
      });
      // every product has ended before the block gives its TMEM back
      umma_commit(done);
      if (!mbar_wait(done, 0)) set_status(p.c.status, SDV_ERR_TIMEOUT);
    }
    __syncwarp();
  };
  auto softmax = [&]() {
    // ---------------- softmax, output: four warps a tile, a thread a row ----------------
    const int t = warp >> 2, i = tid & (BM - 1);
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + t * BK, t_o = tmem + lanes + C::T_O + t * D;
    uint32_t n = 0, oph = 0;  // n: steps so far
    bool dead = dead0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!dead && !bar_wait(bar, parity)) {
        set_status(p.c.status, SDV_ERR_TIMEOUT);
        dead = true;
      }
      __syncwarp();
      tc_fence_after();
    };
    // An item's output is taken from TMEM only after the next item's query is on
    // its way, so that the next scores are made meanwhile.
    bool held = false;
    int turn = 0;
    float m = kNoMax, l = 0.f;
    for (bool more = true;;) {
      Part part;
      if (held) {
        part = s_part[warp];
        more = next_part(part);
      } else {
        more = first_part(part);
      }
      __syncwarp();
      if (lane == 0) s_part[warp] = part;
      __syncwarp();
      if (!more && !held) break;
      const SeqRows& s = part.s;
      const Item& it = part.it;
      Tile x;
      x.s0 = x.s1 = x.rows = 0;
      x.pmin = x.pmax = -1;
      if (more) x = clip(make_tile(s, it, group, window, t), part.b0, part.b1);
      const int row = it.row0 + t * BM + i;
      const bool in_next = i < x.rows;
      float cz = p.scale_log2;
      if (x.s0 < x.s1 && !dead) {
        // this row's query into the tile (its last readers are done: the scores were all seen)
        // the warp's 32 rows, D / 8 lanes a row.  (Short loops here and in the
        // output: this code runs once an item, and unrolled it was fetched
        // anew each time: 9500 cycles an item where this takes 6000.)
        constexpr int QL = D / 8, QR = kWarp / QL;  // lanes a row, rows a pass
        const long long mine = in_next ? (long long)(s.off + row / group) * p.q_stride + (long long)(part.h * group + row % group) * D : -1;
        const int ch = lane % QL, sub = lane / QL;
        uint8_t* q_tile = smem + C::OFF_Q + t * C::SLOT;
#pragma unroll 2
        for (int k = 0; k < QL; ++k) {
          const long long at = __shfl_sync(0xffffffffu, mine, k * QR + sub);
          const int r = (i & ~31) + k * QR + sub;
          cp_async16(q_tile + (ch >> 3) * HALF + r * 128 + (((ch & 7) ^ (r & 7)) << 4), p.q + (at >= 0 ? at + ch * 8 : 0), at >= 0 ? 16 : 0);
        }
        cp_async_wait_all();
        __syncwarp();
        if constexpr (C::kCodes) {
          // each thread its own row: fp16 with the largest magnitude in [1/2, 1)
          __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll 4
          for (int c = 0; c < QL; ++c) {
            const uint4 w = *reinterpret_cast<const uint4*>(q_tile + (c >> 3) * HALF + i * 128 + (((c & 7) ^ (i & 7)) << 4));
            const __nv_bfloat162* v = reinterpret_cast<const __nv_bfloat162*>(&w);
            top = __hmax2(top, __hmax2(__hmax2(__habs2(v[0]), __habs2(v[1])), __hmax2(__habs2(v[2]), __habs2(v[3]))));
          }
          const float a = fmaxf(__low2float(top), __high2float(top));
          const int e = min(max(static_cast<int>(__float_as_uint(a) >> 23) - 126, -100), 100);
          const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
          cz = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll 2
          for (int c = 0; c < QL; ++c) {
            uint4* at = reinterpret_cast<uint4*>(q_tile + (c >> 3) * HALF + i * 128 + (((c & 7) ^ (i & 7)) << 4));
            uint4 w = *at;
            uint32_t* v = &w.x;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const __half2 y = __floats2half2_rn(__uint_as_float(v[x] << 16) * inv, __uint_as_float(v[x] & 0xFFFF0000u) * inv);
              v[x] = *reinterpret_cast<const uint32_t*>(&y);
            }
            *at = w;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[t]);
      }
      if (held) {
        const Held e = s_held[warp];
        const int c_first = e.first, c_last = e.last, e_row = e.row0 + t * BM + i;
        const bool went = e.went != 0, in = t * BM + i < e.rows;
        if (went) {
          wait(&o_full[t], oph);
          oph ^= 1;
          dead = __any_sync(0xffffffffu, dead);
        }
        const int others = c_last - c_first;
        bool join = false, write = in && !dead;
        if (others > 0) {
          // A part: [column][row], then bounds and sums.  Items of few parts are
          // joined here by the last to arrive, whose own part need not leave TMEM
          // (of an item's two parts the one begun earlier ends later as a rule);
          // those of many by chunk_join_kernel, which spreads them over the GPU.
          join = others <= kJoinHere;
          int* count = p.counters + 2 * c_first + t;
          bool last = false;
          if (join && c_first == (int)blockIdx.x) {
            turn ^= 1;
            if (i == 0) {
              s_flag[t][turn] = atomicAdd(count, 0) == others;
              __threadfence();
            }
            named_sync(1 + t, BM);
            last = *reinterpret_cast<volatile int*>(&s_flag[t][turn]) != 0;
          }
          if (!last) {
            float* mine = part_slot(p.part, D, blockIdx.x, c_first, t);
            if (went && !dead) {
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t r[32];
                tmem_ld32(t_o + 32 * c, r);
                tmem_wait_ld(r);
#pragma unroll
                for (int k = 0; k < 32; ++k) mine[(32 * c + k) * BM + i] = __uint_as_float(r[k]);
              }
            }
            mine[D * BM + i] = m;
            mine[(D + 1) * BM + i] = l;
            if (join) {
              turn ^= 1;
              __threadfence();
              named_sync(1 + t, BM);
              if (i == 0) {
                s_flag[t][turn] = atomicAdd(count, 1) == others;
                __threadfence();
              }
              named_sync(1 + t, BM);
              last = *reinterpret_cast<volatile int*>(&s_flag[t][turn]) != 0;
            }
          }
          if (last && i == 0) *count = 0;
          write = write && last;
        }
        // this part's share of the row, and the others'
        float f[kJoinHere + 1];
        if (join && write) {
          float mk[kJoinHere + 1], lk[kJoinHere + 1], top = kNoMax;
#pragma unroll
          for (int k = 0; k <= kJoinHere; ++k) {
            mk[k] = kNoMax;
            lk[k] = 0.f;
            if (k <= others) {
              const float* src = part_slot(p.part, D, c_first + k, c_first, t);
              const bool me = c_first + k == (int)blockIdx.x;
              mk[k] = me ? m : __ldcg(src + D * BM + i);
              lk[k] = me ? l : __ldcg(src + (D + 1) * BM + i);
            }
          }
#pragma unroll
          for (int k = 0; k <= kJoinHere; ++k) top = fmaxf(top, mk[k]);
          l = 0.f;
#pragma unroll
          for (int k = 0; k <= kJoinHere; ++k) {
            f[k] = lk[k] == 0.f ? 0.f : fast_ex2(mk[k] - top);
            l += f[k] * lk[k];
          }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees nothing gives 0
        const long long out_at = write ? (long long)(e.off + e_row / group) * p.out_stride + (long long)(e.h * group + e_row % group) * D : -1;
        if (others == 0 || __any_sync(0xffffffffu, join && write)) {
          // unrolled, the other parts' loads overlap (six prompts, bf16: 84 us against 88); over codes the
          // longer code costs more than that (107 against 101)
#pragma unroll(C::kCodes ? 1 : D / 32)
          for (int c = 0; c < D / 32; ++c) {
            uint32_t r[32];
            if (went && !dead) {
              tmem_ld32(t_o + 32 * c, r);
              tmem_wait_ld(r);
            } else {
#pragma unroll
              for (int k = 0; k < 32; ++k) r[k] = 0;
            }
            if (join && write) {
              float acc[32];
#pragma unroll
              for (int x = 0; x < 32; ++x) acc[x] = 0.f;
#pragma unroll
              for (int k = 0; k <= kJoinHere; ++k)
                if (k <= others && f[k] != 0.f) {  // (a part that saw nothing wrote no columns)
                  if (c_first + k == (int)blockIdx.x) {
#pragma unroll
                    for (int x = 0; x < 32; ++x) acc[x] += f[k] * __uint_as_float(r[x]);
                  } else {
                    const float* src = part_slot(p.part, D, c_first + k, c_first, t) + 32 * c * BM + i;
#pragma unroll
                    for (int x = 0; x < 32; ++x) acc[x] += f[k] * __ldcg(src + x * BM);
                  }
                }
#pragma unroll
              for (int x = 0; x < 32; ++x) r[x] = __float_as_uint(acc[x]);
            }
            // the 32 columns as four pieces of 16 bytes; four lanes trade theirs, so
            // that they store one row's 64 bytes together
            uint32_t o[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int y = 0; y < 4; ++y)
                o[k][y] = l == 0.f ? 0u : pack_bf16x2(__uint_as_float(r[8 * k + 2 * y]) * inv, __uint_as_float(r[8 * k + 2 * y + 1]) * inv);
#pragma unroll
            for (int bit = 1; bit <= 2; bit <<= 1) {
              const bool up = lane & bit;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (k & bit) continue;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  const uint32_t give = up ? o[k][y] : o[k | bit][y];
                  const uint32_t got = __shfl_xor_sync(0xffffffffu, give, bit);
                  if (up) o[k][y] = got;
                  else o[k | bit][y] = got;
                }
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // o[k] is piece lane % 4 of row lane & ~3 + k
              const long long at = __shfl_sync(0xffffffffu, out_at, (lane & ~3) + k);
              if (at >= 0) *reinterpret_cast<uint4*>(p.out + at + 32 * c + (lane & 3) * 8) = make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
            }
          }
        }
        tc_fence_before();
      }
      if (!more) break;
      {
        const long long ua = part.u0 + kItemCost, ub = ua + (long long)(it.blocks - 1) * weight(it);  // the first and last block's units
        const int c_first = ua >= u_begin ? (int)blockIdx.x : static_cast<int>(ua / per_cta);
        const int c_last = ub < u_end ? (int)blockIdx.x : static_cast<int>(ub / per_cta);
        __syncwarp();
        if (lane == 0) s_held[warp] = Held{s.off, part.h, it.row0, it.rows, c_first, c_last, x.s0 < x.s1};
        if (tid == 0 && c_last - c_first > kJoinHere && c_first == (int)blockIdx.x) {
          p.cuts[2 * blockIdx.x] = make_int4(c_last, s.off, part.h, it.row0);
          p.cuts[2 * blockIdx.x + 1].x = it.rows;
        }
        __syncwarp();
      }
      m = kNoMax;
      l = 0.f;
      // step j holds the keys from key_base + 64 j; steps [cut_lo, cut_hi) are seen whole by every row
      const int key_base = it.page_lo * kPage, rel_base = (in_next ? s.pos0 + row / group : -1) - key_base;
      const int cut_hi = (x.pmin - key_base + 1) >> 6;
      const int cut_lo = window > 0 ? ((x.pmax - window - key_base) >> 6) + 1 : 0;
      for (int j = x.s0; j < x.s1; ++j, ++n) {
        wait(&s_full[2 * t + (n & 1)], (n >> 1) & 1);
        const uint32_t t_sb = t_s + (n & 1) * SK;
        const int rel = rel_base - j * SK;  // column c is seen when c <= rel and c > rel - window
        uint32_t buf[2][32];
        if (j >= cut_hi || j < cut_lo) {
          // hide what is not seen, in TMEM, so that what follows is one code for all steps
#pragma unroll
          for (int c = 0; c < SK / 32; ++c) {
            tmem_ld32(t_sb + 32 * c, buf[0]);
            tmem_wait_ld(buf[0]);
            // bit e of `see`: column 32 c + e is seen
            const int hi = rel - 32 * c, lo = window > 0 ? hi - window : -1;
            uint32_t see = hi < 0 ? 0u : hi >= 31 ? 0xFFFFFFFFu : (2u << hi) - 1u;
            if (lo >= 0) see &= lo >= 31 ? 0u : 0xFFFFFFFFu << (lo + 1);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((see >> e) & 1u)) buf[0][e] = 0xFF800000u;
            tmem_st32(t_sb + 32 * c, buf[0]);
          }
          tmem_wait_st();
        }
        auto row_top = [&]() {  // the step's largest logit
          float v = -INFINITY;
#pragma unroll
          for (int c = 0; c < SK / 32; ++c) {
            tmem_ld32(t_sb + 32 * c, buf[0]);
            tmem_wait_ld(buf[0]);
#pragma unroll
            for (int k = 0; k < 32; k += 2) v = fmaxf(v, fmaxf(__uint_as_float(buf[0][k]), __uint_as_float(buf[0][k + 1])));
          }
          return v * cz;
        };
        constexpr float above = C::kCodes ? kAbove : 0.f;
        if (j == x.s0) m = fmaxf(kNoMax, row_top() - above);  // the first step sets the bound
        uint32_t pw[SK / 2];
        for (int again = 0;; ++again) {
          uint64_t sum[2] = {0, 0};
          const uint64_t cc = f2(cz, cz), mm = f2(-m, -m);
          tmem_ld32(t_sb, buf[0]);
#pragma unroll
          for (int c = 0; c < SK / 32; ++c) {
            tmem_wait_ld(buf[c & 1]);
            if (c + 1 < SK / 32) tmem_ld32(t_sb + 32 * (c + 1), buf[(c + 1) & 1]);
            uint32_t (&r)[32] = buf[c & 1];
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              float a, b;
              unf2(fma2(f2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), cc, mm), a, b);
              a = fast_ex2(a);
              b = fast_ex2(b);
              sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], f2(a, b));
              if constexpr (C::kCodes) {
                const __half2 y = __floats2half2_rn(a, b);
                pw[c * 16 + (k >> 1)] = *reinterpret_cast<const uint32_t*>(&y);
              } else {
                pw[c * 16 + (k >> 1)] = pack_bf16x2(a, b);
              }
            }
          }
          float total, other;
          unf2(add2(sum[0], sum[1]), total, other);
          total += other;
          bool move = !(total <= (C::kCodes ? kMostCodes : kMost));
          if constexpr (C::kCodes) move |= total < kLeast && total > 0.f && l <= kSumMost;
          // (a wait that has run out is voted on here too, so that the warp stays one)
          if (!__any_sync(0xffffffffu, (!again && move) || dead)) {
            l += total;
            break;
          }
          dead = __any_sync(0xffffffffu, dead);
          if (dead) break;
          // a row's weights have left what its bound allows (or are not
          // numbers): move the bounds and take the step again
          const float top = row_top() - above;
          float mn = fmaxf(m, top);
          if constexpr (C::kCodes)
            if (move && top < m) mn = fmaxf(top, m - kDropMost);
          const float f = fast_ex2(m - mn);
          m = mn;
          l *= f;
          if (j > x.s0) {
            // the step before has been added (all before it had when these scores were made)
            wait(&v_done[t], (n - 1) & 1);
            const uint64_t ff = f2(f, f);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              tmem_ld32(t_o + 32 * c, buf[0]);
              tmem_wait_ld(buf[0]);
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                float a, b;
                unf2(mul2(f2(__uint_as_float(buf[0][k]), __uint_as_float(buf[0][k + 1])), ff), a, b);
                buf[0][k] = __float_as_uint(a);
                buf[0][k + 1] = __float_as_uint(b);
              }
              tmem_st32(t_o + 32 * c, buf[0]);
            }
            tmem_wait_st();
          }
        }
        if (dead) break;
        tmem_st32(t_sb, pw);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * t + (n & 1)]);
      }
      held = true;
    }
  };
  // a warpgroup changes its registers as one
  if (warp >= CONV_WARP) {
    regs_down<C::R_CONV>();
    if constexpr (C::kCodes) load(0);
  } else if (warp >= MMA_WARP) {
    regs_down<C::R_ISSUE>();
    if (warp < MMA_WARP + 2) multiply(warp - MMA_WARP);
    if constexpr (!C::kCodes)
      if (warp >= TMA_WARP) load(warp - TMA_WARP);
  } else {
    regs_up<C::R_SOFT>();
    softmax();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// Joins the items of many parts (few rows over many keys: up to a part of 128 KB
// on every SM): block (c, y) takes 16 columns of one tile of the item that
// begins in run c, a thread a row, parts in order, four parts' loads in flight.
template <int D>
__global__ void __launch_bounds__(BM) chunk_join_kernel(const ChunkAttnParams p) {
  constexpr int COLS = 16;
  griddep_launch_dependents();
  griddep_wait();
  const int c = blockIdx.x, t = blockIdx.y & 1, col = (blockIdx.y >> 1) * COLS, i = threadIdx.x;
  const int4 cut = p.cuts[2 * c];
  if (cut.x < 0 || read_status(p.c.status) != 0) return;
  const int rows = p.cuts[2 * c + 1].x - t * BM, last = cut.x;
  if (i >= rows) return;
  const int group = p.c.n_q / p.c.n_kv, row = cut.w + t * BM + i;
  float m = kNoMax;
#pragma unroll 8
  for (int k = c; k <= last; ++k) m = fmaxf(m, part_slot(p.part, D, k, c, t)[D * BM + i]);
  float l = 0.f, acc[COLS];
#pragma unroll
  for (int x = 0; x < COLS; ++x) acc[x] = 0.f;
#pragma unroll 4
  for (int k = c; k <= last; ++k) {
    const float* src = part_slot(p.part, D, k, c, t);
    const float lk = src[(D + 1) * BM + i], f = fast_ex2(src[D * BM + i] - m);
    const bool any = lk != 0.f;  // else it saw nothing and wrote no columns
    l += any ? f * lk : 0.f;
#pragma unroll
    for (int x = 0; x < COLS; ++x) {
      const float v = src[(col + x) * BM + i];
      acc[x] += any ? f * v : 0.f;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __nv_bfloat16* dst = p.out + (long long)(cut.y + row / group) * p.out_stride + (long long)(cut.z * group + row % group) * D + col;
#pragma unroll
  for (int x = 0; x < COLS; x += 8)
    *reinterpret_cast<uint4*>(dst + x) =
        make_uint4(pack_bf16x2(acc[x] * inv, acc[x + 1] * inv), pack_bf16x2(acc[x + 2] * inv, acc[x + 3] * inv),
                   pack_bf16x2(acc[x + 4] * inv, acc[x + 5] * inv), pack_bf16x2(acc[x + 6] * inv, acc[x + 7] * inv));
}

template <int D, int FMT>
cudaError_t launch_one(const CUtensorMap& map, const ChunkAttnParams& p, int grid, cudaStream_t stream) {
  const cudaError_t e = launch_pdl(chunk_attn_tc_kernel<D, FMT>, dim3(grid), dim3(Cfg<D, FMT>::THREADS), Cfg<D, FMT>::SMEM, stream, map, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(chunk_join_kernel<D>, dim3(grid, 2 * D / 16), dim3(BM), 0, stream, p);
}

template <int D, int FMT>
cudaError_t setup_one() {
  return cudaFuncSetAttribute(chunk_attn_tc_kernel<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, FMT>::SMEM);
}

}  // namespace

size_t chunk_attn_tc_part_floats(int head_dim, int grid) { return static_cast<size_t>(grid) * 4 * BM * (head_dim + 2); }

cudaError_t setup_chunk_attn_tc(int head_dim, int cache_format) {
  if (head_dim == 64)
    return cache_format == SDV_CACHE_BF16 ? setup_one<64, SDV_CACHE_BF16>() : setup_one<64, SDV_CACHE_E4M3>();
  return cache_format == SDV_CACHE_BF16 ? setup_one<128, SDV_CACHE_BF16>() : setup_one<128, SDV_CACHE_E4M3>();
}

cudaError_t launch_chunk_attn_tc(int head_dim, int cache_format, const CUtensorMap& map, const ChunkAttnParams& p, int grid,
                                 cudaStream_t stream) {
  if (head_dim == 64)
    return cache_format == SDV_CACHE_BF16 ? launch_one<64, SDV_CACHE_BF16>(map, p, grid, stream)
                                          : launch_one<64, SDV_CACHE_E4M3>(map, p, grid, stream);
  return cache_format == SDV_CACHE_BF16 ? launch_one<128, SDV_CACHE_BF16>(map, p, grid, stream)
                                        : launch_one<128, SDV_CACHE_E4M3>(map, p, grid, stream);
}

}  // namespace sdv
