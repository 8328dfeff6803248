// The paged cache's tables of a step, made from the requests' lengths (sdv_cache_plan).
//
// Exclusive sums over the requests give the row offsets and the place of every
// page that moves: page i of those pushed goes to free[top + i], page i of those popped comes from
// free[top + pushed - 1 - i], so both lists move in parallel and the outcome is
// that of one request after another.
//
// A few bytes, so all latency: launch, the lengths, three sums, the moved pages, the rows, one after another.  One request 4.9 us, 64
// requests with 2800 rows and 3900 moved pages 7.0 us, 1024 with 18900 and 37000 12.9 us (one block alone: 9.2 and 41 us).
#include <cooperative_groups.h>

#include "chunk.cuh"

namespace cg = cooperative_groups;

namespace sdv {
namespace {

constexpr int TAB_THREADS = 1024;
static_assert(TAB_THREADS >= kMaxChunkSlots, "a thread takes a request");

// Exclusive sums of a, b and c over the block's threads, in place; totals in tot.
__device__ __forceinline__ void block_sums(long long (&v)[3], long long (&tot)[3], long long (*s_warp)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long own[3];
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    own[j] = v[j];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xFFFFFFFFu, v[j], o);
      if (lane >= o) v[j] += y;
    }
    if (lane == 31) s_warp[warp][j] = v[j];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    long long before = 0, all = lane < TAB_THREADS / 32 ? s_warp[lane][j] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xFFFFFFFFu, all, o);
      if (lane >= o) all += y;
    }
    before = __shfl_sync(0xFFFFFFFFu, all, warp > 0 ? warp - 1 : 0);
    tot[j] = __shfl_sync(0xFFFFFFFFu, all, 31);
    v[j] += (warp > 0 ? before : 0) - own[j];
  }
}

// The request that owns item i of offsets s [B + 1]: the last b with s[b] <= i.
template <typename I>
__device__ __forceinline__ int owner(const I* s, int B, I i) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// One cluster: its first block gives the verdict, all of them move pages and write rows.  Every block makes the
// offsets by itself, from inputs that are written only after all have read them.
__global__ void __launch_bounds__(TAB_THREADS) cache_plan_kernel(const sdv_cache_tables p, int* status) {
  __shared__ long long s_warp[TAB_THREADS / 32][3];
  __shared__ int s_off[kMaxChunkSlots + 1];
  __shared__ long long s_back[kMaxChunkSlots], s_want[kMaxChunkSlots];
  __shared__ int s_first[kMaxChunkSlots];  // first block that moves
  __shared__ int s_len[kMaxChunkSlots];
  __shared__ int s_verdict;
  cg::cluster_group cluster = cg::this_cluster();
  const int t = threadIdx.x, rank = cluster.block_rank(), blocks = cluster.num_blocks();
  griddep_launch_dependents();
  griddep_wait();
  const bool mine = t < p.B;
  const int n = mine ? p.new_rows[t] : 0, len = mine ? p.lens[t] : 0, count = mine ? p.page_counts[t] : 0;
  const int need = (len >> 4) + ((len & 15) != 0), top = *p.num_free;
  int err = 0;
  if (n < 0 || len < 0 || count < 0 || count > p.max_pages_per_seq || top < 0 || top > p.num_pool_pages) err = 1;
  else if (need > p.max_pages_per_seq) err = 2;
  long long v[3] = {n, count > need ? count - need : 0, need > count ? need - count : 0}, tot[3];
  block_sums(v, tot, s_warp);
  if (mine) {
    s_off[t] = static_cast<int>(v[0]);  // (of sums past 32 bits nothing is used)
    s_back[t] = v[1];
    s_want[t] = v[2];
    s_first[t] = min(need, count);
    s_len[t] = len;
  }
  if (t == 0) s_off[p.B] = static_cast<int>(tot[0]);
  const bool bad = __syncthreads_or(err == 1), wide = __syncthreads_or(err == 2);
  const long long have = top + tot[1];
  if (rank == 0 && t == 0) {
    const int found = bad || tot[0] > p.T || have > p.num_pool_pages ? SDV_ERR_BAD_INPUT
                      : wide || tot[2] > have                       ? SDV_ERR_CAPACITY
                                                                    : 0;
    const int before = read_status(status);
    s_verdict = before ? before : found;
    if (found) set_status(status, found);
  }
  cluster.sync();  // every block has its inputs; the verdict
  const int verdict = *cluster.map_shared_rank(&s_verdict, 0), lane0 = rank * TAB_THREADS + t;
  if (verdict == 0) {
    bool out = false;
    for (long long i = lane0; i < tot[1]; i += blocks * TAB_THREADS) {
      const int b = owner(s_back, p.B, i);
      int* entry = p.page_table + (long long)b * p.max_pages_per_seq + s_first[b] + (i - s_back[b]);
      const int page = *entry;
      out |= page < 0 || page >= p.num_pool_pages;
      p.free_pages[top + i] = page;
      *entry = -1;
    }
    if (rank == 0 && mine) {
      p.page_counts[t] = need;
      p.row_offsets[t] = s_off[t];
      if (p.last_rows) p.last_rows[t] = n > 0 ? s_off[t] + n - 1 : -1;
    }
    if (rank == 0 && t >= p.B && t < p.max_B) {
      p.row_offsets[t + 1] = s_off[p.B];
      if (p.last_rows) p.last_rows[t] = -1;
    }
    if (rank == 0 && t == 0) {
      p.row_offsets[p.B] = s_off[p.B];
      *p.num_free = static_cast<int>(have - tot[2]);
    }
    if (out) set_status(status, SDV_ERR_PAGE_RANGE);
  }
  if (tot[1] && tot[2]) cluster.sync();  // pushed pages may be popped (every block has the same sums)
  if (verdict == 0) {
    bool out = false;
    for (long long i = lane0; i < tot[2]; i += blocks * TAB_THREADS) {
      const int b = owner(s_want, p.B, i);
      const int page = __ldcg(p.free_pages + have - 1 - i);
      out |= page < 0 || page >= p.num_pool_pages;
      p.page_table[(long long)b * p.max_pages_per_seq + s_first[b] + (i - s_want[b])] = page;
    }
    if (out) set_status(status, SDV_ERR_PAGE_RANGE);
  }
  cluster.sync();  // the moved pages are in their places; the first block's shared memory has been read
  if (verdict != 0) return;
  const int rows = s_off[p.B];
  for (int r = lane0; r < p.T; r += blocks * TAB_THREADS) {
    int b = -1, pos = -1;
    long long slot = -1;
    if (r < rows) {
      b = owner(s_off, p.B, r);
      pos = s_len[b] - s_off[b + 1] + r;
      if (pos >= 0 && p.slots) {
        const int page = __ldcg(p.page_table + (long long)b * p.max_pages_per_seq + (pos >> 4));
        if (page >= 0 && page < p.num_pool_pages) slot = (long long)page * kPage + (pos & 15);
        else set_status(status, SDV_ERR_PAGE_RANGE);
      }
    }
    if (p.row_request) p.row_request[r] = b;
    if (p.positions) p.positions[r] = pos;
    if (p.slots) p.slots[r] = slot;
  }
}

// Requests and rows up to which one block does it: a cluster of 8 takes about a microsecond to begin and to meet.
constexpr int kPlanSlots = 16, kPlanRows = 1024;

}  // namespace

cudaError_t launch_cache_plan(const sdv_cache_tables& p, int* status, cudaStream_t stream) {
  const int blocks = p.B <= kPlanSlots && p.T <= kPlanRows ? 1 : 8;
  return launch_pdl_cluster(cache_plan_kernel, blocks, dim3(blocks), dim3(TAB_THREADS), 0, stream, p, status);
}

}  // namespace sdv

using namespace sdv;

extern "C" sdv_status sdv_cache_plan(const sdv_cache_tables* p, int* status, void* stream) {
  if (!p || !status) return SDV_ERR_INVALID_ARG;
  if (p->B <= 0 || p->T < 0 || p->T > (1 << 30) || p->max_pages_per_seq <= 0 || p->max_pages_per_seq > (1 << 26) || p->num_pool_pages <= 0)
    return SDV_ERR_INVALID_ARG;
  if (!p->new_rows || !p->lens || !p->page_table || !p->page_counts || !p->free_pages || !p->num_free || !p->row_offsets)
    return SDV_ERR_INVALID_ARG;
  if (p->max_B < 0 || (p->max_B > 0 && p->max_B < p->B)) return SDV_ERR_INVALID_ARG;
  if (p->B > kMaxChunkSlots || p->max_B > kMaxChunkSlots) return SDV_ERR_CAPACITY;
  const cudaError_t e = launch_cache_plan(*p, status, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SDV_OK : cuda_fail(e);
}
