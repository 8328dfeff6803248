// C ABI of the paged cache's operators (include/sdv_cache.h): argument checks,
// the handle and the launches.
#include <cmath>
#include <cstring>
#include <new>

#include "chunk.cuh"

struct sdv_cache {
  sdv_cache_config cfg;
  int device, sms, max_rows, max_slots;
  float *part, *part_tc;
  int *counters, *counters_tc;
  int4* cuts;
  sdv::RopeTurns turns;
};

namespace sdv {
namespace {

bool config_ok(const sdv_cache_config* c) {
  if (!c || c->n_q <= 0 || c->n_kv <= 0 || c->n_q % c->n_kv || c->n_q > 65536) return false;
  if (c->page_size != kPage) return false;
  if (c->cache_format != SDV_CACHE_BF16 && c->cache_format != SDV_CACHE_E4M3) return false;
  return c->rope_theta == 0.f || (c->rope_theta >= 1.f && std::isfinite(c->rope_theta));
}
bool shape_ok(const sdv_cache_config* c) { return c->head_dim == 64 || c->head_dim == 128; }

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

int sms_of(int dev) {
  int n = 0;
  return cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? n : 0;
}

// Packed rows (tokens times heads of a group) of a sequence up to which the
// mma.sync kernel takes it: one of its 16-row items.
constexpr int kSmallRows = 16;

// Whether the sequences of few rows of a step that also brings longer ones go to
// the mma.sync kernel, behind the tcgen05 kernel, or stay with it.  A second
// launch costs 15 to 20 us; a next token costs the tcgen05 kernel an item's start and
// end, and more per key the fewer bytes a key has.  So: where at least half of the sequences
// must be short, and there are enough (sequence, key head)s for it.  One against
// both kernels, 2 pieces of 300 rows and B - 2 next tokens over 600 to 6000 positions, 8 key heads unless said, us:
//   keys of 256 bytes  B 32 105 : 126, 128 328 : 353; over 60 to 600, 2 heads, 256 65 : 68, 1000 198 : 137
//   128 (codes)        B 16 81 : 85, 20 86 : 86, 24 111 : 101, 64 191 : 140; 4 heads, 40 75 : 84, 64 109 : 95; 1 head, 160 76 : 92, 320 131 : 111
//   128 (bf16)         B 16 65 : 70, 20 65 : 65, 24 81 : 78, 64 150 : 120
//   64                 B 8 62 : 65, 12 53 : 54, 20 67 : 57, 64 153 : 92; 2 heads, 40 37 : 48, 80 59 : 59
// and by the share of pieces, codes of 128 bytes: 8 of 24 166 : 161, 31 of 64 557 : 527, 16 of 24 257 : 262.
bool two_kernels(const sdv_cache* h, const sdv_chunk* c) {
  const int key_bytes = h->cfg.head_dim * (h->cfg.cache_format == SDV_CACHE_E4M3 ? 1 : 2);
  if (h->cfg.n_q / h->cfg.n_kv > kSmallRows) return false;  // a single token has too many rows for it
  const int per_sm_x4 = key_bytes <= 64 ? 4 : key_bytes <= 128 ? 5 : 32;
  return 4LL * c->B * h->cfg.n_kv >= (long long)per_sm_x4 * h->sms && c->T <= (long long)c->B * c->max_q / 2;
}

struct Space {
  size_t counters, counters_tc, cuts, part, part_tc, total;
};
Space space(const sdv_cache_config& c, int sms) {
  Space s{};
  s.counters = 0;
  s.counters_tc = up256(chunk_attn_grid_max(sms) * sizeof(int));
  s.cuts = s.counters_tc + up256(2 * sms * sizeof(int));
  s.part = s.cuts + up256(2 * sms * sizeof(int4));
  s.part_tc = s.part + up256(chunk_attn_part_floats(c.head_dim, sms) * sizeof(float));
  s.total = s.part_tc + up256(chunk_attn_tc_part_floats(c.head_dim, sms) * sizeof(float));
  return s;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// row pointers: 16-byte aligned, rows long enough for their heads
sdv_status rows_ok(const void* p, long long stride, long long width, int bytes) {
  if (!p || stride < width || !aligned16(p) || (stride * bytes) % 16) return SDV_ERR_INVALID_ARG;
  return SDV_OK;
}

// Checks a call's common arguments and fills the device's view of the chunk.
sdv_status chunk_params(const sdv_cache* h, const sdv_chunk* c, int* status, ChunkParams* p) {
  if (!h || !c || !status) return SDV_ERR_INVALID_ARG;
  if (c->B <= 0 || c->T < 0 || c->max_q < 0 || c->window < 0 || c->num_pool_pages <= 0 || c->max_pages_per_seq <= 0)
    return SDV_ERR_INVALID_ARG;
  if (c->max_pages_per_seq > (1 << 26)) return SDV_ERR_INVALID_ARG;  // positions below 2^30
  if (!c->row_offsets || !c->kv_lens || !c->kv_pool || !c->page_table || !aligned16(c->kv_pool)) return SDV_ERR_INVALID_ARG;
  if (h->cfg.cache_format == SDV_CACHE_E4M3 && (!c->kv_scales || !aligned16(c->kv_scales))) return SDV_ERR_INVALID_ARG;
  if (c->B > h->max_slots || c->T > h->max_rows) return SDV_ERR_CAPACITY;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != h->device) return SDV_ERR_INVALID_ARG;
  p->B = c->B;
  p->T = c->T;
  p->max_q = c->max_q;
  p->window = c->window < (1 << 30) ? c->window : 0;  // positions end before 2^30: a window as long sees all
  p->row_offsets = c->row_offsets;
  p->kv_lens = c->kv_lens;
  p->pool = static_cast<uint8_t*>(c->kv_pool);
  p->scales = static_cast<uint8_t*>(c->kv_scales);
  p->page_table = c->page_table;
  p->pool_pages = c->num_pool_pages;
  p->max_pages = c->max_pages_per_seq;
  p->n_q = h->cfg.n_q;
  p->n_kv = h->cfg.n_kv;
  p->status = status;
  return SDV_OK;
}

sdv_status launched(cudaError_t e) { return e == cudaSuccess ? SDV_OK : cuda_fail(e); }

}  // namespace
}  // namespace sdv

using namespace sdv;

extern "C" size_t sdv_cache_workspace_size(const sdv_cache_config* cfg, int max_rows, int max_slots) {
  if (!config_ok(cfg) || !shape_ok(cfg) || max_rows <= 0 || max_slots <= 0 || max_slots > kMaxChunkSlots) return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return space(*cfg, sms_of(dev)).total;
}

extern "C" sdv_status sdv_cache_create(const sdv_cache_config* cfg, void* workspace, size_t workspace_bytes, int max_rows,
                                       int max_slots, void* stream, sdv_cache** out) {
  if (!out) return SDV_ERR_INVALID_ARG;
  *out = nullptr;
  if (!config_ok(cfg) || !workspace || max_rows <= 0 || max_slots <= 0 || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return SDV_ERR_INVALID_ARG;
  if (!shape_ok(cfg)) return SDV_ERR_UNSUPPORTED;
  if (max_slots > kMaxChunkSlots || (long long)max_rows * cfg->n_q > 0x3FFFFFFFLL) return SDV_ERR_CAPACITY;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  const int sms = sms_of(dev);
  const Space s = space(*cfg, sms);
  if (workspace_bytes < s.total) return SDV_ERR_CAPACITY;
  e = setup_chunk_attn(cfg->head_dim, cfg->cache_format);
  if (e == cudaSuccess) e = setup_chunk_attn_tc(cfg->head_dim, cfg->cache_format);
  if (e != cudaSuccess) return cuda_fail(e);
  sdv_cache* h = new (std::nothrow) sdv_cache;
  if (!h) return SDV_ERR_INTERNAL;
  h->cfg = *cfg;
  h->device = dev;
  h->sms = sms;
  h->max_rows = max_rows;
  h->max_slots = max_slots;
  h->counters = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + s.counters);
  h->counters_tc = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + s.counters_tc);
  h->cuts = reinterpret_cast<int4*>(static_cast<uint8_t*>(workspace) + s.cuts);
  h->part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + s.part);
  h->part_tc = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + s.part_tc);
  for (int j = 0; j < 64; ++j) {
    h->turns.f[j] = 0;
    if (cfg->rope_theta > 0.f && j < cfg->head_dim / 2) {
      // theta^(-2j/d) <= 1, so at most 0.16 of a turn
      const double turn = std::pow(static_cast<double>(cfg->rope_theta), -2.0 * j / cfg->head_dim) / (2.0 * 3.14159265358979323846);
      h->turns.f[j] = static_cast<unsigned long long>(std::ldexp(turn, 64));
    }
  }
  // cleared before the call returns, so that the first calls may come on any stream
  e = cudaMemsetAsync(h->counters, 0, s.part, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    delete h;
    return cuda_fail(e);
  }
  *out = h;
  return SDV_OK;
}

extern "C" void sdv_cache_destroy(sdv_cache* h) { delete h; }

extern "C" sdv_status sdv_cache_append(sdv_cache* h, const sdv_chunk* chunk, const sdv_append_rows* rows, int* status,
                                       void* stream) {
  AppendParams p;
  sdv_status rc = chunk_params(h, chunk, status, &p.c);
  if (rc != SDV_OK) return rc;
  if (!rows || (rows->x_format != 0 && rows->x_format != 1)) return SDV_ERR_INVALID_ARG;
  if (chunk->T == 0) return SDV_OK;  // no rows: their pointers may be null
  const int bytes = rows->x_format ? 4 : 2, d = h->cfg.head_dim;
  const long long kw = (long long)h->cfg.n_kv * d, qw = (long long)h->cfg.n_q * d;
  if ((rc = rows_ok(rows->k, rows->k_stride, kw, bytes)) != SDV_OK) return rc;
  if ((rc = rows_ok(rows->v, rows->v_stride, kw, bytes)) != SDV_OK) return rc;
  if ((rows->q == nullptr) != (rows->q_out == nullptr)) return SDV_ERR_INVALID_ARG;
  if (rows->q) {
    if ((rc = rows_ok(rows->q, rows->q_stride, qw, bytes)) != SDV_OK) return rc;
    if ((rc = rows_ok(rows->q_out, rows->q_out_stride, qw, 2)) != SDV_OK) return rc;
  }
  p.k = rows->k;
  p.v = rows->v;
  p.q = rows->q;
  p.k_stride = rows->k_stride;
  p.v_stride = rows->v_stride;
  p.q_stride = rows->q_stride;
  p.q_out = rows->q_out;
  p.q_out_stride = rows->q_out_stride;
  p.rope = h->cfg.rope_theta > 0.f;
  return launched(launch_cache_append(d, h->cfg.cache_format, rows->x_format, p, h->turns, h->sms, static_cast<cudaStream_t>(stream)));
}

extern "C" sdv_status sdv_cache_attention(sdv_cache* h, const sdv_chunk* chunk, const void* q, long long q_stride, void* out,
                                          long long out_stride, int* status, void* stream) {
  ChunkAttnParams p;
  sdv_status rc = chunk_params(h, chunk, status, &p.c);
  if (rc != SDV_OK || chunk->T == 0) return rc;
  const int d = h->cfg.head_dim;
  const long long qw = (long long)h->cfg.n_q * d;
  if ((rc = rows_ok(q, q_stride, qw, 2)) != SDV_OK) return rc;
  if ((rc = rows_ok(out, out_stride, qw, 2)) != SDV_OK) return rc;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.scale_log2 = kLog2e / std::sqrt(static_cast<float>(d));
  p.small_rows = 0x7FFFFFFF;
  const int group = h->cfg.n_q / h->cfg.n_kv;
  const long long rows = (long long)(chunk->max_q < chunk->T ? chunk->max_q : chunk->T) * group;  // of a sequence at most
  if (rows > kSmallRows) {
    const bool two = two_kernels(h, chunk);
    p.small_rows = two ? kSmallRows : 0;
    p.part = h->part_tc;
    p.cuts = h->cuts;
    p.counters = h->counters_tc;
    CUtensorMap map;
    if (h->cfg.cache_format == SDV_CACHE_BF16) {
      if (!encode_kv_map(&map, chunk->kv_pool, h->cfg.n_kv, d, chunk->num_pool_pages)) return SDV_ERR_CUDA;
    } else {
      std::memset(&map, 0, sizeof(map));  // the codes are not loaded through it
    }
    const cudaError_t e = launch_chunk_attn_tc(d, h->cfg.cache_format, map, p, h->sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e);
    if (!two) return SDV_OK;
    // (mostly single tokens: items of 8 rows, two for a sequence of up to 16)
    p.part = h->part;
    p.counters = h->counters;
    return launched(launch_chunk_attn(d, h->cfg.cache_format, group <= 8, p, h->sms, static_cast<cudaStream_t>(stream)));
  }
  p.part = h->part;
  p.counters = h->counters;
  return launched(launch_chunk_attn(d, h->cfg.cache_format, rows <= 8, p, h->sms, static_cast<cudaStream_t>(stream)));
}

extern "C" sdv_status sdv_cache_read(sdv_cache* h, const sdv_chunk* chunk, void* k_out, long long k_stride, void* v_out,
                                     long long v_stride, int out_format, int* status, void* stream) {
  ReadParams p;
  sdv_status rc = chunk_params(h, chunk, status, &p.c);
  if (rc != SDV_OK) return rc;
  if (out_format != 0 && out_format != 1) return SDV_ERR_INVALID_ARG;
  if (chunk->T == 0) return SDV_OK;
  const int bytes = out_format ? 4 : 2;
  const long long kw = (long long)h->cfg.n_kv * h->cfg.head_dim;
  if (!k_out && !v_out) return SDV_ERR_INVALID_ARG;
  if (k_out && (rc = rows_ok(k_out, k_stride, kw, bytes)) != SDV_OK) return rc;
  if (v_out && (rc = rows_ok(v_out, v_stride, kw, bytes)) != SDV_OK) return rc;
  p.k = k_out;
  p.v = v_out;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  return launched(launch_cache_read(h->cfg.head_dim, h->cfg.cache_format, out_format, p, h->sms, static_cast<cudaStream_t>(stream)));
}
