// C-ABI layer of the paged cache: argument checks and launches. The entry points are declared and
// documented in include/binattn.h.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "binattn.h"
#include "kernels.h"
#include "paged.cuh"

using namespace binattn;

namespace {

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 4096;  // (token, head) rows of a call
constexpr int64_t kMaxKv = int64_t{1} << 28;
// Rows (new tokens x heads of a group) of a sequence up to which the decoding kernel is taken, with a
// pass over the cache for every 16 rows (8 KV heads, d = 128, decoding kernel and the other one, us):
//              1 x 8192 keys  32 x 4096  128 x 1024  16 x 1024
//   16 rows       18   36       49  126    79  141     16   24
//   32 rows       20   36      100  126   139  142     20   24
//   48 rows       20   37      139  127   201  145     41   24
constexpr int kDecodeRows = 32;
// Up to so many where its tiles fit on the GPU at once and a warp has at most so many blocks of 64 keys:
// there the other kernel's start, cuts and join last longer than the further passes. 48 rows, 1 x 65536
// keys (21 blocks a warp) 66 and 76 us, 64 rows (28 blocks) 82 and 76; 128 rows, 1 x 8192 keys (7 blocks)
// 29 and 40 us. 64 rows, 16 x 1024 keys, twice as many tiles as fit: 48 and 24.
constexpr int kDraftRows = 128, kDraftBlocks = 24;
constexpr int kChunkRows = 256;  // row tile of the kernel for more
constexpr int64_t kMaxCtas = (int64_t{1} << 31) - 1;

bool aligned(const void* p, unsigned n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

ba_status check_cache(const ba_kv_cache* c, CacheView* out) {
  if (c == nullptr || c->num_pages < 0 || c->n_kv_heads < 0) return BA_ERR_INVALID_ARG;
  if (ba_kv_block_bytes(c->page_size, c->d) == 0 || c->n_kv_heads < 1 || c->n_kv_heads > 65535)
    return BA_ERR_UNSUPPORTED;
  if (c->num_pages > (int64_t{1} << 40) / c->page_size) return BA_ERR_UNSUPPORTED;
  if (c->num_pages > 0 && c->data == nullptr) return BA_ERR_INVALID_ARG;
  if (!aligned(c->data, 16)) return BA_ERR_ALIGNMENT;
  out->data = static_cast<uint8_t*>(c->data);
  out->num_pages = c->num_pages;
  out->page_size = c->page_size;
  out->heads = c->n_kv_heads;
  out->d = c->d;
  out->dp = v_row_bytes(c->d);
  out->block_bytes = static_cast<int64_t>(ba_kv_block_bytes(c->page_size, c->d));
  return BA_OK;
}

int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) {
    if (dev < 64 && (sms = known[dev].load()) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) {
      if (dev < 64) known[dev].store(sms);
      return sms;
    }
  }
  cudaGetLastError();  // no device here: the workspace query still answers
  return 148;
}

size_t align_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Regions of the workspace of a launch whose CTAs share the line of units; their size in bytes.
size_t line_workspace(const PagedAttnParams& p, PagedAttnParams* out) {
  const size_t ctas = p.whole ? 0 : p.ctas, n = ctas * 2 * p.row_tile;
  const size_t ml = align_up(n * p.cache.dp * 4), notes = ml + align_up(n * 8);
  const size_t bits = notes + align_up(ctas * sizeof(JoinNote));
  const size_t rows = p.row_tile == kChunkRows ? static_cast<size_t>(p.T) * p.heads : 0, mu = bits + align_up(rows * 16);
  if (out != nullptr) {
    char* base = reinterpret_cast<char*>(out->part_o);
    out->part_ml = reinterpret_cast<float2*>(base + ml);
    out->notes = reinterpret_cast<JoinNote*>(base + notes);
    out->q_bits = reinterpret_cast<uint4*>(base + bits);
    out->q_mu = reinterpret_cast<float*>(base + mu);
  }
  return mu + align_up(rows * 4);
}

// Everything of a call that does not depend on its tensors: sizes, the kernel's tiles and splits,
// and the workspace.
ba_status plan(const ba_kv_cache* cache, const ba_paged_seqs* s, PagedAttnParams* p, size_t* ws) {
  *ws = 0;
  ba_status st = check_cache(cache, &p->cache);
  if (st != BA_OK) return st;
  if (s == nullptr || s->B < 0 || s->T < 0 || s->n_heads < 1 || s->max_q_len < 0 || s->max_kv_len < 0 ||
      s->max_pages < 0 || s->table_stride < 0 || s->window < 0 || s->sinks < 0)
    return BA_ERR_INVALID_ARG;
  if (s->causal != 0 && s->causal != 1) return BA_ERR_INVALID_ARG;
  if (s->window > 0 && s->causal != 1) return BA_ERR_INVALID_ARG;
  if (s->n_heads % cache->n_kv_heads != 0) return BA_ERR_INVALID_ARG;
  if (s->max_kv_len > kMaxKv || s->T > kMaxRows / s->n_heads) return BA_ERR_UNSUPPORTED;
  if (cache->num_pages > ((int64_t{1} << 31) - 1) / cache->n_kv_heads) return BA_ERR_UNSUPPORTED;
  p->B = s->B;
  p->heads = s->n_heads;
  p->group = s->n_heads / cache->n_kv_heads;
  p->T = s->T;
  p->max_q_len = static_cast<int>(std::min<int64_t>(s->cu_seqlens_q != nullptr ? s->max_q_len : std::min(s->max_q_len, 1), s->T));
  p->max_kv_len = static_cast<int>(std::min<int64_t>(s->max_kv_len, static_cast<int64_t>(s->max_pages) * cache->page_size));
  p->cu = s->cu_seqlens_q;
  p->kv_lens = s->kv_lens;
  p->table = s->page_table;
  p->table_stride = s->table_stride;
  p->causal = s->causal;
  // Positions lie within +-2^28: longer windows and more sinks hide nothing either, and sums with these
  // stay within an int.
  p->window = static_cast<int>(std::min<int64_t>(s->window, 2 * kMaxKv));
  p->sinks = static_cast<int>(std::min<int64_t>(s->sinks, kMaxKv));
  if (p->B == 0 || p->max_q_len == 0) return BA_OK;  // nothing to launch
  const int64_t rows = static_cast<int64_t>(p->max_q_len) * p->group;
  const int64_t tiles16 = ceil_div(rows, 16) * p->B * p->cache.heads, at_once = 2 * sm_count();
  const bool few = rows <= kDecodeRows || (rows <= kDraftRows && tiles16 <= at_once &&
                                           tiles16 * most_blocks(*p, 16, 64) <= at_once * 4 * kDraftBlocks);
  p->row_tile = rows <= 8 ? 8 : (few ? 16 : kChunkRows);
  const int64_t tiles = ceil_div(rows, p->row_tile);
  if (tiles > kMaxCtas / (static_cast<int64_t>(p->B) * p->cache.heads)) return BA_ERR_UNSUPPORTED;
  p->row_tiles = static_cast<int>(tiles);
  p->by_group = FastDiv::of(p->group);
  p->by_kv_heads = FastDiv::of(p->cache.heads);
  p->by_page = FastDiv::of(p->cache.page_size);
  p->by_tiles = FastDiv::of(p->row_tiles);
  const int64_t all = tiles * p->B * p->cache.heads;
  // A CTA's share of the key blocks (64 or 128 keys) counts in 31 bits.
  if (all > (int64_t{1} << 38) / (p->max_kv_len / 64 + 16)) return BA_ERR_UNSUPPORTED;
  if (p->row_tile == kChunkRows)
    paged_chunk_plan(p, sm_count());
  else
    paged_decode_plan(p, sm_count());
  if (p->ctas > 0) *ws = line_workspace(*p, nullptr);
  return BA_OK;
}

}  // namespace

extern "C" {

size_t ba_kv_block_bytes(int page_size, int d) {
  if (d < 1 || d > 128 || page_size < kPageUnit || page_size > kMaxPage || page_size % kPageUnit != 0) return 0;
  return static_cast<size_t>(page_size) * (v_row_bytes(d) + 19);
}

ba_status ba_cache_write(const void* k, int64_t k_stride_t, int64_t k_stride_h, const void* v, int64_t v_stride_t,
                         int64_t v_stride_h, ba_dtype dt, int64_t T, const int64_t* slots, const ba_kv_cache* cache,
                         void* stream) {
  CacheWriteParams p{};
  const ba_status st = check_cache(cache, &p.cache);
  if (st != BA_OK) return st;
  if (dt != BA_F16 && dt != BA_BF16) return BA_ERR_INVALID_ARG;
  if (T < 0 || k_stride_t < 0 || k_stride_h < 0 || v_stride_t < 0 || v_stride_h < 0) return BA_ERR_INVALID_ARG;
  if (T > kMaxRows / cache->n_kv_heads) return BA_ERR_UNSUPPORTED;
  if (T == 0 || cache->num_pages == 0) return BA_OK;
  if (!k || !v || !slots) return BA_ERR_INVALID_ARG;
  if (!aligned(k, 2) || !aligned(v, 2) || !aligned(slots, 8)) return BA_ERR_ALIGNMENT;
  p.k = k;
  p.v = v;
  p.k_stride_t = k_stride_t;
  p.k_stride_h = k_stride_h;
  p.v_stride_t = v_stride_t;
  p.v_stride_h = v_stride_h;
  p.T = T;
  p.slots = slots;
  p.wide = cache->d % 8 == 0 && aligned(k, 16) && aligned(v, 16) &&
           (k_stride_t | k_stride_h | v_stride_t | v_stride_h) % 8 == 0;
  p.by_heads = FastDiv::of(cache->n_kv_heads);
  p.by_page = FastDiv::of(cache->page_size);
  return report_cuda(launch_cache_write(p, dt, static_cast<cudaStream_t>(stream)));
}

ba_status ba_cache_read(const ba_kv_cache* cache, const int64_t* slots, int64_t T, void* k, void* v, ba_dtype dt,
                        void* stream) {
  CacheReadParams p{};
  const ba_status st = check_cache(cache, &p.cache);
  if (st != BA_OK) return st;
  if (dt != BA_F16 && dt != BA_BF16 && dt != BA_F32) return BA_ERR_INVALID_ARG;
  if (T < 0) return BA_ERR_INVALID_ARG;
  if (T > kMaxRows / cache->n_kv_heads) return BA_ERR_UNSUPPORTED;
  if (T == 0 || (!k && !v)) return BA_OK;
  if (!slots) return BA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return BA_ERR_ALIGNMENT;
  p.slots = slots;
  p.T = T;
  p.k = k;
  p.v = v;
  p.by_heads = FastDiv::of(cache->n_kv_heads);
  p.by_page = FastDiv::of(cache->page_size);
  return report_cuda(launch_cache_read(p, dt, static_cast<cudaStream_t>(stream)));
}

size_t ba_paged_workspace_bytes(const ba_kv_cache* cache, const ba_paged_seqs* seqs) {
  PagedAttnParams p{};
  size_t ws = 0;
  return plan(cache, seqs, &p, &ws) == BA_OK ? ws : static_cast<size_t>(-1);
}

ba_status ba_attention_paged(const void* q, int64_t q_stride_t, int64_t q_stride_h, ba_dtype dt,
                             const ba_kv_cache* cache, const ba_paged_seqs* seqs, float softmax_scale, void* o,
                             ba_dtype o_dt, float* lse, void* ws, size_t ws_bytes, void* stream) {
  PagedAttnParams p{};
  size_t need = 0;
  const ba_status st = plan(cache, seqs, &p, &need);
  if (st != BA_OK) return st;
  if (dt != BA_F16 && dt != BA_BF16) return BA_ERR_INVALID_ARG;
  if (o_dt != BA_F16 && o_dt != BA_BF16 && o_dt != BA_F32) return BA_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale) || q_stride_t < 0 || q_stride_h < 0) return BA_ERR_INVALID_ARG;
  if (p.B == 0 || p.max_q_len == 0) return BA_OK;
  if (!q || !o || !p.kv_lens || (p.max_kv_len > 0 && !p.table)) return BA_ERR_INVALID_ARG;
  if (!aligned(q, 2) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(p.cu, 4) || !aligned(p.kv_lens, 4) ||
      !aligned(p.table, 4))
    return BA_ERR_ALIGNMENT;
  if (need > 0) {
    if (ws == nullptr || ws_bytes < need) return BA_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return BA_ERR_ALIGNMENT;
    p.part_o = static_cast<float*>(ws);
    line_workspace(p, &p);
  }
  p.q = q;
  p.q_stride_t = q_stride_t;
  p.q_stride_h = q_stride_h;
  const float scale = softmax_scale > 0.0f ? softmax_scale : 1.0f / std::sqrt(static_cast<float>(cache->d));
  p.scale_log2 = scale * 1.4426950408889634f;
  p.o = o;
  p.o_dt = o_dt;
  p.lse = lse;
  const cudaStream_t st_ = static_cast<cudaStream_t>(stream);
  return report_cuda(p.row_tile == kChunkRows ? launch_paged_chunk(p, dt, st_) : launch_paged_decode(p, dt, st_));
}

}  // extern "C"
