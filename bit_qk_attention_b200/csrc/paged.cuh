// The paged KV cache as the kernels see it (the layout is documented in include/binattn.h).
#pragma once

#include "common.cuh"

namespace binattn {

constexpr int kMinExp = -24, kMaxExp = 9;  // exponents of a cached V row
constexpr int kPageUnit = 16;              // a page holds a multiple of this many tokens
constexpr int kMaxPage = 1024;

struct CacheView {
  uint8_t* data;
  int64_t num_pages;
  int page_size, heads, d, dp;
  int64_t block_bytes;

  // Offsets of the parts of a block.
  __host__ __device__ int off_bits() const { return page_size * dp; }
  __host__ __device__ int off_mu() const { return page_size * (dp + 16); }
  __host__ __device__ int off_exp() const { return page_size * (dp + 18); }
  __device__ uint8_t* block(int64_t page, int head) const { return data + (page * heads + head) * block_bytes; }
};

// n / d for 0 <= n < 2^31, without a division: mul = ceil(2^(31 + s) / d) with 2^(s-1) < d <= 2^s is
// off by less than 2^s / 2^(31 + s) of the quotient's scale, too little to reach the next whole number.
struct FastDiv {
  uint32_t mul, shift;
  static FastDiv of(int d) {
    uint32_t s = 0;
    while ((int64_t{1} << s) < d) ++s;
    return {static_cast<uint32_t>(((uint64_t{1} << (31 + s)) + d - 1) / d), 31 + s};
  }
  __host__ __device__ int operator()(int n) const {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul) >> shift);
  }
};

struct CacheWriteParams {
  CacheView cache;
  const void* k;
  const void* v;
  int64_t k_stride_t, k_stride_h, v_stride_t, v_stride_h;  // elements
  int64_t T;
  const int64_t* slots;
  bool wide;  // every row of k and v starts on 16 bytes and d is a multiple of 8
  FastDiv by_heads, by_page;
};

struct CacheReadParams {
  CacheView cache;
  const int64_t* slots;
  int64_t T;
  void* k;
  void* v;
  FastDiv by_heads, by_page;
};

// Page of a slot and the offset in it; page -1 outside the cache.
__device__ __forceinline__ int64_t page_of_slot(const CacheView& cv, const FastDiv& by_page, int64_t slot, int& off) {
  if (slot < 0 || slot >= cv.num_pages * cv.page_size) return -1;
  const int64_t page = (slot >> 31) == 0 ? by_page(static_cast<int>(slot)) : slot / cv.page_size;
  off = static_cast<int>(slot - page * cv.page_size);
  return page;
}

// Attention of new tokens over the cache.
struct JoinNote;
struct PagedAttnParams {
  CacheView cache;
  const void* q;
  int64_t q_stride_t, q_stride_h;  // elements
  int B, heads, group;             // group = query heads per KV head
  FastDiv by_group, by_kv_heads, by_page, by_tiles;  // divide by group, KV heads, page size, row tiles
  int64_t T;
  int max_q_len, max_kv_len;  // max_kv_len also within the page table
  const int32_t* cu;          // null: one row per sequence
  const int32_t* kv_lens;
  const int32_t* table;
  int64_t table_stride;
  int causal, window, sinks;
  float scale_log2;  // softmax scale * log2(e)
  void* o;
  int o_dt;
  float* lse;
  int row_tile;    // rows (token, head of the group) of a CTA's tile
  int row_tiles;   // tiles of a sequence and KV head (most)
  float* part_o;     // [ctas][2][row_tile][dp] unnormalised sums of cut (tile, head)s, by slot
  float2* part_ml;   // [ctas][2][row_tile] (maximum in log2, sum)
  int ctas;          // CTAs that share the line of units; 0: a cluster of CTAs per (tile, head)
  int cluster;       // its size
  int whole;         // many rows: each CTA has one (tile, head), nothing is cut
  JoinNote* notes;   // [ctas]
  const uint4* q_bits;  // [T * heads] sign words of q (many rows)
  const float* q_mu;    // [T * heads] their scales
};

// What a CTA works on: a tile of rows r = i * group + g (i-th new token, g-th head of the group) of
// one sequence and KV head, against the keys that any of them sees. The keys are counted in blocks
// of `bk` tokens: the blocks of the sinks, then those from the window's start to the last key.
struct RowTile {
  int64_t t0;     // row of q of the sequence's first new token
  int nq, kv;     // new tokens, tokens in the cache
  int r0, rows;   // first row of the tile, rows in it (<= 0: nothing to do)
  int lo;         // no row sees keys below it, but for the sinks
  int nsink, first, nblk;  // sink blocks, first block after them, blocks in all

  __device__ int block_at(int v) const { return v < nsink ? v : first + (v - nsink); }
  __device__ int pos0() const { return kv - nq; }  // position of the first new token
};

__device__ __forceinline__ RowTile row_tile(const PagedAttnParams& p, int b, int tile, int bk) {
  RowTile w;
  int64_t n;
  if (p.cu != nullptr) {
    w.t0 = min(max(static_cast<int64_t>(p.cu[b]), int64_t{0}), p.T);
    n = min(max(static_cast<int64_t>(p.cu[b + 1]), w.t0), p.T) - w.t0;
  } else {
    w.t0 = b;
    n = b < p.T ? 1 : 0;
  }
  w.nq = static_cast<int>(min(n, int64_t{1} << 28));
  w.kv = min(max(p.kv_lens[b], 0), p.max_kv_len);
  w.r0 = tile * p.row_tile;
  w.rows = static_cast<int>(min(static_cast<int64_t>(p.row_tile),
                                static_cast<int64_t>(min(w.nq, p.max_q_len)) * p.group - w.r0));
  int lo = 0, hi = w.kv;
  if (p.causal && w.rows > 0) {
    hi = min(hi, w.pos0() + p.by_group(w.r0 + w.rows - 1) + 1);
    if (p.window > 0) lo = max(0, w.pos0() + p.by_group(w.r0) - p.window + 1);
  }
  w.lo = lo;
  w.first = lo / bk;
  w.nsink = min(static_cast<int>(ceil_div(p.sinks, bk)), w.first);
  w.nblk = hi <= 0 || w.rows <= 0 ? 0 : w.nsink + static_cast<int>(ceil_div(hi, bk)) - w.first;
  return w;
}

// Row of o (and of lse) of the tile's row r.
__device__ __forceinline__ int64_t out_row(const PagedAttnParams& p, const RowTile& w, int head, int r) {
  const int i = p.by_group(w.r0 + r);
  return (w.t0 + i) * p.heads + head * p.group + (w.r0 + r - i * p.group);
}

// The work of a launch is a line of units, for all sequences' row tiles, one KV head after the other:
// `cost` units that stand for starting and ending a (tile, head), then one for each of its key blocks.
// Each CTA takes the same number of units, whatever the lengths are, so the blocks of a (tile, head)
// may be cut at the ends of CTAs. What a CTA computes of a cut one goes into the workspace: slot 0 if
// it began before the CTA, else slot 1. The CTA in which a cut one begins leaves a note for the
// kernel that joins the parts.
struct JoinNote {
  int entry, head;  // entry = b * row_tiles + tile
  int last;         // CTA with the last part; the CTAs between have it in slot 0. -1: nothing to join
};

__device__ __forceinline__ RowTile entry_tile(const PagedAttnParams& p, int entry, int bk) {
  const int b = p.by_tiles(entry);
  return row_tile(p, b, entry - b * p.row_tiles, bk);
}

__device__ __forceinline__ int units_of(const RowTile& w, int cost) { return w.rows > 0 ? cost + w.nblk : 0; }

// The entry after one: the next tile, or, behind a sequence's last row, where there may be any number of tiles
// without rows (as many as max_q_len has), the next sequence.
__device__ __forceinline__ int entry_after(const PagedAttnParams& p, int entry, const RowTile& w) {
  return w.rows > 0 ? entry + 1 : (p.by_tiles(entry) + 1) * p.row_tiles;
}

// Units of the line per CTA, rounded up: below 2^31 (the plan sees to it). In 32 bits where the sum fits, since
// every CTA waits for this division.
__host__ __device__ __forceinline__ int share_of(int64_t total, uint32_t ctas) {
  const int64_t up = total + ctas - 1;
  return static_cast<int>((up >> 32) == 0 ? static_cast<uint32_t>(up) / ctas : up / ctas);
}

// A CTA's stretch [at, end) of the line, `per` units or fewer; `at` lies in `entry`, whose units
// start at `base`.
struct Stretch {
  int64_t at, end, base;
  int per, entry;
};

template <int THREADS>
__device__ __forceinline__ Stretch find_stretch(const PagedAttnParams& p, int bk, int cost, int min_units,
                                                int64_t* scratch) {  // shared memory: THREADS / 32 + 2
  int64_t* s_warp = scratch;
  int64_t& s_base = scratch[THREADS / 32];
  int64_t& s_entry = scratch[THREADS / 32 + 1];
  // n < 2^31, but rounded up to a multiple of THREADS it may not be.
  const int heads = p.cache.heads, n = p.B * p.row_tiles;
  const unsigned end = n, each = (end + THREADS - 1) / THREADS;
  const int i0 = min(end, threadIdx.x * each), i1 = min(end, (threadIdx.x + 1) * each);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t sum = 0;
  for (int i = i0; i < i1;) {
    const RowTile w = entry_tile(p, i, bk);
    sum += units_of(w, cost);
    i = entry_after(p, i, w);
  }
  int64_t upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) s_warp[warp] = upto;
  __syncthreads();
  int64_t total = 0, before = upto - sum;
#pragma unroll
  for (int k = 0; k < THREADS / 32; ++k) {
    if (k < warp) before += s_warp[k];
    total += s_warp[k];
  }
  total *= heads;
  Stretch st;
  st.per = max(min_units, share_of(total, gridDim.x));
  st.at = static_cast<int64_t>(blockIdx.x) * st.per;
  st.end = min(total, st.at + st.per);
  int64_t base = before * heads;
  if (st.at < st.end && base <= st.at && st.at < base + sum * heads) {
    int i = i0;
    while (true) {
      const RowTile w = entry_tile(p, i, bk);
      const int64_t u = static_cast<int64_t>(units_of(w, cost)) * heads;
      if (st.at < base + u) break;
      base += u;
      i = entry_after(p, i, w);
    }
    s_entry = i;
    s_base = base;
  }
  __syncthreads();
  st.entry = static_cast<int>(s_entry);
  st.base = s_base;
  return st;
}

// Page of the 16 tokens from j on (a multiple of 16) and their offset in it; page -1 where there is
// none: behind the sequence, or outside the cache.
struct PageAt {
  int page, off;
};

__device__ __forceinline__ PageAt page_at(const PagedAttnParams& p, const int32_t* table, int kv, int j) {
  PageAt at{-1, 0};
  if (j < kv) {
    const int e = p.by_page(j);
    at.page = table[e];
    at.off = j - e * p.cache.page_size;
    if (at.page < 0 || at.page >= p.cache.num_pages) at.page = -1;
  }
  return at;
}

// The mean of d numbers |x| is the sum of |x| * kMeanStep over d * kMeanStep: exact steps of a power of two that
// keep 128 of the largest bf16 numbers within fp32's range (and the least ones above its end).
constexpr float kMeanStep = 0.0078125f;
__device__ __forceinline__ float mean_of(float sum, int d) { return sum / (static_cast<float>(d) * kMeanStep); }

// A 16-bit number, widened.
__device__ __forceinline__ float widen(uint16_t x, int f16) {
  return f16 ? __half2float(__ushort_as_half(x)) : __uint_as_float(static_cast<uint32_t>(x) << 16);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Key blocks of bk tokens that a tile of `rows` rows can see, at most.
inline int64_t most_blocks(const PagedAttnParams& p, int rows, int bk) {
  int64_t keys = p.max_kv_len;
  if (p.causal && p.window > 0) {
    const int64_t near = static_cast<int64_t>(p.window) + rows / p.group + p.sinks + 2 * bk;
    keys = keys < near ? keys : near;
  }
  return ceil_div(keys, bk);
}

cudaError_t launch_paged_decode(const PagedAttnParams& p, int dt, cudaStream_t s);
cudaError_t launch_paged_chunk(const PagedAttnParams& p, int dt, cudaStream_t s);
// Sets p's `ctas` and `cluster` for a device of `sms` SMs.
void paged_decode_plan(PagedAttnParams* p, int sms);
void paged_chunk_plan(PagedAttnParams* p, int sms);
// The kernel behind both that joins cut (tile, head)s (key blocks of bk tokens).
cudaError_t launch_line_join(const PagedAttnParams& p, int bk, cudaStream_t s);

cudaError_t launch_cache_write(const CacheWriteParams& p, int dt, cudaStream_t s);
cudaError_t launch_cache_read(const CacheReadParams& p, int dt, cudaStream_t s);

}  // namespace binattn
