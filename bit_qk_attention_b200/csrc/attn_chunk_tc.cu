// Attention of many query rows over the paged cache on 5th-generation tensor cores (sm_100a).
//
// 256 rows (new tokens x query heads of a group, which share every key) of one sequence and KV head
// meet the 128-key blocks that any of them sees, as two tiles of 128 rows. The products run on tcgen05
// with fp32 accumulators in tensor memory:
//   S = Q K^T  e4m3, both +-1: the whole number d - 2 popc comes out exact; mu_j follows in the softmax
//   O += P V   fp16: P = 2^(s - M), rounded to fp16, V = code 2^e, exact in that type. M is 2^3 to 2^7 below the
//              largest score, not at it: fp16 then loses precision only 2^17 to 2^21 below the largest weight
// One CTA per SM (it owns all tensor memory) walks its stretch of the line of all key blocks, so that
// every SM has the same number of them whatever the lengths and the mask are:
//   * The cache holds K in bits and V in bytes. One warp brings a block's rows by TMA (V through a
//     swizzled tensor map); four expanding warps, one key per lane, read them into registers, which
//     frees the stage for the next block, and write the operands: two instructions per four K channels,
//     seven per four V channels. K and V operands are double-buffered. (K as +-mu_j in bf16 needed no
//     product in the softmax, but twice the instructions, MMAs and shared memory: the call timed below then took
//     1.03 ms instead of 0.97; it is 0.88 by what came after.)
//   * Two warpgroups of softmax, one per tile, one thread per row. Most scores are read once, without a
//     maximum: the weights 2^(s - M) are made with the M of the keys before, and their sum, which is
//     needed anyway, shows whether any of them grew too large for fp16 (weights are positive: a sum up
//     to 65504 has none above). Only then, in a row's first keys and behind a mask, the scores are read
//     again, M moves to 2^3 to 2^7 below the maximum if that is 2^9.9 above it, and O is rescaled in tensor
//     memory.
//   * A block's scores come in two halves of 64 keys, each with its weights over it: a half's P V and
//     the scores two halves on follow its weights in the order of issue, while the softmax works on the
//     other half. It reads the next half's first scores before it waits for its weights to arrive.
//   * At the end of a (tile, head) a softmax warpgroup writes the next one's Q before it reads O, so that
//     the next scores are made meanwhile.
// A block of 256 x 128 scores at d = 128 costs 2048 cycles of exponentials (16 per cycle and SM), and
// 1792 of MMAs; that is the bound. A block takes about 4000: 4096 new tokens of 16 heads over 32768 keys
// of 4 heads take 880 us (1.17 PFLOP/s). What it spends beyond the exponentials is the softmax warps' own
// latency, two of them per scheduler: without any expanding or MMAs they take 850 us. (Four softmax
// warpgroups, two per tile, with 80 registers a thread and a vote between them per half, took 1.05 ms;
// asking for the next half's scores before the half is done 1.01.) 2 x 8192 new tokens of 16 heads (8 KV heads, d = 64)
// in a window of 1024 with 4 sinks take 202 us: 8000 cycles for a block, with a mask in a quarter of the halves.
//
// Every wait is bounded (1 s): on expiry the kernel records a timeout in a device status word, all
// roles leave, copies and MMAs in flight are waited for, and tensor memory is freed.
#include <math_constants.h>

#include <algorithm>

#include "kernels.h"
#include "paged.cuh"
#include "tc_ptx.cuh"
#include "tensormap.h"

namespace binattn {

__device__ int g_chunk_status = 0;

namespace {

using namespace ptx;

constexpr int kBlk = 128;      // keys per block: N of QK, K of PV
constexpr int kTile = 128;     // rows per tile: M
// Blocks that a CTA could do while it starts and ends a (tile, head): with 1, 2, 4 and 6 a prompt of 2 x
// 8192 tokens in a window took 235, 201, 199 and 200 us (with M at the largest score; see kBelow), chunks of 4 x 1000
// over 9000 keys 192, 189, 180, 180.
constexpr int kCost = 4;
constexpr int kWholeBlocks = 10; // blocks that cutting a (tile, head) has to save
constexpr int kMinUnits = 6;   // units (blocks, and kCost) a CTA takes at least
constexpr int kThreads = 512;  // service, expanding and two softmax warpgroups
// Weights are 2^(s - M), and M is set some way below the largest score, so that fp16 has its full precision down
// to 2^-14 of 1, not of the largest weight, and steps of 2^-24 below: kBelow, or less (kLeastBelow at least) where
// the bound on a masked half's scores would then pass kMostLog2 and its maximum be read for nothing (7 always: a
// prompt of 2 x 8192 tokens in a window took 205.5 us instead of 202.2). M moves where a maximum would reach 2^kHigh:
// 64 weights up to that sum to less than kMostSum, so a half whose sum is larger always moves it.
constexpr float kBelow = 7.0f, kLeastBelow = 3.0f;
constexpr float kHigh = 9.9f;
constexpr float kMostLog2 = 15.9f;    // log2 of weights that fp16 surely holds
constexpr float kBoundUp = 1.000001f; // more than the roundings of a score and of its bound
constexpr float kMostSum = 65504.0f;  // fp16's largest number: a sum of weights up to this has none above it
// A row's factor of its scores is this at least, also for a row of zeros, so that -inf in masked places stays -inf:
// fp32's least number, which makes nothing of any finite score.
constexpr float kLeastFactor = 1.4e-45f;
constexpr uint64_t kTimeoutNs = 1000000000ull;

template <int CH>  // channels of the operands: 64 or 128 (>= d)
struct Cfg {
  static constexpr int kOp8 = kBlk * CH;      // bytes of an operand tile of 128 rows: Q and K
  static constexpr int kOp16 = kBlk * CH * 2;  // and V
  static constexpr int kRow = CH;            // bytes of a V row in the stage
  static constexpr int offQ = 0;
  static constexpr int offK = offQ + 2 * kOp8;
  static constexpr int offV = offK + 2 * kOp8;
  static constexpr int offRaw = offV + 2 * kOp16;  // the cache rows of a block: codes, sign rows, mu, exponents
  static constexpr int offBits = offRaw + kBlk * kRow;
  static constexpr int offMu = offBits + kBlk * 16;
  static constexpr int offExp = offMu + kBlk * 2;
  static constexpr int offScale = offExp + kBlk;  // [block % 4][key]: mu as floats
  static constexpr int offBar = offScale + 4 * kBlk * 4;
  static constexpr int kToken = kRow + 16 + 2 + 1;  // bytes that a token brings
  static constexpr int kNumBars = 26;
  static constexpr int offMisc = offBar + kNumBars * 8;  // tensor memory base, abort flag, page masks [4]
  static constexpr int offTop = offMisc + 8 + 16;  // [block % 4][expanding warp]: bits of the largest mu of its keys
  static constexpr int offScratch = offTop + 64;
  static constexpr int kBytes = offScratch + (kThreads / 32 + 2) * 8;
  static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
  // Tensor memory: S of tile q in two halves of 64 keys, each with its P over it, then O.
  static __host__ __device__ constexpr uint32_t tS(int q) { return q * 128; }
  static __host__ __device__ constexpr uint32_t tO(int q) { return 256 + q * CH; }
  // Byte offset of the 16-byte piece c of key j's V row: the swizzle of 128- or 64-byte rows.
  static __device__ __forceinline__ int piece(int j, int c) {
    return kRow == 128 ? (j * 8 + (c ^ (j & 7))) * 16 : (j * 4 + (c ^ ((j >> 1) & 3))) * 16;
  }
};

// Barriers. K and V operands: per stage. The others: per tile; S, P and P V by halves of the keys, since
// who waits for the last P V may not have seen the one before.
constexpr int bKfull = 0, bKempty = 2, bVfull = 4, bVempty = 6, bQfull = 8, bS = 10, bP = 14, bPV = 18, bDrain = 22,
              bRawFull = 24, bRawEmpty = 25;

// The (tile, head)s of a CTA one after the other, as every role walks them.
struct Walk {
  Stretch line;
  RowTile w;
  int b, head, entry, v0, n_blk, slot, last;  // slot as in attn_paged.cu; last: the CTA of the last part

  __device__ __forceinline__ bool next(const PagedAttnParams& p) {
    while (line.at < line.end) {
      w = entry_tile(p, line.entry, kBlk);
      const int units = units_of(w, kCost);
      if (units == 0) {  // a tile without rows
        line.entry = entry_after(p, line.entry, w);
        continue;
      }
      entry = line.entry;
      b = p.by_tiles(entry);
      const int64_t in = line.at - line.base;
      head = (in >> 32) == 0 ? static_cast<uint32_t>(in) / static_cast<uint32_t>(units) : static_cast<int>(in / units);
      const int u0 = static_cast<int>(in - static_cast<int64_t>(head) * units);
      const int u1 = static_cast<int>(min(static_cast<int64_t>(units), u0 + line.end - line.at));
      const int64_t stop = line.at + (units - u0);  // where the (tile, head) ends
      v0 = max(0, u0 - kCost);
      const int v1 = max(0, u1 - kCost);
      n_blk = v1 - v0;
      slot = v0 > 0 ? 0 : (v1 < w.nblk ? 1 : -1);
      last = slot == 1 && v1 > 0 ? static_cast<int>((stop - 1) / line.per) : -1;
      line.at += u1 - u0;
      if (u1 == units && head == p.cache.heads - 1) {
        line.base += static_cast<int64_t>(units) * p.cache.heads;
        ++line.entry;
      }
      if (v1 == 0 && u1 < units) continue;  // cut before the first block: all of it is the next CTA's
      return true;
    }
    return false;
  }
  __device__ __forceinline__ int tiles() const { return w.rows > kTile ? 2 : 1; }
};

// Waits for a phase, a second at most. SLEEP: with a suspend hint, for the roles that mostly wait; the
// polls of the others are on the softmax's path.
template <bool SLEEP>
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag, bool yield = true) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
    if (SLEEP ? mbar_try_wait_sleep(bar, parity, 20000u) : mbar_try_wait(bar, parity)) return true;
    if (yield && *abort_flag) return false;
    if (globaltimer() - t0 > kTimeoutNs) {
      *abort_flag = 1;
      atomicExch(&g_chunk_status, 1);
      return false;
    }
  }
}

template <bool SLEEP>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_bar<SLEEP>(bar, parity, abort_flag));
}

// The n lowest bits (none below 0, all from 32 on).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }

// Sign bits of 32 channels -> +-1 in e4m3, two 16-byte pieces of a K-major operand row. Byte b of word i
// is channel 8 b + i, so that one shift and one mask place four signs; Q and K have the same order, and
// a dot product does not mind. `live`: channels that exist, the others are 0.
__device__ __forceinline__ void expand_signs(uint32_t dst, uint32_t word, uint32_t live) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = ((word << (7 - 4 * c - i)) & 0x80808080u) ^ 0x38383838u;
      if (live != 0xffffffffu) x[i] &= ((live >> (4 * c + i)) & 0x01010101u) * 255u;
    }
    sts128(dst + c * 2048, x[0], x[1], x[2], x[3]);
  }
}

// Eight codes (two words, 8 bits each) times 2^e -> eight fp16 numbers.
__device__ __forceinline__ void expand_codes(uint32_t dst, uint32_t a, uint32_t b, __half2 step) {
  const uint32_t w[2] = {a ^ 0x80808080u, b ^ 0x80808080u};
  const __half2 bias = __floats2half2_rn(-1152.0f, -1152.0f);
  uint32_t x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = __byte_perm(w[i >> 1], 0x64646464u, i & 1 ? 0x4342 : 0x4140);
    const __half2 y = __hmul2(__hadd2(*reinterpret_cast<const __half2*>(&u), bias), step);
    x[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  sts128(dst, x[0], x[1], x[2], x[3]);
}

// Sign words and scale mu of the rows of q: one warp per row, a channel per lane and word. (In the
// attention kernel itself, 32 rows a warp, this took as long as two blocks for every (tile, head).)
template <typename T>
__global__ void __launch_bounds__(256) paged_q_kernel(PagedAttnParams p, uint4* bits, float* mu) {
  allow_dependents();
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / 32;
  const int lane = threadIdx.x & 31;
  if (row >= p.T * p.heads) return;
  const int64_t t = row / p.heads;
  const T* src = static_cast<const T*>(p.q) + t * p.q_stride_t + (row - t * p.heads) * p.q_stride_h;
  uint32_t word[4];
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float x = 32 * k + lane < p.cache.d ? load1<T>(src + 32 * k + lane) : 0.0f;
    word[k] = __ballot_sync(0xffffffffu, x < 0.0f);
    sum += fabsf(x) * kMeanStep;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) {
    bits[row] = make_uint4(word[0], word[1], word[2], word[3]);
    mu[row] = mean_of(sum, p.cache.d);
  }
}

template <int CH>
__global__ void __launch_bounds__(kThreads, 1) paged_chunk_kernel(PagedAttnParams p, int unit, const __grid_constant__ CUtensorMap v_map) {
  using C = Cfg<CH>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::offBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::offMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::offMisc + 4);
  volatile uint32_t* page_ok = reinterpret_cast<volatile uint32_t*>(smem + C::offMisc + 8);  // [block % 4]: which 16 keys have a page
  const CacheView& cv = p.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem);

  allow_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[bKfull + i], 4);
      mbar_init(&bars[bVfull + i], 4);
      mbar_init(&bars[bKempty + i], 2);
      mbar_init(&bars[bVempty + i], 2);
      mbar_init(&bars[bDrain + i], 1);
      mbar_init(&bars[bQfull + i], 4);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&bars[bS + 2 * i + h], 1);
        mbar_init(&bars[bP + 2 * i + h], 4);
        mbar_init(&bars[bPV + 2 * i + h], 1);
      }
    }
    mbar_init(&bars[bRawFull], 1);
    mbar_init(&bars[bRawEmpty], 4);
    *abort_flag = 0;
    mbar_fence_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  Walk k;
  if (p.whole) {  // one (tile, head) per CTA
    const int entry = p.by_kv_heads(blockIdx.x), units = units_of(entry_tile(p, entry, kBlk), kCost);
    const int64_t at = static_cast<int64_t>(blockIdx.x - entry * cv.heads) * units;
    k.line = Stretch{at, at + units, 0, units, entry};
  } else {
    k.line = find_stretch<kThreads>(p, kBlk, kCost, kMinUnits, reinterpret_cast<int64_t*>(smem + C::offScratch));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    setmaxnreg_dec<56>();
    if (warp < 2 && lane == 0) {
      // ---------------------------------------------------------- MMA issue of tile `warp`
      const int q = warp;
      const uint32_t id_qk = (1u << 4) | ((kBlk / 2 >> 3) << 17) | ((kTile >> 4) << 24);
      const uint32_t id_pv = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(cv.dp >> 3) << 17) | ((kTile >> 4) << 24);
      const int qk_steps = (cv.d + 31) / 32;
      const uint32_t s_t = tmem + C::tS(q), o_t = tmem + C::tO(q);
      // Descriptors: the address part (in units of 16 bytes) of the first step, and what is fixed.
      const uint64_t k_desc = smem_desc(0, 2048, 128), v_desc = smem_desc(0, 128, 2048);
      const uint32_t q_at = (base + C::offQ + q * C::kOp8) >> 4, k_at = (base + C::offK) >> 4, v_at = (base + C::offV) >> 4;
      // Scores of the keys 64 h .. 64 h + 63 of the block in stage st.
      auto qk = [&](int st, int h) {
        const uint32_t ka = k_at + st * (C::kOp8 / 16) + h * 64;
#pragma unroll
        for (int i = 0; i < CH / 32; ++i)
          if (i < qk_steps)
            mma_f8_ss(s_t + 64 * h, k_desc | (q_at + i * 256), k_desc | (ka + i * 256), id_qk, i > 0 ? 1u : 0u);
        tc_commit(&bars[bS + 2 * q + h]);
      };
      // P V of those keys.
      auto pv = [&](int st, int h, uint32_t more) {
        const uint32_t va = v_at + st * (C::kOp16 / 16) + h * 64;
#pragma unroll
        for (int i = 0; i < kBlk / 32; ++i)
          mma_f16_ts(o_t, s_t + 64 * h + 8 * i, v_desc | (va + 16 * i), id_pv, i > 0 ? 1u : more);
        tc_commit(&bars[bPV + 2 * q + h]);
      };
      int g = 0, c = 0, seg = 0;  // blocks of the CTA, blocks and (tile, head)s of this tile so far
      bool ok = true;
      auto wait = [&](int bar, int n) { return ok = ok && wait_bar<true>(&bars[bar], n & 1, abort_flag); };
      while (ok && k.next(p)) {
        if (k.n_blk == 0) continue;
        if (q >= k.tiles()) {  // no rows in this tile: its stages are free as soon as they are full
          for (int n = 0; n < k.n_blk && ok; ++n, ++g) {
            if (wait(bKfull + (g & 1), g >> 1)) tc_commit(&bars[bKempty + (g & 1)]);
            if (wait(bVfull + (g & 1), g >> 1)) tc_commit(&bars[bVempty + (g & 1)]);
          }
          continue;
        }
        // S of the last (tile, head) has been read when its successor's Q is there, and its P V comes
        // before these scores in the order of issue, which is the order in which MMAs run.
        if (!wait(bQfull + q, seg) || !wait(bKfull + (g & 1), g >> 1)) break;
        tc_fence_after();
        qk(g & 1, 0);
        qk(g & 1, 1);
        tc_commit(&bars[bKempty + (g & 1)]);
        for (int n = 0; n < k.n_blk && ok; ++n, ++g, ++c) {
          const bool more = n + 1 < k.n_blk;
#pragma unroll
          for (int h = 0; h < 2 && ok; ++h) {
            if (!wait(bP + 2 * q + h, c) || (h == 0 && !wait(bVfull + (g & 1), g >> 1))) break;
            tc_fence_after();
            pv(g & 1, h, n > 0 || h > 0 ? 1u : 0u);
            if (h == 1) tc_commit(&bars[bVempty + (g & 1)]);
            if (more) {  // the next block's scores take the place of these weights, after P V
              if (h == 0 && !wait(bKfull + ((g + 1) & 1), (g + 1) >> 1)) break;
              tc_fence_after();
              qk((g + 1) & 1, h);
              if (h == 1) tc_commit(&bars[bKempty + ((g + 1) & 1)]);
            }
          }
        }
        ++seg;
      }
      tc_commit(&bars[bDrain + q]);
      wait_bar<true>(&bars[bDrain + q], 0, abort_flag, false);
    }
    __syncwarp();
    if (warp == 2) {
      // ---------------------------------------------------------- a block's cache rows
      // A block comes as `per` pieces of `unit` tokens, each within a page. Lane l keeps the page and
      // the offset in it of the piece l % 8 of the block l / 8 after the last look-up. Lane 4 i + k
      // brings, of piece i, the V rows (k = 0), the sign rows, mu or the exponents.
      const int per = kBlk / unit, piece = lane >> 2, kind = lane & 3;
      const int xoff = kind == 1 ? cv.off_bits() : (kind == 2 ? cv.off_mu() : cv.off_exp());
      const int xsize = kind == 1 ? 16 : (kind == 2 ? 2 : 1);
      const uint32_t extra = base + (kind == 1 ? C::offBits : (kind == 2 ? C::offMu : C::offExp)) + unit * piece * xsize;
      const uint32_t bar = smem_u32(&bars[bRawFull]);
      int g = 0;
      bool ok = true;
      while (ok && k.next(p)) {
        const int32_t* table = p.table + k.b * p.table_stride;
        PageAt at{-1, 0};
        for (int n = 0; n < k.n_blk; ++n, ++g) {
          if ((n & 3) == 0) {
            at.page = -1;
            const int m = n + (lane >> 3);
            if (m < k.n_blk && (lane & 7) < per)
              at = page_at(p, table, k.w.kv, k.w.block_at(k.v0 + m) * kBlk + (lane & 7) * unit);
          }
          const int page = __shfl_sync(0xffffffffu, at.page, 8 * (n & 3) + piece);
          const int off = __shfl_sync(0xffffffffu, at.off, 8 * (n & 3) + piece);
          // Bits 0, 4, .. 28 of the vote: the pieces with a page; `have`: the 16-key parts with one.
          const uint32_t vote = __ballot_sync(0xffffffffu, page >= 0 && piece < per) & 0x11111111u;
          const uint32_t have = __ballot_sync(0xffffffffu, lane < 8 && (vote >> (4 * (lane * kPageUnit / unit))) & 1u);
          if (g > 0 && !(ok = wait_warp<true>(&bars[bRawEmpty], (g - 1) & 1, abort_flag))) break;
          // No page: the rows are not seen, but what they are made into stays finite. These zeros come before
          // the arrival, which may complete the phase by itself.
          if (piece < per && page < 0 && kind > 0)
            for (int i = 0; i < unit / 16 * xsize; ++i) sts128(extra + 16 * i, 0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            page_ok[g & 3] = have;
            mbar_arrive_expect_tx(&bars[bRawFull], __popc(vote) * unit * C::kToken);
          }
          __syncwarp();
          if (piece < per && page >= 0) {
            if (kind == 0)
              tma_load_3d(base + C::offRaw + unit * piece * C::kRow, &v_map, bar, 0, off, page * cv.heads + k.head);
            else
              bulk_load(extra, cv.block(page, k.head) + xoff + off * xsize, unit * xsize, bar);
          }
          __syncwarp();
        }
      }
      // Nothing on its way when the CTA ends.
      if (g > 0) wait_bar<true>(&bars[bRawFull], (g - 1) & 1, abort_flag, false);
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ expanding K and V
    setmaxnreg_dec<88>();
    const int row = (warp - 4) * 32 + lane;  // key of the block
    int g = 0;
    bool ok = true;
    while (ok && k.next(p)) {
      for (int n = 0; n < k.n_blk; ++n, ++g) {
        const int st = g & 1;
        if (!(ok = wait_warp<true>(&bars[bRawFull], g & 1, abort_flag))) break;
        const uint4 bits = lds128(base + C::offBits + row * 16);
        const uint32_t mu = lds16(base + C::offMu + row * 2);
        const int e8 = static_cast<int8_t>(lds16(base + C::offExp + (row & ~1)) >> (8 * (row & 1)));
        // A row that nobody sees may hold a negative mu, whose sign would hide the others, or NaN: as whole
        // numbers, bits without a sign have the order of what they stand for, with NaN above all.
        const uint32_t mu_top = __reduce_max_sync(0xffffffffu, mu & 0x7fffu);
        if (lane == 0) *reinterpret_cast<volatile uint32_t*>(smem + C::offTop + (g & 3) * 16 + (warp - 4) * 4) = mu_top << 16;
        *reinterpret_cast<volatile float*>(smem + C::offScale + ((g & 3) * kBlk + row) * 4) = __uint_as_float(mu << 16);
        uint4 code[CH / 16];
#pragma unroll
        for (int c = 0; c < CH / 16; ++c)
          if (c * 16 < cv.dp) code[c] = lds128(base + C::offRaw + C::piece(row, c));
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[bRawEmpty]);
        if (g >= 2 && !(ok = wait_warp<true>(&bars[bKempty + st], ((g >> 1) - 1) & 1, abort_flag))) break;
        const uint32_t kd = base + C::offK + st * C::kOp8 + row * 16;
        const uint32_t word[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
        for (int i = 0; i < CH / 32; ++i)
          if (32 * i < cv.d) expand_signs(kd + i * 4096, word[i], 0xffffffffu);
        fence_proxy_async_smem();
        __syncwarp();
#ifdef BA_TEST_SKIP_ARRIVE
        // Test build only: the first block's arrival is withheld, so that the waits behind it run into the limit.
        if (lane == 0 && g != 0) mbar_arrive(&bars[bKfull + st]);
#else
        if (lane == 0) mbar_arrive(&bars[bKfull + st]);
#endif
        if (g >= 2 && !(ok = wait_warp<true>(&bars[bVempty + st], ((g >> 1) - 1) & 1, abort_flag))) break;
        const uint32_t vd = base + C::offV + st * C::kOp16 + row * 16;
        // A row that no query row sees may hold anything: times 0 it is finite, as its weight of 0 needs.
        const int j = k.w.block_at(k.v0 + n) * kBlk + row;
        const bool in = j < k.w.kv && (j >= k.w.lo || j < p.sinks);
        const __half2 step = __float2half2_rn(
            in ? __uint_as_float(static_cast<uint32_t>(127 + min(max(e8, kMinExp), kMaxExp)) << 23) : 0.0f);
#pragma unroll
        for (int c = 0; c < CH / 16; ++c) {
          if (c * 16 < cv.dp) {
            expand_codes(vd + (2 * c) * 2048, code[c].x, code[c].y, step);
            expand_codes(vd + (2 * c + 1) * 2048, code[c].z, code[c].w, step);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[bVfull + st]);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<184>();
    const int q = (warp - 8) >> 2, w4 = warp & 3;
    const int r = q * kTile + w4 * 32 + lane;  // row of a (tile, head)
    const uint32_t lane_base = static_cast<uint32_t>(w4 * 32) << 16;
    const uint32_t aS = tmem + lane_base + C::tS(q), aO = tmem + lane_base + C::tO(q);
    int g = 0, c = 0;
    // Q of the (tile, head) `to` and the factor of its scores, from what the preparation kernel left.
    auto write_q = [&](const Walk& to) {
      uint4 word = make_uint4(0u, 0u, 0u, 0u);
      float mu = 0.0f;
      if (r < to.w.rows) {
        const int64_t at = out_row(p, to.w, to.head, r);
        word = p.q_bits[at];
        mu = p.q_mu[at];
      }
      const uint32_t w4x[4] = {word.x, word.y, word.z, word.w};
      const uint32_t qd = base + C::offQ + q * C::kOp8 + (w4 * 32 + lane) * 16;
#pragma unroll
      for (int i = 0; i < CH / 32; ++i) {
        const int n = cv.d - 32 * i;
        if (n > 0) expand_signs(qd + i * 4096, w4x[i], low_bits(n));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[bQfull + q]);
      return fmaxf(p.scale_log2 * mu, kLeastFactor);
    };
    grid_dependency_wait();  // for the rows of q
    bool ok = true, more = k.next(p);
    float cq_next = kLeastFactor;
    if (!more && threadIdx.x == 8 * 32 && !p.whole) p.notes[blockIdx.x].last = -1;  // nothing but the start of a cut one
    if (more && q < k.tiles() && k.n_blk > 0) cq_next = write_q(k);
    while (ok && more) {
      const RowTile w = k.w;
      const int head = k.head, n_blk = k.n_blk, v0 = k.v0, slot = k.slot;
      const bool mine = q < k.tiles();  // this (tile, head) has rows in the tile
      if (threadIdx.x == 8 * 32 && !p.whole) p.notes[blockIdx.x] = JoinNote{k.entry, head, k.last};  // the last one's stays
      more = k.next(p);
      const bool write_next = more && q < k.tiles() && k.n_blk > 0;
      const float cq = cq_next;
      const bool live = mine && r < w.rows;
      const int pos = w.pos0() + p.by_group(w.r0 + r);
      const int last = live ? (p.causal ? min(pos, w.kv - 1) : w.kv - 1) : -1;
      const int wlo = p.causal && p.window > 0 ? pos - p.window + 1 : 0;
      // What every row of the warp sees.
      const int all_last = __reduce_min_sync(0xffffffffu, live ? last : 0x7fffffff);
      const int all_lo = __reduce_max_sync(0xffffffffu, live ? wlo : -0x7fffffff);
      float M = -CUDART_INF_F, l = 0.0f;
      if (!mine) g += n_blk;
      // A score passes M by more than the slack: M moves, and what there is of the row is rescaled. O
      // holds the halves before half h of block n.
      auto move_to = [&](float top, float bound, int n, int h) {
        const bool moves = top - M > kHigh;
        // The bound may grow by 1 with the scales of the keys to come.
        const float to = fminf(top - kLeastBelow, fmaxf(top - kBelow, bound + (1.0f - kMostLog2)));
        const float f = moves ? ex2_approx(M - to) : 1.0f;  // 0 for a row's first keys
        if (moves) M = to;
        l *= f;
        if (n + h > 0 && (ok = wait_warp<false>(&bars[bPV + 2 * q + 1 - h], (c - 1 + h) & 1, abort_flag))) {
          tc_fence_after();
#pragma unroll 1
          for (int i = 0; i < cv.dp; i += 16) {
            uint32_t o[16];
            tmem_ld16p(aO + i, o);
            tmem_ld_wait();
            reg_fence8(o);
            reg_fence8(o + 8);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st16p(aO + i, o);
          }
        }
      };
      auto arrive = [&](int bar) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[bar]);
      };
      // Sixteen scores of the keys from j on, -inf for those that the row does not see.
      auto read16 = [&](uint32_t from, int j, bool page, uint32_t mu, uint32_t (&s)[16]) {
        tmem_ld16p(from, s);
        const uint32_t see = page ? low_bits(last - j + 1) & (~low_bits(wlo - j) | low_bits(p.sinks - j)) : 0u;
        tmem_ld_wait();
        reg_fence8(s);
        reg_fence8(s + 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 m = *reinterpret_cast<const uint4*>(smem + mu + 16 * i);
          const uint32_t m4[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
          for (int e = 4 * i; e < 4 * i + 4; ++e)
            s[e] = (see >> e) & 1u ? __float_as_uint(__uint_as_float(s[e]) * __uint_as_float(m4[e % 4])) : 0xff800000u;
        }
      };
      // The weight of two keys as an fp16 pair; its numbers are added to `sum`.
      auto weigh = [&](float2 x, float ref, float2& sum) {
        x = __ffma2_rn(x, make_float2(cq, cq), make_float2(-ref, -ref));
        const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
        sum = __fadd2_rn(sum, e);
        const __half2 y = __floats2half2_rn(e.x, e.y);
        return *reinterpret_cast<const uint32_t*>(&y);
      };
      // Of sixteen keys with the scales at `mu`.
      auto weigh16 = [&](const uint32_t (&s)[16], uint32_t mu, uint32_t* to, float2 (&sum)[2]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 m = *reinterpret_cast<const uint4*>(smem + mu + 16 * i);
          const float2 a = __fmul2_rn(make_float2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])),
                                      make_float2(__uint_as_float(m.x), __uint_as_float(m.y)));
          const float2 b = __fmul2_rn(make_float2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])),
                                      make_float2(__uint_as_float(m.z), __uint_as_float(m.w)));
          to[2 * i] = weigh(a, M, sum[0]);
          to[2 * i + 1] = weigh(b, M, sum[1]);
        }
      };
      bool fresh = true;  // a row has seen nothing yet
      int owed = -1;      // half whose weights are on their way to tensor memory
      auto hand_over = [&] {
        tmem_st_wait();
        arrive(bP + 2 * q + owed);
      };
      for (int n = 0; n < n_blk && mine && ok; ++n, ++g, ++c) {
        const int j0 = w.block_at(v0 + n) * kBlk;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const uint32_t at = aS + 64 * h;
          const int j = j0 + 64 * h;
          const uint32_t mu = C::offScale + ((g & 3) * kBlk + 64 * h) * 4;
          if (!(ok = wait_warp<false>(&bars[bS + 2 * q + h], c & 1, abort_flag))) break;
          tc_fence_after();
          uint32_t x[2][16];
          tmem_ld16p(at, x[0]);
          if (owed >= 0) hand_over();
          const uint32_t have = page_ok[g & 3] >> (4 * h) & 15u;
          float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
          bool done = have == 15u && j + 63 <= all_last && j >= all_lo && !fresh;
          if (done) {
            uint32_t pw[32];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              tmem_ld_wait();
              reg_fence16(x[k & 1]);
              if (k < 3) tmem_ld16p(at + 16 * k + 16, x[(k + 1) & 1]);
              weigh16(x[k & 1], mu + 64 * k, pw + 8 * k, sum);
            }
            const float all = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            done = __all_sync(0xffffffffu, !live || all <= kMostSum);
            if (done) {
              l += all;
              tmem_st32p(at, pw);
            }
          }
          // The rare case in loops of 16 keys: unrolled, it took registers from the common one, which ran at
          // four fifths of its speed.
          if (!done) {
            // A mask alone needs no maximum where none can pass M by 2^15.9: |score| <= factor * d * mu. A NaN
            // among the half's scales, seen or not, fails the comparison.
            const volatile uint32_t* most = reinterpret_cast<volatile uint32_t*>(smem + C::offTop + (g & 3) * 16 + h * 8);
            const float mu_top = __uint_as_float(max(most[0], most[1]));
            const float bound = cq * (static_cast<float>(cv.d) * kBoundUp) * mu_top;
            uint32_t z[16], y[8];
            if (!__all_sync(0xffffffffu, !live || bound - M <= kMostLog2)) {
              float top = -CUDART_INF_F;
#pragma unroll 1
              for (int k = 0; k < 4; ++k) {
                read16(at + 16 * k, j + 16 * k, have >> k & 1u, mu + 64 * k, z);
#pragma unroll
                for (int i = 0; i < 16; i += 2) top = fmax3(top, __uint_as_float(z[i]), __uint_as_float(z[i + 1]));
              }
              top *= cq;
              if (__any_sync(0xffffffffu, top - M > kHigh)) {
                move_to(top, bound, n, h);
                if (!ok) break;
              }
            }
            sum[0] = sum[1] = make_float2(0.0f, 0.0f);
            // Upwards: the weights lie over scores that have been read.
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              read16(at + 16 * k, j + 16 * k, have >> k & 1u, mu + 64 * k, z);
              const float ref = M == -CUDART_INF_F ? 0.0f : M;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                y[i] = weigh(make_float2(__uint_as_float(z[2 * i]), __uint_as_float(z[2 * i + 1])), ref, sum[i & 1]);
              tmem_st8(at + 8 * k, y);
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            fresh = __any_sync(0xffffffffu, live && M == -CUDART_INF_F);
          }
          owed = h;
        }
      }
      if (owed >= 0) hand_over();
      if (!ok) break;
      // The next (tile, head)'s scores can be made while this one's rows are written.
      if (write_next) cq_next = write_q(k);
      if (!mine) continue;
      // ------------------------------------------------------------ the rows' results
      if (n_blk > 0 && !(ok = wait_warp<false>(&bars[bPV + 2 * q + 1], (c - 1) & 1, abort_flag))) break;
      tc_fence_after();
      const int64_t out = out_row(p, w, head, r);
      const float inv = slot >= 0 ? 1.0f : (l > 0.0f ? 1.0f / l : 0.0f);
      const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + slot) * (2 * kTile) + r;
      const bool wide = cv.d % 8 == 0;
#pragma unroll 1
      for (int j = 0; j < cv.dp; j += 16) {
        uint32_t o[16];
        __syncwarp();
        if (n_blk > 0) {
          tmem_ld16p(aO + j, o);
          tmem_ld_wait();
          reg_fence8(o);
          reg_fence8(o + 8);
        }
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = n_blk > 0 ? __uint_as_float(o[i]) * inv : 0.0f;
        if (!live) {
        } else if (slot >= 0) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + part * cv.dp + j);
#pragma unroll
          for (int i = 0; i < 4; ++i) dst[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
        } else if (wide && p.o_dt != BA_F32) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = f[8 * h + 2 * i], bb = f[8 * h + 2 * i + 1];
              if (p.o_dt == BA_F16) {
                const __half2 y = __floats2half2_rn(a, bb);
                x[i] = *reinterpret_cast<const uint32_t*>(&y);
              } else {
                const __nv_bfloat162 y = __floats2bfloat162_rn(a, bb);
                x[i] = *reinterpret_cast<const uint32_t*>(&y);
              }
            }
            if (j + 8 * h < cv.d)
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + out * cv.d + j + 8 * h) =
                  make_uint4(x[0], x[1], x[2], x[3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (j + i < cv.d) store_out(p.o, out * cv.d + j + i, f[i], p.o_dt);
        }
      }
      if (live) {
        if (slot >= 0)
          p.part_ml[part] = make_float2(M, l);
        else if (p.lse != nullptr)
          p.lse[out] = l > 0.0f ? (M + log2f(l)) * CUDART_LN2_F : -CUDART_INF_F;
      }
    }
  }
  grid_dependency_wait();  // also without work: this grid must not complete before the one before it
  tc_fence_before();
  named_barrier_sync(1, kThreads);
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int CH>
cudaError_t launch_chunk(const PagedAttnParams& p, int dt, cudaStream_t s) {
  // At least half of the shared memory: the CTA owns all of the SM's tensor memory.
  const int smem = std::max(Cfg<CH>::kBytes, 116 * 1024);
  cudaError_t e = allow_smem<paged_chunk_kernel<CH>>(smem);
  if (e != cudaSuccess) return e;
  const int unit = v_unit(p.cache, kBlk);
  CUtensorMap map;
  if (!v_rows_map(p.cache, CH, unit, &map)) return cudaErrorInvalidValue;
  const unsigned q_grid = static_cast<unsigned>(ceil_div(p.T * p.heads, 8));
  uint4* bits = const_cast<uint4*>(p.q_bits);
  float* mu = const_cast<float*>(p.q_mu);
  if (dt == BA_F16)
    paged_q_kernel<__half><<<q_grid, 256, 0, s>>>(p, bits, mu);
  else
    paged_q_kernel<__nv_bfloat16><<<q_grid, 256, 0, s>>>(p, bits, mu);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, paged_chunk_kernel<CH>, p, unit, map)) != cudaSuccess) return e;
  return p.whole ? cudaSuccess : launch_line_join(p, kBlk, s);
}

}  // namespace

cudaError_t launch_paged_chunk(const PagedAttnParams& p, int dt, cudaStream_t s) {
  return p.cache.dp > 64 ? launch_chunk<128>(p, dt, s) : launch_chunk<64>(p, dt, s);
}

void paged_chunk_plan(PagedAttnParams* p, int sms) {
  const int64_t blocks = most_blocks(*p, p->row_tile, kBlk), tiles = static_cast<int64_t>(p->B) * p->row_tiles * p->cache.heads;
  p->cluster = 1;
  // Cutting (tile, head)s to fill the GPU costs what kWholeBlocks blocks do (finding the cuts, and the
  // second launch): 80 of 12 blocks took 38 us whole and 58 us cut, 80 of 23 blocks 62 and 73 us, 8 of 8
  // blocks 27 and 31 us, but 8 of 16 blocks 42 and 35 us.
  const int64_t even = std::max<int64_t>((blocks + kCost) * tiles / sms, kMinUnits - kCost);
  p->whole = tiles <= sms && blocks - even <= kWholeBlocks ? 1 : 0;
  p->ctas = p->whole ? static_cast<int>(tiles) : static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(sms, (blocks + kCost) * tiles / kMinUnits)));
}

static cudaError_t read_chunk_status(int* value, cudaStream_t s) { return read_word(g_chunk_status, value, s); }
static cudaError_t clear_chunk_status(cudaStream_t s) { return clear_word(g_chunk_status, s); }
StatusWord chunk_status() { return {read_chunk_status, clear_chunk_status}; }

}  // namespace binattn
