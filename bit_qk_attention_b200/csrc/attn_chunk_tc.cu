// Attention of many query rows over the paged cache on 5th-generation tensor cores (sm_100a).
//
// A CTA takes 256 rows (new tokens x query heads of a group, which share every key) of one sequence
// and KV head against the 128-key blocks that any of them sees, as two tiles of 128 rows whose MMAs
// and softmax alternate. The products run on tcgen05 with fp32 accumulators in tensor memory:
//   S = Q K^T  bf16: Q is +-1, K is +-mu_j, so S = mu_j (d - 2 popc) comes out exact
//   O += P V   fp16: P = 2^(s - M), V = code 2^e, both numbers of the cache exact in their type
// The cache holds K in bits and V in bytes, so the operands are made in shared memory:
//   * Four expanding warps take 32 keys of a block each. A warp copies its rows with cp.async into
//     a stage of its own, one key per lane, reads them into registers, starts the next block's copy
//     into the same stage, and writes the 16-bit operands: two instructions per pair of K channels
//     (the pair is (c, c + 16), so that one shift and one mask place both signs; Q has the same
//     order, and a dot product does not mind), seven per four V channels.
//   * One thread issues the MMAs. K and V operands are double-buffered.
//   * Two warpgroups of softmax, one per tile, one thread per row: the row of S comes from tensor
//     memory, P goes back over it. The running maximum M moves, and O is rescaled in tensor memory,
//     only when a score passes it by more than 2^8, which hardly ever happens after the first
//     blocks; the weights stay far inside fp16 and the sums are fp32.
// A block of 256 x 128 scores costs 2048 cycles of exponentials (16 per cycle and SM) and as many
// of MMAs (4096 products per cycle); that is the bound.
//
// Every wait is bounded (1 s): on expiry the kernel records a timeout in a device status word, all
// roles leave, copies and MMAs in flight are waited for, and tensor memory is freed.
#include <math_constants.h>

#include <algorithm>

#include "kernels.h"
#include "paged.cuh"
#include "tc_ptx.cuh"

namespace binattn {

__device__ int g_chunk_status = 0;

namespace {

using namespace ptx;

constexpr int kBlk = 128;      // keys per block: N of QK, K of PV
constexpr int kTile = 128;     // rows per tile: M
constexpr int kMinBlocks = 4;  // blocks a split takes at least
constexpr int kThreads = 512;  // service, expanding and two softmax warpgroups
constexpr float kSlack = 8.0f;
constexpr uint64_t kTimeoutNs = 1000000000ull;

template <int CH>  // channels of the operands: 64 or 128 (>= d)
struct Cfg {
  static constexpr int kOp = kBlk * CH * 2;  // bytes of an operand tile of 128 rows
  static constexpr int kRow = CH;            // bytes of a V row in a stage
  static constexpr int offBits = 32 * kRow;
  static constexpr int offMu = offBits + 32 * 16;
  static constexpr int offExp = offMu + 32 * 2;
  static constexpr int kStage = offExp + 32;  // a warp's 32 keys
  static constexpr int offQ = 0;
  static constexpr int offK = offQ + 2 * kOp;
  static constexpr int offV = offK + 2 * kOp;
  static constexpr int offRaw = offV + 2 * kOp;
  static constexpr int offBar = offRaw + 4 * kStage;
  static constexpr int kNumBars = 17;
  static constexpr int offMisc = offBar + kNumBars * 8;  // tensor memory base, abort flag, page masks [4][4]
  static constexpr int kBytes = offMisc + 8 + 16 + 8;
  // Tensor memory: S of tile q (P over its first half), then O.
  static __host__ __device__ constexpr uint32_t tS(int q) { return q * 128; }
  static __host__ __device__ constexpr uint32_t tO(int q) { return 256 + q * CH; }
  // 16-byte piece c of key j's V row in a stage, moved so that eight neighbouring keys' loads of
  // one piece touch all banks.
  static __device__ __forceinline__ int piece(int j, int c) {
    return kRow == 128 ? (j * 8 + (c ^ (j & 7))) * 16 : (j * 4 + (c ^ ((j >> 1) & 3))) * 16;
  }
};

// Barriers.
constexpr int bKfull = 0, bKempty = 2, bVfull = 4, bVempty = 6, bQfull = 8, bSfull = 10, bPfull = 12, bPV = 14,
              bDrain = 16;

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag, bool yield = true) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (yield && *abort_flag) return false;
    if (globaltimer() - t0 > kTimeoutNs) {
      *abort_flag = 1;
      atomicExch(&g_chunk_status, 1);
      return false;
    }
  }
}

__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag));
}

// Sign bits of 32 channels -> 16 pairs (channel p, channel p + 16) of +-m, m the bf16 pair (mu, mu):
// four 16-byte pieces of a K-major operand row. keep[i] masks channels that do not exist.
__device__ __forceinline__ void expand_signs(uint32_t dst, uint32_t word, uint32_t m, uint32_t live) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = 4 * c + i;
      const uint32_t mm = live == 0xffffffffu
                              ? m
                              : ((live >> p) & 1u ? m & 0xffffu : 0u) | ((live >> (p + 16)) & 1u ? m & 0xffff0000u : 0u);
      x[i] = ((word << (15 - p)) & 0x80008000u) ^ mm;
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

// Sign words and sum of |x| of one row of q.
template <typename T>
__device__ __forceinline__ float read_row(const T* src, int d, bool wide, uint32_t (&word)[4]) {
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    word[k] = 0u;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int c0 = 32 * k + 8 * c;
      float f[8];
      if (wide) {
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (c0 < d) u = __ldg(reinterpret_cast<const uint4*>(src + c0));
        unpack8<T>(u, f);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = c0 + i < d ? load1<T>(src + c0 + i) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        word[k] |= (f[i] < 0.0f ? 1u : 0u) << (8 * c + i);
        sum += fabsf(f[i]);
      }
    }
  }
  return sum;
}

template <int CH>
__global__ void __launch_bounds__(kThreads, 1) paged_chunk_kernel(PagedAttnParams p, int q_f16, int q_wide) {
  using C = Cfg<CH>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::offBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::offMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::offMisc + 4);
  volatile uint8_t* page_ok = smem + C::offMisc + 8;  // [block % 4][warp]: which 16-key halves have a page
  const CacheView& cv = p.cache;
  // The last row tiles come first: with a causal mask they have the most keys.
  int b, tile, head, split;
  cta_of(p, gridDim.x - 1 - blockIdx.x, p.nsplit, b, tile, head, split);
  const RowTile w = row_tile(p, b, tile, kBlk);
  if (w.rows <= 0) return;
  const int used = splits_used(p, w.nblk);
  if (split >= used) return;
  const int v0 = static_cast<int>(static_cast<int64_t>(w.nblk) * split / used);
  const int n_blk = static_cast<int>(static_cast<int64_t>(w.nblk) * (split + 1) / used) - v0;
  const int tiles = w.rows > kTile ? 2 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[bKfull + i], 4);
      mbar_init(&bars[bVfull + i], 4);
      mbar_init(&bars[bKempty + i], 1);
      mbar_init(&bars[bVempty + i], 1);
      mbar_init(&bars[bQfull + i], 4);
      mbar_init(&bars[bSfull + i], 1);
      mbar_init(&bars[bPfull + i], 4);
      mbar_init(&bars[bPV + i], 1);
    }
    mbar_init(&bars[bDrain], 1);
    *abort_flag = 0;
    mbar_fence_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t base = smem_u32(smem);

  if (warp < 4) {
    setmaxnreg_dec<56>();
    if (warp == 0 && lane == 0 && n_blk > 0) {
      // ---------------------------------------------------------- MMA issue
      const uint32_t id_qk = (1u << 4) | (1u << 7) | (1u << 10) | ((kBlk >> 3) << 17) | ((kTile >> 4) << 24);
      const uint32_t id_pv = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(cv.dp >> 3) << 17) | ((kTile >> 4) << 24);
      const int qk_steps = 2 * ((cv.d + 31) / 32);
      auto qk = [&](int q, int n) -> bool {
        if (n == 0 && !wait_bar(&bars[bQfull + q], 0, abort_flag)) return false;
        if (q == 0 && !wait_bar(&bars[bKfull + (n & 1)], (n >> 1) & 1, abort_flag)) return false;
        tc_fence_after();
        const uint32_t qa = base + C::offQ + q * C::kOp, ka = base + C::offK + (n & 1) * C::kOp;
        for (int k = 0; k < qk_steps; ++k)
          mma_f16_ss(tmem + C::tS(q), smem_desc(qa + k * 4096, 2048, 128), smem_desc(ka + k * 4096, 2048, 128), id_qk,
                     k > 0 ? 1u : 0u);
        tc_commit(&bars[bSfull + q]);
        if (q == tiles - 1) tc_commit(&bars[bKempty + (n & 1)]);
        return true;
      };
      auto pv = [&](int q, int n) -> bool {
        if (!wait_bar(&bars[bPfull + q], n & 1, abort_flag)) return false;
        if (q == 0 && !wait_bar(&bars[bVfull + (n & 1)], (n >> 1) & 1, abort_flag)) return false;
        tc_fence_after();
        const uint32_t va = base + C::offV + (n & 1) * C::kOp;
#pragma unroll
        for (int k = 0; k < kBlk / 16; ++k)
          mma_f16_ts(tmem + C::tO(q), tmem + C::tS(q) + 8 * k, smem_desc(va + 256 * k, 128, 2048), id_pv,
                     n > 0 || k > 0 ? 1u : 0u);
        tc_commit(&bars[bPV + q]);
        if (q == tiles - 1) tc_commit(&bars[bVempty + (n & 1)]);
        return true;
      };
      // P of a tile lies over its S, and the MMAs of a CTA run in the order of their issue: S is
      // rewritten by the next QK only after PV has read P.
      bool ok = qk(0, 0) && (tiles == 1 || qk(1, 0));
      for (int n = 0; n < n_blk && ok; ++n)
        for (int q = 0; q < tiles && ok; ++q) ok = pv(q, n) && (n + 1 == n_blk || qk(q, n + 1));
      tc_commit(&bars[bDrain]);
      wait_bar(&bars[bDrain], 0, abort_flag, false);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ expanding K and V
    setmaxnreg_dec<88>();
    const int ew = warp - 4;
    const uint32_t raw = base + C::offRaw + ew * C::kStage;
    const int32_t* table = p.table + b * p.table_stride;
    PageAt at{-1, 0};
    uint32_t ok_next = 0;
    auto issue = [&](int n) {
      if (n >= n_blk) return;
      if ((n & 15) == 0) {
        at.page = -1;
        if (n + (lane >> 1) < n_blk)
          at = page_at(p, table, w.kv, w.block_at(v0 + n + (lane >> 1)) * kBlk + ew * 32 + (lane & 1) * kPageUnit);
      }
      ok_next = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int page = __shfl_sync(0xffffffffu, at.page, 2 * (n & 15) + h);
        const int off = __shfl_sync(0xffffffffu, at.off, 2 * (n & 15) + h);
        const bool ok = page >= 0;
        ok_next |= (ok ? 1u : 0u) << h;
        const uint8_t* blk = ok ? cv.block(page, head) : cv.data;
        constexpr int PPR = C::kRow / 16;
#pragma unroll
        for (int i = 0; i < kPageUnit * PPR / 32; ++i) {
          const int idx = lane + 32 * i, j = idx / PPR, c = idx % PPR;
          if (c * 16 < cv.dp)
            cp_async16(raw + C::piece(kPageUnit * h + j, c), ok ? blk + (off + j) * cv.dp + c * 16 : blk, ok);
        }
        if (lane < 19) {
          const uint8_t* src = lane < 16 ? blk + cv.off_bits() + (off + lane) * 16
                                         : (lane < 18 ? blk + cv.off_mu() + off * 2 + (lane - 16) * 16
                                                      : blk + cv.off_exp() + off);
          const uint32_t to = lane < 16 ? C::offBits + (kPageUnit * h + lane) * 16
                                        : (lane < 18 ? C::offMu + kPageUnit * h * 2 + (lane - 16) * 16
                                                     : C::offExp + kPageUnit * h);
          cp_async16(raw + to, ok ? src : blk, ok);
        }
      }
      cp_async_commit();
    };
    issue(0);
    const int row = ew * 32 + lane;  // key of the block
    for (int n = 0; n < n_blk; ++n) {
      cp_async_wait<0>();
      __syncwarp();
      const uint4 bits = lds128(raw + C::offBits + lane * 16);
      const uint32_t mu = lds16(raw + C::offMu + lane * 2);
      const int e8 = static_cast<int8_t>(lds16(raw + C::offExp + (lane & ~1)) >> (8 * (lane & 1)));
      uint4 code[CH / 16];
#pragma unroll
      for (int c = 0; c < CH / 16; ++c)
        if (c * 16 < cv.dp) code[c] = lds128(raw + C::piece(lane, c));
      if (lane == 0) page_ok[(n & 3) * 4 + ew] = static_cast<uint8_t>(ok_next);
      __syncwarp();
      issue(n + 1);
      const int st = n & 1;
      if (n >= 2 && !wait_warp(&bars[bKempty + st], ((n >> 1) - 1) & 1, abort_flag)) break;
      const uint32_t kd = base + C::offK + st * C::kOp + row * 16;
      const uint32_t word[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
      for (int k = 0; k < CH / 32; ++k)
        if (32 * k < cv.d) expand_signs(kd + k * 8192, word[k], mu | (mu << 16), 0xffffffffu);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[bKfull + st]);
      if (n >= 2 && !wait_warp(&bars[bVempty + st], ((n >> 1) - 1) & 1, abort_flag)) break;
      const uint32_t vd = base + C::offV + st * C::kOp + row * 16;
      // A row behind the sequence may hold anything: times 0 it is finite, as its weight of 0 needs.
      const bool in = w.block_at(v0 + n) * kBlk + row < w.kv;
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
    cp_async_wait<0>();
  } else {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<184>();
    const int q = (warp - 8) >> 2, w4 = warp & 3;
    const int r = q * kTile + w4 * 32 + lane;  // row of the CTA
    const bool live = r < w.rows;
    const int i = (w.r0 + r) / p.group, hq = head * p.group + (w.r0 + r) % p.group;
    const uint32_t lane_base = static_cast<uint32_t>(w4 * 32) << 16;
    const uint32_t aS = tmem + lane_base + C::tS(q), aO = tmem + lane_base + C::tO(q);
    float cq = 1e-30f;  // above 0 also for a row of zeros, so that -inf in masked places stays -inf
    if (q < tiles) {
      uint32_t word[4] = {0u, 0u, 0u, 0u};
      if (live && n_blk > 0) {
        const int64_t at = (w.t0 + i) * p.q_stride_t + hq * p.q_stride_h;
        const float sum = q_f16 ? read_row(static_cast<const __half*>(p.q) + at, cv.d, q_wide, word)
                                : read_row(static_cast<const __nv_bfloat16*>(p.q) + at, cv.d, q_wide, word);
        cq = fmaxf(p.scale_log2 * (sum / static_cast<float>(cv.d)), cq);
      }
      const uint32_t qd = base + C::offQ + q * C::kOp + (w4 * 32 + lane) * 16;
#pragma unroll
      for (int k = 0; k < CH / 32; ++k) {
        const int n = cv.d - 32 * k;
        if (n > 0) expand_signs(qd + k * 8192, word[k], 0x3f803f80u, n >= 32 ? 0xffffffffu : (1u << n) - 1u);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[bQfull + q]);
    }
    const int pos = w.pos0() + i;
    const int last = live ? (p.causal ? min(pos, w.kv - 1) : w.kv - 1) : -1;
    const int wlo = p.causal && p.window > 0 ? pos - p.window + 1 : 0;
    // What every row of the warp sees.
    const int all_last = __reduce_min_sync(0xffffffffu, live ? last : 0x7fffffff);
    const int all_lo = __reduce_max_sync(0xffffffffu, live ? wlo : -0x7fffffff);
    float M = -CUDART_INF_F, l = 0.0f;
    bool ok = q < tiles;
    for (int n = 0; n < n_blk && ok; ++n) {
      if (!(ok = wait_warp(&bars[bSfull + q], n & 1, abort_flag))) break;
      tc_fence_after();
      uint32_t s[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32p(aS + 32 * c, s + 32 * c);
      const int j0 = w.block_at(v0 + n) * kBlk;
      const uint32_t have = *reinterpret_cast<volatile uint32_t*>(smem + C::offMisc + 8 + (n & 3) * 4);
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 16; ++c) reg_fence8(s + 8 * c);
      if (!(have == 0x03030303u && j0 + kBlk - 1 <= all_last && j0 >= all_lo)) {
#pragma unroll
        for (int c = 0; c < kBlk; ++c) {
          const int j = j0 + c;
          const bool see = ((have >> (8 * (c / 32) + (c / 16) % 2)) & 1u) && j <= last && (j >= wlo || j < p.sinks);
          if (!see) s[c] = 0xff800000u;  // -inf
        }
      }
      float mx[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) mx[k] = fmax3(__uint_as_float(s[k]), __uint_as_float(s[k + 4]), __uint_as_float(s[k + 8]));
#pragma unroll
      for (int c = 12; c < 124; c += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = fmax3(mx[k], __uint_as_float(s[c + k]), __uint_as_float(s[c + 4 + k]));
#pragma unroll
      for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], __uint_as_float(s[124 + k]));
      const float top = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * cq;
      if (__any_sync(0xffffffffu, top > M + kSlack)) {
        const bool moves = top > M + kSlack;
        const float f = moves ? ex2_approx(M - top) : 1.0f;  // 0 for a row's first keys
        if (moves) M = top;
        l *= f;
        if (n > 0) {
          if (!(ok = wait_warp(&bars[bPV + q], (n - 1) & 1, abort_flag))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < cv.dp; c += 16) {
            uint32_t o[16];
            tmem_ld16p(aO + c, o);
            tmem_ld_wait();
            reg_fence8(o);
            reg_fence8(o + 8);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st16p(aO + c, o);
          }
        }
      }
      const float ref = M == -CUDART_INF_F ? 0.0f : M;
      const float2 c2 = make_float2(cq, cq), m2 = make_float2(-ref, -ref);
      float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
      for (int c = 0; c < 64; ++c) {
        const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), c2, m2);
        const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
        sum[c & 1] = __fadd2_rn(sum[c & 1], e);
        const __half2 h = __floats2half2_rn(e.x, e.y);
        s[c] = *reinterpret_cast<const uint32_t*>(&h);
      }
      tmem_st32p(aS, s);
      tmem_st32p(aS + 32, s + 32);
      sum[0] = __fadd2_rn(sum[0], sum[1]);
      l += sum[0].x + sum[0].y;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[bPfull + q]);
    }
    // ------------------------------------------------------------ the rows' results
    if (q < tiles && n_blk > 0 && ok) ok = wait_warp(&bars[bPV + q], (n_blk - 1) & 1, abort_flag);
    tc_fence_after();
    if (ok) {
      const int64_t out = (w.t0 + i) * p.heads + hq;
      const float inv = used > 1 ? 1.0f : (l > 0.0f ? 1.0f / l : 0.0f);
      const int64_t part = split * p.T * p.heads + out;
      const bool wide = cv.d % 8 == 0;
#pragma unroll 1
      for (int c = 0; c < cv.dp; c += 16) {
        uint32_t o[16];
        __syncwarp();
        if (n_blk > 0) {
          tmem_ld16p(aO + c, o);
          tmem_ld_wait();
          reg_fence8(o);
          reg_fence8(o + 8);
        }
        float f[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) f[k] = n_blk > 0 ? __uint_as_float(o[k]) * inv : 0.0f;
        if (!live) {
        } else if (used > 1) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + part * cv.dp + c);
#pragma unroll
          for (int k = 0; k < 4; ++k) dst[k] = make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
        } else if (wide && p.o_dt != BA_F32) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float a = f[8 * h + 2 * k], bb = f[8 * h + 2 * k + 1];
              if (p.o_dt == BA_F16) {
                const __half2 y = __floats2half2_rn(a, bb);
                x[k] = *reinterpret_cast<const uint32_t*>(&y);
              } else {
                const __nv_bfloat162 y = __floats2bfloat162_rn(a, bb);
                x[k] = *reinterpret_cast<const uint32_t*>(&y);
              }
            }
            if (c + 8 * h < cv.d)
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + out * cv.d + c + 8 * h) =
                  make_uint4(x[0], x[1], x[2], x[3]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (c + k < cv.d) store_out(p.o, out * cv.d + c + k, f[k], p.o_dt);
        }
      }
      if (live) {
        if (used > 1)
          p.part_ml[part] = make_float2(M, l);
        else if (p.lse != nullptr)
          p.lse[out] = l > 0.0f ? (M + log2f(l)) * CUDART_LN2_F : -CUDART_INF_F;
      }
    }
  }
  allow_dependents();
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
  const bool wide = p.cache.d % 8 == 0 && reinterpret_cast<uintptr_t>(p.q) % 16 == 0 &&
                    (p.q_stride_t | p.q_stride_h) % 8 == 0;
  const int64_t grid = static_cast<int64_t>(p.B) * p.row_tiles * p.cache.heads * p.nsplit;
  paged_chunk_kernel<CH><<<static_cast<unsigned>(grid), kThreads, smem, s>>>(p, dt == BA_F16 ? 1 : 0, wide ? 1 : 0);
  if ((e = cudaGetLastError()) != cudaSuccess || p.nsplit == 1) return e;
  return launch_paged_join(p, kBlk, s);
}

}  // namespace

cudaError_t launch_paged_chunk(const PagedAttnParams& p, int dt, cudaStream_t s) {
  return p.cache.dp > 64 ? launch_chunk<128>(p, dt, s) : launch_chunk<64>(p, dt, s);
}

int paged_chunk_split_blocks(const PagedAttnParams& p, int sms, int* max_blocks) {
  int64_t keys = p.max_kv_len;
  if (p.causal && p.window > 0)
    keys = std::min<int64_t>(keys, static_cast<int64_t>(p.window) + p.row_tile / p.group + p.sinks + 2 * kBlk);
  const int64_t blocks = ceil_div(keys, kBlk), tiles = static_cast<int64_t>(p.B) * p.row_tiles * p.cache.heads;
  *max_blocks = static_cast<int>(blocks);
  const int64_t parts = std::max<int64_t>(1, std::min(sms / tiles, blocks / kMinBlocks));
  return static_cast<int>(std::max<int64_t>(1, ceil_div(blocks, parts)));
}

cudaError_t read_and_clear_chunk_status(int* value, cudaStream_t s) {
  return read_and_clear_status(g_chunk_status, value, s);
}

}  // namespace binattn
