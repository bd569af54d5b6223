// Attention of few query rows over the paged cache (sm_100a): decoding and drafts.
//
// With few rows per KV head the kernel is bound by reading the cache once: dp + 19 bytes per token
// and head, and at HBM's rate a key of 147 bytes leaves an SM some 6.5 cycles. So the work per key
// is kept small:
//   * A CTA takes one sequence, one KV head, up to 8 NR rows (new tokens x heads of the group, which
//     share every key) and a part of the key axis. Each of its warps walks 32-key blocks of its own
//     through a ring of cp.async stages, with no synchronisation between warps until the end.
//   * Scores are products of whole numbers on the tensor cores (mma.sync m16n8k32, int8). With K's
//     sign bits k in {0, 1} and Q in {-1, +1}, x = sum q - 2 sum q k. The bits need no expanding: a
//     word masked by 0x01010101 << s holds four of them as bytes of value 2^s, and the byte of Q that
//     meets it holds 2^(6 - s), so that every product is 64 q k. (XOR and popc per (key, row) pair
//     took three times the instructions for 8 rows.) The accumulators start at the bit pattern of
//     1.5 * 2^23, which makes the whole-number result a float as it is.
//   * P.V is a product of whole numbers too, V^T P^T: 16 channels x 32 keys of V codes against 32
//     keys x 8 rows, so that 8 rows fill the instruction (a 128-row tcgen05 tile would be mostly
//     empty). The codes go from ldmatrix, which transposes bytes, into the product as they are;
//     making fp16 numbers of them took more instructions than all the rest. The weights of a block
//     are 16-bit fixed-point numbers, round(65280 2^(s - m)) with m the row's maximum in the block:
//     a product each for their high and low bytes, whose exact sums are weighted by 2^(m - M) and
//     added in fp32. A weight's error is 2^-17 of the block's largest.
//   * A value row's exponent e_j joins the score instead of the codes: the weight is
//     2^(s_j + e_j - m) with m a maximum of s_j + e_j, and the softmax sum adds weight * 2^-e_j. The
//     reference M moves (and the sums are rescaled) only when a block's m passes it by 2^40, far
//     inside fp32's range, so that hardly any block rescales.
//   * Parts of the key axis leave (M, sum, unnormalised o) in fp32, joined by a second kernel that
//     is launched as a programmatic dependent. Short sequences use fewer parts, down to one, which
//     writes the result itself.
#include <math_constants.h>

#include <algorithm>

#include "kernels.h"
#include "paged.cuh"

namespace binattn {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kBlk = 32;       // keys per stage of a warp
constexpr int kStages = 3;
constexpr int kCost = 12;       // blocks that a CTA could do while it starts and ends a (tile, head)
constexpr float kSlack = 40.0f;  // log2 by which a block's maximum may pass the reference
constexpr float kUnit = 65280.0f;  // weight 1 in fixed point: 255 * 256
constexpr int kMagicBits = 0x4B400000;  // 1.5 * 2^23
constexpr float kMagic = 12582912.0f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  const uint4 u = lds128(a);
  return make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts_f32(uint32_t a, float x) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory");
}

// c += A B: A 16 x 32 signed bytes (rows g and g + 8 of Q), B 32 x 8 unsigned bytes (keys' bits).
__device__ __forceinline__ void mma_i8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// c = start + A B.
__device__ __forceinline__ void mma_i8_first(int (&c)[4], const int (&start)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(start[0]), "r"(start[1]), "r"(start[2]),
        "r"(start[3]));
}

// Two 16 x 16 matrices of bytes, transposed. Lanes 0-15 and 16-31 give the rows' addresses; the lane
// (g, t) gets, of each matrix, columns g and g + 8 of rows 4 t .. 4 t + 3.
__device__ __forceinline__ void ldmatrix_t8(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}

// Whole-number results (kMagicBits + n, |n| < 2^22) as floats n.
__device__ __forceinline__ float2 whole(int x, int y) {
  return __fadd2_rn(make_float2(__int_as_float(x), __int_as_float(y)), make_float2(-kMagic, -kMagic));
}

// Shared memory of a warp: V rows of kRow bytes for each stage (16-byte pieces permuted), then each
// stage's sign rows, mu and exponents. Once a block's sign rows are read, what its scores need per
// key as floats (mu, e, 2^-e) takes their place. Four CTAs of four warps just fit an SM.
template <int CPG>  // eighths of the channels: 16 (rows of 128 bytes) or 8 (rows of 64)
struct Ring {
  static constexpr int kRow = CPG * 8;
  static constexpr int kV = kBlk * kRow;
  static constexpr int offX = kStages * kV;
  static constexpr int xMu = kBlk * 16, xExp = xMu + kBlk * 2, kX = xExp + kBlk;
  static constexpr int kBytes = offX + kStages * kX;
  static_assert(3 * kBlk * 4 <= xMu, "the floats replace the sign rows");
  // Byte offset of the 16-byte piece c of key j: eight neighbouring keys' pieces c lie in
  // different banks.
  static __device__ __forceinline__ int piece(int j, int c) {
    return kRow == 128 ? (j * 8 + (c ^ (j & 7))) * 16 : (j * 4 + (c ^ ((j >> 1) & 3))) * 16;
  }
};

// One row of q by a warp: sign words and sum of |x|.
template <typename T>
__device__ __forceinline__ void scan_row(const T* src, int d, int lane, uint32_t (&word)[4], float& sum) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = 32 * k + lane;
    const float x = c < d ? load1<T>(src + c) : 0.0f;
    word[k] = __ballot_sync(0xffffffffu, x < 0.0f);
    sum += fabsf(x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
}

template <int CPG, int NR, bool FULL>  // FULL: dp is the whole CPG * 8
__global__ void __launch_bounds__(kThreads, NR == 1 ? 4 : 3) paged_decode_kernel(PagedAttnParams p, int q_f16) {
  using S = Ring<CPG>;
  constexpr int MT = CPG / 2;  // 16-channel tiles
  constexpr int R = 8 * NR;    // rows of a CTA
  constexpr int CH = CPG * 8;  // channels of the accumulators (>= d)
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t s_bits[R][4];
  __shared__ float s_mu[R];
  __shared__ float2 s_ml[kWarps][R];

  allow_dependents();
  const CacheView& cv = p.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // The V stages of all warps come first (they start on 128 bytes).
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const uint32_t vring = base + warp * S::offX, xring = base + kWarps * S::offX + warp * kStages * S::kX;
  Stretch line{};
  if (p.ctas > 0) {
    line = find_stretch<kThreads>(p, kBlk, kCost, kWarps);
    if (line.at >= line.end) {
      if (threadIdx.x == 0) p.notes[blockIdx.x].last = -1;
      return;
    }
  } else {
    line.entry = blockIdx.x / cv.heads;
  }

  for (bool more = true; more;) {
  // The next (tile, head) of the CTA: its blocks v0 .. v1 - 1 of all.
  const RowTile w = entry_tile(p, line.entry, kBlk);
  const int b = line.entry / p.row_tiles;
  int head = blockIdx.x % cv.heads, v0 = 0, v1 = w.nblk, slot = -1;  // slot -1: nothing is cut
  if (p.ctas > 0) {
    const int units = units_of(w, kCost);
    if (units == 0) {  // a tile without rows
      ++line.entry;
      continue;
    }
    const int entry = line.entry;
    const int64_t in = line.at - line.base;
    head = static_cast<int>(in / units);
    const int u0 = static_cast<int>(in - static_cast<int64_t>(head) * units);
    const int u1 = static_cast<int>(min(static_cast<int64_t>(units), u0 + line.end - line.at));
    const int64_t stop = line.at + (units - u0);  // where the (tile, head) ends
    v0 = max(0, u0 - kCost);
    v1 = max(0, u1 - kCost);
    if (v0 > 0 || v1 < w.nblk) slot = v0 > 0 ? 0 : 1;
    line.at += u1 - u0;
    more = line.at < line.end;
    if (u1 == units && head == cv.heads - 1) {
      line.base += static_cast<int64_t>(units) * cv.heads;
      ++line.entry;
    }
    const bool none = v1 == 0 && u1 < units;  // cut before the first block: all of it is the next CTA's
    if (!more && threadIdx.x == 0)
      p.notes[blockIdx.x] = JoinNote{entry, head, slot == 1 && !none ? static_cast<int>((stop - 1) / line.per) : -1};
    if (none) continue;
  } else {
    more = false;
    if (w.rows <= 0) return;
  }

  // The warp's blocks are v0 + warp, v0 + warp + kWarps, ... Lane l keeps the page and the offset
  // in it of the 16 tokens (l % 2) of the block l / 2 after the last look-up: 16 blocks at a time.
  const int nmine = max(0, (v1 - v0 - warp + kWarps - 1) / kWarps);
  const int32_t* table = p.table + b * p.table_stride;
  uint64_t at = 0;    // V rows of those 16 tokens, 0 where there is no page
  int at_off = 0;     // their offset in the page
  uint32_t seen = 0;  // two bits per stage: which halves of the block have a page
  const int dp = FULL ? CH : cv.dp;
  constexpr int PPR = S::kRow / 16;   // pieces of a V row
  constexpr int RPI = 32 / PPR;       // rows that the warp copies per instruction
  const int vrow = lane / PPR, vcol = lane % PPR;
  const bool vok = FULL || vcol * 16 < dp;
  const int vsrc = vrow * dp + vcol * 16;
  // The half's other pieces: 16 sign rows, two pieces of mu, one of exponents, at a distance of
  // xsrc + offset * xmul from its V rows.
  const int xsrc = lane < 16 ? cv.off_bits() + lane * 16 : (lane < 18 ? cv.off_mu() + (lane - 16) * 16 : cv.off_exp());
  const int xsize = lane < 16 ? 16 : (lane < 18 ? 2 : 1);
  const int xmul = xsize - dp;
  const uint32_t xdst = lane < 16 ? lane * 16 : (lane < 18 ? S::xMu + (lane - 16) * 16 : S::xExp);
  auto issue = [&](int n, int st) {
    if (n < nmine) {
      if ((n & 15) == 0) {
        at = 0;
        const int m = n + (lane >> 1);
        if (m < nmine) {
          const PageAt pg = page_at(p, table, w.kv, w.block_at(v0 + warp + m * kWarps) * kBlk + (lane & 1) * kPageUnit);
          at_off = pg.off;
          if (pg.page >= 0) at = reinterpret_cast<uint64_t>(cv.block(pg.page, head)) + pg.off * dp;
        }
      }
      const uint32_t dst = vring + st * S::kV, extra = xring + st * S::kX + xdst;
      uint32_t ok2 = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint64_t rows = __shfl_sync(0xffffffffu, at, 2 * (n & 15) + h);
        const int off = __shfl_sync(0xffffffffu, at_off, 2 * (n & 15) + h);
        const uint32_t to = dst + kPageUnit * h * S::kRow;
        if (rows != 0) {
          ok2 |= 1u << h;
          const uint8_t* src = reinterpret_cast<const uint8_t*>(rows);
          if (vok) {
#pragma unroll
            for (int i = 0; i < kPageUnit / RPI; ++i)
              cp_async16(to + S::piece(i * RPI + vrow, vcol), src + vsrc + i * RPI * dp);
          }
          if (lane < 19) cp_async16(extra + kPageUnit * h * xsize, src + xsrc + off * xmul);
        } else {
          // No page: the rows are not seen, and their weights of 0 need finite scales.
          if (lane < 19) sts128(extra + kPageUnit * h * xsize, 0u, 0u, 0u, 0u);
        }
      }
      seen = (seen & ~(3u << (2 * st))) | (ok2 << (2 * st));
    }
    cp_async_commit();
  };
#pragma unroll
  for (int n = 0; n < kStages - 1; ++n) issue(n, n);

  // Sign bits and scale of the rows, while the first blocks are on their way.
  for (int r = warp; r < R; r += kWarps) {
    uint32_t word[4] = {0u, 0u, 0u, 0u};
    float sum = 0.0f;
    if (r < w.rows) {
      const int i = (w.r0 + r) / p.group, hq = head * p.group + (w.r0 + r) % p.group;
      const int64_t src = (w.t0 + i) * p.q_stride_t + hq * p.q_stride_h;
      if (q_f16)
        scan_row(static_cast<const __half*>(p.q) + src, cv.d, lane, word, sum);
      else
        scan_row(static_cast<const __nv_bfloat16*>(p.q) + src, cv.d, lane, word, sum);
    }
    if (lane < 4) s_bits[r][lane] = lane == 0 ? word[0] : (lane == 1 ? word[1] : (lane == 2 ? word[2] : word[3]));
    if (lane == 0) s_mu[r] = sum / static_cast<float>(cv.d);
  }
  __syncthreads();

  // Q as the A operand: this thread's bytes meet word t of the keys; byte i of step s is channel
  // 32 t + 8 i + s, and holds +-2^(6 - s) (s = 7: +-1, its bit is moved down by one).
  uint32_t qa[NR][8];
  float cq[NR], qsum[NR];
  int last[NR], wlo[NR];  // the row sees keys j <= last with j >= wlo or j < sinks
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int r = 8 * n + g;
    const uint32_t word = s_bits[r][t];
    const int nc = cv.d - 32 * t;  // channels of this word
    const uint32_t live = nc >= 32 ? 0xffffffffu : (nc <= 0 ? 0u : (1u << nc) - 1u);
#pragma unroll
    for (int st = 0; st < 8; ++st) {
      // Bytes mag, or 256 - mag where the bit is set; 0 where there is no channel.
      const uint32_t mag = 1u << (st == 7 ? 0 : 6 - st);
      qa[n][st] = (0x01010101u * mag + ((word >> st) & 0x01010101u) * (256u - 2u * mag)) &
                  (((live >> st) & 0x01010101u) * 255u);
    }
    const int neg = __popc(s_bits[r][0]) + __popc(s_bits[r][1]) + __popc(s_bits[r][2]) + __popc(s_bits[r][3]);
    qsum[n] = static_cast<float>(cv.d - 2 * neg);
    cq[n] = p.scale_log2 * s_mu[r];
    const int pos = w.pos0() + (w.r0 + r) / p.group;
    last[n] = r < w.rows ? (p.causal ? min(pos, w.kv - 1) : w.kv - 1) : -1;
    wlo[n] = p.causal && p.window > 0 ? pos - p.window + 1 : 0;
  }
  // What every row of the tile sees: keys <= all_last from all_lo on.
  const int all_last = p.causal ? min(w.pos0() + w.r0 / p.group, w.kv - 1) : w.kv - 1;
  const int all_lo = p.causal && p.window > 0 ? w.pos0() + (w.r0 + w.rows - 1) / p.group - p.window + 1 : 0;

  float acc[NR][MT][4];
  float M[NR];
  float2 l[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    M[n] = -CUDART_INF_F;
    l[n] = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][m][i] = 0.0f;
  }
  // Key of column g of the first of two score products of 16 keys (the second: two further on), such
  // that a thread's four scores are the keys 4 t .. 4 t + 3.
  const uint32_t kword = (4 * (g >> 1) + (g & 1)) * 16 + 4 * t;
  // Row of V that this lane gives to ldmatrix: tile 0's piece of key `lane`; tile m's is the same
  // address with the bits of 16 m flipped (stages start on 128 bytes).
  const uint32_t vbase = vring + S::piece(lane, 0);
  int start[4];  // a register quad of its own for the products' start
#pragma unroll
  for (int i = 0; i < 4; ++i) asm volatile("mov.u32 %0, %1;" : "=r"(start[i]) : "n"(kMagicBits));

  int st = 0;
  for (int n = 0; n < nmine; ++n) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    issue(n + kStages - 1, st == 0 ? kStages - 1 : st - 1);  // into the stage that the last block left
    const uint32_t stage = st * S::kV, fl = xring + st * S::kX;
    const int j0 = w.block_at(v0 + warp + n * kWarps) * kBlk;
    const uint32_t ok2 = (seen >> (2 * st)) & 3u;
    st = st == kStages - 1 ? 0 : st + 1;
    uint32_t word[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 2; ++k) word[h][k] = lds32(fl + kword + (16 * h + 2 * k) * 16);
    {
      const int e = static_cast<int8_t>(lds16(fl + S::xExp + (lane & ~1)) >> (8 * (lane & 1)));
      const int ec = min(max(e, kMinExp), kMaxExp);
      const float mu = __uint_as_float(lds16(fl + S::xMu + 2 * lane) << 16);
      __syncwarp();
      sts_f32(fl + 4 * lane, mu);
      sts_f32(fl + 4 * (kBlk + lane), static_cast<float>(ec));
      sts_f32(fl + 4 * (2 * kBlk + lane), __uint_as_float(static_cast<uint32_t>(127 - ec) << 23));
    }
    // 64 sum q k of 16 keys each (h), keys 4 t .. 4 t + 3 of them in the order 0, 1 | 2, 3.
    int x[2][2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        mma_i8_first(x[h][k], start, qa[0][0], NR == 2 ? qa[NR - 1][0] : 0u, qa[0][1], NR == 2 ? qa[NR - 1][1] : 0u,
                     word[h][k] & 0x01010101u, word[h][k] & 0x02020202u);
#pragma unroll
        for (int s = 1; s < 4; ++s)
          mma_i8(x[h][k], qa[0][2 * s], NR == 2 ? qa[NR - 1][2 * s] : 0u, qa[0][2 * s + 1],
                 NR == 2 ? qa[NR - 1][2 * s + 1] : 0u, word[h][k] & (0x01010101u << (2 * s)),
                 s == 3 ? (word[h][k] >> 1) & 0x40404040u : word[h][k] & (0x02020202u << (2 * s)));
      }
    __syncwarp();
    // Scores + e: sc[r][h][k] holds the keys 16 h + 4 t + 2 k and the next.
    float2 sc[NR][2][2], down[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 mu = lds_f4(fl + 64 * h + 16 * t), e = lds_f4(fl + 4 * kBlk + 64 * h + 16 * t),
                   dn = lds_f4(fl + 8 * kBlk + 64 * h + 16 * t);
      const float2 mu2[2] = {make_float2(mu.x, mu.y), make_float2(mu.z, mu.w)};
      const float2 e2[2] = {make_float2(e.x, e.y), make_float2(e.z, e.w)};
      down[h][0] = make_float2(dn.x, dn.y);
      down[h][1] = make_float2(dn.z, dn.w);
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // x = sum q - 2 sum q k: exact, the constant of the accumulator's start taken off with it.
          const float back = qsum[r] + kMagic / 32.0f;
          const float2 y = __ffma2_rn(make_float2(__int_as_float(x[h][k][2 * r]), __int_as_float(x[h][k][2 * r + 1])),
                                      make_float2(-0.03125f, -0.03125f), make_float2(back, back));
          sc[r][h][k] = __ffma2_rn(__fmul2_rn(y, mu2[k]), make_float2(cq[r], cq[r]), e2[k]);
        }
    }
    if (!(ok2 == 3u && j0 + kBlk - 1 <= all_last && j0 >= all_lo)) {
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int j = j0 + 16 * h + 4 * t + k;
            const bool see = ((ok2 >> h) & 1u) && j <= last[r] && (j >= wlo[r] || j < p.sinks);
            float& v = (k & 1) ? sc[r][h][k >> 1].y : sc[r][h][k >> 1].x;
            if (!see) v = -CUDART_INF_F;
          }
    }
    uint32_t bw[NR][2][2];  // weights: high and low bytes of the keys 16 h + 4 t .. + 3
    float2 f2[NR];          // what they count, for the rows 2 t and 2 t + 1
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float mx = fmaxf(fmaxf(fmaxf(sc[r][0][0].x, sc[r][0][0].y), fmaxf(sc[r][0][1].x, sc[r][0][1].y)),
                       fmaxf(fmaxf(sc[r][1][0].x, sc[r][1][0].y), fmaxf(sc[r][1][1].x, sc[r][1][1].y)));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (__any_sync(0xffffffffu, mx > M[r] + kSlack)) {
        const float to = mx > M[r] + kSlack ? mx : M[r];
        const float f = M[r] == -CUDART_INF_F ? 0.0f : ex2(M[r] - to);
        M[r] = to;
        l[r].x *= f;
        l[r].y *= f;
        const float f0 = __shfl_sync(0xffffffffu, f, 8 * t), f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          acc[r][m][0] *= f0;
          acc[r][m][1] *= f1;
          acc[r][m][2] *= f0;
          acc[r][m][3] *= f1;
        }
      }
      const bool none = mx == -CUDART_INF_F;  // the row sees nothing of the block
      const float ref = none ? 0.0f : -mx, f = none ? 0.0f : ex2(mx - M[r]);
      float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w16[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 y = __fadd2_rn(sc[r][h][k], make_float2(ref, ref));
          const float2 e = make_float2(ex2(y.x), ex2(y.y));
          sum = __ffma2_rn(e, down[h][k], sum);
          const float2 z = __ffma2_rn(e, make_float2(kUnit, kUnit), make_float2(kMagic, kMagic));
          w16[2 * k] = __float_as_uint(z.x);
          w16[2 * k + 1] = __float_as_uint(z.y);
        }
        const uint32_t u = __byte_perm(w16[0], w16[1], 0x5140), v = __byte_perm(w16[2], w16[3], 0x5140);
        bw[r][1][h] = __byte_perm(u, v, 0x5410);
        bw[r][0][h] = __byte_perm(u, v, 0x7632);
      }
      l[r] = __ffma2_rn(sum, make_float2(f, f), l[r]);
      const float fu = f * (1.0f / kUnit);
      f2[r] = make_float2(__shfl_sync(0xffffffffu, fu, 8 * t), __shfl_sync(0xffffffffu, fu, 8 * t + 4));
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (FULL || 16 * m < cv.dp) {
        uint32_t a[4];  // channels g and g + 8 of the tile: keys 4 t .. + 3 of the block's halves
        ldmatrix_t8((vbase + stage) ^ (m * 16), a);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          int hi[4], lo[4];
          mma_i8_first(hi, start, a[0], a[1], a[2], a[3], bw[r][0][0], bw[r][0][1]);
          mma_i8_first(lo, start, a[0], a[1], a[2], a[3], bw[r][1][0], bw[r][1][1]);
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            float2 o = make_float2(acc[r][m][i], acc[r][m][i + 1]);
            const float2 y = __ffma2_rn(whole(hi[i], hi[i + 1]), make_float2(256.0f, 256.0f), whole(lo[i], lo[i + 1]));
            o = __ffma2_rn(y, f2[r], o);
            acc[r][m][i] = o.x;
            acc[r][m][i + 1] = o.y;
          }
        }
      }
    }
    __syncwarp();
  }
  cp_async_wait<0>();
  __syncthreads();

  // Join the warps: each leaves its (M, l) and its sums in shared memory. A thread holds, for the
  // rows 8 n + 2 t and 8 n + 2 t + 1, the channels 16 m + g and 16 m + g + 8.
  float* s_o = reinterpret_cast<float*>(smem);  // [kWarps][R][CH]
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    float sum = l[n].x + l[n].y;
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if (t == 0) s_ml[warp][8 * n + g] = make_float2(M[n], sum);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s_o[(warp * R + 8 * n + 2 * t + (i & 1)) * CH + 16 * m + g + 8 * (i >> 1)] = acc[n][m][i];
  }
  __syncthreads();
  for (int r = warp; r < w.rows; r += kWarps) {
    float Mr = -CUDART_INF_F, lr = 0.0f, f[kWarps];
#pragma unroll
    for (int k = 0; k < kWarps; ++k) Mr = fmaxf(Mr, s_ml[k][r].x);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      f[k] = s_ml[k][r].x == -CUDART_INF_F ? 0.0f : ex2(s_ml[k][r].x - Mr);
      lr += f[k] * s_ml[k][r].y;
    }
    const int64_t row = (w.t0 + (w.r0 + r) / p.group) * p.heads + head * p.group + (w.r0 + r) % p.group;
    const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + slot) * R + r;
    const float inv = lr > 0.0f ? 1.0f / lr : 0.0f;
    for (int c = lane; c < dp; c += 32) {
      float x = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) x += f[k] * s_o[(k * R + r) * CH + c];
      if (slot >= 0)
        p.part_o[part * dp + c] = x;
      else if (c < cv.d)
        store_out(p.o, row * cv.d + c, x * inv, p.o_dt);
    }
    if (lane == 0) {
      if (slot >= 0)
        p.part_ml[part] = make_float2(Mr, lr);
      else if (p.lse != nullptr)
        p.lse[row] = lr > 0.0f ? (Mr + log2f(lr)) * CUDART_LN2_F : -CUDART_INF_F;
    }
  }
  __syncthreads();  // before the next (tile, head) uses the shared memory
  }
}

// Joins the parts of a (tile, head) that the line of units cut: o = sum_k 2^(M_k - M) o_k / sum_k
// 2^(M_k - M) l_k. One CTA per CTA of the first kernel and row of a tile; its warps take every fourth
// part, four channels per lane, and meet in shared memory.
__global__ void __launch_bounds__(kThreads) line_join_kernel(PagedAttnParams p, int bk) {
  __shared__ float s_x[kWarps][128];
  __shared__ float s_l[kWarps];
  const CacheView& cv = p.cache;
  const int cta = blockIdx.x % p.ctas, r = blockIdx.x / p.ctas;
  // Every CTA waits, also one with nothing to join: this grid must not complete before the one
  // whose parts it joins.
  grid_dependency_wait();
  const JoinNote note = p.notes[cta];
  if (note.last < 0) return;
  const RowTile w = entry_tile(p, note.entry, bk);
  if (r >= w.rows) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = note.last - cta + 1;
  // Part k: slot 1 of the first CTA, slot 0 of the others.
  auto part = [&](int k) { return (static_cast<int64_t>(cta + k) * 2 + (k == 0 ? 1 : 0)) * p.row_tile + r; };
  float M = -CUDART_INF_F;
  for (int k = lane; k < n; k += 32) M = fmaxf(M, p.part_ml[part(k)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float ref = M == -CUDART_INF_F ? 0.0f : M;
  float l = 0.0f;
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const bool on = 4 * lane < cv.dp;
#pragma unroll 8
  for (int k = warp; k < n; k += kWarps) {
    const int64_t at = part(k);
    const float2 ml = p.part_ml[at];
    const float4 o = on ? *reinterpret_cast<const float4*>(p.part_o + at * cv.dp + 4 * lane)
                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float f = ex2(ml.x - ref);
    l = __fmaf_rn(f, ml.y, l);
    x.x = __fmaf_rn(f, o.x, x.x);
    x.y = __fmaf_rn(f, o.y, x.y);
    x.z = __fmaf_rn(f, o.z, x.z);
    x.w = __fmaf_rn(f, o.w, x.w);
  }
  *reinterpret_cast<float4*>(&s_x[warp][4 * lane]) = x;
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  const float lt = s_l[0] + s_l[1] + s_l[2] + s_l[3];
  const int64_t row = (w.t0 + (w.r0 + r) / p.group) * p.heads + note.head * p.group + (w.r0 + r) % p.group;
  const int c = threadIdx.x;
  if (c < cv.d) {
    const float sum = s_x[0][c] + s_x[1][c] + s_x[2][c] + s_x[3][c];
    store_out(p.o, row * cv.d + c, lt > 0.0f ? sum / lt : 0.0f, p.o_dt);
  }
  if (c == 0 && p.lse != nullptr) p.lse[row] = lt > 0.0f ? (M + log2f(lt)) * CUDART_LN2_F : -CUDART_INF_F;
}

// Joins the parts of each row: o = sum_k 2^(M_k - M) o_k / sum_k 2^(M_k - M) l_k. One CTA per row: its
// warps take every fourth part, four channels per lane, and meet in shared memory.
__global__ void __launch_bounds__(kThreads) paged_join_kernel(PagedAttnParams p, int bk) {
  __shared__ float s_x[kWarps][128];
  __shared__ float s_l[kWarps];
  const CacheView& cv = p.cache;
  int b, tile, head, r;
  cta_of(p, blockIdx.x, p.row_tile, b, tile, head, r);
  // Every CTA waits, also one with nothing to join: this grid must not complete before the one
  // whose parts it joins.
  grid_dependency_wait();
  const RowTile w = row_tile(p, b, tile, bk);
  if (r >= w.rows) return;
  const int used = splits_used(p, w.nblk);
  if (used == 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t all = p.T * p.heads;
  const int64_t row = (w.t0 + (w.r0 + r) / p.group) * p.heads + head * p.group + (w.r0 + r) % p.group;
  float M = -CUDART_INF_F;
  for (int k = lane; k < used; k += 32) M = fmaxf(M, p.part_ml[k * all + row].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float ref = M == -CUDART_INF_F ? 0.0f : M;
  float l = 0.0f;
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const bool on = 4 * lane < cv.dp;
#pragma unroll 4
  for (int k = warp; k < used; k += kWarps) {
    const float2 ml = p.part_ml[k * all + row];
    const float4 o = on ? *reinterpret_cast<const float4*>(p.part_o + (k * all + row) * cv.dp + 4 * lane) : x;
    const float f = ex2(ml.x - ref);
    l = __fmaf_rn(f, ml.y, l);
    x.x = __fmaf_rn(f, o.x, x.x);
    x.y = __fmaf_rn(f, o.y, x.y);
    x.z = __fmaf_rn(f, o.z, x.z);
    x.w = __fmaf_rn(f, o.w, x.w);
  }
  *reinterpret_cast<float4*>(&s_x[warp][4 * lane]) = x;
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  const float lt = s_l[0] + s_l[1] + s_l[2] + s_l[3];
  const int c = threadIdx.x;
  if (c < cv.d) {
    const float sum = s_x[0][c] + s_x[1][c] + s_x[2][c] + s_x[3][c];
    store_out(p.o, row * cv.d + c, lt > 0.0f ? sum / lt : 0.0f, p.o_dt);
  }
  if (c == 0 && p.lse != nullptr) p.lse[row] = lt > 0.0f ? (M + log2f(lt)) * CUDART_LN2_F : -CUDART_INF_F;
}

template <int CPG, int NR, bool FULL>
cudaError_t launch_decode_full(const PagedAttnParams& p, int dt, cudaStream_t s) {
  constexpr int ring = kWarps * Ring<CPG>::kBytes, out = kWarps * 8 * NR * CPG * 8 * 4;
  constexpr int smem = ring > out ? ring : out;
  auto kernel = paged_decode_kernel<CPG, NR, FULL>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(p.B) * p.row_tiles * p.cache.heads;
  kernel<<<static_cast<unsigned>(p.ctas > 0 ? p.ctas : tiles), kThreads, smem, s>>>(p, dt == BA_F16 ? 1 : 0);
  if ((e = cudaGetLastError()) != cudaSuccess || p.ctas == 0) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.ctas * p.row_tile));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, line_join_kernel, p, kBlk);
}

template <int CPG, int NR>
cudaError_t launch_decode(const PagedAttnParams& p, int dt, cudaStream_t s) {
  return p.cache.dp == CPG * 8 ? launch_decode_full<CPG, NR, true>(p, dt, s)
                               : launch_decode_full<CPG, NR, false>(p, dt, s);
}

}  // namespace

cudaError_t launch_paged_join(const PagedAttnParams& p, int bk, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(p.B) * p.row_tiles * p.cache.heads * p.row_tile));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel, p, bk);
}

cudaError_t launch_paged_decode(const PagedAttnParams& p, int dt, cudaStream_t s) {
  if (p.cache.dp > 64) return p.row_tile > 8 ? launch_decode<16, 2>(p, dt, s) : launch_decode<16, 1>(p, dt, s);
  return p.row_tile > 8 ? launch_decode<8, 2>(p, dt, s) : launch_decode<8, 1>(p, dt, s);
}

int paged_decode_ctas(const PagedAttnParams& p, int sms) {
  // Keys that a tile can see, in blocks.
  int64_t keys = p.max_kv_len;
  if (p.causal && p.window > 0)
    keys = std::min<int64_t>(keys, static_cast<int64_t>(p.window) + p.row_tile + p.sinks + 2 * kBlk);
  const int64_t blocks = ceil_div(keys, kBlk), tiles = static_cast<int64_t>(p.B) * p.row_tiles * p.cache.heads;
  // Two blocks per warp or fewer: cutting would cost more (a second launch) than it saves.
  if (blocks <= 2 * kWarps) return 0;
  // As many CTAs as fit at once (by registers), each with one block per warp at least.
  return static_cast<int>(std::min<int64_t>(sms * (p.row_tile == 8 ? 4 : 3), ceil_div((blocks + kCost) * tiles, kWarps)));
}

}  // namespace binattn
