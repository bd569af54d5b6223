// Attention of few query rows over the paged cache (sm_100a): decoding and drafts.
//
// With few rows per KV head the kernel is bound by reading the cache once: dp + 19 bytes per token
// and head, and at HBM's rate a key of 147 bytes leaves an SM some 6.5 cycles. So the work per key
// is kept small:
//   * A CTA takes one sequence, one KV head, up to 8 NR rows (new tokens x heads of the group, which
//     share every key) and a part of the key axis. Each of its warps walks 64-key blocks of its own
//     through a ring of TMA stages (V through a tensor map whose swizzle keeps ldmatrix free of bank
//     conflicts, the rest as plain bulk copies), with no synchronisation between warps until the end.
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
//     added in fp32. A weight's error is 2^-17 of the block's largest. Scores come out by key and
//     weights go in by row; movmatrix turns them, as 16-bit numbers, in between.
//   * A value row's exponent e_j joins the score instead of the codes: the weight is
//     2^(s_j + e_j - m) with m a maximum of s_j + e_j, and the softmax sum adds weight * 2^-e_j. The
//     reference M moves (and the sums are rescaled) only when a block's m passes it by 2^40, far
//     inside fp32's range, so that hardly any block rescales.
//   * Short contexts: a cluster of up to eight CTAs per (tile, head), each with a part of the key axis,
//     joined through distributed shared memory. Else the CTAs share the line of all units evenly, and the
//     parts of what they cut leave (M, sum, unnormalised o) in fp32, joined by a second kernel that is
//     launched as a programmatic dependent.
// Measured with 32 query heads, 8 KV heads, d = 128: 128 contexts up to 8192 tokens 105 to 107 us (5.6 to
// 5.7 TB/s, 87 % of a copy; further keys come at 6.3 TB/s); one context of 1024 tokens 8 us, of which a few
// dependent loads and cold instructions are most; 4 KV heads, one context of 131072 tokens 27 us (2.8
// TB/s: 10 us are start and join). d = 64, one query head for each of 16 KV heads, a window of 4096 tokens
// in 32 contexts: 42 us (3.7 TB/s), bound by instructions: seven of eight rows are empty.
#include <math_constants.h>

#include <algorithm>

#include "kernels.h"
#include "paged.cuh"
#include "tc_ptx.cuh"
#include "tensormap.h"

namespace binattn {

__device__ int g_decode_status = 0;

namespace {

using namespace ptx;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kBlk = 64;       // keys per stage of a warp
constexpr int kStages = 2;
constexpr int kQ = kBlk / 16;  // quarters of a block: 16 keys each
// Blocks that a CTA could do while it starts and ends a (tile, head): with 8, 12, 16 and 32 a batch of 128
// contexts up to 8192 took 119, 107, 106 and 109 us, one of 16 contexts 22.9, 23.0, 24.2 and 25.8 us.
constexpr int kCost = 12;
constexpr int kShort = 3;  // blocks of a warp that the joining launch costs
constexpr float kSlack = 40.0f;  // log2 by which a block's maximum may pass the reference
constexpr float kUnit = 65280.0f;  // weight 1 in fixed point: 255 * 256
constexpr int kMagicBits = 0x4B400000;  // 1.5 * 2^23
constexpr float kMagic = 12582912.0f;

__device__ __forceinline__ float ex2(float x) { return ex2_approx(x); }

__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  const uint4 u = lds128(a);
  return make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// c (+)= A B: A 16 x 32 unsigned bytes (keys g and g + 8), B 32 x 8 signed bytes (rows of Q).
__device__ __forceinline__ void mma_qk_first(int (&c)[4], const int (&start)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(start[0]), "r"(start[1]), "r"(start[2]),
        "r"(start[3]));
}
__device__ __forceinline__ void mma_qk(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// c (+)= A B: A 16 channels x 32 keys of signed codes, B 32 keys x 8 rows of unsigned bytes.
__device__ __forceinline__ void mma_pv_first(int (&c)[4], const int (&start)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(start[0]), "r"(start[1]), "r"(start[2]),
        "r"(start[3]));
}
__device__ __forceinline__ void mma_pv(int (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two 16 x 16 matrices of bytes, transposed. Lanes 0-15 and 16-31 give the rows' addresses; the lane
// (g, t) gets, of each matrix, columns g and g + 8 of rows 4 t .. 4 t + 3.
__device__ __forceinline__ void ldmatrix_t8(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}

// 8 x 8 matrix of 16-bit numbers, transposed: the lane (g, t) gives row g, columns 2 t and 2 t + 1.
__device__ __forceinline__ uint32_t turn8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Whole-number results (kMagicBits + n, |n| <= 255 * 128 * 64 < 2^22) as floats n.
__device__ __forceinline__ float2 whole(int x, int y) {
  return __fadd2_rn(make_float2(__int_as_float(x), __int_as_float(y)), make_float2(-kMagic, -kMagic));
}

// Shared memory of a warp: V rows of kRow bytes for each stage as the tensor map's swizzle leaves
// them, then each stage's sign rows, mu and exponents. Once a block's sign rows are read, what its
// scores need per key as floats (mu, e, 2^-e) takes their place. Three CTAs of four warps just fit an SM
template <int CPG>  // eighths of the channels: 16 (rows of 128 bytes) or 8 (rows of 64)
struct Ring {
  static constexpr int kRow = CPG * 8;
  static constexpr int kV = kBlk * kRow;
  static constexpr int offX = kStages * kV;
  static constexpr int xMu = kBlk * 16, xExp = xMu + kBlk * 2, kX = xExp + kBlk;
  static constexpr int kBytes = offX + kStages * kX;  // of a warp
  // Behind the warps' rings: barriers, sums of the warps, sign words and scales of the rows, scratch.
  static constexpr int offFull = kWarps * kBytes;
  static constexpr int offMl = offFull + kWarps * kStages * 8;
  static __host__ __device__ constexpr int offBits(int rows) { return offMl + kWarps * rows * 8; }
  static __host__ __device__ constexpr int offMu(int rows) { return offBits(rows) + rows * 16; }
  static __host__ __device__ constexpr int offScratch(int rows) { return offMu(rows) + rows * 4; }
  static __host__ __device__ constexpr int total(int rows) { return offScratch(rows) + (kWarps + 2) * 8; }
  static constexpr int kToken = kRow + 16 + 2 + 1;  // bytes that a token brings
  // Byte offset of the 16-byte piece c of key j: the swizzle of 128- or 64-byte rows.
  static __device__ __forceinline__ int piece(int j, int c) {
    return kRow == 128 ? (j * 8 + (c ^ (j & 7))) * 16 : (j * 4 + (c ^ ((j >> 1) & 3))) * 16;
  }
};

// Waits, a second at most, for a stage's copies; records a timeout.
__device__ __forceinline__ bool wait_stage(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer() - t0 > 1000000000ull) {
      atomicExch(&g_decode_status, 1);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// A float at the shared-memory address `a` of the cluster's CTA `rank`.
__device__ __forceinline__ float lds_cluster(uint32_t a, int rank) {
  uint32_t at;
  float x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
  return x;
}

// CTAs on an SM. Two tiles of 8 rows need 255 registers: with three CTAs, and 230 bytes of spills, 16 rows
// of 32 x 4096 keys and 8 KV heads (d = 128) took 70 us instead of 49. Up to 64 channels fit 128 registers:
// 16 heads of 32 x 4096 keys in a window (d = 64) take 41 us with four, 46 with three, 43 with five and spills.
constexpr int ctas_per_sm(int cpg, int nr) { return nr == 2 ? 2 : (cpg == 16 ? 3 : 4); }

template <int CPG, int NR>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(CPG, NR))
    paged_decode_kernel(PagedAttnParams p, int q_f16, int unit, const __grid_constant__ CUtensorMap v_map) {
  using S = Ring<CPG>;
  constexpr int MT = CPG / 2;  // 16-channel tiles
  constexpr int R = 8 * NR;    // rows of a CTA
  constexpr int CH = CPG * 8;  // channels of the accumulators (>= d)
  constexpr int KS = CPG / 2;  // steps of QK, four channels of each thread
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int oBits = S::offBits(R), oMu = S::offMu(R), oScratch = S::offScratch(R);
  auto s_full = reinterpret_cast<uint64_t(*)[kStages]>(smem + S::offFull);
  auto s_ml = reinterpret_cast<float2(*)[R]>(smem + S::offMl);
  auto s_bits = reinterpret_cast<uint32_t(*)[4]>(smem + oBits);
  auto s_mu = reinterpret_cast<float*>(smem + oMu);

  allow_dependents();
  grid_dependency_wait();
  const CacheView& cv = p.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int dp = cv.dp;
  // The V stages of all warps come first (they start on 1024 bytes, where the swizzle starts).
  const uint32_t base = smem_u32(smem);
  const uint32_t vring = base + warp * S::offX, xring = base + kWarps * S::offX + warp * kStages * S::kX;
  if (lane < kStages) {
    mbar_init(&s_full[warp][lane], 1);
    mbar_fence_init();
  }
  __syncwarp();
  int st = 0;          // stage of the next block, and the parity of its next arrival
  uint32_t phase = 0;
  bool ok = true;
  Stretch line{};
  if (p.ctas > 0) {
    line = find_stretch<kThreads>(p, kBlk, kCost, kWarps, reinterpret_cast<int64_t*>(smem + oScratch));
    if (line.at >= line.end) {
      if (threadIdx.x == 0) p.notes[blockIdx.x].last = -1;
      return;
    }
  } else {
    line.entry = p.by_kv_heads(blockIdx.x / p.cluster);
  }

  // One (tile, head) per cluster: its CTAs take equal parts and join them through their shared memory.
  const int rank = p.ctas > 0 ? 0 : blockIdx.x % p.cluster;

  for (bool more = true; more;) {
  // The next (tile, head) of the CTA: its blocks v0 .. v1 - 1 of all.
  const RowTile w = entry_tile(p, line.entry, kBlk);
  const int b = p.by_tiles(line.entry);
  int head = blockIdx.x / p.cluster - line.entry * cv.heads, v0 = 0, v1 = w.nblk, slot = -1;  // slot -1: nothing is cut
  if (p.ctas > 0) {
    const int units = units_of(w, kCost);
    if (units == 0) {  // a tile without rows
      line.entry = entry_after(p, line.entry, w);
      continue;
    }
    const int entry = line.entry;
    const int64_t in = line.at - line.base;
    head = (in >> 32) == 0 ? static_cast<uint32_t>(in) / static_cast<uint32_t>(units) : static_cast<int>(in / units);
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
    v0 = w.nblk * rank / p.cluster;  // a power of two below 16; nblk < 2^23
    v1 = w.nblk * (rank + 1) / p.cluster;
  }

  // The rows of q are asked for first; their signs are taken while the first blocks are on their way.
  constexpr int QR = R / kWarps;
  uint16_t q_raw[QR][4];
#pragma unroll
  for (int u = 0; u < QR; ++u) {
    const int r = warp + u * kWarps, i = p.by_group(w.r0 + r);
    const uint16_t* src = static_cast<const uint16_t*>(p.q) + (w.t0 + i) * p.q_stride_t +
                          (head * p.group + w.r0 + r - i * p.group) * p.q_stride_h;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      q_raw[u][k] = 0;
      if (32 * k < CH && r < w.rows && 32 * k + lane < cv.d) q_raw[u][k] = __ldg(src + 32 * k + lane);
    }
  }

  // The warp's blocks are v0 + warp, v0 + warp + kWarps, ... A block comes as `per` pieces of `unit`
  // tokens, each within a page. Lane l keeps the page and the offset in it of the piece l % 4 of the
  // block l / 4 after the last look-up: 8 blocks at a time.
  const int nmine = ok ? max(0, (v1 - v0 - warp + kWarps - 1) / kWarps) : 0;
  const int32_t* table = p.table + b * p.table_stride;
  const int per = kBlk / unit;
  PageAt at{-1, 0};
  uint32_t seen = 0;  // four bits per stage: which quarters of the block have a page
  // Copies of a block: lane 4 i + k brings, of its piece i, the V rows (k = 0), the sign rows, mu or
  // the exponents, which lie at off + offset * size in the page's block.
  const int piece = (lane >> 2) & 3, kind = lane & 3;
  const int xoff = kind == 1 ? cv.off_bits() : (kind == 2 ? cv.off_mu() : cv.off_exp());
  const int xsize = kind == 1 ? 16 : (kind == 2 ? 2 : 1);
  const int xdst = (kind == 1 ? 0 : (kind == 2 ? S::xMu : S::xExp)) + unit * piece * xsize;
  auto issue = [&](int n, int to) {  // block n of the warp into stage `to`
    if (n >= nmine) return;
    if ((n & 7) == 0) {
      at.page = -1;
      const int m = n + (lane >> 2);
      if (m < nmine && (lane & 3) < per)
        at = page_at(p, table, w.kv, w.block_at(v0 + warp + m * kWarps) * kBlk + (lane & 3) * unit);
    }
    const int page = __shfl_sync(0xffffffffu, at.page, 4 * (n & 7) + piece);
    const int off = __shfl_sync(0xffffffffu, at.off, 4 * (n & 7) + piece);
    // Bits 0, 4, 8 and 12 of the vote: the pieces with a page.
    const uint32_t vote = __ballot_sync(0xffffffffu, page >= 0 && lane < 16) & 0x1111u;
    const uint32_t bar = smem_u32(&s_full[warp][to]), extra = xring + to * S::kX + xdst;
#ifdef BA_TEST_SKIP_ARRIVE
    // Test build only: the first block waits for 16 bytes that nobody brings, so that its wait runs into the limit.
    const uint32_t missing = n == 0 ? 16u : 0u;
#else
    constexpr uint32_t missing = 0u;
#endif
    if (lane == 0) mbar_arrive_expect_tx(&s_full[warp][to], __popc(vote) * unit * S::kToken + missing);
    __syncwarp();
    if (lane < 4 * per) {
      if (page < 0) {
        // No page: the rows are not seen, but what their scores are made of stays finite.
        if (kind > 0)
          for (int i = 0; i < unit / 16 * xsize; ++i) sts128(extra + 16 * i, 0u, 0u, 0u, 0u);
      } else if (kind == 0) {
        tma_load_3d(vring + to * S::kV + unit * piece * S::kRow, &v_map, bar, 0, off, page * cv.heads + head);
      } else {
        bulk_load(extra, cv.block(page, head) + xoff + off * xsize, unit * xsize, bar);
      }
    }
    // Per quarter: of one piece (all four), two (two each) or four.
    const uint32_t have = per == 4 ? (vote * 0x1248u >> 12) & 15u : (per == 2 ? (vote & 1u) * 3u + (vote >> 4 & 1u) * 12u : vote * 15u);
    seen = (seen & ~(15u << (4 * to))) | (have << (4 * to));
  };
#pragma unroll
  for (int n = 0; n < kStages; ++n) issue(n, st + n >= kStages ? st + n - kStages : st + n);

  // Sign words and scales of the rows.
#pragma unroll
  for (int u = 0; u < QR; ++u) {
    uint32_t word[4];
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x = widen(q_raw[u][k], q_f16);
      word[k] = __ballot_sync(0xffffffffu, x < 0.0f);
      sum += fabsf(x) * kMeanStep;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int r = warp + u * kWarps;
    if (lane < 4) s_bits[r][lane] = lane == 0 ? word[0] : (lane == 1 ? word[1] : (lane == 2 ? word[2] : word[3]));
    if (lane == 0) s_mu[r] = mean_of(sum, cv.d);
  }
  __syncthreads();

  // Q as the B operand, row g: this thread's bytes meet word t of the keys; byte i of step s is
  // channel 32 t + 8 i + s, and holds +-2^(6 - s) (s = 7: +-1, its bit is moved down by one). Up to 64
  // channels: word t % 2, of each of its bytes the upper half if t > 1.
  const int tw = CPG == 16 ? t : t & 1, sh = CPG == 16 ? 0 : 4 * (t >> 1);
  uint32_t qb[NR][KS];
  // Of the rows 2 t and 2 t + 1, which this thread's scores belong to:
  float2 cq[NR], back[NR];
  int last[NR][2], wlo[NR][2];  // the row sees keys j <= last with j >= wlo or j < sinks
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const uint32_t word = s_bits[8 * n + g][tw] >> sh;
    const int nc = cv.d - 32 * tw;  // channels of this word
    const uint32_t live = (nc >= 32 ? 0xffffffffu : (nc <= 0 ? 0u : (1u << nc) - 1u)) >> sh;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      // Bytes mag, or 256 - mag where the bit is set; 0 where there is no channel.
      const uint32_t mag = 1u << (s == 7 ? 0 : 6 - s);
      qb[n][s] = (0x01010101u * mag + ((word >> s) & 0x01010101u) * (256u - 2u * mag)) &
                 (((live >> s) & 0x01010101u) * 255u);
    }
    float c2[2], b2[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 8 * n + 2 * t + i;
      const int neg = __popc(s_bits[r][0]) + __popc(s_bits[r][1]) + __popc(s_bits[r][2]) + __popc(s_bits[r][3]);
      b2[i] = static_cast<float>(cv.d - 2 * neg) + kMagic / 32.0f;
      c2[i] = p.scale_log2 * s_mu[r];
      const int pos = w.pos0() + p.by_group(w.r0 + r);
      last[n][i] = r < w.rows ? (p.causal ? min(pos, w.kv - 1) : w.kv - 1) : -1;
      wlo[n][i] = p.causal && p.window > 0 ? pos - p.window + 1 : 0;
    }
    cq[n] = make_float2(c2[0], c2[1]);
    back[n] = make_float2(b2[0], b2[1]);
  }
  // What every row of the tile sees: keys <= all_last from all_lo on.
  const int all_last = p.causal ? min(w.pos0() + p.by_group(w.r0), w.kv - 1) : w.kv - 1;
  const int all_lo = p.causal && p.window > 0 ? w.pos0() + p.by_group(w.r0 + w.rows - 1) - p.window + 1 : 0;

  float acc[NR][MT][4];
  float2 M[NR], l[NR];  // of the rows 2 t and 2 t + 1
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    M[n] = make_float2(-CUDART_INF_F, -CUDART_INF_F);
    l[n] = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][m][i] = 0.0f;
  }
  // Keys of this thread's scores: 16 h + key0 + 2 k. (Row g of an 8 x 8 matrix is the key
  // 4 (g / 2) + g % 2, the second matrix two further on, so that the turned matrices hold the keys
  // 4 t .. 4 t + 3 as ldmatrix holds V's.)
  const int key0 = 4 * (g >> 1) + (g & 1);
  // Row of V that this lane gives to ldmatrix: tile 0's piece of key `lane`; tile m's is the same
  // address with the bits of 16 m flipped.
  const uint32_t vbase = vring + S::piece(lane, 0);
  int start[4];  // a register quad of its own for the products' start
#pragma unroll
  for (int i = 0; i < 4; ++i) asm volatile("mov.u32 %0, %1;" : "=r"(start[i]) : "n"(kMagicBits));

  for (int n = 0; n < nmine && ok; ++n) {
    const uint32_t stage = st * S::kV, fl = xring + st * S::kX;
    const int j0 = w.block_at(v0 + warp + n * kWarps) * kBlk;
    ok = __all_sync(0xffffffffu, wait_stage(&s_full[warp][st], (phase >> st) & 1u));
    if (!ok) break;
    phase ^= 1u << st;
    const uint32_t have = (seen >> (4 * st)) & 15u;
    // The block's sign words, before floats take their place.
    uint32_t word[kQ][2];
#pragma unroll
    for (int h = 0; h < kQ; ++h)
#pragma unroll
      for (int k = 0; k < 2; ++k) word[h][k] = lds32(fl + (16 * h + key0 + 2 * k) * 16 + 4 * tw) >> sh;
    {
      uint32_t mu[kBlk / 32];
      int e[kBlk / 32];
#pragma unroll
      for (int i = 0; i < kBlk / 32; ++i) {
        const int j = 32 * i + lane;
        e[i] = min(max(static_cast<int>(static_cast<int8_t>(lds16(fl + S::xExp + (j & ~1)) >> (8 * (lane & 1)))), kMinExp), kMaxExp);
        mu[i] = lds16(fl + S::xMu + 2 * j) << 16;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kBlk / 32; ++i)
        sts128(fl + 16 * (32 * i + lane), mu[i], __float_as_uint(static_cast<float>(e[i])),
               static_cast<uint32_t>(127 - e[i]) << 23, 0u);
      __syncwarp();
    }
    // Scores + e of the keys 16 h + key0 + 2 k and the rows 2 t and 2 t + 1.
    float2 sc[NR][kQ][2];
#pragma unroll
    for (int h = 0; h < kQ; ++h) {
      int x[NR][4];  // 64 sum q k of 16 keys and 8 rows
#pragma unroll
      for (int s = 0; s < KS / 2; ++s) {
        const uint32_t a0 = word[h][0] & (0x01010101u << (2 * s)), a1 = word[h][1] & (0x01010101u << (2 * s));
        const uint32_t a2 = s == 3 ? (word[h][0] >> 1) & 0x40404040u : word[h][0] & (0x02020202u << (2 * s));
        const uint32_t a3 = s == 3 ? (word[h][1] >> 1) & 0x40404040u : word[h][1] & (0x02020202u << (2 * s));
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          if (s == 0)
            mma_qk_first(x[r], start, a0, a1, a2, a3, qb[r][0], qb[r][1]);
          else
            mma_qk(x[r], a0, a1, a2, a3, qb[r][2 * s], qb[r][2 * s + 1]);
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float4 f = lds_f4(fl + (16 * h + key0 + 2 * k) * 16);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          // x = sum q - 2 sum q k: exact, the constant of the accumulator's start taken off with it.
          float2 y = __ffma2_rn(make_float2(__int_as_float(x[r][2 * k]), __int_as_float(x[r][2 * k + 1])),
                                make_float2(-0.03125f, -0.03125f), back[r]);
          y = __fmul2_rn(y, cq[r]);
          sc[r][h][k] = make_float2(__fmaf_rn(y.x, f.x, f.y), __fmaf_rn(y.y, f.x, f.y));
        }
      }
    }
    if (!(have == 15u && j0 + kBlk - 1 <= all_last && j0 >= all_lo)) {
      __syncwarp();  // keeps this a branch: most blocks need no mask
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int h = 0; h < kQ; ++h)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int j = j0 + 16 * h + key0 + 2 * k;
            const bool in = (have >> h) & 1u, sink = j < p.sinks;
            if (!(in && j <= last[r][0] && (j >= wlo[r][0] || sink))) sc[r][h][k].x = -CUDART_INF_F;
            if (!(in && j <= last[r][1] && (j >= wlo[r][1] || sink))) sc[r][h][k].y = -CUDART_INF_F;
          }
    }
    uint32_t bw[NR][2][kQ];  // weights of row g: high and low bytes of the keys 16 h + 4 t .. + 3
    float2 f2[NR];           // what they count, for the rows 2 t and 2 t + 1
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float2 mx = make_float2(fmaxf(sc[r][0][0].x, sc[r][0][1].x), fmaxf(sc[r][0][0].y, sc[r][0][1].y));
#pragma unroll
      for (int h = 1; h < kQ; ++h) {
        mx.x = fmax3(mx.x, sc[r][h][0].x, sc[r][h][1].x);
        mx.y = fmax3(mx.y, sc[r][h][0].y, sc[r][h][1].y);
      }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mx.x = fmaxf(mx.x, __shfl_xor_sync(0xffffffffu, mx.x, o));
        mx.y = fmaxf(mx.y, __shfl_xor_sync(0xffffffffu, mx.y, o));
      }
      if (__any_sync(0xffffffffu, mx.x > M[r].x + kSlack || mx.y > M[r].y + kSlack)) {
        const float2 to = make_float2(mx.x > M[r].x + kSlack ? mx.x : M[r].x, mx.y > M[r].y + kSlack ? mx.y : M[r].y);
        const float2 f = make_float2(M[r].x == -CUDART_INF_F ? 0.0f : ex2(M[r].x - to.x),
                                     M[r].y == -CUDART_INF_F ? 0.0f : ex2(M[r].y - to.y));
        M[r] = to;
        l[r] = __fmul2_rn(l[r], f);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          acc[r][m][0] *= f.x;
          acc[r][m][1] *= f.y;
          acc[r][m][2] *= f.x;
          acc[r][m][3] *= f.y;
        }
      }
      // A row that sees nothing of the block has weights 0 (2^-inf) and counts for nothing.
      const float2 ref = make_float2(mx.x == -CUDART_INF_F ? 0.0f : -mx.x, mx.y == -CUDART_INF_F ? 0.0f : -mx.y);
      const float2 f = make_float2(mx.x == -CUDART_INF_F ? 0.0f : ex2(mx.x - M[r].x),
                                   mx.y == -CUDART_INF_F ? 0.0f : ex2(mx.y - M[r].y));
      float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int h = 0; h < kQ; ++h) {
        uint32_t w16[2];  // 16-bit weights of the keys 16 h + 4 t + 2 k and the next, of row g
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 y = __fadd2_rn(sc[r][h][k], ref);
          const float2 e = make_float2(ex2(y.x), ex2(y.y));
          const float down = __uint_as_float(lds32(fl + (16 * h + key0 + 2 * k) * 16 + 8));  // 2^-e
          sum.x = __fmaf_rn(e.x, down, sum.x);
          sum.y = __fmaf_rn(e.y, down, sum.y);
          const float2 z = __ffma2_rn(e, make_float2(kUnit, kUnit), make_float2(kMagic, kMagic));
          w16[k] = turn8(__byte_perm(__float_as_uint(z.x), __float_as_uint(z.y), 0x5410));
        }
        bw[r][0][h] = __byte_perm(w16[0], w16[1], 0x7531);
        bw[r][1][h] = __byte_perm(w16[0], w16[1], 0x6420);
      }
      l[r] = __ffma2_rn(sum, f, l[r]);
      f2[r] = __fmul2_rn(f, make_float2(1.0f / kUnit, 1.0f / kUnit));
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (16 * m < dp) {
        uint32_t a[2][4];  // channels g and g + 8 of the tile: keys 4 t .. + 3 of two quarters each
        ldmatrix_t8((vbase + stage) ^ (m * 16), a[0]);
        ldmatrix_t8((vbase + stage + 32 * S::kRow) ^ (m * 16), a[1]);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          int hi[4], lo[4];
          mma_pv_first(hi, start, a[0], bw[r][0][0], bw[r][0][1]);
          mma_pv_first(lo, start, a[0], bw[r][1][0], bw[r][1][1]);
          mma_pv(hi, a[1], bw[r][0][2], bw[r][0][3]);
          mma_pv(lo, a[1], bw[r][1][2], bw[r][1][3]);
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
    // The stage's next block: what this warp wrote there comes before what the copies write.
    fence_proxy_async_smem();
    __syncwarp();
    issue(n + kStages, st);
    st = st == kStages - 1 ? 0 : st + 1;
  }
  // After a timeout: the copies still on their way get one more limited wait.
  if (!ok)
    for (int n = 0; n < min(nmine, kStages); ++n) wait_stage(&s_full[warp][n], (phase >> n) & 1u);
  __syncthreads();

  // Join the warps: each leaves its (M, l) and its sums in shared memory. A thread holds, for the
  // rows 8 n + 2 t and 8 n + 2 t + 1, the channels 16 m + g and 16 m + g + 8.
  float* s_o = reinterpret_cast<float*>(smem);  // [kWarps][R][CH]
  float* s_sum = s_o + kWarps * R * CH;         // [R][CH], and (M, l) of the rows: what a cluster joins
  float2* s_fin = reinterpret_cast<float2*>(s_sum + R * CH);
  const bool clustered = p.ctas == 0 && p.cluster > 1;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    float2 sum = l[n];
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      sum.x += __shfl_xor_sync(0xffffffffu, sum.x, o);
      sum.y += __shfl_xor_sync(0xffffffffu, sum.y, o);
    }
    if (g == 0) {
      s_ml[warp][8 * n + 2 * t] = make_float2(M[n].x, sum.x);
      s_ml[warp][8 * n + 2 * t + 1] = make_float2(M[n].y, sum.y);
    }
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
    const int64_t row = out_row(p, w, head, r);
    const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + slot) * R + r;
    const float inv = lr > 0.0f ? 1.0f / lr : 0.0f;
    for (int c = lane; c < dp; c += 32) {
      float x = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) x += f[k] * s_o[(k * R + r) * CH + c];
      if (slot >= 0)
        p.part_o[part * dp + c] = x;
      else if (clustered)
        s_sum[r * CH + c] = x;
      else if (c < cv.d)
        store_out(p.o, row * cv.d + c, x * inv, p.o_dt);
    }
    if (lane == 0) {
      if (slot >= 0)
        p.part_ml[part] = make_float2(Mr, lr);
      else if (clustered)
        s_fin[r] = make_float2(Mr, lr);
      else if (p.lse != nullptr)
        p.lse[row] = lr > 0.0f ? (Mr + log2f(lr)) * CUDART_LN2_F : -CUDART_INF_F;
    }
  }
  if (clustered) {
    // Rows of the tile by turns: each CTA joins all parts of its rows.
    cluster_arrive();
    cluster_wait();
    for (int r = rank + p.cluster * warp; r < w.rows; r += p.cluster * kWarps) {
      // Lane k has the (M, l) of part k.
      const bool is = lane < p.cluster;
      const float Mk = is ? lds_cluster(smem_u32(&s_fin[r]), lane) : -CUDART_INF_F;
      const float lk = is ? lds_cluster(smem_u32(&s_fin[r]) + 4, lane) : 0.0f;
      float x[8][CH / 32];
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int i = 0; i < CH / 32; ++i)
          x[k][i] = k < p.cluster ? lds_cluster(smem_u32(&s_sum[r * CH + 32 * i + lane]), k) : 0.0f;
      float Mr = Mk;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) Mr = fmaxf(Mr, __shfl_xor_sync(0xffffffffu, Mr, o));
      const float f = Mk == -CUDART_INF_F ? 0.0f : ex2(Mk - Mr);
      float lr = f * lk;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) lr += __shfl_xor_sync(0xffffffffu, lr, o);
      Mr = __shfl_sync(0xffffffffu, Mr, 0);
      lr = __shfl_sync(0xffffffffu, lr, 0);
      const float inv = lr > 0.0f ? 1.0f / lr : 0.0f;
      const int64_t row = out_row(p, w, head, r);
#pragma unroll
      for (int i = 0; i < CH / 32; ++i) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum = __fmaf_rn(__shfl_sync(0xffffffffu, f, k), x[k][i], sum);
        if (32 * i + lane < cv.d) store_out(p.o, row * cv.d + 32 * i + lane, sum * inv, p.o_dt);
      }
      if (lane == 0 && p.lse != nullptr) p.lse[row] = lr > 0.0f ? (Mr + log2f(lr)) * CUDART_LN2_F : -CUDART_INF_F;
    }
    // No CTA leaves while another reads its shared memory.
    cluster_arrive();
    cluster_wait();
  }
  // Before the next (tile, head) uses the shared memory, by copies too.
  fence_proxy_async_smem();
  __syncthreads();
  }
}

// Joins the parts of a (tile, head) that the line of units cut: o = sum_k 2^(M_k - M) o_k / sum_k
// 2^(M_k - M) l_k. A CTA takes `rows` rows of what one CTA of the first kernel left a note of, one after
// the other; of a row its warps take every fourth part, four channels per lane, and meet in shared
// memory.
__global__ void __launch_bounds__(kThreads) line_join_kernel(PagedAttnParams p, int bk, int rows) {
  __shared__ float s_x[2][kWarps][128];
  __shared__ float s_l[2][kWarps];
  const CacheView& cv = p.cache;
  const int cta = blockIdx.x % p.ctas, r0 = blockIdx.x / p.ctas * rows;
  // Every CTA waits, also one with nothing to join: this grid must not complete before the one
  // whose parts it joins.
  grid_dependency_wait();
  const JoinNote note = p.notes[cta];
  if (note.last < 0) return;
  const RowTile w = entry_tile(p, note.entry, bk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = note.last - cta + 1;
  const bool on = 4 * lane < cv.dp;
  for (int r = r0; r < min(r0 + rows, w.rows); ++r) {
    // Part k: slot 1 of the first CTA, slot 0 of the others.
    auto part = [&](int k) { return (static_cast<int64_t>(cta + k) * 2 + (k == 0 ? 1 : 0)) * p.row_tile + r; };
    float M = -CUDART_INF_F;
    for (int k = lane; k < n; k += 32) M = fmaxf(M, p.part_ml[part(k)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float ref = M == -CUDART_INF_F ? 0.0f : M;
    float l = 0.0f;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
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
    const int buf = r & 1;  // by turns, so that one barrier per row is enough
    *reinterpret_cast<float4*>(&s_x[buf][warp][4 * lane]) = x;
    if (lane == 0) s_l[buf][warp] = l;
    __syncthreads();
    const float lt = s_l[buf][0] + s_l[buf][1] + s_l[buf][2] + s_l[buf][3];
    const int64_t row = out_row(p, w, note.head, r);
    const int c = threadIdx.x;
    if (c < cv.d) {
      const float sum = s_x[buf][0][c] + s_x[buf][1][c] + s_x[buf][2][c] + s_x[buf][3][c];
      store_out(p.o, row * cv.d + c, lt > 0.0f ? sum / lt : 0.0f, p.o_dt);
    }
    if (c == 0 && p.lse != nullptr) p.lse[row] = lt > 0.0f ? (M + log2f(lt)) * CUDART_LN2_F : -CUDART_INF_F;
  }
}

template <int CPG, int NR>
cudaError_t launch_decode(const PagedAttnParams& p, int dt, cudaStream_t s) {
  static_assert((kWarps + 1) * 8 * NR * CPG * 8 * 4 + 8 * NR * 8 <= kWarps * Ring<CPG>::kBytes, "the warps' sums replace their rings");
  constexpr int smem = Ring<CPG>::total(8 * NR);
  cudaError_t e = allow_smem<paged_decode_kernel<CPG, NR>>(smem);
  if (e != cudaSuccess) return e;
  const CacheView& cv = p.cache;
  const int unit = v_unit(cv, kBlk);
  CUtensorMap map;
  if (!v_rows_map(cv, CPG * 8, unit, &map)) return cudaErrorInvalidValue;
  const int64_t tiles = static_cast<int64_t>(p.B) * p.row_tiles * cv.heads;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(static_cast<unsigned>(p.ctas > 0 ? p.ctas : tiles * p.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  // Its launch overlaps the end of the kernel before it; it waits for that one before it reads anything.
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (p.ctas == 0 && p.cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  e = cudaLaunchKernelEx(&cfg, paged_decode_kernel<CPG, NR>, p, dt == BA_F16 ? 1 : 0, unit, map);
  return e != cudaSuccess || p.ctas == 0 ? e : launch_line_join(p, kBlk, s);
}

}  // namespace

cudaError_t launch_line_join(const PagedAttnParams& p, int bk, cudaStream_t s) {
  // Few rows come in many parts, many rows in a few.
  const int rows = p.row_tile > 16 ? 8 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.ctas * (p.row_tile / rows)));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, line_join_kernel, p, bk, rows);
}

cudaError_t launch_paged_decode(const PagedAttnParams& p, int dt, cudaStream_t s) {
  if (p.cache.dp > 64) return p.row_tile > 8 ? launch_decode<16, 2>(p, dt, s) : launch_decode<16, 1>(p, dt, s);
  return p.row_tile > 8 ? launch_decode<8, 2>(p, dt, s) : launch_decode<8, 1>(p, dt, s);
}

void paged_decode_plan(PagedAttnParams* p, int sms) {
  const int64_t blocks = std::max<int64_t>(1, most_blocks(*p, p->row_tile, kBlk));
  const int64_t tiles = static_cast<int64_t>(p->B) * p->row_tiles * p->cache.heads;
  const int64_t fit = static_cast<int64_t>(sms) * ctas_per_sm(p->cache.dp > 64 ? 16 : 8, p->row_tile / 8);  // CTAs at once
  // Short contexts: a cluster of up to eight CTAs per (tile, head), down to a block per warp, joins
  // its parts itself. Where that leaves a warp more than kShort blocks beyond its share of an even
  // split over the GPU (or more than kShort of them, when the CTAs do not fit at once and ragged
  // lengths would leave some SMs waiting), the line of units and its second launch are faster. (8 KV
  // heads, d = 128, cluster and line: 1 x 4096 keys 9.1 and 11.2 us, 16 x 1024 11.3 and 14.8, 1 x 16384
  // 18.0 and 16.9, 64 x 4096 78 and 61.)
  int cluster = 1;
  while (cluster < 8 && blocks > cluster * kWarps && tiles * cluster * 2 <= fit) cluster *= 2;
  const int64_t mine = ceil_div(blocks, cluster * kWarps);
  const int64_t even = tiles * cluster <= fit ? blocks * tiles / (fit * kWarps) : 0;
  p->cluster = cluster;
  p->ctas = 0;
  if (mine - even > kShort)
    p->ctas = static_cast<int>(std::min<int64_t>(fit, ceil_div((blocks + kCost) * tiles, kWarps)));
}

static cudaError_t read_decode_status(int* value, cudaStream_t s) { return read_word(g_decode_status, value, s); }
static cudaError_t clear_decode_status(cudaStream_t s) { return clear_word(g_decode_status, s); }
StatusWord decode_status() { return {read_decode_status, clear_decode_status}; }

}  // namespace binattn
