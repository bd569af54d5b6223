// Attention of few query rows over the paged cache (sm_100a): decoding and drafts.
//
// With few rows per KV head the kernel is bound by reading the cache once: dp + 19 bytes per token
// and head. The work is laid out so that the arithmetic stays beside those loads:
//   * A CTA takes one sequence, one KV head, up to 8 NR rows (new tokens x heads of the group, which
//     share every key) and a part of the key axis. Each of its warps walks 32-key blocks of its own
//     through a ring of cp.async stages, with no synchronisation between warps until the end.
//   * Scores are XOR / popc on the CUDA cores: x = d - 2 popc, s = (scale mu_q mu_j log2 e) x, one
//     (key, row) pair per thread, placed so that the weights are the B fragment of the product.
//   * P.V runs on the tensor cores as V^T P^T (mma.sync m16n8k16, fp16 in, fp32 out): 16 channels x
//     16 keys of V against 16 keys x 8 rows, so that 8 rows fill the instruction (a 128-row
//     tcgen05 tile would be mostly empty, and the kernel waits for memory, not for the product).
//     The codes are whole numbers, exact in fp16; the order of the channels in a fragment is chosen
//     so that a thread's channels are neighbours in memory.
//   * A value row's exponent e_j joins the score instead of the codes: the weight is
//     2^(s_j + e_j - M) with M the running maximum of s_j + e_j, and the softmax sum adds
//     weight * 2^-e_j. M moves (and the sums are rescaled) only when a score passes it by more than
//     2^8, so that most blocks rescale nothing; the weights then reach 2^8, far inside fp16.
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
constexpr int kBlk = 32;        // keys per stage of a warp
constexpr int kStages = 3;
constexpr int kMinBlocks = 16;  // blocks (of 32 keys) a split takes at least
constexpr float kSlack = 8.0f;  // log2 by which scores may pass the running maximum

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes of two keys (4 channels each, biased by 128) -> fp16 pairs (key 0, key 1) of each channel.
// A byte u under the exponent of 1024 reads 1024 + u, so 1024 + u - 1152 is the signed code.
__device__ __forceinline__ void codes_to_half(uint32_t wa, uint32_t wb, uint32_t (&h)[4]) {
  wa ^= 0x80808080u;
  wb ^= 0x80808080u;
  const uint32_t lo = __byte_perm(wa, wb, 0x5140), hi = __byte_perm(wa, wb, 0x7362);
  const uint32_t x[4] = {__byte_perm(lo, 0x64646464u, 0x4140), __byte_perm(lo, 0x64646464u, 0x4342),
                         __byte_perm(hi, 0x64646464u, 0x4140), __byte_perm(hi, 0x64646464u, 0x4342)};
  const __half2 bias = __floats2half2_rn(-1152.0f, -1152.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 y = __hadd2(*reinterpret_cast<const __half2*>(&x[i]), bias);
    h[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// Shared memory of a warp's stage: V rows of kRow bytes (16-byte pieces permuted, see v_piece),
// sign rows, mu, exponents.
template <int CPG>  // channels per fragment row group: 16 (rows of 128 bytes) or 8 (rows of 64)
struct Stage {
  static constexpr int kRow = CPG * 8;
  static constexpr int offBits = kBlk * kRow;
  static constexpr int offMu = offBits + kBlk * 16;
  static constexpr int offExp = offMu + kBlk * 2;
  static constexpr int kBytes = offExp + kBlk;
  // Byte offset of the 16-byte piece c of key j. A warp's load of the fragment rows touches keys
  // 2t (t = 0..3) and neighbouring pieces: moving the pieces of key j by 2 ((j / 2) % 4) puts them
  // into different banks.
  static __device__ __forceinline__ int v_piece(int j, int c) {
    return ((j * (kRow / 16) + c) ^ (2 * ((j >> 1) & 3))) * 16;
  }
};

template <typename T, int CPG, int NR>
__global__ void __launch_bounds__(kThreads) paged_decode_kernel(PagedAttnParams p) {
  using S = Stage<CPG>;
  constexpr int MT = CPG / 2;   // 16-channel tiles
  constexpr int R = 8 * NR;     // rows of a CTA
  constexpr int CH = CPG * 8;   // channels of the accumulators (>= d)
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint4 s_bits[R];
  __shared__ float s_mu[R];
  __shared__ float2 s_ml[kWarps][R];

  const CacheView& cv = p.cache;
  int b, tile, head, split;
  cta_of(p, blockIdx.x, p.nsplit, b, tile, head, split);
  const RowTile w = row_tile(p, b, tile, kBlk);
  if (w.rows <= 0) return;
  const int used = splits_used(p.nsplit, w.nblk, kMinBlocks);
  if (split >= used) return;
  const int v0 = static_cast<int>(static_cast<int64_t>(w.nblk) * split / used);
  const int v1 = static_cast<int>(static_cast<int64_t>(w.nblk) * (split + 1) / used);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * kStages * S::kBytes;

  // The warp's blocks are v0 + warp, v0 + warp + kWarps, ... Lane l keeps the page and the offset
  // in it of the 16 tokens (l % 2) of the block l / 2 from `base` on: 16 blocks at a time.
  const int nmine = max(0, (v1 - v0 - warp + kWarps - 1) / kWarps);
  const int32_t* table = p.table + b * p.table_stride;
  PageAt at{-1, 0};
  auto look_up = [&](int base) {
    const int n = base + (lane >> 1);
    at.page = -1;
    if (n < nmine)
      at = page_at(p, table, w.kv, w.block_at(v0 + warp + n * kWarps) * kBlk + (lane & 1) * kPageUnit);
  };
  uint32_t seen = 0;  // two bits per stage: which halves of the block have a page
  auto issue = [&](int n) {
    if (n < nmine) {
      if ((n & 15) == 0) look_up(n);
      const int st = n % kStages;
      const uint32_t dst = ring + st * S::kBytes;
      uint32_t ok2 = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int page = __shfl_sync(0xffffffffu, at.page, 2 * (n & 15) + h);
        const int off = __shfl_sync(0xffffffffu, at.off, 2 * (n & 15) + h);
        const bool ok = page >= 0;
        ok2 |= (ok ? 1u : 0u) << h;
        const uint8_t* blk = ok ? cv.block(page, head) : cv.data;
        constexpr int PPR = S::kRow / 16;  // pieces of a row
#pragma unroll
        for (int i = 0; i < kPageUnit * PPR / 32; ++i) {
          const int idx = lane + 32 * i, j = idx / PPR, c = idx % PPR;
          if (c * 16 < cv.dp)
            cp_async16(dst + S::v_piece(kPageUnit * h + j, c), ok ? blk + (off + j) * cv.dp + c * 16 : blk, ok);
        }
        // The half's other pieces: 16 sign rows, two pieces of mu, one of exponents.
        if (lane < 19) {
          const uint8_t* src = lane < 16 ? blk + cv.off_bits() + (off + lane) * 16
                                         : (lane < 18 ? blk + cv.off_mu() + off * 2 + (lane - 16) * 16
                                                      : blk + cv.off_exp() + off);
          const uint32_t to = lane < 16 ? S::offBits + (kPageUnit * h + lane) * 16
                                        : (lane < 18 ? S::offMu + kPageUnit * h * 2 + (lane - 16) * 16
                                                     : S::offExp + kPageUnit * h);
          cp_async16(dst + to, ok ? src : blk, ok);
        }
      }
      seen = (seen & ~(3u << (2 * st))) | (ok2 << (2 * st));
    }
    cp_async_commit();
  };
#pragma unroll
  for (int n = 0; n < kStages - 1; ++n) issue(n);

  // Sign bits and scale of the rows, while the first blocks are on their way.
  for (int r = warp; r < R; r += kWarps) {
    uint4 bits = make_uint4(0u, 0u, 0u, 0u);
    float sum = 0.0f;
    if (r < w.rows) {
      const int i = (w.r0 + r) / p.group, hq = head * p.group + (w.r0 + r) % p.group;
      const T* src = static_cast<const T*>(p.q) + (w.t0 + i) * p.q_stride_t + hq * p.q_stride_h;
      uint32_t word[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = 32 * k + lane;
        const float x = c < cv.d ? load1<T>(src + c) : 0.0f;
        word[k] = __ballot_sync(0xffffffffu, x < 0.0f);
        sum += fabsf(x);
      }
      bits = make_uint4(word[0], word[1], word[2], word[3]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane == 0) {
      s_bits[r] = bits;
      s_mu[r] = sum / static_cast<float>(cv.d);
    }
  }
  __syncthreads();

  uint4 qb[NR];
  float cq[NR];
  int last[NR], wlo[NR];  // the row sees keys j <= last with j >= wlo or j < sinks
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int r = 8 * n + g;
    qb[n] = s_bits[r];
    cq[n] = p.scale_log2 * s_mu[r];
    const int pos = w.pos0() + (w.r0 + r) / p.group;
    last[n] = r < w.rows ? (p.causal ? min(pos, w.kv - 1) : w.kv - 1) : -1;
    wlo[n] = p.causal && p.window > 0 ? pos - p.window + 1 : 0;
  }
  // What every row of the tile sees: keys <= all_last from all_lo on.
  const int all_last = p.causal ? min(w.pos0() + w.r0 / p.group, w.kv - 1) : w.kv - 1;
  const int all_lo = p.causal && p.window > 0 ? w.pos0() + (w.r0 + w.rows - 1) / p.group - p.window + 1 : 0;

  float acc[NR][MT][4];
  float M[NR], l[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    M[n] = -CUDART_INF_F;
    l[n] = 0.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][m][i] = 0.0f;
  }
  const float dfl = static_cast<float>(cv.d);

  for (int n = 0; n < nmine; ++n) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    issue(n + kStages - 1);  // into the stage that the block before this one has left
    const int st = n % kStages;
    const uint32_t src = ring + st * S::kBytes;
    const int j0 = w.block_at(v0 + warp + n * kWarps) * kBlk;
    const uint32_t ok2 = (seen >> (2 * st)) & 3u;
    const bool whole = ok2 == 3u && j0 + kBlk - 1 <= all_last && j0 >= all_lo;

    // Scores s + e of this thread's 8 keys: key(u) = 16 (u / 4) + 2 t + {0, 1, 8, 9}[u % 4].
    float sc[NR][8], down[8];  // down = 2^-e
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int key = 16 * (u >> 2) + 2 * t + (u & 1) + 8 * ((u >> 1) & 1);
      const uint4 kb = lds128(src + S::offBits + key * 16);
      const float mu = __uint_as_float(lds16(src + S::offMu + key * 2) << 16);
      const int e = min(max(static_cast<int>(static_cast<int8_t>(lds16(src + S::offExp + (key & ~1)) >> (8 * (key & 1)))),
                            kMinExp), kMaxExp);
      down[u] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int diff = __popc(qb[r].x ^ kb.x) + __popc(qb[r].y ^ kb.y) + __popc(qb[r].z ^ kb.z) + __popc(qb[r].w ^ kb.w);
        const float x = __fmaf_rn(-2.0f, static_cast<float>(diff), dfl);
        sc[r][u] = __fmaf_rn(cq[r] * mu, x, static_cast<float>(e));
        if (!whole) {
          const int j = j0 + key;
          const bool see = ((ok2 >> (u >> 2)) & 1u) && j <= last[r] && (j >= wlo[r] || j < p.sinks);
          if (!see) sc[r][u] = -CUDART_INF_F;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float mx = sc[r][0];
#pragma unroll
      for (int u = 1; u < 8; ++u) mx = fmaxf(mx, sc[r][u]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const bool moves = mx > M[r] + kSlack;
      if (__any_sync(0xffffffffu, moves)) {
        const float to = moves ? mx : M[r];
        const float f = M[r] == -CUDART_INF_F ? 0.0f : ex2(M[r] - to);
        M[r] = to;
        l[r] *= f;
        const float f0 = __shfl_sync(0xffffffffu, f, 8 * t), f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          acc[r][m][0] *= f0;
          acc[r][m][1] *= f1;
          acc[r][m][2] *= f0;
          acc[r][m][3] *= f1;
        }
      }
      const float ref = M[r] == -CUDART_INF_F ? 0.0f : M[r];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        sc[r][u] = ex2(sc[r][u] - ref);
        l[r] = __fmaf_rn(sc[r][u], down[u], l[r]);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t bf[NR][2];
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const __half2 x = __floats2half2_rn(sc[r][4 * h + 2 * k], sc[r][4 * h + 2 * k + 1]);
          bf[r][k] = *reinterpret_cast<const uint32_t*>(&x);
        }
      uint32_t code[4][CPG / 4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = 16 * h + 2 * t + (k & 1) + 8 * (k >> 1);
        if constexpr (CPG == 16) {
          const uint4 x = lds128(src + S::v_piece(key, g));
          code[k][0] = x.x;
          code[k][1] = x.y;
          code[k][2] = x.z;
          code[k][3] = x.w;
        } else {
          const uint2 x = lds64(src + S::v_piece(key, g >> 1) + (g & 1) * 8);
          code[k][0] = x.x;
          code[k][1] = x.y;
        }
      }
#pragma unroll
      for (int x = 0; x < CPG / 4; ++x) {
        uint32_t ha[4], hb[4];
        codes_to_half(code[0][x], code[1][x], ha);
        codes_to_half(code[2][x], code[3][x], hb);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          mma16816(acc[r][2 * x], ha[0], ha[1], hb[0], hb[1], bf[r][0], bf[r][1]);
          mma16816(acc[r][2 * x + 1], ha[2], ha[3], hb[2], hb[3], bf[r][0], bf[r][1]);
        }
      }
    }
    __syncwarp();
  }
  cp_async_wait<0>();
  __syncthreads();

  // Join the warps: each leaves its (M, l) and its sums in shared memory. A thread holds, for the
  // rows 8 n + 2 t and 8 n + 2 t + 1, the channels CPG g .. CPG g + CPG - 1.
  float* s_o = reinterpret_cast<float*>(smem);  // [kWarps][R][CH]
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    l[n] += __shfl_xor_sync(0xffffffffu, l[n], 1);
    l[n] += __shfl_xor_sync(0xffffffffu, l[n], 2);
    if (t == 0) s_ml[warp][8 * n + g] = make_float2(M[n], l[n]);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<float2*>(s_o + (warp * R + 8 * n + 2 * t + i) * CH + CPG * g + 2 * m) =
            make_float2(acc[n][m][i], acc[n][m][2 + i]);
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
    const float inv = used > 1 ? 1.0f : (lr > 0.0f ? 1.0f / lr : 0.0f);
    for (int c = lane; c < cv.d; c += 32) {
      float x = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) x += f[k] * s_o[(k * R + r) * CH + c];
      if (used > 1)
        p.part_o[(split * p.T * p.heads + row) * cv.dp + c] = x;
      else
        store_out(p.o, row * cv.d + c, x * inv, p.o_dt);
    }
    if (lane == 0) {
      if (used > 1)
        p.part_ml[split * p.T * p.heads + row] = make_float2(Mr, lr);
      else if (p.lse != nullptr)
        p.lse[row] = lr > 0.0f ? (Mr + log2f(lr)) * CUDART_LN2_F : -CUDART_INF_F;
    }
  }
  allow_dependents();
}

// Joins the parts of each row: o = sum_k 2^(M_k - M) o_k / sum_k 2^(M_k - M) l_k. One warp per row.
__global__ void __launch_bounds__(kThreads) paged_join_kernel(PagedAttnParams p, int per_tile, int bk, int min_blocks) {
  const CacheView& cv = p.cache;
  int b, tile, head, part;
  cta_of(p, blockIdx.x, per_tile, b, tile, head, part);
  // Every CTA waits, also one with nothing to join: this grid must not complete before the one
  // whose parts it joins.
  grid_dependency_wait();
  const RowTile w = row_tile(p, b, tile, bk);
  if (w.rows <= 0) return;
  const int used = splits_used(p.nsplit, w.nblk, min_blocks);
  if (used == 1) return;
  const int lane = threadIdx.x & 31;
  const int64_t all = p.T * p.heads;
  for (int r = part * kWarps + (threadIdx.x >> 5); r < w.rows; r += per_tile * kWarps) {
    const int64_t row = (w.t0 + (w.r0 + r) / p.group) * p.heads + head * p.group + (w.r0 + r) % p.group;
    float M = -CUDART_INF_F;
    for (int k = lane; k < used; k += 32) M = fmaxf(M, p.part_ml[k * all + row].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float l = 0.0f, x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = 0; k < used; ++k) {
      const float2 ml = p.part_ml[k * all + row];
      if (ml.x == -CUDART_INF_F) continue;
      const float f = ex2(ml.x - M);
      l = __fmaf_rn(f, ml.y, l);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < cv.d) x[i] = __fmaf_rn(f, p.part_o[(k * all + row) * cv.dp + lane + 32 * i], x[i]);
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 32 * i < cv.d) store_out(p.o, row * cv.d + lane + 32 * i, x[i] * inv, p.o_dt);
    if (lane == 0 && p.lse != nullptr) p.lse[row] = l > 0.0f ? (M + log2f(l)) * CUDART_LN2_F : -CUDART_INF_F;
  }
}

template <typename T, int CPG, int NR>
cudaError_t launch_decode(const PagedAttnParams& p, cudaStream_t s) {
  constexpr int ring = kWarps * kStages * Stage<CPG>::kBytes, out = kWarps * 8 * NR * CPG * 8 * 4;
  constexpr int smem = ring > out ? ring : out;
  auto kernel = paged_decode_kernel<T, CPG, NR>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(p.B) * p.row_tiles * p.cache.heads;
  kernel<<<static_cast<unsigned>(tiles * p.nsplit), kThreads, smem, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess || p.nsplit == 1) return e;
  return launch_paged_join(p, kBlk, kMinBlocks, s);
}

template <typename T>
cudaError_t launch_decode_t(const PagedAttnParams& p, cudaStream_t s) {
  if (p.cache.dp > 64) return p.row_tile > 8 ? launch_decode<T, 16, 2>(p, s) : launch_decode<T, 16, 1>(p, s);
  return p.row_tile > 8 ? launch_decode<T, 8, 2>(p, s) : launch_decode<T, 8, 1>(p, s);
}

}  // namespace

cudaError_t launch_paged_join(const PagedAttnParams& p, int bk, int min_blocks, cudaStream_t s) {
  // A CTA joins two rows per warp.
  const int per_tile = p.row_tile / (2 * kWarps);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(p.B) * p.row_tiles * p.cache.heads * per_tile));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel, p, per_tile, bk, min_blocks);
}

cudaError_t launch_paged_decode(const PagedAttnParams& p, int dt, cudaStream_t s) {
  return dt == BA_F16 ? launch_decode_t<__half>(p, s) : launch_decode_t<__nv_bfloat16>(p, s);
}

int paged_decode_splits(const PagedAttnParams& p, int sms) {
  // Keys that a tile can see, in blocks; four CTAs of a split fill an SM.
  int64_t keys = p.max_kv_len;
  if (p.causal && p.window > 0)
    keys = std::min<int64_t>(keys, static_cast<int64_t>(p.window) + p.row_tile + p.sinks + 2 * kBlk);
  const int64_t blocks = ceil_div(keys, kBlk), tiles = static_cast<int64_t>(p.B) * p.row_tiles * p.cache.heads;
  const int64_t want = ceil_div(static_cast<int64_t>(sms) * 4, tiles);
  return static_cast<int>(std::max<int64_t>(1, std::min(want, blocks / kMinBlocks)));
}

}  // namespace binattn
