// Writing rows of K and V into the paged cache, and reading them back (sm_100a).
//
// Per (token, head) row: the sign bits of k, mu = bf16(mean |k|), the least exponent e with
// max |v| <= 127 2^e, and the codes rne(v 2^-e). Both kernels are bound by memory: a written row
// reads 4 d bytes and writes dp + 19.
//
// A half-warp takes a row of one head at a time, eight channels per lane: 16-byte loads of k and v, one
// sign byte and eight code bytes per lane, so that a row's 16 sign bytes and its codes leave as one
// piece each. The two reductions (sum |k|, max |v|) are four shuffles each. Neighbouring half-warps take
// neighbouring heads of a token, whose rows lie next to each other in k and v. (Two, four or eight rows
// in flight per half-warp were no faster on large calls and slower on small ones; so was a half-warp's
// neighbour taking the next token of the same head.) Stores of read rows are streaming: they are as
// large as all of L2 on long contexts.
//
// 16384 tokens x 8 heads x 128 channels (d): written in 20 us (4.3 TB/s of 512 bytes read and 147 written a row, 19 of
// which in pieces of 16, 2 and 1; what binds it is not established), read in 14 us (6.2 TB/s, all from L2); 65536
// tokens read in 72 to 78 us (4.4 to 4.8 TB/s, nor there); 8 tokens of 16 heads 1.8 us each way, of which a launch
// alone is most.
#include "kernels.h"
#include "paged.cuh"

namespace binattn {

namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 16;  // lanes of a row
constexpr int kHalves = kThreads / kLanes;  // rows of a CTA

// The least e with amax <= 127 * 2^e, held to [kMinExp, kMaxExp]. amax = f * 2^x with
// 1 <= f < 2 gives x - 6 when f <= 127/64 (mantissa bits up to 0x7e0000), else x - 5. Zero and
// numbers below fp32's normal range have a zero exponent field and end at kMinExp.
__device__ __forceinline__ int row_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int x = static_cast<int>(u >> 23) - 127;
  const int e = x - ((u & 0x7fffffu) <= 0x7e0000u ? 6 : 5);
  return min(max(e, kMinExp), kMaxExp);
}

// Eight channels of a row of k or v as they come (channels from d on are 0).
template <typename T, bool WIDE>
__device__ __forceinline__ uint4 load_row8(const T* row, int c0, int d) {
  uint4 u = make_uint4(0u, 0u, 0u, 0u);
  if (WIDE) {
    if (c0 < d) u = ldg_stream(row + c0);
  } else {
    const uint16_t* x = reinterpret_cast<const uint16_t*>(row);
    uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + i < d) w[i / 2] |= static_cast<uint32_t>(__ldg(x + c0 + i)) << (16 * (i % 2));
  }
  return u;
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(CacheWriteParams p) {
  const CacheView& cv = p.cache;
  const int c0 = (threadIdx.x % kLanes) * 8, row = blockIdx.x * kHalves + threadIdx.x / kLanes;
  // Every lane stays for the shuffles; lanes of a row that is not written load nothing.
  const bool in = row < static_cast<int>(p.T) * cv.heads;
  const int t = in ? p.by_heads(row) : 0, h = in ? row - t * cv.heads : 0;
  int off = 0;
  const int64_t page = in ? page_of_slot(cv, p.by_page, p.slots[t], off) : -1;
  const int d = page >= 0 ? cv.d : 0;
  float k[8], v[8];
  unpack8<T>(load_row8<T, WIDE>(static_cast<const T*>(p.k) + t * p.k_stride_t + h * p.k_stride_h, c0, d), k);
  unpack8<T>(load_row8<T, WIDE>(static_cast<const T*>(p.v) + t * p.v_stride_t + h * p.v_stride_h, c0, d), v);
  uint32_t neg = 0;
  float sum = 0.0f, amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    neg |= (k[i] < 0.0f ? 1u : 0u) << i;
    sum += fabsf(k[i]) * kMeanStep;
    amax = fmaxf(amax, fabsf(v[i]));
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  }
  if (page < 0) return;
  uint8_t* blk = cv.block(page, h);
  blk[cv.off_bits() + off * 16 + c0 / 8] = static_cast<uint8_t>(neg);
  const int e = row_exp(amax);
  if (c0 == 0) {
    *reinterpret_cast<__nv_bfloat16*>(blk + cv.off_mu() + off * 2) = __float2bfloat16_rn(mean_of(sum, cv.d));
    *reinterpret_cast<int8_t*>(blk + cv.off_exp() + off) = static_cast<int8_t>(e);
  }
  if (c0 < cv.dp) {
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e: v * inv is exact
    if (e == kMaxExp) {  // only there can a value lie beyond 127 steps
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(v[i], -127.0f * 512.0f), 127.0f * 512.0f);
    }
    // v * inv + 1.5 * 2^23 rounds to the nearest whole number, ties to even, in the low bits.
    uint32_t q[8], w[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __float_as_uint(__fmaf_rn(v[i], inv, 12582912.0f));
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = __byte_perm(__byte_perm(q[4 * i], q[4 * i + 1], 0x0040), __byte_perm(q[4 * i + 2], q[4 * i + 3], 0x0040),
                         0x5410);
    *reinterpret_cast<uint2*>(blk + off * cv.dp + c0) = make_uint2(w[0], w[1]);
  }
}

template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half narrow<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <typename T, bool WIDE>
__device__ __forceinline__ void store_row8(T* row, int c0, int d, const float f[8]) {
  if (WIDE) {
    if (c0 >= d) return;
    alignas(16) T out[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = narrow<T>(f[i]);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(out) / 16); ++i)
      __stcs(reinterpret_cast<uint4*>(row + c0) + i, reinterpret_cast<const uint4*>(out)[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + i < d) row[c0 + i] = narrow<T>(f[i]);
  }
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(CacheReadParams p) {
  const CacheView& cv = p.cache;
  const int c0 = (threadIdx.x % kLanes) * 8, row = blockIdx.x * kHalves + threadIdx.x / kLanes;
  if (row >= static_cast<int>(p.T) * cv.heads || c0 >= cv.d) return;
  const int t = p.by_heads(row);
  int off = 0;
  const int64_t page = page_of_slot(cv, p.by_page, p.slots[t], off);
  uint32_t neg = 0;
  float mu = 0.0f, step = 0.0f;
  uint2 code = make_uint2(0u, 0u);
  if (page >= 0) {
    const uint8_t* blk = cv.block(page, row - t * cv.heads);
    neg = blk[cv.off_bits() + off * 16 + c0 / 8];
    mu = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(blk + cv.off_mu() + off * 2));
    const int e = *reinterpret_cast<const int8_t*>(blk + cv.off_exp() + off);
    step = __uint_as_float(static_cast<uint32_t>(127 + max(e, -126)) << 23);
    code = *reinterpret_cast<const uint2*>(blk + off * cv.dp + c0);
  }
  const int64_t at = static_cast<int64_t>(row) * cv.d;
  float f[8];
  if (p.k != nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (neg >> i) & 1u ? -mu : mu;
    store_row8<T, WIDE>(static_cast<T*>(p.k) + at, c0, cv.d, f);
  }
  if (p.v != nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f[i] = static_cast<float>(static_cast<int8_t>((i < 4 ? code.x : code.y) >> (8 * (i % 4)))) * step;
    store_row8<T, WIDE>(static_cast<T*>(p.v) + at, c0, cv.d, f);
  }
}

unsigned grid_for(int64_t rows) { return static_cast<unsigned>(ceil_div(rows, kHalves)); }

template <typename T>
cudaError_t launch_write(const CacheWriteParams& p, cudaStream_t s) {
  const unsigned grid = grid_for(p.T * p.cache.heads);
  if (p.wide)
    cache_write_kernel<T, true><<<grid, kThreads, 0, s>>>(p);
  else
    cache_write_kernel<T, false><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_read(const CacheReadParams& p, cudaStream_t s) {
  const unsigned grid = grid_for(p.T * p.cache.heads);
  if (p.cache.d % 8 == 0)
    cache_read_kernel<T, true><<<grid, kThreads, 0, s>>>(p);
  else
    cache_read_kernel<T, false><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteParams& p, int dt, cudaStream_t s) {
  return dt == BA_F16 ? launch_write<__half>(p, s) : launch_write<__nv_bfloat16>(p, s);
}

cudaError_t launch_cache_read(const CacheReadParams& p, int dt, cudaStream_t s) {
  if (dt == BA_F16) return launch_read<__half>(p, s);
  if (dt == BA_BF16) return launch_read<__nv_bfloat16>(p, s);
  return launch_read<float>(p, s);
}

}  // namespace binattn
