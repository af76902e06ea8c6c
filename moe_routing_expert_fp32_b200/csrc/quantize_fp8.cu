// quantize_fp8.cu -- bf16 to the library's 8-bit block-scaled format: e4m3
// values q with an fp32 scale s per block, value = q * s.
//
//   a = max |x| over the block (a NaN stays a NaN)
//   s = fl32(max(a, 2^-100) / 448), with power-of-two scales rounded up to one
//   q = e4m3(fl32(x * fl32(1 / s))), to nearest even, at most 448 in magnitude
//
// The floor 2^-100 keeps 1/s finite for a block of zeros (all q = 0).  x * 1/s
// instead of x / s costs one rounding of 2^-24, against the 2^-4 of e4m3, and
// saves a division per element; with power-of-two scales the product is exact.
// An infinity gives s = inf and q = NaN at its place, so it reaches every
// product of its row as a NaN.
//
// A block is 128 columns of one row (activations) or 128 x 128 (weights).
// Both kernels make one pass: a block's values stay in registers between the
// maximum and the rounding.  Bound by HBM: 2 bytes read and 1 written per value.
#include "fp8.cuh"
#include "moe_internal.cuh"

namespace moe {
namespace {

using fp8::block_scale;
using fp8::pack4;

// max over the two bf16 magnitudes of each word, as 16-bit integers: the
// order of the magnitudes, with NaN above infinity
__device__ __forceinline__ uint32_t amax2(uint32_t m, uint32_t w) {
  return __vmaxu2(m, w & 0x7fff7fffu);
}
__device__ __forceinline__ uint32_t amax8(uint32_t m, const uint4& v) {
  return amax2(amax2(amax2(amax2(m, v.x), v.y), v.z), v.w);
}
__device__ __forceinline__ uint2 quant8(const uint4& v, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __fmul_rn(__uint_as_float(w[i] << 16), inv);
    f[2 * i + 1] = __fmul_rn(__uint_as_float(w[i] & 0xffff0000u), inv);
  }
  return make_uint2(pack4(f[0], f[1], f[2], f[3]), pack4(f[4], f[5], f[6], f[7]));
}

// Eight lanes per block of 128 columns, 16 columns each (two 16-byte loads, one
// 16-byte store).
// SCATTER: row t goes to the `top_k` rows pos[t * top_k + k] (a dispatched
// token; -1 where the slot was left out).  Its values are read and quantised
// before the wait on the kernel before (the sort, which writes only pos).
template <bool SCATTER>
__global__ void __launch_bounds__(256) k_quantize_rows(const __nv_bfloat16* __restrict__ x,
                                                       int64_t M, int K, int KB, int pow2,
                                                       uint8_t* __restrict__ q,
                                                       float* __restrict__ scale,
                                                       const int32_t* __restrict__ pos,
                                                       int top_k, int64_t S) {
  if (!SCATTER) pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, l8 = lane & 7;
  const int64_t blocks = M * KB;
  const int64_t b = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3);
  if ((int64_t)blockIdx.x * 32 + (threadIdx.x >> 5) * 4 >= blocks) return;  // whole warp
  const bool live = b < blocks;
  int64_t row;
  int kb;
  if (blocks <= 0x7fffffff) {
    const uint32_t r = (uint32_t)b / (uint32_t)KB;
    row = r;
    kb = (int)((uint32_t)b - r * (uint32_t)KB);
  } else {
    row = b / KB;
    kb = (int)(b - row * KB);
  }
  const int c = kb * 128 + 16 * l8;
  const bool in = live && c < K;  // K is a multiple of 16
  const uint4* src = reinterpret_cast<const uint4*>(x + row * K + c);
  uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
  if (in) {
    v0 = __ldg(src);
    v1 = __ldg(src + 1);
  }
  uint32_t m2 = amax8(amax8(0u, v0), v1);
  uint32_t m = max(m2 >> 16, m2 & 0xffffu);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  float inv;
  const float s = block_scale(__uint_as_float(m << 16), pow2, inv);
  const uint2 q0 = quant8(v0, inv), q1 = quant8(v1, inv);
  if (SCATTER) pdl_wait();
  if (!live) return;
  auto store = [&](int64_t r) {
    if (in) *reinterpret_cast<uint4*>(q + r * K + c) = make_uint4(q0.x, q0.y, q1.x, q1.y);
    if (l8 == 0) scale[r * KB + kb] = s;
  };
  if (SCATTER) {
    for (int k = 0; k < top_k; ++k) {
      const int32_t p = pos[row * top_k + k];
      if (p >= 0 && p < S) store(p);
    }
  } else {
    store(row);
  }
}

// One CTA per 128 x 128 block: 16 lanes cover a row of the block, the CTA 16
// rows at a time, eight times; 32 KB per CTA are loaded before any is used.
__global__ void __launch_bounds__(256) k_quantize_blocks(const __nv_bfloat16* __restrict__ x,
                                                         int64_t M, int K, int MB, int KB,
                                                         int pow2, uint8_t* __restrict__ q,
                                                         float* __restrict__ scale) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint32_t part[8];
  const int64_t blk = blockIdx.x;
  const int64_t bm = blk / KB;  // batch * MB + row block
  const int kb = (int)(blk - bm * KB);
  const int64_t batch = bm / MB;
  const int64_t r0 = (bm - batch * MB) * 128;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = kb * 128 + 8 * (threadIdx.x & 15), rr = threadIdx.x >> 4;
  const int64_t base = batch * M * K;
  uint4 v[8];
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i + rr;
    v[i] = make_uint4(0, 0, 0, 0);
    if (r < M && c < K) v[i] = __ldg(reinterpret_cast<const uint4*>(x + base + r * K + c));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m2 = amax8(m2, v[i]);
  uint32_t m = max(m2 >> 16, m2 & 0xffffu);
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) part[warp] = m;
  __syncthreads();
  m = part[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max(m, part[i]);
  float inv;
  const float s = block_scale(__uint_as_float(m << 16), pow2, inv);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i + rr;
    if (r < M && c < K) *reinterpret_cast<uint2*>(q + base + r * K + c) = quant8(v[i], inv);
  }
  if (threadIdx.x == 0) scale[blk] = s;
}

}  // namespace

cudaError_t launch_quantize_rows(const __nv_bfloat16* x, int64_t M, int K, bool pow2, uint8_t* q,
                                 float* scale, const int32_t* pos, int top_k, int64_t S,
                                 cudaStream_t s) {
  const int KB = (K + 127) / 128;
  const unsigned grid = (unsigned)((M * KB + 31) / 32);
  if (pos)
    return launch_pdl(k_quantize_rows<true>, dim3(grid), dim3(256), 0, s, x, M, K, KB,
                      pow2 ? 1 : 0, q, scale, pos, top_k, S);
  return launch_pdl(k_quantize_rows<false>, dim3(grid), dim3(256), 0, s, x, M, K, KB,
                    pow2 ? 1 : 0, q, scale, pos, 0, (int64_t)0);
}

cudaError_t launch_quantize_blocks(const __nv_bfloat16* x, int64_t B, int64_t M, int K, bool pow2,
                                   uint8_t* q, float* scale, cudaStream_t s) {
  const int KB = (K + 127) / 128;
  const int MB = (int)((M + 127) / 128);
  return launch_pdl(k_quantize_blocks, dim3((unsigned)(B * MB * KB)), dim3(256), 0, s, x, M, K,
                    MB, KB, pow2 ? 1 : 0, q, scale);
}

}  // namespace moe
