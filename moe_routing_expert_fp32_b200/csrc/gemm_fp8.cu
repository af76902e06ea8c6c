// gemm_fp8.cu -- products of 8-bit block-scaled operands on the 5th-generation
// tensor cores: the dense Linear, the Linear grouped by expert over ragged row
// segments, and the expert MLP (gate/up products, activation, requantisation;
// down product).
//
//   y[m, n] = sum_b  sx[m, b] * sw[n / 128, b] * sum_{k in block b} qx[m, k] qw[n, k]
//
// The scales change every 128 columns of K, so a product cannot run through K
// in the tensor core's accumulator: the MMAs of one K block (4 of K = 32,
// kind::f8f6f4, e4m3 x e4m3 -> fp32) write a fresh TMEM buffer, and the epilogue
// warps add it, times sx * sw, to fp32 sums in registers, while the MMAs of the
// next block fill another buffer.
//
// Layout: token rows are the MMA's M side (TMEM lane = token row), weight rows
// its N side.  Each thread then owns part of one row: its scale of a K block is
// one register times one value shared by the warp, and the largest |h| of a
// 128-column block is a maximum over its own registers (and one neighbour's).
//   * gate_up: the N side is 128 rows of w1 over the same 128 rows of w3, so a
//     unit yields whole 128-column blocks of h, which it rounds to e4m3 itself;
//   * few rows per segment: k_gemm_fp8_dec turns the sides round.
// Roles: 8 epilogue warps (lane quarter = warp % 4, column half = warp / 4), one
// TMA warp, one MMA warp; a ring of stages guarded by mbarriers; a persistent
// grid over units (token tile, weight block), weight block fastest.  Every wait
// is bounded as in expert_gemm.cu.
#include <cuda.h>

#include <cuda_fp16.h>
#include <float.h>

#include "fp8.cuh"
#include "moe_internal.cuh"
#include "sm100.cuh"

namespace moe {
namespace {

using sm100::mbar_arrive;
using sm100::mbar_arrive_expect_tx;
using sm100::mbar_init;
using sm100::mbar_wait;
using sm100::smem_u32;
using sm100::tc_fence_after;
using sm100::tc_fence_before;
using sm100::tma_load_2d;
using sm100::tma_load_3d;
using sm100::umma_commit;

constexpr int BM = 128;        // MMA M: token rows
constexpr int BK = 128;        // K per stage = scale block = one 128-byte swizzle row
constexpr int UK = 32;         // K per tcgen05.mma for 8-bit inputs
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarps + 4);  // + TMA warp, MMA warp, two idle (whole warpgroups)
// Registers per thread after the split of the launch's 168 x 384: the epilogue
// holds 128 sums and a 32-column TMEM load, the other warpgroup next to nothing.
constexpr int kEpiRegs = 216, kCtlRegs = 72;
static_assert(kEpiRegs * 32 * kEpiWarps + kCtlRegs * 128 <= 168 * kThreads, "register split");
constexpr int kTmemCols = 512;
constexpr int kSmallBox = 16;  // token rows per small TMA box
constexpr int kMaxSegments = 1024;

constexpr int kBarBytes = 320;
// On the abort path: how long a role waits for copies or MMAs still in flight.
constexpr uint64_t kDrainNs = 100000000ull;

enum Mode { kPlain = 0, kGateUp = 1 };

// BN weight rows per unit: 256 keep the tensor cores busiest (a K block's tokens
// are read from L2 once for twice the MMAs); 128 make twice the units, for
// products whose units would not fill the GPU.  gate_up: 128 rows of w1 and the
// same 128 of w3.
template <int MODE, int BN>
struct Cfg {
  static constexpr int kStages = BN == 256 ? 4 : 6;
  static constexpr int kABytes = BM * BK;
  static constexpr int kBBytes = BN * BK;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kBufs = kTmemCols / BN;
  static constexpr int kStartBytes = (kMaxSegments + 1) * 4;
  static constexpr int kAmaxBytes = 2 * 2 * BM * 4;  // unit parity x half x row
  static constexpr int kOutCols = 32;  // columns that a warp stores at a time
  static constexpr int kOutBytes = 32 * kOutCols * 2;  // of a warp's 32 rows
  static constexpr size_t kSmem = (size_t)kStages * kStageBytes + 1024 + kBarBytes +
                                  kAmaxBytes + kEpiWarps * kOutBytes + 2 * kStartBytes;
  static constexpr int kCache = kMaxSegments + 1;  // offsets held in shared memory
  static_assert(kABytes % 1024 == 0 && kBBytes % 1024 == 0, "1024-byte aligned operands");
  static_assert(MODE == kPlain || BN == 256, "gate_up: 128 rows of w1 and of w3");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct Args {
  const int32_t* offsets;  // [E + 1], or nullptr: one segment of all S rows
  int E;
  int64_t S;
  int N;    // output columns (gate_up: d_ff)
  int K;
  const float* xs;   // [S, KB]
  const float* ws0;  // [E, NB, KB]
  const float* ws1;  // gate_up: w3's
  __nv_bfloat16* y;  // plain: [S, N]
  const __nv_bfloat16* res;
  uint8_t* hq;       // gate_up: [S, N] e4m3
  float* hs;         // gate_up: [S, NB]
  int act_kind;
  float beta, lbeta;
  int pow2;
  int early;  // offsets were complete before the preceding kernel started
  int reset;  // the first kernel of its call: it clears the status word
  int probe;
  DeviceStatus* st;
};

__device__ __forceinline__ void umma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}
// Instruction descriptor: e4m3 x e4m3 -> fp32, both K-major.
__device__ __forceinline__ uint32_t idesc_e4m3(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// (acc.x, acc.y) += (lo, hi) * (c.x, c.y), each rounded once: one instruction
// for two sums.
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t lo, uint32_t hi, uint64_t c) {
  asm("{\n\t.reg .b64 t;\n\tmov.b64 t, {%1, %2};\n\tfma.rn.f32x2 %0, t, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(lo), "r"(hi), "l"(c));
}
__device__ __forceinline__ uint64_t pair_of(float v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// The activation in fp32.  sigmoid(g) = 1/(1 + e^-g); beta tanh(x) with x = g/beta is
// beta (1 - e^-2|x|)/(1 + e^-2|x|) with x's sign, and below |x| = 0.125, where the
// numerator would cancel, g times tanh(x)/x by its Taylor series to x^4 (the next term
// is 2^-22 of it).  Nothing here grows past its result, however large the parameters
// are: each tanh takes its own before the two meet.  The two share one reciprocal.  Error against the value: the rounded argument of 2^x gives
// |g| 2^-24 of it (2^-18.5 at g = -80), the cancellation 2^-21 per tanh at |x| = 0.125;
// elsewhere a few steps of fp32.  The forms of 2^x and 1/x that flush subnormals take
// one instruction each; sigmoid is 0 for g below -87.  At 4096 rows over 32 experts,
// 2048 to 1024 and back, the MLP takes 70 us with SiTU and 59 with SiLU.
struct Act {
  bool situ, has_lb;
  float beta, lbeta, inv_beta, inv_lbeta;
};
__device__ __forceinline__ Act make_act(int kind, float beta, float lbeta) {
  Act t;
  t.situ = kind == MOE_ACT_SITU;
  t.has_lb = !(lbeta == 0.0f || lbeta != lbeta);
  t.beta = (beta == 0.0f || beta != beta) ? 1.0f : beta;
  t.lbeta = lbeta;
  // (finite below 2^-128 too, where 0 times an infinity would make a gate of 0 NaN;
  // arguments that such a limit does not saturate are subnormal themselves)
  auto inverse = [](float b) { return fmaxf(-FLT_MAX, fminf(__fdiv_rn(1.0f, b), FLT_MAX)); };
  t.inv_beta = inverse(t.beta);
  t.inv_lbeta = t.has_lb ? inverse(lbeta) : 0.0f;
  return t;
}
__device__ __forceinline__ float exp2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;
// The same for one element (T = float) or two (a pair in 64 bits), which halves the
// instructions on sums and products.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
template <typename T>
__device__ __forceinline__ T all_of(float v) {
  if constexpr (sizeof(T) == 8) return pair_of(v);
  else return v;
}
__device__ __forceinline__ float mul(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ float add(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ float mad(float a, float b, float c) { return __fmaf_rn(a, b, c); }
__device__ __forceinline__ uint64_t mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mad(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
template <typename F>
__device__ __forceinline__ float each(F f, float v) { return f(v); }
template <typename F>
__device__ __forceinline__ uint64_t each(F f, uint64_t v) {
  return pair_of(f(lo_of(v)), f(hi_of(v)));
}
__device__ __forceinline__ float where_below(float x, float limit, float a, float b) {
  return x < limit ? a : b;
}
__device__ __forceinline__ uint64_t where_below(uint64_t x, float limit, uint64_t a, uint64_t b) {
  return pair_of(lo_of(x) < limit ? lo_of(a) : lo_of(b), hi_of(x) < limit ? hi_of(a) : hi_of(b));
}
__device__ __forceinline__ float sign_of(float v, float s) { return copysignf(v, s); }
__device__ __forceinline__ uint64_t sign_of(uint64_t v, uint64_t s) {
  return pair_of(copysignf(lo_of(v), lo_of(s)), copysignf(hi_of(v), hi_of(s)));
}
// b tanh(v / b) = num / den, 1 <= den <= 2; inv = 1 / b
template <typename T>
__device__ __forceinline__ void tanh_parts(T v, float b, float inv, T& num, T& den) {
  const T one = all_of<T>(1.0f), x = mul(v, all_of<T>(inv)), x2 = mul(x, x);
  const T p = mul(v, mad(x2, mad(x2, all_of<T>(2.0f / 15), all_of<T>(-1.0f / 3)), one));
  const T e = each([](float y) { return exp2_ftz(-fabsf(y)); }, mul(x, all_of<T>(2.0f * kLog2e)));
  num = where_below(x2, 0.015625f, p,
                    mul(sign_of(mad(e, all_of<T>(-1.0f), one), x), all_of<T>(b)));
  den = where_below(x2, 0.015625f, one, add(e, one));
}
template <typename T>
__device__ __forceinline__ T sigmoid(T g) {
  return each(rcp_ftz, add(each(exp2_ftz, mul(g, all_of<T>(-kLog2e))), all_of<T>(1.0f)));
}
// f(h function): one copy of the caller's loop for each activation, so that the
// choice is not made per element.
template <typename F>
__device__ __forceinline__ void with_act(const Act& t, F&& f) {
  if (!t.situ) {
    f([](auto g, auto u) { return mul(mul(g, sigmoid(g)), u); });
  } else if (!t.has_lb) {
    f([&](auto g, auto u) {
      decltype(g) n, d;
      tanh_parts(g, t.beta, t.inv_beta, n, d);
      return mul(mul(mul(n, each(rcp_ftz, d)), sigmoid(g)), u);
    });
  } else {
    f([&](auto g, auto u) {
      decltype(g) n1, d1, n2, d2;
      tanh_parts(g, t.beta, t.inv_beta, n1, d1);
      tanh_parts(u, t.lbeta, t.inv_lbeta, n2, d2);
      return mul(mul(mul(n1, each(rcp_ftz, mul(d1, d2))), sigmoid(g)), n2);
    });
  }
}

// Token tiles of `tile` rows per segment and their prefix into tile_start
// [E + 1] (shared memory), by every CTA for itself.  A segment that is not
// inside [0, S] or runs backwards is recorded and gets no tile, so no row out
// of range is touched.  Every thread of the CTA calls it, after the wait on the
// kernel before; it ends with a __syncthreads.  Returns the offsets: a copy in
// `cache` (shared memory, CACHE entries), since every role looks them up for
// every unit, or the caller's where they are too many.
template <int THREADS, int CACHE>
__device__ __forceinline__ const int32_t* build_tiles(const Args& a, int tile,
                                                      int32_t* tile_start, int32_t* cache,
                                                      int32_t* warp_tot) {
  constexpr int kPer = (kMaxSegments + THREADS) / THREADS;  // segments per thread, and E itself
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.E;
  if (a.reset && blockIdx.x == 0) {
    // instead of a memset before the kernel; the other CTAs record nothing but
    // waits that have run out, long after this
    if (threadIdx.x == 0) *a.st = DeviceStatus{0, 0};
    __syncwarp();  // (the first warp may record next; for the others, the barrier below)
  }
  if (E <= 128) {
    // few segments (or one, of all rows): the first warp alone, four a lane
    if (warp == 0) {
      const int f0 = 4 * lane;
      int32_t o[5], n4[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 5; ++i)
        o[i] = f0 + i > E ? 0 : a.offsets ? a.offsets[f0 + i] : f0 + i ? (int32_t)a.S : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        n4[i] = 0;
        if (f0 + i < E) {
          const bool bad = o[i] < 0 || o[i + 1] < o[i] || o[i + 1] > a.S || (f0 + i == 0 && o[0]);
          if (!bad) n4[i] = (int32_t)(((int64_t)o[i + 1] - o[i] + tile - 1) / tile);
          else if (blockIdx.x == 0) record_error(a.st, MOE_ERR_DEVICE_BOUNDS, 300);
        }
        sum += n4[i];
      }
      int32_t x = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int32_t t = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += t;
      }
      x -= sum;
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        if (f0 + i <= E && (i < 4 || lane == 31)) {
          tile_start[f0 + i] = x;
          cache[f0 + i] = o[i];
        }
        if (i < 4) x += n4[i];
      }
    }
    __syncthreads();
    return cache;
  }
  const int32_t* off = a.offsets;
  if (E < CACHE) {
    for (int e = threadIdx.x; e <= E; e += THREADS)
      cache[e] = a.offsets[e];
    off = cache;
  }
  __syncthreads();
  const int e0 = kPer * threadIdx.x;
  int32_t n[kPer], sum = 0;
  if (e0 < E) {
    int32_t lo = off[e0];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      n[i] = 0;
      if (e0 + i < E) {
        const int32_t hi = off[e0 + i + 1];
        const bool bad = lo < 0 || hi < lo || hi > a.S || (e0 + i == 0 && lo != 0);
        if (!bad) n[i] = (int32_t)(((int64_t)hi - lo + tile - 1) / tile);
        else if (blockIdx.x == 0) record_error(a.st, MOE_ERR_DEVICE_BOUNDS, 300);
        lo = hi;
      }
      sum += n[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) n[i] = 0;
  }
  int32_t x = sum;
#pragma unroll
  for (int off1 = 1; off1 < 32; off1 <<= 1) {
    const int32_t o = __shfl_up_sync(0xffffffffu, x, off1);
    if (lane >= off1) x += o;
  }
  if (lane == 31) warp_tot[warp] = x;
  __syncthreads();
  int32_t run = x - sum;
  for (int w = 0; w < warp; ++w) run += warp_tot[w];
  if (e0 <= E) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (e0 + i <= E) tile_start[e0 + i] = run;
      run += n[i];
    }
  }
  __syncthreads();
  return off;
}

struct Unit {
  int e, row0, nrows, nb;
};
// Fewer than 2^31 for segments that do not overlap.  Behind one that runs backwards
// others may: what is more of them then is left out.
__device__ __forceinline__ uint32_t units_of(int tiles, int RB) {
  const uint64_t n = (uint64_t)tiles * (uint32_t)RB;
  return n < 0x7fffffffu ? (uint32_t)n : 0x7fffffffu;
}
// Unit u: weight block u % RB of token tile u / RB.
__device__ __forceinline__ Unit unit_at(int E, const int32_t* offsets, const int32_t* tile_start,
                                        int RB, int tile, uint32_t u) {
  Unit r;
  const int tt = (int)(u / (uint32_t)RB);
  r.nb = (int)(u - (uint32_t)tt * (uint32_t)RB);
  int lo = 0, hi = E - 1;
  while (lo < hi) {  // largest e with tile_start[e] <= tt
    const int mid = (lo + hi + 1) >> 1;
    if (tile_start[mid] <= tt) lo = mid;
    else hi = mid - 1;
  }
  r.e = lo;
  r.row0 = offsets[lo] + (tt - tile_start[lo]) * tile;
  const int end = offsets[lo + 1];
  r.nrows = end - r.row0 < tile ? end - r.row0 : tile;
  return r;
}

template <int MODE, int BN>
__global__ void __launch_bounds__(kThreads, 1)
    k_gemm_fp8(const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
               const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA128,
               const __grid_constant__ Args a) {
  using C = Cfg<MODE, BN>;
  constexpr int STAGES = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* tail = smem + STAGES * C::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(tail);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + C::kBufs;
  uint64_t* hmax = tempty + C::kBufs;  // gate_up: the two halves of a lane quarter met
  uint64_t* never = hmax + 4;          // the diagnostics hook's (nothing arrives on it)
  uint64_t* drain = never + 1;         // abort path: the MMAs issued have completed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* amax_x = reinterpret_cast<float*>(tail + kBarBytes);
  uint8_t* out_x = tail + kBarBytes + C::kAmaxBytes;
  int32_t* tile_start = reinterpret_cast<int32_t*>(out_x + kEpiWarps * C::kOutBytes);
  int32_t* off_x = tile_start + kMaxSegments + 1;
  static_assert((2 * STAGES + 2 * C::kBufs + 6) * 8 + 8 <= kBarBytes, "barriers");
  __shared__ int32_t warp_tot[kThreads / 32];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KB = (a.K + BK - 1) / BK;
  const int NB = (a.N + 127) / 128;           // weight scale rows
  constexpr int kUnitCols = MODE == kGateUp ? 128 : BN;  // output columns per unit
  const int RB = (a.N + kUnitCols - 1) / kUnitCols;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kEpiWarps);
    }
    for (int q = 0; q < 4; ++q) mbar_init(&hmax[q], 2);
    mbar_init(never, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    sm100::mbar_init_fence();
  }
  if (warp == kEpiWarps && lane == 0) {
    prefetch_map(&tmB0);
    prefetch_map(&tmA);
    prefetch_map(&tmA128);
    if (MODE == kGateUp) prefetch_map(&tmB1);
  }
  if (warp == kEpiWarps + 1) sm100::tmem_alloc(tmem_slot, kTmemCols);
  if (!a.early) pdl_wait();

  tc_fence_before();
  const int32_t* off = build_tiles<kThreads, C::kCache>(a, BM, tile_start, off_x, warp_tot);
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t total_units = units_of(tile_start[a.E], RB);

  auto unit_of = [&](uint32_t u) { return unit_at(a.E, off, tile_start, RB, BM, u); };

  if (warp >= kEpiWarps) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtlRegs));
  if (warp == kEpiWarps) {
    // ------------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int64_t filled = 0;  // stages handed to TMA so far
      bool ok = true;
      if (a.probe)  // the diagnostics hook: a wait that runs out
        ok = mbar_wait(never, 0, abort_flag, kProbeLimitNs);
      bool dep_pending = a.early != 0;
      for (uint32_t u = blockIdx.x; u < total_units && ok; u += gridDim.x) {
        const Unit w = unit_of(u);
        // token rows: one box of 128, or 16-row boxes for a short tile
        const bool big = w.nrows > 2 * kSmallBox;
        const int box = big ? BM : kSmallBox;
        const int nbox = (w.nrows + box - 1) / box;
        // (a narrow last block needs only its 128-row box)
        const bool second = BN == 256 && (MODE == kGateUp || w.nb * BN + 128 < a.N);
        const uint32_t bytes = (second ? 256 : 128) * BK + nbox * box * BK;
        auto load_b = [&](int kb, int s) {
          mbar_arrive_expect_tx(&full[s], bytes);
          uint8_t* sB = smem + s * C::kStageBytes + C::kABytes;
#pragma unroll
          for (int i = 0; i < BN / 128; ++i)
            if (i == 0 || second) tma_load_3d(MODE == kGateUp && i == 1 ? &tmB1 : &tmB0, &full[s], sB + i * 128 * BK,
                        kb * BK, MODE == kGateUp ? w.nb * 128 : w.nb * BN + i * 128, w.e);
        };
        auto load_a = [&](int kb, int s) {
          uint8_t* sA = smem + s * C::kStageBytes;
          for (int i = 0; i < nbox; ++i)
            tma_load_2d(big ? &tmA128 : &tmA, &full[s], sA + i * box * BK, kb * BK,
                        w.row0 + i * box);
        };
        int kb = 0;
        if (dep_pending) {
          // the weights of up to STAGES blocks first, then the wait for the
          // kernel that writes the rows, then their rows
          for (; kb < STAGES && kb < KB; ++kb) {
            if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) { ok = false; break; }
            load_b(kb, stage);
            ++filled;
            if (++stage == STAGES) { stage = 0; phase ^= 1; }
          }
          pdl_wait();
          dep_pending = false;
          for (int j = 0; j < kb; ++j) load_a(j, j);
          if (!ok) break;
        }
        for (; kb < KB; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) { ok = false; break; }
          load_b(kb, stage);
          load_a(kb, stage);
          ++filled;
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
      }
      if (dep_pending) pdl_wait();
      pdl_trigger();
      if (!ok) {
        record_error(a.st, MOE_ERR_DEVICE_TIMEOUT, 310 + MODE);
        *abort_flag = 1;
        volatile int go_on = 0;  // the CTA's copies in flight land before it ends
        for (int64_t f = filled > STAGES ? filled - STAGES : 0; f < filled; ++f)
          mbar_wait(&full[f % STAGES], (uint32_t)(f / STAGES) & 1, &go_on, kDrainNs);
      }
    }
  } else if (warp == kEpiWarps + 1) {
    // ------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int stage = 0, buf = 0;
      uint32_t phase = 0, tphase = 0;
      bool ok = true;
      const uint64_t desc0 = sm100::smem_desc(smem_u32(smem), 1024, 2);
      for (uint32_t u = blockIdx.x; u < total_units && ok; u += gridDim.x) {
        // the last block of columns may be narrower
        const int cols = MODE == kPlain ? a.N - (int)(u % (uint32_t)RB) * BN : BN;
        const uint32_t idesc = idesc_e4m3(BM, cols < BN ? (cols + 15) / 16 * 16 : BN);
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&tempty[buf], tphase ^ 1, abort_flag) ||
              !mbar_wait(&full[stage], phase, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = desc0 + (uint64_t)(stage * (C::kStageBytes >> 4));
          const uint64_t db = da + (uint64_t)(C::kABytes >> 4);
          const uint32_t d = tmem_base + buf * BN;
#pragma unroll
          for (int k = 0; k < BK / UK; ++k)
            umma_e4m3(d, da + (uint64_t)(k * UK / 16), db + (uint64_t)(k * UK / 16), idesc,
                      k != 0);
          umma_commit(&empty[stage]);
          umma_commit(&tfull[buf]);
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
          if (++buf == C::kBufs) { buf = 0; tphase ^= 1; }
        }
      }
      if (!ok) {
        record_error(a.st, MOE_ERR_DEVICE_TIMEOUT, 320 + MODE);
        *abort_flag = 1;
        volatile int go_on = 0;
        umma_commit(drain);
        mbar_wait(drain, 0, &go_on, kDrainNs);
      }
    }
  }
  } else {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    // ------------------------------------------------------ epilogue
    // Warp: the token rows of TMEM lane quarter `quarter`, half of the columns:
    // 128 of y, or 64 of g and the same 64 of u.
    const int quarter = warp & 3, half = warp >> 2;
    constexpr int NC = BN / 2;  // sums per thread
    const int row = quarter * 32 + lane;
    const Act act = make_act(a.act_kind, a.beta, a.lbeta);
    const uint32_t t_lane = tmem_base + ((uint32_t)(quarter * 32) << 16);
    if (a.early) pdl_wait();
    int buf = 0;
    uint32_t tphase = 0, parity = 0;
    bool ok = true;
    for (uint32_t u = blockIdx.x; u < total_units && ok; u += gridDim.x) {
      const Unit w = unit_of(u);
      const int rows = w.nrows - quarter * 32;  // this warp's (<= 0: none)
      const int64_t row0 = (int64_t)w.row0 + quarter * 32;
      const bool live = lane < rows;
      const int cols = MODE == kPlain ? a.N - w.nb * BN - half * NC : NC;  // of this warp that exist
      // scales of a K block: the row's, times the one or two of the columns
      const float* sxp = a.xs + (live ? row0 + lane : (int64_t)w.row0) * KB;
      int sb = w.nb;
      if (MODE == kPlain && BN == 256) sb = 2 * w.nb + half < NB ? 2 * w.nb + half : NB - 1;
      const float* w0p = a.ws0 + ((int64_t)w.e * NB + sb) * KB;
      const float* w1p = MODE == kGateUp ? a.ws1 + ((int64_t)w.e * NB + sb) * KB : w0p;
      // those of four K blocks, and of the next four, in flight meanwhile
      float sx[4], s0[4], s1[4], nx[4], n0[4], n1[4];
      auto fetch = [&](int k0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int b = k0 + j < KB ? k0 + j : KB - 1;
          nx[j] = __ldg(sxp + b);
          n0[j] = __ldg(w0p + b);
          if (MODE == kGateUp) n1[j] = __ldg(w1p + b);
        }
      };
      fetch(0);
      // plain: kOutCols columns of y, and of the residual before them, pass through the
      // warp's shared memory, a row's 16-byte words permuted against bank conflicts.
      // The residual's first columns are copied while the K blocks run, the next ones
      // after each store, from L2 (4096 rows, 2048 to 7168: 143 us when each lane
      // loaded them there, 105 so, 88 without a residual; held in registers instead,
      // the sums spill: 133).
      constexpr int kW = C::kOutCols / 8;  // 16-byte words per row
      constexpr int kRowsAt = 32 / kW;     // rows per warp-wide access
      uint8_t* ob = out_x + warp * C::kOutBytes;
      auto word = [&](int r, int j) {
        return reinterpret_cast<uint4*>(ob + r * (16 * kW) + 16 * (j ^ ((r >> 1) & 3)));
      };
      auto res_async = [&](int c) {  // of columns c .. c + kOutCols - 1
        const int n = c + 8 * (lane % kW);
        const __nv_bfloat16* p = a.res + row0 * a.N + w.nb * BN + NC * half + n;
#pragma unroll
        for (int i = 0; i < kW; ++i) {
          const int r = i * kRowsAt + lane / kW;
          if (n < cols && r < rows)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             smem_u32(word(r, lane % kW))),
                         "l"(p + (int64_t)r * a.N)
                         : "memory");
        }
      };
      if (MODE == kPlain && a.res) {
        // the residual of the first columns to shared memory, of the others into L2
        res_async(0);
        const __nv_bfloat16* p = a.res + row0 * a.N + w.nb * BN + NC * half;
#pragma unroll
        for (int c = C::kOutCols; c < NC; c += C::kOutCols)
          if (live && c < cols)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p + (int64_t)lane * a.N + c));
      }
      uint64_t acc2[NC / 2];  // the sums of columns 2i and 2i + 1
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) acc2[i] = 0;
      for (int kb = 0; kb < KB; ++kb) {
        if ((kb & 3) == 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sx[j] = nx[j];
            s0[j] = n0[j];
            s1[j] = n1[j];
          }
          fetch(kb + 4);
        }
        auto pick = [&](const float* v) {
          return (kb & 2) ? ((kb & 1) ? v[3] : v[2]) : ((kb & 1) ? v[1] : v[0]);
        };
        const float fx = pick(sx);
        const uint64_t c0 = pair_of(fx * pick(s0));
        const uint64_t c1 = MODE == kGateUp ? pair_of(fx * pick(s1)) : c0;
        if (!__all_sync(0xffffffffu, mbar_wait(&tfull[buf], tphase, abort_flag))) {
          if (lane == 0) record_error(a.st, MOE_ERR_DEVICE_TIMEOUT, 330 + MODE);
          *abort_flag = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        if (rows > 0) {
#pragma unroll
          for (int c = 0; c < NC; c += 32) {
            if (MODE == kPlain && c >= cols) break;
            // gate_up: the thread's first 64 sums are g (w1), the next 64 u (w3)
            const bool second = MODE == kGateUp && c >= 64;
            uint32_t r[32];
            sm100::tmem_ld32(t_lane + buf * BN + (MODE == kGateUp ? (second ? 128 : 0) + 64 * half + (c & 63)
                                                   : half * NC + c), r);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              fma2(acc2[c / 2 + i], r[2 * i], r[2 * i + 1], second ? c1 : c0);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[buf]);
        if (++buf == C::kBufs) { buf = 0; tphase ^= 1; }
      }
      if (!ok) break;
      if constexpr (MODE == kPlain) {
        // Through shared memory a store covers whole sectors of few rows (each
        // lane's own row, 16 bytes at a time, took 6,000 cycles a unit).
        const int n_first = w.nb * BN + NC * half;
#pragma unroll
        for (int c = 0; c < NC; c += C::kOutCols) {
          const int n = n_first + c + 8 * (lane % kW);  // of this lane's accesses to y
          const bool in = n < a.N;                      // N is a multiple of 8
          if (a.res) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
          }
#pragma unroll
          for (int j = 0; j < kW; ++j) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[2 * i] = lo_of(acc2[c / 2 + 4 * j + i]);
              v[2 * i + 1] = hi_of(acc2[c / 2 + 4 * j + i]);
            }
            if (a.res) {
              const uint4 t = *word(lane, j);
              const uint32_t tw[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                v[2 * i] += __uint_as_float(tw[i] << 16);
                v[2 * i + 1] += __uint_as_float(tw[i] & 0xffff0000u);
              }
            }
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
              o[i] = *reinterpret_cast<const uint32_t*>(&p);
            }
            *word(lane, j) = make_uint4(o[0], o[1], o[2], o[3]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < kW; ++i) {
            const int r = i * kRowsAt + lane / kW;
            if (in && r < rows)
              *reinterpret_cast<uint4*>(a.y + (row0 + r) * a.N + n) = *word(r, lane % kW);
          }
          __syncwarp();
          if (a.res && c + C::kOutCols < NC) res_async(c + C::kOutCols);
        }
      } else {
        // h of 64 columns in acc2[0..31]; the block's largest |h| needs the
        // other half's too: exchanged through shared memory (the buffer
        // alternates, so a fast warp's next unit cannot overwrite it)
        uint32_t m = 0;  // magnitudes as integers, NaN above infinity
        with_act(act, [&](auto h) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            acc2[i] = h(acc2[i], acc2[32 + i]);
            m = max(m, max((uint32_t)acc2[i] & 0x7fffffffu,
                           (uint32_t)(acc2[i] >> 32) & 0x7fffffffu));
          }
        });
        uint32_t* xch = reinterpret_cast<uint32_t*>(amax_x) + parity * 2 * BM;
        xch[half * BM + row] = m;
        __syncwarp();
        if (lane == 0) mbar_arrive(&hmax[quarter]);
        if (!__all_sync(0xffffffffu, mbar_wait(&hmax[quarter], parity, abort_flag))) {
          if (lane == 0) record_error(a.st, MOE_ERR_DEVICE_TIMEOUT, 340);
          *abort_flag = 1;
          break;
        }
        m = max(m, xch[(half ^ 1) * BM + row]);
        parity ^= 1;
        float inv;
        const float s = fp8::block_scale(__uint_as_float(m), a.pow2, inv);
        // the warp's 32 x 64 bytes through shared memory, as in the plain form
        static_assert(C::kOutBytes == 32 * 64 && kW == 4, "32 rows of 64 bytes");
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t* v = acc2 + 8 * j + 2 * i;
            o[i] = fp8::pack4(lo_of(v[0]) * inv, hi_of(v[0]) * inv, lo_of(v[1]) * inv,
                              hi_of(v[1]) * inv);
          }
          *word(lane, j) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        __syncwarp();
        const int f = w.nb * 128 + 64 * half + 16 * (lane & 3);  // of this lane's stores
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * i + (lane >> 2);
          if (r < rows && f < a.N)  // N is a multiple of 16
            *reinterpret_cast<uint4*>(a.hq + (row0 + r) * a.N + f) = *word(r, lane & 3);
        }
        if (live && half == 0) a.hs[(row0 + lane) * NB + w.nb] = s;
        __syncwarp();
      }
    }
    // a unit that was given up may have left copies of the residual in flight
    if (MODE == kPlain) asm volatile("cp.async.wait_all;" ::: "memory");
  }  // roles
  tc_fence_before();
  __syncthreads();
  if (warp == kEpiWarps + 1) {
    __syncwarp();
    tc_fence_after();
    sm100::tmem_dealloc(tmem_base, kTmemCols);
  }
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void st_cluster_f32(const void* local, uint32_t rank, float v) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(r), "f"(v) : "memory");
}

// --------------------------------------------------------- decode variant
// A few rows per segment: the product is a stream of weights.  Here the weight
// rows are the MMA's M side (128 of them; gate_up 128 of w1 and the same 128 of
// w3, each with its accumulator) and up to 32 token rows its N side, rounded up
// to 16, so an MMA costs little more than reading the weights from shared
// memory, and a K block leaves 16 or 32 sums per thread to add instead of 128.
// (With the token rows on the M side a stream of 8-bit weights ran at 4.9-5.4
// TB/s, paced by the MMAs on 128 mostly empty rows and by the two epilogue
// warps that hold the 32 rows; the loads alone reach 7.)
// The row scales then differ by column: each epilogue warp forms its 32 products
// sx * sw, one per lane, and passes them round through shared memory.
// A stage holds KSUB K blocks, so that 256 contiguous bytes of a weight row are
// asked for together.
// SPLIT: a cluster of 2, 4 or 8 CTAs shares a unit, each takes a part of K,
// and the parts are added in rank order through distributed shared memory:
// for a Linear of few rows, whose units alone would leave most SMs idle.  Every
// cluster has one unit at most.
constexpr int kNt = 32;         // token rows per tile
constexpr int kDecThreads = 192;  // warps 0-3 epilogue, 4 TMA, 5 MMA

template <int MODE, int STAGES, int KSUB>
struct DecCfg {
  static constexpr int kTiles = MODE == kGateUp ? 2 : 1;  // weight tiles (accumulators) per unit
  static constexpr int kWBytes = kTiles * 128 * BK;
  static constexpr int kTBytes = kNt * BK;
  static constexpr int kSubBytes = kWBytes + kTBytes;
  static constexpr int kStageBytes = KSUB * kSubBytes;
  static constexpr int kBufs = 4;
  static constexpr int kBufCols = kTiles * kNt;
  static constexpr int kTmem = kBufs * kBufCols;
  static constexpr int kScaleBytes = 4 * 2 * kTiles * kNt * 4;  // warp x parity x tile x row
  static constexpr int kStartBytes = (kMaxSegments + 1) * 4;
  static constexpr int kMaxBytes = 2 * 4 * kNt * 4;  // gate_up: unit parity x warp x row
  static constexpr int kPartBytes = MODE == kPlain ? 128 * kNt * 4 : 0;  // SPLIT's partial sums
  static constexpr int kCache = 640;  // offsets held in shared memory
  static constexpr size_t kSmem = (size_t)STAGES * kStageBytes + 1024 + kBarBytes + kScaleBytes +
                                  kMaxBytes + kPartBytes + kStartBytes + 4 * kCache;
  static_assert(kTmem <= 512 && (kTmem & (kTmem - 1)) == 0, "TMEM columns");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

template <int MODE, int STAGES, int KSUB, bool SPLIT>
__global__ void __launch_bounds__(kDecThreads, 1)
    k_gemm_fp8_dec(const __grid_constant__ CUtensorMap tmW0,
                   const __grid_constant__ CUtensorMap tmW1,
                   const __grid_constant__ CUtensorMap tmT, const __grid_constant__ Args a) {
  using C = DecCfg<MODE, STAGES, KSUB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* tail = smem + STAGES * C::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(tail);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + C::kBufs;
  uint64_t* hmax = tempty + C::kBufs;  // gate_up: the four warps' maxima are there
  uint64_t* never = hmax + 1;
  uint64_t* drain = never + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((2 * STAGES + 2 * C::kBufs + 3) * 8 + 8 <= kBarBytes, "barriers");
  float* scale_x = reinterpret_cast<float*>(tail + kBarBytes);
  uint32_t* max_x = reinterpret_cast<uint32_t*>(tail + kBarBytes + C::kScaleBytes);
  float* part = reinterpret_cast<float*>(tail + kBarBytes + C::kScaleBytes + C::kMaxBytes);
  int32_t* tile_start = reinterpret_cast<int32_t*>(tail + kBarBytes + C::kScaleBytes +
                                                   C::kMaxBytes + C::kPartBytes);
  int32_t* off_x = tile_start + kMaxSegments + 1;
  __shared__ int32_t warp_tot[kDecThreads / 32];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KB = (a.K + BK - 1) / BK;
  const int NB = (a.N + 127) / 128;  // weight blocks = scale rows
  const uint32_t csize = SPLIT ? cluster_size() : 1, crank = SPLIT ? cluster_rank() : 0;
  const uint32_t unit0 = blockIdx.x / csize, unit_step = gridDim.x / csize;
  const int kb0 = (int)((int64_t)crank * KB / csize);
  const int kb1 = (int)((int64_t)(crank + 1) * KB / csize);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 4);
    }
    mbar_init(hmax, 4);
    mbar_init(never, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    sm100::mbar_init_fence();
  }
  if (warp == 4 && lane == 0) {
    prefetch_map(&tmW0);
    prefetch_map(&tmT);
    if (MODE == kGateUp) prefetch_map(&tmW1);
  }
  if (warp == 5) sm100::tmem_alloc(tmem_slot, C::kTmem);
  if (!a.early) pdl_wait();
  tc_fence_before();
  const int32_t* off = build_tiles<kDecThreads, C::kCache>(a, kNt, tile_start, off_x, warp_tot);
  tc_fence_after();
  if (SPLIT) cluster_sync();  // the other CTAs run: their shared memory may be written
  const uint32_t tmem_base = *tmem_slot;
  uint32_t total_units = units_of(tile_start[a.E], NB);
  if (SPLIT && total_units > unit_step) total_units = unit_step;  // (overlapping segments)
  auto unit_of = [&](uint32_t u) { return unit_at(a.E, off, tile_start, NB, kNt, u); };

  if (warp == 4) {
    // ------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t wpol = sm100::l2_evict_first_policy();
      int stage = 0;
      uint32_t phase = 0;
      int64_t filled = 0;  // stages handed to TMA so far
      bool ok = true;
      if (a.probe) ok = mbar_wait(never, 0, abort_flag, kProbeLimitNs);
      bool dep_pending = a.early != 0;
      for (uint32_t u = unit0; u < total_units && ok; u += unit_step) {
        const Unit w = unit_of(u);
        const int nbox = (w.nrows + kSmallBox - 1) / kSmallBox;
        const uint32_t bytes = C::kWBytes + nbox * kSmallBox * BK;  // of a K block
        auto load_w = [&](int kb, int s) {
          mbar_arrive_expect_tx(&full[s], bytes * (kb1 - kb < KSUB ? kb1 - kb : KSUB));
#pragma unroll
          for (int i = 0; i < C::kTiles; ++i)
#pragma unroll
            for (int j = 0; j < KSUB; ++j)
              if (kb + j < kb1)
                sm100::tma_load_3d_hint(i == 0 ? &tmW0 : &tmW1, &full[s],
                                        smem + s * C::kStageBytes + j * C::kSubBytes +
                                            i * 128 * BK,
                                        (kb + j) * BK, w.nb * 128, w.e, wpol);
        };
        auto load_t = [&](int kb, int s) {
#pragma unroll
          for (int j = 0; j < KSUB; ++j)
            if (kb + j < kb1)
              for (int i = 0; i < nbox; ++i)
                tma_load_2d(&tmT, &full[s],
                            smem + s * C::kStageBytes + j * C::kSubBytes + C::kWBytes +
                                i * kSmallBox * BK,
                            (kb + j) * BK, w.row0 + i * kSmallBox);
        };
        int kb = kb0;
        if (dep_pending) {
          // the weights of up to STAGES stages first, then the wait for the
          // kernel that writes the rows, then their rows
          for (int j = 0; j < STAGES && kb < kb1; ++j, kb += KSUB) {
            load_w(kb, stage);
            ++filled;
            if (++stage == STAGES) { stage = 0; phase ^= 1; }
          }
          pdl_wait();
          dep_pending = false;
          for (int j = 0; kb0 + j * KSUB < kb; ++j) load_t(kb0 + j * KSUB, j);
        }
        for (; kb < kb1; kb += KSUB) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) { ok = false; break; }
          load_w(kb, stage);
          load_t(kb, stage);
          ++filled;
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
      }
      if (dep_pending) pdl_wait();
      pdl_trigger();
      if (!ok) {
        record_error(a.st, MOE_ERR_DEVICE_TIMEOUT, 350 + MODE);
        *abort_flag = 1;
        volatile int go_on = 0;  // the CTA's copies in flight land before it ends
        for (int64_t f = filled > STAGES ? filled - STAGES : 0; f < filled; ++f)
          mbar_wait(&full[f % STAGES], (uint32_t)(f / STAGES) & 1, &go_on, kDrainNs);
      }
    }
  } else if (warp == 5) {
    // ------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int stage = 0, buf = 0;
      uint32_t phase = 0, tphase = 0;
      bool ok = true;
      const uint64_t desc0 = sm100::smem_desc(smem_u32(smem), 1024, 2);
      for (uint32_t u = unit0; u < total_units && ok; u += unit_step) {
        const Unit w = unit_of(u);
        const uint32_t idesc = idesc_e4m3(128, (w.nrows + 15) / 16 * 16);
        for (int kb = kb0; kb < kb1 && ok; kb += KSUB) {
          if (!mbar_wait(&full[stage], phase, abort_flag)) { ok = false; break; }
#pragma unroll
          for (int j = 0; j < KSUB; ++j) {
            if (kb + j >= kb1) break;
            if (!mbar_wait(&tempty[buf], tphase ^ 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint64_t dw =
                desc0 + (uint64_t)(stage * (C::kStageBytes >> 4) + j * (C::kSubBytes >> 4));
            const uint64_t dt = dw + (uint64_t)(C::kWBytes >> 4);
            const uint32_t d = tmem_base + buf * C::kBufCols;
#pragma unroll
            for (int k = 0; k < BK / UK; ++k)
#pragma unroll
              for (int i = 0; i < C::kTiles; ++i)
                umma_e4m3(d + i * kNt, dw + (uint64_t)((i * 128 * BK + k * UK) >> 4),
                          dt + (uint64_t)(k * UK >> 4), idesc, k != 0);
            umma_commit(&tfull[buf]);
            if (++buf == C::kBufs) { buf = 0; tphase ^= 1; }
          }
          if (ok) umma_commit(&empty[stage]);
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok) {
        record_error(a.st, MOE_ERR_DEVICE_TIMEOUT, 360 + MODE);
        *abort_flag = 1;
        volatile int go_on = 0;
        umma_commit(drain);
        mbar_wait(drain, 0, &go_on, kDrainNs);
      }
    }
  } else {
    // ------------------------------------------------------ epilogue
    const Act act = make_act(a.act_kind, a.beta, a.lbeta);
    const uint32_t lanes0 = tmem_base + ((uint32_t)(warp * 32) << 16);
    float* sc = scale_x + warp * 2 * C::kTiles * kNt;
    if (a.early) pdl_wait();
    int buf = 0;
    uint32_t tphase = 0, parity = 0;
    bool ok = true;
    for (uint32_t u = unit0; u < total_units && ok; u += unit_step) {
      const Unit w = unit_of(u);
      // lane t fetches the scales of token row t, kAhead blocks before their use
      const float* sxp =
          a.xs + ((int64_t)w.row0 + (lane < w.nrows ? lane : w.nrows - 1)) * KB;
      const float* w0p = a.ws0 + ((int64_t)w.e * NB + w.nb) * KB;
      const float* w1p = MODE == kGateUp ? a.ws1 + ((int64_t)w.e * NB + w.nb) * KB : nullptr;
      uint64_t acc2[C::kTiles][kNt / 2];  // the sums of token rows 2i and 2i + 1
#pragma unroll
      for (int t = 0; t < C::kTiles; ++t)
#pragma unroll
        for (int i = 0; i < kNt / 2; ++i) acc2[t][i] = 0;
      constexpr int kAhead = 2;
      float sxr[kAhead], w0r[kAhead], w1r[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int b = kb0 + j < KB ? kb0 + j : KB - 1;
        sxr[j] = __ldg(sxp + b);
        w0r[j] = __ldg(w0p + b);
        w1r[j] = MODE == kGateUp ? __ldg(w1p + b) : 0.0f;
      }
      for (int kb = kb0; kb < kb1; ++kb) {
        float* scp = sc + (kb & 1) * C::kTiles * kNt;
        scp[lane] = sxr[0] * w0r[0];
        if (MODE == kGateUp) scp[kNt + lane] = sxr[0] * w1r[0];
#pragma unroll
        for (int j = 0; j + 1 < kAhead; ++j) {
          sxr[j] = sxr[j + 1];
          w0r[j] = w0r[j + 1];
          w1r[j] = w1r[j + 1];
        }
        const int b = kb + kAhead < KB ? kb + kAhead : KB - 1;
        sxr[kAhead - 1] = __ldg(sxp + b);
        w0r[kAhead - 1] = __ldg(w0p + b);
        if (MODE == kGateUp) w1r[kAhead - 1] = __ldg(w1p + b);
        if (!__all_sync(0xffffffffu, mbar_wait(&tfull[buf], tphase, abort_flag))) {
          if (lane == 0) record_error(a.st, MOE_ERR_DEVICE_TIMEOUT, 370 + MODE);
          *abort_flag = 1;
          ok = false;
          break;
        }
        __syncwarp();  // the products sx * sw are in shared memory
        tc_fence_after();
        const uint32_t t0 = lanes0 + buf * C::kBufCols;
        if (w.nrows <= 8) {  // the usual decode step: a quarter of the columns
#pragma unroll
          for (int t = 0; t < C::kTiles; ++t) {
            uint32_t r[8];
            sm100::tmem_ld8(t0 + t * kNt, r);
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
              const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(scp + t * kNt + i);
              fma2(acc2[t][i / 2], r[i], r[i + 1], f.x);
              fma2(acc2[t][i / 2 + 1], r[i + 2], r[i + 3], f.y);
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < kNt; c += 16) {
            if (c < w.nrows) {
#pragma unroll
              for (int t = 0; t < C::kTiles; ++t) {
                uint32_t r[16];
                sm100::tmem_ld16(t0 + t * kNt + c, r);
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                  const ulonglong2 f =
                      *reinterpret_cast<const ulonglong2*>(scp + t * kNt + c + i);
                  fma2(acc2[t][(c + i) / 2], r[i], r[i + 1], f.x);
                  fma2(acc2[t][(c + i) / 2 + 1], r[i + 2], r[i + 3], f.y);
                }
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[buf]);
        if (++buf == C::kBufs) { buf = 0; tphase ^= 1; }
      }
      if (!ok) break;
      const int m = 32 * warp + lane;  // this thread's row of the weight block
      const int n = w.nb * 128 + m;
      float acc[C::kTiles][kNt];
#pragma unroll
      for (int t = 0; t < C::kTiles; ++t)
#pragma unroll
        for (int i = 0; i < kNt / 2; ++i) {
          acc[t][2 * i] = lo_of(acc2[t][i]);
          acc[t][2 * i + 1] = hi_of(acc2[t][i]);
        }
      if (MODE == kPlain && SPLIT) {
        // weight row m is finished by CTA m / rpc of the cluster
        const int rpc = 128 / csize;
#pragma unroll
        for (int i = 0; i < kNt; ++i) {
          if (i >= w.nrows) break;
          st_cluster_f32(part + ((int)crank * kNt + i) * rpc + m % rpc, m / rpc, acc[0][i]);
        }
      } else if (MODE == kPlain) {
        if (n < a.N) {
          const int64_t at = (int64_t)w.row0 * a.N + n;
#pragma unroll
          for (int i = 0; i < kNt; ++i) {
            if (i >= w.nrows) break;
            float v = acc[0][i];
            if (a.res) v += __bfloat162float(a.res[at + (int64_t)i * a.N]);
            a.y[at + (int64_t)i * a.N] = __float2bfloat16_rn(v);
          }
        }
      } else {
        // h of one d_ff row and all token rows; the largest |h| of a token row
        // over the 128 d_ff rows: over the warp, then over the four warps
        // through shared memory (two buffers, so a fast warp's next unit cannot
        // overwrite what a slow one still reads)
        uint32_t mine = 0;  // lane i: the warp's largest magnitude of token row i
        uint32_t* mx = max_x + parity * 4 * kNt;
        with_act(act, [&](auto h) {
#pragma unroll
          for (int i0 = 0; i0 < kNt; i0 += 8) {  // eight at a time: independent chains
            if (i0 >= w.nrows) break;
#pragma unroll
            for (int i = i0; i < i0 + 8; ++i) {
              acc[0][i] = h(acc[0][i], acc[C::kTiles - 1][i]);
              const uint32_t v =
                  __reduce_max_sync(0xffffffffu, __float_as_uint(acc[0][i]) & 0x7fffffffu);
              if (lane == i) mine = v;
            }
          }
        });
        mx[warp * kNt + lane] = mine;
        __syncwarp();
        if (lane == 0) mbar_arrive(hmax);
        if (!__all_sync(0xffffffffu, mbar_wait(hmax, parity, abort_flag))) {
          if (lane == 0) record_error(a.st, MOE_ERR_DEVICE_TIMEOUT, 380);
          *abort_flag = 1;
          break;
        }
        mine = max(max(mx[lane], mx[kNt + lane]), max(mx[2 * kNt + lane], mx[3 * kNt + lane]));
        parity ^= 1;
        float inv;
        const float s = fp8::block_scale(__uint_as_float(mine), a.pow2, inv);
        if (warp == 0 && lane < w.nrows) a.hs[((int64_t)w.row0 + lane) * NB + w.nb] = s;
        uint8_t* dst = a.hq + (int64_t)w.row0 * a.N + n;
#pragma unroll
        for (int i = 0; i < kNt; i += 2) {
          if (i >= w.nrows) break;
          const float q0 = acc[0][i] * __shfl_sync(0xffffffffu, inv, i);
          const float q1 = acc[0][i + 1] * __shfl_sync(0xffffffffu, inv, i + 1);
          const uint32_t q = fp8::pack4(q0, q1, 0.0f, 0.0f);
          if (n < a.N) {
            dst[(int64_t)i * a.N] = (uint8_t)q;
            if (i + 1 < w.nrows) dst[(int64_t)(i + 1) * a.N] = (uint8_t)(q >> 8);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (SPLIT) {
    cluster_sync();  // every CTA's part of this CTA's rows has arrived
    if (unit0 < total_units && !*abort_flag) {
      const Unit w = unit_of(unit0);
      const int rpc = 128 / csize;
      for (int i = threadIdx.x; i < rpc * w.nrows; i += kDecThreads) {
        const int t = i / rpc, m = i - t * rpc;
        const int n = w.nb * 128 + (int)crank * rpc + m;
        float v = part[t * rpc + m];
        for (int r = 1; r < (int)csize; ++r) v += part[(r * kNt + t) * rpc + m];
        if (n < a.N) {
          const int64_t at = ((int64_t)w.row0 + t) * a.N + n;
          if (a.res) v += __bfloat162float(a.res[at]);
          a.y[at] = __float2bfloat16_rn(v);
        }
      }
    }
  }
  if (warp == 5) {
    __syncwarp();
    tc_fence_after();
    sm100::tmem_dealloc(tmem_base, C::kTmem);
  }
}

// ------------------------------------------------------------ few rows
// A dense product of at most kFewRows rows: a matrix-vector product on the CUDA
// cores.  One warp per weight row, 16 bytes a lane and step, so a step covers
// 512 contiguous bytes, four K blocks, and eight lanes share a block: each lane
// sums its 16 products in fp32, times sx * sw, over the steps, and the warp adds
// its lanes at the end.  The rows of x are in shared memory as fp32.  There is
// nothing to stage or hand over, so it ends sooner than the decode
// kernel, whose cluster and barriers cost more than the work: one row, K = 7168,
// N = 2048: 5.1 us, and 8.5 there; its 14.7 MB alone take 2.2.
constexpr int kFewRows = 4;
constexpr int kFewWarps = 16;
constexpr int kFewMaxSmem = 128 * 1024;

template <int M>
__global__ void __launch_bounds__(32 * kFewWarps, 1)
    k_linear_few(const uint8_t* __restrict__ w, const uint8_t* __restrict__ xq, const Args a) {
  // x as it is read: float4 word i (0 .. 3) of lane l in step t of row m is
  // x4[((m * steps + t) * 4 + i) * 32 + l], free of bank conflicts
  extern __shared__ float4 x4[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KB = (a.K + BK - 1) / BK, steps = (a.K + 511) / 512, words16 = a.K / 16;
  pdl_wait();
  pdl_trigger();
  if (a.reset && blockIdx.x == 0 && threadIdx.x == 0) *a.st = DeviceStatus{0, 0};
  auto two = [](uint32_t e4m3x2) {  // the lower two e4m3 as floats (exact)
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)e4m3x2));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
  };
  for (int i = threadIdx.x; i < M * words16; i += 32 * kFewWarps) {
    const int m = i / words16, c = i - m * words16;
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(xq + (int64_t)m * a.K) + c);
    const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = two(words[j]), q = two(words[j] >> 16);
      x4[((m * steps + (c >> 5)) * 4 + j) * 32 + (c & 31)] = make_float4(p.x, p.y, q.x, q.y);
    }
  }
  __syncthreads();
  for (int n = blockIdx.x * kFewWarps + warp; n < a.N; n += gridDim.x * kFewWarps) {
    const uint8_t* row = w + (int64_t)n * a.K;
    const float* sw = a.ws0 + (int64_t)(n >> 7) * KB;
    float acc[M];
#pragma unroll
    for (int m = 0; m < M; ++m) acc[m] = 0.0f;
    // Loads in flight per lane.  More of them wait longer for the last and hold more
    // registers, fewer leave memory idle: over K of 512 to 14336 and N of 1024 to 7168,
    // weights from HBM, the mean time with 4, 5, 6, 7 and 8 was 0.95, 0.95, 0.96, 1 and
    // 1.00 at one row, 0.95, 0.96, 0.98, 1 and 1.03 at two, 0.98, 0.99, 1.00, 1 and 1.03
    // at four (1 row, N = 2048: K = 2048 2.9, 2.9, 3.0, 3.1, 3.1 us, K = 4096 4.2, 4.5,
    // 4.7, 5.0, 4.4, K = 7168 6.3, 6.0, 6.4, 6.2, 6.3).  With 4, one row needs 64
    // registers and two CTAs fit on an SM: a launch whose CTAs are placed while the one
    // before it still holds its SMs then doubles up on the others, and calls in a loop took
    // 5.2 or 7.9 us from one run to the next (K = 7168, N = 2048; 5.1 with 5).
    constexpr int kBatch = 5;
    for (int k0 = 16 * lane; k0 - 16 * lane < a.K; k0 += 512 * kBatch) {
      uint4 v[kBatch];
      float f[kBatch][M];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int k = k0 + 512 * j;
        v[j] = make_uint4(0, 0, 0, 0);
        if (k < a.K) v[j] = __ldg(reinterpret_cast<const uint4*>(row + k));
        const int b = k < a.K ? k >> 7 : KB - 1;
        const float s = __ldg(sw + b);
#pragma unroll
        for (int m = 0; m < M; ++m) f[j][m] = s * __ldg(a.xs + (int64_t)m * KB + b);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int k = k0 + 512 * j;
        if (k >= a.K) break;
        float p[M];
#pragma unroll
        for (int m = 0; m < M; ++m) p[m] = 0.0f;
        const uint32_t words[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 lo = two(words[i]), hi = two(words[i] >> 16);
#pragma unroll
          for (int m = 0; m < M; ++m) {
            const float4 x = x4[((m * steps + (k >> 9)) * 4 + i) * 32 + lane];
            p[m] = fmaf(lo.x, x.x, p[m]);
            p[m] = fmaf(lo.y, x.y, p[m]);
            p[m] = fmaf(hi.x, x.z, p[m]);
            p[m] = fmaf(hi.y, x.w, p[m]);
          }
        }
#pragma unroll
        for (int m = 0; m < M; ++m) acc[m] = fmaf(p[m], f[j][m], acc[m]);
      }
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[m] += __shfl_xor_sync(0xffffffffu, acc[m], o);
      if (lane == 0) {
        const int64_t at = (int64_t)m * a.N + n;
        float y = acc[m];
        if (a.res) y += __bfloat162float(a.res[at]);
        a.y[at] = __float2bfloat16_rn(y);
      }
    }
  }
}

// ------------------------------------------------------------ tensor maps
typedef CUresult (*EncodeTiledFn8)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn8 encode_8() {
  static const EncodeTiledFn8 fn = [] {  // looked up once (thread-safe static)
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn8>(p);
    return static_cast<EncodeTiledFn8>(nullptr);
  }();
  return fn;
}

// [batch, rows, cols] bytes, box 128 columns x box_rows x 1, 128-byte swizzle;
// what a box reaches beyond the tensor reads as zeros (e4m3 0), which the
// products then ignore: K and N need not be multiples of 128.
bool map_weights(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t batch) {
  EncodeTiledFn8 fn = encode_8();
  if (!fn) return false;
  cuuint64_t dims[3] = {cols, rows, batch};
  cuuint64_t strides[2] = {cols, cols * rows};
  cuuint32_t box[3] = {(cuuint32_t)BK, 128, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool map_rows(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows) {
  EncodeTiledFn8 fn = encode_8();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols};
  cuuint32_t box[2] = {(cuuint32_t)BK, box_rows};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Token tiles that S rows in E segments can need at most.
int64_t max_tiles(const Args& a, int tile) {
  if (!a.offsets) return (a.S + tile - 1) / tile;
  return a.S / tile + (a.S < a.E ? a.S : a.E);
}

template <int MODE, int BN>
cudaError_t launch(const CUtensorMap& b0, const CUtensorMap& b1, const CUtensorMap& a16,
                   const CUtensorMap& a128, const Args& args, cudaStream_t s) {
  using C = Cfg<MODE, BN>;
  constexpr auto kernel = k_gemm_fp8<MODE, BN>;
  static std::once_flag once[kMaxDevices];
  static cudaError_t set_up[kMaxDevices];
  const cudaError_t e = once_per_device(once, set_up, [&](int) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)C::kSmem);
  });
  if (e != cudaSuccess) return e;
  const int cols = MODE == kGateUp ? 128 : BN;
  const int64_t units = max_tiles(args, BM) * ((args.N + cols - 1) / cols);
  const int sms = dev_info()->sm_count;
  return launch_pdl(kernel, dim3((unsigned)(units < sms ? units : sms)), dim3(kThreads), C::kSmem,
                    s, b0, b1, a16, a128, args);
}

template <int MODE, int STAGES, int KSUB, bool SPLIT>
cudaError_t launch_dec(const CUtensorMap& w0, const CUtensorMap& w1, const CUtensorMap& t,
                       const Args& args, unsigned grid, unsigned cluster, cudaStream_t s) {
  using C = DecCfg<MODE, STAGES, KSUB>;
  constexpr auto kernel = k_gemm_fp8_dec<MODE, STAGES, KSUB, SPLIT>;
  static std::once_flag once[kMaxDevices];
  static cudaError_t set_up[kMaxDevices];
  const cudaError_t e = once_per_device(once, set_up, [&](int) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)C::kSmem);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kDecThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return counted(cudaLaunchKernelEx(&cfg, kernel, w0, w1, t, args));
}

// How many clusters of the split decode kernel, of 2, 4 and 8 CTAs, can run at once.
int max_clusters(unsigned c) {
  constexpr int kLog = 4;
  static std::once_flag once[kMaxDevices];
  static cudaError_t set_up[kMaxDevices];
  static int most[kMaxDevices][kLog];
  using C = DecCfg<kPlain, 5, 2>;
  constexpr auto kernel = k_gemm_fp8_dec<kPlain, 5, 2, true>;
  const cudaError_t e = once_per_device(once, set_up, [&](int dev) {
    cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)C::kSmem);
    for (int i = 1; i < kLog && r == cudaSuccess; ++i) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 1u << i;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3((unsigned)(dev_info()->sm_count >> i) << i);
      cfg.blockDim = dim3(kDecThreads);
      cfg.dynamicSmemBytes = C::kSmem;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      r = cudaOccupancyMaxActiveClusters(&most[dev][i], kernel, &cfg);
    }
    return r;
  });
  int dev = 0;
  if (e != cudaSuccess || cudaGetDevice(&dev) != cudaSuccess) return 0;
  return most[dev][c == 8 ? 3 : c == 4 ? 2 : 1];
}

size_t few_smem(int64_t M, int K) { return (size_t)M * ((K + 511) / 512) * 512 * sizeof(float); }

// The variant of a product, by an estimate of its time from the sizes alone, with
// segments taken as equally long (their lengths are on the device; with 75 % of the rows
// on a tenth of 384 experts the MLP of 8192 and 32768 rows takes 16 and 23 % more than
// with equal segments): the waves of units over the SMs, times what a
// unit costs, its K blocks and its end.  In microseconds, measured on a B200:
//   decode          0.33 a K block with at most 16 rows a tile, 0.36 with more, 1.0
//                   at the end; gate_up 0.70, 0.74 and 1.0;
//   decode, split   at the end 2.4 and 0.08 a row (the parts' exchange);
//   BN = 128        0.45 and 1.2;
//   BN = 256        0.72 and 2.0, gate_up 0.74 and 2.5;
//   few rows        0.12 + 0.14 a row for 512 columns of K.
// Some borders, measured on both sides (us): 32 segments, K = 2048, N = 7168:
// decode against 256 rows 78 and 92 with 8 rows each, 86 and 96 with 32, 147
// and 95 with 40; 16 segments, K = N = 512, 128 rows each: decode, 128 and 256
// rows 7.6, 6.3 and 8.4.  Few rows against decode, K = 7168: one row 5.1 and 8.5
// with N = 2048, 33 and 24 with N = 18944; two rows 7.2 and 8.5, three 9.5 and 8.5
// with N = 2048.  One segment, K = 7168, N = 2048: decode split 4 ways, not
// split, 128 and 256 rows 9.5, 21, 23 and 36 with 16 rows; decode, 128 and 256 rows
// 41, 26 and 39 with 384; 135, 51 and 40 with 2048.  K = N = 512, 64 rows: split
// 6.4, not split 4.5, 128 rows 4.9.
struct Choice {
  int variant;        // 0 decode, 1 BN = 128, 2 BN = 256, 3 few rows
  unsigned clusters;  // decode: CTAs that share a unit's K
};

Choice choose(const Args& a, bool gate_up) {
  const int sms = dev_info()->sm_count;
  const int64_t KB = (a.K + BK - 1) / BK, NB = (a.N + 127) / 128;
  const int64_t segs = !a.offsets ? 1 : a.S < a.E ? a.S : a.E;
  const int64_t rows = (a.S + segs - 1) / segs;
  auto tiles = [&](int tile) { return segs * ((rows + tile - 1) / tile); };
  auto cost = [&](int64_t units, int64_t kbs, double per_kb, double end) {
    return (double)((units + sms - 1) / sms) * ((double)kbs * per_kb + end);
  };
  Choice c{0, 1};
  const double dec = gate_up ? (rows <= 16 ? 0.70 : 0.74) : (rows <= 16 ? 0.33 : 0.36);
  double best = cost(tiles(kNt) * NB, KB, dec, 1.0);
  if (!gate_up) {
    // every cluster has one unit at most, all can run at once, and each CTA has
    // a K block
    const int64_t most = max_tiles(a, kNt) * NB;
    for (unsigned k = 2; k <= 8 && most * k <= sms && KB >= k && most <= max_clusters(k); k *= 2) {
      const double t =
          cost(most * k, (KB + k - 1) / k, dec, 2.4 + 0.08 * (double)(rows < kNt ? rows : kNt));
      if (t < best) {
        best = t;
        c.clusters = k;
      }
    }
    const double t = cost(tiles(BM) * NB, KB, 0.45, 1.2);
    if (t < best) {
      best = t;
      c.variant = 1;
    }
  }
  const double t = gate_up ? cost(tiles(BM) * NB, KB, 0.74, 2.5)
                           : cost(tiles(BM) * ((a.N + 255) / 256), KB, 0.72, 2.0);
  if (t < best) {
    best = t;
    c.variant = 2;
  }
  if (!gate_up && !a.offsets && a.S <= kFewRows && few_smem(a.S, a.K) <= kFewMaxSmem) {
    const int64_t per_wave = (int64_t)sms * kFewWarps;
    const double few = (double)((a.N + per_wave - 1) / per_wave) * ((a.K + 511) / 512) *
                           (0.12 + 0.14 * (double)a.S);
    if (few < best) c.variant = 3;
  }
  return c;
}

struct Operands {
  const uint8_t* xq;
  const uint8_t* w0;
  const uint8_t* w1;  // gate_up
};

template <int M>
cudaError_t launch_few(const Operands& o, const Args& args, cudaStream_t s) {
  static std::once_flag once[kMaxDevices];
  static cudaError_t set_up[kMaxDevices];
  const cudaError_t e = once_per_device(once, set_up, [](int) {
    return cudaFuncSetAttribute(k_linear_few<M>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kFewMaxSmem);
  });
  if (e != cudaSuccess) return e;
  const int ctas = (args.N + kFewWarps - 1) / kFewWarps, sms = dev_info()->sm_count;
  const size_t smem = few_smem(M, args.K);
  return launch_pdl(k_linear_few<M>, dim3(ctas < sms ? ctas : sms), dim3(32 * kFewWarps), smem, s,
                    o.w0, o.xq, args);
}

template <int MODE>
int run_product(const Operands& o, const Args& args, cudaStream_t s) {
  const Choice c = choose(args, MODE == kGateUp);
  if (c.variant == 3) {
    const cudaError_t e = args.S == 1   ? launch_few<1>(o, args, s)
                          : args.S == 2 ? launch_few<2>(o, args, s)
                          : args.S == 3 ? launch_few<3>(o, args, s)
                                        : launch_few<4>(o, args, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  CUtensorMap w0, w1, t, t128;
  if (!map_weights(&w0, o.w0, args.K, args.N, args.E) ||
      !map_rows(&t, o.xq, args.K, args.S, kSmallBox))
    return MOE_ERR_CUDA;
  if (MODE == kGateUp && !map_weights(&w1, o.w1, args.K, args.N, args.E)) return MOE_ERR_CUDA;
  const CUtensorMap& v1 = MODE == kGateUp ? w1 : w0;
  cudaError_t e;
  if (c.variant == 0) {
    const int sms = dev_info()->sm_count;
    const int64_t units = max_tiles(args, kNt) * ((args.N + 127) / 128);
    const unsigned grid = (unsigned)(units < sms ? units : sms);
    if constexpr (MODE == kGateUp)
      e = launch_dec<MODE, 3, 2, false>(w0, w1, t, args, grid, 1, s);
    else
      e = c.clusters > 1 ? launch_dec<MODE, 5, 2, true>(w0, w0, t, args, (unsigned)units * c.clusters,
                                                        c.clusters, s)
                         : launch_dec<MODE, 5, 2, false>(w0, w0, t, args, grid, 1, s);
  } else {
    if (!map_rows(&t128, o.xq, args.K, args.S, BM)) return MOE_ERR_CUDA;
    if constexpr (MODE == kGateUp)
      e = launch<MODE, 256>(w0, v1, t, t128, args, s);
    else
      e = c.variant == 1 ? launch<MODE, 128>(w0, v1, t, t128, args, s)
                         : launch<MODE, 256>(w0, v1, t, t128, args, s);
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

// Units are counted in 31 bits (more would be a terabyte of weights or outputs),
// tiles too, even where segments behind a bad one overlap.
bool fp8_units_fit(int64_t S, int E, int N) {
  return S / kNt + (S < E ? S : E) <= INT32_MAX / (((int64_t)N + 127) / 128) &&
         (S / kNt + 1) * E <= INT32_MAX;
}

int grouped_fp8_run(const uint8_t* xq, const float* xs, const int32_t* offsets, int E, int64_t S,
                    int K, const uint8_t* w, const float* ws, int N, const __nv_bfloat16* residual,
                    __nv_bfloat16* y, DeviceStatus* st, cudaStream_t s, bool early, bool reset) {
  Args a{};
  a.offsets = offsets;
  a.E = E;
  a.S = S;
  a.N = N;
  a.K = K;
  a.xs = xs;
  a.ws0 = ws;
  a.y = y;
  a.res = residual;
  a.early = early ? 1 : 0;
  a.reset = reset ? 1 : 0;
  a.probe = wait_probe();
  a.st = st;
  return run_product<kPlain>({xq, w, nullptr}, a, s);
}

size_t expert_fp8_scratch_bytes(int64_t S, int F) {
  return align_up((size_t)S * (size_t)F, 256) +
         align_up(sizeof(float) * (size_t)S * (size_t)((F + 127) / 128), 256);
}

int expert_ffn_fp8_run(const uint8_t* xq, const float* xs, const int32_t* offsets, int E, int64_t S,
                       int d, int F, const uint8_t* w1, const float* w1s, const uint8_t* w3,
                       const float* w3s, const uint8_t* w2, const float* w2s,
                       const moe_act_cfg& act, bool pow2, __nv_bfloat16* y, void* scratch,
                       DeviceStatus* st, cudaStream_t s, bool reset) {
  uint8_t* hq = static_cast<uint8_t*>(scratch);
  float* hs = reinterpret_cast<float*>(hq + align_up((size_t)S * (size_t)F, 256));
  Args a{};
  a.offsets = offsets;
  a.E = E;
  a.S = S;
  a.N = F;
  a.K = d;
  a.xs = xs;
  a.ws0 = w1s;
  a.ws1 = w3s;
  a.hq = hq;
  a.hs = hs;
  a.act_kind = act.kind;
  a.beta = act.beta;
  a.lbeta = act.linear_beta;
  a.pow2 = pow2 ? 1 : 0;
  a.reset = reset ? 1 : 0;
  a.probe = wait_probe();
  a.st = st;
  const int rc = run_product<kGateUp>({xq, w1, w3}, a, s);
  if (rc) return rc;
  // offsets were read by the kernel just launched, after its own wait: the
  // down kernel may read them, and fetch weights, before that kernel ends
  return grouped_fp8_run(hq, hs, offsets, E, S, F, w2, w2s, d, nullptr, y, st, s, true, false);
}

}  // namespace moe
