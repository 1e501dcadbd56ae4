// Device helpers shared by the kernels of this library: bf16 packing, mbarrier and TMA wrappers
// (inline PTX for sm_100a), bounded waits and the sticky device error word.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gqa.h"

namespace gqa {

// A pipeline wait gives up after this many nanoseconds of %globaltimer (about 2 s): the kernel
// then records GQA_DEVERR_TIMEOUT and returns instead of spinning forever.
constexpr unsigned long long kWaitLimitNs = 2000000000ull;

__device__ __forceinline__ unsigned long long global_timer_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Record the first device-side error (later ones are dropped). err may be null.
__device__ __forceinline__ void set_device_error(unsigned* err, unsigned code) {
  if (err) atomicCAS(err, 0u, code);
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---------------------------------------------------------------------------------------------
// mbarrier
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

// CTA-wide barrier for code where a warp's lanes may have diverged before it (one lane running a
// producer loop while the others skip it, a loop over threadIdx). __syncthreads is the aligned
// form of the barrier, which expects every warp to arrive converged: a warp whose lanes got there
// at different times counted twice, and the barrier ending an item of the backward kernel let
// thread 0 through two to five microseconds before the MMA and elementwise warps arrived (a
// __syncwarp in front did not change that). The unaligned form counts threads one by one.
__device__ __forceinline__ void cta_sync() {
  asm volatile("barrier.sync 0;" ::: "memory");
}

// Invalidates an mbarrier (before its shared memory is initialised again or used for data).
__device__ __forceinline__ void mbar_inval(uint32_t bar) {
  asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_barrier_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes)
      : "memory");
}

// Non-blocking: has the phase with this parity completed?
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Wait until the phase with the given parity has completed. Returns false (after recording
// GQA_DEVERR_TIMEOUT) if that takes longer than kWaitLimitNs.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, unsigned* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_timer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 0u && global_timer_ns() - t0 > kWaitLimitNs) {
      set_device_error(err, GQA_DEVERR_TIMEOUT);
      return false;
    }
  }
}

// ---------------------------------------------------------------------------------------------
// TMA (cp.async.bulk.tensor): each CTA loads its own tiles
// ---------------------------------------------------------------------------------------------
// Ask for `bytes` of global memory at `p` to be brought into L2 (both 16-byte aligned/multiples);
// nothing waits for it.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(__cvta_generic_to_global(p)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void tma_prefetch_desc(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// 2-D tile load into shared memory; completion is signalled on `bar` as transaction bytes.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

// 3-D tile load (x innermost).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// 4-D tile load (x innermost).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// n / d for 0 <= n < 2^31 and 1 <= d < 2^31 by a multiply and a shift (division by an invariant
// integer, Granlund and Montgomery 1994): q = (umulhi(n, m) + n) >> s with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1. An integer divide by a run-time value is a chain of a few
// dozen instructions through the reciprocal unit, which the exponential-heavy warps of the same
// SM keep busy; the persistent kernels' per-item bookkeeping divides with this instead.
struct FastDiv {
  uint32_t m, s;
  static FastDiv make(uint32_t d) {
    FastDiv f;
    f.s = 0;
    while ((1ull << f.s) < d) ++f.s;
    f.m = (uint32_t)((((1ull << 32) * ((1ull << f.s) - d)) / d) + 1);
    return f;
  }
  __device__ __forceinline__ int div(int n) const {
    return (int)((__umulhi((uint32_t)n, m) + (uint32_t)n) >> s);
  }
};

// ---------------------------------------------------------------------------------------------
// Warp-level helpers
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Packed fp32 pairs (sm_100: two lanes of work per instruction).
__device__ __forceinline__ float2 pair_fma(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mov.b64 rc, {%6, %7};\n\tfma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 pair_add(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 pair_mul(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// ---------------------------------------------------------------------------------------------
// Modified scores: a cap by tanh, a bias that grows with distance, a range of keys per row
// ---------------------------------------------------------------------------------------------
// Kernel-side form of gqa_score_mod. With x = s k1 (s the raw product q.k, k1 = scale / cap) the base-2 score is
// cap2 tanh(x) - slope2 |p - j|, cap2 = cap log2 e; without a cap it is s scale log2 e - slope2 |p - j|.
struct ModArgs {
  float k1 = 0.f, cap2 = 0.f;     // cap2 = 0: no cap
  const float* slopes = nullptr;  // (h_q) natural-log slopes, or none
  const int2* range = nullptr;    // (B, S_q) (decode: (B)) keys lo <= j < hi of each row, or none
  const int4* hull = nullptr;     // per row block: least lo and largest hi of the rows that see any, then
                                  // largest lo and least hi of all rows (RowStart)
};

// Check mode: the score of one pair in natural units, `t` its tanh (for the gradient; 0 without a cap).
__device__ __forceinline__ float mod_score(float dot, float scale, float cap, float slope, long long away, float* t) {
  float s = dot * scale;
  *t = 0.f;
  if (cap > 0.f) {
    *t = tanhf(s / cap);
    s = cap * *t;
  }
  return slope != 0.f ? fmaf(-slope, fabsf((float)away), s) : s;
}

// Bits [lo, hi) of 32, the bounds clamped to them. A test of one bit costs an instruction, where two bounds cost two
// comparisons.
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
  uint32_t a, b;  // shl.b32 by 32 or more gives 0
  asm("shl.b32 %0, %1, %2;" : "=r"(a) : "r"(0xffffffffu), "r"(max(lo, 0)));
  asm("shl.b32 %0, %1, %2;" : "=r"(b) : "r"(0xffffffffu), "r"(max(hi, 0)));
  return a & ~b;
}

// tanh of a pair with |x| <= kTanhSmall: x times a polynomial in z = x^2. Its coefficients are the fit of tanh(x) / x with
// the least maximum relative error, by Lawson's method: least squares over points of (0, 0.6], again and again, each time
// with the weights multiplied by the errors, until these are level (7.3e-8). Rounded to fp32 they give 9.2e-8, and 1.8e-7
// with the roundings of the evaluation. (The first one is not 1: the error is spread over the interval.)
constexpr float kTanhSmall = 0.6f;
__device__ __forceinline__ float2 pair_tanh_small(float2 x) {
  const float2 z = pair_mul(x, x);
  float2 p = pair_fma(make_float2(0x1.fb194ap-7f, 0x1.fb194ap-7f), z, make_float2(-0x1.aad0bap-5f, -0x1.aad0bap-5f));
  p = pair_fma(p, z, make_float2(0x1.1097a4p-3f, 0x1.1097a4p-3f));
  p = pair_fma(p, z, make_float2(-0x1.5552a6p-2f, -0x1.5552a6p-2f));
  p = pair_fma(p, z, make_float2(0x1.fffffep-1f, 0x1.fffffep-1f));
  return pair_mul(p, x);
}
// tanh of a pair of any size: x P(z) / Q(z), Q(0) = 1, the fit of tanh(x) / x over (0, kTanhMost] by the same method (least
// squares of (P - Q tanh(x) / x), divided by the Q of the step before): 1.2e-7, with the roundings of the evaluation and
// an ulp of the reciprocal 5.2e-7. Past kTanhMost the value there, 1 - 3e-7. P and Q have positive coefficients only, so
// nothing cancels: small scores keep their accuracy however large the cap is, and the result is never above 1.
constexpr float kTanhMost = 7.8f;
__device__ __forceinline__ float within_nan(float x, float most) {  // x held to [-most, most]; NaN stays NaN
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(-most));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(y), "f"(most));
  return y;
}
__device__ __forceinline__ float2 pair_tanh_any(float2 x) {
  x = make_float2(within_nan(x.x, kTanhMost), within_nan(x.y, kTanhMost));
  const float2 z = pair_mul(x, x);
  float2 p = pair_fma(make_float2(0x1.866e26p-17f, 0x1.866e26p-17f), z, make_float2(0x1.8544f8p-9f, 0x1.8544f8p-9f));
  float2 q = pair_fma(make_float2(0x1.0f40bcp-22f, 0x1.0f40bcp-22f), z, make_float2(0x1.fa2856p-13f, 0x1.fa2856p-13f));
  p = pair_fma(p, z, make_float2(0x1.091336p-3f, 0x1.091336p-3f));
  q = pair_fma(q, z, make_float2(0x1.8773fep-6f, 0x1.8773fep-6f));
  p = pair_fma(p, z, make_float2(0x1.fffffcp-1f, 0x1.fffffcp-1f));
  q = pair_fma(q, z, make_float2(0x1.d9debp-2f, 0x1.d9debp-2f));
  q = pair_fma(q, z, make_float2(1.f, 1.f));
  float2 r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(q.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(q.y));
  return pair_mul(pair_mul(x, p), r);
}
// s[k] = tanh(s[k] k1) for a thread's N scores, by the polynomial when every score of the warp is small enough (returns
// whether). Called by whole warps. `vote` is k1, or infinity (the same in the whole warp) for the way that holds for any
// size. The two differ in the last bits, so the choice must not hang on memory that may hold anything: callers pass
// infinity where some score is of a key that no row sees.
template <int N>
__device__ __forceinline__ bool tanh_scores(float* s, float k1, float vote) {
  float m0 = 0.f, m1 = 0.f;
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    m0 = fmaxf(m0, fabsf(s[k]));
    m1 = fmaxf(m1, fabsf(s[k + 1]));
  }
  const float2 k2 = make_float2(k1, k1);
  // (zero times infinity is no number, so not at most kTanhSmall either)
  const bool small = __all_sync(0xffffffffu, fmaxf(m0, m1) * vote <= kTanhSmall) != 0;
  if (small) {
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      const float2 t = pair_tanh_small(pair_mul(make_float2(s[k], s[k + 1]), k2));
      s[k] = t.x;
      s[k + 1] = t.y;
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      const float2 t = pair_tanh_any(pair_mul(make_float2(s[k], s[k + 1]), k2));
      s[k] = t.x;
      s[k + 1] = t.y;
    }
  }
  return small;
}

// Barrier among `threads` threads (whole warps) on barrier `id`, aligned form: only where every
// warp taking part arrives converged (no role or lane-divergent loop right before it; the
// unaligned form, as in cta_sync, measured 2% slower on the decode_8k step).
__device__ __forceinline__ void named_barrier_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// 128B-swizzled address of the 16-byte chunk `chunk` (0..7) of row `row` inside a region whose
// rows are 128 bytes and whose base is 1024-byte aligned (the TMA SWIZZLE_128B layout).
__device__ __forceinline__ uint32_t swz128(uint32_t base, int row, int chunk) {
  return base + row * 128 + ((chunk ^ (row & 7)) << 4);
}

}  // namespace gqa
