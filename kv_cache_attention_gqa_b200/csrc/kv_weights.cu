// Attention weight of every cached key: w[b, g, j] (+)= sum over the heads a of group g and the query
// rows i that see key j of P = exp(scale q_{a,i} . k_j - lse_{a,i}), lse from the forward pass.
//
// Mathematics. Given lse the softmax needs no further statistics, so the weight of a key is a plain sum
// over query rows of exp2(c s - lse2) with c = scale log2 e. The probabilities are never stored.
//
// bf16 kernel: key-stationary on the tensor cores. A unit of work is 128 keys of one (sequence, KV head)
// against the query rows that see them (all of them, or one of `parts` shares of them). The keys sit on
// the 128 TMEM lanes, S^T = K Q^T (tcgen05.mma, A = K tile, B = Q tile, both K-major in shared memory), so
// the sum over rows runs along the columns a thread reads of its own lane: no exchange between threads, no
// atomics, the same result every time. A Q tile is kNQ columns: P positions (a power of two) of H heads.
//   kNQ = 128: prompts and windows of queries. Bound by the exponentials (one per visible pair; 16 a clock
//              and SM) next to the MMA (512 clocks a 128 x 128 x 128 tile). Two warpgroups take half of the
//              columns of each tile; S^T is buffered four deep.
//   kNQ = 32:  a few rows per group (one decoded token): one Q tile a unit, bound by reading K once.
// When the units are fewer than the SMs need, or uneven (causal), the query rows of a unit are cut into
// `parts`, whose sums meet in a second launch in a fixed order.
// The grid is persistent, one CTA per SM; all roles walk the same units:
//   warp 0      producer: K tiles and Q tiles by TMA into two rings; -lse2 and position of each column
//   warp 1      issues the MMAs
//   warps 2...  one thread per key and warpgroup: exponentials and sums (compensated, so that thousands of
//               rows keep fp32 accuracy)
//
// fp32 check mode: one thread per key, scalar FFMA.

#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace gqa {
namespace kw {

constexpr int kBK = 128;  // keys of a unit (= TMEM lanes)
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kFar = 0x7ffffffe;  // the position of a row that sees every key (no causal mask)
constexpr int kUnitsPerSm = 12;   // units wanted per SM before query rows are cut into parts
constexpr int kTilesPerPart = 4;  // a part holds at least this many Q tiles (of the fullest unit)

struct WArgs {
  float* w;
  const float* lse;
  const int32_t* q_start;
  const int32_t* kv_len;
  int B, h_q, h_kv, r, S_q, T_max;
  int P, H, hblocks, npb;  // Q tile: P positions x H heads; blocks of heads, of positions
  int N;                   // columns of a Q tile (MMA N)
  int nkt;                 // key tiles of a sequence
  int parts;
  long long n_units;
  float sl2;
  int causal, window, accumulate;
  float* part;  // (parts, B * h_kv, nkt * 128) partial sums, when parts > 1
  const int32_t* block_table;
  int max_pages, page_size, num_pages, sub;  // sub: keys per K copy (128, or 64 / 16 on a paged cache)
  unsigned* err;
};

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort,
                                         unsigned* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_timer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0u) {
      if (*abort) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        set_device_error(err, GQA_DEVERR_TIMEOUT);
        *abort = 1;
        return false;
      }
    }
  }
}

// One unit: keys k0 .. k0 + 127 of (b, g), and the Q tiles t0 .. t1 - 1 of the list (head block, position
// block pb_lo + ...) of the tiles whose rows see any of them.
struct Unit {
  int b, g, part, k0, kv, qs;
  int pb_lo, npb;  // position blocks in sight
  int t0, t1;
  bool valid;
  __device__ __forceinline__ int n() const { return t1 - t0; }
};

__device__ __forceinline__ Unit make_unit(const WArgs& a, long long idx) {
  Unit u;
  // key tiles slowest: the tiles that most rows see (causal) come first, and a CTA's units spread over
  // the sequences
  const int bg_n = a.B * a.h_kv;
  const int kp = (int)(idx / bg_n), bg = (int)(idx - (long long)kp * bg_n);
  const int kt = kp / a.parts;
  u.part = kp - kt * a.parts;
  u.b = bg / a.h_kv;
  u.g = bg - u.b * a.h_kv;
  u.k0 = kt * kBK;
  u.kv = a.kv_len ? a.kv_len[u.b] : a.T_max;
  u.qs = a.q_start ? a.q_start[u.b] : u.kv - a.S_q;
  u.valid = u.kv >= 1 && u.kv <= a.T_max && u.qs >= 0;
  u.pb_lo = u.npb = u.t0 = u.t1 = 0;
  if (!u.valid || u.k0 >= u.kv) return u;
  int i_lo = 0, i_hi = a.S_q - 1;  // rows that may see one of the keys
  if (a.causal) {
    if (u.k0 - u.qs > 0) i_lo = u.k0 - u.qs;
    if (a.window > 0) {
      const long long hi = (long long)min(u.k0 + kBK, u.kv) - 1 + a.window - 1 - u.qs;
      if (hi < i_hi) i_hi = (int)(hi < -1 ? -1 : hi);
    }
  }
  if (i_lo > i_hi) return u;
  u.pb_lo = i_lo / a.P;
  u.npb = i_hi / a.P - u.pb_lo + 1;
  const long long n = (long long)u.npb * a.hblocks;
  u.t0 = (int)(n * u.part / a.parts);
  u.t1 = (int)(n * (u.part + 1) / a.parts);
  return u;
}

// CTA c of G takes units c, 2G - 1 - c, 2G + c, ...: a snake over the heaviest-first order.
__device__ __forceinline__ long long unit_of(int it) {
  const long long base = (long long)it * gridDim.x;
  return base + ((it & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

template <int D, int kNQ>
struct Cfg {
  static constexpr int kNch = D / 64;
  static constexpr int kWG = kNQ == 128 ? 2 : 1;  // epilogue warpgroups
  static constexpr int kThreads = 64 + 128 * kWG;
  static constexpr int kKStages = kNQ == 128 ? 2 : 5;
  static constexpr int kQStages = kNQ == 128 ? 4 : 5;
  static constexpr int kBufs = kNQ == 128 ? 4 : 8;  // S^T buffers in TMEM and their column statistics
  static constexpr uint32_t kTmemCols = kBufs * kNQ;
  static constexpr int kKChunk = kBK * 128, kKBytes = kNch * kKChunk;
  static constexpr int kQChunkMax = kNQ * 128, kQBytes = kNch * kQChunkMax;
  static constexpr int kOffQ = kKStages * kKBytes;
  static constexpr int kOffStat = kOffQ + kQStages * kQBytes;
  // per buffer: -lse2 of the columns, their positions, and (min, max) position of each 32 columns
  static constexpr int kStatWords = 2 * kNQ + 2 * (kNQ / 32);
  static constexpr int kOffX = kOffStat + kBufs * kStatWords * 4;  // second warpgroup's sums, two units
  static constexpr int kOffBar = kOffX + (kWG == 2 ? 2 * 128 * 4 : 0);
  static constexpr int kSmemRaw = kOffBar + 512 + 1024;
  // at least half of an SM's shared memory: one CTA per SM (it allocates up to all TMEM columns)
  static constexpr int kSmem = kSmemRaw > 120 * 1024 ? kSmemRaw : 120 * 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  // barriers
  static constexpr int bKFull = 0, bKEmpty = bKFull + kKStages, bQFull = bKEmpty + kKStages,
                       bQEmpty = bQFull + kQStages, bS = bQEmpty + kQStages, bStat = bS + kBufs,
                       bFree = bStat + kBufs, bX = bFree + kBufs, bY = bX + 2, bDone = bY + 2,
                       kBars = bDone + 1;
  static_assert(kBars * 8 + 16 <= 512, "barrier block");
};

template <int D, int kNQ>
__global__ void __launch_bounds__(Cfg<D, kNQ>::kThreads, 1)
    kv_weights_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmq,
                      const __grid_constant__ WArgs a) {
  using C = Cfg<D, kNQ>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t sK = smem_u32(smem), sQ = smem_u32(smem + C::kOffQ);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  // column statistics of a buffer
  auto nl2 = [&](int bf) { return reinterpret_cast<float*>(smem + C::kOffStat) + bf * C::kStatWords; };
  auto cpos = [&](int bf) { return reinterpret_cast<int*>(nl2(bf) + kNQ); };
  auto crange = [&](int bf) { return reinterpret_cast<int*>(nl2(bf) + 2 * kNQ); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kKStages; ++i) {
      mbar_init(bar(C::bKFull + i), 1);
      mbar_init(bar(C::bKEmpty + i), 1);
    }
    for (int i = 0; i < C::kQStages; ++i) {
      mbar_init(bar(C::bQFull + i), 1);
      mbar_init(bar(C::bQEmpty + i), 1);
    }
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(bar(C::bS + i), 1);
      mbar_init(bar(C::bStat + i), 32);
      mbar_init(bar(C::bFree + i), 4 * C::kWG);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::bX + i), 128);
      mbar_init(bar(C::bY + i), 128);
    }
    mbar_init(bar(C::bDone), 1);
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  cta_sync();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int q_chunk = a.N * 128;  // bytes of one 64-column chunk of a Q tile

  if (warp == 0) {
    // ------------------------------ producer ------------------------------------------------
    if (lane == 0) {
      tma_prefetch_desc(&tmk);
      tma_prefetch_desc(&tmq);
    }
    int nk = 0, nt = 0;  // K tiles and Q tiles issued
    int ok = 1;
    for (int it = 0; ok; ++it) {
      const long long idx = unit_of(it);
      if (idx >= a.n_units) break;
      const Unit u = make_unit(a, idx);
      if (!u.valid && u.k0 == 0 && u.part == 0 && u.g == 0 && lane == 0)
        set_device_error(a.err, u.kv < 1 || u.kv > a.T_max ? GQA_DEVERR_KV_LEN : GQA_DEVERR_POSITION);
      if (u.n() == 0) continue;
      // K tile: one copy per 64-column chunk and sub-tile that holds cached keys
      {
        const int st = nk % C::kKStages, f = nk / C::kKStages;
        const int n_sub = (min(kBK, u.kv - u.k0) + a.sub - 1) / a.sub;
        int row = 0;
        if (a.block_table) {
          if (lane < n_sub) {
            const int key = u.k0 + lane * a.sub;
            int page = __ldg(a.block_table + (long long)u.b * a.max_pages + key / a.page_size);
            if (page < 0 || page >= a.num_pages) {
              set_device_error(a.err, GQA_DEVERR_PAGE);
              page = 0;
            }
            row = (page * a.h_kv + u.g) * a.page_size + key % a.page_size;
          }
        } else {
          row = (u.b * a.h_kv + u.g) * a.T_max + u.k0;
        }
        if (lane == 0) {
          if (f > 0) ok = wait_bar(bar(C::bKEmpty + st), (uint32_t)((f - 1) & 1), abort, a.err);
          if (ok) mbar_arrive_expect_tx(bar(C::bKFull + st), (uint32_t)(n_sub * a.sub * 128 * C::kNch));
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (lane < n_sub) {
#pragma unroll
          for (int ch = 0; ch < C::kNch; ++ch)
            tma_load_2d(sK + st * C::kKBytes + ch * C::kKChunk + lane * a.sub * 128, &tmk,
                        bar(C::bKFull + st), ch * 64, row);
        }
        ++nk;
      }
      for (int t = u.t0; t < u.t1; ++t, ++nt) {
        const int hb = t / u.npb, pb = u.pb_lo + t - hb * u.npb;
        const int head0 = u.g * a.r + hb * a.H, i0 = pb * a.P;
        // statistics of this lane's columns: the loads are on their way before the ring is waited for
        constexpr int kPer = kNQ / 32;
        float l[kPer];
        int ps[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const int n = e * 32 + lane;
          const int h = n / a.P, i = i0 + n - h * a.P;
          const bool in = n < a.N && hb * a.H + h < a.r && i < a.S_q;
          l[e] = in ? __ldg(a.lse + ((long long)u.b * a.h_q + head0 + h) * a.S_q + i) : -INFINITY;
          ps[e] = a.causal ? (int)min((long long)u.qs + i, (long long)kFar) : kFar;
        }
        const int st = nt % C::kQStages, f = nt / C::kQStages;
        if (lane == 0) {
          if (f > 0) ok = wait_bar(bar(C::bQEmpty + st), (uint32_t)((f - 1) & 1), abort, a.err);
          if (ok) {
            mbar_arrive_expect_tx(bar(C::bQFull + st), (uint32_t)(C::kNch * q_chunk));
            for (int ch = 0; ch < C::kNch; ++ch)
              tma_load_3d(sQ + st * C::kQBytes + ch * q_chunk, &tmq, bar(C::bQFull + st), ch * 64, i0,
                          u.b * a.h_q + head0);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        const int bf = nt % C::kBufs, fb = nt / C::kBufs;
        if (lane == 0 && fb > 0) ok = wait_bar(bar(C::bFree + bf), (uint32_t)((fb - 1) & 1), abort, a.err);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) {
          ++nt;
          break;
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          // a row without a finite lse (no visible key, padding) takes part in nothing
          const bool in = l[e] != -INFINITY && l[e] == l[e];
          const int pos = in ? ps[e] : -1;
          nl2(bf)[e * 32 + lane] = in ? -l[e] * kLog2e : 0.f;
          cpos(bf)[e * 32 + lane] = pos;
          const int lo = __reduce_min_sync(0xffffffffu, pos), hi = __reduce_max_sync(0xffffffffu, pos);
          if (lane == 0) {
            crange(bf)[2 * e] = lo;
            crange(bf)[2 * e + 1] = hi;
          }
        }
        mbar_arrive(bar(C::bStat + bf));
      }
    }
    // drain (bounded): no copy may still land in shared memory at exit
    if (lane == 0) {
      volatile int no_abort = 0;
#pragma unroll
      for (int s = 0; s < C::kKStages; ++s)
        if (nk > s) wait_bar(bar(C::bKFull + s), (uint32_t)(((nk - 1 - s) / C::kKStages) & 1), &no_abort, a.err);
#pragma unroll
      for (int s = 0; s < C::kQStages; ++s)
        if (nt > s) wait_bar(bar(C::bQFull + s), (uint32_t)(((nt - 1 - s) / C::kQStages) & 1), &no_abort, a.err);
    }
  } else if (warp == 1) {
    // ------------------------------ MMA issuer ----------------------------------------------
    const uint32_t idesc = tc::idesc_bf16(kBK, a.N, false);
    const uint64_t dK = tc::smem_desc(sK, 16, 1024), dQ = tc::smem_desc(sQ, 16, 1024);
    auto wait = [&](int b_, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_bar(bar(b_), parity, abort, a.err)) != 0;
    };
    int nk = 0, nt = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const long long idx = unit_of(it);
      if (idx >= a.n_units) break;
      const Unit u = make_unit(a, idx);
      if (u.n() == 0) continue;
      const int ks = nk % C::kKStages;
      if (!(ok = wait(C::bKFull + ks, (uint32_t)((nk / C::kKStages) & 1)))) break;
      const uint64_t kd = dK + (uint64_t)((ks * C::kKBytes) >> 4);
      for (int t = u.t0; t < u.t1; ++t, ++nt) {
        const int st = nt % C::kQStages, bf = nt % C::kBufs, fb = nt / C::kBufs;
        ok = wait(C::bQFull + st, (uint32_t)((nt / C::kQStages) & 1)) &&
             (fb == 0 || wait(C::bFree + bf, (uint32_t)((fb - 1) & 1)));
        if (!ok) break;
        tc::fence_after_sync();
        const uint64_t qd = dQ + (uint64_t)((st * C::kQBytes) >> 4);
        if (tc::elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc::mma_ss(tmem + bf * kNQ, kd + tc::koff(k, C::kKChunk), qd + tc::koff(k, q_chunk), idesc,
                       k > 0 ? 1u : 0u);
          tc::commit(bar(C::bS + bf));
          tc::commit(bar(C::bQEmpty + st));
          if (t + 1 == u.t1) tc::commit(bar(C::bKEmpty + ks));
        }
        __syncwarp();
      }
      ++nk;
    }
    if (tc::elect_one()) tc::commit(bar(C::bDone));
    __syncwarp();
    volatile int no_abort = 0;
    wait_bar(bar(C::bDone), 0, &no_abort, a.err);
  } else {
    // ------------------------------ exponentials and sums: one key per thread ---------------
    const int wg = (warp - 2) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;  // TMEM lane = key of the unit
    const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
    float* xs = reinterpret_cast<float*>(smem + C::kOffX);
    constexpr int kCols = kNQ / C::kWG;  // columns of this warpgroup
    const int col0 = wg * kCols;
    int nt = 0, nu = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const long long idx = unit_of(it);
      if (idx >= a.n_units) break;
      const Unit u = make_unit(a, idx);
      const int key = u.k0 + row;
      float sum = 0.f, comp = 0.f;  // compensated sum of the 32-column sums
      for (int t = u.t0; t < u.t1; ++t, ++nt) {
        const int bf = nt % C::kBufs;
        const uint32_t ph = (uint32_t)((nt / C::kBufs) & 1);
        ok = wait_bar(bar(C::bS + bf), ph, abort, a.err) && wait_bar(bar(C::bStat + bf), ph, abort, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll
        for (int cc = 0; cc < kCols / 32; ++cc) {
          const int c0 = col0 + cc * 32;
          const int lo = crange(bf)[2 * (c0 / 32)], hi = crange(bf)[2 * (c0 / 32) + 1];
          if (hi < u.k0) continue;  // no column of these sees any of the keys
          float s[32];
          tc::ld32f(lane_addr + bf * kNQ + c0, s);
          tc::wait_ld();
          const bool all = lo >= u.k0 + kBK - 1 && (a.window == 0 || u.k0 > hi - a.window);
          const float* nl = nl2(bf) + c0;
          float s0 = 0.f, s1 = 0.f;
          if (all) {
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              s0 += fast_exp2(fmaf(s[k], a.sl2, nl[k]));
              s1 += fast_exp2(fmaf(s[k + 1], a.sl2, nl[k + 1]));
            }
          } else {
            const int* cp = cpos(bf) + c0;
            const int reach = a.window > 0 ? a.window : 0x7fffffff;
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              // key <= position, and within the window: position - key < window
              const bool v0 = key <= cp[k] && cp[k] - key < reach;
              const bool v1 = key <= cp[k + 1] && cp[k + 1] - key < reach;
              s0 += v0 ? fast_exp2(fmaf(s[k], a.sl2, nl[k])) : 0.f;
              s1 += v1 ? fast_exp2(fmaf(s[k + 1], a.sl2, nl[k + 1])) : 0.f;
            }
          }
          const float y = (s0 + s1) - comp, tot = sum + y;
          comp = (tot - sum) - y;
          sum = tot;
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::bFree + bf));
      }
      if (!ok) break;
      if (C::kWG == 2 && u.n() > 0) {
        // the second warpgroup hands its sums to the first (two units may be under way)
        const int sl = nu & 1;
        const uint32_t ph = (uint32_t)((nu >> 1) & 1);
        if (wg == 1) {
          if (nu >= 2) ok = wait_bar(bar(C::bY + sl), ph ^ 1u, abort, a.err);
          xs[sl * 128 + row] = sum;
          mbar_arrive(bar(C::bX + sl));
        } else {
          ok = wait_bar(bar(C::bX + sl), ph, abort, a.err);
          sum += xs[sl * 128 + row];
          mbar_arrive(bar(C::bY + sl));
        }
        ok = __all_sync(0xffffffffu, ok);
        ++nu;
        if (!ok) break;
      }
      if (wg == 0) {
        const long long bg = (long long)u.b * a.h_kv + u.g;
        if (a.parts > 1) {
          a.part[((long long)u.part * a.B * a.h_kv + bg) * ((long long)a.nkt * kBK) + key] = sum;
        } else if (key < a.T_max) {
          float* dst = a.w + bg * a.T_max + key;
          const bool in = u.valid && key < u.kv;
          if (!a.accumulate) *dst = in ? sum : 0.f;
          else if (in && u.n() > 0) *dst += sum;
        }
      }
    }
  }
  tc::fence_before_sync();
  cta_sync();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::kTmemCols);
  }
}

// The sums of the parts of each key, in their order.
__global__ void __launch_bounds__(256) kv_weights_join_kernel(const __grid_constant__ WArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int key = blockIdx.x * 256 + threadIdx.x;
  const long long bg = blockIdx.y;
  if (key >= a.T_max) return;
  const int b = (int)(bg / a.h_kv);
  const int kv = a.kv_len ? a.kv_len[b] : a.T_max;
  const int qs = a.q_start ? a.q_start[b] : kv - a.S_q;
  const bool in = kv >= 1 && kv <= a.T_max && qs >= 0 && key < kv;
  float* dst = a.w + bg * a.T_max + key;
  if (!in) {
    if (!a.accumulate) *dst = 0.f;
    return;
  }
  const long long stride = (long long)a.B * a.h_kv * a.nkt * kBK;
  const float* src = a.part + bg * a.nkt * kBK + key;
  float sum = 0.f;
  for (int p = 0; p < a.parts; ++p) sum += __ldcg(src + p * stride);
  *dst = a.accumulate ? *dst + sum : sum;
}

// =============================================================================================
// fp32 check mode: 128 keys per block, one per thread; 16 query rows at a time
// =============================================================================================
constexpr int kF32Rows = 16, kF32Cols = 32;

__global__ void __launch_bounds__(128) kv_weights_fp32_kernel(WArgs a, const float* q, const float* k, int D,
                                                              float scale) {
  __shared__ float ks[kF32Cols][kBK + 1];
  __shared__ float qsm[kF32Cols][kF32Rows];
  __shared__ float ls[kF32Rows];
  __shared__ int ps[kF32Rows];
  const int kt = blockIdx.x, g = blockIdx.y % a.h_kv, b = blockIdx.y / a.h_kv;
  const int k0 = kt * kBK, key = k0 + threadIdx.x;
  const int kv = a.kv_len ? a.kv_len[b] : a.T_max;
  const int qs = a.q_start ? a.q_start[b] : kv - a.S_q;
  const bool valid = kv >= 1 && kv <= a.T_max && qs >= 0;
  if (!valid && kt == 0 && g == 0 && threadIdx.x == 0)
    set_device_error(a.err, kv < 1 || kv > a.T_max ? GQA_DEVERR_KV_LEN : GQA_DEVERR_POSITION);
  const long long bg = (long long)b * a.h_kv + g;
  // this thread's key row (nullptr: not a cached key)
  const float* kr = nullptr;
  if (valid && key < kv) {
    long long row = bg * a.T_max + key;
    if (a.block_table) {
      int page = a.block_table[(long long)b * a.max_pages + key / a.page_size];
      if (page < 0 || page >= a.num_pages) {
        set_device_error(a.err, GQA_DEVERR_PAGE);
        page = 0;
      }
      row = ((long long)page * a.h_kv + g) * a.page_size + key % a.page_size;
    }
    kr = k + row * D;
  }
  float sum = 0.f, comp = 0.f;
  if (valid && k0 < kv) {
    const long long rows = (long long)a.r * a.S_q, q0 = ((long long)b * a.h_q + (long long)g * a.r) * a.S_q;
    for (long long r0 = 0; r0 < rows; r0 += kF32Rows) {
      float acc[kF32Rows];
#pragma unroll
      for (int i = 0; i < kF32Rows; ++i) acc[i] = 0.f;
      for (int c0 = 0; c0 < D; c0 += kF32Cols) {
        __syncthreads();
        for (int c = 0; c < kF32Cols; ++c) ks[c][threadIdx.x] = kr && c0 + c < D ? kr[c0 + c] : 0.f;
        for (int e = threadIdx.x; e < kF32Rows * kF32Cols; e += 128) {
          const int i = e / kF32Cols, c = e - i * kF32Cols;
          qsm[c][i] = r0 + i < rows && c0 + c < D ? q[(q0 + r0 + i) * D + c0 + c] : 0.f;
        }
        if (c0 == 0 && threadIdx.x < kF32Rows) {
          const long long rr = r0 + threadIdx.x;
          const float l = rr < rows ? a.lse[q0 + rr] : -INFINITY;
          const long long pos = (long long)qs + rr % a.S_q;
          ls[threadIdx.x] = l;
          ps[threadIdx.x] = l == -INFINITY || l != l ? -1 : a.causal ? (int)min(pos, (long long)kFar) : kFar;
        }
        __syncthreads();
#pragma unroll 4
        for (int c = 0; c < kF32Cols; ++c) {
          const float kc = ks[c][threadIdx.x];
#pragma unroll
          for (int i = 0; i < kF32Rows; ++i) acc[i] = fmaf(kc, qsm[c][i], acc[i]);
        }
      }
      const int reach = a.window > 0 ? a.window : 0x7fffffff;
#pragma unroll
      for (int i = 0; i < kF32Rows; ++i) {
        if (key > ps[i] || ps[i] - key >= reach) continue;
        const float y = expf(fmaf(acc[i], scale, -ls[i])) - comp, tot = sum + y;
        comp = (tot - sum) - y;
        sum = tot;
      }
    }
  }
  if (key >= a.T_max) return;
  float* dst = a.w + bg * a.T_max + key;
  if (!a.accumulate) *dst = kr ? sum : 0.f;
  else if (kr) *dst += sum;
}

// -------------------------------------------------------------------------------------------------
// host side
// -------------------------------------------------------------------------------------------------
// Tile geometry: P positions (the power of two at or above S_q, at most the tile) of H heads.
struct Geometry {
  bool small;
  int P, H, N, hblocks, npb, parts;
};
Geometry geometry(int B, int h_q, int h_kv, int S_q, int T_max, int num_sms) {
  Geometry m;
  const int r = h_q / h_kv;
  int p2 = 1;
  while (p2 < S_q && p2 < 128) p2 <<= 1;
  // every row of the group fits 32 columns: one small Q tile per unit, and more K tiles in flight
  m.small = S_q <= 32 && (long long)p2 * r <= 32;
  m.N = m.small ? (p2 * r <= 16 ? 16 : 32) : 128;
  m.P = p2;
  m.H = m.N / m.P;
  m.hblocks = (r + m.H - 1) / m.H;
  m.npb = (S_q + m.P - 1) / m.P;
  m.parts = 1;
  const long long units = (long long)B * h_kv * ((T_max + kBK - 1) / kBK);
  const long long tiles = (long long)m.hblocks * m.npb;
  const long long want = ((long long)kUnitsPerSm * num_sms + units - 1) / units;
  const long long most = (tiles + kTilesPerPart - 1) / kTilesPerPart;
  if (!m.small && num_sms > 0) m.parts = (int)(want < most ? want : most);
  if (m.parts < 1) m.parts = 1;
  return m;
}

template <int D, int kNQ>
cudaError_t launch_typed(const WArgs& w, const CUtensorMap* tm, int num_sms, cudaStream_t s) {
  using C = Cfg<D, kNQ>;
  auto kern = kv_weights_kernel<D, kNQ>;
  static bool attr_set[64] = {false};  // per device: the shared-memory opt-in is set once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const unsigned grid = (unsigned)(w.n_units < num_sms ? w.n_units : num_sms);
  kern<<<grid, C::kThreads, C::kSmem, s>>>(tm[0], tm[1], w);
  e = cudaGetLastError();
  if (e != cudaSuccess || w.parts == 1) return e;
  kv_weights_join_kernel<<<dim3((w.T_max + 255) / 256, w.B * w.h_kv), 256, 0, s>>>(w);
  return cudaGetLastError();
}

WArgs make_args(const KvWeightsArgs& a, const Geometry& m) {
  WArgs w;
  w.w = a.w;
  w.lse = a.lse;
  w.q_start = a.q_start;
  w.kv_len = a.kv_len;
  w.B = a.B;
  w.h_q = a.h_q;
  w.h_kv = a.h_kv;
  w.r = a.h_q / a.h_kv;
  w.S_q = a.S_q;
  w.T_max = a.T_max;
  w.P = m.P;
  w.H = m.H;
  w.hblocks = m.hblocks;
  w.npb = m.npb;
  w.N = m.N;
  w.nkt = (a.T_max + kBK - 1) / kBK;
  w.parts = m.parts;
  w.n_units = (long long)a.B * a.h_kv * w.nkt * m.parts;
  w.sl2 = a.scale * kLog2e;
  w.causal = a.causal;
  w.window = a.window;
  w.accumulate = a.accumulate;
  w.part = reinterpret_cast<float*>(a.workspace);
  w.block_table = a.block_table;
  w.max_pages = a.max_pages;
  w.page_size = a.page_size;
  w.num_pages = a.num_pages;
  w.sub = kv_weights_sub(a.block_table != nullptr, a.page_size);
  w.err = a.err;
  return w;
}

}  // namespace kw

int kv_weights_sub(bool paged, int page_size) { return !paged ? 128 : page_size % 64 == 0 ? 64 : 16; }

void kv_weights_tile(int h_q, int h_kv, int S_q, int* P, int* H) {
  const kw::Geometry m = kw::geometry(1, h_q, h_kv, S_q, 1, 0);
  *P = m.P;
  *H = m.H;
}

size_t kv_weights_workspace_bytes(int B, int h_q, int h_kv, int S_q, int T_max, gqa_dtype dtype, int num_sms) {
  if (dtype == GQA_FP32) return 0;
  const kw::Geometry m = kw::geometry(B, h_q, h_kv, S_q, T_max, num_sms);
  if (m.parts == 1) return 0;
  return (size_t)m.parts * B * h_kv * ((T_max + kw::kBK - 1) / kw::kBK) * kw::kBK * sizeof(float);
}

cudaError_t launch_kv_weights_bf16(const KvWeightsArgs& a, const CUtensorMap* tmaps, int num_sms, cudaStream_t s) {
  const kw::Geometry m = kw::geometry(a.B, a.h_q, a.h_kv, a.S_q, a.T_max, num_sms);
  const kw::WArgs w = kw::make_args(a, m);
  if (a.d_h == 128) return m.small ? kw::launch_typed<128, 32>(w, tmaps, num_sms, s) : kw::launch_typed<128, 128>(w, tmaps, num_sms, s);
  if (a.d_h == 64) return m.small ? kw::launch_typed<64, 32>(w, tmaps, num_sms, s) : kw::launch_typed<64, 128>(w, tmaps, num_sms, s);
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv_weights_fp32(const KvWeightsArgs& a, cudaStream_t s) {
  const kw::Geometry m = kw::geometry(a.B, a.h_q, a.h_kv, a.S_q, a.T_max, 0);
  const kw::WArgs w = kw::make_args(a, m);
  const long long bg = (long long)a.B * a.h_kv;
  if (bg > 65535) return cudaErrorInvalidConfiguration;
  kw::kv_weights_fp32_kernel<<<dim3(w.nkt, (unsigned)bg), 128, 0, s>>>(
      w, reinterpret_cast<const float*>(a.q), reinterpret_cast<const float*>(a.k), a.d_h, a.scale);
  return cudaGetLastError();
}

}  // namespace gqa
