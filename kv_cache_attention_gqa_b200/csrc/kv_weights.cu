// Attention weight of every cached key: w[b, g, j] (+)= sum over the heads a of group g and the query
// rows i that see key j of P = exp(scale q_{a,i} . k_j - lse_{a,i}), lse from the forward pass.
//
// Mathematics. Given lse the softmax needs no further statistics, so the weight of a key is a plain sum
// over query rows of exp2(c s - lse2) with c = scale log2 e. The probabilities are never stored. The exponent is one fp32
// fused multiply-add, so a weight's relative error is that of lse2 in fp32: 2^-24 |lse2| ln 2, 7e-7 at an lse2 of 16.
//
// bf16, more than 32 query rows a group (prompts, windows of queries): key-stationary on the tensor cores.
// A unit of work is 256 keys of one (sequence, KV head) against the query rows that see them (all of them,
// or one of `parts` shares of them). The keys of a K tile sit on the 128 TMEM lanes, S^T = K Q^T (tcgen05.mma, A = K tile, B = Q tile, both K-major in shared memory), so
// the sum over rows runs along the columns a thread reads of its own lane: no exchange between threads, no
// atomics, the same result every time. A Q tile is 128 columns: positions of one head, or with
// fewer than 128 positions the rows of the group's heads end to end.
// Four warpgroups: one per 128 keys and half of the columns; S^T is buffered twice. Bound by the exponentials (one
// per visible pair, 16 a clock and SM: 2048 of the 3300 clocks a 256 x 128 tile takes; the rest is TMEM loads and
// waits between the roles). Measured (B200, d = 128): 32 heads over 8 KV heads, 4096 rows, causal: 111 us, 617
// TFLOP/s; 33 rows over 2 x 32768 ragged keys in 16-key pages: 51 us. What did not help, at 4096 rows (best
// other form 115 us): even tiles to two warpgroups and odd ones to the other two, 137 us (each pair waits for its
// only buffer's MMA); a quarter, a half, three quarters of the exponentials as polynomials on the multiply-add
// pipe, 115, 124, 141 us; K as the A operand from TMEM with three 128-column score tiles, 126 us; 128 keys a
// unit, 109 us before the other steps, for twice the L2 reads of Q.
// When the units are fewer than the SMs need, or uneven (causal), the query rows of a unit are cut into
// `parts`, whose sums meet in a second launch in a fixed order.
// The grid is persistent, one CTA per SM; all roles walk the same units:
//   warp 0      producer: K tiles and Q tiles by TMA into two rings
//   warp 1      issues the MMAs
//   warp 2      -lse2 and position of each column of a Q tile
//   warps 4...  one thread per key and warpgroup: exponentials and sums (compensated, so that thousands of
//               rows keep fp32 accuracy)
//
// bf16, up to 32 query rows a group (one decoded token): bound by reading K once. A producer warp streams
// 128-key K tiles with the group's rows, eight warps take 16 keys of each tile: S = Q K^T by m16n8k16 MMAs
// (16 or 32 query rows are too few for a tcgen05 tile: its 128 x 16 MMAs took 1200 clocks a K tile against
// 1450 for the tile's bytes, 34 us for the case below), and the sum over rows is three shuffles. Measured:
// 8 sequences of 8192 keys, 8 KV heads, 4 rows each, d = 128 (138 MB): 31.0 us, 4.5 TB/s; two groups of
// eight warps taking tiles in turn: 32.8 us, so what is left is the start and the end of a launch this short.
//
// fp32 check mode: up to four threads to a key, one per group of 32 query rows, scalar FFMA.

#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace gqa {
namespace kw {

constexpr int kBK = 128;  // keys of a K tile (= TMEM lanes)
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSeqTable = 1024;  // sequences whose length and first position are kept in shared memory
constexpr int kFar = 0x7ffffffe;  // the position of a row that sees every key (no causal mask)
constexpr int kUnitsPerSm = 6;    // units wanted per SM before query rows are cut into parts
constexpr int kTilesPerPart = 4;  // a part holds at least this many Q tiles (of the fullest unit)

struct WArgs {
  float* w;
  const float* lse;
  const int32_t* q_start;
  const int32_t* kv_len;
  int B, h_q, h_kv, r, S_q, T_max;
  int P, H, hblocks, npb;  // Q tile: P positions x H heads; blocks of heads, of positions
  int N;                   // MMA columns of a Q tile: P H rounded up to 16 (the rest is masked)
  int flat;                // 1 (S_q < 128): a Q tile is 128 of the group's r S_q rows, which lie end to end
  int nkt;                 // units along the keys of a sequence
  int parts;
  int n_units;
  FastDiv div_bg, div_nkt, div_parts, div_hkv, div_P;
  float sl2;
  int causal, window, accumulate;
  float* part;  // (parts, B * h_kv, keys of all units) partial sums, when parts > 1
  int part_keys;
  const int32_t* block_table;
  int max_pages, page_size, num_pages, sub;  // sub: keys per K copy (128, or 64 / 16 on a paged cache)
  // Where a K tile's rows lie in shared memory: `k_chunk` bytes between its 64-column chunks, `k_group` between
  // groups of 8 rows. Plane by plane (16384, 1024), or on a paged cache with d = 128 both chunks of a group side by
  // side (1024, 2048): the copy of a sub-tile is then one box of four dimensions instead of one per chunk (33 rows
  // over paged keys 54 -> 51 us).
  int k_chunk, k_group, k_4d;
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

// One unit: kKeys keys from k0 on of (b, g), and the Q tiles t0 .. t1 - 1 of the list (head block, position
// block pb_lo + ...) of the tiles whose rows see any of them.
struct Unit {
  int b, g, part, k0, kv, qs;
  int pb_lo, npb;  // position blocks in sight
  int t0, t1;
  bool valid;
  __device__ __forceinline__ int n() const { return t1 - t0; }
};

// (kv_len, q_start) of a sequence
__device__ __forceinline__ int2 sequence(const WArgs& a, int b) {
  const int kv = a.kv_len ? a.kv_len[b] : a.T_max;
  return make_int2(kv, a.q_start ? a.q_start[b] : kv - a.S_q);
}

// seq: the first kSeqTable sequences' lengths and positions (a global load is a trip to L2 here, ~600
// clocks in every role: shared memory leaves no L1).
// kStream (the small kernel): key tiles fastest, so that the SMs together read the cache in its order.
template <int kKeys, bool kStream = false>
__device__ __forceinline__ Unit make_unit(const WArgs& a, const int2* seq, int idx) {
  Unit u;
  int kt, bg;
  if constexpr (kStream) {
    bg = a.div_nkt.div(idx);
    kt = idx - bg * a.nkt;
    u.part = 0;
  } else {
    // key tiles slowest: the tiles that most rows see (causal) come first, and a CTA's units spread over
    // the sequences
    const int kp = a.div_bg.div(idx);
    bg = idx - kp * (a.B * a.h_kv);
    kt = a.div_parts.div(kp);
    u.part = kp - kt * a.parts;
  }
  u.b = a.div_hkv.div(bg);
  u.g = bg - u.b * a.h_kv;
  u.k0 = kt * kKeys;
  const int2 sq = u.b < kSeqTable ? seq[u.b] : sequence(a, u.b);
  u.kv = sq.x;
  u.qs = sq.y;
  u.valid = u.kv >= 1 && u.kv <= a.T_max && u.qs >= 0;
  u.pb_lo = u.npb = u.t0 = u.t1 = 0;
  if (!u.valid || u.k0 >= u.kv) return u;
  int i_lo = 0, i_hi = a.S_q - 1;  // rows that may see one of the keys
  if (a.causal) {
    if (u.k0 - u.qs > 0) i_lo = u.k0 - u.qs;
    if (a.window > 0) {
      const long long hi = (long long)min(u.k0 + kKeys, u.kv) - 1 + a.window - 1 - u.qs;
      if (hi < i_hi) i_hi = (int)(hi < -1 ? -1 : hi);
    }
  }
  if (i_lo > i_hi) return u;
  u.pb_lo = a.div_P.div(i_lo);
  u.npb = a.div_P.div(i_hi) - u.pb_lo + 1;
  const int n = u.npb * a.hblocks;  // times parts below 2^31 (the host bounds the list by it)
  u.t0 = a.div_parts.div(n * u.part);
  u.t1 = a.div_parts.div(n * (u.part + 1));
  return u;
}

// Sub-tile `sub` (a.sub rows from `row` of the cache on) of a K tile.
template <int kNch>
__device__ __forceinline__ void load_keys(const WArgs& a, uint32_t tile, const CUtensorMap* map, uint32_t bar, int sub,
                                          int row) {
  if (a.k_4d) {
    tma_load_4d(tile + sub * (a.sub / 8) * a.k_group, map, bar, 0, 0, 0, row / 8);
  } else {
#pragma unroll
    for (int ch = 0; ch < kNch; ++ch) tma_load_2d(tile + ch * a.k_chunk + sub * a.sub * 128, map, bar, ch * 64, row);
  }
}

// CTA c of G takes units c, 2G - 1 - c, 2G + c, ...: a snake over the heaviest-first order.
__device__ __forceinline__ long long unit_of(int it) {
  const long long base = (long long)it * gridDim.x;
  return base + ((it & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

constexpr int kNQ = 128;  // columns of a Q tile

template <int D>
struct Cfg {
  static constexpr int kNch = D / 64;
  static constexpr int kWG = 4;  // warpgroups of exponentials
  static constexpr int kKT = 2;  // K tiles of a unit
  static constexpr int kKeys = kKT * kBK;
  static constexpr int kThreads = 128 + 128 * kWG;
  static constexpr int kKStages = 3;
  static constexpr int kQStages = 3;
  static constexpr int kBufs = 2;  // S^T buffers in TMEM and their column statistics
  static constexpr uint32_t kBufCols = kKT * kNQ;  // one buffer: a tile of scores per K tile
  static constexpr uint32_t kTmemCols = kBufs * kBufCols;
  static constexpr int kKChunk = kBK * 128, kKBytes = kNch * kKChunk;
  static constexpr int kQChunk = kNQ * 128, kQBytes = kNch * kQChunk;
  static constexpr int kOffQ = kKStages * kKBytes;
  static constexpr int kOffStat = kOffQ + kQStages * kQBytes;
  // per buffer: -lse2 of the columns, their positions, and (min, max) position of each 32 columns
  static constexpr int kStatWords = 2 * kNQ + 2 * (kNQ / 32);
  static constexpr int kOffX = kOffStat + kBufs * kStatWords * 4;  // sums over the second columns, two units
  static constexpr int kOffSeq = kOffX + 2 * kKeys * 4;
  static constexpr int kOffBar = kOffSeq + kSeqTable * 8;
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

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    kv_weights_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmq,
                      const __grid_constant__ WArgs a) {
  using C = Cfg<D>;
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
      mbar_init(bar(C::bX + i), 256);
      mbar_init(bar(C::bY + i), 256);
    }
    mbar_init(bar(C::bDone), 1);
    *abort = 0;
    fence_barrier_init();
  }
  int2* seq = reinterpret_cast<int2*>(smem + C::kOffSeq);
  for (int b = threadIdx.x; b < min(a.B, kSeqTable); b += C::kThreads) seq[b] = sequence(a, b);
  if (warp == 1) {
    tc::tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  cta_sync();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

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
      const Unit u = make_unit<C::kKeys>(a, seq, (int)idx);
      if (!u.valid && u.k0 == 0 && u.part == 0 && u.g == 0 && lane == 0)
        set_device_error(a.err, u.kv < 1 || u.kv > a.T_max ? GQA_DEVERR_KV_LEN : GQA_DEVERR_POSITION);
      if (u.n() == 0) continue;
      // K tiles that hold cached keys: one copy per 64-column chunk and sub-tile that holds any
      const int n_kt = min(C::kKT, (u.kv - u.k0 + kBK - 1) / kBK);
      for (int kt = 0; kt < n_kt; ++kt, ++nk) {
        const int st = nk % C::kKStages, f = nk / C::kKStages;
        const int k0 = u.k0 + kt * kBK;
        const int n_sub = (min(kBK, u.kv - k0) + a.sub - 1) / a.sub;
        int row = 0;
        if (a.block_table) {
          if (lane < n_sub) {
            const int key = k0 + lane * a.sub;
            int page = __ldg(a.block_table + (long long)u.b * a.max_pages + key / a.page_size);
            if (page < 0 || page >= a.num_pages) {
              set_device_error(a.err, GQA_DEVERR_PAGE);
              page = 0;
            }
            row = (page * a.h_kv + u.g) * a.page_size + key % a.page_size;
          }
        } else {
          row = (u.b * a.h_kv + u.g) * a.T_max + k0;
        }
        if (lane == 0) {
          if (f > 0) ok = wait_bar(bar(C::bKEmpty + st), (uint32_t)((f - 1) & 1), abort, a.err);
          if (ok) mbar_arrive_expect_tx(bar(C::bKFull + st), (uint32_t)(n_sub * a.sub * 128 * C::kNch));
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (lane < n_sub) load_keys<C::kNch>(a, sK + st * C::kKBytes, &tmk, bar(C::bKFull + st), lane, row);
      }
      if (!ok) break;
      if (lane == 0) {
        int hb = u.t0 / u.npb, pb = u.t0 - hb * u.npb;
        for (int t = u.t0; t < u.t1; ++t, ++nt) {
          const int st = nt % C::kQStages, f = nt / C::kQStages;
          if (f > 0) ok = wait_bar(bar(C::bQEmpty + st), (uint32_t)((f - 1) & 1), abort, a.err);
          if (!ok) break;
          const int head = u.b * a.h_q + u.g * a.r;
          mbar_arrive_expect_tx(bar(C::bQFull + st), (uint32_t)(C::kNch * (a.flat ? kNQ : a.P * a.H) * 128));
          for (int ch = 0; ch < C::kNch; ++ch)
            tma_load_3d(sQ + st * C::kQBytes + ch * C::kQChunk, &tmq, bar(C::bQFull + st), ch * 64,
                        a.flat ? head * a.S_q + t * kNQ : (u.pb_lo + pb) * a.P, a.flat ? 0 : head + hb * a.H);
          if (++pb == u.npb) {
            pb = 0;
            ++hb;
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
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
    const int rows = a.r * a.S_q;
    const uint64_t dK = tc::smem_desc(sK, 16, (uint32_t)a.k_group), dQ = tc::smem_desc(sQ, 16, 1024);
    const uint64_t khi = dK & 0xffffffff00000000ull, khi_q = dQ & 0xffffffff00000000ull;
    auto uniform = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
    auto wait = [&](int b_, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_bar(bar(b_), parity, abort, a.err)) != 0;
    };
    int nk = 0, nt = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const long long idx = unit_of(it);
      if (idx >= a.n_units) break;
      const Unit u = make_unit<C::kKeys>(a, seq, (int)idx);
      if (u.n() == 0) continue;
      const int n_kt = min(C::kKT, (u.kv - u.k0 + kBK - 1) / kBK);
      for (int kt = 0; kt < n_kt && ok; ++kt)
        ok = wait(C::bKFull + (nk + kt) % C::kKStages, (uint32_t)(((nk + kt) / C::kKStages) & 1));
      if (!ok) break;
      for (int t = u.t0; t < u.t1; ++t, ++nt) {
        const int st = nt % C::kQStages, bf = nt % C::kBufs, fb = nt / C::kBufs;
        ok = wait(C::bQFull + st, (uint32_t)((nt / C::kQStages) & 1)) &&
             (fb == 0 || wait(C::bFree + bf, (uint32_t)((fb - 1) & 1)));
        if (!ok) break;
        tc::fence_after_sync();
        // Everything an MMA takes is made warp-uniform first (the unit comes from shared memory, so the compiler
        // cannot know it): the low words of the descriptors, which hold the address, the TMEM column and the shape.
        const uint32_t ql = uniform((uint32_t)dQ + ((st * C::kQBytes) >> 4));
        const uint32_t kl0 = uniform((uint32_t)dK + (((nk % C::kKStages) * C::kKBytes) >> 4));
        const uint32_t kl1 = uniform((uint32_t)dK + ((((nk + 1) % C::kKStages) * C::kKBytes) >> 4));
        const uint32_t col = uniform(tmem + bf * C::kBufCols), two = uniform(n_kt > 1 ? 1u : 0u);
        const uint32_t idesc =
            uniform(tc::idesc_bf16(kBK, a.flat ? min(kNQ, (rows - t * kNQ + 15) / 16 * 16) : a.N, false));
        if (tc::elect_one()) {
          // the two K tiles' MMAs alternate: each waits for its own accumulator's last step
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t q = khi_q | (ql + (uint32_t)tc::koff(k, C::kQChunk));
            const uint32_t ko = (uint32_t)tc::koff(k, (uint32_t)a.k_chunk);
            tc::mma_ss(col, khi | (kl0 + ko), q, idesc, k > 0 ? 1u : 0u);
            if (two) tc::mma_ss(col + kNQ, khi | (kl1 + ko), q, idesc, k > 0 ? 1u : 0u);
          }
          tc::commit(bar(C::bS + bf));
          tc::commit(bar(C::bQEmpty + st));
          if (t + 1 == u.t1)
            for (int kt = 0; kt < n_kt; ++kt) tc::commit(bar(C::bKEmpty + (nk + kt) % C::kKStages));
        }
        __syncwarp();
      }
      nk += n_kt;
    }
    if (tc::elect_one()) tc::commit(bar(C::bDone));
    __syncwarp();
    volatile int no_abort = 0;
    wait_bar(bar(C::bDone), 0, &no_abort, a.err);
  } else if (warp == 2) {
    // ------------------------------ column statistics ---------------------------------------
    constexpr int kPer = kNQ / 32;
    int hn[kPer], pn[kPer];  // head and position of this lane's columns inside a tile
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int n = e * 32 + lane;
      hn[e] = n / a.P;
      pn[e] = n - hn[e] * a.P;
    }
    int nt = 0, ok = 1;
    for (int it = 0; ok; ++it) {
      const long long idx = unit_of(it);
      if (idx >= a.n_units) break;
      const Unit u = make_unit<C::kKeys>(a, seq, (int)idx);
      if (u.n() == 0) continue;
      int hb = u.t0 / u.npb, pb = u.t0 - hb * u.npb;
      for (int t = u.t0; t < u.t1; ++t, ++nt) {
        float l[kPer];
        int ps[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          int h = hb * a.H + hn[e], i = (u.pb_lo + pb) * a.P + pn[e];
          bool in = hn[e] < a.H && h < a.r && i < a.S_q;
          if (a.flat) {
            const int x = t * kNQ + e * 32 + lane;
            h = a.div_P.div(x);  // P = S_q
            i = x - h * a.S_q;
            in = h < a.r;
          }
          l[e] = in ? __ldg(a.lse + ((long long)u.b * a.h_q + u.g * a.r + h) * a.S_q + i) : -INFINITY;
          ps[e] = a.causal ? (int)min((long long)u.qs + i, (long long)kFar) : kFar;
        }
        if (++pb == u.npb) {
          pb = 0;
          ++hb;
        }
        const int bf = nt % C::kBufs, fb = nt / C::kBufs;
        if (lane == 0 && fb > 0) ok = wait_bar(bar(C::bFree + bf), (uint32_t)((fb - 1) & 1), abort, a.err);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
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
  } else if (warp >= 4) {
    // ------------------------------ exponentials and sums: one key per thread ---------------
    const int wg = (warp >> 2) - 1, quarter = warp & 3;
    const int row = quarter * 32 + lane;  // TMEM lane = key of the K tile
    const int kh = wg >> 1, ch = wg & 1;  // K tile and half of the columns of this warpgroup
    const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16) + kh * kNQ;
    float* xs = reinterpret_cast<float*>(smem + C::kOffX);
    const int reach = a.window > 0 ? a.window : 0x7fffffff;
    int nt = 0, nu = 0;            // Q tiles and units with any so far
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const long long idx = unit_of(it);
      if (idx >= a.n_units) break;
      const Unit u = make_unit<C::kKeys>(a, seq, (int)idx);
      const int k0 = u.k0 + kh * kBK, key = k0 + row;
      const long long bg = (long long)u.b * a.h_kv + u.g;
      const bool writes = ch == 0;
      const bool in = u.valid && key < u.kv;
      float* const dst = a.w + bg * a.T_max + key;
      // the entry to be added to is loaded ahead of the sum
      const float old = writes && a.accumulate && a.parts == 1 && in && u.n() > 0 ? *dst : 0.f;
      float sum = 0.f, comp = 0.f;  // compensated sum of the column groups' sums
      for (int t = u.t0; t < u.t1; ++t, ++nt) {
        const int bf = nt % C::kBufs;
        const uint32_t ph = (uint32_t)((nt / C::kBufs) & 1);
        ok = wait_bar(bar(C::bS + bf), ph, abort, a.err) && wait_bar(bar(C::bStat + bf), ph, abort, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc::fence_after_sync();
        const float2 c2 = make_float2(a.sl2, a.sl2);
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          const int c0 = cc * 64 + ch * 32;
          const int lo = crange(bf)[c0 / 16], hi = crange(bf)[c0 / 16 + 1];
          if (hi < k0 || k0 >= u.kv) continue;  // no column sees one of the keys, or there are none
          float s[32];
          tc::ld32f(lane_addr + bf * C::kBufCols + c0, s);
          tc::wait_ld();
          const bool all = lo >= k0 + kBK - 1 && (a.window == 0 || k0 > hi - a.window);
          const float* nl = nl2(bf) + c0;
          float2 acc = make_float2(0.f, 0.f);
          auto expo = [&](int k, float2 n) {
            const float2 x = pair_fma(make_float2(s[k], s[k + 1]), c2, n);
            return make_float2(fast_exp2(x.x), fast_exp2(x.y));
          };
          if (all) {
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const float4 n = *reinterpret_cast<const float4*>(nl + k);
              acc = pair_add(acc, expo(k, make_float2(n.x, n.y)));
              acc = pair_add(acc, expo(k + 2, make_float2(n.z, n.w)));
            }
          } else {
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              float2 p = expo(k, *reinterpret_cast<const float2*>(nl + k));
              // key <= position, and within the window: position - key < window
              const int2 at = *reinterpret_cast<const int2*>(cpos(bf) + c0 + k);
              if (key > at.x || at.x - key >= reach) p.x = 0.f;
              if (key > at.y || at.y - key >= reach) p.y = 0.f;
              acc = pair_add(acc, p);
            }
          }
          const float y = (acc.x + acc.y) - comp, tot = sum + y;
          comp = (tot - sum) - y;
          sum = tot;
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::bFree + bf));
      }
      if (!ok) break;
      if (u.n() > 0) {
        // the sums over the second columns join the first (two units may be under way)
        const int sl = nu & 1;
        const uint32_t ph = (uint32_t)((nu >> 1) & 1);
        float* x = xs + sl * C::kKeys + kh * kBK + row;
        if (ch == 1) {
          if (nu >= 2) ok = wait_bar(bar(C::bY + sl), ph ^ 1u, abort, a.err);
          *x = sum;
          mbar_arrive(bar(C::bX + sl));
        } else {
          ok = wait_bar(bar(C::bX + sl), ph, abort, a.err);
          sum += *x;
          mbar_arrive(bar(C::bY + sl));
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      if (u.n() > 0) ++nu;
      if (!writes) continue;
      if (a.parts > 1) a.part[((long long)u.part * a.B * a.h_kv + bg) * a.part_keys + key] = sum;
      else if (!a.accumulate && key < a.T_max) *dst = in ? sum : 0.f;
      else if (a.accumulate && in && u.n() > 0) *dst = old + sum;
    }
  }
  tc::fence_before_sync();
  cta_sync();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::kTmemCols);
  }
}

// =============================================================================================
// up to 32 query rows per group: K streams through, m16n8k16 MMAs
// =============================================================================================
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int MT>
struct SCfg {
  static constexpr int kNch = D / 64;
  static constexpr int kStages = D == 64 ? 8 : MT == 1 ? 6 : 5;
  static constexpr int kRows = 16 * MT;  // query rows of the tile
  static constexpr int kWarps = 8;       // consumers
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kKChunk = kBK * 128, kKBytes = kNch * kKChunk;
  static constexpr int kQChunk = kRows * 128, kQBytes = kNch * kQChunk;
  static constexpr int kStage = kKBytes + kQBytes;
  static constexpr int kOffStat = kStages * kStage;              // per stage: -lse2 and position of the rows
  static constexpr int kOffSeq = kOffStat + kStages * kRows * 8;
  static constexpr int kOffBar = kOffSeq + kSeqTable * 8;
  static constexpr int kSmem = kOffBar + 256 + 1024;
  static_assert(kSmem <= 227 * 1024 && 2 * kStages * 8 + 8 <= 256, "shared memory budget");
};

template <int D, int MT>
__global__ void __launch_bounds__(SCfg<D, MT>::kThreads, 1)
    kv_weights_small_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmq,
                            const __grid_constant__ WArgs a) {
  using C = SCfg<D, MT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);  // full (stages), empty (stages)
  volatile int* abort = reinterpret_cast<volatile int*>(bars + 2 * C::kStages);
  int2* seq = reinterpret_cast<int2*>(smem + C::kOffSeq);
  const uint32_t base = smem_u32(smem);
  auto full = [&](int st) { return smem_u32(&bars[st]); };
  auto empty = [&](int st) { return smem_u32(&bars[C::kStages + st]); };
  auto nl2 = [&](int st) { return reinterpret_cast<float*>(smem + C::kOffStat) + st * 2 * C::kRows; };
  auto cpos = [&](int st) { return reinterpret_cast<int*>(nl2(st) + C::kRows); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(full(i), 1 + 32);  // copies; the producer lanes' statistics
      mbar_init(empty(i), C::kWarps);
    }
    *abort = 0;
    fence_barrier_init();
  }
  for (int b = threadIdx.x; b < min(a.B, kSeqTable); b += C::kThreads) seq[b] = sequence(a, b);
  cta_sync();
  const int R = a.r * a.S_q;  // query rows of a group

  if (warp == C::kWarps) {
    // ------------------------------ producer ------------------------------------------------
    if (lane == 0) {
      tma_prefetch_desc(&tmk);
      tma_prefetch_desc(&tmq);
    }
    // lane = query row of the group: its head and row, and its lse, loaded one unit ahead
    const int h = lane / a.S_q, i = lane - h * a.S_q;
    auto lse_of = [&](const Unit& u) {
      return lane < R ? __ldg(a.lse + ((long long)u.b * a.h_q + u.g * a.r + h) * a.S_q + i) : -INFINITY;
    };
    int n = 0, ok = 1;
    int it = 0;
    // the next unit with keys to read (n_units: none)
    auto next = [&](Unit& u) {
      for (;; ++it) {
        const long long idx = unit_of(it);
        if (idx >= a.n_units) return false;
        u = make_unit<kBK, true>(a, seq, (int)idx);
        if (!u.valid && u.k0 == 0 && u.g == 0 && lane == 0)
          set_device_error(a.err, u.kv < 1 || u.kv > a.T_max ? GQA_DEVERR_KV_LEN : GQA_DEVERR_POSITION);
        if (u.n() > 0) {
          ++it;
          return true;
        }
      }
    };
    Unit u, v;
    bool have = next(u);
    float l = have ? lse_of(u) : 0.f;
    while (have && ok) {
      const bool more = next(v);
      const float l_next = more ? lse_of(v) : 0.f;
      const int st = n % C::kStages, f = n / C::kStages;
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
        if (f > 0) ok = wait_bar(empty(st), (uint32_t)((f - 1) & 1), abort, a.err);
        if (ok) {
          mbar_arrive_expect_tx(full(st), (uint32_t)(n_sub * a.sub * 128 * C::kNch + C::kQBytes));
          for (int ch = 0; ch < C::kNch; ++ch)
            tma_load_2d(base + st * C::kStage + C::kKBytes + ch * C::kQChunk, &tmq, full(st), ch * 64,
                        (u.b * a.h_q + u.g * a.r) * a.S_q);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      if (lane < n_sub) load_keys<C::kNch>(a, base + st * C::kStage, &tmk, full(st), lane, row);
      if (lane < C::kRows) {
        // a row without a finite lse (no visible key, padding) takes part in nothing
        const bool in = l != -INFINITY && l == l;
        nl2(st)[lane] = in ? -l * kLog2e : 0.f;
        cpos(st)[lane] = !in ? -1 : a.causal ? (int)min((long long)u.qs + i, (long long)kFar) : kFar;
      }
      mbar_arrive(full(st));
      ++n;
      u = v;
      l = l_next;
      have = more;
    }
    if (lane == 0) {  // drain (bounded): no copy may still land in shared memory at exit
      volatile int no_abort = 0;
#pragma unroll
      for (int s = 0; s < C::kStages; ++s)
        if (n > s) wait_bar(full(s), (uint32_t)(((n - 1 - s) / C::kStages) & 1), &no_abort, a.err);
    }
    return;
  }

  // ------------------------------ consumers: 16 keys of each tile per warp -------------------
  const int gid = lane >> 2, tq = lane & 3;
  const int reach = a.window > 0 ? a.window : 0x7fffffff;
  int n = 0;
  for (int it = 0;; ++it) {
    const long long idx = unit_of(it);
    if (idx >= a.n_units) break;
    const Unit u = make_unit<kBK, true>(a, seq, (int)idx);
    // lane gid = 2 j + e (below 4) of each quad column tq ends up with key 8 j + 2 tq + e of the warp's 16
    const int kq = u.k0 + warp * 16 + 2 * tq;  // keys kq, kq + 1, kq + 8, kq + 9
    const int key = kq + 8 * (gid >> 1) + (gid & 1);
    const bool writer = gid < 4 && key < a.T_max;
    const bool in = u.valid && key < u.kv;
    float* const dst = a.w + ((long long)u.b * a.h_kv + u.g) * a.T_max + key;
    if (u.n() == 0) {
      if (writer && !a.accumulate) *dst = 0.f;
      continue;
    }
    // the entry to be added to is loaded ahead of the sum
    const float old = writer && in && a.accumulate ? *dst : 0.f;
    const int st = n % C::kStages;
    // ldmatrix / mma.sync below need the whole warp: leave together if the wait ran out
    if (!__all_sync(0xffffffffu, wait_bar(full(st), (uint32_t)((n / C::kStages) & 1), abort, a.err))) return;
    const uint32_t kb = base + st * C::kStage, qb = kb + C::kKBytes;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};  // over this lane's rows, of keys kq, kq + 1, kq + 8, kq + 9
    if (u.k0 + warp * 16 < u.kv) {
      float sc[MT][2][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j) sc[m][j][0] = sc[m][j][1] = sc[m][j][2] = sc[m][j][3] = 0.f;
      const int krow = warp * 16 + ((lane >> 4) << 3) + (lane & 7);
      const int qi = lane >> 3;
      const int qrow = (qi & 1) * 8 + (lane & 7);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const int d8k = ks * 2 + ((lane >> 3) & 1), d8q = ks * 2 + (qi >> 1);
        uint32_t b0, b1, b2, b3;
        ldsm_x4(swz128(kb + (krow >> 3) * a.k_group + (d8k >> 3) * a.k_chunk, krow & 7, d8k & 7), b0, b1, b2, b3);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint32_t qf[4];
          ldsm_x4(swz128(qb + (d8q >> 3) * C::kQChunk, m * 16 + qrow, d8q & 7), qf[0], qf[1], qf[2], qf[3]);
          mma_bf16(sc[m][0], qf, b0, b1);
          mma_bf16(sc[m][1], qf, b2, b3);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int row = m * 16 + half * 8 + gid;
          const float nl = nl2(st)[row];
          const int at = cpos(st)[row];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = kq + 8 * (e >> 1) + (e & 1);
            // key <= position, and within the window: position - key < window
            const bool vis = k <= at && at - k < reach;
            sum[e] += vis ? fast_exp2(fmaf(sc[m][e >> 1][2 * half + (e & 1)], a.sl2, nl)) : 0.f;
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty(st));
    ++n;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 4);
      sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 8);
      sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 16);
    }
    const float total = gid == 0 ? sum[0] : gid == 1 ? sum[1] : gid == 2 ? sum[2] : sum[3];
    if (!writer) continue;
    if (!a.accumulate) *dst = in ? total : 0.f;
    else if (in) *dst = old + total;
  }
}

// The sums of the parts of each key, in their order.
__global__ void __launch_bounds__(256) kv_weights_join_kernel(const __grid_constant__ WArgs a) {
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
  const long long stride = (long long)a.B * a.h_kv * a.part_keys;
  const float* src = a.part + bg * a.part_keys + key;
  float sum = 0.f;
  for (int p = 0; p < a.parts; ++p) sum += __ldcg(src + p * stride);
  *dst = a.accumulate ? *dst + sum : sum;
}

// =============================================================================================
// fp32 check mode: 128 keys per block, kGroups threads to a key, each with kRows query rows at a time (8, 16 or 32
// rows and one group where those hold the KV head's rows; else 32 rows and 2 or 4 groups, which share the keys' loads
// and give the few blocks of a short cache enough warps). Keys come in 32 columns at a time, a warp to a row. Rows that see no
// key of the block are passed over 32 kGroups at a time.
// Measured: 64 heads, 35 rows over 845 keys, d = 96: 41 us; one row over 2000 keys, d = 128: 24 us (113 and 86 us
// with each thread reading its own key's elements, 16 rows at a time); 9 x 4 heads, 184 rows over 77 keys: 47 us
// (74 us with one group).
// =============================================================================================
constexpr int kF32Cols = 32;

template <int kRows, int kGroups>
__global__ void __launch_bounds__(kBK * kGroups) kv_weights_fp32_kernel(WArgs a, const float* q, const float* k, int D,
                                                                        float scale) {
  constexpr int kAll = kRows * kGroups;   // query rows under way
  constexpr int kPer = 32 / kGroups;      // rows of the key tile a warp loads
  constexpr int kFly = kPer < 16 ? kPer : 16;
  __shared__ float ks[kF32Cols][kBK + 1];
  __shared__ __align__(16) float qsm[kF32Cols][kAll];
  __shared__ long long s_row[kBK];  // this block's cache rows (-1: not a cached key)
  __shared__ float ls[kAll], part[kGroups][kBK];
  __shared__ int ps[kAll];
  __shared__ bool s_on[kGroups];  // the group's rows see any of the keys
  const int kt = blockIdx.x, g = blockIdx.y % a.h_kv, b = blockIdx.y / a.h_kv;
  const int t = threadIdx.x % kBK, grp = threadIdx.x / kBK;
  const int k0 = kt * kBK, key = k0 + t;
  const int kv = a.kv_len ? a.kv_len[b] : a.T_max;
  const int qs = a.q_start ? a.q_start[b] : kv - a.S_q;
  const bool valid = kv >= 1 && kv <= a.T_max && qs >= 0;
  if (!valid && kt == 0 && g == 0 && threadIdx.x == 0)
    set_device_error(a.err, kv < 1 || kv > a.T_max ? GQA_DEVERR_KV_LEN : GQA_DEVERR_POSITION);
  const long long bg = (long long)b * a.h_kv + g;
  const bool cached = valid && key < kv;
  if (grp == 0) {
    long long row = -1;
    if (cached) {
      row = bg * a.T_max + key;
      if (a.block_table) {
        int page = a.block_table[(long long)b * a.max_pages + key / a.page_size];
        if (page < 0 || page >= a.num_pages) {
          set_device_error(a.err, GQA_DEVERR_PAGE);
          page = 0;
        }
        row = ((long long)page * a.h_kv + g) * a.page_size + key % a.page_size;
      }
    }
    s_row[t] = row;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int reach = a.window > 0 ? a.window : 0x7fffffff;
  const int k_end = min(k0 + kBK, kv);
  float sum = 0.f, comp = 0.f;
  if (valid && k0 < kv) {
    const long long rows = (long long)a.r * a.S_q, q0 = ((long long)b * a.h_q + (long long)g * a.r) * a.S_q;
    for (long long r0 = 0; r0 < rows; r0 += kAll) {
      bool sees = false;
      __syncthreads();  // the rows before are done with
      if (threadIdx.x < kAll) {
        const long long rr = r0 + threadIdx.x;
        const float l = rr < rows ? a.lse[q0 + rr] : -INFINITY;
        const long long pos = (long long)qs + rr % a.S_q;
        const int at = l == -INFINITY || l != l ? -1 : a.causal ? (int)min(pos, (long long)kFar) : kFar;
        ls[threadIdx.x] = l;
        ps[threadIdx.x] = at;
        sees = at >= k0 && at - (k_end - 1) < reach;
        if constexpr (kGroups > 1) {  // 32 rows: a warp to a group
          const bool any = __any_sync(0xffffffffu, sees);
          if (lane == 0) s_on[warp] = any;
        }
      }
      if (!__syncthreads_or(sees)) continue;
      float acc[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) acc[i] = 0.f;
      for (int c0 = 0; c0 < D; c0 += kF32Cols) {
        if (c0 > 0) __syncthreads();
#pragma unroll 1
        for (int j0 = 0; j0 < kPer; j0 += kFly) {
          float x[kFly];
#pragma unroll
          for (int u = 0; u < kFly; ++u) {
            const long long at = s_row[4 * kGroups * (j0 + u) + warp];
            x[u] = at >= 0 && c0 + lane < D ? __ldg(k + at * D + c0 + lane) : 0.f;
          }
#pragma unroll
          for (int u = 0; u < kFly; ++u) ks[lane][4 * kGroups * (j0 + u) + warp] = x[u];
        }
        for (int e = threadIdx.x; e < kAll * kF32Cols; e += kBK * kGroups) {
          const int i = e / kF32Cols, c = e - i * kF32Cols;
          qsm[c][i] = r0 + i < rows && c0 + c < D ? __ldg(q + (q0 + r0 + i) * D + c0 + c) : 0.f;
        }
        __syncthreads();
        if (kGroups > 1 && !s_on[grp]) continue;
#pragma unroll 4
        for (int c = 0; c < kF32Cols; ++c) {
          const float kc = ks[c][t];
#pragma unroll
          for (int i = 0; i < kRows; ++i) acc[i] = fmaf(kc, qsm[c][grp * kRows + i], acc[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int at = ps[grp * kRows + i];
        if (key > at || at - key >= reach) continue;
        const float y = expf(fmaf(acc[i], scale, -ls[grp * kRows + i])) - comp, tot = sum + y;
        comp = (tot - sum) - y;
        sum = tot;
      }
    }
  }
  if constexpr (kGroups > 1) {  // the groups' sums, in their order
    part[grp][t] = sum;
    __syncthreads();
    if (grp > 0) return;
    for (int k_ = 1; k_ < kGroups; ++k_) sum += part[k_][t];
  }
  if (key >= a.T_max) return;
  float* dst = a.w + bg * a.T_max + key;
  if (!a.accumulate) *dst = cached ? sum : 0.f;
  else if (cached) *dst += sum;
}

// -------------------------------------------------------------------------------------------------
// host side
// -------------------------------------------------------------------------------------------------
// Tile geometry: P = min(S_q, 128) positions of as many heads as fit (small: all rows of the group).
struct Geometry {
  bool small, flat;
  int keys;  // of a unit
  int P, H, N, hblocks, npb, parts;
};
Geometry geometry(int B, int h_q, int h_kv, int S_q, int T_max, int num_sms) {
  Geometry m;
  const int r = h_q / h_kv;
  // every row of the group fits 32 columns: one small Q tile per unit, and more K tiles in flight
  m.small = (long long)S_q * r <= 32;
  m.P = S_q < 128 ? S_q : 128;
  m.H = m.small ? r : 128 / m.P;
  m.H = (r + (r + m.H - 1) / m.H - 1) / ((r + m.H - 1) / m.H);  // the same number in every block
  m.keys = m.small ? kBK : Cfg<64>::kKeys;
  m.N = (m.P * m.H + 15) / 16 * 16;
  m.hblocks = (r + m.H - 1) / m.H;
  m.flat = !m.small && S_q < 128;
  if (m.flat) m.hblocks = (int)(((long long)r * S_q + 127) / 128);
  m.npb = (S_q + m.P - 1) / m.P;
  m.parts = 1;
  const long long units = (long long)B * h_kv * ((T_max + m.keys - 1) / m.keys);
  const long long tiles = (long long)m.hblocks * m.npb;
  const long long want = ((long long)kUnitsPerSm * num_sms + units - 1) / units;
  const long long most = (tiles + kTilesPerPart - 1) / kTilesPerPart;
  if (!m.small && num_sms > 0) m.parts = (int)(want < most ? want : most);
  if (m.parts < 1) m.parts = 1;
  return m;
}

template <typename Kernel>
cudaError_t launch_kernel(Kernel kern, int threads, int smem, bool (&attr_set)[64], const WArgs& w,
                          const CUtensorMap* tm, int num_sms, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {  // per device: the shared-memory opt-in is set once
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  kern<<<w.n_units < num_sms ? w.n_units : num_sms, threads, smem, s>>>(tm[0], tm[1], w);
  e = cudaGetLastError();
  if (e != cudaSuccess || w.parts == 1) return e;
  kv_weights_join_kernel<<<dim3((w.T_max + 255) / 256, w.B * w.h_kv), 256, 0, s>>>(w);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch_tiles(const WArgs& w, const CUtensorMap* tm, int num_sms, cudaStream_t s) {
  static bool attr_set[64] = {false};
  return launch_kernel(kv_weights_kernel<D>, Cfg<D>::kThreads, Cfg<D>::kSmem, attr_set, w, tm, num_sms, s);
}
template <int D, int MT>
cudaError_t launch_small(const WArgs& w, const CUtensorMap* tm, int num_sms, cudaStream_t s) {
  static bool attr_set[64] = {false};
  using C = SCfg<D, MT>;
  return launch_kernel(kv_weights_small_kernel<D, MT>, C::kThreads, C::kSmem, attr_set, w, tm, num_sms, s);
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
  w.flat = m.flat ? 1 : 0;
  w.nkt = (a.T_max + m.keys - 1) / m.keys;
  w.part_keys = w.nkt * m.keys;
  w.parts = m.parts;
  w.n_units = (int)((long long)a.B * a.h_kv * w.nkt * m.parts);
  w.div_bg = FastDiv::make((uint32_t)(a.B * a.h_kv));
  w.div_nkt = FastDiv::make((uint32_t)w.nkt);
  w.div_parts = FastDiv::make((uint32_t)m.parts);
  w.div_hkv = FastDiv::make((uint32_t)a.h_kv);
  w.div_P = FastDiv::make((uint32_t)m.P);
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
  w.k_4d = kv_weights_4d(a.block_table != nullptr, a.d_h) ? 1 : 0;
  w.k_chunk = w.k_4d ? 1024 : kBK * 128;
  w.k_group = w.k_4d ? 2048 : 1024;
  w.err = a.err;
  return w;
}

}  // namespace kw

bool kv_weights_4d(bool paged, int d_h) { return paged && d_h == 128; }

int kv_weights_sub(bool paged, int page_size) { return !paged ? 128 : page_size % 64 == 0 ? 64 : 16; }

KvWeightsTile kv_weights_tile(int h_q, int h_kv, int S_q) {
  const kw::Geometry m = kw::geometry(1, h_q, h_kv, S_q, 1, 0);
  return {m.small, m.flat, m.P, m.H, S_q * (h_q / h_kv) > 16 ? 32 : 16};
}

size_t kv_weights_workspace_bytes(int B, int h_q, int h_kv, int S_q, int T_max, gqa_dtype dtype, int num_sms) {
  if (dtype == GQA_FP32) return 0;
  const kw::Geometry m = kw::geometry(B, h_q, h_kv, S_q, T_max, num_sms);
  if (m.parts == 1) return 0;
  return (size_t)m.parts * B * h_kv * ((T_max + m.keys - 1) / m.keys) * m.keys * sizeof(float);
}

cudaError_t launch_kv_weights_bf16(const KvWeightsArgs& a, const CUtensorMap* tmaps, int num_sms, cudaStream_t s) {
  const kw::Geometry m = kw::geometry(a.B, a.h_q, a.h_kv, a.S_q, a.T_max, num_sms);
  const kw::WArgs w = kw::make_args(a, m);
  // units and a unit's tile list times the parts are counted in 32 bits
  if ((long long)a.B * a.h_kv * w.nkt * m.parts >= (1ll << 31) || (long long)m.npb * m.hblocks * m.parts >= (1ll << 31))
    return cudaErrorInvalidConfiguration;
  const bool two = a.S_q * w.r > 16;  // m-tiles of the small kernel
  if (a.d_h == 128) {
    if (!m.small) return kw::launch_tiles<128>(w, tmaps, num_sms, s);
    return two ? kw::launch_small<128, 2>(w, tmaps, num_sms, s) : kw::launch_small<128, 1>(w, tmaps, num_sms, s);
  }
  if (a.d_h == 64) {
    if (!m.small) return kw::launch_tiles<64>(w, tmaps, num_sms, s);
    return two ? kw::launch_small<64, 2>(w, tmaps, num_sms, s) : kw::launch_small<64, 1>(w, tmaps, num_sms, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv_weights_fp32(const KvWeightsArgs& a, cudaStream_t s) {
  const kw::Geometry m = kw::geometry(a.B, a.h_q, a.h_kv, a.S_q, a.T_max, 0);
  const kw::WArgs w = kw::make_args(a, m);
  const long long bg = (long long)a.B * a.h_kv;
  if (bg > 65535) return cudaErrorInvalidConfiguration;
  const long long rows = (long long)(a.h_q / a.h_kv) * a.S_q;
  const int groups = rows <= 32 ? 1 : rows <= 64 ? 2 : 4;
  auto kern = rows <= 8    ? kw::kv_weights_fp32_kernel<8, 1>
              : rows <= 16 ? kw::kv_weights_fp32_kernel<16, 1>
              : rows <= 32 ? kw::kv_weights_fp32_kernel<32, 1>
              : rows <= 64 ? kw::kv_weights_fp32_kernel<32, 2>
                           : kw::kv_weights_fp32_kernel<32, 4>;
  kern<<<dim3((a.T_max + kw::kBK - 1) / kw::kBK, (unsigned)bg), kw::kBK * groups, 0, s>>>(
      w, reinterpret_cast<const float*>(a.q), reinterpret_cast<const float*>(a.k), a.d_h, a.scale);
  return cudaGetLastError();
}

}  // namespace gqa
