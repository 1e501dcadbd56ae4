// Check mode of attention with modified scores (fp32 in and out, scalar FFMA): prefill and its backward, by tiles in
// shared memory. Same mathematics as the bf16 kernels: s = scale q.k, capped (c tanh(s / c)) and biased
// (-slope |p - j|), masked by position, window, length and the row's key range; online softmax; the backward
// recomputes P from the saved lse and multiplies dS by the cap's derivative 1 - tanh^2.
//
// 256 threads, 8 to a row of the stationary tile (16 rows x 16 threads for dkdv). A thread forms four scores from
// 16-byte loads of both operands' rows (16 FFMA per 5 loads) and owns NC float4 columns of its row's output, where
// NC = ceil(d / 32): the rows are padded with zeros to 32 NC columns and 4 more, which keeps 16-byte alignment and
// spreads the banks. Key (query) tiles that no pair of the stationary tile sees are skipped. Bound: shared-memory
// loads. Calls whose 32-row tiles leave SMs without a block are bound by latency (two warps a scheduler waiting for
// shared memory): they take tiles of 8 rows, and of 8 keys, with a warp to each. dq and dkdv need nothing of each
// other and are blocks of one launch. Measured (B200), 2 x 6 heads of 67 rows over 2 KV heads, d = 96: forward 18 us,
// backward 32 us (29, and 32 + 36 in two launches, with tiles of 32 rows and 16 keys); one warp per row with a shuffle
// reduction per key, the layout of the plain check-mode kernels, took 77 and 95 + 166 us.

#include <cooperative_groups.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace gqa {
namespace mf {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kRows = 32;  // rows of a query tile (8: small calls); keys of the key tiles it meets
constexpr int kKeys = 16;  // stationary keys of a dkdv block (8: small calls)
constexpr int kKvQ = 64;   // query rows of its tiles

struct FArgs {
  const float* q;
  const float* k;
  const float* v;
  const float* o;
  const float* d_o;
  const float* lse_in;
  const float* drow;
  float* out;  // o, or dq
  float* lse;
  float* dk;
  float* dv;
  const int32_t* q_start;
  const int32_t* kv_len;
  int B, h_q, h_kv, r, S_q, T_max, D;
  float scale, cap;
  int causal, window;
  const float* slopes;
  const int2* range;
  unsigned* err;
};

// keys [x, y) that row i of sequence b (at position pos) sees
__device__ __forceinline__ int2 row_keys(const FArgs& a, int b, int i, long long pos, int kv) {
  long long lo = 0, hi = kv;
  if (a.causal) {
    if (pos + 1 < hi) hi = pos + 1;
    if (a.window > 0 && pos - a.window + 1 > lo) lo = pos - a.window + 1;
  }
  if (a.range) {
    const int2 rg = a.range[(long long)b * a.S_q + i];
    if (rg.x > lo) lo = rg.x;
    if (rg.y < hi) hi = rg.y;
  }
  return lo < hi ? make_int2((int)lo, (int)hi) : make_int2(0, 0);
}

// rows [r0, r0 + N) of a (rows, D) matrix into shared memory, zeros outside [lo, hi) and past column D; eight loads in
// flight per thread (one at a time, this was most of the time of a small call)
template <int NC, int N>
__device__ __forceinline__ void load_rows(float* to, const float* from, int r0, int lo, int hi, int D) {
  constexpr int kW = 32 * NC, kStride = kW + 4, kIter = N * kW / kThreads;
  static_assert(N * kW % kThreads == 0, "whole rounds");
#pragma unroll 1
  for (int i0 = 0; i0 < kIter; i0 += 8) {
    float x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int e = threadIdx.x + (i0 + u) * kThreads, r = e / kW, c = e - r * kW, at = r0 + r;
      x[u] = i0 + u < kIter && at >= lo && at < hi && c < D ? __ldg(from + (long long)at * D + c) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int e = threadIdx.x + (i0 + u) * kThreads, r = e / kW, c = e - r * kW;
      if (i0 + u < kIter) to[r * kStride + c] = x[u];
    }
  }
}

// products of one row (x) with the N rows y, y + kStep rows, ...; four sums are under way whatever N is
template <int NC, int kStep, int N>
__device__ __forceinline__ void dots(const float* x, const float* y, float (&s)[N]) {
  constexpr int kStride = 32 * NC + 4, kSplit = 4 / N;
  static_assert(N * kSplit == 4, "1, 2 or 4 rows");
  float p[N][kSplit];
#pragma unroll
  for (int u = 0; u < N; ++u)
#pragma unroll
    for (int e = 0; e < kSplit; ++e) p[u][e] = 0.f;
#pragma unroll (N == 4 ? 4 : 8)
  for (int c = 0; c < 32 * NC; c += 4) {
    const float4 a = *reinterpret_cast<const float4*>(x + c);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const float4 b = *reinterpret_cast<const float4*>(y + u * kStep * kStride + c);
      p[u][0 % kSplit] = fmaf(a.x, b.x, p[u][0 % kSplit]);
      p[u][1 % kSplit] = fmaf(a.y, b.y, p[u][1 % kSplit]);
      p[u][2 % kSplit] = fmaf(a.z, b.z, p[u][2 % kSplit]);
      p[u][3 % kSplit] = fmaf(a.w, b.w, p[u][3 % kSplit]);
    }
  }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    s[u] = p[u][0];
#pragma unroll
    for (int e = 1; e < kSplit; ++e) s[u] += p[u][e];
  }
}

// acc += w * row, over this thread's float4 columns tx, tx + kLanes, ... of 8 NC
template <int NC, int kLanes>
__device__ __forceinline__ void axpy(float4* acc, float w, const float* row, int tx) {
#pragma unroll
  for (int n = 0; n < (8 * NC + kLanes - 1) / kLanes; ++n) {
    if (8 * NC % kLanes != 0 && tx + kLanes * n >= 8 * NC) continue;
    const float4 x = *reinterpret_cast<const float4*>(row + 4 * (tx + kLanes * n));
    acc[n].x = fmaf(w, x.x, acc[n].x);
    acc[n].y = fmaf(w, x.y, acc[n].y);
    acc[n].z = fmaf(w, x.z, acc[n].z);
    acc[n].w = fmaf(w, x.w, acc[n].w);
  }
}

template <int NC, int kLanes>
__device__ __forceinline__ void store_row(float* to, const float4* acc, float f, int tx, int D) {
#pragma unroll
  for (int n = 0; n < (8 * NC + kLanes - 1) / kLanes; ++n) {
    const int c = 4 * (tx + kLanes * n);
    const float x[4] = {acc[n].x, acc[n].y, acc[n].z, acc[n].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < D) to[c + e] = x[e] * f;
  }
}

// Query tiles: kR rows of one head. kGrad: the dq pass (lse, drow and dO given), else the forward.
template <int NC, bool kGrad, int kR>
__device__ __forceinline__ void rows_block(const FArgs& a, int block) {
  constexpr int kStride = 32 * NC + 4;
  constexpr int kLanes = kThreads / kR, kS = kRows / kLanes;  // threads of a row, scores of a thread
  constexpr int kN = (8 * NC + kLanes - 1) / kLanes;          // float4 columns of a thread
  extern __shared__ float4 smem4[];
  float* sq = reinterpret_cast<float*>(smem4);
  float* sk = sq + kR * kStride;
  float* sv = sk + kRows * kStride;
  float* sdo = sv + kRows * kStride;             // kGrad
  float* sp = sdo + (kGrad ? kR * kStride : 0);  // weights of the tile: [row][key]
  __shared__ int s_lo, s_hi;
  const int n_tiles = (a.S_q + kR - 1) / kR;
  const int tile = n_tiles - 1 - block % n_tiles, bh = block / n_tiles;  // late rows first
  const int b = bh / a.h_q, head = bh - b * a.h_q, g = head / a.r;
  const int ty = threadIdx.x / kLanes, tx = threadIdx.x % kLanes;
  const int i = tile * kR + ty;
  const int kv = a.kv_len ? a.kv_len[b] : a.T_max;
  const int qs = a.q_start ? a.q_start[b] : 0;
  const bool valid = kv >= 1 && kv <= a.T_max && qs >= 0;
  if (!valid && threadIdx.x == 0 && tile == 0 && head == 0)
    set_device_error(a.err, kv < 1 || kv > a.T_max ? GQA_DEVERR_KV_LEN : GQA_DEVERR_POSITION);
  const long long row = (long long)bh * a.S_q + i;
  const bool live = valid && i < a.S_q;
  const long long pos = (long long)qs + i;
  int2 see = live ? row_keys(a, b, i, pos, kv) : make_int2(0, 0);
  float lse = 0.f, dr = 0.f;
  if (kGrad && live) {
    lse = a.lse_in[row];
    dr = a.drow[row];
    if (!(lse > -INFINITY)) see = make_int2(0, 0);
  }
  if (threadIdx.x == 0) {
    s_lo = 0x7fffffff;
    s_hi = 0;
  }
  __syncthreads();
  if (tx == 0 && see.x < see.y) {
    atomicMin(&s_lo, see.x);
    atomicMax(&s_hi, see.y);
  }
  const float* qp = a.q + (long long)bh * a.S_q * a.D;
  load_rows<NC, kR>(sq, qp, tile * kR, 0, a.S_q, a.D);
  if (kGrad) load_rows<NC, kR>(sdo, a.d_o + (long long)bh * a.S_q * a.D, tile * kR, 0, a.S_q, a.D);
  __syncthreads();
  const int lo = s_lo, hi = s_hi;
  const float slope = a.slopes ? a.slopes[head] : 0.f;
  const long long kvb = ((long long)b * a.h_kv + g) * a.T_max * a.D;
  float4 acc[kN];
#pragma unroll
  for (int n = 0; n < kN; ++n) acc[n] = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  for (int k0 = lo / kRows * kRows; k0 < hi; k0 += kRows) {
    if (!__syncthreads_or(see.x < k0 + kRows && see.y > k0)) continue;  // (also: the last tile's readers are done)
    load_rows<NC, kRows>(sk, a.k + kvb, k0, lo, hi, a.D);
    load_rows<NC, kRows>(sv, a.v + kvb, k0, lo, hi, a.D);
    __syncthreads();
    float s[kS], t[kS], w[kS];
    dots<NC, kLanes, kS>(sq + ty * kStride, sk + tx * kStride, s);
#pragma unroll
    for (int u = 0; u < kS; ++u) {
      const int key = k0 + tx + kLanes * u;
      s[u] = mod_score(s[u], a.scale, a.cap, slope, pos - key, &t[u]);
      if (key < see.x || key >= see.y) s[u] = -INFINITY;
    }
    if constexpr (kGrad) {
      float dp[kS];
      dots<NC, kLanes, kS>(sdo + ty * kStride, sv + tx * kStride, dp);
#pragma unroll
      for (int u = 0; u < kS; ++u)
        w[u] = s[u] == -INFINITY ? 0.f : expf(s[u] - lse) * (dp[u] - dr) * (1.f - t[u] * t[u]);
    } else {
      float mx = s[0];
#pragma unroll
      for (int u = 1; u < kS; ++u) mx = fmaxf(mx, s[u]);
#pragma unroll
      for (int off = 1; off < kLanes; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float mn = fmaxf(m, mx);
      const float f = m == -INFINITY ? 0.f : expf(m - mn);
      float sum = 0.f;
#pragma unroll
      for (int u = 0; u < kS; ++u) {
        w[u] = s[u] == -INFINITY ? 0.f : expf(s[u] - mn);
        sum += w[u];
      }
#pragma unroll
      for (int off = 1; off < kLanes; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      l = fmaf(l, f, sum);
      m = mn;
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        acc[n].x *= f;
        acc[n].y *= f;
        acc[n].z *= f;
        acc[n].w *= f;
      }
    }
#pragma unroll
    for (int u = 0; u < kS; ++u) sp[ty * kRows + tx + kLanes * u] = w[u];
    __syncwarp();  // a row's threads share a warp
    const float* from = kGrad ? sk : sv;
#pragma unroll 4
    for (int j = 0; j < kRows; ++j) {
      const float x = sp[ty * kRows + j];
      if (x != 0.f) axpy<NC, kLanes>(acc, x, from + j * kStride, tx);  // rows with no weight may hold anything
    }
  }
  if (i >= a.S_q) return;
  if (!kGrad) {
    if (valid && l == 0.f && tx == 0 && !a.range) set_device_error(a.err, GQA_DEVERR_NO_VISIBLE);
    if (a.lse && tx == 0) a.lse[row] = l > 0.f ? m + logf(l) : -INFINITY;
  }
  store_row<NC, kLanes>(a.out + row * a.D, acc, kGrad ? a.scale : l > 0.f ? 1.f / l : 0.f, tx, a.D);
}

template <int NC, int kR>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ FArgs a) {
  rows_block<NC, false, kR>(a, blockIdx.x);
}

// Key tiles: kK keys of one (sequence, KV head), all rows of all its heads that see them. The (head, 64 rows) tiles are
// shared by the blocks of a cluster, whose sums meet through distributed shared memory in the order of their ranks.
template <int NC, int kK>
__device__ __forceinline__ void keys_block(const FArgs& a) {
  constexpr int kStride = 32 * NC + 4;
  constexpr int kLanes = kThreads / kK, kS = kKvQ / kLanes;  // threads of a key, scores of a thread
  extern __shared__ float4 smem4[];
  float* sk = reinterpret_cast<float*>(smem4);
  float* sv = sk + kK * kStride;
  float* sq = sv + kK * kStride;
  float* sdo = sq + kKvQ * kStride;
  float* sp = sdo + kKvQ * kStride;  // [key][row]: P, then dS
  float* sds = sp + kK * kKvQ;
  __shared__ int2 s_see[kKvQ];
  __shared__ float s_lse[kKvQ], s_dr[kKvQ];
  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int n_tiles = (a.T_max + kK - 1) / kK;
  const int tile = blockIdx.x / ranks % n_tiles, bg = blockIdx.x / ranks / n_tiles;
  const int b = bg / a.h_kv, g = bg - b * a.h_kv;
  const int ty = threadIdx.x / kLanes, tx = threadIdx.x % kLanes;
  const int k0 = tile * kK, key = k0 + ty;
  const int kv = a.kv_len ? a.kv_len[b] : a.T_max;
  const int qs = a.q_start ? a.q_start[b] : 0;
  const bool valid = kv >= 1 && kv <= a.T_max && qs >= 0;
  constexpr int kN = (8 * NC + kLanes - 1) / kLanes;  // float4 columns of a thread
  float4 ak[kN], av[kN];
#pragma unroll
  for (int n = 0; n < kN; ++n) ak[n] = av[n] = make_float4(0.f, 0.f, 0.f, 0.f);
  const long long kvb = (long long)bg * a.T_max * a.D;
  if (valid && k0 < kv) {
    load_rows<NC, kK>(sk, a.k + kvb, k0, 0, kv, a.D);
    load_rows<NC, kK>(sv, a.v + kvb, k0, 0, kv, a.D);
    const int nq = (a.S_q + kKvQ - 1) / kKvQ;
    for (long long it = rank; it < (long long)a.r * nq; it += ranks) {
      const int head = g * a.r + (int)(it / nq), i0 = (int)(it % nq) * kKvQ;
      const long long base = ((long long)b * a.h_q + head) * a.S_q;
      const float slope = a.slopes ? a.slopes[head] : 0.f;
      __syncthreads();  // the last tile's readers are done
      bool any = false;
      if (threadIdx.x < kKvQ) {
        const int i = i0 + threadIdx.x;
        int2 see = i < a.S_q ? row_keys(a, b, i, (long long)qs + i, kv) : make_int2(0, 0);
        const float l = i < a.S_q ? a.lse_in[base + i] : -INFINITY;
        if (!(l > -INFINITY)) see = make_int2(0, 0);
        any = see.x < k0 + kK && see.y > k0;
        s_see[threadIdx.x] = see;
        s_lse[threadIdx.x] = l;
        s_dr[threadIdx.x] = i < a.S_q ? a.drow[base + i] : 0.f;
      }
      if (!__syncthreads_or(any)) continue;
      load_rows<NC, kKvQ>(sq, a.q + base * a.D, i0, 0, a.S_q, a.D);
      load_rows<NC, kKvQ>(sdo, a.d_o + base * a.D, i0, 0, a.S_q, a.D);
      __syncthreads();
      float s[kS], dp[kS];
      dots<NC, kLanes, kS>(sk + ty * kStride, sq + tx * kStride, s);
      dots<NC, kLanes, kS>(sv + ty * kStride, sdo + tx * kStride, dp);
#pragma unroll
      for (int u = 0; u < kS; ++u) {
        const int x = tx + kLanes * u;
        const int2 see = s_see[x];
        float t;
        const float z = mod_score(s[u], a.scale, a.cap, slope, (long long)qs + i0 + x - key, &t);
        const float p = key >= see.x && key < see.y ? expf(z - s_lse[x]) : 0.f;
        sp[ty * kKvQ + x] = p;
        sds[ty * kKvQ + x] = p == 0.f ? 0.f : p * (dp[u] - s_dr[x]) * (1.f - t * t);
      }
      __syncwarp();  // a key's threads share a warp
#pragma unroll 4
      for (int x = 0; x < kKvQ; ++x) {
        const float p = sp[ty * kKvQ + x], ds = sds[ty * kKvQ + x];
        if (p == 0.f && ds == 0.f) continue;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          const int c = 4 * (tx + kLanes * n);
          if (kN * kLanes > 8 * NC && c >= 32 * NC) continue;
          const float4 d = *reinterpret_cast<const float4*>(sdo + x * kStride + c);
          const float4 q = *reinterpret_cast<const float4*>(sq + x * kStride + c);
          av[n].x = fmaf(p, d.x, av[n].x);
          av[n].y = fmaf(p, d.y, av[n].y);
          av[n].z = fmaf(p, d.z, av[n].z);
          av[n].w = fmaf(p, d.w, av[n].w);
          ak[n].x = fmaf(ds, q.x, ak[n].x);
          ak[n].y = fmaf(ds, q.y, ak[n].y);
          ak[n].z = fmaf(ds, q.z, ak[n].z);
          ak[n].w = fmaf(ds, q.w, ak[n].w);
        }
      }
    }
  }
  // every block's sums into its own shared memory, then each block adds up its share of the keys
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem4);  // [dK, dV][key][column]
  constexpr int kW = 32 * NC;
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    const int c = 4 * (tx + kLanes * n);
    if (kN * kLanes > 8 * NC && c >= kW) continue;
    *reinterpret_cast<float4*>(part + ty * kW + c) = ak[n];
    *reinterpret_cast<float4*>(part + (kK + ty) * kW + c) = av[n];
  }
  cluster.sync();
  for (int e = rank * kThreads + threadIdx.x; e < 2 * kK * kW; e += ranks * kThreads) {
    const int y = e / kW, c = e - y * kW, is_v = y / kK, j = k0 + y - is_v * kK;
    if (c >= a.D || j >= a.T_max) continue;
    float sum = 0.f;
    for (int k = 0; k < ranks; ++k) sum += cluster.map_shared_rank(part, k)[e];
    (is_v ? a.dv : a.dk)[kvb + (long long)j * a.D + c] = valid && j < kv ? (is_v ? sum : sum * a.scale) : 0.f;
  }
  cluster.sync();  // no block leaves while its sums may be read
}

// The first key_blocks blocks (whole clusters) take key tiles, the others query tiles.
template <int NC, int kR, int kK>
__global__ void __launch_bounds__(kThreads) backward_kernel(const __grid_constant__ FArgs a, int key_blocks,
                                                            int row_blocks) {
  if ((int)blockIdx.x < key_blocks) {
    keys_block<NC, kK>(a);
  } else if ((int)blockIdx.x - key_blocks < row_blocks) {
    rows_block<NC, true, kR>(a, blockIdx.x - key_blocks);
  }
}

// D = rowsum(dO * O), one warp per row
__global__ void __launch_bounds__(kThreads) rowsum_kernel(const __grid_constant__ FArgs a, float* drow) {
  const long long row = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (row >= (long long)a.B * a.h_q * a.S_q) return;
  float s = 0.f;
  for (int c = lane; c < a.D; c += 32) s = fmaf(a.o[row * a.D + c], a.d_o[row * a.D + c], s);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (lane == 0) drow[row] = s;
}

template <typename Kernel, typename... Args>
cudaError_t launch(Kernel kern, long long blocks, size_t smem, cudaStream_t s, int ranks, const Args&... args) {
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  // the opt-in is set on every call: a check-mode call is no hot path
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// query tiles of `rows` rows
long long row_tiles(const FArgs& f, int rows) { return (long long)f.B * f.h_q * ((f.S_q + rows - 1) / rows); }

template <int NC, int kR>
cudaError_t forward(const FArgs& f, cudaStream_t s) {
  const size_t smem = ((kR + 2 * kRows) * (32 * NC + 4) + kR * kRows) * sizeof(float);
  return launch(rows_kernel<NC, kR>, row_tiles(f, kR), smem, s, 1, f);
}
template <int NC, int kR, int kK>
cudaError_t backward(const FArgs& f, int num_sms, cudaStream_t s) {
  const size_t row_smem = ((2 * kR + 2 * kRows) * (32 * NC + 4) + kR * kRows) * sizeof(float);
  const size_t key_smem = (2 * (kK + kKvQ) * (32 * NC + 4) + 2 * kK * kKvQ) * sizeof(float);
  // blocks of a cluster: up to 8, while there are tiles for them and SMs without a block
  const long long tiles = (long long)f.B * f.h_kv * ((f.T_max + kK - 1) / kK);
  const long long its = (long long)f.r * ((f.S_q + kKvQ - 1) / kKvQ);
  int ranks = 1;
  while (ranks < 8 && 2 * ranks <= its && 2 * ranks * tiles <= 2 * num_sms) ranks *= 2;
  const long long keys = tiles * ranks, rows = row_tiles(f, kR), blocks = keys + (rows + ranks - 1) / ranks * ranks;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch(backward_kernel<NC, kR, kK>, blocks, row_smem > key_smem ? row_smem : key_smem, s, ranks, f,
                (int)keys, (int)rows);
}

template <typename F>
cudaError_t by_width(int D, F&& f) {
  switch ((D + 31) / 32) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 5:
    case 6: return f(std::integral_constant<int, 6>());
    default: return f(std::integral_constant<int, 8>());
  }
}

}  // namespace mf

cudaError_t launch_prefill_fp32_mod(const PrefillArgs& a, int num_sms, cudaStream_t s) {
  mf::FArgs f = {};
  f.q = reinterpret_cast<const float*>(a.q);
  f.k = reinterpret_cast<const float*>(a.k);
  f.v = reinterpret_cast<const float*>(a.v);
  f.out = reinterpret_cast<float*>(a.o);
  f.lse = a.lse;
  f.q_start = a.q_start;
  f.kv_len = a.kv_len;
  f.B = a.B;
  f.h_q = a.h_q;
  f.h_kv = a.h_kv;
  f.r = a.h_q / a.h_kv;
  f.S_q = a.S_q;
  f.T_max = a.T_max;
  f.D = a.d_h;
  f.scale = a.scale;
  f.cap = a.mod.softcap;
  f.causal = a.causal;
  f.window = a.window;
  f.slopes = a.mod.slopes;
  f.range = reinterpret_cast<const int2*>(a.mod.range);
  f.err = a.err;
  const bool small = mf::row_tiles(f, mf::kRows) < num_sms;
  return mf::by_width(a.d_h, [&](auto nc) {
    return small ? mf::forward<decltype(nc)::value, 8>(f, s) : mf::forward<decltype(nc)::value, mf::kRows>(f, s);
  });
}

cudaError_t launch_backward_fp32_mod(const BackwardArgs& a, int num_sms, cudaStream_t s) {
  mf::FArgs f = {};
  f.q = reinterpret_cast<const float*>(a.q);
  f.k = reinterpret_cast<const float*>(a.k);
  f.v = reinterpret_cast<const float*>(a.v);
  f.o = reinterpret_cast<const float*>(a.o);
  f.d_o = reinterpret_cast<const float*>(a.d_o);
  f.lse_in = a.lse;
  f.drow = a.drow;
  f.out = reinterpret_cast<float*>(a.dq);
  f.dk = reinterpret_cast<float*>(a.dk);
  f.dv = reinterpret_cast<float*>(a.dv);
  f.q_start = a.q_start;
  f.kv_len = a.kv_len;
  f.B = a.B;
  f.h_q = a.h_q;
  f.h_kv = a.h_kv;
  f.r = a.h_q / a.h_kv;
  f.S_q = a.S_q;
  f.T_max = a.T_max;
  f.D = a.d_h;
  f.scale = a.scale;
  f.cap = a.mod.softcap;
  f.causal = a.causal;
  f.window = a.window;
  f.slopes = a.mod.slopes;
  f.range = reinterpret_cast<const int2*>(a.mod.range);
  f.err = a.err;
  const long long rows = (long long)a.B * a.h_q * a.S_q;
  if ((rows * 32 + mf::kThreads - 1) / mf::kThreads > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  mf::rowsum_kernel<<<(unsigned)((rows * 32 + mf::kThreads - 1) / mf::kThreads), mf::kThreads, 0, s>>>(f, a.drow);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const bool small = mf::row_tiles(f, mf::kRows) < num_sms;
  return mf::by_width(a.d_h, [&](auto nc) {
    return small ? mf::backward<decltype(nc)::value, 8, 8>(f, num_sms, s)
                 : mf::backward<decltype(nc)::value, mf::kRows, mf::kKeys>(f, num_sms, s);
  });
}

}  // namespace gqa
