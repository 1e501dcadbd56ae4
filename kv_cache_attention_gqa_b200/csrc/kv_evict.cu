// Eviction from the KV cache by accumulated attention weight: of each (sequence, KV head)'s n cached keys
// the first `sink`, the last `recent` and the budget - sink - recent heaviest of the others are kept and
// moved to the front, in their order, in the caller's cache (in place) or into another.
//
// Two launches.
//   select  one CTA, or for long rows a cluster of them, per (sequence, KV head); each keeps its share of the keys.
//           The threshold weight is found by a radix selection over the weights' bits mapped to unsigned integers
//           of the same order: passes of 11, 11 and 10 bits, each a
//           histogram in shared memory and a scan of its counts (with 8 bits the first pass would be the
//           exponent alone, a handful of bins that every thread of a warp adds to in turn); the weights are
//           read from DRAM once and kept in shared memory while they fit. The blocks of a cluster read each
//           other's counts (distributed shared memory) and find the same threshold. Then one pass over the keys in
//           order writes the kept indices: everything above the threshold, and of the keys equal to it the
//           first ones. Bound by latency: a few thousand keys per block, a dozen dependent phases.
//   move    rows of K, V and the weights, bound by DRAM (kept rows once in, once out). Kept indices ascend, so
//           a row's source is at or behind its destination (kept[i] >= i): moving in order, batch by batch,
//           with every load of a batch before its first store, never overwrites a row still to be read, also
//           in place. Columns are independent, so a (sequence, head, tensor) is cut into column slices,
//           one CTA each, which need no order among them; a copy into another cache or other pages is cut along
//           the rows too. The next batch's loads are issued before the current batch's stores (its sources lie
//           behind the current destinations).
//
// Measured (B200, d = 128 bf16): 64 rows of 8192 keys to 2048: 39 us (select 13, move 26 for 134 MB); 32 rows of 3001 to
// 32768 keys to 4096, 16-key pages: 44 us (select 18, move 26); the moves cut along the rows into 4 blocks an SM (8:
// 39.5 / 46.7 us, 16: 40.1 / 49.1 us).

#include <cooperative_groups.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace gqa {
namespace ev {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelKeep = 48 * 1024;  // weights kept in shared memory (192 KiB)
constexpr int kMinShare = 4096;  // keys of a block of a cluster, at least
constexpr int kBins = 2048;  // 11 bits a pass: two bins a thread
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;  // vectors in flight per thread and batch
constexpr int kTable = 1024;    // rows whose addresses are worked out together

// Weights in the order of eviction: unsigned, larger = kept longer; NaN ranks lowest.
__device__ __forceinline__ uint32_t rank_bits(float w) {
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);  // -0 equals 0
  if (w != w) return 0u;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads, 1) kv_evict_select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint4 keep4[];  // ranks of the competing keys, when they fit (a whole number of fours)
  uint32_t* const keep = reinterpret_cast<uint32_t*>(keep4);
  __shared__ int hists[3][kBins];  // one per pass: the cluster reads a pass's counts while the next pass counts
  __shared__ int totals[2];        // this block's keys above the threshold, and equal to it
  __shared__ int warp_sum[kSelWarps], warp_gt[kSelWarps], warp_eq[kSelWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank_ = (int)cluster.block_rank();
  const int g = blockIdx.x / ranks % a.h_kv, b = blockIdx.x / ranks / a.h_kv;
  const long long bg = blockIdx.x / ranks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = a.kv_len ? a.kv_len[b] : a.T_max;
  const bool valid = n >= 0 && n <= a.T_max;
  int32_t* kept = a.kept + bg * a.budget;
  const int len = !valid ? 0 : n < a.budget ? n : a.budget;
  if (threadIdx.x == 0 && rank_ == 0) {
    if (!valid && g == 0) set_device_error(a.err, GQA_DEVERR_KV_LEN);
    if (g == 0) a.new_len[b] = valid ? len : n;
  }
  if (!valid || n <= a.budget) {  // everything stays (the whole cluster takes this way)
    for (int i = rank_ * kSelThreads + threadIdx.x; i < a.budget; i += ranks * kSelThreads) kept[i] = i < len ? i : -1;
    return;
  }
  const float* w = a.w + bg * a.T_max;
  // the keys that compete, [lo0, hi0), and this block's share of them, [lo, lo + m)
  const int lo0 = a.sink, hi0 = n - a.recent, share = ((hi0 - lo0 + ranks - 1) / ranks + 3) / 4 * 4;
  const int lo = min(hi0, lo0 + rank_ * share), m = min(hi0 - lo, share);
  const int need = a.budget - a.sink - a.recent;          // of which so many stay (fewer than compete)
  const bool fits = m <= kSelKeep;
  auto rank = [&](int i) { return fits ? keep[i] : rank_bits(__ldg(w + lo + i)); };
  if (fits) {
    constexpr int kU = 8;  // loads in flight per thread
    for (int i0 = threadIdx.x; i0 < m; i0 += kU * kSelThreads) {
      float x[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) x[u] = i0 + u * kSelThreads < m ? __ldg(w + lo + i0 + u * kSelThreads) : 0.f;
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (i0 + u * kSelThreads < m) keep[i0 + u * kSelThreads] = rank_bits(x[u]);
    }
  }
  if (rank_ == 0) {
    for (int i = threadIdx.x; i < a.sink; i += kSelThreads) kept[i] = i;
    for (int i = threadIdx.x; i < a.recent; i += kSelThreads) kept[a.budget - a.recent + i] = hi0 + i;
  }
  if (need == 0) return;

  // threshold: the need-th largest rank, 11, 11 and 10 bits at a time
  uint32_t prefix = 0;
  int left = need;  // how many of the keys that share the prefix stay
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, top = pass == 0 ? 32 : pass == 1 ? 21 : 10;
    int* const hist = hists[pass];
    for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t mask = (1u << (top - shift)) - 1u;
    // four neighbours a thread; where they share a bin (equal weights, above all zeros) they are added at once
    for (int i = 4 * threadIdx.x; i < m; i += 4 * kSelThreads) {
      uint32_t r[4];
      if (fits) {
        const uint4 q = keep4[i / 4];
        r[0] = q.x, r[1] = q.y, r[2] = q.z, r[3] = q.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = i + e < m ? rank(i + e) : 0u;
      }
      int bin[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool in = i + e < m && (pass == 0 || (r[e] >> top) == (prefix >> top));
        bin[e] = in ? (int)(r[e] >> shift & mask) : -1;
      }
      if (bin[0] == bin[1] && bin[0] == bin[2] && bin[0] == bin[3]) {
        if (bin[0] >= 0) atomicAdd(&hist[bin[0]], 4);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (bin[e] >= 0) atomicAdd(&hist[bin[e]], 1);
      }
    }
    if (ranks > 1) cluster.sync();
    else __syncthreads();
    // thread t holds bins 2047 - 2t and 2046 - 2t of all blocks; counts of the bins above them by a scan
    int c0 = 0, c1 = 0;
    for (int k = 0; k < ranks; ++k) {
      const int2 c = *reinterpret_cast<const int2*>((ranks > 1 ? cluster.map_shared_rank(hist, k) : hist) + kBins - 2 -
                                                    2 * threadIdx.x);
      c0 += c.y;
      c1 += c.x;
    }
    int above = c0 + c1;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, above, off);
      if (lane >= off) above += t;
    }
    if (lane == 31) warp_sum[warp] = above;
    __syncthreads();
    above += __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0) - c0 - c1;
    if (above < left && above + c0 + c1 >= left) {  // exactly one thread
      const bool second = above + c0 < left;
      s_prefix = prefix | (uint32_t)(kBins - 1 - 2 * (int)threadIdx.x - (second ? 1 : 0)) << shift;
      s_need = left - above - (second ? c0 : 0);
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_need;
  }

  // kept indices in order: ranks above the threshold, and the first `left` equal to it. A warp takes a
  // contiguous range; counts of the warps before it give its places.
  const int per = ((m + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int i0 = min(m, warp * per), i1 = min(m, i0 + per);
  int gt = 0, eq = 0;
  for (int i = i0; i < i1; i += 32) {
    const uint32_t r = i + lane < i1 ? rank(i + lane) : 0u;
    const bool in = i + lane < i1;
    gt += __popc(__ballot_sync(0xffffffffu, in && r > prefix));
    eq += __popc(__ballot_sync(0xffffffffu, in && r == prefix));
  }
  if (lane == 0) {
    warp_gt[warp] = gt;
    warp_eq[warp] = eq;
  }
  __syncthreads();
  int gt0 = 0, eq0 = 0;  // before this warp's range
  if (ranks > 1) {
    if (threadIdx.x == 0) {
      totals[0] = totals[1] = 0;
      for (int k = 0; k < kSelWarps; ++k) {
        totals[0] += warp_gt[k];
        totals[1] += warp_eq[k];
      }
    }
    cluster.sync();
    for (int k = 0; k < rank_; ++k) {
      const int* other = cluster.map_shared_rank(totals, k);
      gt0 += other[0];
      eq0 += other[1];
    }
    cluster.sync();  // no block leaves while its counts may be read
  }
  for (int k = 0; k < warp; ++k) {
    gt0 += warp_gt[k];
    eq0 += warp_eq[k];
  }
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1;
    const uint32_t r = in ? rank(i + lane) : 0u;
    const uint32_t bg_ = __ballot_sync(0xffffffffu, in && r > prefix);
    const uint32_t be = __ballot_sync(0xffffffffu, in && r == prefix);
    const uint32_t below = (1u << lane) - 1u;
    const int g_at = gt0 + __popc(bg_ & below), e_at = eq0 + __popc(be & below);
    if (in && (r > prefix || (r == prefix && e_at < left)))
      kept[a.sink + g_at + min(e_at, left)] = lo + i + lane;
    gt0 += __popc(bg_);
    eq0 += __popc(be);
  }
}

// Rows kept[i] -> i of one column slice of K or of V, or (the last job) the weights.
template <typename Vec>
__global__ void __launch_bounds__(kMoveThreads) kv_evict_move_kernel(const __grid_constant__ EvictArgs a, int vecs,
                                                                     int slice, int n_slices, int row_split) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the kept indices are written
  const long long bg = blockIdx.y;
  const int b = (int)(bg / a.h_kv), g = (int)(bg - (long long)b * a.h_kv);
  const int n = a.kv_len ? a.kv_len[b] : a.T_max;
  if (n < 0 || n > a.T_max) return;
  const int len = n < a.budget ? n : a.budget;
  const int32_t* kept = a.kept + bg * a.budget;
  const int job = blockIdx.x;
  if (job == 2 * n_slices * row_split) {
    // the weights: one float a row, and zero from the new length on, where appended keys will count from
    const float* src = a.w + bg * a.T_max;
    float* dst = a.w_out + bg * a.T_out;
    const bool stay = a.w_out == a.w && n <= a.budget;
    for (int base = 0; base < len && !stay; base += kMoveThreads) {
      const int i = base + threadIdx.x;
      const float x = i < len ? src[kept[i]] : 0.f;
      __syncthreads();
      if (i < len) dst[i] = x;
    }
    if (a.w_out == a.w) __syncthreads();
    for (int i = len + threadIdx.x; i < a.T_out; i += kMoveThreads) dst[i] = 0.f;
    return;
  }
  if (a.in_place && n <= a.budget) return;
  const int part = job % row_split, sl = (job / row_split) % n_slices, is_v = job / (row_split * n_slices);
  const Vec* src = reinterpret_cast<const Vec*>(is_v ? a.v : a.k);
  Vec* dst = reinterpret_cast<Vec*>(is_v ? a.v_out : a.k_out);
  const int c0 = sl * slice, nc = min(slice, vecs - c0);  // this slice's vectors of a row
  const int rows = kMoveThreads / slice;                  // rows a block moves at once
  const int rl = threadIdx.x / slice, c = threadIdx.x - rl * slice;
  const bool lane_ok = rl < rows && c < nc;
  // rows [r0, r1) of this block. A move in place (onto the same rows, or by a table that keeps any of the sequence's
  // own pages in its column) has an order: its first block takes all rows.
  bool ordered = a.in_place;
  if (!ordered && a.block_table) {
    const int32_t* from = a.block_table + (long long)b * a.max_pages;
    const int32_t* to = a.block_table_out + (long long)b * a.max_pages_out;
    bool same = false;
    for (int c_ = threadIdx.x; c_ < (len + a.page_size - 1) / a.page_size; c_ += kMoveThreads) same |= from[c_] == to[c_];
    ordered = __syncthreads_or(same) != 0;
  }
  const int per = ordered ? (part == 0 ? len : 0) : (len + row_split - 1) / row_split;
  const int r0 = ordered ? 0 : min(len, part * per), r1 = min(len, r0 + per);
  // Source and destination rows, a table of kTable at a time (dst < 0: not moved). Every thread of a row
  // working them out for itself, kept index, table entry and divisions, was the longer part of the kernel.
  __shared__ int s_src[2][kTable], s_dst[2][kTable];
  auto row_of = [&](const int32_t* table, int max_pages, int T, int at) -> int {
    if (!table) return (int)(bg * T + at);
    const int pg = at / a.page_size;
    const int page = table[(long long)b * max_pages + pg];
    if (page < 0 || page >= a.num_pages) {
      set_device_error(a.err, GQA_DEVERR_PAGE);
      return -1;
    }
    return (page * a.h_kv + g) * a.page_size + at - pg * a.page_size;
  };
  auto fill = [&](int t) {  // table t: rows r0 + t kTable ...
    for (int k = threadIdx.x; k < kTable; k += kMoveThreads) {
      const int i = r0 + t * kTable + k;
      int from = 0, to = -1;
      if (i < r1) {
        const int at = kept[i];
        if (!a.in_place || at != i) {
          from = row_of(a.block_table, a.max_pages, a.T_max, at);
          to = from < 0 ? -1 : row_of(a.block_table_out, a.max_pages_out, a.T_out, i);
        }
      }
      s_src[t & 1][k] = from;
      s_dst[t & 1][k] = to;
    }
  };
  const int batch = rows * kMoveUnroll;  // divides kTable
  const int per_table = kTable / batch, n_batches = (r1 - r0 + batch - 1) / batch;
  Vec cur[kMoveUnroll], nxt[kMoveUnroll];
  auto load = [&](int n_, Vec (&x)[kMoveUnroll]) {
    const int t = (n_ / per_table) & 1, k0 = n_ % per_table * batch + rl;
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u)
      if (lane_ok && s_dst[t][k0 + u * rows] >= 0) x[u] = src[(long long)s_src[t][k0 + u * rows] * vecs + c0 + c];
  };
  auto store = [&](int n_, const Vec (&x)[kMoveUnroll]) {
    const int t = (n_ / per_table) & 1, k0 = n_ % per_table * batch + rl;
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int to = s_dst[t][k0 + u * rows];
      if (lane_ok && to >= 0) dst[(long long)to * vecs + c0 + c] = x[u];
    }
  };
  if (n_batches == 0) return;
  fill(0);
  __syncthreads();
  load(0, cur);
  for (int i = 0; i < n_batches; ++i) {
    if (i + 1 < n_batches) {
      if ((i + 1) % per_table == 0) {
        // over the table before last, which its last stores have read: they lie behind a batch's barrier, unless a
        // batch fills a table (rows of one vector)
        if (per_table == 1) __syncthreads();
        fill((i + 1) / per_table);
        __syncthreads();
      }
      load(i + 1, nxt);
    }
    __syncthreads();  // every load of this batch (and the next) comes before its stores
    store(i, cur);
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) cur[u] = nxt[u];
  }
}

template <typename Vec>
cudaError_t launch_move(const EvictArgs& a, long long row_bytes, int num_sms, cudaStream_t s) {
  const int vecs = (int)(row_bytes / sizeof(Vec));
  const long long bg = (long long)a.B * a.h_kv;
  // Column slices (a power of two of vectors). A move in place has only these to share: 128 bytes where that gives
  // every SM two blocks, down to 32 (a DRAM sector) where not. A copy into another cache or other pages has no
  // order and is cut along the rows instead: whole rows up to 256 bytes.
  const bool ordered = a.in_place;
  int slice = (ordered ? 128 : 256) / (int)sizeof(Vec);
  const int least = 32 / (int)sizeof(Vec);
  auto slices = [&](int w) { return (vecs + w - 1) / w; };
  while (ordered && slice > least && bg * 2 * slices(slice) < 2ll * num_sms) slice /= 2;
  while (slice > 1 && slice / 2 >= vecs) slice /= 2;
  const int n_slices = slices(slice);
  int split = 1;
  if (!ordered) {
    const int rows = kMoveThreads / slice * kMoveUnroll;
    const int most = (a.budget + rows - 1) / rows;
    const long long want = (4ll * num_sms + bg * 2 * n_slices - 1) / (bg * 2 * n_slices);
    split = (int)(want < most ? want : most);
    if (split < 1) split = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * n_slices * split + 1), (unsigned)bg);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv_evict_move_kernel<Vec>, a, vecs, slice, n_slices, split);
  if (e != cudaSuccess) {  // a stream that does not take dependent launches
    (void)cudaGetLastError();
    cfg.numAttrs = 0;
    e = cudaLaunchKernelEx(&cfg, kv_evict_move_kernel<Vec>, a, vecs, slice, n_slices, split);
  }
  return e;
}

}  // namespace ev

cudaError_t launch_kv_evict(const EvictArgs& a, int d_h, int elem_bytes, int num_sms, cudaStream_t s) {
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(ev::kv_evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             ev::kSelKeep * 4);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  // Blocks per row: up to 8, each with kMinShare keys at least, while every block has an SM (one fills it; a
  // second wave costs more than the split gains). 32 rows of 3001 to 32768 keys: 1, 4, 8 blocks 30.7, 17.7, 35 us; 64
  // rows of 8192: 1, 2, 4 blocks 13.2, 13.2, 26 us.
  const long long bg = (long long)a.B * a.h_kv;
  int ranks = 1;
  while (ranks < 8 && a.T_max / (2 * ranks) >= ev::kMinShare && 2 * ranks * bg <= num_sms) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(bg * ranks));
  cfg.blockDim = dim3(ev::kSelThreads);
  const int share = (a.T_max + ranks - 1) / ranks;  // a block's ranks, a whole number of fours
  cfg.dynamicSmemBytes = (size_t)((share < ev::kSelKeep ? share : ev::kSelKeep) + 3) / 4 * 16;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, ev::kv_evict_select_kernel, a);
  if (e != cudaSuccess) return e;
  const long long row_bytes = (long long)d_h * elem_bytes;
  const uintptr_t all = (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.k_out | (uintptr_t)a.v_out;
  if (row_bytes % 16 == 0 && all % 16 == 0) return ev::launch_move<uint4>(a, row_bytes, num_sms, s);
  if (row_bytes % 4 == 0 && all % 4 == 0) return ev::launch_move<uint32_t>(a, row_bytes, num_sms, s);
  return ev::launch_move<uint16_t>(a, row_bytes, num_sms, s);
}

}  // namespace gqa
