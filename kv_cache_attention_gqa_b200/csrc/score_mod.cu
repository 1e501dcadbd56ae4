// Host and device pieces shared by the attention kernels with modified scores: the kernel-side arguments
// and the hulls of key ranges.

#include "common.cuh"
#include "internal.h"

namespace gqa {

ModArgs mod_args(const ScoreMod& m, float scale) {
  ModArgs a;
  if (m.softcap > 0.f) {
    a.k1 = (float)((double)scale / m.softcap);
    a.cap2 = (float)((double)m.softcap * 1.4426950408889634);
  }
  a.slopes = m.slopes;
  a.range = reinterpret_cast<const int2*>(m.range);
  return a;
}

namespace {

// One warp per block of `rows` query rows of one sequence. x, y: the least lo and the largest hi of the rows
// that see any key (y = 0: none does); z, w: the largest lo and the least hi of all of them, so that keys
// z <= j < w are in every row's range (a row without a key makes that empty). Resets the ticket counter of the kernel
// that follows, where it has one.
__global__ void __launch_bounds__(256) row_hull_kernel(const int2* range, int4* hull, int B, int S_q, int rows,
                                                       int n_blocks, int* ticket) {
  if (ticket && blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;
  const long long wid = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (wid >= (long long)B * n_blocks) return;
  const int b = (int)(wid / n_blocks), blk = (int)(wid - (long long)b * n_blocks);
  const int i0 = blk * rows, i1 = min(S_q, i0 + rows);
  int4 h = make_int4(0x7fffffff, 0, 0, 0x7fffffff);
  for (int i = i0 + lane; i < i1; i += 32) {
    const int2 r = range[(long long)b * S_q + i];
    const int lo = max(r.x, 0);
    if (lo < r.y) {
      h.x = min(h.x, lo);
      h.y = max(h.y, r.y);
      h.z = max(h.z, lo);
      h.w = min(h.w, r.y);
    } else {
      h.w = 0;
    }
  }
  h.x = __reduce_min_sync(0xffffffffu, h.x);
  h.y = __reduce_max_sync(0xffffffffu, h.y);
  h.z = __reduce_max_sync(0xffffffffu, h.z);
  h.w = __reduce_min_sync(0xffffffffu, h.w);
  if (lane == 0) hull[wid] = h;
}

}  // namespace

cudaError_t launch_row_hull(const int32_t* range, void* hull, int B, int S_q, int rows, int n_blocks,
                            int* ticket, cudaStream_t s) {
  const long long warps = (long long)B * n_blocks;
  row_hull_kernel<<<(unsigned)((warps + 7) / 8), 256, 0, s>>>(reinterpret_cast<const int2*>(range),
                                                              reinterpret_cast<int4*>(hull), B, S_q, rows, n_blocks,
                                                              ticket);
  return cudaGetLastError();
}

}  // namespace gqa
