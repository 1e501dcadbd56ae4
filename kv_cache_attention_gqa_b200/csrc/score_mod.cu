// Host and device pieces shared by the attention kernels with modified scores: the kernel-side arguments
// and the launch in front of them (hulls of key ranges, row terms).

#include <float.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace gqa {

ModArgs mod_args(const ScoreMod& m, float scale) {
  ModArgs a;
  if (m.softcap > 0.f) {
    // within fp32 for every finite cap: cap log2 e overflows past 2.3e38 (2^100 is out of any score's reach), and
    // scale / cap under a cap far below one, where a score of zero times infinity would be no number
    const double cap = fmin(m.softcap, 0x1p100);
    a.k1 = (float)fmin(scale / cap, (double)FLT_MAX);
    a.cap2 = (float)(cap * 1.4426950408889634);
  }
  a.slopes = m.slopes;
  a.range = reinterpret_cast<const int2*>(m.range);
  return a;
}

namespace {

constexpr int kStartThreads = 256;

// The small work in front of a kernel with modified scores, in one launch (three took 10 us of a training step over
// short documents): the first blocks take a query row a thread, the others a hull a warp.
__global__ void __launch_bounds__(kStartThreads) row_start_kernel(const __grid_constant__ RowStart a, int row_blocks) {
  if (blockIdx.x == 0 && (int)threadIdx.x < a.n_tickets) a.tickets[threadIdx.x] = 0;
  if ((int)blockIdx.x < row_blocks) {
    const long long row = (long long)blockIdx.x * kStartThreads + threadIdx.x;
    if (row >= a.n_rows) return;
    const float l = a.lse[row];
    a.lse2[row] = l == -INFINITY || l != l ? INFINITY : l * 1.4426950408889634f;
    a.d[0][row] = a.d[1][row] = 0.f;
    return;
  }
  long long wid = ((long long)(blockIdx.x - row_blocks) * kStartThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const long long first = (long long)a.B * a.blocks[0];
  const int which = wid >= first;
  if (which) wid -= first;
  const int n_blocks = a.blocks[which];
  if (wid >= (long long)a.B * n_blocks) return;
  const int b = (int)(wid / n_blocks), blk = (int)(wid - (long long)b * n_blocks);
  const int i0 = blk * a.rows[which], i1 = min(a.S_q, i0 + a.rows[which]);
  int4 h = make_int4(0x7fffffff, 0, 0, 0x7fffffff);
  for (int i = i0 + lane; i < i1; i += 32) {
    const int2 r = a.range[(long long)b * a.S_q + i];
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
  if (lane == 0) a.hull[which][wid] = h;
}

}  // namespace

cudaError_t launch_row_start(const RowStart& a, cudaStream_t s) {
  const long long row_blocks = (a.n_rows + kStartThreads - 1) / kStartThreads;
  const long long warps = (long long)a.B * (a.blocks[0] + a.blocks[1]);
  const long long grid = row_blocks + (warps * 32 + kStartThreads - 1) / kStartThreads;
  row_start_kernel<<<(unsigned)(grid > 0 ? grid : 1), kStartThreads, 0, s>>>(a, (int)row_blocks);
  return cudaGetLastError();
}

}  // namespace gqa
