// Rotary position embedding, alone and fused with the append to the KV cache.
//
// Mathematics. Element pair i of a row at position p turns by the angle p f_i (f = inv_freq):
//   (x0, x1) -> (x0 c - x1 s, x0 s + x1 c),  c = scale cos(p f_i), s = +-scale sin(p f_i)
// (s negated: the transpose, which is the gradient). Half layout pairs elements i and i + d_rot / 2 of
// the rotated segment, interleaved layout 2i and 2i + 1; elements outside the segment are copied.
// The angle is formed in 64 bits and reduced to a fraction of a turn before it is rounded to fp32
// (p f_i reaches 10^6 radians in long contexts, where an fp32 product is off by 0.06); the rotation
// itself is fp32, rounded once to the output type.
//
// Bound: every row is read and written once, so DRAM at length and launch latency at one token. A block
// takes a few tokens and all (or some) of their heads: it computes each token's cos / sin once into
// shared memory, for all heads that share them, and then moves rows. A thread moves `slots`: the two
// vectors of up to 16 bytes that hold kVec pairs (half layout: kVec elements of either half; interleaved:
// 2 kVec elements in a row), or two vectors to be copied. With an append, q goes to its output, k rotated
// and v unchanged straight to their cache rows (contiguous or paged), so neither is written and read
// again in between.

#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace gqa {
namespace rp {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;            // slots whose loads are in flight together in one thread
constexpr int kMaxTableBytes = 32768;  // cos / sin of a block's tokens

template <int kBytes>
struct Raw;
template <>
struct Raw<16> { using T = uint4; };
template <>
struct Raw<8> { using T = uint2; };
template <>
struct Raw<4> { using T = uint32_t; };
template <>
struct Raw<2> { using T = uint16_t; };

template <typename T, int kVec>
union Vec {
  typename Raw<(int)sizeof(T) * kVec>::T raw;
  T e[kVec];
  __device__ Vec() {}
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& d, float x) { d = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

// Where one slot reads and writes: two vectors at element offsets e0 and e1 (< 0: none) of a row.
template <typename T>
struct Place {
  const T* src;
  T* dst;      // nullptr: the row is not written (flagged)
  int mode;    // 0 rotate, 1 copy, 2 zeros
  int tl;      // the token's row of the cos / sin table
};

template <typename T, int kVec, bool kInter>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs a, int tb, int hc, int slots) {
  // A decode launched as a programmatic dependent may start its prologue now (it waits for this
  // grid's completion before it reads anything).
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ float2 table[];  // [token][pair]: (c, s)
  const int half = a.d_rot >> 1;
  const int n_tok = a.B * a.S;  // below 2^31 (checked on the host), as is every tok below
  const int tok0 = blockIdx.x * tb;
  const int nt = n_tok - tok0 < tb ? n_tok - tok0 : tb;
  const int H = a.h + 2 * a.h_kv;  // rows per token: q heads, then k heads, then v heads
  const int head0 = blockIdx.y * hc;
  const int nh = H - head0 < hc ? H - head0 : hc;

  // position of a token: < 0 when invalid
  auto position = [&](int tok, int b, int t) -> long long {
    if (a.per_token) return a.positions[tok];
    const long long p = a.positions[b];
    return p < 0 ? p : p + t;
  };
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int tl = i / half, pr = i - tl * half;
    const int tok = tok0 + tl;
    const int b = tok / a.S;
    const long long p = position(tok, b, tok - b * a.S);
    double turn = (double)(p < 0 ? 0 : p) * a.inv_freq[pr] * 0.15915494309189533577;  // 1 / (2 pi)
    turn -= rint(turn);
    float s, c;
    sincospif(2.f * (float)turn, &s, &c);
    table[i] = make_float2(c * a.scale, a.inverse ? -s * a.scale : s * a.scale);
  }
  __syncthreads();

  const int per_row = kThreads / slots > 0 ? kThreads / slots : 1;  // rows a block covers at once
  const int step = slots <= kThreads ? per_row : 1;
  const int lane_slots = slots <= kThreads ? slots : kThreads;
  const int row_lane = threadIdx.x / lane_slots;
  if (row_lane >= step) return;
  const int rows = nt * nh;
  const int n_rot = half / kVec;             // rotated slots of a row
  const int n_keep = (a.d - a.d_rot) / kVec;  // copied vectors of a rotated row

  for (int slot = threadIdx.x - row_lane * lane_slots; slot < slots; slot += lane_slots) {
    // element offsets of the slot's two vectors, in a rotated row and in a copied one
    int e0, e1;
    const bool turn = slot < n_rot;
    if (turn) {
      e0 = a.offset + (kInter ? 2 * slot * kVec : slot * kVec);
      e1 = kInter ? e0 + kVec : e0 + half;
    } else {
      const int v0 = 2 * (slot - n_rot), v1 = v0 + 1;  // vectors outside the rotated segment
      e0 = v0 < n_keep ? v0 * kVec : -1;
      e1 = v1 < n_keep ? v1 * kVec : -1;
      if (e0 >= a.offset) e0 += a.d_rot;
      if (e1 >= a.offset) e1 += a.d_rot;
    }
    const int n_all = a.d / kVec;
    const int c0 = 2 * slot < n_all ? 2 * slot * kVec : -1;
    const int c1 = 2 * slot + 1 < n_all ? (2 * slot + 1) * kVec : -1;

    auto place = [&](int row) {
      Place<T> pl;
      const int tl = row / nh, head = head0 + (row - tl * nh);
      const int tok = tok0 + tl;
      const int b = tok / a.S, t = tok - b * a.S;
      const bool ok = position(tok, b, t) >= 0;
      pl.tl = tl;
      pl.mode = ok ? 0 : 2;
      if (!ok && head == 0 && slot == 0) set_device_error(a.err, GQA_DEVERR_POSITION);
      if (head < a.h) {
        pl.src = reinterpret_cast<const T*>(a.x) + b * a.xs[0] + head * a.xs[1] + t * a.xs[2];
        pl.dst = reinterpret_cast<T*>(a.out) + b * a.os[0] + head * a.os[1] + t * a.os[2];
        return pl;
      }
      const bool is_v = head >= a.h + a.h_kv;
      const int g = head - a.h - (is_v ? a.h_kv : 0);
      const long long* st = is_v ? a.vs : a.ks;
      pl.src = reinterpret_cast<const T*>(is_v ? a.v : a.k) + b * st[0] + g * st[1] + t * st[2];
      pl.dst = nullptr;
      if (is_v) pl.mode = 1;
      if (!ok) return pl;  // a token without a position is not cached
      const int p = a.pos[b];
      if (p < 0 || (long long)p + a.S > a.T_max) {
        if (slot == 0 && g == 0 && !is_v) set_device_error(a.err, GQA_DEVERR_POSITION);
        return pl;
      }
      long long row_at;
      if (a.block_table) {
        const int pt = p + t;
        const int page = a.block_table[(long long)b * a.max_pages + pt / a.page_size];
        if (page < 0 || page >= a.num_pages) {
          if (slot == 0) set_device_error(a.err, GQA_DEVERR_PAGE);
          return pl;
        }
        row_at = ((long long)page * a.h_kv + g) * a.page_size + pt % a.page_size;
      } else {
        row_at = ((long long)b * a.h_kv + g) * a.T_max + p + t;
      }
      pl.dst = reinterpret_cast<T*>(is_v ? a.v_cache : a.k_cache) + row_at * a.d;
      return pl;
    };

    for (int r0 = row_lane; r0 < rows; r0 += step * kUnroll) {
      Place<T> pl[kUnroll];
      Vec<T, kVec> x0[kUnroll], x1[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int row = r0 + u * step;
        pl[u].dst = nullptr;
        if (row >= rows) continue;
        pl[u] = place(row);
        if (!pl[u].dst || pl[u].mode == 2) continue;
        const int f0 = pl[u].mode == 1 ? c0 : e0, f1 = pl[u].mode == 1 ? c1 : e1;
        if (f0 >= 0) x0[u].raw = *reinterpret_cast<const decltype(x0[u].raw)*>(pl[u].src + f0);
        if (f1 >= 0) x1[u].raw = *reinterpret_cast<const decltype(x1[u].raw)*>(pl[u].src + f1);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (!pl[u].dst) continue;
        const int f0 = pl[u].mode == 1 ? c0 : e0, f1 = pl[u].mode == 1 ? c1 : e1;
        if (pl[u].mode == 2) {
#pragma unroll
          for (int k = 0; k < kVec; ++k) {
            from_f(x0[u].e[k], 0.f);
            from_f(x1[u].e[k], 0.f);
          }
        } else if (pl[u].mode == 0 && turn) {
          const float2* cs = table + pl[u].tl * half + slot * kVec;
#pragma unroll
          for (int k = 0; k < kVec; ++k) {
            const float2 w = cs[k];
            if constexpr (kInter) {
              // pair k: elements 2k and 2k + 1 of the two vectors laid end to end
              T& lo = 2 * k < kVec ? x0[u].e[(2 * k) % kVec] : x1[u].e[(2 * k) % kVec];
              T& hi = 2 * k + 1 < kVec ? x0[u].e[(2 * k + 1) % kVec] : x1[u].e[(2 * k + 1) % kVec];
              const float p = to_f(lo), q = to_f(hi);
              from_f(lo, p * w.x - q * w.y);
              from_f(hi, q * w.x + p * w.y);
            } else {
              const float p = to_f(x0[u].e[k]), q = to_f(x1[u].e[k]);
              from_f(x0[u].e[k], p * w.x - q * w.y);
              from_f(x1[u].e[k], q * w.x + p * w.y);
            }
          }
        }
        if (f0 >= 0) *reinterpret_cast<decltype(x0[u].raw)*>(pl[u].dst + f0) = x0[u].raw;
        if (f1 >= 0) *reinterpret_cast<decltype(x1[u].raw)*>(pl[u].dst + f1) = x1[u].raw;
      }
    }
  }
}

template <typename T, int kVec>
cudaError_t launch_typed(const RopeArgs& a, int num_sms, cudaStream_t s) {
  const int slots = a.d_rot / 2 / kVec + ((a.d - a.d_rot) / kVec + 1) / 2;
  const int lanes = slots < kThreads ? kThreads / slots : 1;
  const int H = a.h + 2 * a.h_kv;
  const long long n_tok = (long long)a.B * a.S, rows = n_tok * H;
  // rows per block: enough for kUnroll slots a thread twice over when there is work for every SM
  // several times, down to one slot a thread for a few tokens (latency)
  long long per_block = rows / ((long long)num_sms * 4);
  if (per_block > 2ll * kUnroll * lanes) per_block = 2ll * kUnroll * lanes;
  if (per_block < lanes) per_block = lanes;
  const int hc = (int)(per_block < H ? per_block : H);
  const int half = a.d_rot / 2;
  int tb = (int)(per_block / H);
  if (tb > kMaxTableBytes / (half * 8)) tb = kMaxTableBytes / (half * 8);
  if (tb < 1) tb = 1;
  const long long gx = (n_tok + tb - 1) / tb;
  const int gy = (H + hc - 1) / hc;
  if (gx > 0x7fffffffLL || gy > 65535) return cudaErrorInvalidConfiguration;
  const size_t smem = (size_t)tb * half * sizeof(float2);
  const dim3 grid((unsigned)gx, (unsigned)gy);
  if (a.interleaved) rope_kernel<T, kVec, true><<<grid, kThreads, smem, s>>>(a, tb, hc, slots);
  else rope_kernel<T, kVec, false><<<grid, kThreads, smem, s>>>(a, tb, hc, slots);
  return cudaGetLastError();
}

// The widest vector that divides every offset and stride the call uses.
int vector_elems(const RopeArgs& a, int elem_bytes) {
  int v = 16 / elem_bytes;
  long long mix = a.d | a.d_rot / 2 | a.offset;
  uintptr_t ptr = (uintptr_t)a.x | (uintptr_t)a.out;
  for (int i = 0; i < 3; ++i) mix |= a.xs[i] | a.os[i];
  if (a.h_kv > 0) {
    ptr |= (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.k_cache | (uintptr_t)a.v_cache;
    for (int i = 0; i < 3; ++i) mix |= a.ks[i] | a.vs[i];
  }
  while (v > 1 && (mix % v != 0 || ptr % ((uintptr_t)v * elem_bytes) != 0)) v >>= 1;
  return v;
}

}  // namespace rp

cudaError_t launch_rope(const RopeArgs& a, gqa_dtype dtype, int num_sms, cudaStream_t s) {
  if (dtype == GQA_FP32) {
    switch (rp::vector_elems(a, 4)) {
      case 4: return rp::launch_typed<float, 4>(a, num_sms, s);
      case 2: return rp::launch_typed<float, 2>(a, num_sms, s);
      default: return rp::launch_typed<float, 1>(a, num_sms, s);
    }
  }
  switch (rp::vector_elems(a, 2)) {
    case 8: return rp::launch_typed<__nv_bfloat16, 8>(a, num_sms, s);
    case 4: return rp::launch_typed<__nv_bfloat16, 4>(a, num_sms, s);
    case 2: return rp::launch_typed<__nv_bfloat16, 2>(a, num_sms, s);
    default: return rp::launch_typed<__nv_bfloat16, 1>(a, num_sms, s);
  }
}

}  // namespace gqa
