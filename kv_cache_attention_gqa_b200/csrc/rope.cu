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
// again in between. The first rows' loads are issued before the angles are worked out.
//
// Measured (B200): gradient of 32 heads of 2 x 8192 tokens, d = 128, 268 MB: 50.0 us, 5.4 TB/s (0.82 of
// the measured copy rate); one launch for a 512-token chunk of four sequences, 48 heads, paged: 12.2 us;
// one token of eight sequences: 2.7 us. Two rows in flight per thread at 64 registers, four blocks an SM,
// beat four rows at 80 registers (50.9 / 18.0 us) and one row at 40 (48.6 / 17.4 us); eight rows a thread
// beat four (50.8 / 13.1) and two (54.3 / 14.5).

#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace gqa {
namespace rp {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;             // rows whose loads are in flight together in one thread
constexpr int kBlocksPerSm = 4;        // resident blocks the register budget allows (64 a thread)
constexpr int kRowsPerLane = 8;        // rows a thread moves when there is work for every SM
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

template <typename T, int kVec, bool kInter, bool kAppend>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    rope_kernel(const __grid_constant__ RopeArgs a, int tl_n, int hl_n, int hc, int slots) {
  // A decode launched as a programmatic dependent may start its prologue now (it waits for this
  // grid's completion before it reads anything).
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ float2 table[];  // [token][pair]: (c, s)
  using Raw_t = typename Raw<(int)sizeof(T) * kVec>::T;
  const int half = a.d_rot >> 1;
  const int n_tok = a.B * a.S;  // below 2^31 (checked on the host)
  const int tok0 = blockIdx.x * tl_n;
  const int nt = min(tl_n, n_tok - tok0);
  // position of a token: < 0 when invalid
  auto position = [&](int tok, int b, int t) -> long long {
    if (a.per_token) return a.positions[tok];
    const long long p = a.positions[b];
    return p < 0 ? p : p + t;
  };

  // this thread's slot, token and first head
  const int width = min(slots, kThreads);  // threads of one row
  const int lane = threadIdx.x / width;
  const int slot = blockIdx.z * kThreads + threadIdx.x - lane * width;
  const int tl = lane / hl_n;
  const bool active = slot < slots && tl < nt;
  const int tok = tok0 + (active ? tl : 0), b = tok / a.S, t = tok - b * a.S;
  const bool ok = position(tok, b, t) >= 0;
  const int H = kAppend ? a.h + 2 * a.h_kv : a.h;  // rows per token: q heads, then k heads, then v heads
  const int head0 = blockIdx.y * hc, head1 = active ? min(H, head0 + hc) : 0;
  const int n_rot = half / kVec;  // rotated slots of a row
  const bool turns = slot < n_rot;
  // element offsets of the slot's two vectors (< 0: none), in a rotated row and in a copied one
  int e0, e1;
  if (turns) {
    e0 = a.offset + (kInter ? 2 * slot * kVec : slot * kVec);
    e1 = kInter ? e0 + kVec : e0 + half;
  } else {
    const int n_keep = (a.d - a.d_rot) / kVec;  // vectors outside the rotated segment
    const int v0 = 2 * (slot - n_rot), v1 = v0 + 1;
    e0 = v0 < n_keep ? v0 * kVec : -1;
    e1 = v1 < n_keep ? v1 * kVec : -1;
    if (e0 >= a.offset) e0 += a.d_rot;
    if (e1 >= a.offset) e1 += a.d_rot;
  }
  const int n_all = a.d / kVec;
  const int c0 = 2 * slot < n_all ? 2 * slot * kVec : -1;
  const int c1 = 2 * slot + 1 < n_all ? (2 * slot + 1) * kVec : -1;

  if (active && !ok && slot == 0 && head0 == 0 && lane == tl * hl_n) set_device_error(a.err, GQA_DEVERR_POSITION);
  const T* xq = reinterpret_cast<const T*>(a.x) + b * a.xs[0] + t * a.xs[2];
  T* yq = reinterpret_cast<T*>(a.out) + b * a.os[0] + t * a.os[2];
  // the token's cache row of KV head 0 (-1: not cached), and the distance to the next head's
  long long row0 = -1;
  if (kAppend && ok && head1 > a.h) {
    const int p = a.pos[b];
    if (p < 0 || (long long)p + a.S > a.T_max) {
      set_device_error(a.err, GQA_DEVERR_POSITION);
    } else if (a.block_table) {
      const int pt = p + t;
      const int page = a.block_table[(long long)b * a.max_pages + pt / a.page_size];
      if (page < 0 || page >= a.num_pages) set_device_error(a.err, GQA_DEVERR_PAGE);
      else row0 = (long long)page * a.h_kv * a.page_size + pt % a.page_size;
    } else {
      row0 = (long long)b * a.h_kv * a.T_max + p + t;
    }
  }
  const int row_step = a.block_table ? a.page_size : a.T_max;

  Vec<T, kVec> x0[kUnroll], x1[kUnroll];
  // what a row is: 0 not written, 1 rotated, 2 copied, 3 written as zeros
  auto kind = [&](int head) {
    if (head >= head1) return 0;
    if (!kAppend || head < a.h) return ok ? 1 : 3;
    return row0 < 0 ? 0 : head < a.h + a.h_kv ? 1 : 2;
  };
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int head = h0 + u * hl_n, kd = kind(head);
      if (kd == 0 || kd == 3) continue;
      const T* src = xq + head * a.xs[1];
      if (kAppend && head >= a.h)
        src = kd == 1 ? reinterpret_cast<const T*>(a.k) + b * a.ks[0] + (head - a.h) * a.ks[1] + t * a.ks[2]
                      : reinterpret_cast<const T*>(a.v) + b * a.vs[0] + (head - a.h - a.h_kv) * a.vs[1] + t * a.vs[2];
      const int f0 = kd == 2 ? c0 : e0, f1 = kd == 2 ? c1 : e1;
      if (f0 >= 0) x0[u].raw = *reinterpret_cast<const Raw_t*>(src + f0);
      if (f1 >= 0) x1[u].raw = *reinterpret_cast<const Raw_t*>(src + f1);
    }
  };
  // the first rows are on their way while the block works out its angles
  int h0 = head0 + lane - tl * hl_n;
  load(h0);

  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int il = i / half, pr = i - il * half;
    const int itok = tok0 + il, ib = itok / a.S;
    const long long p = position(itok, ib, itok - ib * a.S);
    double turn = (double)(p < 0 ? 0 : p) * a.inv_freq[pr] * 0.15915494309189533577;  // 1 / (2 pi)
    turn -= rint(turn);
    float s, c;
    sincospif(2.f * (float)turn, &s, &c);
    table[i] = make_float2(c * a.scale, a.inverse ? -s * a.scale : s * a.scale);
  }
  __syncthreads();

  const float2* cs = table + tl * half + slot * kVec;
  while (h0 < head1) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int head = h0 + u * hl_n, kd = kind(head);
      if (kd == 0) continue;
      if (kd == 3) {
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
          from_f(x0[u].e[k], 0.f);
          from_f(x1[u].e[k], 0.f);
        }
      } else if (kd == 1 && turns) {
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
          // half layout: pair k is element k of either vector; interleaved: elements 2k and 2k + 1 of the
          // two vectors laid end to end
          const float2 w = cs[k];
          T& lo = !kInter ? x0[u].e[k] : 2 * k < kVec ? x0[u].e[(2 * k) % kVec] : x1[u].e[(2 * k) % kVec];
          T& hi = !kInter ? x1[u].e[k] : 2 * k + 1 < kVec ? x0[u].e[(2 * k + 1) % kVec] : x1[u].e[(2 * k + 1) % kVec];
          const float p = to_f(lo), q = to_f(hi);
          from_f(lo, p * w.x - q * w.y);
          from_f(hi, q * w.x + p * w.y);
        }
      }
      T* dst = yq + head * a.os[1];
      if (kAppend && head >= a.h)
        dst = kd == 1 ? reinterpret_cast<T*>(a.k_cache) + (row0 + (long long)(head - a.h) * row_step) * a.d
                      : reinterpret_cast<T*>(a.v_cache) + (row0 + (long long)(head - a.h - a.h_kv) * row_step) * a.d;
      const int f0 = kd == 2 ? c0 : e0, f1 = kd == 2 ? c1 : e1;
      if (f0 >= 0) *reinterpret_cast<Raw_t*>(dst + f0) = x0[u].raw;
      if (f1 >= 0) *reinterpret_cast<Raw_t*>(dst + f1) = x1[u].raw;
    }
    h0 += hl_n * kUnroll;
    load(h0);
  }
}

template <typename T, int kVec>
cudaError_t launch_typed(const RopeArgs& a, int num_sms, cudaStream_t s) {
  const int slots = a.d_rot / 2 / kVec + ((a.d - a.d_rot) / kVec + 1) / 2;
  const int lanes = slots < kThreads ? kThreads / slots : 1;  // rows a block moves at once
  const int H = a.h + 2 * a.h_kv;
  const long long n_tok = (long long)a.B * a.S;
  const int half = a.d_rot / 2;
  // Lanes are split between the heads of a token (hl_n) and tokens. With work for every SM several
  // times over, a lane takes kRowsPerLane heads; with few tokens every row gets a lane of its own.
  const bool many = n_tok * H >= 2ll * kRowsPerLane * num_sms * lanes;
  int hl_n = many ? (H + kRowsPerLane - 1) / kRowsPerLane : H;
  if (hl_n > lanes) hl_n = lanes;
  int tl_n = lanes / hl_n;
  if (tl_n > n_tok) tl_n = (int)n_tok;
  while (tl_n > 1 && tl_n * half * 8 > kMaxTableBytes) --tl_n;
  const int hc = many ? hl_n * kRowsPerLane : hl_n;  // heads of a block
  const long long gx = (n_tok + tl_n - 1) / tl_n;
  const int gy = (H + hc - 1) / hc, gz = (slots + kThreads - 1) / kThreads;
  if (gx > 0x7fffffffLL || gy > 65535) return cudaErrorInvalidConfiguration;
  const size_t smem = (size_t)tl_n * half * sizeof(float2);
  const dim3 grid((unsigned)gx, (unsigned)gy, (unsigned)gz);
  auto kern = a.h_kv > 0 ? (a.interleaved ? rope_kernel<T, kVec, true, true> : rope_kernel<T, kVec, false, true>)
                         : (a.interleaved ? rope_kernel<T, kVec, true, false> : rope_kernel<T, kVec, false, false>);
  kern<<<grid, kThreads, smem, s>>>(a, tl_n, hl_n, hc, slots);
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
