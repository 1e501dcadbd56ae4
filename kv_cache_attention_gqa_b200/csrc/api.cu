// C ABI of the library (declared in include/gqa.h): host-side argument checks, TMA descriptor
// encoding and dispatch to the kernels. No per-call allocation; no per-request state.

#include <cudaTypedefs.h>
#include <math.h>
#include <atomic>
#include <mutex>
#include <string.h>

#include "common.cuh"
#include "internal.h"

namespace gqa {

// Sticky device error word (one per device that loads the library). Kernels receive its address.
__device__ unsigned g_device_error_word;

namespace {

constexpr int kMaxDevices = 64;

// Test hook set by gqa_debug_expire_waits: the bf16 prefill, the contiguous bf16 decode and the
// tensor-core MLA decode pass it to their kernels, whose CTA 0 then waits on a barrier that nothing
// signals.
std::atomic<int> g_expire_waits{0};

unsigned* device_error_ptr() {
  static unsigned* ptrs[kMaxDevices] = {nullptr};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!ptrs[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_device_error_word) != cudaSuccess) return nullptr;
    ptrs[dev] = reinterpret_cast<unsigned*>(p);
  }
  return ptrs[dev];
}

int sm_count() {
  static int cached[kMaxDevices] = {0};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < kMaxDevices && cached[dev] > 0) return cached[dev];
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < kMaxDevices) cached[dev] = n;
  return n;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Encode a bf16 tensor map over a row-major matrix viewed as (rows, inner) with a 128-byte
// swizzle. Dimensions are listed innermost first, as the driver expects.
bool encode_bf16(CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
                 const uint64_t* strides_bytes, const uint32_t* box) {
  auto fn = encode_fn();
  if (!fn) return false;
  uint32_t elem_strides[5] = {1, 1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank,
                        const_cast<void*>(base), dims, strides_bytes, box, elem_strides,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// scale: finite and > 0, or exactly 0 for the default 1/sqrt(d_h) (computed in double, then
// rounded once to fp32, so every caller of the C ABI gets the same fp32 value)
bool valid_scale(float s) { return isfinite(s) && s >= 0.f; }
float resolve_scale(float s, int d) { return s == 0.f ? (float)(1.0 / sqrt((double)d)) : s; }

bool aligned(const void* p, uintptr_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// modified scores: a cap finite and > 0, or 0 for none; key ranges are read as pairs
bool valid_mod(const gqa_score_mod* m) {
  return !m || (isfinite(m->softcap) && m->softcap >= 0.f && aligned(m->key_range, 8));
}
ScoreMod score_mod(const gqa_score_mod* m) {
  ScoreMod s;
  if (m) {
    s.softcap = m->softcap;
    s.slopes = m->alibi_slopes;
    s.range = m->key_range;
  }
  return s;
}

gqa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA; }

}  // namespace

}  // namespace gqa

namespace gqa {
gqa_status decode_check_args(const void* q, const void* k_cache, const void* v_cache, const void* o,
                             int B, int h_q, int h_kv, int T_max, int d_h, float scale, int window,
                             gqa_dtype dtype, int num_splits, long long cache_rows) {
  if (!q || !k_cache || !v_cache || !o) return GQA_ERR_INVALID_ARG;
  if (window < 0) return GQA_ERR_INVALID_ARG;
  if (B <= 0 || h_q <= 0 || h_kv <= 0 || T_max <= 0 || d_h <= 0 || num_splits < 0)
    return GQA_ERR_INVALID_ARG;
  if (h_q % h_kv != 0 || !valid_scale(scale)) return GQA_ERR_INVALID_ARG;
  if (dtype != GQA_BF16 && dtype != GQA_FP32) return GQA_ERR_INVALID_ARG;
  if (B > decode_max_batch()) return GQA_ERR_UNSUPPORTED;
  if (dtype == GQA_FP32 && d_h > 256) return GQA_ERR_UNSUPPORTED;
  if (dtype == GQA_BF16 && d_h != 64 && d_h != 128) return GQA_ERR_UNSUPPORTED;
  if (cache_rows >= (1ll << 31) || (long long)B * h_q >= (1ll << 31)) return GQA_ERR_UNSUPPORTED;
  return GQA_OK;
}
}  // namespace gqa

using namespace gqa;

namespace {
// Shared body of gqa_decode and gqa_decode_paged. A paged call passes block_table != nullptr and
// T_max = max_pages * page_size; k_cache / v_cache are then the page pools.
gqa_status decode_impl(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                       const int32_t* kv_len, const int32_t* q_pos, int B, int h_q, int h_kv,
                       int T_max, int d_h, float scale, int window, gqa_dtype dtype, void* workspace,
                       size_t workspace_bytes, int num_splits, void* stream,
                       const int32_t* block_table, int max_pages, int page_size, int num_pages,
                       const gqa_score_mod* mod = nullptr) {
  using namespace gqa;
  const long long cache_rows =
      block_table ? (long long)num_pages * h_kv * page_size : (long long)B * h_kv * T_max;
  const gqa_status st = decode_check_args(q, k_cache, v_cache, o, B, h_q, h_kv, T_max, d_h, scale,
                                          window, dtype, num_splits, cache_rows);
  if (st != GQA_OK) return st;
  if (!valid_mod(mod)) return GQA_ERR_INVALID_ARG;
  scale = resolve_scale(scale, d_h);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return GQA_ERR_WORKSPACE;
  // the workspace check needs no device query when num_splits is given
  if (num_splits > 0 && workspace_bytes < decode_workspace_bytes(B, h_q, h_kv, T_max, d_h, num_splits, 1))
    return GQA_ERR_WORKSPACE;
  const int sms = sm_count();
  if (sms <= 0) return GQA_ERR_CUDA;
  if (workspace_bytes < decode_workspace_bytes(B, h_q, h_kv, T_max, d_h, num_splits, sms, false, false,
                                               score_mod(mod).on()))
    return GQA_ERR_WORKSPACE;
  DecodeArgs a;
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.o = o;
  a.lse = lse;
  a.kv_len = kv_len;
  a.q_pos = q_pos;
  a.B = B;
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.T_max = T_max;
  a.d_h = d_h;
  a.scale = scale;
  a.window = window;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  a.num_splits = num_splits;
  a.num_sms = sms;
  a.block_table = block_table;
  a.max_pages = max_pages;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.expire_wait = g_expire_waits.load(std::memory_order_relaxed);
  a.mod = score_mod(mod);
  a.err = device_error_ptr();
  if (!a.err) return GQA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == GQA_FP32) return from_cuda(launch_decode_fp32(a, s));
  // Query rows per TMA box = the kernel's m-tiles x 16: units hold min(r, 32) heads (the decode
  // kernel's heads-per-unit limit), two m-tiles above 16. The box height and the kernel's expected
  // bytes must agree, or its full barriers never complete (the bounded waits then report a timeout).
  const int r = h_q / h_kv;
  const uint32_t qrows = r > 16 ? 32 : 16;
  CUtensorMap maps[3];
  // K/V: rows of d_h elements; a paged pool is (num_pages * h_kv * page_size) rows loaded in
  // 64-row boxes when pages hold a multiple of 64 keys, else in 16-row boxes (one per 16-key
  // sub-tile); a contiguous cache (B * h_kv * T_max) in 64-row boxes
  const uint64_t kdims[2] = {(uint64_t)d_h, (uint64_t)cache_rows};
  const uint64_t qdims[2] = {(uint64_t)d_h, (uint64_t)B * h_q};
  const uint64_t strides[1] = {(uint64_t)d_h * 2};
  const uint32_t box[2] = {64, (block_table && page_size % 64 != 0) ? 16u : 64u};
  const uint32_t qbox[2] = {64, qrows};
  if (!encode_bf16(&maps[2], q, 2, qdims, strides, qbox)) return GQA_ERR_CUDA;
  if (block_table && page_size % 64 != 0 && d_h == 128) {
    // 16-row sub-tiles at d_h = 128: a 3-D view whose third dimension steps over the two 128-byte
    // column chunks of a row, so one box carries a whole 16 x 128 sub-tile (half the copies of
    // two 2-D boxes). Falls back to the 2-D boxes if the driver declines the view.
    const uint64_t dims3[3] = {64, (uint64_t)cache_rows, 2};
    const uint64_t strides3[2] = {(uint64_t)d_h * 2, 128};
    const uint32_t box3[3] = {64, 16, 2};
    if (encode_bf16(&maps[0], k_cache, 3, dims3, strides3, box3) &&
        encode_bf16(&maps[1], v_cache, 3, dims3, strides3, box3)) {
      a.paged_3d = 1;
      return from_cuda(launch_decode_bf16(a, maps, s));
    }
  }
  if (!encode_bf16(&maps[0], k_cache, 2, kdims, strides, box) ||
      !encode_bf16(&maps[1], v_cache, 2, kdims, strides, box))
    return GQA_ERR_CUDA;
  return from_cuda(launch_decode_bf16(a, maps, s));
}
}  // namespace

namespace {
void rope_strides(long long* to, const int64_t* from, int B, int h, int S, int d) {
  const long long dense[3] = {(long long)h * S * d, (long long)S * d, d};
  const int size[3] = {B, h, S};
  for (int i = 0; i < 3; ++i) to[i] = size[i] == 1 ? 0 : from ? (long long)from[i] : dense[i];
}

// Rows of d adjacent elements at strides s over n[0] x n[1] x n[2] (s[i] = 0 where n[i] = 1): the elements' extent.
void rows_extent(const long long* s, const int* n, int d, long long& lo, long long& hi) {
  lo = 0;
  hi = d;
  for (int i = 0; i < 3; ++i) (s[i] < 0 ? lo : hi) += (n[i] - 1) * s[i];
}

// Whether two sets of rows share memory. Exact for sets of the same sizes and strides in which each dimension steps
// over the whole of the inner ones (slices of one fused projection lie between each other's rows); sets of other
// shapes count as sharing where their extents meet.
bool rows_overlap(const void* x, const long long* xs, const int* xn, const void* y, const long long* ys, const int* yn,
                  int d, long long elem) {
  long long x0, x1, y0, y1;
  rows_extent(xs, xn, d, x0, x1);
  rows_extent(ys, yn, d, y0, y1);
  const long long delta = (long long)(reinterpret_cast<uintptr_t>(y) - reinterpret_cast<uintptr_t>(x));  // bytes
  if (delta + y0 * elem >= x1 * elem || delta + y1 * elem <= x0 * elem) return false;
  int dim[3] = {0, 1, 2};  // by stride, largest first
  for (int i = 0; i < 3; ++i) {
    if (xs[i] != ys[i] || xn[i] != yn[i] || xs[i] < 0) return true;
    for (int j = i; j > 0 && xs[dim[j]] > xs[dim[j - 1]]; --j) {
      const int t = dim[j];
      dim[j] = dim[j - 1];
      dim[j - 1] = t;
    }
  }
  if (delta % elem != 0) return true;
  long long inner = d;  // extent of the dimensions within
  for (int i = 2; i >= 0; --i) {
    const int k = dim[i];
    if (xn[k] == 1) continue;
    if (xs[k] < inner) return true;
    inner += (xn[k] - 1) * xs[k];
  }
  // is delta within d of a sum of steps? In each dimension only the two steps around what is left can lead there.
  for (int way = 0; way < 8; ++way) {
    long long left = delta / elem;
    for (int i = 0; i < 3; ++i) {
      const long long s = xs[dim[i]], most = xn[dim[i]] - 1;
      if (s == 0) continue;
      long long step = left / s - (left % s < 0) + ((way >> i) & 1);
      step = step < -most ? -most : step > most ? most : step;
      left -= step * s;
    }
    if (left > -d && left < d) return true;
  }
  return false;
}

// Checks and fills the arguments of a rotation (rows x -> out); strides are host arrays of three, in
// elements, or NULL for dense rows. The stride of a dimension of size 1 is never used: it is taken as
// zero, so that it does not narrow the vectors.
gqa_status rope_args(RopeArgs& a, const void* x, void* out, const double* inv_freq,
                     const int32_t* positions, int per_token, int B, int h, int S, int d, int d_rot,
                     int offset, const int64_t* xs, const int64_t* os, int interleaved, int inverse,
                     float scale, gqa_dtype dtype) {
  if (B <= 0 || h <= 0 || S < 0 || d <= 0 || offset < 0) return GQA_ERR_INVALID_ARG;
  if (d_rot <= 0 || d_rot % 2 != 0 || (long long)offset + d_rot > d) return GQA_ERR_INVALID_ARG;
  if ((per_token | 1) != 1 || (interleaved | 1) != 1 || (inverse | 1) != 1) return GQA_ERR_INVALID_ARG;
  if (!isfinite(scale)) return GQA_ERR_INVALID_ARG;
  if (dtype != GQA_BF16 && dtype != GQA_FP32) return GQA_ERR_INVALID_ARG;
  if (S > 0 && (!x || !out || !inv_freq || !positions)) return GQA_ERR_INVALID_ARG;
  if (d > 4096 || (long long)B * S >= (1ll << 31)) return GQA_ERR_UNSUPPORTED;
  a.x = x;
  a.out = out;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.per_token = per_token;
  a.B = B;
  a.h = h;
  a.S = S;
  a.d = d;
  a.d_rot = d_rot;
  a.offset = offset;
  rope_strides(a.xs, xs, B, h, S, d);
  rope_strides(a.os, os, B, h, S, d);
  a.interleaved = interleaved;
  a.inverse = inverse;
  a.scale = scale;
  // in place (every row onto itself), or no memory in common
  const int size[3] = {B, h, S};
  const bool in_place = x == out && a.xs[0] == a.os[0] && a.xs[1] == a.os[1] && a.xs[2] == a.os[2];
  if (h > 0 && S > 0 && !in_place && rows_overlap(x, a.xs, size, out, a.os, size, d, dtype == GQA_BF16 ? 2 : 4))
    return GQA_ERR_INVALID_ARG;
  return GQA_OK;
}

gqa_status rope_launch(RopeArgs& a, gqa_dtype dtype, void* stream) {
  a.err = device_error_ptr();
  const int sms = sm_count();
  if (!a.err || sms <= 0) return GQA_ERR_CUDA;
  return from_cuda(launch_rope(a, dtype, sms, reinterpret_cast<cudaStream_t>(stream)));
}

// Shared body of kv_rope_append and kv_rope_append_paged (block_table != nullptr, T_max = max_pages *
// page_size, k_cache / v_cache the page pools).
gqa_status rope_append_impl(const void* q, const void* k_new, const void* v_new, void* q_out,
                            void* k_cache, void* v_cache, const double* inv_freq, const int32_t* pos,
                            const int32_t* positions, int per_token, int B, int h_q, int h_kv, int S_new,
                            int T_max, int d_h, int d_rot, int offset, const int64_t* qs,
                            const int64_t* ks, const int64_t* vs, int interleaved, float scale,
                            gqa_dtype dtype, void* stream, const int32_t* block_table, int max_pages,
                            int page_size, int num_pages) {
  if (!k_cache || !v_cache || h_kv <= 0 || T_max <= 0) return GQA_ERR_INVALID_ARG;
  if (S_new > 0 && (!k_new || !v_new || !pos)) return GQA_ERR_INVALID_ARG;
  RopeArgs a;
  // without positions a token's position is its cache row
  const gqa_status st = rope_args(a, q, q_out, inv_freq, positions ? positions : pos,
                                  positions ? per_token : 0, B, h_q, S_new, d_h, d_rot, offset, qs, nullptr,
                                  interleaved, 0, scale, dtype);
  if (st != GQA_OK) return st;
  if (S_new > T_max) return GQA_ERR_INVALID_ARG;
  if ((long long)h_q + 2ll * h_kv >= (1ll << 31)) return GQA_ERR_UNSUPPORTED;
  if (S_new == 0) return GQA_OK;  // nothing to rotate or copy
  a.h_kv = h_kv;
  a.k = k_new;
  a.v = v_new;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  rope_strides(a.ks, ks, B, h_kv, S_new, d_h);
  rope_strides(a.vs, vs, B, h_kv, S_new, d_h);
  const int q_size[3] = {B, h_q, S_new}, kv_size[3] = {B, h_kv, S_new};
  const long long elem = dtype == GQA_BF16 ? 2 : 4;
  if (h_q > 0 && (rows_overlap(k_new, a.ks, kv_size, q_out, a.os, q_size, d_h, elem) ||
                  rows_overlap(v_new, a.vs, kv_size, q_out, a.os, q_size, d_h, elem)))
    return GQA_ERR_INVALID_ARG;
  a.pos = pos;
  a.T_max = T_max;
  a.block_table = block_table;
  a.max_pages = max_pages;
  a.page_size = page_size;
  a.num_pages = num_pages;
  return rope_launch(a, dtype, stream);
}

// Shared body of gqa_kv_weights and gqa_kv_weights_paged (block_table != nullptr, T_max = max_pages *
// page_size, k the page pool).
gqa_status kv_weights_impl(KvWeightsArgs a, gqa_dtype dtype, size_t workspace_bytes, void* stream) {
  if (!a.q || !a.k || !a.lse || !a.w) return GQA_ERR_INVALID_ARG;
  if (a.B <= 0 || a.h_q <= 0 || a.h_kv <= 0 || a.S_q <= 0 || a.T_max <= 0 || a.d_h <= 0) return GQA_ERR_INVALID_ARG;
  if (a.h_q % a.h_kv != 0 || !valid_scale(a.scale)) return GQA_ERR_INVALID_ARG;
  if ((a.causal | 1) != 1 || (a.accumulate | 1) != 1) return GQA_ERR_INVALID_ARG;
  if (a.window < 0 || (a.window > 0 && a.causal != 1)) return GQA_ERR_INVALID_ARG;
  if (dtype != GQA_BF16 && dtype != GQA_FP32) return GQA_ERR_INVALID_ARG;
  if (dtype == GQA_FP32 && a.d_h > 256) return GQA_ERR_UNSUPPORTED;
  if (dtype == GQA_BF16 && a.d_h != 64 && a.d_h != 128) return GQA_ERR_UNSUPPORTED;
  const long long k_rows = a.block_table ? (long long)a.num_pages * a.h_kv * a.page_size
                                         : (long long)a.B * a.h_kv * a.T_max;
  if (k_rows >= (1ll << 31) || (long long)a.B * a.h_kv * a.T_max >= (1ll << 31) ||
      (long long)a.B * a.h_q * a.S_q >= (1ll << 31) || (long long)a.B * a.h_kv > 65535)
    return GQA_ERR_UNSUPPORTED;
  a.scale = resolve_scale(a.scale, a.d_h);
  const int sms = sm_count();
  if (sms <= 0) return GQA_ERR_CUDA;
  const size_t need = kv_weights_workspace_bytes(a.B, a.h_q, a.h_kv, a.S_q, a.T_max, dtype, sms);
  if (need > 0 && (!a.workspace || (reinterpret_cast<uintptr_t>(a.workspace) & 255u) || workspace_bytes < need))
    return GQA_ERR_WORKSPACE;
  a.err = device_error_ptr();
  if (!a.err) return GQA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == GQA_FP32) return from_cuda(launch_kv_weights_fp32(a, s));
  const KvWeightsTile t = kv_weights_tile(a.h_q, a.h_kv, a.S_q);
  CUtensorMap maps[2];
  const uint64_t strides[1] = {(uint64_t)a.d_h * 2};
  const uint32_t sub = (uint32_t)kv_weights_sub(a.block_table != nullptr, a.page_size);
  bool ok;
  if (kv_weights_4d(a.block_table != nullptr, a.d_h)) {
    // groups of 8 rows (pages hold whole ones) with their two 64-column chunks side by side
    const uint64_t dims[4] = {64, 8, 2, (uint64_t)k_rows / 8};
    const uint64_t strides4[3] = {256, 128, 2048};
    const uint32_t box[4] = {64, 8, 2, sub / 8};
    ok = encode_bf16(&maps[0], a.k, 4, dims, strides4, box);
  } else {
    const uint64_t kdims[2] = {(uint64_t)a.d_h, (uint64_t)k_rows};
    const uint32_t kbox[2] = {64, sub};
    ok = encode_bf16(&maps[0], a.k, 2, kdims, strides, kbox);
  }
  if (!ok) return GQA_ERR_CUDA;
  if (t.small) {
    const uint64_t qdims[2] = {(uint64_t)a.d_h, (uint64_t)a.B * a.h_q * a.S_q};
    const uint32_t qbox[2] = {64, (uint32_t)t.rows};
    ok = encode_bf16(&maps[1], a.q, 2, qdims, strides, qbox);
  } else {
    const uint64_t rows = (uint64_t)a.B * a.h_q;
    const uint64_t qdims[3] = {(uint64_t)a.d_h, t.flat ? rows * a.S_q : (uint64_t)a.S_q, t.flat ? 1 : rows};
    const uint64_t qstrides[2] = {(uint64_t)a.d_h * 2, qdims[1] * a.d_h * 2};
    const uint32_t qbox[3] = {64, t.flat ? 128u : (uint32_t)t.P, t.flat ? 1u : (uint32_t)t.H};
    ok = encode_bf16(&maps[1], a.q, 3, qdims, qstrides, qbox);
  }
  if (!ok) return GQA_ERR_CUDA;
  return from_cuda(launch_kv_weights_bf16(a, maps, sms, s));
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// Checks shared by kv_evict and kv_evict_paged, and the launch.
gqa_status evict_impl(EvictArgs& a, int d_h, gqa_dtype dtype, void* stream) {
  if (!a.k || !a.v || !a.k_out || !a.v_out || !a.w || !a.w_out || !a.kept || !a.new_len) return GQA_ERR_INVALID_ARG;
  if (a.B <= 0 || a.h_kv <= 0 || a.T_max <= 0 || a.T_out <= 0 || d_h <= 0) return GQA_ERR_INVALID_ARG;
  if (a.budget <= 0 || a.sink < 0 || a.recent < 0 || (long long)a.sink + a.recent > a.budget) return GQA_ERR_INVALID_ARG;
  if (a.budget > a.T_out) return GQA_ERR_INVALID_ARG;
  if (dtype != GQA_BF16 && dtype != GQA_FP32) return GQA_ERR_INVALID_ARG;
  // every block reads kv_len after new_len may be written
  if (a.kv_len && overlap(a.kv_len, (size_t)a.B * 4, a.new_len, (size_t)a.B * 4)) return GQA_ERR_INVALID_ARG;
  const size_t bg = (size_t)a.B * a.h_kv;
  if (a.w_out == a.w ? a.T_out != a.T_max
                     : overlap(a.w, bg * a.T_max * 4, a.w_out, bg * a.T_out * 4))
    return GQA_ERR_INVALID_ARG;
  // rows are counted in 32 bits, by threads that look up to a few blocks' width past the last one
  const long long most = (1ll << 31) - (1ll << 16);
  const long long rows = a.block_table ? (long long)a.num_pages * a.h_kv * a.page_size : (long long)bg * a.T_max;
  if (rows >= most || (long long)bg * a.T_max >= most || (long long)bg * a.T_out >= most || (long long)bg > 65535)
    return GQA_ERR_UNSUPPORTED;
  a.err = device_error_ptr();
  const int sms = sm_count();
  if (!a.err || sms <= 0) return GQA_ERR_CUDA;
  return from_cuda(launch_kv_evict(a, d_h, dtype == GQA_BF16 ? 2 : 4, sms, reinterpret_cast<cudaStream_t>(stream)));
}
}  // namespace

extern "C" {

const char* gqa_status_string(gqa_status s) {
  switch (s) {
    case GQA_OK: return "GQA_OK";
    case GQA_ERR_INVALID_ARG: return "GQA_ERR_INVALID_ARG";
    case GQA_ERR_UNSUPPORTED: return "GQA_ERR_UNSUPPORTED";
    case GQA_ERR_CUDA: return "GQA_ERR_CUDA";
    case GQA_ERR_DEVICE: return "GQA_ERR_DEVICE";
    case GQA_ERR_WORKSPACE: return "GQA_ERR_WORKSPACE";
  }
  return "GQA_ERR_UNKNOWN";
}

const char* gqa_version(void) { return "gqa-b200 0.2.0 (sm_100a)"; }

gqa_status gqa_debug_expire_waits(int enable) {
  if (enable != 0 && enable != 1) return GQA_ERR_INVALID_ARG;
  g_expire_waits.store(enable, std::memory_order_relaxed);
  return GQA_OK;
}

gqa_status gqa_get_device_error(int* code, void* stream) {
  if (!code) return GQA_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  unsigned v = 0;
  if (cudaStreamSynchronize(s) != cudaSuccess) return GQA_ERR_CUDA;
  if (cudaMemcpyFromSymbol(&v, g_device_error_word, sizeof(v)) != cudaSuccess) return GQA_ERR_CUDA;
  *code = (int)v;
  if (v != 0) {
    const unsigned zero = 0;
    if (cudaMemcpyToSymbol(g_device_error_word, &zero, sizeof(zero)) != cudaSuccess)
      return GQA_ERR_CUDA;
    return GQA_ERR_DEVICE;
  }
  return GQA_OK;
}

gqa_status kv_append(void* k_cache, void* v_cache, const void* k_new, const void* v_new,
                     const int32_t* pos, int B, int h_kv, int S_new, int T_max, int d_h,
                     gqa_dtype dtype, void* stream) {
  if (!k_cache || !v_cache) return GQA_ERR_INVALID_ARG;
  if (S_new > 0 && (!k_new || !v_new || !pos)) return GQA_ERR_INVALID_ARG;  // S_new = 0: no-op
  if (B <= 0 || h_kv <= 0 || S_new < 0 || T_max <= 0 || d_h <= 0) return GQA_ERR_INVALID_ARG;
  if (dtype != GQA_BF16 && dtype != GQA_FP32) return GQA_ERR_INVALID_ARG;
  if (S_new > T_max) return GQA_ERR_INVALID_ARG;
  if (S_new == 0) return GQA_OK;  // nothing to copy
  AppendArgs a;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_new = k_new;
  a.v_new = v_new;
  a.pos = pos;
  a.B = B;
  a.h_kv = h_kv;
  a.S_new = S_new;
  a.T_max = T_max;
  a.d_h = d_h;
  a.elem_bytes = dtype == GQA_BF16 ? 2 : 4;
  a.err = device_error_ptr();
  if (!a.err) return GQA_ERR_CUDA;
  return from_cuda(launch_kv_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

gqa_status gqa_prefill(const void* q, const void* k_cache, const void* v_cache, void* o,
                       float* lse, const int32_t* q_start, const int32_t* kv_len,
                       int B, int h_q, int h_kv, int S_q, int T_max, int d_h,
                       float scale, int causal, int window, gqa_dtype dtype, void* stream) {
  return gqa_prefill_mod(q, k_cache, v_cache, o, lse, q_start, kv_len, nullptr, B, h_q, h_kv, S_q, T_max, d_h,
                         scale, causal, window, dtype, nullptr, 0, stream);
}

size_t gqa_prefill_mod_workspace_size(int B, int h_q, int h_kv, int S_q) {
  if (B <= 0 || h_q <= 0 || h_kv <= 0 || S_q <= 0 || h_q % h_kv != 0) return 0;
  return (prefill_hull_bytes(B, h_q, h_kv, S_q) + 255) / 256 * 256;
}

gqa_status gqa_prefill_mod(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                           const int32_t* q_start, const int32_t* kv_len, const gqa_score_mod* mod,
                           int B, int h_q, int h_kv, int S_q, int T_max, int d_h, float scale,
                           int causal, int window, gqa_dtype dtype, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (!q || !k_cache || !v_cache || !o) return GQA_ERR_INVALID_ARG;
  // a window is measured back from each row's own position, so it needs the causal mask
  if (window < 0 || (window > 0 && causal != 1)) return GQA_ERR_INVALID_ARG;
  if (B <= 0 || h_q <= 0 || h_kv <= 0 || S_q <= 0 || T_max <= 0 || d_h <= 0)
    return GQA_ERR_INVALID_ARG;
  if (h_q % h_kv != 0 || !valid_scale(scale)) return GQA_ERR_INVALID_ARG;
  scale = resolve_scale(scale, d_h);
  if (causal != 0 && causal != 1) return GQA_ERR_INVALID_ARG;
  // every host-detectable problem is reported before the first CUDA call
  if (dtype != GQA_BF16 && dtype != GQA_FP32) return GQA_ERR_INVALID_ARG;
  if (dtype == GQA_FP32 && d_h > 256) return GQA_ERR_UNSUPPORTED;
  if (dtype == GQA_BF16) {
    if (d_h != 64 && d_h != 128) return GQA_ERR_UNSUPPORTED;
    if ((long long)B * h_kv * T_max >= (1ll << 31) || (long long)B * h_q * S_q >= (1ll << 31))
      return GQA_ERR_UNSUPPORTED;
    if (!aligned(o, 16)) return GQA_ERR_INVALID_ARG;  // written in 16-byte vectors
  }
  if (!valid_mod(mod)) return GQA_ERR_INVALID_ARG;
  if (dtype == GQA_BF16 && mod && mod->key_range &&
      (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
       workspace_bytes < gqa_prefill_mod_workspace_size(B, h_q, h_kv, S_q)))
    return GQA_ERR_WORKSPACE;
  PrefillArgs a;
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.o = o;
  a.lse = lse;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.B = B;
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.S_q = S_q;
  a.T_max = T_max;
  a.d_h = d_h;
  a.scale = scale;
  a.causal = causal;
  a.window = window;
  a.expire_wait = g_expire_waits.load(std::memory_order_relaxed);
  a.mod = score_mod(mod);
  a.workspace = workspace;
  a.err = device_error_ptr();
  if (!a.err) return GQA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == GQA_FP32) return from_cuda(a.mod.on() ? launch_prefill_fp32_mod(a, sm_count(), s) : launch_prefill_fp32(a, s));
  // TMA views: Q as (d_h, S_q, B*h_q) with box (64, P, H): one box holds the H heads x P
  // positions of a tile, head-major; K, V as rows (B*h_kv*T_max, d_h) with box (64, 128).
  const int H = prefill_heads_per_tile(h_q, h_kv);
  const uint32_t P = (uint32_t)(128 / H);
  CUtensorMap maps[3];
  const uint64_t qdims[3] = {(uint64_t)d_h, (uint64_t)S_q, (uint64_t)B * h_q};
  const uint64_t qstrides[2] = {(uint64_t)d_h * 2, (uint64_t)S_q * d_h * 2};
  const uint32_t qbox[3] = {64, P, (uint32_t)H};
  const uint64_t kdims[2] = {(uint64_t)d_h, (uint64_t)B * h_kv * T_max};
  const uint64_t strides[1] = {(uint64_t)d_h * 2};
  const uint32_t box[2] = {64, 128};
  if (!encode_bf16(&maps[0], q, 3, qdims, qstrides, qbox) ||
      !encode_bf16(&maps[1], k_cache, 2, kdims, strides, box) ||
      !encode_bf16(&maps[2], v_cache, 2, kdims, strides, box))
    return GQA_ERR_CUDA;
  return from_cuda(launch_prefill_bf16(a, maps, sm_count(), s));
}

size_t gqa_prefill_backward_workspace_size(int B, int h_q, int S_q) {
  if (B <= 0 || h_q <= 0 || S_q <= 0) return 0;
  const size_t rows = (size_t)B * h_q * S_q;
  return 2 * ((rows * 4 + 255) / 256 * 256) + 256;  // lse2, D, the work-item counter
}

gqa_status gqa_prefill_backward(const void* q, const void* k_cache, const void* v_cache,
                                const void* o, const void* d_o, const float* lse, void* dq,
                                void* dk, void* dv, const int32_t* q_start, const int32_t* kv_len,
                                int B, int h_q, int h_kv, int S_q, int T_max, int d_h, float scale,
                                int causal, int window, gqa_dtype dtype, void* workspace,
                                size_t workspace_bytes, void* stream) {
  return gqa_prefill_backward_mod(q, k_cache, v_cache, o, d_o, lse, dq, dk, dv, q_start, kv_len, nullptr, B, h_q,
                                  h_kv, S_q, T_max, d_h, scale, causal, window, dtype, workspace, workspace_bytes,
                                  stream);
}

size_t gqa_prefill_backward_mod_workspace_size(int B, int h_q, int h_kv, int S_q) {
  if (B <= 0 || h_q <= 0 || h_kv <= 0 || S_q <= 0 || h_q % h_kv != 0) return 0;
  const size_t rows = (size_t)B * h_q * S_q;  // the second part of D
  return gqa_prefill_backward_workspace_size(B, h_q, S_q) + (rows * 4 + 255) / 256 * 256 +
         (backward_hull_bytes(B, h_q, h_kv, S_q) + 255) / 256 * 256;
}

gqa_status gqa_prefill_backward_mod(const void* q, const void* k_cache, const void* v_cache, const void* o,
                                    const void* d_o, const float* lse, void* dq, void* dk, void* dv,
                                    const int32_t* q_start, const int32_t* kv_len,
                                    const gqa_score_mod* mod, int B, int h_q, int h_kv, int S_q,
                                    int T_max, int d_h, float scale, int causal, int window,
                                    gqa_dtype dtype, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  if (!q || !k_cache || !v_cache || !o || !d_o || !lse || !dq || !dk || !dv) return GQA_ERR_INVALID_ARG;
  if (B <= 0 || h_q <= 0 || h_kv <= 0 || S_q <= 0 || T_max <= 0 || d_h <= 0) return GQA_ERR_INVALID_ARG;
  if (h_q % h_kv != 0 || !valid_scale(scale)) return GQA_ERR_INVALID_ARG;
  scale = resolve_scale(scale, d_h);
  if (causal != 0 && causal != 1) return GQA_ERR_INVALID_ARG;
  if (window < 0 || (window > 0 && causal != 1)) return GQA_ERR_INVALID_ARG;
  if (dtype != GQA_BF16 && dtype != GQA_FP32) return GQA_ERR_INVALID_ARG;
  if (dtype == GQA_FP32 && d_h > 256) return GQA_ERR_UNSUPPORTED;
  if (dtype == GQA_BF16 && d_h != 64 && d_h != 128) return GQA_ERR_UNSUPPORTED;
  if ((long long)B * h_kv * T_max >= (1ll << 31) || (long long)B * h_q * S_q >= (1ll << 31))
    return GQA_ERR_UNSUPPORTED;
  if (!valid_mod(mod)) return GQA_ERR_INVALID_ARG;
  if (dtype == GQA_BF16 && !(aligned(dq, 16) && aligned(dk, 16) && aligned(dv, 16))) return GQA_ERR_INVALID_ARG;
  const size_t base = gqa_prefill_backward_workspace_size(B, h_q, S_q);
  const size_t need = score_mod(mod).on() ? gqa_prefill_backward_mod_workspace_size(B, h_q, h_kv, S_q) : base;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < need)
    return GQA_ERR_WORKSPACE;
  BackwardArgs a;
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.o = o;
  a.d_o = d_o;
  a.lse = lse;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.B = B;
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.S_q = S_q;
  a.T_max = T_max;
  a.d_h = d_h;
  a.scale = scale;
  a.causal = causal;
  a.window = window;
  const size_t half = (base - 256) / 2;
  a.lse2 = reinterpret_cast<float*>(workspace);
  a.drow = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace) + half);
  a.ticket = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(workspace) + 2 * half);
  a.mod = score_mod(mod);
  a.dpart1 = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace) + base);
  a.hull = reinterpret_cast<uint8_t*>(workspace) + base + half;
  a.err = device_error_ptr();
  if (!a.err) return GQA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == GQA_FP32) return from_cuda(a.mod.on() ? launch_backward_fp32_mod(a, sm_count(), s) : launch_backward_fp32(a, s));
  // TMA views: Q and dO as (d_h, S_q, B*h_q) with box (64, 64, 1) for the key-stationary dK/dV
  // kernel and (64, P, H) for the query-stationary dQ kernel; K, V as rows with box (64, 128) for
  // dK/dV (its 128 stationary keys) and (64, 64) for dQ (its 64-key blocks).
  const int H = prefill_heads_per_tile(h_q, h_kv);
  const uint32_t P = (uint32_t)(128 / H);
  CUtensorMap maps[8];
  const uint64_t qdims[3] = {(uint64_t)d_h, (uint64_t)S_q, (uint64_t)B * h_q};
  const uint64_t qstrides[2] = {(uint64_t)d_h * 2, (uint64_t)S_q * d_h * 2};
  const uint32_t qbox_rows[3] = {64, 64, 1};
  const uint32_t qbox_tile[3] = {64, P, (uint32_t)H};
  const uint64_t kdims[2] = {(uint64_t)d_h, (uint64_t)B * h_kv * T_max};
  const uint64_t strides[1] = {(uint64_t)d_h * 2};
  const uint32_t box[2] = {64, 128};
  const uint32_t box64[2] = {64, 64};
  if (!encode_bf16(&maps[6], k_cache, 2, kdims, strides, box64) ||
      !encode_bf16(&maps[7], v_cache, 2, kdims, strides, box64) ||
      !encode_bf16(&maps[0], q, 3, qdims, qstrides, qbox_rows) ||
      !encode_bf16(&maps[1], d_o, 3, qdims, qstrides, qbox_rows) ||
      !encode_bf16(&maps[2], k_cache, 2, kdims, strides, box) ||
      !encode_bf16(&maps[3], v_cache, 2, kdims, strides, box) ||
      !encode_bf16(&maps[4], q, 3, qdims, qstrides, qbox_tile) ||
      !encode_bf16(&maps[5], d_o, 3, qdims, qstrides, qbox_tile))
    return GQA_ERR_CUDA;
  const int sms = sm_count();
  if (sms <= 0) return GQA_ERR_CUDA;
  return from_cuda(launch_backward_bf16(a, maps, sms, s));
}

namespace {
size_t decode_workspace_size(int B, int h_q, int h_kv, int T_max, int d_h, gqa_dtype dtype, int num_splits, bool mod) {
  if (B <= 0 || h_q <= 0 || h_kv <= 0 || T_max <= 0 || d_h <= 0 || h_q % h_kv != 0) return 0;
  if (num_splits < 0 || (dtype != GQA_BF16 && dtype != GQA_FP32)) return 0;
  const int sms = num_splits > 0 ? 1 : sm_count();
  if (sms <= 0) return 0;
  return decode_workspace_bytes(B, h_q, h_kv, T_max, d_h, num_splits, sms, false, false, mod);
}
}  // namespace

size_t gqa_decode_workspace_size(int B, int h_q, int h_kv, int T_max, int d_h, gqa_dtype dtype,
                                 int num_splits) {
  return decode_workspace_size(B, h_q, h_kv, T_max, d_h, dtype, num_splits, false);
}

size_t gqa_decode_mod_workspace_size(int B, int h_q, int h_kv, int T_max, int d_h, gqa_dtype dtype,
                                     int num_splits) {
  return decode_workspace_size(B, h_q, h_kv, T_max, d_h, dtype, num_splits, true);
}

gqa_status gqa_decode(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                      const int32_t* kv_len, const int32_t* q_pos,
                      int B, int h_q, int h_kv, int T_max, int d_h, float scale, int window,
                      gqa_dtype dtype, void* workspace, size_t workspace_bytes, int num_splits,
                      void* stream) {
  return decode_impl(q, k_cache, v_cache, o, lse, kv_len, q_pos, B, h_q, h_kv, T_max, d_h, scale,
                     window, dtype, workspace, workspace_bytes, num_splits, stream, nullptr, 0, 0, 0);
}

size_t gqa_mla_decode_workspace_size(int B, int h_q, int T_max, int d_v, gqa_dtype dtype,
                                     int num_splits) {
  if (B <= 0 || h_q <= 0 || T_max <= 0 || d_v <= 0 || num_splits < 0) return 0;
  if (dtype != GQA_BF16 && dtype != GQA_FP32) return 0;
  const int sms = num_splits > 0 ? 1 : sm_count();
  if (sms <= 0) return 0;
  return decode_workspace_bytes(B, h_q, 1, T_max, d_v, num_splits, sms, true, mla_uses_tc(h_q, dtype) != 0);
}

gqa_status gqa_mla_decode(const void* q, const void* cache, void* o, float* lse,
                          const int32_t* kv_len, const int32_t* q_pos, int B, int h_q, int T_max,
                          int d_qk, int d_v, float scale, gqa_dtype dtype, void* workspace,
                          size_t workspace_bytes, int num_splits, void* stream) {
  if (!q || !cache || !o) return GQA_ERR_INVALID_ARG;
  if (B <= 0 || h_q <= 0 || T_max <= 0 || d_qk <= 0 || d_v <= 0 || d_v > d_qk || num_splits < 0)
    return GQA_ERR_INVALID_ARG;
  if (!valid_scale(scale)) return GQA_ERR_INVALID_ARG;
  scale = resolve_scale(scale, d_qk);
  if (dtype != GQA_BF16 && dtype != GQA_FP32) return GQA_ERR_INVALID_ARG;
  if (dtype == GQA_BF16 && !mla_dims_supported_bf16(d_qk, d_v)) return GQA_ERR_UNSUPPORTED;
  if (dtype == GQA_FP32 && (d_qk > 768 || d_v > 512)) return GQA_ERR_UNSUPPORTED;
  if (dtype == GQA_BF16 && !aligned(o, 16)) return GQA_ERR_INVALID_ARG;
  if (B > decode_max_batch()) return GQA_ERR_UNSUPPORTED;
  if ((long long)B * T_max >= (1ll << 31) || (long long)B * h_q >= (1ll << 31)) return GQA_ERR_UNSUPPORTED;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return GQA_ERR_WORKSPACE;
  const bool tc = mla_uses_tc(h_q, dtype) != 0;
  if (num_splits > 0 && workspace_bytes < decode_workspace_bytes(B, h_q, 1, T_max, d_v, num_splits, 1, true, tc))
    return GQA_ERR_WORKSPACE;
  const int sms = sm_count();
  if (sms <= 0) return GQA_ERR_CUDA;
  if (workspace_bytes < decode_workspace_bytes(B, h_q, 1, T_max, d_v, num_splits, sms, true, tc))
    return GQA_ERR_WORKSPACE;
  DecodeArgs a;
  a.q = q;
  a.k = cache;
  a.v = cache;  // values are the first d_v entries of each cache row
  a.o = o;
  a.lse = lse;
  a.kv_len = kv_len;
  a.q_pos = q_pos;
  a.B = B;
  a.h_q = h_q;
  a.h_kv = 1;
  a.T_max = T_max;
  a.d_h = d_qk;
  a.d_v = d_v;
  a.mla = 1;
  a.mla_tc = tc ? 1 : 0;
  a.expire_wait = g_expire_waits.load(std::memory_order_relaxed);
  a.scale = scale;
  a.window = 0;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  a.num_splits = num_splits;
  a.num_sms = sms;
  a.err = device_error_ptr();
  if (!a.err) return GQA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == GQA_FP32) return from_cuda(launch_decode_fp32(a, s));
  CUtensorMap maps[4];
  const uint64_t cdims[2] = {(uint64_t)d_qk, (uint64_t)B * T_max};
  const uint64_t qdims[2] = {(uint64_t)d_qk, (uint64_t)B * h_q};
  const uint64_t strides[1] = {(uint64_t)d_qk * 2};
  const uint32_t cbox[2] = {64, 64};
  const uint32_t qbox[2] = {64, 16};
  // The tensor-core kernel reads rows as (64 columns, rows, 9 column chunks): one copy brings a
  // tile's chunks (the chunk dimension outermost in shared memory, one 128-byte row per key and
  // chunk) -- 32-key cache tiles, and the query's last 3 chunks of 128 heads.
  const uint64_t cdims3[3] = {64, (uint64_t)B * T_max, (uint64_t)d_qk / 64};
  const uint64_t qdims3[3] = {64, (uint64_t)B * h_q, (uint64_t)d_qk / 64};
  const uint64_t strides3[2] = {(uint64_t)d_qk * 2, 128};
  const uint32_t cbox_tc[3] = {64, 32, (uint32_t)d_qk / 64};
  const uint32_t qbox_tc[3] = {64, 128, 3};
  if (!encode_bf16(&maps[0], cache, 2, cdims, strides, cbox) ||
      !encode_bf16(&maps[1], q, 2, qdims, strides, qbox) ||
      (tc && (!encode_bf16(&maps[2], q, 3, qdims3, strides3, qbox_tc) ||
              !encode_bf16(&maps[3], cache, 3, cdims3, strides3, cbox_tc))))
    return GQA_ERR_CUDA;
  return from_cuda(launch_mla_bf16(a, maps, s));
}

gqa_status gqa_decode_paged(const void* q, const void* k_pages, const void* v_pages, void* o,
                            float* lse, const int32_t* kv_len, const int32_t* q_pos,
                            const int32_t* block_table, int B, int h_q, int h_kv, int num_pages,
                            int page_size, int max_pages, int d_h, float scale, int window,
                            gqa_dtype dtype, void* workspace, size_t workspace_bytes,
                            int num_splits, void* stream) {
  if (!block_table || num_pages <= 0 || page_size <= 0 || max_pages <= 0) return GQA_ERR_INVALID_ARG;
  if (page_size % 16 != 0) return GQA_ERR_UNSUPPORTED;
  const long long T_max = (long long)max_pages * page_size;
  if (T_max >= (1ll << 31)) return GQA_ERR_UNSUPPORTED;
  return decode_impl(q, k_pages, v_pages, o, lse, kv_len, q_pos, B, h_q, h_kv, (int)T_max, d_h,
                     scale, window, dtype, workspace, workspace_bytes, num_splits, stream, block_table,
                     max_pages, page_size, num_pages);
}

gqa_status kv_append_paged(void* k_pages, void* v_pages, const void* k_new, const void* v_new,
                           const int32_t* pos, const int32_t* block_table, int B, int h_kv,
                           int S_new, int num_pages, int page_size, int max_pages, int d_h,
                           gqa_dtype dtype, void* stream) {
  using namespace gqa;
  if (!k_pages || !v_pages) return GQA_ERR_INVALID_ARG;
  if (S_new > 0 && (!k_new || !v_new || !pos || !block_table)) return GQA_ERR_INVALID_ARG;  // S_new = 0: no-op
  if (B <= 0 || h_kv <= 0 || S_new < 0 || d_h <= 0) return GQA_ERR_INVALID_ARG;
  if (num_pages <= 0 || page_size <= 0 || max_pages <= 0) return GQA_ERR_INVALID_ARG;
  if (dtype != GQA_BF16 && dtype != GQA_FP32) return GQA_ERR_INVALID_ARG;
  const long long T_max = (long long)max_pages * page_size;
  if (T_max >= (1ll << 31)) return GQA_ERR_UNSUPPORTED;
  if (S_new > T_max) return GQA_ERR_INVALID_ARG;
  if (S_new == 0) return GQA_OK;  // nothing to copy
  AppendArgs a;
  a.k_cache = k_pages;
  a.v_cache = v_pages;
  a.k_new = k_new;
  a.v_new = v_new;
  a.pos = pos;
  a.B = B;
  a.h_kv = h_kv;
  a.S_new = S_new;
  a.T_max = (int)T_max;
  a.d_h = d_h;
  a.elem_bytes = dtype == GQA_BF16 ? 2 : 4;
  a.block_table = block_table;
  a.max_pages = max_pages;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.err = device_error_ptr();
  if (!a.err) return GQA_ERR_CUDA;
  return from_cuda(launch_kv_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

gqa_status gqa_rope(const void* x, void* out, const double* inv_freq, const int32_t* positions,
                    int per_token, int B, int h, int S, int d, int d_rot, int offset,
                    const int64_t* x_strides, const int64_t* out_strides, int interleaved, int inverse,
                    float scale, gqa_dtype dtype, void* stream) {
  if (h <= 0) return GQA_ERR_INVALID_ARG;
  RopeArgs a;
  const gqa_status st = rope_args(a, x, out, inv_freq, positions, per_token, B, h, S, d, d_rot, offset,
                                  x_strides, out_strides, interleaved, inverse, scale, dtype);
  if (st != GQA_OK || S == 0) return st;
  return rope_launch(a, dtype, stream);
}

gqa_status kv_rope_append(const void* q, const void* k_new, const void* v_new, void* q_out,
                          void* k_cache, void* v_cache, const double* inv_freq, const int32_t* pos,
                          const int32_t* positions, int per_token, int B, int h_q, int h_kv, int S_new,
                          int T_max, int d_h, int d_rot, int offset, const int64_t* q_strides,
                          const int64_t* k_strides, const int64_t* v_strides, int interleaved,
                          float scale, gqa_dtype dtype, void* stream) {
  return rope_append_impl(q, k_new, v_new, q_out, k_cache, v_cache, inv_freq, pos, positions, per_token, B,
                          h_q, h_kv, S_new, T_max, d_h, d_rot, offset, q_strides, k_strides, v_strides,
                          interleaved, scale, dtype, stream, nullptr, 0, 0, 0);
}

gqa_status kv_rope_append_paged(const void* q, const void* k_new, const void* v_new, void* q_out,
                                void* k_pages, void* v_pages, const double* inv_freq,
                                const int32_t* pos, const int32_t* positions, int per_token,
                                const int32_t* block_table, int B, int h_q, int h_kv, int S_new,
                                int num_pages, int page_size, int max_pages, int d_h, int d_rot,
                                int offset, const int64_t* q_strides, const int64_t* k_strides,
                                const int64_t* v_strides, int interleaved, float scale,
                                gqa_dtype dtype, void* stream) {
  if (num_pages <= 0 || page_size <= 0 || max_pages <= 0) return GQA_ERR_INVALID_ARG;
  if (S_new > 0 && !block_table) return GQA_ERR_INVALID_ARG;
  const long long T_max = (long long)max_pages * page_size;
  if (T_max >= (1ll << 31)) return GQA_ERR_UNSUPPORTED;
  return rope_append_impl(q, k_new, v_new, q_out, k_pages, v_pages, inv_freq, pos, positions, per_token, B,
                          h_q, h_kv, S_new, (int)T_max, d_h, d_rot, offset, q_strides, k_strides, v_strides,
                          interleaved, scale, dtype, stream, block_table, max_pages, page_size, num_pages);
}

size_t gqa_kv_weights_workspace_size(int B, int h_q, int h_kv, int S_q, int T_max, gqa_dtype dtype) {
  if (B <= 0 || h_q <= 0 || h_kv <= 0 || S_q <= 0 || T_max <= 0 || h_q % h_kv != 0) return 0;
  return kv_weights_workspace_bytes(B, h_q, h_kv, S_q, T_max, dtype, sm_count());
}

gqa_status gqa_kv_weights(const void* q, const void* k_cache, const float* lse, float* weights,
                          const int32_t* q_start, const int32_t* kv_len, int B, int h_q, int h_kv,
                          int S_q, int T_max, int d_h, float scale, int causal, int window,
                          int accumulate, gqa_dtype dtype, void* workspace, size_t workspace_bytes,
                          void* stream) {
  KvWeightsArgs a;
  a.q = q;
  a.k = k_cache;
  a.lse = lse;
  a.w = weights;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.B = B;
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.S_q = S_q;
  a.T_max = T_max;
  a.d_h = d_h;
  a.scale = scale;
  a.causal = causal;
  a.window = window;
  a.accumulate = accumulate;
  a.workspace = workspace;
  return kv_weights_impl(a, dtype, workspace_bytes, stream);
}

gqa_status gqa_kv_weights_paged(const void* q, const void* k_pages, const float* lse, float* weights,
                                const int32_t* q_start, const int32_t* kv_len,
                                const int32_t* block_table, int B, int h_q, int h_kv, int S_q,
                                int num_pages, int page_size, int max_pages, int d_h, float scale,
                                int causal, int window, int accumulate, gqa_dtype dtype,
                                void* workspace, size_t workspace_bytes, void* stream) {
  if (!block_table || num_pages <= 0 || page_size <= 0 || max_pages <= 0) return GQA_ERR_INVALID_ARG;
  if (page_size % 16 != 0) return GQA_ERR_UNSUPPORTED;
  const long long T_max = (long long)max_pages * page_size;
  if (T_max >= (1ll << 31)) return GQA_ERR_UNSUPPORTED;
  KvWeightsArgs a;
  a.q = q;
  a.k = k_pages;
  a.lse = lse;
  a.w = weights;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.B = B;
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.S_q = S_q;
  a.T_max = (int)T_max;
  a.d_h = d_h;
  a.scale = scale;
  a.causal = causal;
  a.window = window;
  a.accumulate = accumulate;
  a.workspace = workspace;
  a.block_table = block_table;
  a.max_pages = max_pages;
  a.page_size = page_size;
  a.num_pages = num_pages;
  return kv_weights_impl(a, dtype, workspace_bytes, stream);
}

gqa_status kv_evict(const void* k_cache, const void* v_cache, void* k_out, void* v_out,
                    const float* weights, float* weights_out, int32_t* kept, int32_t* new_len,
                    const int32_t* kv_len, int B, int h_kv, int T_max, int T_out, int budget, int sink,
                    int recent, int d_h, gqa_dtype dtype, void* stream) {
  EvictArgs a;
  a.k = k_cache;
  a.v = v_cache;
  a.k_out = k_out;
  a.v_out = v_out;
  a.w = weights;
  a.w_out = weights_out;
  a.kept = kept;
  a.new_len = new_len;
  a.kv_len = kv_len;
  a.B = B;
  a.h_kv = h_kv;
  a.T_max = T_max;
  a.T_out = T_out;
  a.budget = budget;
  a.sink = sink;
  a.recent = recent;
  a.in_place = k_cache == k_out ? 1 : 0;
  if (B > 0 && h_kv > 0 && T_max > 0 && T_out > 0 && d_h > 0) {
    // in place both caches are, over the same rows; else no output overlaps an input or the other output
    const size_t row = (size_t)d_h * (dtype == GQA_BF16 ? 2 : 4);
    const size_t in = (size_t)B * h_kv * T_max * row, out = (size_t)B * h_kv * T_out * row;
    if (a.in_place ? v_cache != v_out || T_out != T_max
                   : overlap(k_cache, in, k_out, out) || overlap(v_cache, in, v_out, out))
      return GQA_ERR_INVALID_ARG;
    if (overlap(k_cache, in, v_out, out) || overlap(v_cache, in, k_out, out) || overlap(k_out, out, v_out, out))
      return GQA_ERR_INVALID_ARG;
  }
  return evict_impl(a, d_h, dtype, stream);
}

gqa_status kv_evict_paged(void* k_pages, void* v_pages, const int32_t* block_table,
                          const int32_t* block_table_out, const float* weights, float* weights_out,
                          int32_t* kept, int32_t* new_len, const int32_t* kv_len, int B, int h_kv,
                          int num_pages, int page_size, int max_pages, int max_pages_out, int budget,
                          int sink, int recent, int d_h, gqa_dtype dtype, void* stream) {
  if (!block_table || num_pages <= 0 || page_size <= 0 || max_pages <= 0) return GQA_ERR_INVALID_ARG;
  if (!block_table_out) max_pages_out = max_pages;
  if (max_pages_out <= 0) return GQA_ERR_INVALID_ARG;
  const long long T_max = (long long)max_pages * page_size, T_out = (long long)max_pages_out * page_size;
  if (T_max >= (1ll << 31) || T_out >= (1ll << 31)) return GQA_ERR_UNSUPPORTED;
  if (k_pages == v_pages) return GQA_ERR_INVALID_ARG;
  EvictArgs a;
  a.k = a.k_out = k_pages;
  a.v = a.v_out = v_pages;
  a.w = weights;
  a.w_out = weights_out;
  a.kept = kept;
  a.new_len = new_len;
  a.kv_len = kv_len;
  a.B = B;
  a.h_kv = h_kv;
  a.T_max = (int)T_max;
  a.T_out = (int)T_out;
  a.budget = budget;
  a.sink = sink;
  a.recent = recent;
  a.in_place = block_table_out ? 0 : 1;
  a.block_table = block_table;
  a.block_table_out = block_table_out ? block_table_out : block_table;
  a.max_pages = max_pages;
  a.max_pages_out = max_pages_out;
  a.page_size = page_size;
  a.num_pages = num_pages;
  return evict_impl(a, d_h, dtype, stream);
}

gqa_status gqa_decode_mod(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                          const int32_t* kv_len, const int32_t* q_pos, const gqa_score_mod* mod, int B,
                          int h_q, int h_kv, int T_max, int d_h, float scale, int window,
                          gqa_dtype dtype, void* workspace, size_t workspace_bytes, int num_splits,
                          void* stream) {
  return decode_impl(q, k_cache, v_cache, o, lse, kv_len, q_pos, B, h_q, h_kv, T_max, d_h, scale, window, dtype,
                     workspace, workspace_bytes, num_splits, stream, nullptr, 0, 0, 0, mod);
}

gqa_status gqa_decode_paged_mod(const void* q, const void* k_pages, const void* v_pages, void* o,
                                float* lse, const int32_t* kv_len, const int32_t* q_pos,
                                const int32_t* block_table, const gqa_score_mod* mod, int B, int h_q,
                                int h_kv, int num_pages, int page_size, int max_pages, int d_h,
                                float scale, int window, gqa_dtype dtype, void* workspace,
                                size_t workspace_bytes, int num_splits, void* stream) {
  if (!block_table || num_pages <= 0 || page_size <= 0 || max_pages <= 0) return GQA_ERR_INVALID_ARG;
  if (page_size % 16 != 0) return GQA_ERR_UNSUPPORTED;
  const long long T_max = (long long)max_pages * page_size;
  if (T_max >= (1ll << 31)) return GQA_ERR_UNSUPPORTED;
  return decode_impl(q, k_pages, v_pages, o, lse, kv_len, q_pos, B, h_q, h_kv, (int)T_max, d_h, scale, window,
                     dtype, workspace, workspace_bytes, num_splits, stream, block_table, max_pages, page_size,
                     num_pages, mod);
}

}  // extern "C"
