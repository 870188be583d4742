// Attention of one query token per row over a paged key/value cache.

#include <cuda_fp8.h>
#include <math.h>

#include "cache.h"
#include "common.cuh"

namespace xmod {

namespace {

struct DecodeArgs {
  int M, hq, hkv, ldq;
  const void* q;
  const int32_t *seq, *len;
  void* o;
  float* lse;
  xmod_kv_cache cache;
  int* status;
};

template <typename T, bool FP8>
__device__ __forceinline__ float cache_value(const void* base, int64_t at) {
  if constexpr (FP8) {
    const __half_raw r = __nv_cvt_fp8_to_halfraw(((const uint8_t*)base)[at], __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&r));
  } else {
    return Elem<T>::to_f(((const T*)base)[at]);
  }
}

// One warp per (row, query head): the softmax's running maximum and sum over the keys in
// order; lane l holds dimensions l, l + 32, ...
template <typename T, int HD, bool FP8>
__global__ void __launch_bounds__(256) cache_attention_rows_kernel(DecodeArgs a) {
  constexpr int E = HD / 32;
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (item >= (int64_t)a.M * a.hq) return;
  const int m = (int)(item / a.hq), h = (int)(item % a.hq), g = h / (a.hq / a.hkv);
  const xmod_kv_cache& c = a.cache;
  const int seq = a.seq ? a.seq[m] : m;
  if (seq < 0) return;
  if (seq >= c.n_seqs) {
    if (lane == 0) report_status(a.status, XMOD_ERR_DEVICE_CHECK);
    return;
  }
  int n = a.len[m];
  if (n < 0 || n > c.max_pages * c.page_size) {
    if (lane == 0) report_status(a.status, XMOD_ERR_DEVICE_CHECK);
    n = n < 0 ? 0 : c.max_pages * c.page_size;
  }
  const T* qp = (const T*)a.q + (int64_t)m * a.ldq + (int64_t)h * HD;
  const float scale = rsqrtf((float)HD);
  float q[E], acc[E], top = -INFINITY, sum = 0.f;
  for (int e = 0; e < E; ++e) {
    q[e] = Elem<T>::to_f(qp[lane + 32 * e]) * scale;
    acc[e] = 0.f;
  }
  for (int i = 0; i < n; ++i) {
    int page = c.table[(int64_t)seq * c.max_pages + i / c.page_size];
    if (page < 0 || page >= c.n_pages) {
      if (lane == 0) report_status(a.status, XMOD_ERR_DEVICE_CHECK);
      page = 0;
    }
    const int64_t row = ((int64_t)page * a.hkv + g) * c.page_size + i % c.page_size;
    float s = 0.f;
    for (int e = 0; e < E; ++e)
      s = fmaf(q[e], cache_value<T, FP8>(c.k, row * HD + lane + 32 * e), s);
    s = warp_sum(s);
    float vs = 1.f;
    if (FP8) {
      s *= c.k_scale[row];
      vs = c.v_scale[row];
    }
    const float top2 = fmaxf(top, s);
    const float base = top2 == -INFINITY ? 0.f : top2;
    const float keep = expf(top - base), p = expf(s - base);
    top = top2;
    sum = sum * keep + p;
    for (int e = 0; e < E; ++e)
      acc[e] = acc[e] * keep + p * vs * cache_value<T, FP8>(c.v, row * HD + lane + 32 * e);
  }
  T* op = (T*)a.o + (int64_t)m * a.hq * HD + (int64_t)h * HD;
  for (int e = 0; e < E; ++e) op[lane + 32 * e] = Elem<T>::from_f(n ? acc[e] / sum : 0.f);
  if (a.lse && lane == 0) a.lse[(int64_t)m * a.hq + h] = n ? top + logf(sum) : -INFINITY;
}

template <typename T, bool FP8>
cudaError_t launch_rows(const Ctx& c, const DecodeArgs& a, int hd) {
  const dim3 grid((unsigned)(((int64_t)a.M * a.hq + 7) / 8));
  if (hd == 128) cache_attention_rows_kernel<T, 128, FP8><<<grid, 256, 0, c.stream>>>(a);
  else if (hd == 64) cache_attention_rows_kernel<T, 64, FP8><<<grid, 256, 0, c.stream>>>(a);
  else cache_attention_rows_kernel<T, 32, FP8><<<grid, 256, 0, c.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace xmod

using namespace xmod;

extern "C" {

size_t xmod_cache_attention_workspace_bytes(const xmod_dims* dm, int M) {
  if (!dims_ok(dm) || M < 0) return 0;
  return 256;
}

int xmod_cache_attention(const xmod_dims* dm, const xmod_kv_cache* cache, int M, const void* q,
                         int ldq, const int32_t* seq, const int32_t* len, void* o, float* lse,
                         void* ws, size_t ws_bytes, void* stream) {
  const int st = cache_status(dm, cache);
  if (st) return st;
  if (M < 0) return XMOD_ERR_INVALID_ARG;
  if (M == 0) return XMOD_OK;
  const int qw = dm->n_heads * dm->head_dim;
  if (!ptr16(q) || ldq < qw || ldq % 8 || !ptr4_or_null(seq) || !len || !ptr4_or_null(len) ||
      !ptr16(o) || !ptr4_or_null(lse))
    return XMOD_ERR_INVALID_ARG;
  if (!ptr16(ws) || ws_bytes < xmod_cache_attention_workspace_bytes(dm, M))
    return XMOD_ERR_WORKSPACE;
  DecodeArgs a{M, dm->n_heads, dm->n_kv_heads, ldq, q, seq, len, o, lse, *cache, (int*)ws};
  const Ctx c{(cudaStream_t)stream, (int*)ws};
  if (cache->format == XMOD_CACHE_E4M3)
    XMOD_LAUNCH(c, "cache_attention", (launch_rows<__nv_bfloat16, true>(c, a, dm->head_dim)));
  else if (dm->dtype == XMOD_BF16)
    XMOD_LAUNCH(c, "cache_attention", (launch_rows<__nv_bfloat16, false>(c, a, dm->head_dim)));
  else
    XMOD_LAUNCH(c, "cache_attention", (launch_rows<float, false>(c, a, dm->head_dim)));
  return XMOD_OK;
}

}  // extern "C"
