// Log probabilities of given tokens with the entropy and the largest alternatives, and
// their gradient at the logits.

#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace xmod {

namespace {

struct LogprobArgs {
  int V, top_k;
  int64_t ld;
  const void* logits;
  const int32_t* target;
  float *logp, *entropy, *lse;
  int32_t* top_idx;
  float* top_logp;
  int* status;
};

// Order of two logits as unsigned keys: larger value, larger key; -0 equals +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  if (x != x) return 0xffffffffu;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One block per row.
template <typename T>
__global__ void __launch_bounds__(256) token_logprobs_rows_kernel(LogprobArgs a) {
  __shared__ float red[8];
  __shared__ unsigned long long best_s[8];
  const int64_t n = blockIdx.x;
  const T* x = (const T*)a.logits + n * a.ld;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float m = -INFINITY;
  bool bad = false;
  for (int v = tid; v < a.V; v += 256) {
    const float f = Elem<T>::to_f(x[v]);
    m = fmaxf(m, f);
    bad |= !(f < INFINITY);   // NaN or +infinity
  }
  m = warp_max(m);
  if (lane == 0) red[warp] = m;
  bad = __syncthreads_or(bad);
  for (int i = 0; i < 8; ++i) m = fmaxf(m, red[i]);
  __syncthreads();
  bad |= m == -INFINITY;
  float l = 0.f, u = 0.f;
  for (int v = tid; v < a.V; v += 256) {
    const float y = Elem<T>::to_f(x[v]) - m, e = expf(y);
    l += e;
    if (e > 0.f) u = fmaf(e, y, u);
  }
  l = warp_sum(l);
  if (lane == 0) red[warp] = l;
  __syncthreads();
  l = 0.f;
  for (int i = 0; i < 8; ++i) l += red[i];
  __syncthreads();
  u = warp_sum(u);
  if (lane == 0) red[warp] = u;
  __syncthreads();
  u = 0.f;
  for (int i = 0; i < 8; ++i) u += red[i];
  const float nan = __int_as_float(0x7fc00000);
  const float ll = logf(l);
  if (tid == 0) {
    if (bad) report_status(a.status, XMOD_ERR_DEVICE_CHECK);
    if (a.lse) a.lse[n] = bad ? nan : m + ll;
    if (a.entropy) a.entropy[n] = bad ? nan : ll - u / l;
    if (a.logp) {
      const int t = a.target[n];
      if (t >= a.V) report_status(a.status, XMOD_ERR_DEVICE_CHECK);
      a.logp[n] = t < 0 ? 0.f : bad || t >= a.V ? nan : (Elem<T>::to_f(x[t]) - m) - ll;
    }
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < a.top_k; ++k) {
    unsigned long long best = 0;
    for (int v = tid; v < a.V; v += 256) {
      const unsigned long long key =
          ((unsigned long long)order_key(Elem<T>::to_f(x[v])) << 32) | (0xffffffffu - (uint32_t)v);
      if (key < last && key > best) best = key;
    }
    for (int o = 16; o; o >>= 1) {
      const unsigned long long other = __shfl_xor_sync(0xffffffffu, best, o);
      best = other > best ? other : best;
    }
    if (lane == 0) best_s[warp] = best;
    __syncthreads();
    for (int i = 0; i < 8; ++i) best = best_s[i] > best ? best_s[i] : best;
    __syncthreads();
    last = best;
    const int v = (int)(0xffffffffu - (uint32_t)best);
    if (tid == 0) {
      a.top_idx[n * a.top_k + k] = v;
      a.top_logp[n * a.top_k + k] = bad ? nan : (Elem<T>::to_f(x[v]) - m) - ll;
    }
  }
}

struct LogprobBwdArgs {
  int V;
  int64_t ld, ldd;
  const void* logits;
  const int32_t* target;
  const float *lse, *entropy, *g_logp, *g_entropy;
  void* dlogits;
  int* status;
};

template <typename T>
__global__ void __launch_bounds__(256) token_logprobs_bwd_kernel(LogprobBwdArgs a) {
  const int64_t n = blockIdx.x;
  const T* x = (const T*)a.logits + n * a.ld;
  T* d = (T*)a.dlogits + n * a.ldd;
  int t = a.g_logp ? a.target[n] : -1;
  if (t >= a.V) {
    if (threadIdx.x == 0) report_status(a.status, XMOD_ERR_DEVICE_CHECK);
    t = -1;
  }
  const float g = t >= 0 ? a.g_logp[n] : 0.f, gh = a.g_entropy ? a.g_entropy[n] : 0.f;
  const float lse = a.lse[n], ent = a.g_entropy ? a.entropy[n] : 0.f;
  for (int v = threadIdx.x; v < a.V; v += 256) {
    float r = 0.f;
    if (g != 0.f || gh != 0.f) {
      const float y = Elem<T>::to_f(x[v]) - lse, p = expf(y);
      r = -p * (p > 0.f ? fmaf(gh, y + ent, g) : g);
      if (v == t) r += g;
    }
    d[v] = Elem<T>::from_f(r);
  }
}

bool ptr16(const void* p) { return p && ((uintptr_t)p & 15u) == 0; }
bool ptr4_or_null(const void* p) { return ((uintptr_t)p & 3u) == 0; }

}  // namespace
}  // namespace xmod

using namespace xmod;

extern "C" {

int xmod_token_logprobs(xmod_dtype dt, int64_t N, int V, const void* logits, int64_t ld,
                        const int32_t* target, float* logp, float* entropy, float* lse, int top_k,
                        int32_t* top_idx, float* top_logp, int* status_out, void* stream) {
  if ((dt != XMOD_BF16 && dt != XMOD_FP32) || N < 0 || V <= 0 || ld < V || top_k < 0)
    return XMOD_ERR_INVALID_ARG;
  if (top_k > V || (top_k > 0) != (top_idx != nullptr) || (top_k > 0) != (top_logp != nullptr) ||
      (target != nullptr) != (logp != nullptr))
    return XMOD_ERR_INVALID_ARG;
  if (N == 0) return XMOD_OK;
  if (!ptr16(logits)) return XMOD_ERR_INVALID_ARG;
  const void* ps[] = {target, logp, entropy, lse, top_idx, top_logp, status_out};
  for (const void* p : ps)
    if (!ptr4_or_null(p)) return XMOD_ERR_INVALID_ARG;
  if (top_k > XMOD_MAX_TOP_K || N > INT32_MAX) return XMOD_ERR_UNSUPPORTED;
  const LogprobArgs a{V, top_k, ld, logits, target, logp, entropy, lse, top_idx, top_logp,
                      status_out};
  const Ctx c{(cudaStream_t)stream, status_out};
  if (dt == XMOD_BF16)
    token_logprobs_rows_kernel<__nv_bfloat16><<<(unsigned)N, 256, 0, c.stream>>>(a);
  else
    token_logprobs_rows_kernel<float><<<(unsigned)N, 256, 0, c.stream>>>(a);
  XMOD_LAUNCH(c, "token_logprobs", cudaGetLastError());
  return XMOD_OK;
}

int xmod_token_logprobs_bwd(xmod_dtype dt, int64_t N, int V, const void* logits, int64_t ld,
                            const int32_t* target, const float* lse, const float* entropy,
                            const float* g_logp, const float* g_entropy, void* dlogits,
                            int64_t ldd, int* status_out, void* stream) {
  if ((dt != XMOD_BF16 && dt != XMOD_FP32) || N < 0 || V <= 0 || ld < V || ldd < V)
    return XMOD_ERR_INVALID_ARG;
  if (N == 0) return XMOD_OK;
  if (!ptr16(logits) || !ptr16(dlogits) || !lse || (g_logp && !target) ||
      (g_entropy && !entropy) || (dlogits == logits && ldd != ld))
    return XMOD_ERR_INVALID_ARG;
  const void* ps[] = {target, lse, entropy, g_logp, g_entropy, status_out};
  for (const void* p : ps)
    if (!ptr4_or_null(p)) return XMOD_ERR_INVALID_ARG;
  if (N > INT32_MAX) return XMOD_ERR_UNSUPPORTED;
  const LogprobBwdArgs a{V, ld, ldd, logits, target, lse, entropy, g_logp, g_entropy, dlogits,
                         status_out};
  const Ctx c{(cudaStream_t)stream, status_out};
  if (dt == XMOD_BF16)
    token_logprobs_bwd_kernel<__nv_bfloat16><<<(unsigned)N, 256, 0, c.stream>>>(a);
  else
    token_logprobs_bwd_kernel<float><<<(unsigned)N, 256, 0, c.stream>>>(a);
  XMOD_LAUNCH(c, "token_logprobs_bwd", cudaGetLastError());
  return XMOD_OK;
}

}  // extern "C"
