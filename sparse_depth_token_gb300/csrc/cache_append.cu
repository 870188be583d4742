// Appending new tokens to a paged key/value cache: QK-norm and rotary embedding of the
// projections q | k | v on the way, k and v to their slots (bf16, fp32, or e4m3 codes with
// one scale per slot and head), q to the caller.

#include <cuda_fp8.h>
#include <float.h>
#include <math.h>

#include "cache.h"
#include "common.cuh"

namespace xmod {

namespace {

// Rotation angle of pair c at position pos, in turns: pos * f[c] modulo 1, f[c] =
// theta^(-2c/hd) / 2 pi as a 64-bit binary fraction. The product wraps at whole turns by
// itself, so the angle is as exact at position 2^31 as at 1 (f's own error, 2^-53 relative,
// is 2e-7 turns there), without double arithmetic on the device.
struct Turns {
  uint64_t f[64];
};

void make_turns(float theta, int hd, Turns& t) {
  constexpr double kInvTwoPi = 0.15915494309189535;
  double coarse[8], fine[8];   // theta^(-2c/hd), c = 8 i + j: two short tables of powers
  const double lg = -2.0 * log2((double)theta) / hd;
  for (int i = 0; i < 8; ++i) {
    coarse[i] = exp2(8 * i * lg) * kInvTwoPi;
    fine[i] = exp2(i * lg);
  }
  for (int c = 0; c < hd / 2; ++c) {
    const double r = coarse[c >> 3] * fine[c & 7];
    t.f[c] = (uint64_t)((r - floor(r)) * 18446744073709551616.0);
  }
}

__device__ __forceinline__ float2 rotation(uint64_t f, int pos) {
  const uint64_t turn = f * (uint64_t)(int64_t)pos;
  // the top 32 bits as a signed half-turn count in [-1, 1)
  const float half = (float)(int32_t)(turn >> 32) * 4.656612873077393e-10f;
  float2 r;
  sincospif(half, &r.y, &r.x);
  return r;
}

struct AppendArgs {
  int M, hq, hkv, ldqkv, ldq;
  const void *qkv, *q_gain, *k_gain;
  void* q_out;
  const int32_t *seq, *slot, *pos;
  xmod_kv_cache cache;
  float eps;
  bool rope;
  int* status;
};

// One warp per (row, head); lane l holds dimensions l, l + 32, ...
template <typename T, int HD, bool FP8>
__global__ void __launch_bounds__(256) cache_append_kernel(AppendArgs a, Turns turns) {
  constexpr int E = HD / 32;
  const int heads = a.hq + 2 * a.hkv;
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (item >= (int64_t)a.M * heads) return;
  const int m = (int)(item / heads), h = (int)(item % heads);
  const int seq = a.seq ? a.seq[m] : m;
  if (seq < 0) return;
  const int slot = a.slot[m];
  const xmod_kv_cache& c = a.cache;
  if (seq >= c.n_seqs || slot < 0 || slot >= c.max_pages * c.page_size) {
    if (lane == 0) report_status(a.status, XMOD_ERR_DEVICE_CHECK);
    return;
  }
  const int page = c.table[(int64_t)seq * c.max_pages + slot / c.page_size];
  if (page < 0 || page >= c.n_pages) {
    if (lane == 0) report_status(a.status, XMOD_ERR_DEVICE_CHECK);
    return;
  }
  const bool is_q = h < a.hq, is_v = h >= a.hq + a.hkv;
  if (is_q && !a.q_out) return;
  const T* src = (const T*)a.qkv + (int64_t)m * a.ldqkv + (int64_t)h * HD;
  float v[E];
  for (int e = 0; e < E; ++e) v[e] = Elem<T>::to_f(src[lane + 32 * e]);
  const T* gain = is_v ? nullptr : (const T*)(is_q ? a.q_gain : a.k_gain);
  if (gain) {
    float ss = 0.f;
    for (int e = 0; e < E; ++e) ss = fmaf(v[e], v[e], ss);
    const float inv = rsqrtf(warp_sum(ss) / (float)HD + a.eps);
    for (int e = 0; e < E; ++e) v[e] = v[e] * inv * Elem<T>::to_f(gain[lane + 32 * e]);
  }
  if (a.rope && !is_v) {
    const int pos = a.pos ? a.pos[m] : slot;
    for (int e = 0; e < E; ++e) {
      const int d = lane + 32 * e, c2 = d % (HD / 2);
      const float2 cs = rotation(turns.f[c2], pos);
      float other;
      if (HD == 32) {
        other = __shfl_xor_sync(0xffffffffu, v[e], 16);
        v[e] = d < HD / 2 ? v[e] * cs.x - other * cs.y : v[e] * cs.x + other * cs.y;
      } else if (e < E / 2) {
        other = v[(e + E / 2) % E];
        const float lo = v[e] * cs.x - other * cs.y, hi = other * cs.x + v[e] * cs.y;
        v[e] = lo;
        v[(e + E / 2) % E] = hi;
      }
    }
  }
  if (is_q) {
    T* dst = (T*)a.q_out + (int64_t)m * a.ldq + (int64_t)h * HD;
    for (int e = 0; e < E; ++e) dst[lane + 32 * e] = Elem<T>::from_f(v[e]);
    return;
  }
  const int g = is_v ? h - a.hq - a.hkv : h - a.hq;
  const int64_t row = ((int64_t)page * a.hkv + g) * c.page_size + slot % c.page_size;
  if constexpr (FP8) {
    float amax = 0.f;
    bool bad = false;
    for (int e = 0; e < E; ++e) {
      amax = fmaxf(amax, fabsf(v[e]));
      bad |= !(fabsf(v[e]) <= FLT_MAX);
    }
    bad = __any_sync(0xffffffffu, bad);
    float scale = warp_max(amax) / 448.0f;
    if (scale < FLT_MIN) scale = 0.0f;
    if (bad) scale = __int_as_float(0x7fc00000);
    uint8_t* dst = (uint8_t*)(is_v ? c.v : c.k) + row * HD;
    for (int e = 0; e < E; ++e) {
      const float x = bad ? scale : scale > 0.0f ? v[e] / scale : 0.0f;
      dst[lane + 32 * e] = (uint8_t)__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
    }
    if (lane == 0) (is_v ? c.v_scale : c.k_scale)[row] = scale;
  } else {
    T* dst = (T*)(is_v ? c.v : c.k) + row * HD;
    for (int e = 0; e < E; ++e) dst[lane + 32 * e] = Elem<T>::from_f(v[e]);
  }
}

template <typename T, bool FP8>
cudaError_t launch_append(const Ctx& c, const AppendArgs& a, int hd, const Turns& turns) {
  const int64_t items = (int64_t)a.M * (a.hq + 2 * a.hkv);
  const dim3 grid((unsigned)((items + 7) / 8));
  if (hd == 128) cache_append_kernel<T, 128, FP8><<<grid, 256, 0, c.stream>>>(a, turns);
  else if (hd == 64) cache_append_kernel<T, 64, FP8><<<grid, 256, 0, c.stream>>>(a, turns);
  else cache_append_kernel<T, 32, FP8><<<grid, 256, 0, c.stream>>>(a, turns);
  return cudaGetLastError();
}

}  // namespace
}  // namespace xmod

using namespace xmod;

extern "C" {

int xmod_cache_append(const xmod_dims* dm, const xmod_kv_cache* cache, int M, const void* qkv,
                      int ldqkv, const xmod_layer_weights* w, const int32_t* seq,
                      const int32_t* slot, const int32_t* pos, void* q_out, int ldq,
                      int* status_out, void* stream) {
  const int st = cache_status(dm, cache);
  if (st) return st;
  if (M < 0) return XMOD_ERR_INVALID_ARG;
  if (M == 0) return XMOD_OK;
  const int qw = dm->n_heads * dm->head_dim, kw = dm->n_kv_heads * dm->head_dim;
  if (!ptr16(qkv) || ldqkv < qw + 2 * kw || ldqkv % 8 || !slot || !ptr4_or_null(slot) ||
      !ptr4_or_null(seq) || !ptr4_or_null(pos) || !ptr4_or_null(status_out))
    return XMOD_ERR_INVALID_ARG;
  if (q_out && (!ptr16(q_out) || ldq < qw || ldq % 8)) return XMOD_ERR_INVALID_ARG;
  if (q_out == qkv && ldq != ldqkv) return XMOD_ERR_INVALID_ARG;
  if (w && (!ptr16_or_null(w->q_norm) || !ptr16_or_null(w->k_norm) || !isfinite(w->rope_theta) ||
            w->rope_theta < 0.0f))
    return XMOD_ERR_INVALID_ARG;
  AppendArgs a{};
  a.M = M;
  a.hq = dm->n_heads;
  a.hkv = dm->n_kv_heads;
  a.ldqkv = ldqkv;
  a.ldq = ldq;
  a.qkv = qkv;
  a.q_gain = w ? w->q_norm : nullptr;
  a.k_gain = w ? w->k_norm : nullptr;
  a.q_out = q_out;
  a.seq = seq;
  a.slot = slot;
  a.pos = pos;
  a.cache = *cache;
  a.eps = dm->rms_eps;
  a.rope = w && w->rope_theta > 0.0f;
  a.status = status_out;
  Turns turns{};
  if (a.rope) make_turns(w->rope_theta, dm->head_dim, turns);
  const Ctx c{(cudaStream_t)stream, status_out};
  if (cache->format == XMOD_CACHE_E4M3)
    XMOD_LAUNCH(c, "cache_append",
                (launch_append<__nv_bfloat16, true>(c, a, dm->head_dim, turns)));
  else if (dm->dtype == XMOD_BF16)
    XMOD_LAUNCH(c, "cache_append",
                (launch_append<__nv_bfloat16, false>(c, a, dm->head_dim, turns)));
  else
    XMOD_LAUNCH(c, "cache_append", (launch_append<float, false>(c, a, dm->head_dim, turns)));
  return XMOD_OK;
}

}  // extern "C"
