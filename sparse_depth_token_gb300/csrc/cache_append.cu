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

// Bound: memory. A token's (hq + 2 hkv) hd elements are read once and written once, the
// arithmetic (7 operations an element) is far below what that takes. So every thread moves
// two 16-byte vectors: V elements c .. c + V - 1 of a head and their rotation partners
// hd/2 further, LPH = hd / (2 V) lanes to a head, and a CTA holds as many tokens as fill
// about 256 threads, which keeps an SM's 2048 threads loading. The angles of a token are
// the same for all its heads: HD/2 threads compute them once into shared memory while the
// vectors are on their way.
template <typename T, int HD, bool FP8>
__global__ void __launch_bounds__(512, 3)
cache_append_kernel(const AppendArgs a, const __grid_constant__ Turns turns, int rows_per_cta) {
  constexpr int V = 16 / sizeof(T), LPH = HD / (2 * V), HALF = HD / 2;
  __shared__ float2 angle[8][HALF];
  const int heads = a.hq + 2 * a.hkv, units = heads * LPH;
  const int64_t m0 = (int64_t)blockIdx.x * rows_per_cta;
  const int rows = (int)min((int64_t)rows_per_cta, a.M - m0), total = rows * units;
  const xmod_kv_cache& c = a.cache;
  pdl_trigger();
  pdl_wait();

  for (int u0 = 0; u0 < total; u0 += blockDim.x) {
    const int u = u0 + threadIdx.x;
    const int lr = min(u, total - 1) / units, un = min(u, total - 1) % units;
    const int h = un / LPH, l = un % LPH;
    const int64_t m = m0 + lr;
    const bool is_q = h < a.hq, is_v = h >= a.hq + a.hkv;
    const int seq = a.seq ? a.seq[m] : (int)m, slot = a.slot[m];
    bool live = u < total && seq >= 0;
    if (live && (seq >= c.n_seqs || slot < 0 || slot >= c.max_pages * c.page_size)) {
      report_status(a.status, XMOD_ERR_DEVICE_CHECK);
      live = false;
    }
    const T* src = (const T*)a.qkv + m * a.ldqkv + (int64_t)h * HD + l * V;
    Vec16<T> lo, hi;
    lo.raw = hi.raw = make_uint4(0u, 0u, 0u, 0u);
    int page = 0;
    if (live) {
      page = c.table[(int64_t)seq * c.max_pages + slot / c.page_size];
      lo = ld_vec_stream(src);
      hi = ld_vec_stream(src + HALF);
    }
    if (u0 == 0 && a.rope) {
      for (int i = threadIdx.x; i < rows * HALF; i += blockDim.x) {
        const int64_t row = m0 + i / HALF;
        angle[i / HALF][i % HALF] =
            rotation(turns.f[i % HALF], a.pos ? a.pos[row] : a.slot[row]);
      }
    }
    if (u0 == 0) __syncthreads();
    if (live && (page < 0 || page >= c.n_pages)) {
      report_status(a.status, XMOD_ERR_DEVICE_CHECK);
      live = false;
    }
    float x[V], y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = lo.get(i);
      y[i] = hi.get(i);
    }
    if (a.q_gain || a.k_gain) {   // uniform: the shuffles need every lane
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const T* gain = is_v ? nullptr : (const T*)(is_q ? a.q_gain : a.k_gain);
      if (gain) {
        const float inv = rsqrtf(ss / (float)HD + a.eps);
        const Vec16<T> g0 = ld_vec(gain + l * V), g1 = ld_vec(gain + HALF + l * V);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          x[i] = x[i] * inv * g0.get(i);
          y[i] = y[i] * inv * g1.get(i);
        }
      }
    }
    if (a.rope && !is_v) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 cs = angle[lr][l * V + i];
        const float rx = x[i] * cs.x - y[i] * cs.y;
        y[i] = y[i] * cs.x + x[i] * cs.y;
        x[i] = rx;
      }
    }
    const int g = is_v ? h - a.hq - a.hkv : h - a.hq;
    const int64_t row = is_q ? 0 : ((int64_t)page * a.hkv + g) * c.page_size + slot % c.page_size;
    if constexpr (FP8) {
      float amax = 0.f;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        amax = fmaxf(amax, fmaxf(fabsf(x[i]), fabsf(y[i])));
        bad |= !(fabsf(x[i]) <= FLT_MAX) || !(fabsf(y[i]) <= FLT_MAX);
      }
      if (bad) amax = INFINITY;   // fmaxf passes over a NaN
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (live && !is_q) {
        float scale = amax / 448.0f;
        if (scale < FLT_MIN) scale = 0.0f;
        if (amax == INFINITY) scale = __int_as_float(0x7fc00000);
        uint32_t cx[V / 4], cy[V / 4];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          float2 p = make_float2(0.f, 0.f), q = p;
          if (!(scale == 0.0f)) {
            p = make_float2(x[2 * i] / scale, x[2 * i + 1] / scale);
            q = make_float2(y[2 * i] / scale, y[2 * i + 1] / scale);
          }
          const uint32_t px = __nv_cvt_float2_to_fp8x2(p, __NV_SATFINITE, __NV_E4M3);
          const uint32_t qx = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
          cx[i / 2] = i & 1 ? cx[i / 2] | px << 16 : px;
          cy[i / 2] = i & 1 ? cy[i / 2] | qx << 16 : qx;
        }
        uint8_t* dst = (uint8_t*)(is_v ? c.v : c.k) + row * HD + l * V;
        *reinterpret_cast<uint2*>(dst) = make_uint2(cx[0], cx[1]);
        *reinterpret_cast<uint2*>(dst + HALF) = make_uint2(cy[0], cy[1]);
        if (l == 0) (is_v ? c.v_scale : c.k_scale)[row] = scale;
        continue;
      }
    }
    if (live && (!is_q || a.q_out)) {
      T* dst = is_q ? (T*)a.q_out + m * a.ldq + (int64_t)h * HD
                    : (T*)(is_v ? c.v : c.k) + row * HD;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        lo.set(i, x[i]);
        hi.set(i, y[i]);
      }
      st_vec(dst + l * V, lo);
      st_vec(dst + l * V + HALF, hi);
    }
  }
}

template <typename T, int HD, bool FP8>
cudaError_t launch_append_hd(const Ctx& c, const AppendArgs& a, const Turns& turns) {
  const int units = (a.hq + 2 * a.hkv) * (HD / 2) / (16 / (int)sizeof(T));
  int rows = 256 / units;
  rows = rows < 1 ? 1 : rows > 8 ? 8 : rows;
  int threads = (rows * units + 31) / 32 * 32;
  if (threads > 512) threads = 512;
  return launch_pdl(cache_append_kernel<T, HD, FP8>, dim3((unsigned)((a.M + rows - 1) / rows)),
                    dim3(threads), 0, c.stream, a, turns, rows);
}

template <typename T, bool FP8>
cudaError_t launch_append(const Ctx& c, const AppendArgs& a, int hd, const Turns& turns) {
  if (hd == 128) return launch_append_hd<T, 128, FP8>(c, a, turns);
  if (hd == 64) return launch_append_hd<T, 64, FP8>(c, a, turns);
  return launch_append_hd<T, 32, FP8>(c, a, turns);
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
