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

// (cos, sin) of pos * f turns: the nearest quarter turn and a remainder r of at most pi/4,
// by the series of sine (to r^9 / 9!, off by 2e-9) and cosine (to r^8 / 8!, off by 3e-8).
__device__ __forceinline__ float2 rotation(uint64_t f, int pos) {
  const uint32_t turn = (uint32_t)((f * (uint64_t)(int64_t)pos) >> 32);
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const float r = (float)(int32_t)(turn - (quarter << 30)) * 1.4629180792671596e-9f;   // 2 pi / 2^32
  const float r2 = r * r;
  float s = fmaf(r2, 2.7557319e-6f, -1.9841270e-4f);
  s = fmaf(s, r2, 8.3333333e-3f);
  s = fmaf(s, r2, -1.6666667e-1f);
  s = fmaf(s * r2, r, r);
  float c = fmaf(r2, 2.4801587e-5f, -1.3888889e-3f);
  c = fmaf(c, r2, 4.1666667e-2f);
  c = fmaf(c, r2, -0.5f);
  c = fmaf(c, r2, 1.0f);
  float2 cs = quarter & 1 ? make_float2(s, c) : make_float2(c, s);
  // quarters 1 and 2 have a negative cosine, 2 and 3 a negative sine
  if ((quarter + 1) & 2) cs.x = -cs.x;
  if (quarter & 2) cs.y = -cs.y;
  return cs;
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

// Bound: memory, once the instructions are few enough. A token's (hq + 2 hkv) hd elements
// are read once and written once. One warp takes a token (small batches: a part of its
// heads) by itself, without shared memory or barriers. A lane moves two 16-byte vectors of
// a head, elements c .. c + V - 1 and their rotation partners hd/2 further, LPH = hd / (2 V)
// lanes to a head, HPW heads of one kind (q, k or v) a pass, four passes' loads together
// (4 KB a warp). The angles are the same for all heads: every lane computes the 1 or 2 of
// the hd/2 that it owns, once per token, and gets its V by shuffles. The arithmetic runs on
// pairs of fp32; v is copied as it is. Warps stay for many tokens; the next token's
// sequence, slot, position and page are fetched a token ahead.
constexpr int kPasses = 4;        // passes whose loads are in flight together
constexpr int kAppendWarps = 4;
constexpr int kAppendCtas = 24;   // CTAs per SM the grid is limited to

template <typename T, int HD, bool FP8>
__global__ void __launch_bounds__(kAppendWarps * 32)
cache_append_kernel(const AppendArgs a, const __grid_constant__ Turns turns, int chunk) {
  constexpr int V = 16 / sizeof(T), LPH = HD / (2 * V), HALF = HD / 2, HPW = 32 / LPH;
  constexpr int NJ = V > HPW ? V / HPW : 1;   // angles a lane computes
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPH, hl = lane / LPH;
  const int q_passes = (a.hq + HPW - 1) / HPW, kv_passes = (a.hkv + HPW - 1) / HPW;
  // passes: the q heads', the k heads', the v heads'; this warp's are [first, last)
  const int first = max((int)blockIdx.y * chunk, a.q_out ? 0 : q_passes);
  const int last = min(((int)blockIdx.y + 1) * chunk, q_passes + 2 * kv_passes);
  const bool rope = a.rope && first < q_passes + kv_passes;
  const xmod_kv_cache& c = a.cache;
  const int room = c.max_pages * c.page_size;
  const int step = gridDim.x * kAppendWarps;
  // this lane's angles: pairs l V + i, i = hl + HPW j; pair i of a lane comes from lane
  // l + LPH (i % HPW)
  uint64_t freq[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) freq[j] = turns.f[l * V + (hl + HPW * j) % V];
  pdl_trigger();
  pdl_wait();

  struct Where {
    int seq, slot, pos, page;
  };
  auto locate = [&](int64_t m, Where& w) {
    w.seq = -1;
    if (m >= a.M) return;
    w.seq = a.seq ? a.seq[m] : (int)m;
    w.slot = a.slot[m];
    w.pos = a.pos ? a.pos[m] : w.slot;
  };
  auto find_page = [&](Where& w) {   // the page of a row to append, -1: skip the row
    w.page = -1;
    if (w.seq < 0) return;
    if (w.seq < c.n_seqs && w.slot >= 0 && w.slot < room)
      w.page = c.table[(int64_t)w.seq * c.max_pages + w.slot / c.page_size];
    if (w.page >= c.n_pages) w.page = -1;
    if (w.page < 0) {
      report_status(a.status, XMOD_ERR_DEVICE_CHECK);
      w.page = -1;
    }
  };

  int64_t m = (int64_t)blockIdx.x * kAppendWarps + warp;
  Where now, next;
  locate(m, now);
  find_page(now);
  for (; m < a.M; m += step) {
    locate(m + step, next);
    if (now.page >= 0) {   // the same for the whole warp
      const T* src = (const T*)a.qkv + m * a.ldqkv + l * V;
      const int64_t page_row = (int64_t)now.page * a.hkv * c.page_size + now.slot % c.page_size;
      float2 cs[V / 2], sn[V / 2];
      for (int p0 = first; p0 < last; p0 += kPasses) {
        uint4 lo[kPasses], hi[kPasses];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int p = p0 + i;
          const int kind = p < q_passes ? 0 : p < q_passes + kv_passes ? 1 : 2;
          const int h = (kind == 0 ? p : p - q_passes - (kind - 1) * kv_passes) * HPW + hl;
          const int col = kind == 0 ? 0 : a.hq + (kind - 1) * a.hkv;
          lo[i] = hi[i] = make_uint4(0u, 0u, 0u, 0u);
          if (p < last && h < (kind == 0 ? a.hq : a.hkv)) {
            lo[i] = __ldcs(reinterpret_cast<const uint4*>(src + (col + h) * HD));
            hi[i] = __ldcs(reinterpret_cast<const uint4*>(src + (col + h) * HD + HALF));
          }
        }
        if (rope && p0 == first) {
          float2 own[NJ];
#pragma unroll
          for (int j = 0; j < NJ; ++j) own[j] = rotation(freq[j], now.pos);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float x = __shfl_sync(0xffffffffu, own[i / HPW].x, l + LPH * (i % HPW));
            const float y = __shfl_sync(0xffffffffu, own[i / HPW].y, l + LPH * (i % HPW));
            if (i & 1) {
              cs[i / 2].y = x;
              sn[i / 2].y = y;
            } else {
              cs[i / 2].x = x;
              sn[i / 2].x = y;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int p = p0 + i;
          if (p >= last) break;
          const int kind = p < q_passes ? 0 : p < q_passes + kv_passes ? 1 : 2;
          const int h = (kind == 0 ? p : p - q_passes - (kind - 1) * kv_passes) * HPW + hl;
          const bool live = h < (kind == 0 ? a.hq : a.hkv);
          const T* gain = (const T*)(kind == 0 ? a.q_gain : kind == 1 ? a.k_gain : nullptr);
          T* dst;   // of the head's vectors, in q_out or a native cache
          int64_t row = 0;
          if (kind == 0) {
            dst = (T*)a.q_out + m * a.ldq + h * HD + l * V;
          } else {
            row = page_row + (int64_t)h * c.page_size;
            dst = (T*)(kind == 2 ? c.v : c.k) + row * HD + l * V;
          }
          if (kind == 2 && !FP8) {
            if (live) {
              *reinterpret_cast<uint4*>(dst) = lo[i];
              *reinterpret_cast<uint4*>(dst + HALF) = hi[i];
            }
            continue;
          }
          float2 x[V / 2], y[V / 2];
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            x[e] = vec_pair<T>(lo[i], e);
            y[e] = vec_pair<T>(hi[i], e);
          }
          if (gain) {
            float2 ss = mul2(x[0], x[0]);
#pragma unroll
            for (int e = 1; e < V / 2; ++e) ss = fma2(x[e], x[e], ss);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) ss = fma2(y[e], y[e], ss);
            float sum = ss.x + ss.y;
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float inv = rsqrtf(fmaf(sum, 1.0f / (float)HD, a.eps));
            const float2 inv2 = make_float2(inv, inv);
            const uint4 g0 = *reinterpret_cast<const uint4*>(gain + l * V);
            const uint4 g1 = *reinterpret_cast<const uint4*>(gain + HALF + l * V);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
              x[e] = mul2(mul2(x[e], inv2), vec_pair<T>(g0, e));
              y[e] = mul2(mul2(y[e], inv2), vec_pair<T>(g1, e));
            }
          }
          if (rope && kind != 2) {
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
              const float2 neg = make_float2(-sn[e].x, -sn[e].y);
              const float2 rx = fma2(y[e], neg, mul2(x[e], cs[e]));
              y[e] = fma2(x[e], sn[e], mul2(y[e], cs[e]));
              x[e] = rx;
            }
          }
          if (FP8 && kind != 0) {
            if constexpr (FP8) {
              float amax = 0.f;
              bool bad = false;
#pragma unroll
              for (int e = 0; e < V / 2; ++e) {
                const float big = fmaxf(fmaxf(fabsf(x[e].x), fabsf(x[e].y)),
                                        fmaxf(fabsf(y[e].x), fabsf(y[e].y)));
                amax = fmaxf(amax, big);   // passes over a NaN
                bad |= x[e].x != x[e].x || x[e].y != x[e].y || y[e].x != y[e].x || y[e].y != y[e].y;
              }
              if (bad) amax = INFINITY;
#pragma unroll
              for (int o = LPH / 2; o > 0; o >>= 1)
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
              float scale = amax / 448.0f;
              if (scale < FLT_MIN) scale = 0.0f;
              if (amax == INFINITY) scale = __int_as_float(0x7fc00000);
              const float inv = scale == 0.0f ? 0.0f : 1.0f / scale;   // NaN stays
              const float2 inv2 = make_float2(inv, inv);
              uint32_t cx[V / 4], cy[V / 4];
#pragma unroll
              for (int e = 0; e < V / 2; ++e) {
                const uint32_t sx =
                    __nv_cvt_float2_to_fp8x2(mul2(x[e], inv2), __NV_SATFINITE, __NV_E4M3);
                const uint32_t sy =
                    __nv_cvt_float2_to_fp8x2(mul2(y[e], inv2), __NV_SATFINITE, __NV_E4M3);
                cx[e / 2] = e & 1 ? cx[e / 2] | sx << 16 : sx;
                cy[e / 2] = e & 1 ? cy[e / 2] | sy << 16 : sy;
              }
              if (live) {
                uint8_t* codes = (uint8_t*)(kind == 2 ? c.v : c.k) + row * HD + l * V;
                *reinterpret_cast<uint2*>(codes) = make_uint2(cx[0], cx[1]);
                *reinterpret_cast<uint2*>(codes + HALF) = make_uint2(cy[0], cy[1]);
                if (l == 0) (kind == 2 ? c.v_scale : c.k_scale)[row] = scale;
              }
            }
          } else if (live) {
            uint4 w0, w1;
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
              set_vec_pair<T>(w0, e, x[e]);
              set_vec_pair<T>(w1, e, y[e]);
            }
            *reinterpret_cast<uint4*>(dst) = w0;
            *reinterpret_cast<uint4*>(dst + HALF) = w1;
          }
        }
      }
    }
    now = next;
    if (m + step < a.M) find_page(now);
  }
}

template <typename T, int HD, bool FP8>
cudaError_t launch_append_hd(const Ctx& c, const AppendArgs& a, const Turns& turns) {
  constexpr int HPW = 32 / (HD / 2 / (16 / (int)sizeof(T)));
  const int total = (a.hq + HPW - 1) / HPW + 2 * ((a.hkv + HPW - 1) / HPW);
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // Passes a warp does of a token: all of them (the angles once) when the tokens alone fill
  // the GPU, one while even single passes leave it empty (latency), four in between.
  const int64_t M = a.M;
  const int chunk = M * total <= (int64_t)sms * 8 ? 1 : M < (int64_t)sms * 32 && total > 4 ? 4 : total;
  const int chunks = (total + chunk - 1) / chunk;
  const int64_t ctas = (M + kAppendWarps - 1) / kAppendWarps;
  const int64_t most = ((int64_t)sms * kAppendCtas + chunks - 1) / chunks;
  return launch_pdl(cache_append_kernel<T, HD, FP8>,
                    dim3((unsigned)(ctas < most ? ctas : most), chunks), dim3(kAppendWarps * 32), 0,
                    c.stream, a, turns, chunk);
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
