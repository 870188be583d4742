// Appending new tokens to a paged key/value cache: QK-norm and rotary embedding of the
// projections q | k | v on the way, k and v to their slots (bf16, fp32, or e4m3 codes with
// one scale per slot and head), q to the caller.

#include <cuda_fp8.h>
#include <float.h>
#include <math.h>

#include "cache.h"
#include "common.cuh"
#include "rotary.cuh"

namespace xmod {

namespace {

// Rotation angle of pair c at position pos, in turns: pos * f[c] modulo 1, f[c] =
// theta^(-2c/hd) / 2 pi as a 64-bit binary fraction. The product wraps at whole turns by
// itself, without double arithmetic on the device; what is left is f's own error, that of
// double arithmetic: below 2^-52 turns for theta >= 1 (a power's relative error is
// 2^-52 (1.1 E + 3.5) at size 2^-E / 2 pi). The angle is off by pos times that: below fp32's
// half step up to position 2^24, by 5e-7 turns (3e-6 radians) at most at 2^31.
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

struct AppendArgs {
  int M, hq, hkv, ldqkv, ldq;
  const void *qkv, *q_gain, *k_gain;
  void* q_out;
  const int32_t *seq, *slot, *pos;
  xmod_kv_cache cache;
  float eps;
  int page_shift;   // log2 of the page size, -1: not a power of two
  bool rope;
  int* status;
};

// Bound: memory, once the instructions are few enough (a token's elements are read once and
// written once, with 7 operations each). A warp takes tokens by itself, without barriers,
// and of every token the same part: up to four passes over the q heads,
// or one or two over the k heads with the v heads beside them. What depends on the heads
// (columns, gains, this lane's frequencies) is then set up once per warp. A lane moves two
// 16-byte vectors of a head, elements c .. c + V - 1 and their rotation partners hd/2
// further, LPH = hd / (2 V) lanes to a head, HPW heads a pass. The vectors come by
// asynchronous copies into the lane's own places in shared memory, two tokens ahead, so that
// loads are in flight all the time and cost no registers (loading into registers, a token at
// a time, left the memory idle while a token was transformed: 87 us where this took 63).
// The angles are the same for all heads: every lane computes the 1 or 2 of the hd/2 that it
// owns, once per token, and gets its V by shuffles. The arithmetic runs on pairs of fp32; v
// is copied as it is. Sequence, slot and position are fetched three tokens ahead, the page
// one (and looked at only when its token's turn comes: 64 us with a check as it is fetched).
// Measured: 32768 tokens of 12 q and 4 KV heads of 128, bf16 (336 MB): 58 us, 5.8 TB/s, 0.85
// of what a copy reaches, fp32 (672 MB) 134 us; 5003 tokens of 32 and 8 heads to e4m3 (99 MB):
// 22.5 us, with neither memory (32 %) nor issue (35 %) full: 122 registers leave four CTAs an SM,
// too few to hide their latencies; 8 tokens: 2.0 us.
constexpr int kQPasses = 4, kKvPasses = 2;
constexpr int kAppendWarps = 4;
// CTAs per SM the grid is limited to: four are resident, twice as many even out the parts'
// lengths. In us at 4, 8, 16 and 32: 32768 tokens of 12 q and 4 KV heads of 128, bf16 55.8, 58.0,
// 61.5, 67.8, to e4m3 59.8, 62.8, 67.2, 74.5, fp32 167, 134, 115, 115; 5003 tokens of 32 and 8
// heads, bf16 23.6, 20.8, 20.4, 22.7, to e4m3 24.7, 22.3, 22.7, 24.9, fp32 45.6, 38.6, 36.1, 35.7.
constexpr int kAppendCtas = 8;
constexpr int kAppendStages = 3;  // tokens of a warp in shared memory: one at work, two coming

template <typename T, int HD> struct AppendShape {
  static constexpr int V = 16 / sizeof(T), LPH = HD / (2 * V), HALF = HD / 2, HPW = 32 / LPH;
  static constexpr int NJ = V > HPW ? V / HPW : 1;   // angles a lane computes
};

__device__ __forceinline__ void copy16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}

struct Where {
  int seq, slot, pos, page;
};

// QK-norm (gain > 0 elements given) and rotation of a lane's vectors x, y.
template <typename T, int HD>
__device__ __forceinline__ void transform(float2 (&x)[AppendShape<T, HD>::V / 2],
                                          float2 (&y)[AppendShape<T, HD>::V / 2], bool norm,
                                          const uint4& g0, const uint4& g1, float eps, bool rope,
                                          const float2* cs, const float2* sn) {
  using S = AppendShape<T, HD>;
  if (norm) {
    float2 ss = mul2(x[0], x[0]);
#pragma unroll
    for (int e = 1; e < S::V / 2; ++e) ss = fma2(x[e], x[e], ss);
#pragma unroll
    for (int e = 0; e < S::V / 2; ++e) ss = fma2(y[e], y[e], ss);
    float sum = ss.x + ss.y;
#pragma unroll
    for (int o = S::LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = rsqrtf(fmaf(sum, 1.0f / (float)HD, eps));
    const float2 inv2 = make_float2(inv, inv);
#pragma unroll
    for (int e = 0; e < S::V / 2; ++e) {
      x[e] = mul2(mul2(x[e], inv2), vec_pair<T>(g0, e));
      y[e] = mul2(mul2(y[e], inv2), vec_pair<T>(g1, e));
    }
  }
  if (rope) {
#pragma unroll
    for (int e = 0; e < S::V / 2; ++e) {
      const float2 t = mul2(x[e], cs[e]);
      const float2 rx = make_float2(fmaf(-y[e].x, sn[e].x, t.x), fmaf(-y[e].y, sn[e].y, t.y));
      y[e] = fma2(x[e], sn[e], mul2(y[e], cs[e]));
      x[e] = rx;
    }
  }
}

template <typename T, int HD>
__device__ __forceinline__ void store_pair(T* dst, const float2* x, const float2* y) {
  using S = AppendShape<T, HD>;
  uint4 w0, w1;
#pragma unroll
  for (int e = 0; e < S::V / 2; ++e) {
    set_vec_pair<T>(w0, e, x[e]);
    set_vec_pair<T>(w1, e, y[e]);
  }
  *reinterpret_cast<uint4*>(dst) = w0;
  *reinterpret_cast<uint4*>(dst + S::HALF) = w1;
}

// e4m3 codes and scale of a head whose LPH lanes hold x, y (x and y may change).
template <int HD>
__device__ __forceinline__ void store_e4m3(uint8_t* dst, float* scale_at, bool live, bool writes_scale,
                                           float2* x, float2* y) {
  using S = AppendShape<__nv_bfloat16, HD>;
  float amax = 0.f;
  bool bad = false;
#pragma unroll
  for (int e = 0; e < S::V / 2; ++e) {
    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(x[e].x), fabsf(x[e].y)),
                             fmaxf(fabsf(y[e].x), fabsf(y[e].y))));   // passes over a NaN
    bad |= x[e].x != x[e].x || x[e].y != x[e].y || y[e].x != y[e].x || y[e].y != y[e].y;
  }
  if (bad) amax = INFINITY;
#pragma unroll
  for (int o = S::LPH / 2; o > 0; o >>= 1)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  float scale = amax / 448.0f;
  if (scale < FLT_MIN) scale = 0.0f;
  if (amax == INFINITY) scale = __int_as_float(0x7fc00000);
  // The quotients x / scale, rounded as fp32's division rounds them: bf16 values over a scale
  // often lie exactly between two codes, where a product with the rounded reciprocal took the
  // other code (0.05 % of normal values). The reciprocal in two parts gives a quotient q within
  // an ulp of x / scale; then q scale - x is exact, and q - (q scale - x) / scale rounds
  // correctly (P. Markstein, Computation of elementary functions on the IBM RISC System/6000
  // processor, IBM J. Res. Dev. 34, 1990). The values come in negated, and the reciprocal's
  // first part is rounded down, so that zeros keep their signs.
  // 5003 tokens of 32 and 8 heads: 22.5 us; by divisions 25.9, by the product alone 22.0.
  float by = scale;
  if (scale < 0x1p-64f) {   // values and scale enlarged, so that the remainder has its last bits
    by *= 0x1p64f;
#pragma unroll
    for (int e = 0; e < S::V / 2; ++e) {
      x[e] = mul2(x[e], make_float2(0x1p64f, 0x1p64f));
      y[e] = mul2(y[e], make_float2(0x1p64f, 0x1p64f));
    }
  }
  const float inv = scale == 0.0f ? 0.0f : 1.0f / by;   // a NaN stays
  const float down = fmaf(-by, inv, 1.0f) < 0.0f ? __uint_as_float(__float_as_uint(inv) - 1u) : inv;
  const float rest = fmaf(-by, down, 1.0f) * inv;
  const float2 by2 = make_float2(by, by), inv2 = make_float2(-inv, -inv);
  const float2 down2 = make_float2(-down, -down), rest2 = make_float2(-rest, -rest);
  auto codes = [&](const float2& f) {
    const float2 g = make_float2(-f.x, -f.y), q = fma2(g, down2, mul2(g, rest2));
    return (uint32_t)__nv_cvt_float2_to_fp8x2(fma2(fma2(q, by2, g), inv2, q), __NV_SATFINITE, __NV_E4M3);
  };
  uint32_t c[4];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    c[e] = codes(x[2 * e]) | codes(x[2 * e + 1]) << 16;
    c[2 + e] = codes(y[2 * e]) | codes(y[2 * e + 1]) << 16;
  }
  if (!live) return;
  *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
  *reinterpret_cast<uint2*>(dst + S::HALF) = make_uint2(c[2], c[3]);
  if (writes_scale) *scale_at = scale;
}

// The part of the tokens that one warp takes: KV, the k and v heads from head0 on; else the
// q heads from head0 on; `passes` passes of HPW heads.
template <typename T, int HD, bool FP8, bool KV>
__device__ __forceinline__ void append_part(const AppendArgs& a, const Turns& turns, int head0,
                                            int passes, int64_t m, int64_t step,
                                            uint4* ring_base) {
  using S = AppendShape<T, HD>;
  constexpr int V = S::V, LPH = S::LPH, HALF = S::HALF, HPW = S::HPW, NJ = S::NJ;
  constexpr int NP = KV ? kKvPasses : kQPasses;
  const int lane = threadIdx.x & 31, l = lane % LPH, hl = lane / LPH;
  const xmod_kv_cache& c = a.cache;
  const int room = c.max_pages * c.page_size;
  // this lane's angles: pairs l V + i, i = hl + HPW j; pair i of a lane comes from lane
  // l + LPH (i % HPW)
  uint64_t freq[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) freq[j] = turns.f[l * V + (hl + HPW * j) % V];
  const T* gain = (const T*)(KV ? a.k_gain : a.q_gain);
  const bool norm = gain != nullptr;

  auto locate = [&](int64_t m_, Where& w) {
    w.seq = -1;
    if (m_ >= a.M) return;
    w.seq = a.seq ? a.seq[m_] : (int)m_;
    w.slot = a.slot[m_];
    w.pos = a.pos ? a.pos[m_] : w.slot;
  };
  auto find_page = [&](Where& w) {   // looked at an iteration later, when it has arrived
    w.page = -1;
    if (w.seq >= 0 && w.seq < c.n_seqs && w.slot >= 0 && w.slot < room)
      w.page = c.table[(int64_t)w.seq * c.max_pages +
                       (a.page_shift >= 0 ? w.slot >> a.page_shift : w.slot / c.page_size)];
  };

  pdl_trigger();
  pdl_wait();
  uint4 g0 = make_uint4(0u, 0u, 0u, 0u), g1 = g0;
  if (norm) {
    g0 = *reinterpret_cast<const uint4*>(gain + l * V);
    g1 = *reinterpret_cast<const uint4*>(gain + HALF + l * V);
  }
  const int heads = KV ? a.hkv : a.hq, h0 = head0 + hl;
  const T* src0 = (const T*)a.qkv + (KV ? a.hq * HD : 0) + h0 * HD + l * V;
  const int v_off = a.hkv * HD;   // from a k head to the v head beside it
  constexpr int NV = KV ? 2 : 1;
  // [stage][vector][lane]: a lane reads only what it copied itself
  uint4* const ring = ring_base + (threadIdx.x >> 5) * kAppendStages * 8 * 32 + lane;
  static_assert(2 * NP * NV == 8, "vectors of a stage");
  auto issue = [&](int64_t m_, const Where& w, int stage) {
    if (w.seq >= 0) {
      const T* src = src0 + m_ * a.ldqkv;
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (p < passes && h0 + p * HPW < heads) {
            uint4* at = ring + (stage * 8 + (p * NV + j) * 2) * 32;
            copy16(at, src + p * HPW * HD + j * v_off);
            copy16(at + 32, src + p * HPW * HD + j * v_off + HALF);
          }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // tokens m (at work), m + step (page on its way), m + 2 step (vectors about to be asked
  // for), m + 3 step (sequence, slot and position on their way)
  Where w0, w1, w2;
  locate(m, w0);
  locate(m + step, w1);
  locate(m + 2 * step, w2);
  issue(m, w0, 0);
  issue(m + step, w1, 1);
  find_page(w0);
  for (int stage = 0; m < a.M; m += step, stage = stage == kAppendStages - 1 ? 0 : stage + 1) {
    Where w3;
    locate(m + 3 * step, w3);
    issue(m + 2 * step, w2, stage >= 1 ? stage - 1 : kAppendStages - 1);
    find_page(w1);
    asm volatile("cp.async.wait_group 2;" ::: "memory");
    const Where now = w0;
    const bool found = now.page >= 0 && now.page < c.n_pages;   // the same for the whole warp
    if (now.seq >= 0 && !found) report_status(a.status, XMOD_ERR_DEVICE_CHECK);
    if (now.seq >= 0 && found) {
      float2 cs[V / 2], sn[V / 2];
      if (a.rope) {
        float2 own[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) own[j] = rotation(freq[j], now.pos);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float x = __shfl_sync(0xffffffffu, own[i / HPW].x, l + LPH * (i % HPW));
          const float y = __shfl_sync(0xffffffffu, own[i / HPW].y, l + LPH * (i % HPW));
          (i & 1 ? cs[i / 2].y : cs[i / 2].x) = x;
          (i & 1 ? sn[i / 2].y : sn[i / 2].x) = y;
        }
      }
      const int off = a.page_shift >= 0 ? now.slot & (c.page_size - 1) : now.slot % c.page_size;
      // this lane's first row of the cache
      const int64_t row0 = ((int64_t)now.page * a.hkv + h0) * c.page_size + off;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        if (p >= passes) break;
        const bool live = h0 + p * HPW < heads;
        const uint4* at_p = ring + (stage * 8 + p * NV * 2) * 32;
        const uint4 lo = at_p[0], hi = at_p[32];
        float2 x[V / 2], y[V / 2];
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          x[e] = vec_pair<T>(lo, e);
          y[e] = vec_pair<T>(hi, e);
        }
        transform<T, HD>(x, y, norm, g0, g1, a.eps, a.rope, cs, sn);
        if constexpr (!KV) {
          if (live) store_pair<T, HD>((T*)a.q_out + m * a.ldq + (h0 + p * HPW) * HD + l * V, x, y);
        } else {
          const int64_t row = row0 + (int64_t)p * HPW * c.page_size, at = row * HD + l * V;
          if constexpr (FP8) {
            store_e4m3<HD>((uint8_t*)c.k + at, c.k_scale + row, live, l == 0, x, y);
            const uint4 vlo = at_p[64], vhi = at_p[96];
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
              x[e] = vec_pair<T>(vlo, e);
              y[e] = vec_pair<T>(vhi, e);
            }
            store_e4m3<HD>((uint8_t*)c.v + at, c.v_scale + row, live, l == 0, x, y);
          } else if (live) {
            store_pair<T, HD>((T*)c.k + at, x, y);
            *reinterpret_cast<uint4*>((T*)c.v + at) = at_p[64];
            *reinterpret_cast<uint4*>((T*)c.v + at + HALF) = at_p[96];
          }
        }
      }
    }
    w0 = w1;
    w1 = w2;
    w2 = w3;
  }
}

// blockIdx.y: the kv parts first, then the q parts.
template <typename T, int HD, bool FP8>
__global__ void __launch_bounds__(kAppendWarps * 32)
cache_append_kernel(const AppendArgs a, const __grid_constant__ Turns turns, int kv_parts,
                    int kv_passes, int q_passes) {
  constexpr int HPW = AppendShape<T, HD>::HPW;
  const int64_t m = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const int64_t step = (int64_t)gridDim.x * kAppendWarps;
  const int part = blockIdx.y;
  __shared__ uint4 ring[kAppendWarps * kAppendStages * 8 * 32];
  if (part < kv_parts)
    append_part<T, HD, FP8, true>(a, turns, part * kv_passes * HPW, kv_passes, m, step, ring);
  else
    append_part<T, HD, FP8, false>(a, turns, (part - kv_parts) * q_passes * HPW, q_passes, m, step,
                                   ring);
}

template <typename T, int HD, bool FP8>
cudaError_t launch_append_hd(const Ctx& c, const AppendArgs& a, const Turns& turns) {
  constexpr int HPW = AppendShape<T, HD>::HPW;
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int q_all = a.q_out ? (a.hq + HPW - 1) / HPW : 0, kv_all = (a.hkv + HPW - 1) / HPW;
  // Passes a warp does of a token: as many as it holds in flight, or one while the tokens
  // are so few that single passes leave the GPU empty (then only the latency counts; one
  // and several, in us: 12 q and 4 KV heads of 128, bf16, 8 tokens 2.0 and 2.4, 256 tokens
  // 2.7 and 2.8; 32 and 8 heads, 64 tokens 2.5 and 2.8, 512 tokens 6.8 and 4.1).
  const bool few = (int64_t)a.M * (q_all + kv_all) <= (int64_t)sms * 8;
  const int kv_parts = few ? kv_all : (kv_all + kKvPasses - 1) / kKvPasses;
  const int q_parts = few ? q_all : (q_all + kQPasses - 1) / kQPasses;
  const int kv_passes = (kv_all + kv_parts - 1) / kv_parts;
  const int q_passes = q_parts ? (q_all + q_parts - 1) / q_parts : 0;
  const int64_t ctas = ((int64_t)a.M + kAppendWarps - 1) / kAppendWarps;
  const int64_t most = ((int64_t)sms * kAppendCtas + kv_parts + q_parts - 1) / (kv_parts + q_parts);
  return launch_pdl(cache_append_kernel<T, HD, FP8>,
                    dim3((unsigned)(ctas < most ? ctas : most), kv_parts + q_parts),
                    dim3(kAppendWarps * 32), 0, c.stream, a, turns, kv_parts, kv_passes, q_passes);
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
  if (q_out == qkv && M > 1 && ldq != ldqkv) return XMOD_ERR_INVALID_ARG;
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
  a.page_shift = -1;
  for (int i = 4; i < 31; ++i)
    if (cache->page_size == 1 << i) a.page_shift = i;
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
