// QK-norm and rotary positions of q and k heads in any pairing and scaling, and their
// gradient.

#include <math.h>

#include "cache.h"
#include "common.cuh"
#include "rotary.cuh"

namespace xmod {

namespace {

// Turns per position of every pair as 64-bit binary fractions: pos * f wraps at whole turns
// by itself, without double arithmetic on the device.
struct PairTurns {
  uint64_t f[64];
};

// |freq| / (2 pi) with the product's rounding error and 1 / (2 pi) in two doubles, its fraction rounded
// to 2^-64 and negated for a negative freq: a small negative number rounded up to a turn would
// keep no more than 2^-54 of it.
void pair_turns(const xmod_rope& r, PairTurns& t) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
  for (int c = 0; c < r.rot_dim / 2; ++c) {
    const double f = fabs(r.freq[c]), turns = f * kHi;
    const double rest = fma(f, kHi, -turns) + f * kLo;
    // units of 2^-64, and what is left of them
    const double at = (turns - floor(turns)) * 0x1p64, more = (rest - rint(rest)) * 0x1p64;
    const double at_units = floor(at), more_units = floor(more);   // 0 .. 2^64 - 1, -2^63 .. 2^63
    const double left = (at - at_units) + (more - more_units);
    const uint64_t frac = (uint64_t)at_units +
                          (more_units < 0.0 ? 0 - (uint64_t)-more_units : (uint64_t)more_units) +
                          (uint64_t)(left + 0.5);
    t.f[c] = r.freq[c] < 0.0 ? 0 - frac : frac;
  }
}

struct RopeArgs {
  int M, T, hq, hkv, ldx, ldd, ldo;
  const void *x, *q_gain, *k_gain;
  const void* d;      // gradient at the output (backward)
  void* out;
  const int32_t* pos;
  int rot, interleaved;
  float eps, amplitude;
  float turn_sign;    // -1: turned back
  float* part;        // [ctas, 2, hd] of the gains' gradients
  int q_parts, k_parts;   // groups of HPW heads
};

constexpr int kRopeWarps = 4;
// CTAs an SM, and so registers a thread, and the grid: a warp has many tokens, the next one's
// vectors on their way while it works on one. Measured (bf16, 12 and 4 heads of 128): forward of
// 32768 tokens 49.2 us at 5 (4: 51.7, 6: 52.7, 8: 64 with spills; four passes of heads a warp and no
// token ahead: 56), 5.5 TB/s, 0.81 of what a copy reaches; gradient of 16384 tokens 43.3 us at 4 (3:
// 44.9, 5: 77 with spills), 4.7 TB/s with the gains' sums, which take 8; twice the grid 52.
template <bool BWD> constexpr int rope_ctas() { return BWD ? 4 : 5; }
constexpr int kMaxRopeCtas = 2048;

// Bound: memory (a row's q and k heads are read and written once). A lane holds two vectors of V elements of a head, HD / (2 V) lanes to a head, HPW heads a
// pass. Pairs never leave the lane: with halves paired a turning lane holds vector l and its
// partner rot_dim / 2 further, the other lanes two neighbouring vectors of the rest;
// interleaved, any two vectors will do.
template <typename T, int V, int HD> struct RopeShape {
  static constexpr int LPH = HD / (2 * V), HPW = 32 / LPH;
  static constexpr int NJ = V > HPW ? V / HPW : 1;   // angles a lane computes
};

template <int BYTES> __device__ __forceinline__ uint4 load_bytes(const void* p) {
  if constexpr (BYTES == 16) {
    return *reinterpret_cast<const uint4*>(p);
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return make_uint4(v.x, v.y, 0u, 0u);
  }
}
template <int BYTES> __device__ __forceinline__ void store_bytes(void* p, const uint4& v) {
  if constexpr (BYTES == 16)
    *reinterpret_cast<uint4*>(p) = v;
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(v.x, v.y);
}

// Where a lane's two vectors lie in a head, and whether they turn.
struct LaneMap {
  int e0, e1;
  bool turn0, turn1;
};
template <int V, int HD>
__device__ __forceinline__ LaneMap lane_map(int l, int rot, bool interleaved) {
  LaneMap m;
  if (interleaved) {
    m.e0 = l * V;
    m.e1 = HD / 2 + l * V;
    m.turn0 = m.e0 < rot;
    m.turn1 = m.e1 < rot;
  } else {
    const int turning = rot / (2 * V);
    m.turn0 = m.turn1 = l < turning;
    m.e0 = l < turning ? l * V : rot + 2 * (l - turning) * V;
    m.e1 = l < turning ? rot / 2 + l * V : m.e0 + V;
  }
  return m;
}

// Cosines and sines of a lane's V pairs, from the lanes that computed them.
template <typename T, int V, int HD>
__device__ __forceinline__ void lane_angles(const uint64_t (&freq)[RopeShape<T, V, HD>::NJ], int pos,
                                            float amp, float sign, int l, float2 (&cs)[V / 2],
                                            float2 (&sn)[V / 2]) {
  using S = RopeShape<T, V, HD>;
  float2 own[S::NJ];
#pragma unroll
  for (int j = 0; j < S::NJ; ++j) {
    own[j] = rotation(freq[j], pos);
    own[j].x *= amp;
    own[j].y *= amp * sign;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float x = __shfl_sync(0xffffffffu, own[i / S::HPW].x, l + S::LPH * (i % S::HPW));
    const float y = __shfl_sync(0xffffffffu, own[i / S::HPW].y, l + S::LPH * (i % S::HPW));
    (i & 1 ? cs[i / 2].y : cs[i / 2].x) = x;
    (i & 1 ? sn[i / 2].y : sn[i / 2].x) = y;
  }
}

// Turn a lane's vectors: halves paired, x[e] with y[e]; interleaved, the pairs (x.x, x.y) by
// angles 0 .. V/2 - 1 and (y.x, y.y) by V/2 .. V - 1.
template <int V>
__device__ __forceinline__ void turn(float2 (&x)[V / 2], float2 (&y)[V / 2], const float2 (&cs)[V / 2],
                                     const float2 (&sn)[V / 2], const LaneMap& m, bool interleaved) {
  if (!interleaved) {
    if (m.turn0) {
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        const float2 t = mul2(x[e], cs[e]);
        const float2 r = make_float2(fmaf(-y[e].x, sn[e].x, t.x), fmaf(-y[e].y, sn[e].y, t.y));
        y[e] = fma2(x[e], sn[e], mul2(y[e], cs[e]));
        x[e] = r;
      }
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < V / 2; ++e) {
    const int i = e, j = V / 2 + e;
    const float cx = i & 1 ? cs[i / 2].y : cs[i / 2].x, sx = i & 1 ? sn[i / 2].y : sn[i / 2].x;
    const float cy = j & 1 ? cs[j / 2].y : cs[j / 2].x, sy = j & 1 ? sn[j / 2].y : sn[j / 2].x;
    if (m.turn0) x[e] = make_float2(fmaf(-x[e].y, sx, x[e].x * cx), fmaf(x[e].x, sx, x[e].y * cx));
    if (m.turn1) y[e] = make_float2(fmaf(-y[e].y, sy, y[e].x * cy), fmaf(y[e].x, sy, y[e].y * cy));
  }
}

// A warp takes HPW heads (one pass over 32 lanes) of every step-th token, the same heads all along.
// BWD: the gradient with norms (the one without is the forward's with turn_sign -1).
template <typename T, int V, int HD, bool BWD>
__global__ void __launch_bounds__(kRopeWarps * 32, rope_ctas<BWD>())
qk_rope_kernel(const RopeArgs a, const __grid_constant__ PairTurns turns) {
  using S = RopeShape<T, V, HD>;
  constexpr int LPH = S::LPH, HPW = S::HPW, VB = V * sizeof(T);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPH, hl = lane / LPH;
  const bool is_k = (int)blockIdx.y >= a.q_parts;
  const int part = is_k ? blockIdx.y - a.q_parts : blockIdx.y, heads = is_k ? a.hkv : a.hq;
  const int h0 = part * HPW + hl;
  const int64_t column = (int64_t)((is_k ? a.hq : 0) + h0) * HD;
  const LaneMap map = lane_map<V, HD>(l, a.rot, a.interleaved);
  uint64_t freq[S::NJ];
#pragma unroll
  for (int j = 0; j < S::NJ; ++j) {
    const int i = (hl + HPW * j) % V;
    const int e = i < V / 2 ? map.e0 + 2 * i : map.e1 + 2 * i - V;   // interleaved: first of the pair
    const int pair = a.interleaved ? e / 2 : map.e0 + i;
    freq[j] = pair < a.rot / 2 ? turns.f[pair] : 0;
  }
  const T* gain = (const T*)(is_k ? a.k_gain : a.q_gain);
  const bool norm = gain != nullptr, live = h0 < heads;
  // lanes without a head have zeros, and add to the gains' sums: with eps 0 they would have no inverse root
  const float eps = live ? a.eps : 1.0f;
  float2 dg0[V / 2], dg1[V / 2];
#pragma unroll
  for (int e = 0; e < V / 2; ++e) dg0[e] = dg1[e] = make_float2(0.f, 0.f);

  pdl_trigger();
  pdl_wait();
  uint4 g0 = make_uint4(0u, 0u, 0u, 0u), g1 = g0;
  if (norm) {
    g0 = load_bytes<VB>(gain + map.e0);
    g1 = load_bytes<VB>(gain + map.e1);
  }
  const int64_t step = (int64_t)gridDim.x * kRopeWarps;
  auto position = [&](int64_t m) { return m < a.M ? a.pos ? a.pos[m] : (int)(m % a.T) : -1; };
  // x: the projections; d: the gradient
  auto fetch = [&](int64_t m, int pos, uint4 (&x)[2], uint4 (&d)[2]) {
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    const bool in = live && pos >= 0;
    if (!BWD || norm) {
      const T* p = (const T*)a.x + m * a.ldx + column;
      x[0] = in ? load_bytes<VB>(p + map.e0) : none;
      x[1] = in ? load_bytes<VB>(p + map.e1) : none;
    }
    if constexpr (BWD) {
      const T* p = (const T*)a.d + m * a.ldd + column;
      d[0] = in ? load_bytes<VB>(p + map.e0) : none;
      d[1] = in ? load_bytes<VB>(p + map.e1) : none;
    }
  };
  int64_t m = (int64_t)blockIdx.x * kRopeWarps + warp;
  int pos = position(m), pos1 = position(m + step);
  uint4 xv[2], dv[2];
  fetch(m, pos, xv, dv);
  for (; m < a.M; m += step) {
    const int pos2 = position(m + 2 * step);
    uint4 xn[2], dn[2];
    fetch(m + step, pos1, xn, dn);
    if (pos >= 0) {
      float2 cs[V / 2], sn[V / 2];
      lane_angles<T, V, HD>(freq, pos, a.amplitude, a.turn_sign, l, cs, sn);
      float2 x[V / 2], y[V / 2];
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        x[e] = vec_pair<T>(BWD ? dv[0] : xv[0], e);
        y[e] = vec_pair<T>(BWD ? dv[1] : xv[1], e);
      }
      if constexpr (!BWD) {
        if (norm) {
          float2 ss = mul2(x[0], x[0]);
#pragma unroll
          for (int e = 1; e < V / 2; ++e) ss = fma2(x[e], x[e], ss);
#pragma unroll
          for (int e = 0; e < V / 2; ++e) ss = fma2(y[e], y[e], ss);
          float sum = ss.x + ss.y;
#pragma unroll
          for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          const float inv = rsqrtf(fmaf(sum, 1.0f / (float)HD, eps));
          const float2 inv2 = make_float2(inv, inv);
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            x[e] = mul2(mul2(x[e], inv2), vec_pair<T>(g0, e));
            y[e] = mul2(mul2(y[e], inv2), vec_pair<T>(g1, e));
          }
        }
        turn<V>(x, y, cs, sn, map, a.interleaved);
      } else {
        turn<V>(x, y, cs, sn, map, a.interleaved);   // the gradient at the normed head
        if (norm) {
          float2 ss = make_float2(0.f, 0.f), sd = ss;
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            const float2 u = vec_pair<T>(xv[0], e), w = vec_pair<T>(xv[1], e);
            ss = fma2(w, w, fma2(u, u, ss));
            sd = fma2(mul2(x[e], vec_pair<T>(g0, e)), u, sd);
            sd = fma2(mul2(y[e], vec_pair<T>(g1, e)), w, sd);
          }
          float sum = ss.x + ss.y, dot = sd.x + sd.y;
#pragma unroll
          for (int o = LPH / 2; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
          }
          const float inv = rsqrtf(fmaf(sum, 1.0f / (float)HD, eps));
          const float2 inv2 = make_float2(inv, inv);
          const float back = -(inv * dot) * (1.0f / (float)HD) * inv * inv;
          const float2 back2 = make_float2(back, back);
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            const float2 u = vec_pair<T>(xv[0], e), w = vec_pair<T>(xv[1], e);
            dg0[e] = fma2(x[e], mul2(u, inv2), dg0[e]);
            dg1[e] = fma2(y[e], mul2(w, inv2), dg1[e]);
            x[e] = fma2(u, back2, mul2(mul2(x[e], vec_pair<T>(g0, e)), inv2));
            y[e] = fma2(w, back2, mul2(mul2(y[e], vec_pair<T>(g1, e)), inv2));
          }
        }
      }
      if (live) {
        T* op = (T*)a.out + m * a.ldo + column;
        uint4 w0, w1;
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          set_vec_pair<T>(w0, e, x[e]);
          set_vec_pair<T>(w1, e, y[e]);
        }
        store_bytes<VB>(op + map.e0, w0);
        store_bytes<VB>(op + map.e1, w1);
      }
    }
    pos = pos1;
    pos1 = pos2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      xv[i] = xn[i];
      dv[i] = dn[i];
    }
  }
  if constexpr (BWD) {
    if (!a.part) return;
    // the warps' and head groups' sums of this CTA's part, in a fixed order
    __shared__ float sm[kRopeWarps][HD];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float s0 = e & 1 ? dg0[e / 2].y : dg0[e / 2].x, s1 = e & 1 ? dg1[e / 2].y : dg1[e / 2].x;
#pragma unroll
      for (int o = LPH; o < 32; o <<= 1) {
        s0 += __shfl_xor_sync(0xffffffffu, s0, o);
        s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      }
      if (hl == 0) {
        sm[warp][map.e0 + e] = s0;
        sm[warp][map.e1 + e] = s1;
      }
    }
    __syncthreads();
    float* at = a.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * HD;
    for (int e = threadIdx.x; e < HD; e += kRopeWarps * 32) {
      float s = 0.f;
      for (int w = 0; w < kRopeWarps; ++w) s += sm[w][e];
      at[e] = s;
    }
  }
}

// The CTAs' sums of the gains' gradients, 32 dimensions a block (blockIdx.y 0: q's, 1: k's), in
// order, each sum with its rounding errors beside it (D. E. Knuth, The Art of Computer
// Programming 2, 4.2.2; in doubles it took 22 us of 80, one block for all dimensions 76).
constexpr int kGainThreads = 1024;
struct PairSum {
  float hi, lo;
  __device__ __forceinline__ void add(float h, float l) {
    const float t = hi + h, b = t - hi;
    lo += (hi - (t - b)) + (h - b) + l;
    hi = t;
  }
};
__global__ void __launch_bounds__(kGainThreads)
qk_rope_gain_kernel(const float* part, int hd, int ctas, int q_parts, int k_parts, float* dq, float* dk) {
  __shared__ float2 sm[kGainThreads];
  pdl_trigger();
  pdl_wait();
  float* out = blockIdx.y ? dk : dq;
  if (!out) return;
  const int e = blockIdx.x * 32 + (threadIdx.x & 31), rows = kGainThreads / 32;
  const float* at = part + (blockIdx.y ? (int64_t)q_parts * ctas * hd : 0) + e;
  const int n = (blockIdx.y ? k_parts : q_parts) * ctas;
  PairSum s{0.f, 0.f};
  for (int i0 = threadIdx.x >> 5; i0 < n; i0 += 8 * rows) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i0 + j * rows < n ? at[(int64_t)(i0 + j * rows) * hd] : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s.add(v[j], 0.f);
  }
  sm[threadIdx.x] = make_float2(s.hi, s.lo);
  __syncthreads();
  if (threadIdx.x >= 32) return;
  s = PairSum{0.f, 0.f};
#pragma unroll 8
  for (int i = 0; i < rows; ++i) s.add(sm[i * 32 + threadIdx.x].x, sm[i * 32 + threadIdx.x].y);
  out[e] = s.hi + s.lo;
}

template <typename T, int V, int HD, bool BWD>
int launch_rope(const Ctx& c, RopeArgs a, const PairTurns& turns, float* dq, float* dk) {
  constexpr int HPW = RopeShape<T, V, HD>::HPW;
  const int sms = device_sms();
  if (sms <= 0) return XMOD_ERR_CUDA;
  a.q_parts = (a.hq + HPW - 1) / HPW;
  a.k_parts = (a.hkv + HPW - 1) / HPW;
  const int parts = a.q_parts + a.k_parts;
  const int64_t want = ((int64_t)a.M + kRopeWarps - 1) / kRopeWarps;
  int64_t most = ((int64_t)sms * rope_ctas<BWD>() + parts - 1) / parts;
  if (BWD && most * parts > kMaxRopeCtas) most = kMaxRopeCtas / parts > 0 ? kMaxRopeCtas / parts : 1;
  const int ctas = (int)(want < most ? want : most);
  XMOD_LAUNCH(c, "qk_rope", launch_pdl(qk_rope_kernel<T, V, HD, BWD>, dim3(ctas, parts),
                                       dim3(kRopeWarps * 32), 0, c.stream, a, turns));
  if (BWD && a.part)
    XMOD_LAUNCH(c, "qk_rope_gain",
                launch_pdl(qk_rope_gain_kernel, dim3(HD / 32, 2), dim3(kGainThreads), 0, c.stream,
                           (const float*)a.part, HD, ctas, a.q_parts, a.k_parts, dq, dk));
  return XMOD_OK;
}

template <typename T, int V>
int launch_rope_hd(const Ctx& c, const RopeArgs& a, const PairTurns& t, int hd, bool bwd, float* dq, float* dk) {
  if (bwd) {
    if (hd == 128) return launch_rope<T, V, 128, true>(c, a, t, dq, dk);
    if (hd == 64) return launch_rope<T, V, 64, true>(c, a, t, dq, dk);
    return launch_rope<T, V, 32, true>(c, a, t, dq, dk);
  }
  if (hd == 128) return launch_rope<T, V, 128, false>(c, a, t, dq, dk);
  if (hd == 64) return launch_rope<T, V, 64, false>(c, a, t, dq, dk);
  return launch_rope<T, V, 32, false>(c, a, t, dq, dk);
}

int run_rope(const xmod_dims* dm, const RopeArgs& a, const xmod_rope& r, bool bwd, float* dq, float* dk,
             void* stream) {
  PairTurns t{};
  pair_turns(r, t);
  const Ctx c{(cudaStream_t)stream, nullptr};
  if (dm->dtype == XMOD_FP32) return launch_rope_hd<float, 4>(c, a, t, dm->head_dim, bwd, dq, dk);
  // bf16 vectors of 16 bytes, or of 8 where a half is no multiple of them
  if (r.interleaved || r.rot_dim % 16 == 0)
    return launch_rope_hd<__nv_bfloat16, 8>(c, a, t, dm->head_dim, bwd, dq, dk);
  return launch_rope_hd<__nv_bfloat16, 4>(c, a, t, dm->head_dim, bwd, dq, dk);
}

int rope_status(const xmod_dims* dm, const xmod_layer_weights* w, const xmod_rope* r) {
  if (!dims_ok(dm) || !r) return XMOD_ERR_INVALID_ARG;
  if (!head_dim_supported(dm->head_dim)) return XMOD_ERR_UNSUPPORTED;
  if (r->rot_dim < 8 || r->rot_dim % 8 || r->rot_dim > dm->head_dim || !isfinite(r->amplitude))
    return XMOD_ERR_INVALID_ARG;
  for (int c = 0; c < r->rot_dim / 2; ++c)
    if (!isfinite(r->freq[c])) return XMOD_ERR_INVALID_ARG;
  if (w && (!ptr16_or_null(w->q_norm) || !ptr16_or_null(w->k_norm))) return XMOD_ERR_INVALID_ARG;
  return XMOD_OK;
}

bool row_ok(const void* p, int ld, int width) { return ptr16(p) && ld >= width && ld % 8 == 0; }

RopeArgs rope_args(const xmod_dims* dm, int M, const xmod_layer_weights* w, const xmod_rope* r,
                   const int32_t* pos) {
  RopeArgs a{};
  a.M = M;
  a.T = dm->T;
  a.hq = dm->n_heads;
  a.hkv = dm->n_kv_heads;
  a.q_gain = w ? w->q_norm : nullptr;
  a.k_gain = w ? w->k_norm : nullptr;
  a.pos = pos;
  a.rot = r->rot_dim;
  a.interleaved = r->interleaved != 0;
  a.eps = dm->rms_eps;
  a.amplitude = r->amplitude;
  a.turn_sign = 1.0f;
  return a;
}

size_t gain_workspace(const xmod_dims* dm) {
  // one part at least for each of the q and the k heads, whatever the grid
  const size_t parts = (size_t)dm->n_heads + dm->n_kv_heads;
  return ((size_t)kMaxRopeCtas + parts) * dm->head_dim * sizeof(float);
}

}  // namespace
}  // namespace xmod

using namespace xmod;

extern "C" {

int xmod_rope_init(xmod_rope* rope, int rot_dim, int interleaved, double theta,
                   xmod_rope_scaling scaling, double factor, int trained) {
  if (!rope || rot_dim < 8 || rot_dim % 8 || rot_dim > 128 || !isfinite(theta) || !(theta > 1.0))
    return XMOD_ERR_INVALID_ARG;
  if (scaling != XMOD_ROPE_PLAIN && scaling != XMOD_ROPE_LINEAR && scaling != XMOD_ROPE_BASE &&
      scaling != XMOD_ROPE_PARTS)
    return XMOD_ERR_INVALID_ARG;
  if (scaling != XMOD_ROPE_PLAIN && (!isfinite(factor) || !(factor >= 1.0))) return XMOD_ERR_INVALID_ARG;
  if (scaling == XMOD_ROPE_PARTS && trained <= 0) return XMOD_ERR_INVALID_ARG;
  xmod_rope r{};
  r.rot_dim = rot_dim;
  r.interleaved = interleaved != 0;
  r.amplitude = 1.0f;
  if (scaling == XMOD_ROPE_BASE) theta *= pow(factor, (double)rot_dim / (rot_dim - 2));
  double lo = 0.0, hi = 0.0;
  if (scaling == XMOD_ROPE_PARTS) {
    constexpr double kTwoPi = 6.283185307179586;
    auto pair_of = [&](double turns) {
      return rot_dim * log(trained / (kTwoPi * turns)) / (2.0 * log(theta));
    };
    lo = fmax(0.0, floor(pair_of(32.0)));
    hi = fmin(rot_dim - 1.0, ceil(pair_of(1.0)));
    r.amplitude = (float)(0.1 * log(factor) + 1.0);
  }
  for (int c = 0; c < rot_dim / 2; ++c) {
    double f = pow(theta, -2.0 * c / rot_dim);
    if (scaling == XMOD_ROPE_LINEAR) f /= factor;
    if (scaling == XMOD_ROPE_PARTS) {
      const double g = fmin(1.0, fmax(0.0, (c - lo) / fmax(hi - lo, 0.001)));
      f = f * (1.0 - g) + f / factor * g;
    }
    r.freq[c] = f;
  }
  *rope = r;
  return XMOD_OK;
}

int xmod_qk_rope(const xmod_dims* dm, int M, const void* qkv, int ldqkv, const xmod_layer_weights* w,
                 const xmod_rope* rope, const int32_t* pos, void* out, int ldo, void* stream) {
  const int st = rope_status(dm, w, rope);
  if (st) return st;
  if (M < 0) return XMOD_ERR_INVALID_ARG;
  if (M == 0) return XMOD_OK;
  const int width = (dm->n_heads + dm->n_kv_heads) * dm->head_dim;
  if (!row_ok(qkv, ldqkv, width) || !row_ok(out, ldo, width) || !ptr4_or_null(pos) || dm->T <= 0 ||
      (out == qkv && M > 1 && ldo != ldqkv))
    return XMOD_ERR_INVALID_ARG;
  RopeArgs a = rope_args(dm, M, w, rope, pos);
  a.x = qkv;
  a.ldx = ldqkv;
  a.out = out;
  a.ldo = ldo;
  return run_rope(dm, a, *rope, false, nullptr, nullptr, stream);
}

size_t xmod_qk_rope_bwd_workspace_bytes(const xmod_dims* dm, int M) {
  if (!dims_ok(dm) || M < 0 || !head_dim_supported(dm->head_dim)) return 0;
  return gain_workspace(dm);
}

int xmod_qk_rope_bwd(const xmod_dims* dm, int M, const void* qkv, int ldqkv, const xmod_layer_weights* w,
                     const xmod_rope* rope, const int32_t* pos, const void* dout, int lddo, void* din,
                     int lddi, float* dq_norm, float* dk_norm, void* ws, size_t ws_bytes, void* stream) {
  const int st = rope_status(dm, w, rope);
  if (st) return st;
  if (M < 0) return XMOD_ERR_INVALID_ARG;
  const bool norm = w && (w->q_norm || w->k_norm);
  if ((dq_norm && !(w && w->q_norm)) || (dk_norm && !(w && w->k_norm)) || !ptr4_or_null(dq_norm) ||
      !ptr4_or_null(dk_norm))
    return XMOD_ERR_INVALID_ARG;
  const int width = (dm->n_heads + dm->n_kv_heads) * dm->head_dim;
  if (M > 0 && (!row_ok(dout, lddo, width) || !row_ok(din, lddi, width) ||
                (norm && !row_ok(qkv, ldqkv, width)) || !ptr4_or_null(pos) || dm->T <= 0 ||
                (din == dout && M > 1 && lddi != lddo) || (norm && din == qkv)))
    return XMOD_ERR_INVALID_ARG;
  const bool gains = dq_norm || dk_norm;
  if (gains && (!ptr16(ws) || ws_bytes < gain_workspace(dm))) return XMOD_ERR_WORKSPACE;
  if (M == 0) {
    if (!gains) return XMOD_OK;
    const Ctx c{(cudaStream_t)stream, nullptr};
    XMOD_LAUNCH(c, "qk_rope_gain",
                launch_pdl(qk_rope_gain_kernel, dim3(dm->head_dim / 32, 2), dim3(kGainThreads), 0, c.stream,
                           (const float*)ws, dm->head_dim, 0, 0, 0, dq_norm, dk_norm));
    return XMOD_OK;
  }
  RopeArgs a = rope_args(dm, M, w, rope, pos);
  a.out = din;
  a.ldo = lddi;
  a.turn_sign = -1.0f;
  if (!norm) {   // the rotation's transpose
    a.x = dout;
    a.ldx = lddo;
    return run_rope(dm, a, *rope, false, nullptr, nullptr, stream);
  }
  a.x = qkv;
  a.ldx = ldqkv;
  a.d = dout;
  a.ldd = lddo;
  a.part = gains ? (float*)ws : nullptr;
  return run_rope(dm, a, *rope, true, dq_norm, dk_norm, stream);
}

}  // extern "C"
