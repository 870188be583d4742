// Log probabilities of given tokens with the entropy and the largest alternatives, and
// their gradient at the logits.

#include <cuda_bf16.h>
#include <float.h>
#include <limits.h>
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "tc_common.cuh"

namespace xmod {

using namespace tc;

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ---------------------------------------------------------------- forward
//
// One pass: every thread keeps a running maximum m, l = sum e^(x - m) and u = sum e^(x - m)
// (x - m); then lse = m + ln l and the entropy is ln l - u / l, whose terms all have one
// sign. A bf16 logit costs 5 instructions (4 without the entropy), half of the issue slots
// at the full memory rate: the kernel is bound by memory, and laid out to keep reading. A
// CTA works rows off one after the other, in three roles that meet at mbarriers only: a
// producer warp keeps bulk copies into a ring of 16 KB chunks going, across row ends; four
// consumer warps sum, each at its own pace; a finisher warp (or two, taking turns) joins a
// row's sums, finds its alternatives and writes its results while the consumers are at the
// next rows. Few rows are split over the CTAs of a cluster, which join through distributed
// shared memory; short rows go to single warps (below).
//
// Measured: 4096 rows of 50257, bf16 (412 MB): 67 us, 6.2 TB/s, 0.91 of what a copy reaches;
// with 5 alternatives 76 us, 0.80 (the finisher takes issue slots); fp32 (823 MB), with 5
// alternatives 124 us, 0.98; 8 rows with 20 alternatives 10.7 us, without 4.1.
//
// The alternatives. Logits are ranked by 64-bit keys, the value's order above the inverted
// token number: keys are distinct, so ties need no care. All that the consumers do for them
// is to leave every thread's maximum of every chunk. The k-th largest of the threads' maxima
// over the row is a bound that k logits reach and few besides; the finisher reads the
// vectors behind the chunk maxima that reach it once more (from L2), and ranks the logits
// that do by counting the larger ones. Whenever they fill its buffer (many equal ones, a row
// in rising order), only the k best so far stay; a row with fewer than k tokens above
// -infinity is filled up from its first tokens.

constexpr int kLpThreads = 128;    // consumers; then the finishers' warps and the producer's
constexpr int kChunk = 16384;      // bytes
constexpr int kLpStages = 2;
constexpr int kLpCtas = 4;         // an SM
constexpr int kVecs = kChunk / 16 / kLpThreads;   // vectors a thread takes of a chunk
constexpr int kTail = 2;            // vectors at a time of a row's last chunk
constexpr int kSlots = 8;          // maxima a thread leaves of a row, each of `step` chunks
// Logits that a finisher keeps while it looks. 8 rows of 50257 bf16 logits with 20
// alternatives, all but three at the type's lowest value: 99 us (192: 112, 512: 300; reading
// the row once for every alternative instead, 1030); ordinary rows do not fill it.
constexpr int kCandidates = 256;

struct LogprobArgs {
  int V, top_k, splits, per;   // per: logits of a split
  int64_t N, ld;
  const void* logits;
  const int32_t* target;
  float *logp, *entropy, *lse;
  int32_t* top_idx;
  float* top_logp;
  int* status;
};

// Order of a logit as an unsigned number: larger value, larger number; -0 equals +0, NaN on
// top. And back.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return x != x ? 0xffffffffu : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, int token) {
  return (uint64_t)order_of(x) << 32 | (0xffffffffu - (uint32_t)token);
}
__device__ __forceinline__ int token_of(uint64_t key) {
  return (int)(0xffffffffu - (uint32_t)key);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Maximum of two fp32, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Largest element of a 16-byte vector, NaN if there is one.
template <typename T> __device__ __forceinline__ float vec_max(const uint4& v) {
  if constexpr (sizeof(T) == 4) {
    return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                   max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
  } else {
    const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&v);
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(b[0], b[1]), __hmax2_nan(b[2], b[3]));
    const float2 f = __bfloat1622float2(m);
    return max_nan(f.x, f.y);
  }
}
template <typename T> __device__ __forceinline__ float vec_at(const uint4& v, int i) {
  const float2 f = vec_pair<T>(v, i >> 1);
  return i & 1 ? f.y : f.x;
}
// Elements below -2^123 become -2^123; a NaN stays.
template <typename T> __device__ __forceinline__ void vec_finite(uint4& v) {
  if constexpr (sizeof(T) == 4) {
    float* f = reinterpret_cast<float*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = max_nan(f[i], -1.0633824e37f);
  } else {
    __nv_bfloat162* b = reinterpret_cast<__nv_bfloat162*>(&v);
    const __nv_bfloat162_raw low{0xfd00, 0xfd00};
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __hmax2_nan(b[i], __nv_bfloat162(low));
  }
}
template <typename T> __device__ __forceinline__ void vec_clear(uint4& v, int i) {   // to -inf
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
  if constexpr (sizeof(T) == 4)
    w[i] = 0xff800000u;
  else
    w[i >> 1] = i & 1 ? (w[i >> 1] & 0x0000ffffu) | 0xff800000u : (w[i >> 1] & 0xffff0000u) | 0xff80u;
}

// Over a common maximum m (l, u: sums of e^(x - m) and of e^(x - m) log2(e^(x - m))).
// Nothing seen: l = 0.
struct Moments {
  float m, l, u;
  // to a maximum at or above its own
  __device__ __forceinline__ void raise(float m2) {
    const float d = (m - m2) * kLog2e, f = ex2(d);
    u = f > 0.f ? f * fmaf(d, l, u) : 0.f;   // d may be infinite where f is 0
    l *= f;
    m = m2;
  }
};

// A row's (or a split's) logits in 16-byte vectors, aligned: `head` elements of the first
// vector and what follows `count` elements do not belong to it.
struct Span {
  const uint4* vecs;
  int head, count, nvec, full, token0;   // full: vectors wholly inside the buffer
};
template <typename T>
__device__ __forceinline__ Span span_of(const LogprobArgs& a, int64_t row, int split) {
  constexpr int VE = 16 / sizeof(T);
  Span s;
  s.token0 = min(a.V, split * a.per);
  s.count = min(a.V, s.token0 + a.per) - s.token0;
  const uintptr_t at = (uintptr_t)((const T*)a.logits + row * a.ld + s.token0);
  s.head = (int)(at & 15) / (int)sizeof(T);
  s.vecs = (const uint4*)(at & ~(uintptr_t)15);
  s.full = s.count ? (s.head + s.count) / VE : 0;
  s.nvec = s.count ? (s.head + s.count + VE - 1) / VE : 0;
  return s;
}
__device__ __forceinline__ int span_chunks(const Span& s) {
  return (s.nvec + kChunk / 16 - 1) / (kChunk / 16);
}

// What a warp needs to find a row's alternatives.
struct Finisher {
  alignas(16) uint64_t cand[kCandidates + 2];
  uint64_t top[XMOD_MAX_TOP_K];   // the row's (or this CTA's) best, in order
  uint16_t hits[kSlots * kLpThreads];
};

// Shared memory behind the ring. Two of what a row leaves: the consumers may be a row ahead.
struct alignas(16) LpShared {
  uint64_t full[kLpStages], empty[kLpStages];
  uint64_t done[2], freed[2];     // a row's maxima and sums are there; have been read
  Moments moments[2][kLpThreads / 32];
  Moments parts[8];               // of a cluster's CTAs, in the first one
  int abort;
  alignas(16) float tops[2][kSlots][kLpThreads];
  Finisher fin[2];
};

__device__ __forceinline__ void st_cluster(uint32_t at, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster64(uint32_t at, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}

constexpr uint32_t kOrderNone = 0x007fffffu;   // order_of(-infinity)

// The `k` best of `count` candidates to sh.top, in order; one warp.
__device__ __forceinline__ void rank_candidates(Finisher& sh, int count, int k, int lane) {
  if (lane == 0) sh.cand[count] = 0;   // the last pair's other half
  __syncwarp();
  for (int i = lane; i < count; i += 32) {
    const uint64_t mine = sh.cand[i];
    int above = 0;
#pragma unroll 4
    for (int j = 0; j < count; j += 2) {
      const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&sh.cand[j]);
      above += (o.x > mine) + (o.y > mine);
    }
    if (above < k) sh.top[above] = mine;
  }
  __syncwarp();
}

// One warp: the k best of a row (or split) to sh.top, in order; how many there are (all of a
// short one). The row's vectors were read by 32 Q threads: thread t took the vectors
// t + 32 Q j, and its slot i holds the maximum of EACH * step of them from j = i EACH step on;
// tops: those of threads lane, lane + 32, ...
template <typename T, int Q, int S, int EACH>
__device__ __forceinline__ int find_top(const LogprobArgs& a, Finisher& sh,
                                        const float (&tops)[Q][S], const Span& s, int64_t row,
                                        int step, int k, int lane) {
  constexpr int VE = 16 / sizeof(T), THREADS = 32 * Q;
  constexpr int BITS = 8 * sizeof(T), SHIFT = 32 - BITS;   // of an order that differ by type
  const T* p = (const T*)a.logits + row * a.ld + s.token0;
  uint32_t best[Q];   // the threads' orders over the row
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    float m = tops[q][0];
#pragma unroll
    for (int i = 1; i < S; ++i) m = max_nan(m, tops[q][i]);
    best[q] = lane + 32 * q < s.nvec ? order_of(m) : 0u;
  }
  // the k-th largest of the threads' orders: a few by taking the largest away, more by the
  // largest bound that k threads reach, bit by bit (4096 rows of 50257, bf16, either way, in us:
  // 5 alternatives 76.4 and 78.9, 8 of them 81.9 and 84.0, 12 86.8 and 87.4, 16 96.4 and 94.3,
  // 20 101 and 97.9; rows of 16000: 5 of them 41.1 and 42.9, 12 46.4 and 45.9, 20 53.3 and 48.9)
  uint32_t bound = 0;
  if (k <= 12) {
    uint32_t left[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) left[q] = best[q];
    for (int i = 0; i < k; ++i) {
      uint32_t mine = left[0];
#pragma unroll
      for (int q = 1; q < Q; ++q) mine = max(mine, left[q]);
      bound = __reduce_max_sync(0xffffffffu, mine);
      if (lane == __ffs(__ballot_sync(0xffffffffu, mine == bound)) - 1) {
        bool taken = false;
#pragma unroll
        for (int q = 0; q < Q; ++q)
          if (!taken && left[q] == bound) {
            left[q] = 0;
            taken = true;
          }
      }
    }
  } else {
    for (int bit = BITS - 1; bit >= 0; --bit) {
      const uint32_t next = bound | 1u << bit;
      int n = 0;
#pragma unroll
      for (int q = 0; q < Q; ++q) n += __popc(__ballot_sync(0xffffffffu, best[q] >> SHIFT >= next));
      if (n >= k) bound = next;
    }
    bound <<= SHIFT;
  }
  // none at -infinity (see below); 0 stands for -0 too
  bound = max(bound, kOrderNone + 1);
  float least = value_of(bound);
  // the threads' chunks whose maxima reach it: first vectors of them
  uint32_t mask = 0;
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (!(tops[q][i] < least)) mask |= 1u << (q * S + i);
  int at = __popc(mask), hits = at;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, hits, o);
    if (lane >= o) hits += up;
  }
  at = hits - at;
  hits = __shfl_sync(0xffffffffu, hits, 31);
  for (; mask; mask &= mask - 1) {
    const int i = __ffs(mask) - 1;
    sh.hits[at++] = i % S * THREADS + lane + i / S * 32;
  }
  __syncwarp();
  // their vectors, a lane each, two readings under way
  int count = 0;
  uint64_t low = 0;   // keys below it are known not to be among the k best
  float above = least;   // from token `last` on, the least value that can be
  int last = INT_MAX;
  constexpr int HPW = 32 / EACH, AHEAD = 2;
  static_assert(32 % EACH == 0 && Q * S <= 32, "");
  for (int h0 = 0; h0 < hits; h0 += HPW * AHEAD) {
    for (int c = 0; c < step; ++c) {
      uint4 x[AHEAD];
      int e0[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int h = h0 + i * HPW + lane / EACH;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        e0[i] = s.count;
        if (h < hits) {
          const int hit = sh.hits[h];
          const int v = ((hit / THREADS * step + c) * EACH + lane % EACH) * THREADS + hit % THREADS;
          if (v < s.nvec) {
            e0[i] = v * VE - s.head;
            if (v < s.full) {
              x[i] = s.vecs[v];
            } else {
              T* e = reinterpret_cast<T*>(&x[i]);
#pragma unroll
              for (int j = 0; j < VE; ++j)
                if (e0[i] + j >= 0 && e0[i] + j < s.count) e[j] = p[e0[i] + j];
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (h0 + i * HPW >= hits) break;
        const float at_least = s.token0 + e0[i] >= last ? above : least;
        uint32_t in = 0;
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (!(vec_at<T>(x[i], j) < at_least)) in |= 1u << j;
        // elements before the row's first and past its last
        if (e0[i] < 0) in &= ~0u << -e0[i];
        if (e0[i] + VE > s.count) in &= (1u << max(0, s.count - e0[i])) - 1u;
        for (uint32_t who; (who = __ballot_sync(0xffffffffu, in != 0)) != 0; in &= in - 1) {
          if (count > kCandidates - 32) {   // keep the k best
            rank_candidates(sh, count, k, lane);
            for (int j = lane; j < k; j += 32) sh.cand[j] = sh.top[j];
            count = k;
            low = sh.top[k - 1];
            least = value_of((uint32_t)(low >> 32));
            above = value_of((uint32_t)(low >> 32) + 1);
            last = token_of(low);
            __syncwarp();
          }
          uint64_t key = 0;
          if (in) {
            const int j = __ffs(in) - 1;
            float f = vec_at<T>(x[i], 0);
#pragma unroll
            for (int jj = 1; jj < VE; ++jj) f = jj == j ? vec_at<T>(x[i], jj) : f;
            key = key_of(f, s.token0 + e0[i] + j);
          }
          if (low) who = __ballot_sync(0xffffffffu, key > low);
          if (who >> lane & 1) sh.cand[count + __popc(who & ((1u << lane) - 1u))] = key;
          count += __popc(who);
        }
      }
    }
  }
  const int want = min(k, s.count);
  if (count < want) {   // the rest are tokens at -infinity: the lowest, among the first 2 k
    for (int t0 = 0; t0 < min(2 * k, s.count); t0 += 32) {
      const int t = t0 + lane;
      const bool in = t < min(2 * k, s.count) && order_of(Elem<T>::to_f(p[t])) == kOrderNone;
      const uint32_t who = __ballot_sync(0xffffffffu, in);
      if (in) sh.cand[count + __popc(who & ((1u << lane) - 1u))] = key_of(-INFINITY, s.token0 + t);
      count += __popc(who);
    }
  }
  rank_candidates(sh, count, k, lane);
  return want;
}

// One warp: a row's results from its sums, its target's logit and its alternatives' keys.
template <typename T>
__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t row, const Moments& mo,
                                          int target, T x_t, const uint64_t* top, int lane) {
  const bool bad = !(mo.l > 0.f);   // nothing above -infinity, a NaN or +infinity
  const float ll = logf(mo.l), nan = __int_as_float(0x7fc00000);
  if (lane == 0) {
    if (bad || target >= a.V) report_status(a.status, XMOD_ERR_DEVICE_CHECK);
    if (a.lse) a.lse[row] = bad ? nan : mo.m + ll;
    if (a.entropy) a.entropy[row] = bad ? nan : ll - 0.6931471805599453f * mo.u / mo.l;
    if (a.logp)
      a.logp[row] = target < 0 ? 0.f : bad || target >= a.V ? nan : (Elem<T>::to_f(x_t) - mo.m) - ll;
  }
  for (int i = lane; i < a.top_k; i += 32) {
    const uint64_t key = top[i];
    a.top_idx[row * a.top_k + i] = token_of(key);
    a.top_logp[row * a.top_k + i] = bad ? nan : (value_of((uint32_t)(key >> 32)) - mo.m) - ll;
  }
}

// Rows of at most 256 vectors (4 KB): a warp holds one in registers, eight vectors a lane, so
// the maximum comes first and nothing is read twice but the few vectors behind the bound.
// 4096 rows of 1000 logits, bf16, with 5 alternatives: 7.3 us, 18 us by the ring.
constexpr int kShortVecs = 8, kShortWarps = 4, kShortTopK = 32;

template <typename T, bool ENT>
__global__ void __launch_bounds__(kShortWarps * 32)
token_logprobs_short_kernel(const LogprobArgs a) {
  constexpr int VE = 16 / sizeof(T);
  __shared__ Finisher fin[kShortWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  for (int64_t row = (int64_t)blockIdx.x * kShortWarps + warp; row < a.N;
       row += (int64_t)gridDim.x * kShortWarps) {
    const Span s = span_of<T>(a, row, 0);
    const int target = a.logp ? a.target[row] : -1;
    uint4 x[kShortVecs];
#pragma unroll
    for (int i = 0; i < kShortVecs; ++i) {
      const int v = lane + 32 * i;
      const uint32_t ninf = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
      x[i] = make_uint4(ninf, ninf, ninf, ninf);
      if (v < s.full) {
        x[i] = s.vecs[v];
        if (v == 0) {
#pragma unroll
          for (int j = 0; j < VE; ++j)
            if (j < s.head) vec_clear<T>(x[i], j);
        }
      } else if (v < s.nvec) {
        const T* p = reinterpret_cast<const T*>(s.vecs + v);
        T* e = reinterpret_cast<T*>(&x[i]);
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (v * VE + j >= s.head && v * VE + j < s.head + s.count) e[j] = p[j];
      }
    }
    const T x_t = target >= 0 && target < a.V ? ((const T*)a.logits + row * a.ld)[target]
                                              : Elem<T>::from_f(0.f);
    float tops[1][kShortVecs], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kShortVecs; ++i) {
      tops[0][i] = vec_max<T>(x[i]);
      top = max_nan(top, tops[0][i]);
    }
    // a NaN makes the maximum +infinity, the sum 0 or NaN and the row bad
    const bool nan = __any_sync(0xffffffffu, top != top);
    Moments mo{nan ? INFINITY : warp_max(top), 0.f, 0.f};
    float2 l2 = make_float2(0.f, 0.f), u2 = l2;
    if (fabsf(mo.m) < 1e36f) {
      const float2 neg = make_float2(-mo.m, -mo.m), lg = make_float2(kLog2e, kLog2e);
#pragma unroll
      for (int i = 0; i < kShortVecs; ++i) {
        if (32 * i >= s.nvec) break;
        if (ENT) vec_finite<T>(x[i]);
#pragma unroll
        for (int j = 0; j < VE / 2; ++j) {
          const float2 t = mul2(add2(vec_pair<T>(x[i], j), neg), lg);
          const float2 e = make_float2(ex2(t.x), ex2(t.y));
          l2 = add2(l2, e);
          if (ENT) u2 = fma2(e, t, u2);
        }
      }
    } else if (mo.m > -INFINITY) {   // differences that could overflow
#pragma unroll
      for (int i = 0; i < kShortVecs * VE; ++i) {
        const float d = fmaxf(vec_at<T>(x[i / VE], i % VE) - mo.m, -1e30f) * kLog2e, e = ex2(d);
        l2.x += e;
        if (ENT) u2.x = fmaf(e, d, u2.x);
      }
    }
    mo.l = warp_sum(l2.x + l2.y);
    if (ENT) mo.u = warp_sum(u2.x + u2.y);
    if (a.top_k)
      find_top<T, 1, kShortVecs, 1>(a, fin[warp], tops, s, row, 1, a.top_k, lane);
    write_row<T>(a, row, mo, target, x_t, fin[warp].top, lane);
    __syncwarp();
  }
}

template <typename T, bool ENT, int FIN>
__global__ void __launch_bounds__(kLpThreads + 32 * FIN + 32, kLpCtas)
token_logprobs_kernel(const LogprobArgs a) {
  constexpr int VE = 16 / sizeof(T), W = kLpThreads / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  LpShared& sh = *reinterpret_cast<LpShared*>(smem + kLpStages * kChunk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = a.splits > 1 ? (int)cluster_ctarank() : 0;
  const int64_t row0 = blockIdx.x / a.splits, row_step = gridDim.x / a.splits;
  const int k = a.top_k;
  volatile int* abort_flag = &sh.abort;
  const uint32_t bFull = smem_u32(&sh.full[0]), bEmpty = smem_u32(&sh.empty[0]);
  const uint32_t bDone = smem_u32(&sh.done[0]), bFreed = smem_u32(&sh.freed[0]);

  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < kLpStages; ++i) {
      mbar_init(bFull + 8 * i, 1);
      mbar_init(bEmpty + 8 * i, W);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bDone + 8 * i, W);
      mbar_init(bFreed + 8 * i, 1);
    }
    sh.abort = 0;
    fence_barrier_init();
  }
  if (a.splits > 1)
    cluster_sync_all();   // also: the cluster's CTAs run, their shared memory may be written
  else
    __syncthreads();
  pdl_wait();
  // a wait that gives up ends its warp's work; the other warps' waits end by the abort flag

  if (warp == W + FIN) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t n = 0;
      bool ok = true;
      for (int64_t row = row0; ok && row < a.N; row += row_step) {
        const Span s = span_of<T>(a, row, split);
        const int chunks = span_chunks(s);
        for (int c = 0; c < chunks; ++c, ++n) {
          const uint32_t st = n % kLpStages, use = n / kLpStages;
          if (use && !(ok = mbar_wait(bEmpty + 8 * st, (use - 1) & 1, abort_flag, a.status))) break;
          const int v0 = c * (kChunk / 16);
          const int bytes = max(0, min(kChunk / 16, s.full - v0)) * 16;
          mbar_arrive_expect_tx(bFull + 8 * st, bytes);
          if (bytes) bulk_load(smem_u32(smem) + st * kChunk, s.vecs + v0, bytes, bFull + 8 * st);
        }
      }
      // the copies still in flight land before the CTA can end
      for (uint32_t j = n > kLpStages ? n - kLpStages : 0; j < n; ++j)
        mbar_wait(bFull + 8 * (j % kLpStages), (j / kLpStages) & 1, nullptr, a.status);
    }
    __syncwarp();
  } else if (warp >= W) {
    // ------------------------------------------------------------ finishers
    int parity = warp - W;
    Finisher& fin = sh.fin[parity];
    const int64_t first = row0 + parity * row_step, turn = FIN * row_step;
    uint32_t phase = 0;
    bool met = false;   // the cluster's barrier is behind it
    // the target's logit is fetched a row ahead (and kept as it is stored until it is used),
    // the target two rows ahead
    const bool targets = a.logp && split == 0;
    auto target_of = [&](int64_t r) { return targets && r < a.N ? a.target[r] : -1; };
    auto logit_of = [&](int64_t r, int t) {
      return t >= 0 && t < a.V ? ((const T*)a.logits + r * a.ld)[t] : Elem<T>::from_f(0.f);
    };
    int target_1 = target_of(first), target_2 = target_of(first + turn);
    T x_1 = logit_of(first, target_1);
    for (int64_t row = first; row < a.N; row += turn) {
      const Span s = span_of<T>(a, row, split);
      const int chunks = span_chunks(s), step = (chunks + kSlots - 1) / kSlots;
      const int target = target_1;
      const T x_t = x_1;
      target_1 = target_2;
      x_1 = logit_of(row + turn, target_1);
      target_2 = target_of(row + 2 * turn);
      if (!mbar_wait(bDone + 8 * parity, phase, abort_flag, a.status)) break;
      Moments mo = sh.moments[parity][lane % W];
      int found = 0;
      if (k) {
        const int slots = (chunks + step - 1) / step;
        float tops[W][kSlots];
#pragma unroll
        for (int q = 0; q < W; ++q)
#pragma unroll
          for (int i = 0; i < kSlots; ++i)
            tops[q][i] = i < slots ? sh.tops[parity][i][lane + 32 * q] : -INFINITY;
        found = find_top<T, W, kSlots, kVecs>(a, fin, tops, s, row, step, k, lane);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bFreed + 8 * parity);
      mo.raise(warp_max(mo.m));
      if (lane >= W) mo.l = mo.u = 0.f;
      mo.l = warp_sum(mo.l);
      mo.u = warp_sum(mo.u);
      const uint64_t* best = fin.top;
      if (a.splits > 1) {   // the cluster's only row: everything to the first CTA
        if (lane == 0) {
          const uint32_t at = mapa_shared(smem_u32(&sh.parts[split]), 0);
          st_cluster(at, __float_as_uint(mo.m));
          st_cluster(at + 4, __float_as_uint(mo.l));
          st_cluster(at + 8, __float_as_uint(mo.u));
        }
        const int before = split * min(k, a.per);   // all splits but the last are full
        for (int i = lane; i < found; i += 32)
          st_cluster64(mapa_shared(smem_u32(&sh.fin[1].cand[before + i]), 0), fin.top[i]);
        cluster_sync_all();
        met = true;
        if (split != 0) return;
        mo = sh.parts[min(lane, a.splits - 1)];
        mo.raise(warp_max(mo.m));
        if (lane >= a.splits) mo.l = mo.u = 0.f;
        mo.l = warp_sum(mo.l);
        mo.u = warp_sum(mo.u);
        if (k) {
          const int last = a.V - (a.splits - 1) * a.per;
          const int all = (a.splits - 1) * min(k, a.per) + min(k, last);
          rank_candidates(sh.fin[1], all, k, lane);
          best = sh.fin[1].top;   // a second finisher has no row here
        }
      }
      write_row<T>(a, row, mo, target, x_t, best, lane);
      __syncwarp();
      if (FIN == 1) parity ^= 1;
      if (FIN == 2 || !parity) phase ^= 1;
    }
    if (met) return;
  } else {
    // ------------------------------------------------------------ consumers
    int stage = 0, parity = 0;
    uint32_t phase = 0, row_phase = 1;   // the first two rows find their places free
    for (int64_t row = row0; row < a.N; row += row_step) {
      const Span s = span_of<T>(a, row, split);
      const int chunks = span_chunks(s), step = (chunks + kSlots - 1) / kSlots;
      Moments mo{-FLT_MAX, 0.f, 0.f};
      float2 l2 = make_float2(0.f, 0.f), u2 = l2;
      float slot_top = -INFINITY;
      int slot = 0, in_slot = 0;
      if (!mbar_wait(bFreed + 8 * parity, row_phase, abort_flag, a.status)) break;
      bool ok = true;
      for (int c = 0; c < chunks; ++c) {
        if (!(ok = mbar_wait(bFull + 8 * stage, phase, abort_flag, a.status))) break;
        const uint4* buf = reinterpret_cast<const uint4*>(smem + stage * kChunk);
        const int v0 = c * (kChunk / 16);
        auto absorb = [&](auto& x) {   // takes vectors into the sums
          constexpr int N = sizeof(x) / sizeof(uint4);
          float top = vec_max<T>(x[0]);
#pragma unroll
          for (int i = 1; i < N; ++i) top = max_nan(top, vec_max<T>(x[i]));
          if (!(top <= mo.m)) {   // larger, or a NaN: that one makes l 0 and the row bad
            const float d = (mo.m - (top != top ? INFINITY : top)) * kLog2e, f = ex2(d);
            const float2 f2 = make_float2(f, f), d2 = make_float2(d, d);
            if (ENT) u2 = f > 0.f ? mul2(f2, fma2(d2, l2, u2)) : make_float2(0.f, 0.f);
            l2 = mul2(l2, f2);
            mo.m = top != top ? INFINITY : top;
          }
          slot_top = max_nan(slot_top, top);
          if (fabsf(mo.m) < 1e36f) {
            const float2 neg = make_float2(-mo.m, -mo.m), lg = make_float2(kLog2e, kLog2e);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              // an infinite exponent times 0 would be a NaN: such logits become low finite
              // ones, whose terms are 0 as well
              if (ENT) vec_finite<T>(x[i]);
#pragma unroll
              for (int j = 0; j < VE / 2; ++j) {
                // the difference first: exactly 0, and a term of exactly 1, at the maximum
                const float2 t = mul2(add2(vec_pair<T>(x[i], j), neg), lg);
                const float2 e = make_float2(ex2(t.x), ex2(t.y));
                l2 = add2(l2, e);
                if (ENT) u2 = fma2(e, t, u2);
              }
            }
          } else if (top > -INFINITY) {   // differences that could overflow
#pragma unroll
            for (int i = 0; i < N * VE; ++i) {
              const float d = fmaxf(vec_at<T>(x[i / VE], i % VE) - mo.m, -1e30f) * kLog2e, e = ex2(d);
              l2.x += e;
              if (ENT) u2.x = fmaf(e, d, u2.x);
            }
          }
        };
        if (v0 + kChunk / 16 <= s.full) {
          uint4 x[kVecs];
#pragma unroll
          for (int i = 0; i < kVecs; ++i) x[i] = buf[tid + i * kLpThreads];
          __syncwarp();
          if (lane == 0) mbar_arrive(bEmpty + 8 * stage);
          if (v0 + tid == 0) {
#pragma unroll
            for (int j = 0; j < VE; ++j)
              if (j < s.head) vec_clear<T>(x[0], j);
          }
          absorb(x);
        } else {   // the row's last chunk: what there is of it, two vectors at a time
          // (4096 rows of 16000 logits, bf16: 29.0 us; one by one 31.9, four 27.7, but those
          // cost 81 instead of 76 where 50257 logits with 5 alternatives are wanted)
          const uint32_t ninf = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
          // the last vector, not wholly inside the buffer, by elements
          uint4 part = make_uint4(ninf, ninf, ninf, ninf);
          if (s.full < s.nvec && (s.full - v0) % kLpThreads == tid) {
            const T* p = reinterpret_cast<const T*>(s.vecs + s.full);
            T* e = reinterpret_cast<T*>(&part);
#pragma unroll
            for (int j = 0; j < VE; ++j)
              if (s.full * VE + j >= s.head && s.full * VE + j < s.head + s.count) e[j] = p[j];
          }
#pragma unroll 1
          for (int v = v0 + tid; v - lane < s.nvec; v += kTail * kLpThreads) {
            uint4 x[kTail];
#pragma unroll
            for (int i = 0; i < kTail; ++i) {
              const int vi = v + i * kLpThreads;
              x[i] = vi == s.full ? part : make_uint4(ninf, ninf, ninf, ninf);
              if (vi < s.full) x[i] = buf[vi - v0];
            }
            if (v == 0) {
#pragma unroll
              for (int j = 0; j < VE; ++j)
                if (j < s.head) vec_clear<T>(x[0], j);
            }
            absorb(x);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bEmpty + 8 * stage);
        }
        if (++stage == kLpStages) {
          stage = 0;
          phase ^= 1;
        }
        if (++in_slot == step || c + 1 == chunks) {
          sh.tops[parity][slot++][tid] = slot_top;
          slot_top = -INFINITY;
          in_slot = 0;
        }
      }
      if (!ok) break;
      mo.l = l2.x + l2.y;
      mo.u = u2.x + u2.y;
      mo.raise(warp_max(mo.m));
      mo.l = warp_sum(mo.l);
      if (ENT) mo.u = warp_sum(mo.u);
      if (lane == 0) sh.moments[parity][warp] = mo;
      __syncwarp();
      if (lane == 0) mbar_arrive(bDone + 8 * parity);
      parity ^= 1;
      if (!parity) row_phase ^= 1;
    }
  }
  if (a.splits > 1) cluster_sync_all();   // the finishers' one, for the cluster's one row
}

// ---------------------------------------------------------------- gradient
//
// dx_v = g (1[v = t] - p_v) - gH p_v (ln p_v + H): one reading and one writing of the
// logits' size, 5 instructions a logit: bound by memory (4096 rows of 50257, bf16, 823 MB:
// 127 us, 6.5 TB/s, 0.96 of what a copy reaches). A CTA takes 16 KB of a row, four
// 16-byte vectors a thread, aligned in the output; where the logits' rows are aligned
// differently (another row stride), their elements are loaded one by one, which the L1
// cache makes up for.
// Short rows (at most 256 vectors) are taken by warps instead of CTAs, 2 KB at a time.
struct LogprobBwdArgs {
  int V, chunks;   // chunks: pieces of a row
  int64_t N, ld, ldd;
  const void* logits;
  const int32_t* target;
  const float *lse, *entropy, *g_logp, *g_entropy;
  void* dlogits;
  int* status;
};

constexpr int kBwdThreads = 256, kBwdVecs = 4;

// GROUP threads take a piece of GROUP * kBwdVecs vectors of a row.
template <typename T, int GROUP>
__global__ void __launch_bounds__(kBwdThreads) token_logprobs_bwd_kernel(const LogprobBwdArgs a) {
  constexpr int VE = 16 / sizeof(T), GROUPS = kBwdThreads / GROUP;
  const int t_in = threadIdx.x % GROUP;
  pdl_trigger();
  pdl_wait();
  for (int64_t item = (int64_t)blockIdx.x * GROUPS + threadIdx.x / GROUP; item < a.N * a.chunks;
       item += (int64_t)gridDim.x * GROUPS) {
    const int64_t row = item / a.chunks;
    const int chunk = (int)(item - row * a.chunks);
    const T* x = (const T*)a.logits + row * a.ld;
    T* d = (T*)a.dlogits + row * a.ldd;
    // element 0 of the row is element `head` of its first aligned vector
    const int head = (int)((uintptr_t)d & 15) / (int)sizeof(T);
    const bool same = (((uintptr_t)x ^ (uintptr_t)d) & 15) == 0;
    const int e0 = (chunk * GROUP * kBwdVecs + t_in) * VE - head;
    uint4 v[kBwdVecs];
#pragma unroll
    for (int i = 0; i < kBwdVecs; ++i) {
      const int e = e0 + i * GROUP * VE;
      if (same && e >= 0 && e + VE <= a.V) {
        v[i] = *reinterpret_cast<const uint4*>(x + e);
      } else {
        T* w = reinterpret_cast<T*>(&v[i]);
#pragma unroll
        for (int j = 0; j < VE; ++j)
          w[j] = e + j >= 0 && e + j < a.V ? x[e + j] : Elem<T>::from_f(0.f);
      }
    }
    int t = a.g_logp ? a.target[row] : -1;
    if (t >= a.V) {
      if (t_in == 0 && chunk == 0) report_status(a.status, XMOD_ERR_DEVICE_CHECK);
      t = -1;
    }
    const float g = t >= 0 ? a.g_logp[row] : 0.f, gh = a.g_entropy ? a.g_entropy[row] : 0.f;
    const bool zero = g == 0.f && gh == 0.f;
    const float lse = a.lse[row], ent = a.g_entropy ? a.entropy[row] : 0.f;
    const float2 neg = make_float2(-lse, -lse), lg = make_float2(kLog2e, kLog2e);
    // -(g + gH (y + H)) = -gH y - (g + gH H)
    const float b = -fmaf(gh, ent, g);
    const float2 mul = make_float2(-gh, -gh), add = make_float2(b, b);
#pragma unroll
    for (int i = 0; i < kBwdVecs; ++i) {
      const int e = e0 + i * GROUP * VE;
      if (e >= a.V || e + VE <= 0) continue;
      uint4 out;
#pragma unroll
      for (int j = 0; j < VE / 2; ++j) {
        float2 y = add2(vec_pair<T>(v[i], j), neg);
        const float2 tt = mul2(y, lg);
        const float2 p = make_float2(ex2(tt.x), ex2(tt.y));
        y.x = fmaxf(y.x, -1e4f);   // p is 0 long before; -infinity times 0 would be a NaN
        y.y = fmaxf(y.y, -1e4f);
        float2 r = mul2(p, fma2(mul, y, add));
        if (zero) r = make_float2(0.f, 0.f);
        if (e + 2 * j == t) r.x += g;
        if (e + 2 * j + 1 == t) r.y += g;
        set_vec_pair<T>(out, j, r);
      }
      if (e >= 0 && e + VE <= a.V) {
        *reinterpret_cast<uint4*>(d + e) = out;
      } else {
        const T* w = reinterpret_cast<const T*>(&out);
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (e + j >= 0 && e + j < a.V) d[e + j] = w[j];
      }
    }
  }
}

// ---------------------------------------------------------------- host

// Logits: any element of an array (vector accesses stay inside its aligned 16 bytes).
bool elem_ptr(const void* p, xmod_dtype dt) {
  return p && ((uintptr_t)p & (dt == XMOD_BF16 ? 1u : 3u)) == 0;
}
bool ptr4_or_null(const void* p) { return ((uintptr_t)p & 3u) == 0; }

template <typename T, bool ENT, int FIN>
cudaError_t launch_logprobs_fin(const Ctx& c, const LogprobArgs& a0) {
  LogprobArgs a = a0;
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // CTAs of a cluster share a row while there are SMs for them, two 16 KB chunks for each, and
  // not too many candidates to join (8 rows of 50257, bf16, one, two, four CTAs a row: without
  // alternatives 6.3, 5.0, 4.5 us; 5 of them 8.9, 8.3, 8.1; 20 of them 10.6, 10.5, 11.5)
  a.splits = 1;
  while (a.splits < 8 && a.N * a.splits * 2 <= sms && a.splits * 2 * a.top_k <= 48 &&
         (int64_t)a.V * sizeof(T) >= 2 * a.splits * (int64_t)kChunk)
    a.splits *= 2;
  a.per = (a.V + a.splits - 1) / a.splits;
  constexpr int smem = kLpStages * kChunk + (int)sizeof(LpShared);
  static_assert(kLpCtas * (smem + 1024) <= 228 * 1024, "");
  auto kernel = token_logprobs_kernel<T, ENT, FIN>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kernel, smem, done);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)sms * kLpCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.splits > 1 ? a.N * a.splits : a.N < most ? a.N : most));
  cfg.blockDim = dim3(kLpThreads + 32 * FIN + 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Short rows go to warps. Else a second finisher where one would hold the rows up: rows of one
// or two chunks, or many alternatives (it costs the others registers and issue slots). 4096
// rows, bf16, one and two finishers, in us: 5 alternatives of 5000 logits 32.5 and 26.5, of 8191
// 38.1 and 34.1, of 16000 44.8 and 41.2, of 20000 47.9 and 47.1, of 24000 51.6 and 52.0, of 32000
// 59.1 and 61.7, of 50257 76.6 and 80.7; of 50257 20 alternatives 96.8 and 97.9, 32 113 and 108,
// 40 127 and 116, 64 184 and 147.
template <typename T, bool ENT>
cudaError_t launch_logprobs(const Ctx& c, const LogprobArgs& a) {
  const int VE = 16 / (int)sizeof(T);
  if (((int64_t)a.V + 2 * VE - 2) / VE <= 32 * kShortVecs && a.top_k <= kShortTopK) {
    const int sms = device_sms();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const int64_t ctas = (a.N + kShortWarps - 1) / kShortWarps, most = (int64_t)sms * 16;
    return launch_pdl(token_logprobs_short_kernel<T, ENT>, dim3((unsigned)(ctas < most ? ctas : most)),
                      dim3(kShortWarps * 32), 0, c.stream, a);
  }
  return a.top_k > 32 || (a.top_k && (int64_t)a.V * sizeof(T) <= 2 * kChunk)
             ? launch_logprobs_fin<T, ENT, 2>(c, a)
             : launch_logprobs_fin<T, ENT, 1>(c, a);
}

template <typename T, int GROUP>
cudaError_t launch_logprobs_bwd_group(const Ctx& c, const LogprobBwdArgs& a0, int64_t vecs) {
  LogprobBwdArgs a = a0;
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  a.chunks = (int)((vecs + GROUP * kBwdVecs - 1) / (GROUP * kBwdVecs));
  const int64_t items = a.N * a.chunks, groups = kBwdThreads / GROUP;
  const int64_t ctas = (items + groups - 1) / groups, most = (int64_t)sms * 64;
  return launch_pdl(token_logprobs_bwd_kernel<T, GROUP>, dim3((unsigned)(ctas < most ? ctas : most)),
                    dim3(kBwdThreads), 0, c.stream, a);
}

template <typename T>
cudaError_t launch_logprobs_bwd(const Ctx& c, const LogprobBwdArgs& a) {
  const int VE = 16 / (int)sizeof(T);
  const int64_t vecs = ((int64_t)a.V + 2 * VE - 2) / VE;   // of a row at the worst alignment
  return vecs <= 256 ? launch_logprobs_bwd_group<T, 32>(c, a, vecs)
                     : launch_logprobs_bwd_group<T, kBwdThreads>(c, a, vecs);
}

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
  if (!elem_ptr(logits, dt)) return XMOD_ERR_INVALID_ARG;
  const void* ps[] = {target, logp, entropy, lse, top_idx, top_logp, status_out};
  for (const void* p : ps)
    if (!ptr4_or_null(p)) return XMOD_ERR_INVALID_ARG;
  if (top_k > XMOD_MAX_TOP_K || N > INT32_MAX || V > XMOD_MAX_VOCAB) return XMOD_ERR_UNSUPPORTED;
  const LogprobArgs a{V, top_k, 1, V, N, ld, logits, target, logp, entropy, lse, top_idx, top_logp,
                      status_out};
  const Ctx c{(cudaStream_t)stream, status_out};
  if (dt == XMOD_BF16)
    XMOD_LAUNCH(c, "token_logprobs", (entropy ? launch_logprobs<__nv_bfloat16, true>(c, a)
                                              : launch_logprobs<__nv_bfloat16, false>(c, a)));
  else
    XMOD_LAUNCH(c, "token_logprobs",
                (entropy ? launch_logprobs<float, true>(c, a) : launch_logprobs<float, false>(c, a)));
  return XMOD_OK;
}

int xmod_token_logprobs_bwd(xmod_dtype dt, int64_t N, int V, const void* logits, int64_t ld,
                            const int32_t* target, const float* lse, const float* entropy,
                            const float* g_logp, const float* g_entropy, void* dlogits,
                            int64_t ldd, int* status_out, void* stream) {
  if ((dt != XMOD_BF16 && dt != XMOD_FP32) || N < 0 || V <= 0 || ld < V || ldd < V)
    return XMOD_ERR_INVALID_ARG;
  if (N == 0) return XMOD_OK;
  if (!elem_ptr(logits, dt) || !elem_ptr(dlogits, dt) || !lse || (g_logp && !target) ||
      (g_entropy && !entropy) || (dlogits == logits && ldd != ld))
    return XMOD_ERR_INVALID_ARG;
  const void* ps[] = {target, lse, entropy, g_logp, g_entropy, status_out};
  for (const void* p : ps)
    if (!ptr4_or_null(p)) return XMOD_ERR_INVALID_ARG;
  if (N > INT32_MAX || V > XMOD_MAX_VOCAB) return XMOD_ERR_UNSUPPORTED;
  const LogprobBwdArgs a{V, 1, N, ld, ldd, logits, target, lse, entropy, g_logp, g_entropy,
                         dlogits, status_out};
  const Ctx c{(cudaStream_t)stream, status_out};
  if (dt == XMOD_BF16)
    XMOD_LAUNCH(c, "token_logprobs_bwd", launch_logprobs_bwd<__nv_bfloat16>(c, a));
  else
    XMOD_LAUNCH(c, "token_logprobs_bwd", launch_logprobs_bwd<float>(c, a));
  return XMOD_OK;
}

}  // extern "C"
