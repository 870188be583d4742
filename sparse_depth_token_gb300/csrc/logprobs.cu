// Log probabilities of given tokens with the entropy and the largest alternatives, and
// their gradient at the logits.

#include <cuda_bf16.h>
#include <float.h>
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
// sign. A bf16 logit costs 5 instructions (4 without the entropy), half of the issue
// slots at the full memory rate: the kernel is bound by memory, and laid out to keep
// reading. A CTA works rows off one after the other: a producer warp keeps bulk copies into a
// ring of 16 KB chunks going, across row ends, and eight warps consume them, each at its own
// pace but for the first chunk and the end of a row. Few rows are split over the CTAs of a
// cluster, which join through distributed shared memory.
//
// The alternatives. Logits are ranked by 64-bit keys, the value's order above the inverted
// token number: keys are distinct, so ties need no care. The k-th largest of the maxima of
// groups of threads in a row's first chunk is a bound: k logits are at least that large, and
// few are. The row's candidates are the first chunk's logits at or above it and the later
// ones above it (one that equals it loses the tie to those k); a warp looks at one thread's
// logits of a chunk at a time, a lane each. At the row's end they are ranked by counting the
// larger ones. Should there be more than the buffer holds (rising or constant rows), the row
// is read once more for every alternative; a row with fewer than k tokens above -infinity is
// filled up from its first tokens.

constexpr int kLpThreads = 256;    // consumers; one more warp produces
constexpr int kChunk = 16384;      // bytes
constexpr int kLpStages = 3;
constexpr int kVecs = kChunk / 16 / kLpThreads;   // vectors a thread takes of a chunk
constexpr int kMaxCandidates = 1296;   // 2 x 10 KB: three CTAs an SM with the ring

struct LogprobArgs {
  int V, top_k, splits, per, capacity;   // per: logits of a split; capacity: candidates
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
    u = l > 0.f ? f * fmaf(d, l, u) : 0.f;
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
  return (s.nvec * 16 + kChunk - 1) / kChunk;
}

// Shared memory behind the ring.
struct alignas(16) LpShared {
  uint64_t full[kLpStages], empty[kLpStages];
  uint32_t least;           // the row's bound, in orders
  int found, abort;
  int counts[kLpThreads / 32 + 1];   // candidates of the warps, and those filled up
  Moments moments[2][kLpThreads / 32];   // of even and odd rows: a warp may be a row ahead
  Moments total;
  alignas(16) uint32_t group_max[kLpThreads];
  alignas(16) uint64_t top[XMOD_MAX_TOP_K];   // this CTA's best, in order
};

// Threads whose maxima stand together for the bound: at least 4 top_k groups (fewer give a
// looser bound, more cost more to rank).
__device__ __forceinline__ int lp_group(int top_k) {
  return top_k <= 8 ? 8 : top_k <= 16 ? 4 : top_k <= 32 ? 2 : 1;
}

constexpr uint32_t kOrderNone = 0x007fffffu;   // order_of(-infinity)

__device__ __forceinline__ void sync_consumers() {
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(kLpThreads) : "memory");
}

template <typename T, bool ENT>
__global__ void __launch_bounds__(kLpThreads + 32, 3) token_logprobs_kernel(const LogprobArgs a) {
  constexpr int VE = 16 / sizeof(T);
  extern __shared__ __align__(128) uint8_t smem[];
  LpShared& sh = *reinterpret_cast<LpShared*>(smem + kLpStages * kChunk);
  uint64_t* cand = reinterpret_cast<uint64_t*>(&sh + 1);   // the warps' lists, the filled up
  uint64_t* joined = cand + a.capacity;                    // and all together
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = a.splits > 1 ? (int)cluster_ctarank() : 0;
  const int64_t row0 = blockIdx.x / a.splits, row_step = gridDim.x / a.splits;
  const int k = a.top_k, capw = a.capacity / (kLpThreads / 32 + 1);   // candidates of a warp
  volatile int* abort_flag = &sh.abort;
  const uint32_t bFull = smem_u32(&sh.full[0]), bEmpty = smem_u32(&sh.empty[0]);

  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < kLpStages; ++i) {
      mbar_init(bFull + 8 * i, 1);
      mbar_init(bEmpty + 8 * i, kLpThreads / 32);
    }
    sh.abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();

  if (warp == kLpThreads / 32) {
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
    if (a.splits > 1) {   // the consumers' two, for the cluster's one row
      cluster_sync_all();
      cluster_sync_all();
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  // A wait that gives up (abort) lets the loops run on over what the ring holds: every warp
  // still meets the others' barriers.
  int stage = 0;
  uint32_t phase = 0;
  int parity = 0;
  const bool has_target = split == 0 && tid == 0 && a.logp;
  int next_target = has_target && row0 < a.N ? a.target[row0] : -1;
  for (int64_t row = row0; row < a.N; row += row_step, parity ^= 1) {
    const Span s = span_of<T>(a, row, split);
    const int chunks = span_chunks(s);
    // the target's logit, on its way while the row is read; the next row's target too
    float x_t = 0.f;
    const int target = next_target;
    if (target >= 0 && target < a.V) x_t = Elem<T>::to_f(((const T*)a.logits + row * a.ld)[target]);
    if (has_target && row + row_step < a.N) next_target = a.target[row + row_step];
    int mine_n = 0;   // this warp's candidates
    Moments mo{-FLT_MAX, 0.f, 0.f};
    float2 l2 = make_float2(0.f, 0.f), u2 = l2;
    uint32_t bound = kOrderNone;
    float thr = -INFINITY;   // candidates are above it
    const int lane_vec = lane / VE * kLpThreads;   // from a thread's first vector to the lane's
    auto tail_index = [&](int v) {   // the lane's element of vector v, the row's last at most
      return min(v * VE + lane % VE, s.head + s.count - 1);
    };
    for (int c = 0; c < chunks; ++c) {
      mbar_wait(bFull + 8 * stage, phase, abort_flag, a.status);
      const uint4* buf = reinterpret_cast<const uint4*>(smem + stage * kChunk);
      const int v0 = c * (kChunk / 16);
      uint4 x[kVecs];
#pragma unroll
      for (int i = 0; i < kVecs; ++i) x[i] = buf[tid + i * kLpThreads];
      const bool whole = c > 0 && v0 + kChunk / 16 <= s.full;
      if (!whole) {   // the row's ends
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
          const int v = v0 + tid + i * kLpThreads;
          if (v >= s.full) {   // past the row, or its last elements: one by one
            const uint32_t ninf = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
            x[i] = make_uint4(ninf, ninf, ninf, ninf);
            if (v < s.nvec) {
              const T* p = reinterpret_cast<const T*>(s.vecs + v);
              T* e = reinterpret_cast<T*>(&x[i]);
#pragma unroll
              for (int j = 0; j < VE; ++j)
                if (v * VE + j < s.head + s.count) e[j] = p[j];
            }
          }
          if (v == 0) {
#pragma unroll
            for (int j = 0; j < VE; ++j)
              if (j < s.head) vec_clear<T>(x[i], j);
          }
        }
      }
      float top = vec_max<T>(x[0]);
#pragma unroll
      for (int i = 1; i < kVecs; ++i) top = max_nan(top, vec_max<T>(x[i]));
      if (!(top <= mo.m)) {   // larger, or a NaN: that one makes l 0 and the row bad
        const float d = (mo.m - (top != top ? INFINITY : top)) * kLog2e, f = ex2(d);
        const float2 f2 = make_float2(f, f), d2 = make_float2(d, d);
        if (ENT) u2 = l2.x + l2.y > 0.f ? mul2(f2, fma2(d2, l2, u2)) : make_float2(0.f, 0.f);
        l2 = mul2(l2, f2);
        mo.m = top != top ? INFINITY : top;
      }
      if (fabsf(mo.m) < 1e36f) {
        const float2 neg = make_float2(-mo.m, -mo.m), lg = make_float2(kLog2e, kLog2e);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
          if (!whole && v0 + warp * 32 + i * kLpThreads >= s.nvec) break;   // nothing left
          // an infinite exponent times 0 would be a NaN: such logits become low finite ones,
          // whose terms are 0 as well
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
      } else if (mo.m > -FLT_MAX) {   // differences that could overflow
#pragma unroll
        for (int i = 0; i < kVecs * VE; ++i) {
          const float d = fmaxf(vec_at<T>(x[i / VE], i % VE) - mo.m, -1e30f) * kLog2e, e = ex2(d);
          l2.x += e;
          if (ENT) u2.x = fmaf(e, d, u2.x);
        }
      }
      if (k) {
        if (c == 0) {   // the row's bound
          const int lanes = lp_group(k), groups = kLpThreads / lanes;
          uint32_t best = tid < s.nvec ? order_of(top) : 0u;
          for (int o = 1; o < lanes; o <<= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
          if (tid % lanes == 0) sh.group_max[tid / lanes] = best;
          if (tid == 0) sh.least = 0;
          sync_consumers();
          uint32_t g = 0;
          if (groups == 32 || tid < groups) {   // 32 groups: every warp for itself
            g = sh.group_max[groups == 32 ? lane : tid];
            int gt = 0, ge = 0;
#pragma unroll 4
            for (int j = 0; j < groups; j += 4) {
              const uint4 o = *reinterpret_cast<const uint4*>(&sh.group_max[j]);
              gt += (o.x > g) + (o.y > g) + (o.z > g) + (o.w > g);
              ge += (o.x >= g) + (o.y >= g) + (o.z >= g) + (o.w >= g);
            }
            if (gt >= k || ge < k) g = 0;
          }
          if (groups == 32) {
            g = __reduce_max_sync(0xffffffffu, g);
          } else {
            if (g) sh.least = g;   // one value, whoever writes it
            sync_consumers();
            g = sh.least;
          }
          // later logits have to be above the bound (one equal to it loses to the k that reach
          // it), this chunk's at it; none at -infinity is in. g 0: fewer than k groups hold any
          bound = max(g, kOrderNone);
          const uint32_t below = bound - (bound == 0x80000000u ? 2 : 1);   // 0: -0 equals it
          thr = value_of(max(below, kOrderNone));
        }
        uint32_t todo = __ballot_sync(0xffffffffu, !(top <= thr));
        while (todo) {   // a thread's logits of the chunk, one a lane
          const int from = warp * 32 + __ffs(todo) - 1;
          todo &= todo - 1;
          float f = -INFINITY;
          if (lane < kVecs * VE) {
            if (whole || v0 + from + lane_vec < s.full)
              f = Elem<T>::to_f(reinterpret_cast<const T*>(buf + from)[lane_vec * VE + lane % VE]);
            else if (v0 + from + lane_vec < s.nvec)
              f = Elem<T>::to_f(reinterpret_cast<const T*>(s.vecs)[tail_index(v0 + from + lane_vec)]);
          }
          const int e = (v0 + from + lane_vec) * VE + lane % VE - s.head;
          const bool in = !(f <= thr) && (whole || (e >= 0 && e < s.count));
          const uint32_t who = __ballot_sync(0xffffffffu, in);
          const int at = mine_n + __popc(who & ((1u << lane) - 1u));
          mine_n += __popc(who);
          if (in && at < capw) cand[warp * capw + at] = key_of(f, s.token0 + e);
        }
        if (c == 0) thr = value_of(bound);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bEmpty + 8 * stage);
      if (++stage == kLpStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    // ---- the row's end: this CTA's sums and candidates
    mo.l = l2.x + l2.y;
    mo.u = u2.x + u2.y;
    mo.raise(warp_max(mo.m));
    mo.l = warp_sum(mo.l);
    if (ENT) mo.u = warp_sum(mo.u);
    if (lane == 0) {
      sh.moments[parity][warp] = mo;
      sh.counts[warp] = mine_n;
      if (warp == 0) sh.counts[kLpThreads / 32] = 0;
    }
    sync_consumers();
    // the k best of `count` candidates to sh.top, in order: those in the lists of counts[],
    // `stride` apart, are put together and ranked by counting the larger ones
    auto rank = [&](int lists, int stride, int count) {
      for (int i = tid; i < count; i += kLpThreads) {
        int list = 0, j = i;
        while (j >= sh.counts[list]) j -= sh.counts[list++];
        joined[i] = cand[list * stride + j];
      }
      if (tid == 0) joined[count] = 0;   // pairs below
      sync_consumers();
      for (int i = tid; i < count; i += kLpThreads) {
        const uint64_t mine = joined[i];
        int above = 0;
#pragma unroll 4
        for (int j = 0; j < count; j += 2) {
          const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&joined[j]);
          above += (o.x > mine) + (o.y > mine);
        }
        if (above < k) sh.top[above] = mine;
      }
      sync_consumers();
    };
    int found = 0;
    if (k) {
      constexpr int W = kLpThreads / 32;
      bool full = false;
      for (int w = 0; w < W; ++w) {
        found += sh.counts[w];
        full |= sh.counts[w] > capw;
      }
      const T* p = (const T*)a.logits + row * a.ld + s.token0;
      if (found < k) {
        // the rest are tokens at -infinity: the lowest, among the first 2 k
        if (tid < min(2 * k, s.count) && order_of(Elem<T>::to_f(p[tid])) == kOrderNone)
          cand[W * capw + atomicAdd(&sh.counts[W], 1)] = key_of(-INFINITY, s.token0 + tid);
        sync_consumers();
        found += sh.counts[W];
      }
      if (!full) {
        rank(W + 1, capw, found);
      } else {   // too many: one reading for each alternative, the largest key below the last
        uint64_t last = ~0ull;
        for (int i = 0; i < min(k, s.count); ++i) {
          unsigned long long best = 0;
          for (int e = tid; e < s.count; e += kLpThreads) {
            const uint64_t key = key_of(Elem<T>::to_f(p[e]), s.token0 + e);
            if (key < last && key > best) best = key;
          }
          for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
          if (lane == 0) cand[warp] = best;
          sync_consumers();
          for (int w = 0; w < W; ++w) best = max(best, (unsigned long long)cand[w]);
          last = best;
          if (tid == 0) sh.top[i] = best;
          sync_consumers();
        }
      }
      found = min(found, min(k, s.count));
    }
    // the first warp finishes the row; the others meet it again at the next row's barriers,
    // before anything that it reads here is written
    if (a.splits == 1 && warp != 0) continue;
    mo = sh.moments[parity][lane % (kLpThreads / 32)];
    mo.raise(warp_max(mo.m));
    if (lane >= kLpThreads / 32) mo.l = mo.u = 0.f;
    mo.l = warp_sum(mo.l);
    mo.u = warp_sum(mo.u);
    if (a.splits > 1) {
      if (tid == 0) {
        sh.total = mo;
        sh.found = found;
      }
      cluster_sync_all();
      if (split == 0) {
        int all = 0;
        for (int r = 0; r < a.splits; ++r) {
          const uint32_t at = mapa_shared(smem_u32(&sh.total), r);
          Moments other;
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(other.m) : "r"(at) : "memory");
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(other.l) : "r"(at + 4) : "memory");
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(other.u) : "r"(at + 8) : "memory");
          if (r == 0) {
            mo = other;
          } else {
            const float m2 = fmaxf(mo.m, other.m);
            mo.raise(m2);
            other.raise(m2);
            mo.l += other.l;
            mo.u += other.u;
          }
          if (k) {
            int n;
            asm volatile("ld.shared::cluster.s32 %0, [%1];"
                         : "=r"(n)
                         : "r"(mapa_shared(smem_u32(&sh.found), r))
                         : "memory");
            if (tid < n)
              asm volatile("ld.shared::cluster.u64 %0, [%1];"
                           : "=l"(cand[r * XMOD_MAX_TOP_K + tid])
                           : "r"(mapa_shared(smem_u32(&sh.top[0]), r) + 8 * tid)
                           : "memory");
            if (tid == 0) sh.counts[r] = n;
            all += n;
          }
        }
        sync_consumers();
        if (k) rank(a.splits, XMOD_MAX_TOP_K, all);
      }
      cluster_sync_all();   // the other CTAs' shared memory has been read
      if (split != 0 || warp != 0) continue;
    }
    const bool bad = !(mo.l > 0.f);   // nothing above -infinity, a NaN or +infinity
    const float ll = logf(mo.l), nan = __int_as_float(0x7fc00000);
    if (tid == 0) {
      if (bad || target >= a.V) report_status(a.status, XMOD_ERR_DEVICE_CHECK);
      if (a.lse) a.lse[row] = bad ? nan : mo.m + ll;
      if (a.entropy) a.entropy[row] = bad ? nan : ll - 0.6931471805599453f * mo.u / mo.l;
      if (a.logp) a.logp[row] = target < 0 ? 0.f : bad || target >= a.V ? nan : (x_t - mo.m) - ll;
    }
    for (int i = lane; i < k; i += 32) {
      const uint64_t key = sh.top[i];
      a.top_idx[row * k + i] = token_of(key);
      a.top_logp[row * k + i] = bad ? nan : (value_of((uint32_t)(key >> 32)) - mo.m) - ll;
    }
  }
}

// ---------------------------------------------------------------- gradient
//
// dx_v = g (1[v = t] - p_v) - gH p_v (ln p_v + H): one reading and one writing of the
// logits' size, 5 instructions a logit: bound by memory. A CTA takes 16 KB of a row, four
// 16-byte vectors a thread, aligned in the output; where the logits' rows are aligned
// differently (another row stride), their elements are loaded one by one, which the L1
// cache makes up for.
struct LogprobBwdArgs {
  int V, chunks;
  int64_t N, ld, ldd;
  const void* logits;
  const int32_t* target;
  const float *lse, *entropy, *g_logp, *g_entropy;
  void* dlogits;
  int* status;
};

template <typename T>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_bwd_kernel(const LogprobBwdArgs a) {
  constexpr int VE = 16 / sizeof(T);
  pdl_trigger();
  pdl_wait();
  for (int64_t item = blockIdx.x; item < a.N * a.chunks; item += gridDim.x) {
    const int64_t row = item / a.chunks;
    const int chunk = (int)(item - row * a.chunks);
    const T* x = (const T*)a.logits + row * a.ld;
    T* d = (T*)a.dlogits + row * a.ldd;
    // element 0 of the row is element `head` of its first aligned vector
    const int head = (int)((uintptr_t)d & 15) / (int)sizeof(T);
    const bool same = (((uintptr_t)x ^ (uintptr_t)d) & 15) == 0;
    const int e0 = (chunk * (kChunk / 16) + (int)threadIdx.x) * VE - head;
    uint4 v[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int e = e0 + i * kLpThreads * VE;
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
      if (threadIdx.x == 0 && chunk == 0) report_status(a.status, XMOD_ERR_DEVICE_CHECK);
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
    for (int i = 0; i < kVecs; ++i) {
      const int e = e0 + i * kLpThreads * VE;
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

bool ptr16(const void* p) { return p && ((uintptr_t)p & 15u) == 0; }
bool ptr4_or_null(const void* p) { return ((uintptr_t)p & 3u) == 0; }

template <typename T, bool ENT>
cudaError_t launch_logprobs(const Ctx& c, const LogprobArgs& a0) {
  LogprobArgs a = a0;
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // CTAs of a cluster share a row while there are SMs for them and 16 KB chunks enough
  a.splits = 1;
  while (a.splits < 8 && a.N * a.splits * 2 <= sms && (int64_t)a.V * sizeof(T) >= 2 * a.splits * (int64_t)kChunk)
    a.splits *= 2;
  a.per = (a.V + a.splits - 1) / a.splits;
  // about top_k logits of every chunk's size are above a bound from one chunk
  const int64_t want = 2 * (int64_t)a.top_k * ((int64_t)a.per * sizeof(T) / kChunk + 1);
  const int lists = kLpThreads / 32 + 1;   // of at least 128: a list may fill up 2 top_k
  a.capacity = !a.top_k ? 0 : want < 128 * lists ? 128 * lists : want < kMaxCandidates ? (int)want / lists * lists : kMaxCandidates;
  a.capacity += a.capacity & 1;
  const int smem = kLpStages * kChunk + (int)sizeof(LpShared) + 16 * a.capacity + 16;
  auto kernel = token_logprobs_kernel<T, ENT>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kernel, kLpStages * kChunk + (int)sizeof(LpShared) +
                                         16 * kMaxCandidates + 16, done);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)sms * 3;   // resident: by registers, and by shared memory
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.splits > 1 ? a.N * a.splits : a.N < most ? a.N : most));
  cfg.blockDim = dim3(kLpThreads + 32);
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

template <typename T>
cudaError_t launch_logprobs_bwd(const Ctx& c, const LogprobBwdArgs& a0) {
  LogprobBwdArgs a = a0;
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int VE = 16 / (int)sizeof(T);
  // vectors of a row at the worst alignment, in chunks
  a.chunks = (int)(((int64_t)a.V + 2 * VE - 2) / VE / (kChunk / 16)) + 1;
  const int64_t items = a.N * a.chunks, most = (int64_t)sms * 64;
  return launch_pdl(token_logprobs_bwd_kernel<T>, dim3((unsigned)(items < most ? items : most)),
                    dim3(kLpThreads), 0, c.stream, a);
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
  if (!ptr16(logits)) return XMOD_ERR_INVALID_ARG;
  const void* ps[] = {target, logp, entropy, lse, top_idx, top_logp, status_out};
  for (const void* p : ps)
    if (!ptr4_or_null(p)) return XMOD_ERR_INVALID_ARG;
  if (top_k > XMOD_MAX_TOP_K || N > INT32_MAX || V > INT32_MAX - 65536) return XMOD_ERR_UNSUPPORTED;
  const LogprobArgs a{V, top_k, 1, V, 0, N, ld, logits, target, logp, entropy, lse, top_idx, top_logp,
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
  if (!ptr16(logits) || !ptr16(dlogits) || !lse || (g_logp && !target) ||
      (g_entropy && !entropy) || (dlogits == logits && ldd != ld))
    return XMOD_ERR_INVALID_ARG;
  const void* ps[] = {target, lse, entropy, g_logp, g_entropy, status_out};
  for (const void* p : ps)
    if (!ptr4_or_null(p)) return XMOD_ERR_INVALID_ARG;
  if (N > INT32_MAX || V > INT32_MAX - 65536) return XMOD_ERR_UNSUPPORTED;
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
