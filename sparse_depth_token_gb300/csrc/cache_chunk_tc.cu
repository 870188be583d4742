// Attention of a chunk of new tokens over the paged cache on the tcgen05 tensor cores: bf16
// queries over a bf16 or an e4m3 cache.
//
//   o = sum_i p_i V_i,  p = softmax_i(q . K_i / sqrt(hd)),  i < the row's limit
//
// One persistent CTA per SM takes its range of the tile list (cache_chunk.cuh). A segment is two
// MMA tiles, A and B, of 128 query rows each (a row is a token and a query head of one KV head),
// which share every 64-key tile of K and V. Roles:
//   warp 0        TMA of K and V (pages gathered box by box) into rings of stages, K a tile ahead
//   warps 1, 3    they issue A's and B's S = Q K^T (two buffers each, a tile ahead)
//                 and O += P V; warp 1 owns the tensor memory
//   warp 2        the segments' descriptions, and TMA of their query rows, the next segment's as
//                 soon as the last S of this one has been computed
//   warps 4..7    softmax of A, a row a thread: scores from tensor memory, running maximum and
//   warps 8..11   sum, P back over the scores as bf16; the same for B
//   warps 12..15  (e4m3) codes to bf16, exactly
// The reference of the weights, a maximum, only moves when it grows by more than 2^8 (weights stay below 256 and
// keep their relative rounding in bf16); O is then rescaled in tensor memory.
//
// V is used as the cache stores it, [slot, dimension], as an MN-major operand: nothing is
// transposed. A slot that a row does not see must not touch it even if it holds an infinity or
// NaN, which a weight of 0 does not ensure. So in the tiles that some row of the segment sees
// only in part, the softmax warps look at V first: slots past the segment's end become zeros;
// and if another slot that some row does not see holds such a value, those values are added by
// hand to the rows that see them and then replaced by zeros.
//
// Bound by the tensor pipe and its issue beside the softmax warps: 500 tokens at 131072 of 16
// and 4 heads of 128 380 us (1.41 PFLOP/s, 0.74 of the measured burst; at the power cap 406-423), six
// prompts of up to 8192 tokens 990 us (1.40; at the cap 1057-1082; a segment's start and end cost about four
// of its tiles). Over e4m3 by issue: 16 ragged chunks at up to 16384 238 us (0.68 PFLOP/s). Small
// calls by latency: eight chunks of 4 tokens over 4096 29 us with the join, whose plan takes 3.
//
// The weights are rounded to bf16 (8 bits): P is an operand of the same MMA as V and kind::f16 takes
// one type for both. Two bf16 parts of P would keep 16 bits, as the attention of single tokens does, at
// half again the MMAs (twice P V), of the pipe that bounds long chunks. The sums l take the weights
// before the rounding.

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <float.h>
#include <math.h>

#include <atomic>

#include "cache_chunk.cuh"
#include "tc_common.cuh"

namespace xmod {

namespace {

using namespace tc;

constexpr int KB = kChunkKeys;
constexpr int QR = kChunkTcRows;
constexpr float kRescale = 8.0f;   // log2 units

// Whether a wait that ran out has to give up. Some roles wait as long as a segment takes, which has no
// bound (2 s at 146 million slots): not if the loads, of which the word after the abort flag counts
// 1024 tiles at a time, went on since this thread asked last, a limit's time ago; behind it every
// thread has what it saw then. (Kept in the wait's own registers this costs 2 % of the kernel's time.)
__device__ __noinline__ bool stalled(volatile int* abort_flag, int* status) {
  volatile uint16_t* const seen = reinterpret_cast<volatile uint16_t*>(abort_flag + 2) + threadIdx.x;
  const uint16_t now = (uint16_t)(abort_flag[1] | 0x8000);   // 0: has not asked yet
  if (*seen != now) {
    *seen = now;
    return false;
  }
  report_status(status, XMOD_ERR_TIMEOUT);
  *abort_flag = 1;
  return true;
}
// The bounded wait with everything but its first test out of line: it stands in every loop here,
// whose code has to stay small.
__device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = global_timer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 0u) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        if (stalled(abort_flag, status)) return false;
        t0 = global_timer_ns();
      }
    }
  }
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) ok = wait_longer(bar, parity, abort_flag, status);
  return __all_sync(0xffffffffu, ok);   // the whole warp calls it
}

template <int HD, bool FP8> struct Tc {
  static constexpr int RB = HD >= 64 ? 128 : 64;            // bytes of a swizzled row
  static constexpr int HALVES = HD * 2 / RB;                // of a head's dimensions
  static constexpr int Q_HALF = 128 * RB, Q_TILE = HALVES * Q_HALF;
  static constexpr int K_HALF = KB * RB, K_TILE = HALVES * K_HALF;
  static constexpr int NK = FP8 ? 3 : HD == 128 ? 4 : HD == 64 ? 6 : 8;   // stages of K, and of V
  static constexpr int CRB = HD >= 128 ? 128 : HD;          // bytes of a row of codes
  static constexpr int CODES = FP8 ? KB * HD : 0;           // of K, and of V
  static constexpr int NC = FP8 ? 3 : 0;
  static constexpr int SCALES = FP8 ? 2 * KB * 4 : 0;
  // where a warp turns its rows of the output: 32 rows of OUT columns, padded
  static constexpr int OUT = FP8 && HD == 128 ? 16 : 32, OUT_LD = OUT * 2 + 16, TURN = 8 * 32 * OUT_LD;
  static constexpr int DATA = 2 * Q_TILE + 2 * NK * K_TILE + NC * (2 * CODES + SCALES) + NK * SCALES + TURN;
  static constexpr int MISC = 2048 + 512;
  static constexpr int SMEM = DATA + MISC + 1024;
  static constexpr int THREADS = FP8 ? 512 : 384;
  static constexpr int TMEM_COLS = 512;                     // S: 4 x 64, O: 2 x HD
  static constexpr int SW = RB == 128 ? 2 : 4;              // descriptor's swizzle code
  static_assert(SMEM <= 227 * 1024, "");
};

// A segment in a CTA's range, as the loader describes it to the softmax warps.
struct Segment {
  Chunk k;
  int hp, t, tiles, limit, first, last;   // tiles first .. last - 1 are this CTA's; first < 0: no more
  int both;                               // B has rows
};
constexpr int kSegments = 4;

__device__ __forceinline__ bool segment_both(const ChunkArgs& a, const Chunk& k, int t) {
  return k.n - t * a.tpt > a.block_tokens;
}

// K-major operand: rows of RB bytes, groups of 8 rows RB * 8 bytes apart.
template <int RB, int SW> __device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)1 << 16 | (uint64_t)((8 * RB) >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)SW << 61;
}
// MN-major operand: atoms of RB bytes (MN) x 8 rows (K), the atoms along K 8 * RB bytes apart,
// those along MN `stride`.
template <int RB, int SW> __device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t stride) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)((stride >> 4) & 0x3FFFu) << 16 |
         (uint64_t)((8 * RB) >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)SW << 61;
}

// Byte offset of 16-byte chunk c of row r in a tile of `rows` rows.
template <int RB> __device__ __forceinline__ uint32_t swizzled(int r, int c, int rows) {
  constexpr int CH = RB / 16;
  const int x = RB == 128 ? (r & 7) : RB == 64 ? ((r >> 1) & 3) : ((r >> 2) & 1);
  return (uint32_t)((c / CH) * rows * RB + r * RB + (((c % CH) ^ x) << 4));
}

// The tensor-core instructions of a whole warp, issued by one elected lane.
__device__ __forceinline__ void mma_elected(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_tmem_a_elected(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {   // accumulates
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc)
      : "memory");
}
__device__ __forceinline__ void commit_elected(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

__device__ __forceinline__ void sts128(uint32_t at, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Nonzero if one of the two bf16 of w is an infinity or NaN.
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// Two e4m3 codes to bf16, exactly, by way of f16 and fp32 (NaN included; moving the bits to their
// places by hand takes more instructions). The conversion itself ends at f16; the operands are bf16
// because the queries are, whose range f16 has not.
__device__ __forceinline__ uint32_t codes2_bf16(uint32_t codes) {
  const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3));
  const float2 f = __half22float2(h);
  return pack_bf16x2(f.x, f.y);
}
__device__ __forceinline__ void codes_bf16(const uint4& u, uint4& lo, uint4& hi) {
  lo = make_uint4(codes2_bf16(u.x & 0xffffu), codes2_bf16(u.x >> 16), codes2_bf16(u.y & 0xffffu), codes2_bf16(u.y >> 16));
  hi = make_uint4(codes2_bf16(u.z & 0xffffu), codes2_bf16(u.z >> 16), codes2_bf16(u.w & 0xffffu), codes2_bf16(u.w >> 16));
}

// log2 of the significand of the value's scale that belongs to the largest of a row's scores (in
// tensor memory; sc: the keys' scales, then the values'; those below `seen`).
__device__ __noinline__ float scale_shift(uint32_t scores, const float* sc, int seen) {
  float top = -INFINITY, s = 1.0f;
#pragma unroll 1
  for (int c = 0; c < KB; c += 32) {
    float v[32];
    tmem_ld32(scores + c, v);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float x = v[i] * sc[c + i];
      if (c + i < seen && x > top) {
        top = x;
        s = sc[KB + c + i];
      }
    }
  }
  return log2f(__uint_as_float((__float_as_uint(s) & 0x7fffffu) | 0x3f800000u));
}

template <int HD, bool FP8>
__global__ void __launch_bounds__((Tc<HD, FP8>::THREADS), 1)
cache_chunk_tc_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                      const __grid_constant__ CUtensorMap mV, const ChunkArgs a) {
  using C = Tc<HD, FP8>;
  constexpr int NK = C::NK, RB = C::RB;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const uint32_t sQ = base, sK = sQ + 2 * C::Q_TILE, sV = sK + NK * C::K_TILE;
  const uint32_t sCode = sV + NK * C::K_TILE;                       // stages: K codes, V codes
  const uint32_t sCodeScale = sCode + C::NC * 2 * C::CODES;         // stages: K scales, V scales
  const uint32_t sScale = sCodeScale + C::NC * C::SCALES;           // the same beside the V stages
  const uint32_t sTurn = sScale + NK * C::SCALES;                   // a part for each softmax warp
  uint8_t* const misc = gbase + C::DATA;
  const uint32_t sMisc = base + C::DATA;
  // misc: barriers, then what the roles tell one another
  uint32_t bar = sMisc;
  auto take = [&](int n) {
    const uint32_t b = bar;
    bar += 8 * n;
    return b;
  };
  const uint32_t FULL = take(NK), K_EMPTY = take(NK), V_EMPTY = take(NK);   // of K and V together
  const uint32_t S_FULL = take(4), P_FULL = take(4), P_EMPTY = take(4);   // [A, B][2]
  const uint32_t Q_FULL = take(1), Q_EMPTY = take(1), SEG_FULL = take(kSegments), SEG_EMPTY = take(kSegments);
  const uint32_t LOOK = take(2), C_FULL = take(C::NC), C_EMPTY = take(C::NC);
  constexpr int kBarBytes = 8 * (3 * NK + 12 + 2 + 2 * kSegments + 2 + 2 * C::NC);
  static_assert(kBarBytes <= 640, "");
  ChunkPlan* const plan = reinterpret_cast<ChunkPlan*>(misc + 640);
  long long* const scratch = reinterpret_cast<long long*>(misc + 768);                      // [16]
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(misc + 896);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(misc + 1408);            // what stalled() tells
  unsigned long long* const bad_keys = reinterpret_cast<unsigned long long*>(misc + 912);   // [2][3]
  Segment* const segs = reinterpret_cast<Segment*>(misc + 960);
  static_assert(sizeof(ChunkPlan) <= 128 && 960 + kSegments * sizeof(Segment) <= 1408 && 1408 + 8 + 2 * C::THREADS <= C::MISC, "");

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  reinterpret_cast<volatile uint16_t*>(abort_flag + 2)[tid] = 0;
  if (tid == 0) {
    for (int i = 0; i < NK; ++i) {
      mbar_init(FULL + 8 * i, FP8 ? 128 : 1);
      mbar_init(K_EMPTY + 8 * i, 2);   // A's and B's MMAs
      mbar_init(V_EMPTY + 8 * i, 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(S_FULL + 8 * i, 1);
      mbar_init(P_FULL + 8 * i, 128);
      mbar_init(P_EMPTY + 8 * i, 1);
    }
    mbar_init(Q_FULL, 1);
    mbar_init(Q_EMPTY, 2);
    for (int i = 0; i < kSegments; ++i) {
      mbar_init(SEG_FULL + 8 * i, 1);
      mbar_init(SEG_EMPTY + 8 * i, FP8 ? 14 : 10);   // softmax, MMA and conversion warps
    }
    mbar_init(LOOK, 4);       // A's warps alone
    mbar_init(LOOK + 8, 8);   // A's and B's
    for (int i = 0; i < C::NC; ++i) {
      mbar_init(C_FULL + 8 * i, 1);
      mbar_init(C_EMPTY + 8 * i, 128);
    }
    abort_flag[0] = abort_flag[1] = 0;
    for (int i = 0; i < 6; ++i) bad_keys[i] = 0;
    fence_barrier_init();
    prefetch_tensormap(&mQ);
    prefetch_tensormap(&mK);
    prefetch_tensormap(&mV);
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;   // S of A, S of B (two buffers each), O of A, O of B
  // Not before the allocation: a successor that got the columns which a CTA of this grid waits for
  // would hold them while it waits for this grid to end.
  pdl_trigger();
  pdl_wait();
  make_chunk_plan(a, plan, scratch);
  if (tid == 0) a.join[blockIdx.x].first = -1;

  // ------------------------------------------------------------ MMA of A (X = 0), of B
  // The whole warp runs this, with one lane elected at each instruction: control and operands
  // stay uniform, which keeps the descriptors in uniform registers (a lane by itself moves every
  // operand there first, on a scheduler that it shares with two softmax warps: 500 tokens at
  // 131072 487 us, so 402). Every wait costs the issue of MMAs, so there are two a tile.
  auto issue_mma = [&](const int X) {
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, KB);
    constexpr uint32_t idesc_o = idesc_bf16_f32(128, HD) | kIdescBMajorMN;
    constexpr int PER = RB / 32;   // 16-deep steps of a half
    const uint32_t bSF = S_FULL + 16 * X, bPF = P_FULL + 16 * X, bPE = P_EMPTY + 16 * X;
    const uint32_t tS = tmem + 2 * X * KB, tO = tmem + 4 * KB + X * HD;
    const uint64_t dQ = desc_k<RB, C::SW>(sQ + X * C::Q_TILE);
    const uint64_t dK0 = desc_k<RB, C::SW>(sK), dV0 = desc_mn<RB, C::SW>(sV, C::K_HALF);
    int s_st = 0, v_st = 0;    // stages of the next S and P V,
    uint32_t s_ph = 0;         // the phase of S's
    int cs = 0, cp = 0;        // tiles whose S, P V has been issued
    auto next_stage = [&](int& st) {
      if (++st == NK) st = 0;
    };
    // S of the next tile, once its K and V are there
    auto scores = [&](bool mine) {
      if (!wait_for(FULL + 8 * s_st, s_ph, abort_flag, a.status)) return false;
      if (mine) {
        const int b = cs & 1;
        tc_fence_after();
        const uint64_t dK = dK0 + (uint32_t)(s_st * (C::K_TILE >> 4));
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          mma_elected(tS + b * KB, dQ + (kk / PER) * (C::Q_HALF >> 4) + 2 * (kk % PER),
                      dK + (kk / PER) * (C::K_HALF >> 4) + 2 * (kk % PER), idesc_s, kk != 0);
        commit_elected(bSF + 8 * b);
        ++cs;
      }
      commit_elected(K_EMPTY + 8 * s_st);
      if (++s_st == NK) {
        s_st = 0;
        s_ph ^= 1;
      }
      return true;
    };
    for (int s = 0;; ++s) {
      const int e = s % kSegments;
      if (!wait_for(SEG_FULL + 8 * e, (s / kSegments) & 1, abort_flag, a.status)) break;
      const int first = __shfl_sync(0xffffffffu, segs[e].first, 0);
      const int count = __shfl_sync(0xffffffffu, segs[e].last, 0) - first;
      const bool mine = X == 0 || __shfl_sync(0xffffffffu, segs[e].both, 0);
      __syncwarp();
      if (lane == 0) mbar_arrive(SEG_EMPTY + 8 * e);
      if (first < 0 || !wait_for(Q_FULL, s & 1, abort_flag, a.status)) break;
      // S runs two tiles ahead of P V: its buffer held the P before, which that P V has taken (the
      // MMAs of a thread run in order). A tile without rows of this half: its stages are freed, but
      // not before they are full, for a phase has one arrival of each half.
      bool ok = scores(mine) && (count == 1 || scores(mine));
      if (count <= 2) commit_elected(Q_EMPTY);
      for (int i = 0; i < count && ok; ++i) {
        if (mine) {
          const int b = cp & 1;
          ok = wait_for(bPF + 8 * b, (uint32_t)(cp >> 1) & 1u, abort_flag, a.status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dV = dV0 + (uint32_t)(v_st * (C::K_TILE >> 4));
#pragma unroll
          for (int kk = 0; kk < KB / 16; ++kk)   // 16 keys: 8 columns of P, 2 groups of 8 rows of V
            mma_tmem_a_elected(tO, tS + b * KB + 8 * kk, dV + kk * RB, idesc_o);
          commit_elected(bPE + 8 * b);
          ++cp;
        }
        commit_elected(V_EMPTY + 8 * v_st);
        next_stage(v_st);
        if (i + 2 < count) {
          ok = scores(mine);
          if (i + 3 == count) commit_elected(Q_EMPTY);
        }
      }
      if (!ok) break;
    }
  };

  if (plan->begin >= plan->end) {
    // nothing to do
  } else if (warp == 0) {
    // ------------------------------------------------------------ TMA
    ChunkWalk w;
    w.begin(a, *plan);
    int it = 0;
    const int nbox = KB / a.box;
    int page = 0, y_prev = 0, boxes_prev = 0;
    auto page_of = [&](int tile) {   // lane b: the page of box b
      if (lane >= nbox) return 0;   // nor may the sum pass 2^31, which the last tile reaches
      const int key = tile * KB + lane * a.box;
      return key < w.limit ? chunk_page(a, w.k, key) : 0;
    };
    auto load_v = [&](int i, int y, int boxes) {   // V of the i-th tile of the range
      const int st = i % NK;
      const uint32_t full = FULL + 8 * st;
      if (i >= NK && !wait_for(V_EMPTY + 8 * st, ((i / NK) & 1) ^ 1, abort_flag, a.status)) return false;
      if (lane < boxes) {
#pragma unroll
        for (int h = 0; h < C::HALVES; ++h)
          tma_load_2d(sV + st * C::K_TILE + h * C::K_HALF + lane * a.box * RB, &mV, full, h * 64, y);
      }
      return true;
    };
    bool ok = true;
    while (ok && w.next(a)) {
      const int first = w.first, last = w.last, g = chunk_kv_head(a, w.hp);
      page = page_of(first);
      for (int tile = first; tile < last && ok; ++tile, ++it) {
        if (lane == 0 && (it & 1023) == 0) abort_flag[1] = it >> 10;
        const int next = tile + 1 < last ? page_of(tile + 1) : 0;
        // A tile without keys loads a box as well (of page 0, seen by no row): there at once, it would
        // complete FULL again before the softmax of the tile that had its stage waited for that.
        const int valid = max(1, min(KB, w.limit - tile * KB)), boxes = (valid + a.box - 1) / a.box;
        int pg = page;
        if (lane < boxes && (pg < 0 || pg >= a.n_pages)) {
          report_status(a.status, XMOD_ERR_DEVICE_CHECK);
          pg = 0;
        }
        const int key = tile * KB + (lane < nbox ? lane * a.box : 0);
        const int y = (int)(((int64_t)pg * a.hkv + g) * a.page_size + chunk_in_page(a, key));
        if constexpr (!FP8) {
          const int st = it % NK;
          const uint32_t full = FULL + 8 * st;
          ok = it < NK || wait_for(K_EMPTY + 8 * st, ((it / NK) & 1) ^ 1, abort_flag, a.status);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(full, boxes * (uint32_t)a.box * HD * 4);   // V's too
          __syncwarp();
          if (lane < boxes) {
#pragma unroll
            for (int h = 0; h < C::HALVES; ++h)
              tma_load_2d(sK + st * C::K_TILE + h * C::K_HALF + lane * a.box * RB, &mK, full, h * 64, y);
          }
          if (it > 0) ok = load_v(it - 1, y_prev, boxes_prev);
        } else {
          const int st = it % C::NC;
          const uint32_t full = C_FULL + 8 * st;
          ok = it < C::NC || wait_for(C_EMPTY + 8 * st, ((it / C::NC) & 1) ^ 1, abort_flag, a.status);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(full, boxes * (uint32_t)a.box * (2 * HD + 8));
          __syncwarp();
          if (lane < boxes) {
            const uint32_t k = sCode + st * 2 * C::CODES + lane * a.box * C::CRB;
            tma_load_2d(k, &mK, full, 0, y);
            tma_load_2d(k + C::CODES, &mV, full, 0, y);
            const uint32_t s = sCodeScale + st * C::SCALES + lane * a.box * 4;
            bulk_load(s, a.k_scale + y, a.box * 4, full);
            bulk_load(s + KB * 4, a.v_scale + y, a.box * 4, full);
          }
        }
        y_prev = y;
        boxes_prev = boxes;
        page = next;
      }
    }
    if (!FP8 && ok && it > 0) load_v(it - 1, y_prev, boxes_prev);
  } else if (warp == 1 || warp == 3) {
    issue_mma(warp == 3 ? 1 : 0);
  } else if (warp == 2) {
    // ------------------------------------------------------------ segments and their queries
    ChunkWalk w;
    w.begin(a, *plan);
    int s = 0;
    bool ok = true;
    for (;; ++s) {
      const int e = s % kSegments;
      ok = s < kSegments || wait_for(SEG_EMPTY + 8 * e, ((s / kSegments) & 1) ^ 1, abort_flag, a.status);
      if (!ok) break;
      const bool more = w.next(a), both = more && segment_both(a, w.k, w.t);
      if (lane == 0) {
        Segment& g = segs[e];
        g.k = w.k;
        g.hp = w.hp;
        g.t = w.t;
        g.tiles = w.tiles;
        g.limit = w.limit;
        g.first = more ? w.first : -1;
        g.last = w.last;
        g.both = both;
        mbar_arrive(SEG_FULL + 8 * e);
      }
      __syncwarp();
      if (!more) break;
      ok = s == 0 || wait_for(Q_EMPTY, (s - 1) & 1, abort_flag, a.status);
      if (!ok) break;
      if (lane == 0) {
        // rows past the chunk's end come too (zeros past q's); they are worked on but not stored
        const int blocks = both ? 2 : 1, head = chunk_first_head(a, w.hp);
        mbar_arrive_expect_tx(Q_FULL, (uint32_t)(blocks * C::HALVES * RB * a.hpt * a.block_tokens));
        for (int x = 0; x < blocks; ++x)
#pragma unroll
          for (int h = 0; h < C::HALVES; ++h)
            tma_load_3d(sQ + x * C::Q_TILE + h * C::Q_HALF, &mQ, Q_FULL, h * 64, head,
                        w.k.first + w.t * a.tpt + x * a.block_tokens);
      }
      __syncwarp();
    }
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------ softmax
    const int x = (warp - 4) >> 2, quad = warp & 3, row128 = quad * 32 + lane, R = x * 128 + row128;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + lane_off + 2 * x * KB, tO = tmem + lane_off + 4 * KB + x * HD;
    const uint32_t bSF = S_FULL + 16 * x, bPF = P_FULL + 16 * x, bPE = P_EMPTY + 16 * x;
    const float scale_log2 = 1.4426950408889634f * rsqrtf((float)HD);
    int n = 0, i0 = 0;            // tiles this group has worked on; tiles before the segment
    int looks[2] = {0, 0};        // looks at V, by A's warps alone and by all
    uint32_t look_phase = 0;      // of the two barriers
    bool ok = true;
    // all softmax warps that work on the segment
    auto meet = [&](int both) {
      __syncwarp();
      if (lane == 0) mbar_arrive(LOOK + 8 * both);
      const bool r = wait_for(LOOK + 8 * both, (look_phase >> both) & 1u, abort_flag, a.status);
      look_phase ^= 1u << both;
      return r;
    };
    for (int s = 0; ok; ++s) {
      const int e = s % kSegments;
      if (!wait_for(SEG_FULL + 8 * e, (s / kSegments) & 1, abort_flag, a.status)) break;
      const Segment g = segs[e];
      __syncwarp();
      if (lane == 0) mbar_arrive(SEG_EMPTY + 8 * e);
      if (g.first < 0) break;
      const int count = g.last - g.first;
      const int least = (int)max((int64_t)0, g.k.len - g.k.n + 1 + (int64_t)g.t * a.tpt);   // the first row's limit
      if (x == 1 && !g.both) {
        i0 += count;
        continue;
      }
      const ChunkRow row = chunk_row(a, g.k, g.hp, g.t, x, row128);
      const int limit = row.m < 0 ? g.limit : row.limit;
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        float zero[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) zero[i] = 0.f;
        tmem_st32(tO + c * 32, zero);
      }
      tmem_st_wait();
      for (int tile = g.first; tile < g.last; ++tile, ++n) {
        const int b = n & 1, it = i0 + tile - g.first, vs = it % NK, key0 = tile * KB;
        if (!wait_for(bSF + 8 * b, (uint32_t)(n >> 1) & 1u, abort_flag, a.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float v[KB];
        tmem_ld64(tS + b * KB, v);
        tmem_ld_wait();
        const float* sc = reinterpret_cast<const float*>(gbase + (sScale - base) + vs * C::SCALES);
        if constexpr (FP8) {
          // the scales lie there since the codes were converted
          if (!wait_for(FULL + 8 * vs, (uint32_t)(it / NK) & 1u, abort_flag, a.status)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int i = 0; i < KB; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(sc + i);
            const float2 s0 = mul2(make_float2(v[i], v[i + 1]), make_float2(f.x, f.y));
            const float2 s1 = mul2(make_float2(v[i + 2], v[i + 3]), make_float2(f.z, f.w));
            v[i] = s0.x;
            v[i + 1] = s0.y;
            v[i + 2] = s1.x;
            v[i + 3] = s1.y;
          }
        }
        const bool masked = least - key0 < KB;   // some row of the segment does not see all of it
        const int seen = limit - key0;   // of this row
        if (masked) {
#pragma unroll
          for (int c = 0; c < KB; c += 16)
            if (__any_sync(0xffffffffu, seen < c + 16)) {
#pragma unroll
              for (int i = c; i < c + 16; ++i)
                if (i >= seen) v[i] = -INFINITY;
            }
        }
        float mc[KB / 16];
#pragma unroll
        for (int r = 0; r < KB / 16; ++r) {
          const float* u = v + 16 * r;
          float t = max3(u[0], u[1], u[2]);
#pragma unroll
          for (int i = 3; i < 15; i += 2) t = max3(t, u[i], u[i + 1]);
          mc[r] = fmaxf(t, u[15]);
        }
        const float m_cand = fmaxf(max3(mc[0], mc[1], mc[2]), mc[3]) * scale_log2;
        const bool grow = m_cand > m + kRescale;
        float m_new = grow ? m_cand : m;
        if constexpr (FP8) {
          // the largest weight, times its value's scale, becomes a power of two, which bf16 holds (without
          // this a row of one or two keys is off by two roundings that every dimension shares: 1.9
          // times the error of exact weights)
          if (__any_sync(0xffffffffu, grow)) {
            const float shift = scale_shift(tS + b * KB, sc, seen);
            if (grow) m_new += shift;   // any would do: it cancels from the sums
          }
        }
        const float alpha = grow ? exp2f(m - m_new) : 1.0f;
        if (__any_sync(0xffffffffu, grow && m != -INFINITY)) {
          // O holds the tiles before: the last of their products has to have landed
          const int q = n - 1;
          if (!wait_for(bPE + 8 * (q & 1), (uint32_t)(q >> 1) & 1u, abort_flag, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float f = m == -INFINITY ? 1.0f : alpha;
#pragma unroll 1
          for (int c = 0; c < HD / 32; ++c) {
            float ov[32];
            tmem_ld32(tO + c * 32, ov);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] *= f;
            tmem_st32(tO + c * 32, ov);
          }
          tmem_st_wait();
        }
        m = m_new;
        const float negm = m == -INFINITY ? 0.f : -m;
        const float2 scale2 = make_float2(scale_log2, scale_log2), negm2 = make_float2(negm, negm);
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < KB; i += 2) {
          const float2 y = fma2(make_float2(v[i], v[i + 1]), scale2, negm2);
          const float2 p = make_float2(ex2(y.x), ex2(y.y));
          acc[(i >> 1) & 1] = add2(acc[(i >> 1) & 1], p);
          v[i] = p.x;
          v[i + 1] = p.y;
        }
        const float2 both_acc = add2(acc[0], acc[1]);
        l = l * alpha + (both_acc.x + both_acc.y);
        if constexpr (FP8) {
#pragma unroll
          for (int i = 0; i < KB; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(sc + KB + i);
            const float2 s0 = mul2(make_float2(v[i], v[i + 1]), make_float2(f.x, f.y));
            const float2 s1 = mul2(make_float2(v[i + 2], v[i + 3]), make_float2(f.z, f.w));
            v[i] = s0.x;
            v[i + 1] = s0.y;
            v[i + 2] = s1.x;
            v[i + 3] = s1.y;
          }
          if (masked) {   // a scale that is not seen may be anything
#pragma unroll
            for (int i = 0; i < KB; ++i)
              if (i >= seen) v[i] = 0.f;
          }
        }
        if (masked) {
          // ---- V's slots that some row does not see
          if (!wait_for(FULL + 8 * vs, (uint32_t)(it / NK) & 1u, abort_flag, a.status)) {
            ok = false;
            break;
          }
          constexpr int CH = HD / 8;
          const uint32_t vt = sV + vs * C::K_TILE;
          const int from = max(0, least - key0), valid = max(0, min(KB, g.limit - key0));
          const int width = g.both ? 256 : 128;
          unsigned long long bad = 0;
          bool wrote = false;
          // four vectors at a time
#pragma unroll 1
          for (int i0 = from * CH + R; i0 < KB * CH; i0 += 4 * width) {
            uint4 u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int i = min(i0 + j * width, KB * CH - 1);
              u[j] = lds128(vt + swizzled<RB>(i / CH, i % CH, KB));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int i = i0 + j * width, key = i / CH;
              if (i >= KB * CH) break;
              if (key >= valid) {
                sts128(vt + swizzled<RB>(key, i % CH, KB), make_uint4(0u, 0u, 0u, 0u));
                wrote = true;
              } else if (nonfinite2(u[j].x) | nonfinite2(u[j].y) | nonfinite2(u[j].z) | nonfinite2(u[j].w)) {
                bad |= 1ull << key;
              }
            }
          }
          // three slots in turn: the one of the look before last, which all have read before they
          // came to this one, is cleared for the look after next
          const int look = g.both ? looks[1]++ : looks[0]++;
          unsigned long long* const slots = bad_keys + 3 * g.both;
          const int slot = look % 3;
          if (bad) atomicOr(&slots[slot], bad);
          if (wrote) fence_proxy_async_smem();
          if (!meet(g.both)) {
            ok = false;
            break;
          }
          bad = *reinterpret_cast<volatile unsigned long long*>(&slots[slot]);
          if (R == 0) slots[(look + 2) % 3] = 0;
          if (bad) {
            // rare: infinities and NaN of V to the rows that see them, then zeros in their place
            if (n > 0) {
              const int q = n - 1;
              if (!wait_for(bPE + 8 * (q & 1), (uint32_t)(q >> 1) & 1u, abort_flag, a.status)) {
                ok = false;
                break;
              }
            }
            tc_fence_after();
            float weight[KB];   // by key: local memory
#pragma unroll
            for (int i = 0; i < KB; ++i) weight[i] = v[i];
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
              float ov[32];
              tmem_ld32(tO + c * 32, ov);
              tmem_ld_wait();
              for (unsigned long long rest = bad; rest; rest &= rest - 1) {
                const int key = __ffsll((long long)rest) - 1;
                if (key0 + key >= limit) continue;
                const float p = weight[key];
#pragma unroll
                for (int d = 0; d < 32; d += 8) {
                  const uint4 u = lds128(vt + swizzled<RB>(key, c * 4 + d / 8, KB));
#pragma unroll
                  for (int h = 0; h < 4; ++h) {
                    const float2 f = vec_pair<__nv_bfloat16>(u, h);
                    if (!isfinite(f.x)) ov[d + 2 * h] += p * f.x;
                    if (!isfinite(f.y)) ov[d + 2 * h + 1] += p * f.y;
                  }
                }
              }
              __syncwarp();
              tmem_st32(tO + c * 32, ov);
            }
            tmem_st_wait();
            if (!meet(g.both)) {
              ok = false;
              break;
            }
            for (int i = from * CH + R; i < valid * CH; i += width) {
              const uint32_t at = vt + swizzled<RB>(i / CH, i % CH, KB);
              uint4 u = lds128(at);
              uint32_t* h = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t f = nonfinite2(h[k]);
                h[k] &= ~((f & 0x8000u ? 0xffffu : 0u) | (f & 0x80000000u ? 0xffff0000u : 0u));
              }
              sts128(at, u);
            }
            fence_proxy_async_smem();
            if (!meet(g.both)) {
              ok = false;
              break;
            }
          }
        }
        float pk[32];
#pragma unroll
        for (int i = 0; i < KB; i += 2) pk[i / 2] = __uint_as_float(pack_bf16x2(v[i], v[i + 1]));
        tmem_st32(tS + b * KB, pk);   // over the scores
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bPF + 8 * b);
      }
      if (!ok) break;
      i0 += count;
      // ---- the segment's result in this CTA's range
      const int q = n - 1;
      if (!wait_for(bPE + 8 * (q & 1), (uint32_t)(q >> 1) & 1u, abort_flag, a.status)) break;
      tc_fence_after();
      const bool whole = g.first == 0 && g.last == g.tiles;
      const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
      const int64_t head = row.m < 0 ? -1 : row.m * a.hq + row.head;
      float* part = chunk_part<QR, HD>(a, blockIdx.x, g.first > 0);
      if (whole) {
        // through shared memory, so that lanes side by side write one row's columns: PER lanes a row
        constexpr int PER = C::OUT / 8, STEPS = PER;   // 16 bytes a lane, 32 / PER rows a step
        const uint32_t turn_base = sTurn + (warp - 4) * 32 * C::OUT_LD;
        int64_t to[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; ++i) to[i] = __shfl_sync(0xffffffffu, head, i * (32 / PER) + lane / PER);
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
          float ov[32];
          tmem_ld32(tO + c * 32, ov);
          tmem_ld_wait();
#pragma unroll
          for (int part32 = 0; part32 < 32 / C::OUT; ++part32) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < C::OUT; i += 8) {
              const float* f = ov + part32 * C::OUT + i;
              sts128(turn_base + lane * C::OUT_LD + i * 2,
                     make_uint4(pack_bf16x2(f[0] * inv, f[1] * inv), pack_bf16x2(f[2] * inv, f[3] * inv),
                                pack_bf16x2(f[4] * inv, f[5] * inv), pack_bf16x2(f[6] * inv, f[7] * inv)));
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
              const uint4 u = lds128(turn_base + (i * (32 / PER) + lane / PER) * C::OUT_LD + lane % PER * 16);
              if (to[i] >= 0)
                *reinterpret_cast<uint4*>((__nv_bfloat16*)a.o + to[i] * HD + c * 32 + part32 * C::OUT +
                                          lane % PER * 8) = u;
            }
          }
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
          float ov[32];
          tmem_ld32(tO + c * 32, ov);
          tmem_ld_wait();
          if (row.m >= 0) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(part + 2 * QR + ((c * 8 + i / 4) * QR + R) * 4) =
                  make_float4(ov[i], ov[i + 1], ov[i + 2], ov[i + 3]);
          }
        }
      }
      if (row.m >= 0) {
        if (whole) {
          if (a.lse) a.lse[head] = (m + log2f(l)) * 0.6931471805599453f;
        } else {
          part[R] = m;
          part[QR + R] = l;
        }
      }
      if (R == 0 && g.first == 0 && !whole) {
        a.join[blockIdx.x] = chunk_join(*plan, g.k, g.hp, g.t, g.tiles - g.last);
      }
    }
  } else if (FP8 && warp >= 12) {
    // ------------------------------------------------------------ codes to bf16
    // Thread t takes chunk (t / 8) % CH of rows t % 8 + 8 * (t / (8 CH)), and STEP rows on: eight
    // lanes have the same chunk of eight rows, whose swizzled places differ.
    constexpr int CH = HD / 16, N = KB * CH / 128, STEP = 128 / CH;   // 16-byte chunks of a row of codes
    const int t = tid - 384, r0 = (t & 7) + 8 * (t / (8 * CH)), c0 = (t >> 3) % CH;
    const uint32_t from_at = swizzled<C::CRB>(r0, c0, KB), lo_at = swizzled<RB>(r0, 2 * c0, KB),
                   hi_at = swizzled<RB>(r0, 2 * c0 + 1, KB);
    bool ok = true;
    int it = 0;
    for (int s = 0, left = 0; ok; ++it, --left) {
      while (left == 0 && ok) {   // the next segment's tiles
        const int e = s % kSegments;
        ok = wait_for(SEG_FULL + 8 * e, (s / kSegments) & 1, abort_flag, a.status);
        if (!ok) break;
        const int first = segs[e].first;
        left = first < 0 ? -1 : segs[e].last - first;
        __syncwarp();
        if (lane == 0) mbar_arrive(SEG_EMPTY + 8 * e);
        ++s;
      }
      if (!ok || left < 0) break;
      const int cs = it % (C::NC ? C::NC : 1), st = it % NK;
      ok = wait_for(C_FULL + 8 * cs, (it / (C::NC ? C::NC : 1)) & 1, abort_flag, a.status);
      // K's and V's stages are those of the tile NK before: with V's the softmax is done with its scales
      if (ok && it >= NK)
        ok = wait_for(K_EMPTY + 8 * st, ((it / NK) & 1) ^ 1, abort_flag, a.status) &&
             wait_for(V_EMPTY + 8 * st, ((it / NK) & 1) ^ 1, abort_flag, a.status);
      if (!ok) break;
      {
        const float* from = reinterpret_cast<const float*>(gbase + (sCodeScale - base) + cs * C::SCALES);
        float* to = reinterpret_cast<float*>(gbase + (sScale - base) + st * C::SCALES);
        to[t] = from[t];   // 128: K's and V's
      }
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t src = sCode + cs * 2 * C::CODES + kv * C::CODES + from_at;
        const uint32_t dst = (kv ? sV : sK) + st * C::K_TILE;
        // Loops are kept small: unrolled, the roles' code together no longer fits the instruction
        // cache (16 ragged chunks at 16384: 668 us instead of 357).
        uint4 u = lds128(src);
#pragma unroll 1
        for (int j = 0; j < N; ++j) {
          uint4 lo, hi;
          codes_bf16(u, lo, hi);
          if (j + 1 < N) u = lds128(src + (j + 1) * STEP * C::CRB);
          sts128(dst + lo_at + j * STEP * RB, lo);
          sts128(dst + hi_at + j * STEP * RB, hi);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(FULL + 8 * st);
      mbar_arrive(C_EMPTY + 8 * cs);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {   // copies in flight land before the CTA ends
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 20000000ull) {
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int HD, bool FP8> int launch_tc(const Ctx& c, const ChunkArgs& a, int ctas) {
  using C = Tc<HD, FP8>;
  CUtensorMap mq, mk, mv;
  const int64_t rows = (int64_t)a.n_pages * a.hkv * a.page_size;
  const int cols = FP8 ? C::CRB : C::RB / 2;
  if (!tma_map_heads(&mq, a.q, a.M, a.ldq, a.hq, HD, C::RB / 2, a.hpt, a.block_tokens) ||
      !tma_map_rows(&mk, a.k, FP8 ? 1 : 2, rows, HD, cols, a.box) ||
      !tma_map_rows(&mv, a.v, FP8 ? 1 : 2, rows, HD, cols, a.box))
    return XMOD_ERR_CUDA;
  static std::atomic<uint64_t> done{0};
  auto k = cache_chunk_tc_kernel<HD, FP8>;
  if (allow_smem(k, C::SMEM, done) != cudaSuccess) return XMOD_ERR_CUDA;
  XMOD_LAUNCH(c, "cache_chunk", launch_pdl(k, dim3(ctas), dim3(C::THREADS), C::SMEM, c.stream, mq, mk, mv, a));
  return XMOD_OK;
}

template <bool FP8> int launch_tc_hd(const Ctx& c, const ChunkArgs& a, int hd, int ctas) {
  if (hd == 128) return launch_tc<128, FP8>(c, a, ctas);
  if (hd == 64) return launch_tc<64, FP8>(c, a, ctas);
  return launch_tc<32, FP8>(c, a, ctas);
}

}  // namespace

int launch_chunk_tc(const Ctx& c, const ChunkArgs& a, int hd, bool fp8, int ctas) {
  return fp8 ? launch_tc_hd<true>(c, a, hd, ctas) : launch_tc_hd<false>(c, a, hd, ctas);
}

}  // namespace xmod
