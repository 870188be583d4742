// Attention of one query token per row over a paged key/value cache:
//   o = sum_i p_i V_i,  p = softmax_i(q . K_i / sqrt(hd)),  i < len
// in one pass over the cache with the softmax's running maximum and sum.
//
// Bound. Every key costs 2 hd elements of memory traffic per KV head and 4 hd operations
// per query head: at 4 query heads per KV head and bf16 that is 4 operations a byte, far
// below what the tensor cores do in the time the bytes take. So the kernel is built around
// keeping copies in flight: TMA tiles into a ring of shared-memory stages (two CTAs per SM,
// about 190 KB in flight), and the arithmetic, on the warp-level MMA (its rows padded from
// the query heads of one KV head to 16), hides behind them. tcgen05 would not help: its 128
// rows would be 4 to 16 query heads, and the scores would travel through tensor memory.
//
// Measured: 64 rows of up to 8192 slots (32 query and 8 KV heads of 128, bf16, 1.10 GB)
// 171 us, 6.4 TB/s, 0.95 of what a copy reaches; one row of 131079 (16 and 4 heads, 268 MB)
// 49 us, of which 10 are the launch, the plan, the first tile and the join; 32 rows of up to
// 16384 in e4m3 (285 MB) 55 us: the codes stream at 6.3 TB/s (their conversions to f16 double
// the instructions a byte) after 9.5 us of the same latency; 8 rows of up to 512 8.3 us.
//
// Split. The tiles of all rows and KV heads form one list, cut into equal ranges, one per
// CTA, so a single long sequence fills the GPU as well as a batch of ragged ones. A CTA
// walks its range; where a (row, KV head) lies in several CTAs' ranges each leaves its
// maximum, sum and unnormalised output in the workspace and a second small kernel joins
// them, in CTA order: the result is the same bits at every call.

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <float.h>
#include <math.h>

#include <atomic>

#include "cache.h"
#include "common.cuh"
#include "tc_common.cuh"

namespace xmod {

using namespace tc;

namespace {

constexpr int kMaxCtas = 512;        // CTAs the workspace has room for
constexpr int kThreads = 160;        // 4 consumer warps, 1 producer warp
constexpr int kConsumers = 4;

struct DecodeArgs {
  int M, hq, hkv, ldq;
  const void* q;
  const int32_t *seq, *len;
  void* o;
  float* lse;
  const int32_t* table;
  const void *k, *v;
  const float *k_scale, *v_scale;
  int n_pages, page_size, n_seqs, max_pages;
  int passes;      // passes of at most ROWS query heads per KV head
  int box;         // rows of a TMA box: divides the page size and a tile
  float* part;     // partial results, two per CTA
  struct Join* join;   // what each CTA leaves to be joined
  int* status;
};

// A segment (row, KV head, pass) that starts in a CTA's range and ends in a later one's.
struct Join {
  int row, pass, first, last;   // CTAs first .. last hold it; row < 0: none
};

// Keys per tile: 128 bytes of each dimension.
template <bool FP8> constexpr int tile_keys() { return FP8 ? 128 : 64; }

// Length of row m, clamped into its range; -1 for a row to skip.
__device__ __forceinline__ int row_length(const DecodeArgs& a, int m, int* seq_out) {
  const int seq = a.seq ? a.seq[m] : m;
  *seq_out = seq;
  if (seq < 0) return -1;
  if (seq >= a.n_seqs) {
    report_status(a.status, XMOD_ERR_DEVICE_CHECK);
    return -1;
  }
  const int n = a.len[m], most = a.max_pages * a.page_size;
  if (n < 0 || n > most) {
    report_status(a.status, XMOD_ERR_DEVICE_CHECK);
    return n < 0 ? 0 : most;
  }
  return n;
}
// An empty row counts as one tile: its zeros have to be written.
template <int KT> __device__ __forceinline__ int row_tiles(int n) {
  return n < 0 ? 0 : n == 0 ? 1 : (n - 1) / KT + 1;
}

// This CTA's range [begin, end) of the tile list (order: row, KV head and pass, tile) and
// the row it starts in, `off` tiles into that row's.
struct Plan {
  long long begin, end, total, off;
  int row, ctas;
};

// All threads of the CTA; scratch: one int64 per warp.
template <int KT>
__device__ void make_plan(const DecodeArgs& a, Plan* plan, long long* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthreads = blockDim.x;
  const int per = (a.M + nthreads - 1) / nthreads;
  const int m0 = min(a.M, tid * per), m1 = min(a.M, m0 + per);
  const long long P = (long long)a.hkv * a.passes;
  long long mine = 0;
  int seq;
  for (int m = m0; m < m1; ++m) mine += P * row_tiles<KT>(row_length(a, m, &seq));
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
  for (int w = 0; w < nthreads / 32; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  const int ctas = (int)min((long long)gridDim.x, total);
  const int g = blockIdx.x;
  const long long begin = g < ctas ? total * g / ctas : total;
  const long long end = g < ctas ? total * (g + 1) / ctas : total;
  if (tid == 0) {
    plan->begin = begin;
    plan->end = end;
    plan->total = total;
    plan->ctas = ctas;
  }
  if (begin < end && begin >= before && begin < before + mine) {
    long long at = before;
    for (int m = m0; m < m1; ++m) {
      const long long t = P * row_tiles<KT>(row_length(a, m, &seq));
      if (begin < at + t) {
        plan->row = m;
        plan->off = begin - at;
        break;
      }
      at += t;
    }
  }
  __syncthreads();
}

// What the producer tells the consumers about a tile.
struct Tile {
  int row, pass, valid, flags;   // valid: keys of the tile below the row's length
  int left;                      // tiles of the segment after this one
};
enum { kFirst = 1, kLast = 2, kBefore = 4, kAfter = 8 };   // of the segment in this CTA;
                                                           // segment goes on before / after

// The join of a segment whose last tile in this CTA's range is `info`, the range's last: the
// segment ends `left` tiles on, in the last CTA whose range begins at or before that tile.
__device__ __forceinline__ Join make_join(const Plan& plan, const Tile& info) {
  Join j;
  j.row = info.row;
  j.pass = info.pass;
  j.first = blockIdx.x;
  j.last = (int)min((long long)plan.ctas - 1,
                    ((plan.end + info.left) * plan.ctas - 1) / plan.total);
  return j;
}

// Partial result `slot`: per query head maximum and sum (log2 units), then outputs.
template <int HD, int ROWS>
__device__ __forceinline__ float* part_at(const DecodeArgs& a, int slot) {
  return a.part + (int64_t)slot * ROWS * (HD + 2);
}

// ---------------------------------------------------------------- warp MMA

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c[16 x 8] += a[16 x 16] b[16 x 8], fp32 accumulation.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four e4m3 codes to two pairs of f16, exactly.
__device__ __forceinline__ void e4m3x4_f16x2(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// (a, b) rounded to the MMA's 16-bit type, and what the rounding left, rounded again.
template <bool F16>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t& hi, uint32_t& lo) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = pack_f16x2(a - f.x, b - f.y);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    const float2 f = __bfloat1622float2(h);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = pack_bf16x2(a - f.x, b - f.y);
  }
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// f16 weights of e4m3 values (probability times the value's scale) are scaled up to 2^14 (f16
// ends at 65504, its last step is 2^-24): one part keeps 11 bits, two keep 22, and either is off
// by 2^-39 of the reference where that is more, a power of two at or above the largest weight so
// far. The largest weight, not
// the largest scale: a key of little probability with a large scale costs the others nothing.
// (32 rows of up to 16384, 16 and 4 heads: 54.7 us, by the largest scale 54.4; 64 rows of up to
// 8192 with 16 query heads a KV head 42.5 and 41.7.)
constexpr float kWeightScale = 16384.f, kLeastRef = 0x1p-112f;   // 2^14 / 2^-112 is finite
// The power of two at or above x >= 0, within [2^-112, 2^127].
__device__ __forceinline__ float pow2_at_least(float x) {
  const uint32_t b = (__float_as_uint(x) + 0x007fffffu) & 0x7f800000u;
  return fminf(fmaxf(__uint_as_float(b), kLeastRef), 0x1p127f);
}
// kWeightScale / ref of such a power of two.
__device__ __forceinline__ float weight_factor(float ref) {
  return __uint_as_float(((127u + 127u + 14u) << 23) - __float_as_uint(ref));
}

// ---------------------------------------------------------------- tensor-core kernel

template <int HD, bool FP8, int ROWS> struct Cf {
  static constexpr int ES = FP8 ? 1 : 2;
  static constexpr int KT = tile_keys<FP8>();
  static constexpr int RB = HD * ES < 128 ? HD * ES : 128;   // bytes of a box row
  static constexpr int HALVES = HD * ES / RB;                // boxes across the dimensions
  static constexpr int KV = KT * HD * ES;                    // bytes of a K or V tile
  static constexpr int QROW = HD * 2 + 16;                   // padded: rows on distinct banks
  static constexpr int QB = ROWS * QROW;
  static constexpr int SC = FP8 ? 2 * KT * 4 : 0;
  static constexpr int MISC = 2048;   // barriers, plan, tile infos, the warps' maxima and sums
  static constexpr int SM2 = 228 * 1024 / 2 - 1024;          // per CTA at two CTAs an SM
  static constexpr int FIT = (SM2 - MISC - 1024) / (2 * KV + QB + SC);
  static constexpr int NST = FIT < 8 ? FIT : 8;
  static constexpr int SMEM = NST * (2 * KV + QB + SC) + MISC + 1024;
  static constexpr int KSTEPS = HD / 16;
  static constexpr int SUB = KT / 64;   // 16-key groups of a tile per consumer warp
  static constexpr int NT = HD / 8;     // 8-wide output column groups
  static_assert(NST >= 2 && NST * (int)sizeof(Tile) + 16 * NST + 8 + 256 + 1024 <= MISC, "");
  // the consumers' outputs are exchanged through the stage of the segment's last tile
  static_assert(kConsumers * ROWS * HD * 4 <= 2 * KV, "");
};

// Byte offset of 16-byte chunk c (of a whole row) of tile row r, under the TMA's swizzle:
// the chunk index within the 128-, 64- or 32-byte row is XORed with the address bits above
// the 128-byte line's row index.
template <class C>
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
  constexpr int CH = C::RB / 16;
  const int half = c / CH, cc = c % CH;
  const int x = C::RB == 128 ? (r & 7) : C::RB == 64 ? ((r >> 1) & 3) : ((r >> 2) & 1);
  return (uint32_t)(half * C::KT * C::RB + r * C::RB + ((cc ^ x) << 4));
}

template <int HD, bool FP8, int ROWS>
__global__ void __launch_bounds__(kThreads, 2)
cache_attention_kernel(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV,
                       const DecodeArgs a) {
  using C = Cf<HD, FP8, ROWS>;
  constexpr int KT = C::KT, NST = C::NST;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  // stages of K and V, then the stages' q rows and scales, then the small things
  const uint32_t sQ = base + NST * 2 * C::KV, sScale = sQ + NST * C::QB,
                 sMisc = sScale + NST * C::SC;
  uint8_t* misc = gbase + (sMisc - base);
  Plan* plan = reinterpret_cast<Plan*>(misc);
  long long* scratch = reinterpret_cast<long long*>(misc + 64);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 64 + 64);
  const uint32_t bFull = sMisc + 256, bEmpty = bFull + 8 * NST, bSync = bEmpty + 8 * NST;
  float* warp_ml = reinterpret_cast<float*>(misc + 512);   // [2][m, l][4][16]
  Tile* tiles = reinterpret_cast<Tile*>(misc + 512 + 1024);
  static_assert(64 + 64 + 8 <= 256 && 256 + 16 * NST + 8 <= 512 &&
                    512 + 1024 + NST * (int)sizeof(Tile) <= C::MISC, "");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(bFull + 8 * i, 1);
      mbar_init(bEmpty + 8 * i, kConsumers);
    }
    mbar_init(bSync, kConsumers);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&mK);
    prefetch_tensormap(&mV);
  }
  pdl_wait();
  make_plan<KT>(a, plan, scratch);   // its barriers also publish the mbarriers
  const int ntiles = (int)(plan->end - plan->begin);
  if (tid == 0) a.join[blockIdx.x].row = -1;   // the consumers set it where there is one
  if (ntiles <= 0) return;
  const int P = a.hkv * a.passes, group = a.hq / a.hkv;

  if (warp == kConsumers) {
    // ------------------------------------------------------------ producer
    int m = plan->row, batch = m & ~31, seq_l = -1, n_l = -1;
    auto load_batch = [&]() {
      n_l = -1;
      if (batch + lane < a.M) n_l = row_length(a, batch + lane, &seq_l);
    };
    load_batch();
    int n = __shfl_sync(0xffffffffu, n_l, m - batch), seq = __shfl_sync(0xffffffffu, seq_l, m - batch);
    int nt = row_tiles<KT>(n);
    int pass = (int)(plan->off / nt), tile = (int)(plan->off % nt);
    const int nbox = KT / a.box;
    auto page_of = [&](int n_, int seq_, int tile_) {   // lane b: the page of box b
      const int key = tile_ * KT + lane * a.box;
      return lane < nbox && key < n_ ? a.table[(int64_t)seq_ * a.max_pages + key / a.page_size] : 0;
    };
    int page = page_of(n, seq, tile);
    bool first_tile = true;
    int issued = 0;
    for (int it = 0; it < ntiles; ++it) {
      // the next tile, and its pages on their way while this one waits for its stage
      int m2 = m, n2 = n, seq2 = seq, nt2 = nt, pass2 = pass, tile2 = tile + 1;
      if (tile2 == nt) {
        tile2 = 0;
        if (++pass2 == P) {
          pass2 = 0;
          if (it + 1 < ntiles) do {
            if (++m2 >= batch + 32) {
              batch += 32;
              load_batch();
            }
            n2 = __shfl_sync(0xffffffffu, n_l, m2 - batch);
          } while (n2 < 0 && m2 + 1 < a.M);
          seq2 = __shfl_sync(0xffffffffu, seq_l, m2 - batch);
          n2 = max(n2, 0);   // the plan ends with the last row that is not skipped
          nt2 = row_tiles<KT>(n2);
        }
      }
      const int page2 = it + 1 < ntiles ? page_of(n2, seq2, tile2) : 0;

      const int st = it % NST;
      if (it >= NST && !mbar_wait(bEmpty + 8 * st, ((it / NST) & 1) ^ 1, abort_flag, a.status))
        break;
      issued = it + 1;
      const int valid = min(KT, n - tile * KT);
      const int boxes = (valid + a.box - 1) / a.box;
      const bool first = first_tile || tile == 0;
      const int g = pass / a.passes, h0 = (pass % a.passes) * ROWS;
      const int rows = min(ROWS, group - h0);
      const uint32_t full = bFull + 8 * st;
      if (lane == 0) {
        Tile t;
        t.row = m;
        t.pass = pass;
        t.valid = valid;
        // in the range's first segment it - tile is minus the tiles before the range
        t.flags = (first ? kFirst : 0) | (tile == nt - 1 || it == ntiles - 1 ? kLast : 0) |
                  (it < tile ? kBefore : 0) | (tile < nt - 1 ? kAfter : 0);
        t.left = nt - 1 - tile;
        tiles[st] = t;
        uint32_t bytes = boxes * (uint32_t)a.box * (2 * HD * C::ES + (FP8 ? 8 : 0));
        if (first && valid > 0) bytes += rows * HD * 2;
        mbar_arrive_expect_tx(full, bytes);
      }
      __syncwarp();
      if (valid > 0) {
        const uint32_t kS = base + st * 2 * C::KV, vS = kS + C::KV;
        if (lane < boxes) {
          int pg = page;
          if (pg < 0 || pg >= a.n_pages) {
            report_status(a.status, XMOD_ERR_DEVICE_CHECK);
            pg = 0;
          }
          const int key = tile * KT + lane * a.box;
          const int y = (int)(((int64_t)pg * a.hkv + g) * a.page_size + key % a.page_size);
          const uint32_t at = lane * a.box * C::RB;
#pragma unroll
          for (int h = 0; h < C::HALVES; ++h) {
            tma_load_2d(kS + h * KT * C::RB + at, &mK, full, h * 64, y);
            tma_load_2d(vS + h * KT * C::RB + at, &mV, full, h * 64, y);
          }
          if constexpr (FP8) {
            const uint32_t sc = sScale + st * C::SC + lane * a.box * 4;
            bulk_load(sc, a.k_scale + y, a.box * 4, full);
            bulk_load(sc + KT * 4, a.v_scale + y, a.box * 4, full);
          }
        }
        if (first && lane >= 16 && lane - 16 < rows)
          bulk_load(sQ + st * C::QB + (lane - 16) * C::QROW,
                    (const __nv_bfloat16*)a.q + (int64_t)m * a.ldq +
                        (int64_t)(g * group + h0 + lane - 16) * HD,
                    HD * 2, full);
      }
      m = m2; n = n2; seq = seq2; nt = nt2; pass = pass2; tile = tile2; page = page2;
      first_tile = false;
    }
    // the copies still in flight land before the CTA can end, whatever became of the consumers
    for (int j = max(0, issued - NST); j < issued; ++j)
      mbar_wait(bFull + 8 * (j % NST), (j / NST) & 1, nullptr, a.status);
    return;
  }

  // -------------------------------------------------------------- consumers
  // Warp w takes the keys w, w + 4, ... (in groups of 16) of every tile. Scores and
  // probabilities live in MMA fragments: thread (r = lane / 4, t = lane % 4) holds query
  // heads r and r + 8. Probabilities go in as two parts, 16 bits of mantissa in bf16, 22 in f16
  // (e4m3 values; 32 rows of up to 16384, 16 and 4 heads: 54.5 us, by one part 54.4): with
  // at most 8 query heads rows 8 to 15 carry what rounding rows 0 to 7 left over, at no cost;
  // with more a second MMA does, for bf16; over e4m3 values f16's 11 bits stand there (64 rows
  // of up to 8192, 16 query heads a KV head: 42.4 us, 46.4 with the second).
  constexpr bool PAIR = ROWS == 8;
  const int r = lane >> 2, t = lane & 3;
  const float to_log2 = 1.4426950408889634f * rsqrtf((float)HD);
  uint32_t qf[C::KSTEPS][PAIR ? 2 : 4];
  float q_mul[PAIR ? 1 : 2];   // scores' factor (and, for f16 queries, their power of two)
  float o[C::NT][4];
  float mx[2], sum[2];
  float big[2] = {0.f, 0.f}, ref[2] = {kLeastRef, kLeastRef};   // largest weight, its reference
  uint32_t sync_phase = 0;
  int seg_parity = 0;
  auto sync_warps = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(bSync);
    const bool ok = mbar_wait(bSync, sync_phase, abort_flag, a.status);
    sync_phase ^= 1;
    return ok;
  };

  for (int it = 0; it < ntiles; ++it) {
    const int st = it % NST;
    if (!mbar_wait(bFull + 8 * st, (it / NST) & 1, abort_flag, a.status)) return;
    const Tile info = tiles[st];
    const uint32_t kS = base + st * 2 * C::KV, vS = kS + C::KV;
    bool wrote = false;   // this thread wrote to the stage (TMA will overwrite it later)
    if (info.flags & kFirst) {
#pragma unroll
      for (int i = 0; i < C::NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      mx[0] = mx[1] = -INFINITY;
      sum[0] = sum[1] = 0.f;
      big[0] = big[1] = 0.f;
      ref[0] = ref[1] = kLeastRef;
      if (info.valid > 0) {
        // query fragments: bf16 as they are; for e4m3 caches in f16 (the type the codes
        // convert to), each row scaled by a power of two to a largest value in [1, 2)
        // (rows past the query heads are zero: their maxima never move)
        const uint32_t qs = sQ + st * C::QB;
        const int rows = min(ROWS, group - (info.pass % a.passes) * ROWS);
#pragma unroll
        for (int i = 0; i < (PAIR ? 1 : 2); ++i) {
          const uint32_t row = qs + (r + 8 * i) * C::QROW;
          uint32_t w[C::KSTEPS][2];
#pragma unroll
          for (int k = 0; k < C::KSTEPS; ++k) {
            // bf16: columns 2t, 2t+1 and 8 further; e4m3: 4t .. 4t+3 (the order in which a
            // thread finds the codes of K, see below)
            const uint32_t at = row + k * 32 + (FP8 ? t * 8 : t * 4);
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[k][0]) : "r"(at));
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[k][1]) : "r"(at + (FP8 ? 4 : 16)));
            if (r + 8 * i >= rows) w[k][0] = w[k][1] = 0u;
          }
          q_mul[i] = to_log2;
          if constexpr (FP8) {
            float big = 0.f;
#pragma unroll
            for (int k = 0; k < C::KSTEPS; ++k)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float2 f = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w[k][j]));
                big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
              }
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            float p2 = __uint_as_float(__float_as_uint(big) & 0x7f800000u);   // its power of two
            // zeros and tiny rows: 2^-120, whose product with to_log2 is a normal number; rows with
            // an infinity: as they are
            p2 = p2 == INFINITY ? 1.f : fmaxf(p2, 0x1p-120f);
            const float inv = 1.f / p2;
            q_mul[i] *= p2;
#pragma unroll
            for (int k = 0; k < C::KSTEPS; ++k)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float2 f = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w[k][j]));
                w[k][j] = pack_f16x2(f.x * inv, f.y * inv);
              }
          }
#pragma unroll
          for (int k = 0; k < C::KSTEPS; ++k) {
            qf[k][i] = w[k][0];
            qf[k][(PAIR ? 1 : 2) + i] = w[k][1];
          }
        }
      }
    }

    if (warp * 16 < info.valid) {
      // ---- scores of this warp's SUB x 16 keys
      float s[2 * C::SUB][4];
#pragma unroll
      for (int u = 0; u < C::SUB; ++u) {
        const int key0 = (u * 4 + warp) * 16;
#pragma unroll
        for (int j = 0; j < 2; ++j) s[2 * u + j][0] = s[2 * u + j][1] = s[2 * u + j][2] = s[2 * u + j][3] = 0.f;
        if (!FP8) {
#pragma unroll
          for (int k = 0; k < C::KSTEPS; ++k) {
            uint32_t b[4];   // keys 0-7: k 0-7, 8-15; keys 8-15: k 0-7, 8-15
            ldsm4(b, kS + tile_off<C>(key0 + ((lane >> 4) << 3) + (lane & 7), 2 * k + ((lane >> 3) & 1)));
#pragma unroll
            for (int j = 0; j < 2; ++j)
              mma16816<FP8>(s[2 * u + j], qf[k][0], PAIR ? 0u : qf[k][1 % (PAIR ? 2 : 4)],
                            qf[k][PAIR ? 1 : 2], PAIR ? 0u : qf[k][3 % (PAIR ? 2 : 4)], b[2 * j], b[2 * j + 1]);
          }
        } else {
          // a 16-byte chunk holds the 16 codes of one k step; a thread gets codes 4t .. 4t+3
          // of its key, taken as k = 2t, 2t+1 and 2t+8, 2t+9 (the queries' order above)
#pragma unroll
          for (int k = 0; k < C::KSTEPS; k += 2) {
            uint32_t b[4];   // step k: keys 0-7, 8-15; step k + 1: the same
            ldsm4(b, kS + tile_off<C>(key0 + (((lane >> 3) & 1) << 3) + (lane & 7), k + (lane >> 4)));
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                uint32_t b0, b1;
                e4m3x4_f16x2(b[2 * kk + j], b0, b1);
                mma16816<FP8>(s[2 * u + j], qf[k + kk][0], PAIR ? 0u : qf[k + kk][1 % (PAIR ? 2 : 4)],
                              qf[k + kk][PAIR ? 1 : 2], PAIR ? 0u : qf[k + kk][3 % (PAIR ? 2 : 4)],
                              b0, b1);
              }
          }
        }
      }
      // ---- scaling and mask; running maximum
      float vs[2 * C::SUB][2], top[2] = {mx[0], mx[1]};
      const float* sc = reinterpret_cast<const float*>(gbase + (sScale - base) + st * C::SC);
#pragma unroll
      for (int j = 0; j < 2 * C::SUB; ++j) {
        const int key = ((j >> 1) * 4 + warp) * 16 + (j & 1) * 8 + 2 * t;
        float2 ks = make_float2(1.f, 1.f);
        if constexpr (FP8) {
          ks = *reinterpret_cast<const float2*>(sc + key);
          const float2 v2 = *reinterpret_cast<const float2*>(sc + KT + key);
          vs[j][0] = v2.x;
          vs[j][1] = v2.y;
        }
#pragma unroll
        for (int i = 0; i < (PAIR ? 1 : 2); ++i) {
          s[j][2 * i] *= FP8 ? q_mul[i] * ks.x : q_mul[i];
          s[j][2 * i + 1] *= FP8 ? q_mul[i] * ks.y : q_mul[i];
        }
      }
      if (info.valid < KT) {   // slots past the length
#pragma unroll
        for (int j = 0; j < 2 * C::SUB; ++j) {
          const int key = ((j >> 1) * 4 + warp) * 16 + (j & 1) * 8 + 2 * t;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (key + e >= info.valid) {
              s[j][e] = s[j][2 + e] = -INFINITY;
              vs[j][e] = 0.f;
            }
        }
      }
#pragma unroll
      for (int j = 0; j < 2 * C::SUB; ++j) {
#pragma unroll
        for (int i = 0; i < (PAIR ? 1 : 2); ++i) top[i] = fmaxf(top[i], fmaxf(s[j][2 * i], s[j][2 * i + 1]));
      }
      float keep[2], floor2[2];
#pragma unroll
      for (int i = 0; i < (PAIR ? 1 : 2); ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
        floor2[i] = top[i] == -INFINITY ? 0.f : top[i];
        keep[i] = exp2_approx(mx[i] - floor2[i]);
        mx[i] = top[i];
      }
      float moves[2] = {keep[0], PAIR ? keep[0] : keep[PAIR ? 0 : 1]};   // factors of the outputs so far
#pragma unroll
      for (int i = 0; i < (PAIR ? 1 : 2); ++i) {
        float part = 0.f, most = 0.f;
#pragma unroll
        for (int j = 0; j < 2 * C::SUB; ++j) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = s[j][2 * i + e];
            x = exp2_approx(x - floor2[i]);
            part += x;
            if constexpr (FP8) {
              x *= vs[j][e];
              most = fmaxf(most, fabsf(x));
            }
          }
        }
        sum[i] = sum[i] * keep[i] + part;
        if constexpr (FP8) {
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
          big[i] = fmaxf(big[i] * keep[i], most);
          const float now = pow2_at_least(big[i]);
          // it falls with the maximum's rise: keep times their ratio is 2 at most, the ratio
          // alone may be infinite
          if (now != ref[i]) moves[i] = keep[i] == 0.f ? 0.f : keep[i] * (ref[i] / now);
          ref[i] = now;
          const float by = weight_factor(now);
#pragma unroll
          for (int j = 0; j < 2 * C::SUB; ++j) {
            s[j][2 * i] *= by;
            s[j][2 * i + 1] *= by;
          }
        }
      }
      bool moved = moves[0] != 1.f;
      if constexpr (!PAIR) moved |= moves[1] != 1.f;
      if (__any_sync(0xffffffffu, moved)) {
        const float k0 = moves[0], k1 = moves[PAIR ? 0 : 1];
#pragma unroll
        for (int i = 0; i < C::NT; ++i) {
          o[i][0] *= k0;
          o[i][1] *= k0;
          o[i][2] *= k1;
          o[i][3] *= k1;
        }
      }
      // ---- outputs
#pragma unroll
      for (int u = 0; u < C::SUB; ++u) {
        const int key0 = (u * 4 + warp) * 16;
        if (key0 >= info.valid) break;
        if (key0 + 16 > info.valid) {
          // a slot past the length may hold anything; its weight is 0, its value must be too
          constexpr int CH = HD * C::ES / 16;
          const int rows = key0 + 16 - info.valid;
          for (int i = lane; i < rows * CH; i += 32) {
            const uint32_t at = vS + tile_off<C>(info.valid + i / CH, i % CH);
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
          }
          wrote = true;
          __syncwarp();
        }
        uint32_t hi[4], lo[4];
        split_pair<FP8>(s[2 * u][0], s[2 * u][1], hi[0], lo[0]);
        split_pair<FP8>(s[2 * u + 1][0], s[2 * u + 1][1], hi[2], lo[2]);
        if constexpr (!PAIR) {
          split_pair<FP8>(s[2 * u][2], s[2 * u][3], hi[1], lo[1]);
          split_pair<FP8>(s[2 * u + 1][2], s[2 * u + 1][3], hi[3], lo[3]);
        }
        auto accumulate = [&](float (&c)[4], uint32_t b0, uint32_t b1) {
          if constexpr (PAIR) {
            mma16816<FP8>(c, hi[0], lo[0], hi[2], lo[2], b0, b1);
          } else {
            mma16816<FP8>(c, hi[0], hi[1], hi[2], hi[3], b0, b1);
            if (!FP8) mma16816<FP8>(c, lo[0], lo[1], lo[2], lo[3], b0, b1);
          }
        };
#pragma unroll
        for (int c = 0; c < HD / 16; ++c) {
          if constexpr (!FP8) {
            uint32_t b[4];   // columns 16c .. +7: keys 0-7, 8-15; columns 16c + 8 .. +15
            ldsm4_t(b, vS + tile_off<C>(key0 + (((lane >> 3) & 1) << 3) + (lane & 7), 2 * c + (lane >> 4)));
            accumulate(o[2 * c], b[0], b[1]);
            accumulate(o[2 * c + 1], b[2], b[3]);
          } else if ((c & 1) == 0) {
            // transposed as pairs of codes: a register holds dimensions 2r, 2r + 1 of key 2t
            // and of key 2t + 1; with the middle two exchanged, the pair of keys of the even
            // dimension and that of the odd one, which make two column groups
            uint32_t b[4];   // chunk c: keys 0-7, 8-15; chunk c + 1: the same
            ldsm4_t(b, vS + tile_off<C>(key0 + (((lane >> 3) & 1) << 3) + (lane & 7), c + (lane >> 4)));
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
              uint32_t x0, x1, y0, y1;
              e4m3x4_f16x2(__byte_perm(b[2 * cc], 0, 0x3120), x0, x1);
              e4m3x4_f16x2(__byte_perm(b[2 * cc + 1], 0, 0x3120), y0, y1);
              accumulate(o[2 * (c + cc)], x0, y0);
              accumulate(o[2 * (c + cc) + 1], x1, y1);
            }
          }
        }
      }
    }

    if (info.flags & kLast) {
      // ---- the warps' parts of the segment, joined through this tile's stage
      float* ml = warp_ml + seg_parity * 128;
      seg_parity ^= 1;
#pragma unroll
      for (int i = 0; i < (PAIR ? 1 : 2); ++i) {
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        if (t == 0) {
          ml[warp * 16 + r + 8 * i] = mx[i];
          ml[64 + warp * 16 + r + 8 * i] = sum[i];
        }
      }
      if (!sync_warps()) return;
      float top[2], total[2], mine[2];
#pragma unroll
      for (int i = 0; i < (PAIR ? 1 : 2); ++i) {
        top[i] = -INFINITY;
        for (int w = 0; w < kConsumers; ++w) top[i] = fmaxf(top[i], ml[w * 16 + r + 8 * i]);
        const float low = top[i] == -INFINITY ? 0.f : top[i];
        total[i] = 0.f;
        for (int w = 0; w < kConsumers; ++w)
          total[i] += ml[64 + w * 16 + r + 8 * i] * exp2_approx(ml[w * 16 + r + 8 * i] - low);
        mine[i] = exp2_approx(mx[i] - low) * (FP8 ? ref[i] / kWeightScale : 1.f);
      }
      constexpr int W = PAIR ? 2 : 4;   // values a thread keeps per column group
      float* ex = reinterpret_cast<float*>(gbase + st * 2 * C::KV);
#pragma unroll
      for (int i = 0; i < C::NT; ++i) {
        float* at = ex + ((warp * C::NT + i) * 32 + lane) * W;
        if constexpr (PAIR) {
          *reinterpret_cast<float2*>(at) =
              make_float2((o[i][0] + o[i][2]) * mine[0], (o[i][1] + o[i][3]) * mine[0]);
        } else {
          *reinterpret_cast<float4*>(at) = make_float4(o[i][0] * mine[0], o[i][1] * mine[0],
                                                       o[i][2] * mine[PAIR ? 0 : 1], o[i][3] * mine[PAIR ? 0 : 1]);
        }
      }
      wrote = true;
      if (!sync_warps()) return;
      const int g = info.pass / a.passes, h0 = (info.pass % a.passes) * ROWS;
      const int rows = min(ROWS, group - h0);
      const bool whole = !(info.flags & (kBefore | kAfter));
      const int64_t head0 = (int64_t)info.row * a.hq + g * group + h0;
      const int slot = 2 * blockIdx.x + (info.flags & kBefore ? 0 : 1);
      float* part = part_at<HD, ROWS>(a, slot);
      // two column groups (16 dimensions) at a time, as they pair up for e4m3
      for (int c = warp; c < HD / 16; c += kConsumers) {
        float v[2][W];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int e = 0; e < W; ++e) v[j][e] = 0.f;
          for (int w = 0; w < kConsumers; ++w) {
            const float* at = ex + ((w * C::NT + 2 * c + j) * 32 + lane) * W;
#pragma unroll
            for (int e = 0; e < W; ++e) v[j][e] += at[e];
          }
        }
#pragma unroll
        for (int i = 0; i < (PAIR ? 1 : 2); ++i) {
          const int row = r + 8 * i;
          if (row >= rows) continue;
          // dimensions of v[0][0], v[0][1], v[1][0], v[1][1]: e4m3 16c + 4t + {0, 2, 1, 3},
          // bf16 16c + 2t + {0, 1, 8, 9}
          const float x0 = v[0][2 * i], x1 = FP8 ? v[1][2 * i] : v[0][2 * i + 1];
          const float x2 = FP8 ? v[0][2 * i + 1] : v[1][2 * i], x3 = v[1][2 * i + 1];
          const int d0 = 16 * c + (FP8 ? 4 * t : 2 * t), d2 = d0 + (FP8 ? 2 : 8);
          if (whole) {
            const float inv = total[i] > 0.f || total[i] != total[i] ? 1.f / total[i] : 0.f;
            __nv_bfloat16* op = (__nv_bfloat16*)a.o + (head0 + row) * HD;
            *reinterpret_cast<uint32_t*>(op + d0) = pack_bf16x2(x0 * inv, x1 * inv);
            *reinterpret_cast<uint32_t*>(op + d2) = pack_bf16x2(x2 * inv, x3 * inv);
          } else {
            float* pp = part + 2 * ROWS + row * HD;
            *reinterpret_cast<float2*>(pp + d0) = make_float2(x0, x1);
            *reinterpret_cast<float2*>(pp + d2) = make_float2(x2, x3);
          }
        }
      }
      if (warp == 0 && t == 0) {
#pragma unroll
        for (int i = 0; i < (PAIR ? 1 : 2); ++i) {
          const int row = r + 8 * i;
          if (row >= rows) continue;
          if (whole) {
            if (a.lse) a.lse[head0 + row] = (top[i] + log2f(total[i])) * 0.6931471805599453f;
          } else {
            part[row] = top[i];
            part[ROWS + row] = total[i];
          }
        }
      }
      if (warp == 0 && lane == 0 && (info.flags & (kBefore | kAfter)) == kAfter)
        a.join[blockIdx.x] = make_join(*plan, info);
    }
    if (wrote) fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bEmpty + 8 * st);
  }
}

// ---------------------------------------------------------------- fp32 kernel

// fp32 caches: FFMA throughout, as in the layers. Eight lanes share a key (each holds every
// eighth float4 of it), a warp takes 16 keys of each 64-key tile; ROWS query heads share a
// reading of the keys (32 registers of q, 32 of output). The cache's tiles, ranges and joins
// are the tensor-core kernel's.
template <int HD> constexpr int f32_rows() { return 256 / HD; }
// CTAs an SM: as many as the registers allow (24 rows of up to 1000 slots, 4 KV heads of 64:
// two 12.0, three 11.4 us; 64 rows of up to 8192: 113, 95 us; heads of 128 spill at three).
template <int HD> constexpr int f32_ctas() { return HD == 128 ? 2 : 3; }

template <int HD>
__global__ void __launch_bounds__(128, f32_ctas<HD>()) cache_attention_f32_kernel(const DecodeArgs a) {
  constexpr int KT = 64, ROWS = f32_rows<HD>(), CH = HD / 32;
  __shared__ Plan plan_s;
  __shared__ long long scratch[4];
  __shared__ float sm_m[4][ROWS], sm_l[4][ROWS];
  __shared__ __align__(16) float sm_o[4][ROWS][HD];   // written as float4
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane >> 3, l8 = lane & 7;
  pdl_trigger();
  pdl_wait();
  make_plan<KT>(a, &plan_s, scratch);
  const Plan plan = plan_s;
  if (tid == 0) a.join[blockIdx.x].row = -1;
  const int ntiles = (int)(plan.end - plan.begin);
  if (ntiles <= 0) return;
  const int P = a.hkv * a.passes, group = a.hq / a.hkv;
  const float to_log2 = 1.4426950408889634f * rsqrtf((float)HD);
  int m = plan.row, seq;
  int n = row_length(a, m, &seq), nt = row_tiles<KT>(n);
  int pass = (int)(plan.off / nt), tile = (int)(plan.off % nt);
  float4 q[ROWS][CH], o[ROWS][CH];
  float mx[ROWS], sum[ROWS];
  bool first = true;
  for (int it = 0; it < ntiles; ++it) {
    const int g = pass / a.passes, h0 = (pass % a.passes) * ROWS, rows = min(ROWS, group - h0);
    if (first || tile == 0) {
      const float* qp = (const float*)a.q + (int64_t)m * a.ldq + (int64_t)(g * group + h0) * HD;
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        mx[i] = -INFINITY;
        sum[i] = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
          q[i][c] = i < rows ? *reinterpret_cast<const float4*>(qp + i * HD + (c * 8 + l8) * 4)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
    }
    const int key0 = tile * KT + warp * 16;
    if (key0 < n) {
      // the 16 keys lie in one page (page sizes are multiples of 16)
      int page = a.table[(int64_t)seq * a.max_pages + key0 / a.page_size];
      if (page < 0 || page >= a.n_pages) {
        report_status(a.status, XMOD_ERR_DEVICE_CHECK);
        page = 0;
      }
      const int64_t row0 = ((int64_t)page * a.hkv + g) * a.page_size + key0 % a.page_size + sub;
      const float4* kp = reinterpret_cast<const float4*>((const float*)a.k + row0 * HD) + l8;
      const float4* vp = reinterpret_cast<const float4*>((const float*)a.v + row0 * HD) + l8;
      float s[4][ROWS];
      // the values on their way with the keys (plain loads: the launch may begin while the
      // kernel before it still writes the cache, so it is not read-only to this one)
      float4 kk[4][CH], vv[4][CH];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int c = 0; c < CH; ++c)
          kk[j][c] = key0 + 4 * j + sub < n ? kp[j * HD + c * 8]
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int c = 0; c < CH; ++c)
          vv[j][c] = key0 + 4 * j + sub < n ? vp[j * HD + c * 8]
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          float d = 0.f;
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            d = fmaf(q[i][c].x, kk[j][c].x, d);
            d = fmaf(q[i][c].y, kk[j][c].y, d);
            d = fmaf(q[i][c].z, kk[j][c].z, d);
            d = fmaf(q[i][c].w, kk[j][c].w, d);
          }
          d += __shfl_xor_sync(0xffffffffu, d, 1);
          d += __shfl_xor_sync(0xffffffffu, d, 2);
          d += __shfl_xor_sync(0xffffffffu, d, 4);
          s[j][i] = key0 + 4 * j + sub < n ? d * to_log2 : -INFINITY;
        }
      }
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {   // each eight lanes keep the softmax of their keys
        const float top = fmaxf(fmaxf(fmaxf(s[0][i], s[1][i]), fmaxf(s[2][i], s[3][i])), mx[i]);
        const float low = top == -INFINITY ? 0.f : top;
        const float keep = exp2f(mx[i] - low);
        mx[i] = top;
        sum[i] *= keep;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          o[i][c].x *= keep;
          o[i][c].y *= keep;
          o[i][c].z *= keep;
          o[i][c].w *= keep;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = exp2f(s[j][i] - low);
          sum[i] += p;
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            o[i][c].x = fmaf(p, vv[j][c].x, o[i][c].x);
            o[i][c].y = fmaf(p, vv[j][c].y, o[i][c].y);
            o[i][c].z = fmaf(p, vv[j][c].z, o[i][c].z);
            o[i][c].w = fmaf(p, vv[j][c].w, o[i][c].w);
          }
        }
      }
    }
    first = false;
    if (tile == nt - 1 || it == ntiles - 1) {
      // join the warp's four key groups, then the warps
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        float top = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        const float f = exp2f(mx[i] - (top == -INFINITY ? 0.f : top));
        float l = sum[i] * f;
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          float v[4] = {o[i][c].x * f, o[i][c].y * f, o[i][c].z * f, o[i][c].w * f};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] += __shfl_xor_sync(0xffffffffu, v[e], 8);
            v[e] += __shfl_xor_sync(0xffffffffu, v[e], 16);
          }
          if (sub == 0)
            *reinterpret_cast<float4*>(&sm_o[warp][i][(c * 8 + l8) * 4]) =
                make_float4(v[0], v[1], v[2], v[3]);
        }
        if (lane == 0) {
          sm_m[warp][i] = top;
          sm_l[warp][i] = l;
        }
      }
      __syncthreads();
      const bool before = it < tile, after = tile < nt - 1, whole = !before && !after;
      const int64_t head0 = (int64_t)m * a.hq + g * group + h0;
      float* part = part_at<HD, ROWS>(a, 2 * blockIdx.x + (before ? 0 : 1));
      for (int e = tid; e < rows * HD; e += 128) {
        const int i = e / HD, d = e % HD;
        float top = -INFINITY, l = 0.f, v = 0.f;
        for (int w = 0; w < 4; ++w) top = fmaxf(top, sm_m[w][i]);
        const float low = top == -INFINITY ? 0.f : top;
        for (int w = 0; w < 4; ++w) {
          const float f = exp2f(sm_m[w][i] - low);
          l += sm_l[w][i] * f;
          v += sm_o[w][i][d] * f;
        }
        if (whole) {
          ((float*)a.o)[(head0 + i) * HD + d] = l > 0.f || l != l ? v / l : 0.f;
          if (a.lse && d == 0) a.lse[head0 + i] = (top + log2f(l)) * 0.6931471805599453f;
        } else {
          part[2 * ROWS + i * HD + d] = v;
          if (d == 0) {
            part[i] = top;
            part[ROWS + i] = l;
          }
        }
      }
      if (tid == 0 && after && !before) {
        Tile info;
        info.row = m;
        info.pass = pass;
        info.left = nt - 1 - tile;
        a.join[blockIdx.x] = make_join(plan, info);
      }
      __syncthreads();
    }
    if (++tile == nt) {
      tile = 0;
      if (++pass == P) {
        pass = 0;
        if (it + 1 < ntiles) do n = row_length(a, ++m, &seq);
          while (n < 0 && m + 1 < a.M);
        n = max(n, 0);
        nt = row_tiles<KT>(n);
      }
    }
  }
}

// ---------------------------------------------------------------- join

// Segment of CTA blockIdx.x that later CTAs' ranges continue, query head blockIdx.y: the
// parts' maxima and sums, and their outputs weighted to the common maximum. Eight warps take
// every eighth part each, four of them under way at a time; their sums are added in order.
constexpr int kJoinWarps = 8;

template <typename T, int HD, int ROWS>
__global__ void __launch_bounds__(kJoinWarps * 32) cache_attention_join_kernel(const DecodeArgs a) {
  constexpr int E = HD / 32, AHEAD = 4;
  __shared__ float sm_w[kMaxCtas], sm_red[2][kJoinWarps], sm_o[kJoinWarps][HD];
  pdl_trigger();
  pdl_wait();
  const Join j = a.join[blockIdx.x];
  if (j.row < 0) return;
  const int group = a.hq / a.hkv, g = j.pass / a.passes, h0 = (j.pass % a.passes) * ROWS;
  const int row = blockIdx.y;
  if (row >= min(ROWS, group - h0)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = j.last - j.first + 1;
  // part 0 is the starting CTA's second slot, the others their CTAs' first
  auto part = [&](int p) { return part_at<HD, ROWS>(a, 2 * (j.first + p) + (p == 0 ? 1 : 0)); };
  float v[AHEAD][E];   // this warp's first parts, on their way with the maxima
  auto fetch = [&](int p0) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int p = p0 + i * kJoinWarps;
      const float* at = part(min(p, parts - 1)) + 2 * ROWS + row * HD + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) v[i][e] = p < parts ? at[e] : 0.f;
    }
  };
  fetch(warp);
  float m[2], s[2], top = -INFINITY;   // at most kMaxCtas parts: two a thread
  static_assert(kMaxCtas <= 2 * kJoinWarps * 32, "");
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int p = threadIdx.x + i * kJoinWarps * 32;
    m[i] = p < parts ? part(p)[row] : -INFINITY;
    s[i] = p < parts ? part(p)[ROWS + row] : 0.f;
    top = fmaxf(top, m[i]);
  }
  top = warp_max(top);
  if (lane == 0) sm_red[0][warp] = top;
  __syncthreads();
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, sm_red[0][w]);
  const float low = top == -INFINITY ? 0.f : top;
  float l = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int p = threadIdx.x + i * kJoinWarps * 32;
    const float f = exp2f(m[i] - low);
    if (p < parts) sm_w[p] = f;
    l = fmaf(s[i], f, l);
  }
  l = warp_sum(l);
  if (lane == 0) sm_red[1][warp] = l;
  __syncthreads();
  float o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int p0 = warp; p0 < parts; p0 += AHEAD * kJoinWarps) {
    if (p0 != warp) fetch(p0);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int p = p0 + i * kJoinWarps;
      if (p < parts) {
        const float f = sm_w[p];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(v[i][e], f, o[e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = o[e];
  __syncthreads();
  l = 0.f;
  for (int w = 0; w < kJoinWarps; ++w) l += sm_red[1][w];
  const int64_t head = (int64_t)j.row * a.hq + g * group + h0 + row;
  for (int d = threadIdx.x; d < HD; d += kJoinWarps * 32) {
    float x = 0.f;
    for (int w = 0; w < kJoinWarps; ++w) x += sm_o[w][d];
    st_f((T*)a.o + head * HD + d, l > 0.f || l != l ? x / l : 0.f);
  }
  if (a.lse && threadIdx.x == 0) a.lse[head] = (top + log2f(l)) * 0.6931471805599453f;
}

// ---------------------------------------------------------------- host

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

// Query heads per pass: all of a KV head's when they fit the MMA's 16 rows, at most 8 of
// them sharing the rows with the remainders; fp32 see f32_rows.
int pass_rows(const xmod_dims* dm) {
  const int group = dm->n_heads / dm->n_kv_heads;
  if (dm->dtype == XMOD_FP32) return 256 / dm->head_dim;
  return group <= 8 ? 8 : 16;
}

size_t attention_workspace(const xmod_dims* dm) {
  const size_t part = (size_t)pass_rows(dm) * (dm->head_dim + 2) * 4;
  return 256 + round256(kMaxCtas * sizeof(Join)) + 2 * kMaxCtas * part;
}

template <int HD, bool FP8, int ROWS>
int run_tc(const Ctx& c, const DecodeArgs& a, int ctas) {
  using C = Cf<HD, FP8, ROWS>;
  CUtensorMap mk, mv;
  const int64_t rows = (int64_t)a.n_pages * a.hkv * a.page_size;
  if (!tma_map_rows(&mk, a.k, C::ES, rows, HD, C::RB / C::ES, a.box) ||
      !tma_map_rows(&mv, a.v, C::ES, rows, HD, C::RB / C::ES, a.box))
    return XMOD_ERR_CUDA;
  static std::atomic<uint64_t> done{0};
  auto k = cache_attention_kernel<HD, FP8, ROWS>;
  if (allow_smem(k, C::SMEM, done) != cudaSuccess) return XMOD_ERR_CUDA;
  XMOD_LAUNCH(c, "cache_attention",
              launch_pdl(k, dim3(ctas), dim3(kThreads), C::SMEM, c.stream, mk, mv, a));
  const int group = a.hq / a.hkv;
  XMOD_LAUNCH(c, "cache_attn_join",
              launch_pdl(cache_attention_join_kernel<__nv_bfloat16, HD, ROWS>,
                         dim3(ctas, group < ROWS ? group : ROWS), dim3(kJoinWarps * 32), 0,
                         c.stream, a));
  return XMOD_OK;
}

template <int HD>
int run_hd(const Ctx& c, const DecodeArgs& a, int ctas, bool fp32, bool fp8, int rows) {
  if (fp32) {
    XMOD_LAUNCH(c, "cache_attention", launch_pdl(cache_attention_f32_kernel<HD>, dim3(ctas), dim3(128),
                                                 0, c.stream, a));
    constexpr int ROWS = f32_rows<HD>();
    const int group = a.hq / a.hkv;
    XMOD_LAUNCH(c, "cache_attn_join",
                launch_pdl(cache_attention_join_kernel<float, HD, ROWS>,
                           dim3(ctas, group < ROWS ? group : ROWS), dim3(kJoinWarps * 32), 0,
                         c.stream, a));
    return XMOD_OK;
  }
  if (rows == 8) return fp8 ? run_tc<HD, true, 8>(c, a, ctas) : run_tc<HD, false, 8>(c, a, ctas);
  return fp8 ? run_tc<HD, true, 16>(c, a, ctas) : run_tc<HD, false, 16>(c, a, ctas);
}

}  // namespace
}  // namespace xmod

using namespace xmod;

extern "C" {

size_t xmod_cache_attention_workspace_bytes(const xmod_dims* dm, int M) {
  if (!dims_ok(dm) || M < 0 || !head_dim_supported(dm->head_dim)) return 0;
  return attention_workspace(dm);
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
  if (!ptr16(ws) || ws_bytes < attention_workspace(dm)) return XMOD_ERR_WORKSPACE;
  const bool fp32 = dm->dtype == XMOD_FP32, fp8 = cache->format == XMOD_CACHE_E4M3;
  if (!fp32 && !tma_available()) return XMOD_ERR_UNSUPPORTED;
  const int sms = device_sms();
  if (sms <= 0) return XMOD_ERR_CUDA;
  const int per_sm = fp32 && dm->head_dim != 128 ? 3 : 2;   // f32_ctas, Cf: two
  const int ctas = per_sm * sms < kMaxCtas ? per_sm * sms : kMaxCtas;
  const int rows = pass_rows(dm), group = dm->n_heads / dm->n_kv_heads;
  DecodeArgs a{};
  a.M = M;
  a.hq = dm->n_heads;
  a.hkv = dm->n_kv_heads;
  a.ldq = ldq;
  a.q = q;
  a.seq = seq;
  a.len = len;
  a.o = o;
  a.lse = lse;
  a.table = cache->table;
  a.k = cache->k;
  a.v = cache->v;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.n_pages = cache->n_pages;
  a.page_size = cache->page_size;
  a.n_seqs = cache->n_seqs;
  a.max_pages = cache->max_pages;
  a.passes = (group + rows - 1) / rows;
  a.box = cache->page_size % 64 == 0 ? 64 : cache->page_size % 32 == 0 ? 32 : 16;
  a.join = (Join*)((char*)ws + 256);
  a.part = (float*)((char*)ws + 256 + round256(kMaxCtas * sizeof(Join)));
  a.status = (int*)ws;
  const Ctx c{(cudaStream_t)stream, a.status};
  if (dm->head_dim == 128) return run_hd<128>(c, a, ctas, fp32, fp8, rows);
  if (dm->head_dim == 64) return run_hd<64>(c, a, ctas, fp32, fp8, rows);
  return run_hd<32>(c, a, ctas, fp32, fp8, rows);
}

}  // extern "C"
