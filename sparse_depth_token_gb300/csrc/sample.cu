// A token for each row of logits from a given uniform number, with temperature, top-k, top-p
// and min-p.
//
// A CTA has a row: its largest logit, the counts of its values (bf16) or bins' counts and masses
// (fp32) by atomics in shared memory, the cut that top-k, top-p and min-p make, the kept weights
// of a slice of the row for each warp, the token in the slice that the uniform number falls in. Weights
// and sums are whole numbers, so that a sum does not depend on its order; weights have units of
// 2^-62 of the largest and sums 96 bits (in 64 bits, with units that leave room for V weights, 4096 rows
// take 434 us, but 2^22 logits 27 below one were off by 2^-19 of the row's sum). The row is read from
// memory once and from L2 twice or three times. Bound by issue (bf16: 73 thousand instructions a
// row, of all its warps, half of them the counts' and the slices' loops), shared memory's turns, the
// code's way into the instruction cache and the barriers between phases, not by the reads: 4096
// rows of 50257 bf16 logits with top-p 445 us (924 GB/s), 256 rows of fp32 with all settings 114,
// eight rows of bf16 24.

#include <cuda_bf16.h>
#include <math.h>

#include <atomic>

#include "cache.h"   // pointer checks
#include "common.cuh"

namespace xmod {

namespace {

// Tables of powers of two for the weights, in 62-bit fractions: 2^(i / 32) and 2^(i / 1024).
struct PowerTables {
  uint64_t coarse[32], fine[32];
};

const PowerTables& power_tables() {
  static const PowerTables tables = [] {
    PowerTables t{};
    for (int i = 0; i < 32; ++i) {
      t.coarse[i] = (uint64_t)(exp2(i / 32.0) * 4611686018427387904.0);
      t.fine[i] = (uint64_t)(exp2(i / 1024.0) * 4611686018427387904.0);
    }
    return t;
  }();
  return tables;
}

// Weights are whole numbers in units of 2^-62, the largest 2^62; sums of up to 2^22 of them have 96 bits.
constexpr int kUnit = 62;
using wide = unsigned __int128;
static_assert(kUnit + 22 < 96 && XMOD_MAX_VOCAB <= 1 << 22, "");

struct SampleArgs {
  int V;
  int64_t N, ld;
  const void* logits;
  const float *temperature, *top_p, *min_p, *u;
  const int32_t* top_k;
  int32_t* token;
  float* logp;
  int* status;
};

constexpr int kBins = 4096;     // of 1/64 in log2 of the weight, or of a range of keys
constexpr int kList = 1024;     // tokens that are ranked one by one

// What stays of a row, in shared memory. bf16 (table): the table's entries of values that go are
// zeros, `place` is that of the last value kept, of which the first `ties` tokens stay with
// `weight` each; the values too small for the table stay as told. Else tokens above x stay, and
// those at x up to `token`. Weights below `least` go.
struct Cut {
  bool table, small;
  unsigned place;
  uint64_t ties, weight, least;
  float x;
  int token;
};

// The slice that the token lies in: what is left of the target and of the ties there, the kept sum.
struct Choice {
  uint64_t target_lo, target_hi, whole_lo, whole_hi;
  unsigned left;
  int slice;
};

struct Shared {
  uint64_t power[1024];     // 2^(i / 1024) in units of 2^-62, less kRound's bits
  float powerf[1024];       // the same times 2^32
  union {
    struct {
      unsigned mass_lo[kBins], mass_hi[kBins], mass_top[kBins];
    };
    uint64_t value[kBins];  // weights of bf16 values
  };
  unsigned count[kBins];
  uint64_t key[kList], weight[kList];
  uint64_t scan[33], scan2[33];
  uint64_t found[4];
  unsigned long long small_lo, small_hi;   // their mass: small_lo + small_hi 2^32
  unsigned small_n;
  int n;
  Cut cut;
  Choice choice;
};

// Order of a logit as an unsigned number (larger value, larger number; -0 equals +0), above
// the inverted token: keys are distinct and rank as the tokens do.
__device__ __forceinline__ uint64_t key_of(float x, int token) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (uint64_t)(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (0xffffffffu - (uint32_t)token);
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ int key_token(uint64_t key) { return (int)(0xffffffffu - (uint32_t)key); }

// A row's scale: weights are 2^((x - top) c), c = log2(e) / T in two parts.
struct Scale {
  float top, hi, lo;
};

// Where the weight of x lies on a grid of 1/1024 in log2 (0 at the top, descending with x), and
// the rest z: 2^((step + z * 1024) / 1024). The difference and the product are taken with
// their rounding errors (T. J. Dekker, A floating-point technique for extending the available
// precision, 1971), so that the rest is good to 2^-34. kNone: the weight is 0.
constexpr int kNone = -65536;
__device__ __forceinline__ int step_of(const Scale& s, float x, float& z) {
  constexpr float kMagic = 12288.0f;   // its last bit is 2^-10
  const float d = x - s.top, t = d - x;
  const float dd = (x - (d - t)) + (-s.top - t);
  const float p = d * s.hi;
  const float e = fmaf(dd, s.hi, fmaf(d, s.lo, fmaf(d, s.hi, -p)));
  const float n = fmaxf(p, -63.0f) + kMagic;
  z = (p - (n - kMagic)) + e;
  return p > -63.0f ? __float_as_int(n) - __float_as_int(kMagic) : kNone;   // -infinity too
}

// Weight in units of 2^-62: the table's entry for the grid point and a second-order series
// of what is left (at most 2^-11: the next term is below 2^-37), rounded to 2^-32 by adding
// kRound, whose bits the table's entry has less.
constexpr float kRound = 12582912.0f;
__device__ __forceinline__ uint64_t weight_inline(const Shared& sh, const Scale& s, float x) {
  float z;
  const int step = step_of(s, x, z);
  const int j = step & 1023, shift = -(step >> 10);   // 63 at most, or none
  const float q = z * fmaf(z, 0.24022651f, 0.69314718f);
  const int corr = __float_as_int(fmaf(sh.powerf[j], q, kRound));
  const int64_t w = (int64_t)sh.power[j] + (int64_t)corr * (1ll << (kUnit - 32));
  return step == kNone ? 0 : (uint64_t)w >> shift;
}

__device__ __noinline__ uint64_t weight_of(const Shared& sh, Scale s, float x) {
  return weight_inline(sh, s, x);
}

// 16-byte blocks of a row.
template <typename T> struct Row {
  static constexpr int VE = 16 / sizeof(T);
  const T* base;    // aligned
  int off, V, blocks;
  int first, last;   // blocks that lie within the row whole: first .. last - 1
  __device__ Row(const void* logits, int64_t at, int V_) {
    const T* p = (const T*)logits + at;
    off = (int)(((uintptr_t)p & 15) / sizeof(T));
    base = p - off;
    V = V_;
    blocks = (off + V + VE - 1) / VE;
    first = off ? 1 : 0;
    last = (off + V) / VE;
  }
};
// A block that the row's first or last token lies in: -infinity in the others' place.
template <typename T> __device__ __noinline__ uint4 edge_block(const T* base, int off, int V, int v) {
  constexpr int VE = 16 / sizeof(T);
  uint4 r = make_uint4(0, 0, 0, 0);
#pragma unroll 1
  for (int i = VE - 1; i >= 0; --i) {
    const int token = v * VE - off + i;
    const uint32_t x = __float_as_uint(token >= 0 && token < V ? ld_f(base + (int64_t)v * VE + i) : -INFINITY);
    if constexpr (sizeof(T) == 2)
      r = make_uint4(r.x << 16 | x >> 16, __funnelshift_l(r.x, r.y, 16), __funnelshift_l(r.y, r.z, 16),
                     __funnelshift_l(r.z, r.w, 16));
    else
      r = make_uint4(x, r.x, r.y, r.z);
  }
  return r;
}
template <typename T> __device__ __forceinline__ uint4 block_of(const Row<T>& row, int v) {
  return v >= row.first && v < row.last ? *reinterpret_cast<const uint4*>(row.base + (int64_t)v * Row<T>::VE)
                                        : edge_block<T>(row.base, row.off, row.V, v);
}
// Element i of a block.
template <typename T> __device__ __forceinline__ float element(const uint4& u, int i) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w = i < 4 ? i < 2 ? u.x : u.y : i < 6 ? u.z : u.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  } else {
    return __uint_as_float(i < 2 ? i == 0 ? u.x : u.y : i == 2 ? u.z : u.w);
  }
}

// f(v, block) for this thread's blocks v = from, from + STEP, .. below `to`, the next one on its
// way. f's code stands once, rare cases and a row's ends stand out of line: all of a row's phases
// pass through the instruction cache once a row, so longer code costs more than it saves (four
// copies with four loads on their way 786 us for 4096 rows of bf16, one copy 562, that without the
// ends' and the scans' copies 509, with one load ahead 504).
template <typename T, int STEP, typename F>
__device__ __forceinline__ void for_blocks(const Row<T>& row, int from, int to, F&& f) {
  if (from >= to) return;
  uint4 next = block_of(row, from);
#pragma unroll 1
  for (int v = from; v < to; v += STEP) {
    const uint4 now = next;
    if (v + STEP < to) next = block_of(row, v + STEP);
    f(v, now);
  }
}

// Sums of weights. A count of tokens rides in the top 32 bits where both are summed.
struct Sum96 {
  uint64_t lo;
  uint32_t hi;
  __device__ __forceinline__ void add(uint64_t w) {
    asm("add.cc.u64 %0, %0, %2;\n\taddc.u32 %1, %1, 0;" : "+l"(lo), "+r"(hi) : "l"(w));
  }
  __device__ __forceinline__ wide get() const { return (wide)hi << 64 | lo; }
};
__device__ __forceinline__ wide times(uint64_t w, uint32_t n) {   // w below 2^64, n any
  return ((wide)((w >> 32) * n) << 32) + (uint64_t)(uint32_t)w * n;
}
__device__ __forceinline__ wide with_count(uint32_t count, wide mass) { return (wide)count << 96 | mass; }
__device__ __forceinline__ uint32_t count_in(wide v) { return (uint32_t)(v >> 96); }
__device__ __forceinline__ wide mass_in(wide v) { return v & (((wide)1 << 96) - 1); }

__device__ __forceinline__ wide shfl(wide v, int lane) {
  return (wide)__shfl_sync(0xffffffffu, (uint64_t)(v >> 64), lane) << 64 | __shfl_sync(0xffffffffu, (uint64_t)v, lane);
}
// Sum over the lanes up to this one's, of the first `lanes`.
__device__ __forceinline__ wide warp_scan(wide v, int lanes) {
#pragma unroll 1
  for (int o = 1; o < lanes; o <<= 1) {
    const wide up = (wide)__shfl_up_sync(0xffffffffu, (uint64_t)(v >> 64), o) << 64 |
                    __shfl_up_sync(0xffffffffu, (uint64_t)v, o);
    if ((int)(threadIdx.x & 31) >= o) v += up;
  }
  return v;
}

// Sum over the warp of v below 2^80, by pieces of 27 bits.
__device__ __forceinline__ wide warp_sum96(const Sum96& v) {
  const uint32_t p0 = __reduce_add_sync(0xffffffffu, (uint32_t)v.lo & 0x7ffffffu);
  const uint32_t p1 = __reduce_add_sync(0xffffffffu, (uint32_t)(v.lo >> 27) & 0x7ffffffu);
  const uint32_t p2 = __reduce_add_sync(0xffffffffu, (uint32_t)(v.lo >> 54) | v.hi << 10);
  return ((wide)p2 << 54) + (((uint64_t)p1 << 27) + p0);
}

// Sum over the CTA of each thread's v before it; *total the whole sum.
template <int THREADS>
__device__ __forceinline__ wide block_scan(Shared& sh, wide v, wide* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const wide incl = warp_scan(v, 32);
  __syncthreads();
  if (lane == 31) {
    sh.scan[warp] = (uint64_t)incl;
    sh.scan2[warp] = (uint64_t)(incl >> 64);
  }
  __syncthreads();
  // a lane a warp, by one warp: by all of them it costs more than the barrier
  constexpr int WARPS = THREADS / 32;
  if (warp == 0) {
    const wide mine = lane < WARPS ? (wide)sh.scan2[lane] << 64 | sh.scan[lane] : 0;
    const wide upto = warp_scan(mine, WARPS), before = upto - mine;
    __syncwarp();
    if (lane < WARPS) {
      sh.scan[lane] = (uint64_t)before;
      sh.scan2[lane] = (uint64_t)(before >> 64);
    }
    if (lane == WARPS - 1) {
      sh.scan[32] = (uint64_t)upto;
      sh.scan2[32] = (uint64_t)(upto >> 64);
    }
  }
  __syncthreads();
  *total = (wide)sh.scan2[32] << 64 | sh.scan[32];
  return ((wide)sh.scan2[warp] << 64 | sh.scan[warp]) + (incl - v);
}

// f * w rounded down for f >= 0 (w below 2^96), and whether something was cut off.
__device__ __forceinline__ wide scaled(float f, wide w, bool* cut) {
  const uint32_t b = __float_as_uint(f) & 0x7fffffffu;   // -0 is 0
  const int ex = (int)(b >> 23);
  const int right = 150 - (ex ? ex : 1);   // f = m 2^-right, right >= 23 up to 1
  const wide v = w * ((b & 0x7fffffu) | (ex ? 0x800000u : 0u));
  const wide r = right < 128 ? v >> right : 0;
  *cut = right < 128 ? r << right != v : v != 0;
  return r;
}

__device__ __forceinline__ void add_mass(Shared& sh, int b, uint64_t w) {
  const unsigned lo = (unsigned)w, old = atomicAdd(&sh.mass_lo[b], lo);
  const unsigned hi = (unsigned)(w >> 32) + (old + lo < old ? 1u : 0u);
  if (hi) {
    const unsigned before = atomicAdd(&sh.mass_hi[b], hi);
    if (before + hi < before) atomicAdd(&sh.mass_top[b], 1u);
  }
}
__device__ __forceinline__ wide bin_of(const Shared& sh, int b) {   // count and mass
  return (wide)((uint64_t)sh.count[b] << 32 | sh.mass_top[b]) << 64 | ((uint64_t)sh.mass_hi[b] << 32 | sh.mass_lo[b]);
}

template <int THREADS> __device__ __forceinline__ void clear_bins(Shared& sh) {
#pragma unroll 1
  for (int b = threadIdx.x; b < kBins; b += THREADS) sh.mass_lo[b] = sh.mass_hi[b] = sh.mass_top[b] = sh.count[b] = 0;
  __syncthreads();
}

// First bin at which the running sum of counts (by_mass: masses) reaches `need` (bin kBins: none),
// what lies before it, and the whole sums.
struct Crossing {
  int bin;
  uint32_t count;   // before the bin
  wide mass;        // the same
  wide all_mass;
};
template <int THREADS>
__device__ __forceinline__ Crossing find_bin(Shared& sh, bool by_mass, wide need) {
  constexpr int PER = kBins / THREADS;
  wide mine = 0, total;
#pragma unroll 1
  for (int i = 0; i < PER; ++i) mine += bin_of(sh, threadIdx.x * PER + i);
  wide before = block_scan<THREADS>(sh, mine, &total);
  if (threadIdx.x == 0) {   // what a sum that never reaches `need` would leave
    sh.found[0] = kBins;
    sh.found[1] = sh.found[2] = sh.found[3] = 0;
  }
  __syncthreads();
  auto of = [&](wide v) { return by_mass ? mass_in(v) : (wide)count_in(v); };
  if (of(before) < need && need <= of(before + mine)) {
#pragma unroll 1
    for (int i = 0; i < PER; ++i) {
      const int b = threadIdx.x * PER + i;
      const wide upto = before + bin_of(sh, b);
      if (need <= of(upto)) {
        sh.found[0] = b;
        sh.found[1] = count_in(before);
        sh.found[2] = (uint64_t)before;
        sh.found[3] = (uint64_t)(mass_in(before) >> 64);
        break;
      }
      before = upto;
    }
  }
  __syncthreads();
  const Crossing r{(int)sh.found[0], (uint32_t)sh.found[1], (wide)sh.found[3] << 64 | sh.found[2], mass_in(total)};
  __syncthreads();
  return r;
}

// The key at which the running count (by_mass: mass) over the tokens of bin `bin` in their
// order reaches `need`, and the mass up to it. `clobbered`: the bins were used for finer ones.
template <typename T, int THREADS>
__device__ __noinline__ uint64_t find_key(Shared& sh, const Row<T> row, const Scale sc, int bin, bool by_mass,
                                          wide need, wide* mass_to, bool* clobbered) {
  constexpr int VE = Row<T>::VE;
  uint64_t lo = 0, hi = ~0ull;
  wide before_mass = 0;
  bool ranged = false;   // members are those with keys in lo .. hi, else those of the bin
  auto visit = [&](auto&& f) {
    uint4 next = threadIdx.x < row.blocks ? block_of(row, threadIdx.x) : make_uint4(0, 0, 0, 0);
#pragma unroll 1
    for (int v = threadIdx.x; v < row.blocks; v += THREADS) {
      const uint4 u = next;
      if (v + THREADS < row.blocks) next = block_of(row, v + THREADS);
      unsigned in = 0;
#pragma unroll (sizeof(T) == 4 ? 4 : 1)
      for (int i = 0; i < VE; ++i) {
        const float x = element<T>(u, i);
        const uint64_t key = key_of(x, v * VE - row.off + i);
        float z;
        in |= (ranged ? key >= lo && key <= hi : min(kBins - 1, -step_of(sc, x, z) >> 4) == bin) ? 1u << i : 0u;
      }
      // few are members, and none of those outside the row
#pragma unroll 1
      for (; in; in &= in - 1) {
        const int i = __ffs(in) - 1;
        const float x = element<T>(u, i);
        f(key_of(x, v * VE - row.off + i), x);
      }
    }
  };
  // every turn leaves a 4096th of the keys: six are enough for 64 bits
  for (int level = 0; level < 7; ++level) {
    if (threadIdx.x == 0) {
      sh.n = 0;
      sh.found[0] = ~0ull;
      sh.found[1] = 0;
    }
    __syncthreads();
    visit([&](uint64_t key, float x) {
      const int i = atomicAdd(&sh.n, 1);
      if (i < kList) {
        sh.key[i] = key;
        sh.weight[i] = weight_of(sh, sc, x);
      }
    });
    __syncthreads();
    if (sh.n <= kList) break;
    *clobbered = true;
    if (!ranged) {   // the members' range of keys
      uint64_t mn = ~0ull, mx = 0;
      visit([&](uint64_t key, float) {
        mn = key < mn ? key : mn;
        mx = key > mx ? key : mx;
      });
      atomicMin((unsigned long long*)&sh.found[0], (unsigned long long)mn);
      atomicMax((unsigned long long*)&sh.found[1], (unsigned long long)mx);
      __syncthreads();
      lo = sh.found[0];
      hi = sh.found[1];
      ranged = true;
      __syncthreads();
    }
    int shift = 0;
    while ((hi - lo) >> shift >= kBins) ++shift;
    clear_bins<THREADS>(sh);
    visit([&](uint64_t key, float x) {
      const int b = (int)((hi - key) >> shift);
      atomicAdd(&sh.count[b], 1u);
      add_mass(sh, b, weight_of(sh, sc, x));
    });
    __syncthreads();
    const Crossing at = find_bin<THREADS>(sh, by_mass, need);
    const int sub = min(at.bin, kBins - 1);
    need -= by_mass ? at.mass : (wide)at.count;
    before_mass += at.mass;
    hi -= (uint64_t)sub << shift;
    const uint64_t width = (1ull << shift) - 1;
    if (hi - lo > width) lo = hi - width;
    __syncthreads();
  }
  const int n = min(sh.n, kList);
  __syncthreads();
  if (threadIdx.x == 0) sh.found[0] = sh.found[1] = sh.found[2] = 0;
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < n; i += THREADS) {
    const uint64_t key = sh.key[i], w = sh.weight[i];
    unsigned above = 0;
    Sum96 sum{0, 0};
#pragma unroll 4
    for (int j = 0; j < n; ++j)
      if (sh.key[j] > key) {
        ++above;
        sum.add(sh.weight[j]);
      }
    const wide above_mass = sum.get();
    if (by_mass ? above_mass < need && need <= above_mass + w : above + 1 == need) {
      sh.found[0] = key;
      sh.found[1] = (uint64_t)(above_mass + w);
      sh.found[2] = (uint64_t)((above_mass + w) >> 64);
    }
  }
  __syncthreads();
  const uint64_t key = sh.found[0];
  *mass_to = before_mass + ((wide)sh.found[2] << 64 | sh.found[1]);
  __syncthreads();
  return key;
}

// ---------------------------------------------------------------- bf16 values
//
// bf16 rows have few values, so their weights come from a table that a row's CTA works out
// once, 4096 entries for 2^-9 <= |x| < 128. Smaller values are worked out as they come; logits
// below -127.5 count as that, whose weight has to be 0 (else, as with a largest logit outside the
// table, the row goes the general way).
constexpr int kValues = 2048;         // of a sign
constexpr unsigned kLeastValue = 0x3b00;   // 2^-9; the 2048 patterns from here differ in their last 11 bits
constexpr unsigned kLowest = 0xc2ff;       // -127.5

__device__ __forceinline__ unsigned place_of(unsigned bits) { return (bits & 0x7ffu) | (bits >> 4 & 0x800u); }
__device__ __forceinline__ bool in_table(unsigned bits) { return (bits & 0x7fffu) - kLeastValue < kValues; }
__device__ __forceinline__ int place_size(int place) { return (place - (kLeastValue & 0x7ff)) & 0x7ff; }   // by |x|
__device__ __forceinline__ float place_value(int place) {
  return __uint_as_float((kLeastValue + place_size(place) | (place >= kValues ? 0x8000u : 0u)) << 16);
}
// Values in falling order.
__device__ __forceinline__ int place_rank(int place) {
  return place < kValues ? kValues - 1 - place_size(place) : kValues + place_size(place);
}
__device__ __forceinline__ int place_at(int rank) {
  const int size = rank < kValues ? kValues - 1 - rank : rank - kValues;
  return ((kLeastValue + size) & 0x7ff) | (rank < kValues ? 0 : kValues);
}
__device__ __forceinline__ uint4 clamped(const uint4& raw) {
  uint4 r;
  const uint32_t low = kLowest << 16 | kLowest;
  const __nv_bfloat162 l = *reinterpret_cast<const __nv_bfloat162*>(&low);
  const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&raw);
  __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = __hmax2(b[i], l);
  return r;
}
// Whether all eight values of a clamped block of a row below 128 lie in the table.
__device__ __forceinline__ bool all_in_table(const uint4& u) {
  const unsigned m = 0x7fff7fffu, least = kLeastValue << 16 | kLeastValue;
  const unsigned x = __vminu2(__vminu2(u.x & m, u.y & m), __vminu2(u.z & m, u.w & m));
  return __vminu2(x, least) == least;
}
__device__ __forceinline__ unsigned half_of(const uint4& u, int i) {
  const uint32_t w = i < 2 ? u.x : i < 4 ? u.y : i < 6 ? u.z : u.w;
  return i & 1 ? w >> 16 : w & 0xffffu;
}
// Byte offsets of the places of a word's two values in a table of entries of 2^SHIFT bytes.
template <int SHIFT> __device__ __forceinline__ uint32_t offsets(uint32_t w) {
  return (w & 0x07ff07ffu) << SHIFT | (w >> (4 - SHIFT) & 0x08000800u << SHIFT);
}
template <typename E> __device__ __forceinline__ E& entry(E* table, uint32_t bytes) {
  return *reinterpret_cast<E*>(reinterpret_cast<char*>(table) + bytes);
}
// Sum of the entries at two byte offsets past a table's address in shared memory, each if its half
// of x (bf16) is above that of cut. Lanes that do not read cost no bank's turn: with an eighth of
// the values above the cut 818 -> 786 us for 4096 rows.
__device__ __forceinline__ uint64_t sum_above(uint32_t table, uint32_t offsets, uint32_t x, uint32_t cut) {
  uint64_t a, b;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.gt.bf16x2 p|q, %4, %5;\n\tmov.b64 %0, 0;\n\tmov.b64 %1, 0;\n\t"
      "@p ld.shared.b64 %0, [%2];\n\t@q ld.shared.b64 %1, [%3];\n\t}"
      : "=&l"(a), "=&l"(b)
      : "r"(table + (offsets & 0xffffu)), "r"(table + (offsets >> 16)), "r"(x), "r"(cut)
      : "memory");
  return a + b;
}
// The values beside the table, a bit each, and the block with the lowest value in their place: its
// weight is 0 and it ranks last, so that it may be counted without harm.
__device__ __forceinline__ unsigned beside_table(uint4 u) {
  unsigned r = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) r |= in_table(half_of(u, i)) ? 0u : 1u << i;
  return r;
}
__device__ __forceinline__ uint32_t lowest_for(uint32_t w, unsigned beside) {
  const uint32_t m = (beside & 1 ? 0xffffu : 0u) | (beside & 2 ? 0xffff0000u : 0u);
  return (w & ~m) | ((kLowest << 16 | kLowest) & m);
}
__device__ __forceinline__ uint4 lowest_for(const uint4& u, unsigned beside) {
  return make_uint4(lowest_for(u.x, beside), lowest_for(u.y, beside >> 2), lowest_for(u.z, beside >> 4),
                    lowest_for(u.w, beside >> 6));
}

// Counts the clamped values u that `live` tells, which lie beside the table.
__device__ __noinline__ void count_block(Shared& sh, Scale sc, uint4 u, unsigned live) {
  atomicAdd(&sh.small_n, (unsigned)__popc(live));
  uint64_t lo = 0, hi = 0;
#pragma unroll 1
  for (; live; live &= live - 1) {
    const uint64_t w = weight_of(sh, sc, __uint_as_float(half_of(u, __ffs(live) - 1) << 16));
    lo += (uint32_t)w;
    hi += w >> 32;
  }
  atomicAdd(&sh.small_lo, (unsigned long long)lo);
  atomicAdd(&sh.small_hi, (unsigned long long)hi);
}
__device__ __forceinline__ wide small_mass(const Shared& sh) { return ((wide)sh.small_hi << 32) + sh.small_lo; }

// Counts of the table's values and the cut by them. False: the cut lies among the smaller values.
template <int THREADS>
__device__ __forceinline__ bool table_cut(Shared& sh, const Row<__nv_bfloat16> row, const Scale sc, int top_k,
                                       float top_p, bool by_k, bool by_p) {
  const int tid = threadIdx.x;
  for_blocks<__nv_bfloat16, THREADS>(row, tid, row.blocks, [&](int, const uint4& raw) {
    uint4 u = clamped(raw);
    if (!all_in_table(u)) {
      const unsigned beside = beside_table(u);
      count_block(sh, sc, u, beside);
      u = lowest_for(u, beside);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t at = offsets<2>((&u.x)[i]);
      atomicAdd(&entry(sh.count, at & 0xffffu), 1u);
      atomicAdd(&entry(sh.count, at >> 16), 1u);
    }
  });
  __syncthreads();
  // running sums in rank order; the small values lie between the signs
  constexpr int PER = kBins / THREADS;
  const int r0 = tid * PER;
  unsigned c = 0;
  uint64_t m_lo = 0, m_hi = 0;   // of the weights' low and high words: at most 2^57
  {   // the thread's ranks are PER places in a row, from a multiple of PER on
    const int at = min(place_at(r0), place_at(r0 + PER - 1));
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
      const uint4 n = *reinterpret_cast<const uint4*>(&sh.count[at + i]);
      const ulonglong2 v0 = *reinterpret_cast<const ulonglong2*>(&sh.value[at + i]);
      const ulonglong2 v1 = *reinterpret_cast<const ulonglong2*>(&sh.value[at + i + 2]);
      c += n.x + n.y + n.z + n.w;
      m_lo += (v0.x & 0xffffffffu) * n.x + (v0.y & 0xffffffffu) * n.y + (v1.x & 0xffffffffu) * n.z + (v1.y & 0xffffffffu) * n.w;
      m_hi += (v0.x >> 32) * n.x + (v0.y >> 32) * n.y + (v1.x >> 32) * n.z + (v1.y >> 32) * n.w;
    }
  }
  const wide m = ((wide)m_hi << 32) + m_lo;
  wide all;
  const wide before2 = block_scan<THREADS>(sh, with_count(c, m), &all);
  const unsigned cb = count_in(before2) + (r0 >= kValues ? sh.small_n : 0u);
  const wide mb = mass_in(before2) + (r0 >= kValues ? small_mass(sh) : 0);
  // where a sum reaches `need`: found = {place, tokens of it, sum up to it}
  auto reach = [&](bool by_mass, wide need) {
    __syncthreads();
    if (tid < 32) {
      if (by_mass) {   // top_p of what is kept, rounded up, by one warp
        bool more;
        need = scaled(top_p, need, &more);
        need += more;
        if (need == 0) need = 1;
      }
      if (tid == 0) {
        sh.found[0] = kBins;
        sh.choice.target_lo = (uint64_t)need;
        sh.choice.target_hi = (uint64_t)(need >> 64);
      }
    }
    __syncthreads();
    need = (wide)sh.choice.target_hi << 64 | sh.choice.target_lo;
    const wide before = by_mass ? mb : (wide)cb;
    if (before < need && need <= before + (by_mass ? m : (wide)c)) {
      unsigned count = cb;
      wide mass = mb;
#pragma unroll 1
      for (int i = 0; i < PER; ++i) {
        const int at = place_at(r0 + i);
        const unsigned n = sh.count[at];
        const uint64_t w = sh.value[at];
        if (by_mass ? need <= mass + times(w, n) : need <= count + n) {
          unsigned keep = (unsigned)need - count;
          if (by_mass) {   // need - mass over w, rounded up: about, then exactly
            const wide rest = need - mass;
            keep = (unsigned)__fdividef((float)(uint64_t)(rest >> 64) * 0x1p64f + (float)(uint64_t)rest, (float)w);
#pragma unroll 1
            while (times(w, keep) < rest) ++keep;
#pragma unroll 1
            while (keep > 1 && times(w, keep - 1) >= rest) --keep;
          }
          mass += times(w, keep);
          sh.found[0] = at;
          sh.found[1] = keep;
          sh.found[2] = (uint64_t)mass;
          sh.found[3] = (uint64_t)(mass >> 64);
          break;
        }
        count += n;
        mass += times(w, n);
      }
    }
    __syncthreads();
  };
  wide kept = mass_in(all) + small_mass(sh);
  uint64_t ties = 0;
  unsigned place = kBins;
  if (by_k) {
    reach(false, top_k);
    place = (unsigned)sh.found[0];
    if (place == kBins) return false;
    ties = sh.found[1];
    kept = (wide)sh.found[3] << 64 | sh.found[2];
  }
  if (by_p) {
    reach(true, kept);
    const unsigned at = (unsigned)sh.found[0];
    if (at == kBins) return false;
    // of one place p's cut is within k's
    if (place == kBins || place_rank(at) <= place_rank(place)) {
      place = at;
      ties = sh.found[1];
    }
  }
  const uint64_t weight = sh.value[place];
  __syncthreads();
  if (tid == 0) {
    sh.cut.place = place;
    sh.cut.weight = weight;
    sh.cut.ties = weight < sh.cut.least ? 0 : ties;
    sh.cut.small = place >= kValues;
  }
  const int rank = place_rank(place);
#pragma unroll 1
  for (int i = tid; i < kBins; i += THREADS)
    if (place_rank(i) >= rank) sh.value[i] = 0;
  return true;
}

// Counts and masses of a row's bins below `region`; the mass of the others is returned unless by_k
// (what is kept then lies in the bins): small weights are summed aside, not by atomics, unless the
// cut lies among them.
template <typename T, int THREADS>
__device__ __noinline__ wide fill_bins(Shared& sh, const Row<T> row, const Scale sc, bool by_k, bool by_p,
                                           int region) {
  clear_bins<THREADS>(sh);
  Sum96 mass{0, 0};
  for_blocks<T, THREADS>(row, threadIdx.x, row.blocks, [&](int, const uint4& u) {
// fp32 comes this way alone: 122 us for 256 rows with four copies, 129 with one
#pragma unroll (sizeof(T) == 4 ? 4 : 1)
    for (int i = 0; i < Row<T>::VE; ++i) {
      const float x = element<T>(u, i);
      float z;
      const int b = min(kBins - 1, -step_of(sc, x, z) >> 4);
      const uint64_t w = by_p && (b < region || !by_k) ? weight_inline(sh, sc, x) : 0;
      if (b < region) {
        if (by_k) atomicAdd(&sh.count[b], 1u);
        if (w) add_mass(sh, b, w);
      } else {
        mass.add(w);
      }
    }
  });
  wide all;
  block_scan<THREADS>(sh, mass.get(), &all);
  __syncthreads();
  return all;
}

// The lowest key kept by top-k and top-p, of any values.
template <typename T, int THREADS>
__device__ __noinline__ uint64_t general_cut(Shared& sh, const Row<T> row, const Scale sc, int top_k, float top_p,
                                             bool by_k, bool by_p) {
  uint64_t cut = 0;
  wide rest_mass = 0;
  auto fill = [&](int region) { rest_mass = fill_bins<T, THREADS>(sh, row, sc, by_k, by_p, region); };
  int region = 24 * 64;
  fill(region);
  wide kept = 0;
  bool clobbered = false;
  if (by_k) {
    wide to;
    Crossing at = find_bin<THREADS>(sh, false, top_k);
    if (at.bin == kBins && region < kBins) {
      fill(region = kBins);
      at = find_bin<THREADS>(sh, false, top_k);
    }
    kept = at.mass;
    if (at.bin < kBins - 1) {   // the last bin's weights are 0: kept or not is the same
      cut = find_key<T, THREADS>(sh, row, sc, at.bin, false, top_k - at.count, &to, &clobbered);
      kept += to;
    }
  } else {
    kept = find_bin<THREADS>(sh, true, ~(wide)0).all_mass + rest_mass;
  }
  if (by_p) {
    if (clobbered) fill(region);
    bool more;
    wide need = scaled(top_p, kept, &more);
    need += more;
    if (need == 0) need = 1;
    wide to;
    Crossing at = find_bin<THREADS>(sh, true, need);
    if (at.bin == kBins && region < kBins) {
      fill(region = kBins);
      at = find_bin<THREADS>(sh, true, need);
    }
    const uint64_t key = find_key<T, THREADS>(sh, row, sc, at.bin, true, need - at.mass, &to, &clobbered);
    cut = key > cut ? key : cut;
  }
  return cut;
}

// Weights of the clamped values u that `live` tells, which lie beside the table, summed.
__device__ __noinline__ wide sum_block(const Shared& sh, Scale sc, uint4 u, unsigned live) {
  Sum96 sum{0, 0};
#pragma unroll 1
  for (; live; live &= live - 1) {
    const uint64_t t = weight_of(sh, sc, __uint_as_float(half_of(u, __ffs(live) - 1) << 16));
    sum.add(t >= sh.cut.least ? t : 0);
  }
  return sum.get();
}
// Weight of a token if it stays for sure, in the general way.
__device__ __forceinline__ uint64_t key_weight(const Shared& sh, const Scale& sc, const Cut& cut, int token, float x) {
  if (!(x > cut.x || (x == cut.x && token <= cut.token))) return 0;
  const uint64_t t = weight_inline(sh, sc, x);
  return t >= cut.least ? t : 0;
}
// In any way; *tied: it is of the last value kept.
template <typename T>
__device__ __noinline__ uint64_t token_weight(const Shared& sh, Scale sc, int token, float x) {
  const Cut& cut = sh.cut;
  if (sizeof(T) != 2 || !cut.table) return key_weight(sh, sc, cut, token, x);
  const unsigned bits = __float_as_uint(fmaxf(x, -127.5f)) >> 16;
  if (in_table(bits)) return sh.value[place_of(bits)];   // 0 if it goes or is tied
  if (!cut.small) return 0;
  const uint64_t t = weight_of(sh, sc, x);
  return t >= cut.least ? t : 0;
}
// The choice among what stays.
template <typename T, int THREADS>
__device__ __forceinline__ void choose(const SampleArgs& a, Shared& sh, const Row<T> row, const Scale sc, int64_t r,
                                    float u, float temp) {
  constexpr int VE = Row<T>::VE, WARPS = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Cut cut = sh.cut;
  // ---- kept weights by slices of the row, a warp each
  const int per = (row.blocks + WARPS - 1) / WARPS;
  Sum96 sum{0, 0};   // a lane's slice
  unsigned tied = 0;
  // equal to no logit without a cut by the table
  const bool ranked = sizeof(T) == 2 && cut.table && cut.place < kBins;
  const float cut_value = ranked ? place_value(cut.place) : __int_as_float(0x7fc00000);
  const int slice_end = min(row.blocks, (warp + 1) * per);
  if (sizeof(T) == 2 && cut.table) {
    if constexpr (sizeof(T) == 2) {
      // ties of the low and the high halves, 16 bits each; without a cut all are above -infinity
      const uint32_t cut_bits = cut.place < kBins ? __float_as_uint(place_value(cut.place)) : 0xff800000u;
      const uint32_t value = (uint32_t)__cvta_generic_to_shared(sh.value);
      const uint32_t pattern = cut_bits | cut_bits >> 16;
      unsigned ties = 0;
      for_blocks<T, 32>(row, warp * per + lane, slice_end, [&](int, const uint4& raw) {
        uint4 u = raw;
        if (cut.small) {   // else nothing outside the table is above the cut or equal to it
          u = clamped(raw);
          if (!all_in_table(u)) {
            const unsigned beside = beside_table(u);
            const wide t = sum_block(sh, sc, u, beside);
            sum.add((uint64_t)t);
            sum.hi += (uint32_t)(t >> 64);
            u = lowest_for(u, beside);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = (&u.x)[i], at = offsets<3>(w);
          const __nv_bfloat162 x2 = *reinterpret_cast<const __nv_bfloat162*>(&w);
          sum.add(sum_above(value, at, w, pattern));
          ties += __heq2_mask(x2, *reinterpret_cast<const __nv_bfloat162*>(&pattern)) & 0x00010001u;
        }
      });
      tied = (ties & 0xffffu) + (ties >> 16);
    }
  } else {
    for_blocks<T, 32>(row, warp * per + lane, slice_end, [&](int v, const uint4& u) {
#pragma unroll (sizeof(T) == 4 ? 4 : 1)
      for (int i = 0; i < VE; ++i) sum.add(key_weight(sh, sc, cut, v * VE - row.off + i, element<T>(u, i)));
    });
  }
  const wide slice_sum = with_count(__reduce_add_sync(0xffffffffu, tied), warp_sum96(sum));
  __syncthreads();
  if (lane == 0) {
    sh.scan[warp] = (uint64_t)slice_sum;
    sh.scan2[warp] = (uint64_t)(slice_sum >> 64);
  }
  __syncthreads();
  if (warp == 0) {
    // a lane a slice: the ties before it, what is kept of it, and up to it
    const wide slice_of = lane < WARPS ? (wide)sh.scan2[lane] << 64 | sh.scan[lane] : 0;
    const unsigned ties_all = (unsigned)cut.ties, here = count_in(slice_of);
    unsigned met_before = here;
#pragma unroll 1
    for (int o = 1; o < WARPS; o <<= 1) {
      const unsigned up = __shfl_up_sync(0xffffffffu, met_before, o);
      if (lane >= o) met_before += up;
    }
    met_before -= here;
    const unsigned ties_left = ties_all - min(ties_all, met_before);
    const wide mass = mass_in(slice_of) + times(cut.weight, min(here, ties_left));
    const wide upto = warp_scan(mass, WARPS);
    const wide whole = shfl(upto, WARPS - 1);
    bool rest;
    const wide target = scaled(u, whole, &rest);   // the running sum has to exceed it, as the whole does
    const int slice = min(__ffs(__ballot_sync(0xffffffffu, target < upto)) - 1, WARPS - 1);
    if (lane == slice) {
      const wide within = target - (upto - mass);
      sh.choice = Choice{(uint64_t)within, (uint64_t)(within >> 64), (uint64_t)whole, (uint64_t)(whole >> 64), ties_left, slice};
    }
  }
  __syncthreads();
  const int slice = sh.choice.slice;
  wide target = (wide)sh.choice.target_hi << 64 | sh.choice.target_lo;
  unsigned left = sh.choice.left;   // ties not yet met
  // ---- the token within the slice, a block a thread
#pragma unroll 1
  for (int v0 = slice * per; v0 < min(row.blocks, (slice + 1) * per); v0 += THREADS) {
    const int v = v0 + tid;
    // the block's weights and its tokens of the last value kept
    const bool live = v < min(row.blocks, (slice + 1) * per);
    Sum96 sure{0, 0};
    unsigned met = 0;
    uint4 block = make_uint4(0, 0, 0, 0);
    if (live) {
      block = block_of(row, v);
#pragma unroll 1
      for (int i = 0; i < VE; ++i) {
        const float x = element<T>(block, i);
        sure.add(token_weight<T>(sh, sc, v * VE - row.off + i, x));
        met += sizeof(T) == 2 && x == cut_value;
      }
    }
    wide all;
    const wide before2 = block_scan<THREADS>(sh, with_count(met, sure.get()), &all);
    // the first `left` ties stay
    const unsigned ties_before = min(count_in(before2), left), ties_here = min(met, left - ties_before);
    const wide before = mass_in(before2) + times(cut.weight, ties_before);
    const wide mine = sure.get() + times(cut.weight, ties_here);
    if (before <= target && target < before + mine) {
      wide cum = before;
      unsigned stay = ties_here;
      int at = -1;
      float x_at = 0.f;
#pragma unroll 1
      for (int i = 0; i < VE && cum <= target; ++i) {
        x_at = element<T>(block, i);
        at = i;
        if (sizeof(T) == 2 && x_at == cut_value) {
          if (stay) {
            cum += cut.weight;
            --stay;
          }
        } else {
          cum += token_weight<T>(sh, sc, v * VE - row.off + i, x_at);
        }
      }
      a.token[r] = v * VE - row.off + at;
      if (a.logp) {
        // (x - top) / temp - ln(whole 2^-62), each with its rounding errors
        const float d = x_at - sc.top, t = d - x_at, dd = (x_at - (d - t)) + (-sc.top - t);
        const float q = d / temp, qq = temp < INFINITY ? (fmaf(-q, temp, d) + dd) / temp : 0.0f;
        // whole = 2^e (1 + f); it has the largest weight or, at least, the chosen one
        const uint64_t high = sh.choice.whole_hi;
        const wide whole = (wide)high << 64 | sh.choice.whole_lo;
        const int e = high ? 127 - __clzll(high) : 63 - __clzll((uint64_t)whole);
        const uint64_t head = (uint64_t)(e > 63 ? whole >> (e - 63) : whole << (63 - e));
        const float f = (float)(head & 0x7fffffffffffffffull) * 0x1p-63f;
        const float n = (float)(e - kUnit);
        constexpr float kLn2Hi = 0.693145752f, kLn2Lo = 1.42860677e-6f;   // the first of 15 bits: exact times n
        const float big = q - n * kLn2Hi, rest2 = (q - big) - n * kLn2Hi;
        a.logp[r] = big + (rest2 + ((qq - n * kLn2Lo) - log1pf(f)));
      }
    }
    const unsigned ties_here_all = min(count_in(all), left);
    const wide whole_here = mass_in(all) + times(cut.weight, ties_here_all);
    if (target < whole_here) break;
    target -= whole_here;
    left -= ties_here_all;
  }
}

// The largest of two, a NaN if one is.
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
// The row's largest logit, a NaN if it holds one. Every thread has it.
template <typename T, int THREADS>
__device__ __forceinline__ float row_top(Shared& sh, const Row<T> row) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float top = -INFINITY;
  __nv_bfloat162 top2 = __float2bfloat162_rn(-INFINITY);
  for_blocks<T, THREADS>(row, tid, row.blocks, [&](int, const uint4& raw) {
    if constexpr (sizeof(T) == 2) {
      const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&raw);
      top2 = __hmax2_nan(top2, __hmax2_nan(__hmax2_nan(b[0], b[1]), __hmax2_nan(b[2], b[3])));
    } else {
      top = max_nan(top, max_nan(max_nan(__uint_as_float(raw.x), __uint_as_float(raw.y)),
                                 max_nan(__uint_as_float(raw.z), __uint_as_float(raw.w))));
    }
  });
  const float2 f = __bfloat1622float2(top2);
  top = max_nan(top, max_nan(f.x, f.y));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  __syncthreads();
  float* tops = reinterpret_cast<float*>(sh.scan);
  if (lane == 0) tops[warp] = top;
  __syncthreads();
  top = tops[lane < THREADS / 32 ? lane : 0];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  __syncthreads();
  return top + 0.0f;
}
// The first token whose logit is `top`.
template <typename T, int THREADS>
__device__ __noinline__ int first_token(Shared& sh, const Row<T> row, float top) {
  constexpr int VE = Row<T>::VE;
  if (threadIdx.x == 0) sh.n = row.V;
  __syncthreads();
#pragma unroll 1
  for (int v = threadIdx.x; v < row.blocks; v += THREADS) {
    const uint4 u = block_of(row, v);
    unsigned at = 0;
#pragma unroll
    for (int i = 0; i < VE; ++i) at |= element<T>(u, i) == top ? 1u << i : 0u;
    if (at) {
      atomicMin(&sh.n, v * VE - row.off + __ffs(at) - 1);
      break;   // the thread's others come later
    }
  }
  __syncthreads();
  return sh.n;
}

template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
sample_kernel(const SampleArgs a, const __grid_constant__ PowerTables tables) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  const int tid = threadIdx.x;
  pdl_trigger();
  for (int i = tid; i < 1024; i += THREADS) {
    const uint64_t p = __umul64hi(tables.coarse[i >> 5], tables.fine[i & 31]);   // 60-bit fraction
    sh.power[i] = (p << (kUnit - 60)) - ((uint64_t)__float_as_int(kRound) << (kUnit - 32));
    sh.powerf[i] = (float)(p >> 28);
  }
  pdl_wait();
#pragma unroll 1
  for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x) {
    const Row<T> row(a.logits, r * a.ld, a.V);
    const float top = row_top<T, THREADS>(sh, row);
    float temp = a.temperature ? a.temperature[r] : 1.0f;
    const float u = a.u[r], min_p = a.min_p ? a.min_p[r] : 0.0f, top_p = a.top_p ? a.top_p[r] : 1.0f;
    const int top_k = a.top_k ? a.top_k[r] : 0;
    if (!(top > -INFINITY && top < INFINITY) || !(u >= 0.0f && u < 1.0f) || temp != temp ||
        min_p != min_p || top_p != top_p) {
      if (tid == 0) {
        report_status(a.status, XMOD_ERR_DEVICE_CHECK);
        a.token[r] = -1;
        if (a.logp) a.logp[r] = __int_as_float(0x7fc00000);
      }
      continue;
    }
    if (temp <= 0.0f || top_k == 1 || top_p <= 0.0f) {
      const int token = first_token<T, THREADS>(sh, row, top);
      if (tid == 0) {
        a.token[r] = token;
        if (a.logp) a.logp[r] = 0.0f;
      }
      continue;
    }
    Scale sc;
    sc.top = top;
    {   // log2(e) / temp, the division's remainder in the second part
      constexpr float kHi = 1.44269502f, kLo = 1.92596299e-8f;   // log2(e)
      temp = fmaxf(temp, kHi * 0x1p-120f);   // below it sc.hi would pass fp32's range
      sc.hi = kHi / temp;
      sc.lo = temp < INFINITY ? (fmaf(-sc.hi, temp, kHi) + kLo) / temp : 0.0f;
    }
    const bool by_k = top_k > 0 && top_k < a.V, by_p = top_p < 1.0f;
    uint64_t least = 0;
    if (min_p > 0.0f) {
      bool more;
      least = (uint64_t)scaled(fminf(min_p, 1.0f), (wide)1 << kUnit, &more) + more;
    }
    // -127.5 at (-127.5 - top) sc.hi: none of its weight is left 62 below
    bool table = sizeof(T) == 2 && in_table(__float_as_uint(top) >> 16) && (-127.5f - top) * sc.hi < -64.0f;
    if (tid == 0) {
      sh.cut = Cut{table, true, kBins, 0, 0, least, -INFINITY, a.V};
      sh.small_n = 0;
      sh.small_lo = sh.small_hi = 0;
    }
    if constexpr (sizeof(T) == 2) {
      if (table) {
#pragma unroll 1
        for (int i = tid; i < kBins; i += THREADS) {
          const float x = place_value(i);
          sh.value[i] = x <= top ? weight_inline(sh, sc, x) : 0;
          sh.count[i] = 0;
        }
        __syncthreads();
        if (by_k || by_p) table = table_cut<THREADS>(sh, row, sc, top_k, top_p, by_k, by_p);
        if (table && least) {
          __syncthreads();
#pragma unroll 1
          for (int i = tid; i < kBins; i += THREADS)
            if (sh.value[i] < least) sh.value[i] = 0;
        }
      }
    }
    if ((by_k || by_p) && !table) {
      __syncthreads();
      const uint64_t cut = general_cut<T, THREADS>(sh, row, sc, top_k, top_p, by_k, by_p);
      if (tid == 0) {
        sh.cut.table = false;
        sh.cut.x = cut ? key_value(cut) : -INFINITY;
        sh.cut.token = cut ? key_token(cut) : a.V;
      }
    }
    __syncthreads();
    choose<T, THREADS>(a, sh, row, sc, r, u, temp);
  }
}

template <typename T, int THREADS>
cudaError_t launch_sample(const Ctx& c, const SampleArgs& a) {
  static std::atomic<uint64_t> done{0};
  auto k = sample_kernel<T, THREADS>;
  const cudaError_t e = allow_smem(k, (int)sizeof(Shared), done);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)device_sms() * (THREADS == 1024 ? 1 : 2);
  return launch_pdl(k, dim3((unsigned)(a.N < most ? a.N : most)), dim3(THREADS), sizeof(Shared), c.stream, a,
                    power_tables());
}

}  // namespace
}  // namespace xmod

using namespace xmod;

extern "C" {

int xmod_sample_tokens(xmod_dtype dt, int64_t N, int V, const void* logits, int64_t ld,
                       const float* temperature, const int32_t* top_k, const float* top_p,
                       const float* min_p, const float* u, int32_t* token, float* logp,
                       int* status_out, void* stream) {
  if ((dt != XMOD_BF16 && dt != XMOD_FP32) || N < 0 || V <= 0 || ld < V) return XMOD_ERR_INVALID_ARG;
  if (V > XMOD_MAX_VOCAB) return XMOD_ERR_UNSUPPORTED;
  if (N == 0) return XMOD_OK;
  if (!logits || (uintptr_t)logits % (dt == XMOD_BF16 ? 2 : 4) || !ptr4_or_null(temperature) ||
      !ptr4_or_null(top_k) || !ptr4_or_null(top_p) || !ptr4_or_null(min_p) || !u || !ptr4_or_null(u) ||
      !token || !ptr4_or_null(token) || !ptr4_or_null(logp) || !ptr4_or_null(status_out))
    return XMOD_ERR_INVALID_ARG;
  if (device_sms() <= 0) return XMOD_ERR_CUDA;
  SampleArgs a{};
  a.V = V;
  a.N = N;
  a.ld = ld;
  a.logits = logits;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.u = u;
  a.token = token;
  a.logp = logp;
  a.status = status_out;
  const Ctx c{(cudaStream_t)stream, status_out};
  // A row an SM: twice the threads (152 rows of 50257 with top-p, us: bf16 23.1, with 512 threads 24.3;
  // fp32 60 and 80; rows of 1000 13.3 and 11.8, 17.3 and 16.9). More: two CTAs an SM (153 rows of
  // bf16 33.0, with 1024 threads 40.1, 608 rows 70 and 92; fp32 111 and 110, 234 and 244; rows of 1000
  // 15 and 22).
  if (N <= device_sms())
    XMOD_LAUNCH(c, "sample_tokens", (dt == XMOD_BF16 ? launch_sample<__nv_bfloat16, 1024>(c, a)
                                                     : launch_sample<float, 1024>(c, a)));
  else
    XMOD_LAUNCH(c, "sample_tokens", (dt == XMOD_BF16 ? launch_sample<__nv_bfloat16, 512>(c, a)
                                                     : launch_sample<float, 512>(c, a)));
  return XMOD_OK;
}

}  // extern "C"
