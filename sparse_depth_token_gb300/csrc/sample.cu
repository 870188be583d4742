// A token for each row of logits from a given uniform number, with temperature, top-k, top-p
// and min-p.

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

struct SampleArgs {
  int V, unit;     // weights in units of 2^-unit
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

struct Shared {
  uint64_t power[1024];     // 2^(i / 1024) in units of 2^-unit
  float powerf[1024];       // the same times 2^40
  unsigned mass_lo[kBins], mass_hi[kBins], count[kBins];
  uint64_t key[kList], weight[kList];
  uint64_t scan[33], scan2[33];
  uint64_t found[4];
  int n;
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
  int unit;
};

// Where the weight of x lies on a grid of 1/1024 in log2 (0 at the top, descending with x), and
// the rest z: 2^((step + z * 1024) / 1024). The difference and the product are taken with
// their rounding errors (T. J. Dekker, A floating-point technique for extending the available
// precision, 1971), so that the rest is good to 2^-34.
__device__ __forceinline__ int step_of(const Scale& s, float x, float& z) {
  constexpr float kMagic = 12288.0f;   // its last bit is 2^-10
  const float d = x - s.top, t = d - x;
  const float dd = (x - (d - t)) + (-s.top - t);
  const float p = d * s.hi;
  const float e = fmaf(dd, s.hi, fmaf(d, s.lo, fmaf(d, s.hi, -p)));
  const float n = fmaxf(p, -63.0f) + kMagic;
  z = (p - (n - kMagic)) + e;
  return p > -63.0f ? __float_as_int(n) - __float_as_int(kMagic) : -65536;   // -infinity too
}

// Weight in units of 2^-unit: the table's entry for the grid point and a second-order series
// of what is left (at most 2^-11: the next term is below 2^-37).
__device__ __forceinline__ uint64_t weight_of(const Shared& sh, const Scale& s, float x) {
  float z;
  const int step = step_of(s, x, z);
  if (step <= -64512) return 0;
  const int j = step & 1023, shift = -(step >> 10);
  const float q = z * fmaf(z, 0.24022651f, 0.69314718f);
  const int corr = __float2int_rn(sh.powerf[j] * q);
  const int64_t w = (int64_t)sh.power[j] + (int64_t)corr * (1ll << (s.unit - 40));
  return (uint64_t)w >> shift;
}

// Elements of 16-byte block v of a row, -infinity for those outside it.
template <typename T> struct Row {
  static constexpr int VE = 16 / sizeof(T);
  const T* base;    // aligned
  int off, V, blocks;
  __device__ Row(const void* logits, int64_t at, int V_) {
    const T* p = (const T*)logits + at;
    off = (int)(((uintptr_t)p & 15) / sizeof(T));
    base = p - off;
    V = V_;
    blocks = (int)(((int64_t)off + V + VE - 1) / VE);
  }
  __device__ __forceinline__ void load(int v, float (&x)[VE]) const {
    const int e0 = v * VE - off;   // token of the block's first element
    if (e0 >= 0 && e0 + VE <= V) {
      const uint4 raw = *reinterpret_cast<const uint4*>(base + (int64_t)v * VE);
#pragma unroll
      for (int i = 0; i < VE / 2; ++i) {
        const float2 f = vec_pair<T>(raw, i);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i)
        x[i] = e0 + i >= 0 && e0 + i < V ? ld_f(base + (int64_t)v * VE + i) : -INFINITY;
    }
  }
};

__device__ __forceinline__ uint64_t shfl_up64(uint64_t v, int o) { return __shfl_up_sync(0xffffffffu, v, o); }

// Sum over the CTA of each thread's v before it; *total the whole sum.
template <int THREADS>
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* scratch, uint64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t up = shfl_up64(incl, o);
    if (lane >= o) incl += up;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  uint64_t before = 0, sum = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += scratch[w];
    sum += scratch[w];
  }
  *total = sum;
  return before + incl - v;
}

// f * w rounded down for f >= 0, and whether something was cut off.
__device__ __forceinline__ uint64_t scaled(float f, uint64_t w, bool* cut) {
  const uint32_t b = __float_as_uint(f);
  const int ex = (int)(b >> 23);
  const uint64_t m = (b & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int right = 150 - (ex ? ex : 1);   // f = m 2^-right, right >= 24 below 1
  const uint64_t lo = m * w, hi = __umul64hi(m, w);
  if (right < 64) {
    *cut = (lo & ((1ull << right) - 1)) != 0;
    return hi << (64 - right) | lo >> right;
  }
  const int r = right - 64;
  *cut = lo != 0 || (r < 64 ? (hi & ((1ull << r) - 1)) != 0 : hi != 0);
  return r < 64 ? hi >> r : 0;
}

__device__ __forceinline__ void add_mass(Shared& sh, int b, uint64_t w) {
  const unsigned lo = (unsigned)w, old = atomicAdd(&sh.mass_lo[b], lo);
  const unsigned hi = (unsigned)(w >> 32) + (old + lo < old ? 1u : 0u);
  if (hi) atomicAdd(&sh.mass_hi[b], hi);
}

template <int THREADS> __device__ __forceinline__ void clear_bins(Shared& sh) {
  for (int b = threadIdx.x; b < kBins; b += THREADS) sh.mass_lo[b] = sh.mass_hi[b] = sh.count[b] = 0;
  __syncthreads();
}

// First bin at which the running sum of counts (by_mass: masses) reaches `need`; what lies
// before it. The sums reach it.
struct Crossing {
  int bin;
  uint64_t count, mass;   // before the bin
};
template <int THREADS>
__device__ Crossing find_bin(Shared& sh, bool by_mass, uint64_t need, uint64_t* all_mass) {
  constexpr int PER = kBins / THREADS;
  uint64_t c = 0, m = 0, total, total_c;
  for (int i = 0; i < PER; ++i) {
    const int b = threadIdx.x * PER + i;
    c += sh.count[b];
    m += (uint64_t)sh.mass_hi[b] << 32 | sh.mass_lo[b];
  }
  uint64_t cb = block_scan<THREADS>(c, sh.scan, &total_c);
  uint64_t mb = block_scan<THREADS>(m, sh.scan2, &total);
  if (all_mass) *all_mass = total;
  if (threadIdx.x == 0) {   // what a sum that never reaches `need` would leave
    sh.found[0] = kBins - 1;
    sh.found[1] = sh.found[2] = 0;
  }
  __syncthreads();
  const uint64_t before = by_mass ? mb : cb, mine = by_mass ? m : c;
  if (before < need && need <= before + mine) {
    for (int i = 0; i < PER; ++i) {
      const int b = threadIdx.x * PER + i;
      const uint64_t bc = sh.count[b], bm = (uint64_t)sh.mass_hi[b] << 32 | sh.mass_lo[b];
      if (need <= (by_mass ? mb + bm : cb + bc)) {
        sh.found[0] = b;
        sh.found[1] = cb;
        sh.found[2] = mb;
        break;
      }
      cb += bc;
      mb += bm;
    }
  }
  __syncthreads();
  const Crossing r{(int)sh.found[0], sh.found[1], sh.found[2]};
  __syncthreads();
  return r;
}

// The key at which the running count (by_mass: mass) over the tokens of bin `bin` in their
// order reaches `need`, and the mass up to it. `clobbered`: the bins were used for finer ones.
template <typename T, int THREADS>
__device__ uint64_t find_key(Shared& sh, const Row<T>& row, const Scale& sc, int bin, uint64_t members,
                             bool by_mass, uint64_t need, uint64_t* mass_to, bool* clobbered) {
  constexpr int VE = Row<T>::VE;
  uint64_t lo = 0, hi = ~0ull, before_mass = 0;
  bool ranged = false;   // members are those with keys in lo .. hi, else those of the bin
  auto visit = [&](auto&& f) {
    for (int v = threadIdx.x; v < row.blocks; v += THREADS) {
      float x[VE];
      row.load(v, x);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const int token = v * VE - row.off + i;
        if (token < 0 || token >= row.V) continue;
        const uint64_t key = key_of(x[i], token);
        float z;
        const bool in = ranged ? key >= lo && key <= hi : min(kBins - 1, -step_of(sc, x[i], z) >> 4) == bin;
        if (in) f(key, x[i]);
      }
    }
  };
  // every turn leaves a 4096th of the keys: six are enough for 64 bits
  for (int level = 0; members > kList && level < 6; ++level) {
    *clobbered = true;
    if (!ranged) {   // the members' range of keys
      uint64_t mn = ~0ull, mx = 0;
      visit([&](uint64_t key, float) {
        mn = key < mn ? key : mn;
        mx = key > mx ? key : mx;
      });
      __syncthreads();
      if (threadIdx.x == 0) {
        sh.found[0] = ~0ull;
        sh.found[1] = 0;
      }
      __syncthreads();
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
    const Crossing at = find_bin<THREADS>(sh, by_mass, need, nullptr);
    need -= by_mass ? at.mass : at.count;
    before_mass += at.mass;
    members = sh.count[at.bin];
    hi -= (uint64_t)at.bin << shift;
    const uint64_t width = (1ull << shift) - 1;
    if (hi - lo > width) lo = hi - width;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    sh.n = 0;
    sh.found[0] = sh.found[1] = 0;
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
  const int n = min(sh.n, kList);
  for (int i = threadIdx.x; i < n; i += THREADS) {
    const uint64_t key = sh.key[i], w = sh.weight[i];
    uint64_t above = 0, above_mass = 0;
    for (int j = 0; j < n; ++j)
      if (sh.key[j] > key) {
        ++above;
        above_mass += sh.weight[j];
      }
    if (by_mass ? above_mass < need && need <= above_mass + w : above + 1 == need) {
      sh.found[0] = key;
      sh.found[1] = above_mass + w;
    }
  }
  __syncthreads();
  const uint64_t key = sh.found[0];
  *mass_to = before_mass + sh.found[1];
  __syncthreads();
  return key;
}

template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS)
sample_kernel(const SampleArgs a, const __grid_constant__ PowerTables tables) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  constexpr int VE = Row<T>::VE, WARPS = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  for (int i = tid; i < 1024; i += THREADS) {
    const uint64_t p = __umul64hi(tables.coarse[i >> 5], tables.fine[i & 31]);   // 60-bit fraction
    sh.power[i] = a.unit >= 60 ? p << (a.unit - 60) : p >> (60 - a.unit);
    sh.powerf[i] = (float)(p >> 20);
  }
  pdl_wait();
  for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x) {
    const Row<T> row(a.logits, r * a.ld, a.V);
    // ---- the first token in rank; a NaN
    uint64_t best = 0;
    bool bad = false;
    {
      float top = -INFINITY;
      int at = -1;
#pragma unroll 2
      for (int v = tid; v < row.blocks; v += THREADS) {
        float x[VE];
        row.load(v, x);
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          if (x[i] > top) {
            top = x[i];
            at = v * VE - row.off + i;
          }
          bad |= x[i] != x[i];
        }
      }
      if (at >= 0) best = key_of(top, at);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(0xffffffffu, best, o);
      best = other > best ? other : best;
    }
    __syncthreads();
    if (lane == 0) sh.scan[warp] = best;
    bad = __syncthreads_or(bad);
    for (int w = 0; w < WARPS; ++w) best = sh.scan[w] > best ? sh.scan[w] : best;
    __syncthreads();

    const float temp = a.temperature ? a.temperature[r] : 1.0f;
    const float u = a.u[r], min_p = a.min_p ? a.min_p[r] : 0.0f, top_p = a.top_p ? a.top_p[r] : 1.0f;
    const int top_k = a.top_k ? a.top_k[r] : 0;
    const float top = key_value(best);
    if (bad || best == 0 || top == INFINITY || !(u >= 0.0f && u < 1.0f) || temp != temp ||
        min_p != min_p || top_p != top_p) {
      if (tid == 0) {
        report_status(a.status, XMOD_ERR_DEVICE_CHECK);
        a.token[r] = -1;
        if (a.logp) a.logp[r] = __int_as_float(0x7fc00000);
      }
      continue;
    }
    if (temp <= 0.0f || top_k == 1 || top_p <= 0.0f) {
      if (tid == 0) {
        a.token[r] = key_token(best);
        if (a.logp) a.logp[r] = 0.0f;
      }
      continue;
    }
    Scale sc;
    sc.top = top;
    sc.unit = a.unit;
    {   // log2(e) / temp, the division's remainder in the second part
      constexpr float kHi = 1.44269502f, kLo = 1.92596299e-8f;   // log2(e)
      sc.hi = kHi / temp;
      sc.lo = (fmaf(-sc.hi, temp, kHi) + kLo) / temp;
      if (!(sc.hi < 0x1p120f)) {   // any difference between logits is then beyond the last weight
        sc.hi = 0x1p120f;
        sc.lo = 0.0f;
      }
    }
    // ---- the cut of top-k and top-p: the lowest key that is kept
    uint64_t cut = 0;
    const bool by_k = top_k > 0 && top_k < a.V, by_p = top_p < 1.0f;
    if (by_k || by_p) {
      auto fill = [&]() {
        clear_bins<THREADS>(sh);
        for (int v = tid; v < row.blocks; v += THREADS) {
          float x[VE];
          row.load(v, x);
#pragma unroll
          for (int i = 0; i < VE; ++i) {
            const int token = v * VE - row.off + i;
            if (token < 0 || token >= a.V) continue;
            float z;
            const int b = min(kBins - 1, -step_of(sc, x[i], z) >> 4);
            atomicAdd(&sh.count[b], 1u);
            if (by_p) {
              const uint64_t w = weight_of(sh, sc, x[i]);
              if (w) add_mass(sh, b, w);
            }
          }
        }
        __syncthreads();
      };
      fill();
      uint64_t kept = 0;
      bool clobbered = false;
      if (by_k) {
        uint64_t to;
        const Crossing at = find_bin<THREADS>(sh, false, top_k, nullptr);
        kept = at.mass;
        if (at.bin < kBins - 1) {   // the last bin's weights are 0: kept or not is the same
          cut = find_key<T, THREADS>(sh, row, sc, at.bin, sh.count[at.bin], false, top_k - at.count, &to,
                                     &clobbered);
          kept += to;
        }
      }
      if (by_p) {
        if (clobbered) fill();
        uint64_t all;
        if (!by_k) {
          find_bin<THREADS>(sh, false, 1, &all);
          kept = all;
        }
        bool more;
        uint64_t need = scaled(top_p, kept, &more);
        need += more;
        if (need == 0) need = 1;
        uint64_t to;
        const Crossing at = find_bin<THREADS>(sh, true, need, nullptr);
        const uint64_t key = find_key<T, THREADS>(sh, row, sc, at.bin, sh.count[at.bin], true,
                                                  need - at.mass, &to, &clobbered);
        cut = key > cut ? key : cut;
      }
    }
    const float cut_x = cut ? key_value(cut) : -INFINITY;
    const int cut_token = cut ? key_token(cut) : a.V;
    uint64_t least = 0;
    if (min_p > 0.0f) {
      bool more;
      least = scaled(fminf(min_p, 1.0f), 1ull << a.unit, &more);
      least += more;
    }
    auto kept_weight = [&](float x, int token) -> uint64_t {
      if (!(x > cut_x || (x == cut_x && token <= cut_token))) return 0;
      const uint64_t w = weight_of(sh, sc, x);
      return w >= least ? w : 0;
    };
    // ---- kept weights by slices of the row, a warp each
    const int per = (row.blocks + WARPS - 1) / WARPS;
    uint64_t sum = 0;
#pragma unroll 2
    for (int v = warp * per + lane; v < min(row.blocks, (warp + 1) * per); v += 32) {
      float x[VE];
      row.load(v, x);
#pragma unroll
      for (int i = 0; i < VE; ++i) sum += kept_weight(x[i], v * VE - row.off + i);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sh.scan[warp] = sum;
    __syncthreads();
    uint64_t whole = 0;
    for (int w = 0; w < WARPS; ++w) whole += sh.scan[w];
    bool rest;
    uint64_t target = scaled(u, whole, &rest);   // the running sum has to exceed it
    int slice = 0;
    for (; slice < WARPS - 1 && target >= sh.scan[slice]; ++slice) target -= sh.scan[slice];
    __syncthreads();
    // ---- the token within the slice, a block a thread
    for (int v0 = slice * per; v0 < min(row.blocks, (slice + 1) * per); v0 += THREADS) {
      const int v = v0 + tid;
      uint64_t w[VE], mine = 0, all;
      float x[VE];
      if (v < min(row.blocks, (slice + 1) * per)) {
        row.load(v, x);
#pragma unroll
        for (int i = 0; i < VE; ++i) mine += w[i] = kept_weight(x[i], v * VE - row.off + i);
      }
      const uint64_t before = block_scan<THREADS>(mine, sh.scan, &all);
      if (before <= target && target < before + mine) {
        uint64_t cum = before;
        bool done = false;
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          cum += w[i];
          if (!done && cum > target) {
            done = true;
            a.token[r] = v * VE - row.off + i;
            if (a.logp) {
              const int e = 63 - __clzll(whole);
              const float f = (float)(whole - (1ull << e)) * exp2f((float)-e);
              a.logp[r] = (float)(((double)x[i] - (double)top) / (double)temp -
                                  ((double)(e - a.unit) * 0.6931471805599453 + (double)log1pf(f)));
            }
          }
        }
      }
      if (target < all) break;
      target -= all;
    }
    __syncthreads();
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
  int bits = 1;
  while ((1 << bits) < V) ++bits;
  a.unit = 62 - bits;
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
  // few rows: one CTA an SM with twice the threads
  if (N <= device_sms())
    XMOD_LAUNCH(c, "sample_tokens", (dt == XMOD_BF16 ? launch_sample<__nv_bfloat16, 1024>(c, a)
                                                     : launch_sample<float, 1024>(c, a)));
  else
    XMOD_LAUNCH(c, "sample_tokens", (dt == XMOD_BF16 ? launch_sample<__nv_bfloat16, 512>(c, a)
                                                     : launch_sample<float, 512>(c, a)));
  return XMOD_OK;
}

}  // extern "C"
