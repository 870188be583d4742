// Attention of a chunk of new tokens over the paged cache on FFMA: fp32 throughout (tf32 would keep
// ten bits of q, K and the weights). Bound: FFMA, of which 64 x 64 tiles reach 36 TFLOP/s (500
// tokens at 8192 of 16 and 4 heads of 128 910 us, eight chunks of 512 at 4096 of 64 889); small calls
// by the latency of one to three tiles a CTA and the join (six of 100 at 1000 35 us).

#include <limits.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "cache_chunk.cuh"

namespace xmod {

namespace {

constexpr int kRows = kChunkF32Rows, kThreads = 256;

template <int HD> struct Smem {
  static constexpr int QLD = HD + 4, PLD = kChunkKeys + 4;
  // heads of 128: keys and values share a buffer, so that two CTAs fit an SM (500 tokens at 8192 of
  // 16 and 4 heads: 910 us; one CTA with both on their way 1574)
  static constexpr bool kShared = HD == 128;
  float q[kRows * QLD], k[kChunkKeys * QLD], own_v[kShared ? 4 : kChunkKeys * QLD], p[kRows * PLD];
  __device__ __forceinline__ float* v() { return kShared ? k : own_v; }
  ChunkPlan plan;
  long long scratch[kThreads / 32];
};

// 16 x 16 threads: thread (ty, tx) has rows 4 ty .. 4 ty + 3, keys tx + 16 j of the scores and
// dimensions 4 tx + 64 j .. of the output.
template <int HD>
__global__ void __launch_bounds__(kThreads, 2) cache_chunk_f32_kernel(const ChunkArgs a) {
  using S = Smem<HD>;
  constexpr int DW = HD >= 64 ? 4 : 2, DN = HD / (16 * DW);   // DN groups of DW dimensions
  extern __shared__ __align__(16) uint8_t smem[];
  S& s = *reinterpret_cast<S*>(smem);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  pdl_trigger();
  pdl_wait();
  make_chunk_plan(a, &s.plan, s.scratch);
  if (tid == 0) a.join[blockIdx.x].first = -1;
  if (s.plan.begin >= s.plan.end) return;
  ChunkWalk w;
  w.begin(a, s.plan);
  const float to_log2 = 1.4426950408889634f * rsqrtf((float)HD);
  while (w.next(a)) {
    const int first = w.first, last = w.last;
    ChunkRow row[4];
    float mx[4], sum[4], o[4][DN * DW];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      row[i] = chunk_row(a, w.k, w.hp, w.t, 0, 4 * ty + i);
      mx[i] = -INFINITY;
      sum[i] = 0.f;
#pragma unroll
      for (int d = 0; d < DN * DW; ++d) o[i][d] = 0.f;
    }
    __syncthreads();   // the segment before is done with the queries
    for (int i = tid; i < kRows * (HD / 4); i += kThreads) {
      const int R = i / (HD / 4), d = i % (HD / 4) * 4;
      const ChunkRow r = chunk_row(a, w.k, w.hp, w.t, 0, R);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r.m >= 0) {
        const float* p = (const float*)a.q + r.m * a.ldq + r.head * HD + d;
        x = make_float4(ld_f(p) * to_log2, ld_f(p + 1) * to_log2, ld_f(p + 2) * to_log2, ld_f(p + 3) * to_log2);
      }
      *reinterpret_cast<float4*>(&s.q[R * S::QLD + d]) = x;
    }
    // A tile's slots on their way into shared memory, those at and after the segment's limit as
    // zeros. A thread copies vector tid % CH of the keys tid / CH + STEP j; the pages of those are
    // looked up a tile ahead.
    constexpr int CH = HD / 4, STEP = kThreads / CH, N = kChunkKeys / STEP;
    const int g = chunk_kv_head(a, w.hp), c4 = tid % CH * 4, key_in = tid / CH;
    auto pages_of = [&](int tile, int (&page)[N]) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        // tiles past the last one may lie past 2^31
        const int slot = tile < last ? tile * kChunkKeys + key_in + STEP * j : INT_MAX;
        page[j] = slot < w.limit ? chunk_page(a, w.k, slot) : 0;
      }
    };
    auto copy = [&](const float* cache, float* to, int tile, const int (&page)[N]) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int key = key_in + STEP * j, slot = tile * kChunkKeys + key;
        int pg = page[j];
        if (pg < 0 || pg >= a.n_pages) {
          report_status(a.status, XMOD_ERR_DEVICE_CHECK);
          pg = 0;
        }
        const int64_t at = ((int64_t)pg * a.hkv + g) * a.page_size + chunk_in_page(a, slot);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(to + key * S::QLD + c4)),
                     "l"(cache + (slot < w.limit ? at * HD + c4 : 0)), "r"(slot < w.limit ? 16 : 0)
                     : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int page[N], page_next[N];
    pages_of(first, page);
    pages_of(first + 1, page_next);
    copy((const float*)a.k, s.k, first, page);
    if (!S::kShared) copy((const float*)a.v, s.v(), first, page);
    for (int tile = first; tile < last; ++tile) {
      const int key0 = tile * kChunkKeys;
      if (S::kShared)
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      else
        asm volatile("cp.async.wait_group 1;" ::: "memory");   // the keys; the values may be under way
      __syncthreads();
      float sc[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[i][j] = 0.f;
#pragma unroll 2
      for (int d = 0; d < HD; d += 4) {
        float4 qv[4], kv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4*>(&s.q[(4 * ty + i) * S::QLD + d]);
#pragma unroll
        for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(&s.k[(tx + 16 * j) * S::QLD + d]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            sc[i][j] = fmaf(qv[i].x, kv[j].x, fmaf(qv[i].y, kv[j].y, fmaf(qv[i].z, kv[j].z, fmaf(qv[i].w, kv[j].w, sc[i][j]))));
      }
      bool masked = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float top = mx[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (key0 + tx + 16 * j >= row[i].limit) sc[i][j] = -INFINITY;
          top = fmaxf(top, sc[i][j]);
        }
        masked |= row[i].limit - key0 < kChunkKeys;
#pragma unroll
        for (int of = 8; of > 0; of >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, of));
        const float low = top == -INFINITY ? 0.f : top, keep = exp2f(mx[i] - low);
        mx[i] = top;
        float part = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = exp2f(sc[i][j] - low);
          part += p;
          s.p[(4 * ty + i) * S::PLD + tx + 16 * j] = p;
        }
        sum[i] = sum[i] * keep + part;   // this thread's keys; joined at the end
#pragma unroll
        for (int d = 0; d < DN * DW; ++d) o[i][d] *= keep;
      }
      if (S::kShared) {
        __syncthreads();   // the keys are done with
        copy((const float*)a.v, s.v(), tile, page);
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();   // the values are there, the weights too, and the keys are done with
      if (!S::kShared && tile + 1 < last) {
#pragma unroll
        for (int j = 0; j < N; ++j) page[j] = page_next[j];
        pages_of(tile + 2, page_next);
        copy((const float*)a.k, s.k, tile + 1, page);
      }
      // four keys at a time; a key past a row's limit may hold anything: its product is left out,
      // not weighted by 0
      const bool guard = __any_sync(0xffffffffu, masked);
      auto add = [&](auto guarded, int key) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(&s.p[(4 * ty + i) * S::PLD + key]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v[DN * DW];
#pragma unroll
          for (int gd = 0; gd < DN; ++gd) {
            const float* at = &s.v()[(key + e) * S::QLD + (gd * 16 + tx) * DW];
            if constexpr (DW == 4) {
              const float4 f = *reinterpret_cast<const float4*>(at);
              v[4 * gd] = f.x;
              v[4 * gd + 1] = f.y;
              v[4 * gd + 2] = f.z;
              v[4 * gd + 3] = f.w;
            } else {
              const float2 f = *reinterpret_cast<const float2*>(at);
              v[2 * gd] = f.x;
              v[2 * gd + 1] = f.y;
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float pe = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
            if (!decltype(guarded)::value || key0 + key + e < row[i].limit) {
#pragma unroll
              for (int d = 0; d < DN * DW; ++d) o[i][d] = fmaf(pe, v[d], o[i][d]);
            }
          }
        }
      };
      if (guard) {
#pragma unroll 1
        for (int key = 0; key < kChunkKeys; key += 4) add(std::true_type{}, key);
      } else {
#pragma unroll 2
        for (int key = 0; key < kChunkKeys; key += 4) add(std::false_type{}, key);
      }
      __syncthreads();
      if (tile + 1 < last) {
        if (S::kShared) {
#pragma unroll
          for (int j = 0; j < N; ++j) page[j] = page_next[j];
          pages_of(tile + 2, page_next);
          copy((const float*)a.k, s.k, tile + 1, page);
        } else {
          copy((const float*)a.v, s.v(), tile + 1, page);
        }
      }
    }
    const bool whole = first == 0 && last == w.tiles;
    float* part = chunk_part<kRows, HD>(a, blockIdx.x, first > 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int of = 8; of > 0; of >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], of);
      const int R = 4 * ty + i;
      if (row[i].m < 0) continue;
      const int64_t head = row[i].m * a.hq + row[i].head;
      if (whole) {
        const float inv = sum[i] > 0.f || sum[i] != sum[i] ? 1.f / sum[i] : 0.f;
#pragma unroll
        for (int g = 0; g < DN; ++g)
#pragma unroll
          for (int e = 0; e < DW; ++e)
            ((float*)a.o)[head * HD + (g * 16 + tx) * DW + e] = o[i][g * DW + e] * inv;
        if (a.lse && tx == 0) a.lse[head] = (mx[i] + log2f(sum[i])) * 0.6931471805599453f;
      } else {
#pragma unroll
        for (int g = 0; g < DN; ++g)
#pragma unroll
          for (int e = 0; e < DW; ++e)
            part[2 * kRows + (((g * 16 + tx) * DW / 4) * kRows + R) * 4 + (tx * DW + e) % 4] = o[i][g * DW + e];
        if (tx == 0) {
          part[R] = mx[i];
          part[kRows + R] = sum[i];
        }
      }
    }
    if (tid == 0 && first == 0 && !whole) a.join[blockIdx.x] = chunk_join(s.plan, w.k, w.hp, w.t, w.tiles - last);
  }
}

template <int HD> int launch_f32(const Ctx& c, const ChunkArgs& a, int ctas) {
  static std::atomic<uint64_t> done{0};
  auto k = cache_chunk_f32_kernel<HD>;
  if (allow_smem(k, (int)sizeof(Smem<HD>), done) != cudaSuccess) return XMOD_ERR_CUDA;
  XMOD_LAUNCH(c, "cache_chunk",
              launch_pdl(k, dim3(ctas), dim3(kThreads), sizeof(Smem<HD>), c.stream, a));
  return XMOD_OK;
}

}  // namespace

int launch_chunk_f32(const Ctx& c, const ChunkArgs& a, int hd, int ctas) {
  if (hd == 128) return launch_f32<128>(c, a, ctas);
  if (hd == 64) return launch_f32<64>(c, a, ctas);
  return launch_f32<32>(c, a, ctas);
}

}  // namespace xmod
