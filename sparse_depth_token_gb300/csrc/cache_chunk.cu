// Attention of a chunk of new tokens over the paged cache: the entry point, and the join of
// segments that several CTAs worked on.

#include <math.h>

#include "cache_chunk.cuh"

namespace xmod {

namespace {

// Segment of CTA blockIdx.x that later CTAs' ranges continue, 32 rows a block: a lane has a row,
// a warp every eighth group of four dimensions; the parts' outputs are weighted to the running
// maximum, in CTA order, several parts on their way at a time. Latency: the record, the parts, the
// stores (13 us with one part at a time and the maxima before, now 7 for eight chunks of four tokens).
constexpr int kJoinWarps = 8;

template <typename T, int HD, int QR>
__global__ void __launch_bounds__(kJoinWarps * 32) cache_chunk_join_kernel(const ChunkArgs a) {
  constexpr int G = HD / 4, E = G / kJoinWarps, AHEAD = E >= 4 ? 4 : 8;
  pdl_trigger();
  pdl_wait();
  const ChunkJoin j = a.join[blockIdx.x];
  if (j.first < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, R = blockIdx.y * 32 + lane;
  constexpr int BLOCK = QR < 128 ? QR : 128;
  const ChunkRow row = chunk_row(a, j.k, j.hp, j.t, R / BLOCK, R % BLOCK);
  if (row.m < 0) return;
  float top = -INFINITY, sum = 0.f;
  float4 o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int p0 = j.first; p0 <= j.last; p0 += AHEAD) {
    float m[AHEAD], l[AHEAD];
    float4 v[AHEAD][E];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int p = min(p0 + i, j.last);
      const float* part = chunk_part<QR, HD>(a, p, p > j.first);
      m[i] = part[R];
      l[i] = part[QR + R];
#pragma unroll
      for (int e = 0; e < E; ++e)
        v[i][e] = *reinterpret_cast<const float4*>(part + 2 * QR + ((e * kJoinWarps + warp) * QR + R) * 4);
    }
    float now = top;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) now = fmaxf(now, m[i]);   // the last part again, perhaps
    const float low = now == -INFINITY ? 0.f : now, keep = exp2f(top - low);
    top = now;
    sum *= keep;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = make_float4(o[e].x * keep, o[e].y * keep, o[e].z * keep, o[e].w * keep);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (p0 + i > j.last) break;
      const float f = exp2f(m[i] - low);
      sum = fmaf(l[i], f, sum);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        o[e].x = fmaf(v[i][e].x, f, o[e].x);
        o[e].y = fmaf(v[i][e].y, f, o[e].y);
        o[e].z = fmaf(v[i][e].z, f, o[e].z);
        o[e].w = fmaf(v[i][e].w, f, o[e].w);
      }
    }
  }
  const int64_t head = row.m * a.hq + row.head;
  const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    T* dst = (T*)a.o + head * HD + (e * kJoinWarps + warp) * 4;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(dst) = make_float4(o[e].x * inv, o[e].y * inv, o[e].z * inv, o[e].w * inv);
    } else {
      uint4 w;
      set_vec_pair<T>(w, 0, make_float2(o[e].x * inv, o[e].y * inv));
      set_vec_pair<T>(w, 1, make_float2(o[e].z * inv, o[e].w * inv));
      *reinterpret_cast<uint2*>(dst) = make_uint2(w.x, w.y);
    }
  }
  if (a.lse && warp == 0) a.lse[head] = (top + log2f(sum)) * 0.6931471805599453f;
}

template <typename T, int QR> int launch_join(const Ctx& c, const ChunkArgs& a, int hd, int ctas) {
  const dim3 grid(ctas, QR / 32), block(kJoinWarps * 32);
  if (hd == 128)
    XMOD_LAUNCH(c, "cache_chunk_join", launch_pdl(cache_chunk_join_kernel<T, 128, QR>, grid, block, 0, c.stream, a));
  else if (hd == 64)
    XMOD_LAUNCH(c, "cache_chunk_join", launch_pdl(cache_chunk_join_kernel<T, 64, QR>, grid, block, 0, c.stream, a));
  else
    XMOD_LAUNCH(c, "cache_chunk_join", launch_pdl(cache_chunk_join_kernel<T, 32, QR>, grid, block, 0, c.stream, a));
  return XMOD_OK;
}

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

size_t chunk_workspace(const xmod_dims* dm) {
  const bool fp32 = dm->dtype == XMOD_FP32;
  const size_t part = (size_t)(fp32 ? kChunkF32Rows : kChunkTcRows) * (dm->head_dim + 2) * 4;
  return 256 + round256(kChunkMaxCtas * sizeof(ChunkJoin)) +
         2 * (size_t)(fp32 ? kChunkMaxCtas : kChunkTcMaxCtas) * part;
}

}  // namespace
}  // namespace xmod

using namespace xmod;

extern "C" {

size_t xmod_cache_attention_chunk_workspace_bytes(const xmod_dims* dm, int n_chunks, int M) {
  if (!dims_ok(dm) || n_chunks < 0 || M < 0 || !head_dim_supported(dm->head_dim)) return 0;
  return chunk_workspace(dm);
}

int xmod_cache_attention_chunk(const xmod_dims* dm, const xmod_kv_cache* cache, int n_chunks, int M,
                               const void* q, int ldq, const int32_t* start, const int32_t* seq,
                               const int32_t* len, void* o, float* lse, void* ws, size_t ws_bytes,
                               void* stream) {
  const int st = cache_status(dm, cache);
  if (st) return st;
  if (n_chunks < 0 || M < 0) return XMOD_ERR_INVALID_ARG;
  if (M > XMOD_MAX_CHUNK_ROWS) return XMOD_ERR_UNSUPPORTED;
  if (n_chunks == 0 || M == 0) return XMOD_OK;
  const int qw = dm->n_heads * dm->head_dim;
  if (!ptr16(q) || ldq < qw || ldq % 8 || !start || !ptr4_or_null(start) || !ptr4_or_null(seq) || !len ||
      !ptr4_or_null(len) || !ptr16(o) || o == q || !ptr4_or_null(lse))
    return XMOD_ERR_INVALID_ARG;
  if (!ptr16(ws) || ws_bytes < chunk_workspace(dm)) return XMOD_ERR_WORKSPACE;
  const bool fp32 = dm->dtype == XMOD_FP32, fp8 = cache->format == XMOD_CACHE_E4M3;
  if (!fp32 && !tma_available()) return XMOD_ERR_UNSUPPORTED;
  const int sms = device_sms();
  if (sms <= 0) return XMOD_ERR_CUDA;
  const int want = fp32 ? 2 * sms : sms, most = fp32 ? kChunkMaxCtas : kChunkTcMaxCtas;
  const int ctas = want < most ? want : most, rows = fp32 ? kChunkF32Rows : kChunkTcRows;
  const int group = dm->n_heads / dm->n_kv_heads;
  ChunkArgs a{};
  a.n_chunks = n_chunks;
  a.M = M;
  a.hq = dm->n_heads;
  a.hkv = dm->n_kv_heads;
  a.ldq = ldq;
  a.q = q;
  a.start = start;
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
  const int block = fp32 ? kChunkF32Rows : 128;
  a.group = group;
  a.hpt = group < block ? group : block;
  a.block_tokens = block / a.hpt;
  a.tpt = rows / block * a.block_tokens;
  a.passes = (group + a.hpt - 1) / a.hpt;
  a.lead = fp32 ? 1 : 4;
  a.hpt_inverse = (65536 + a.hpt - 1) / a.hpt;
  a.page_shift = -1;
  for (int i = 4; i < 31; ++i)
    if (cache->page_size == 1 << i) a.page_shift = i;
  a.box = cache->page_size % 64 == 0 ? 64 : cache->page_size % 32 == 0 ? 32 : 16;
  a.join = (ChunkJoin*)((char*)ws + 256);
  a.part = (float*)((char*)ws + 256 + round256(kChunkMaxCtas * sizeof(ChunkJoin)));
  a.status = (int*)ws;
  const Ctx c{(cudaStream_t)stream, a.status};
  if (fp32) {
    const int r = launch_chunk_f32(c, a, dm->head_dim, ctas);
    return r ? r : launch_join<float, kChunkF32Rows>(c, a, dm->head_dim, ctas);
  }
  const int r = launch_chunk_tc(c, a, dm->head_dim, fp8, ctas);
  return r ? r : launch_join<__nv_bfloat16, kChunkTcRows>(c, a, dm->head_dim, ctas);
}

}  // extern "C"
