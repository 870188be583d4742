// What the kernels of a chunk's attention over the paged cache share: the chunks' shapes, the
// division of the work over the CTAs, and the partial results where a division cuts it.
//
// A segment is up to QR query rows of one chunk and KV head: one block of rows (FFMA) or two of
// 128 (tensor cores), a block `block_tokens` tokens with hpt query heads of the KV head each (row
// r: token r / hpt, head r % hpt), so that a key tile read once serves them all. A segment's key
// tiles are those below its last token's limit. The tiles of all
// segments form one list (order: chunk, KV head and pass of heads, tokens, keys), cut into
// ranges of equal cost, one per CTA: a single long sequence fills the GPU as well as a batch of ragged
// ones, and causal segments of all lengths even out. Where a segment lies in several CTAs'
// ranges each leaves its maximum, sum and unnormalised output in the workspace, and a second
// kernel joins them in CTA order: the result is the same bits at every call.
#pragma once

#include "cache.h"
#include "common.cuh"

namespace xmod {

constexpr int kChunkKeys = 64;        // keys of a tile
constexpr int kChunkMaxCtas = 512;    // CTAs the workspace has room for
constexpr int kChunkTcRows = 256;     // query rows of a segment: tensor cores, one CTA an SM
constexpr int kChunkTcMaxCtas = 192;
constexpr int kChunkF32Rows = 64;     // FFMA, two CTAs an SM

struct Chunk {
  int first, n, len, seq;   // first row, tokens (0: nothing to do), slots, sequence
};

// A segment that starts in a CTA's range and ends in a later one's.
struct ChunkJoin {
  int hp, t, first, last;   // CTAs first .. last hold it; first < 0: none
  Chunk k;
};

struct ChunkArgs {
  int n_chunks, M, hq, hkv, ldq;
  const void* q;
  const int32_t *start, *seq, *len;
  void* o;
  float* lse;
  const int32_t* table;
  const void *k, *v;
  const float *k_scale, *v_scale;
  int n_pages, page_size, n_seqs, max_pages;
  int group;              // query heads of a KV head
  int hpt, tpt, passes;   // heads and tokens of a segment, passes over a KV head's query heads
  int block_tokens;       // tokens of a block of rows
  int lead;               // what a segment costs beside its tiles, in tiles: tensor cores 4 (six prompts 993 us,
                          // with 0 1291), FFMA 1 (six of 100 at 1000 34.6 us, with 0 39.2, with 2 41.0;
                          // six prompts of up to 2048, 16 and 4 heads of 64: 662, 745, 688)
  int hpt_inverse;        // ceil(2^16 / hpt): r / hpt for r, hpt <= 256 (their product is below 2^16)
  int page_shift;         // log2 of the page size, -1: not a power of two
  int box;                // rows of a TMA box: divides the page size and a tile
  float* part;            // partial results, two per CTA
  ChunkJoin* join;        // what each CTA leaves to be joined
  int* status;
};

static __device__ __noinline__ Chunk read_chunk(const ChunkArgs& a, int c) {
  Chunk k;
  k.first = a.start[c];
  const int end = a.start[c + 1];
  k.seq = a.seq ? a.seq[c] : c;
  k.len = 0;
  k.n = 0;
  if (k.seq < 0) return k;
  if (k.seq >= a.n_seqs || k.first < 0 || end < k.first || end > a.M) {
    report_status(a.status, XMOD_ERR_DEVICE_CHECK);
    return k;
  }
  k.n = end - k.first;
  if (k.n == 0) return k;
  const int n = a.len[c], most = a.max_pages * a.page_size;
  if (n < 0 || n > most) report_status(a.status, XMOD_ERR_DEVICE_CHECK);
  k.len = min(max(n, 0), most);
  return k;
}

__device__ __forceinline__ int chunk_segments(const ChunkArgs& a, const Chunk& k) {
  return (k.n + a.tpt - 1) / a.tpt;
}
// Slots that the last token of segment t attends to (may be 0 or less).
__device__ __forceinline__ int segment_limit(const ChunkArgs& a, const Chunk& k, int t) {
  const int64_t end = min((int64_t)k.n, (int64_t)(t + 1) * a.tpt);
  return (int)(k.len - k.n + end);
}
// A segment without keys counts as one tile: its zeros have to be written.
__device__ __forceinline__ int segment_tiles(int limit) {
  return limit <= 0 ? 1 : (limit - 1) / kChunkKeys + 1;
}

// Tiles of the first t segments of a chunk, in closed form. Segment i has ceil((b + (i + 1) tpt)
// / 64) tiles with b = len - n, at least one, the last one ceil(len / 64).
// Small code (a loop, not inlined): what a kernel runs once costs mostly its fetching.
static __device__ __noinline__ long long tiles_before(int tpt, int tokens, int slots, int segments, int t) {
  long long sum = 0;
  if (t == segments && t > 0) {
    sum += segment_tiles(slots);
    --t;
  }
  const int b = slots - tokens;   // below 2^31 in size both
  const int empty = b < 0 ? min(t, -b / tpt) : 0;
  sum += empty;
  const int n = t - empty;
  if (n <= 0) return sum;
  // sum over j < n of floor((tpt j + c) / 64)
  const long long c = (long long)b + kChunkKeys - 1 + (long long)tpt * (empty + 1);
  const int qa = tpt / kChunkKeys, ra = tpt % kChunkKeys;
  const long long qc = c / kChunkKeys;
  const int rc = (int)(c % kChunkKeys);
  sum += (long long)qa * ((long long)n * (n - 1) / 2) + qc * n;
  if (ra == 0) return sum;
  if (kChunkKeys % ra == 0) {
    // j = p u + v, p = 64 / ra: floor((ra j + rc) / 64) = u, and one more from v = z on
    const int p = kChunkKeys / ra, z = (kChunkKeys - rc + ra - 1) / ra;
    const long long u = n / p;
    const int w = n % p;
    return sum + p * (u * (u - 1) / 2) + u * w + u * max(0, p - z) + max(0, w - z);
  }
  // j = 64 u + v: floor((ra j + rc) / 64) = ra u + floor((ra v + rc) / 64)
  const long long u = n / kChunkKeys;
  const int w = n % kChunkKeys;
  int whole = 0, part = 0;
#pragma unroll 4
  for (int v = 0; v < kChunkKeys; ++v) {
    const int f = (ra * v + rc) / kChunkKeys;
    whole += f;
    part += v < w ? f : 0;
  }
  return sum + ra * (kChunkKeys * (u * (u - 1) / 2) + u * w) + u * whole + part;
}

// x / y for 0 <= x, 0 < y: in 32 bits where they fit (a division in 64 is long).
static __device__ __noinline__ long long divide(long long x, long long y) {
  if (((x | y) >> 32) == 0) return (uint32_t)x / (uint32_t)y;
  return x / y;
}

// The list's cut: positions are tiles, with `lead` more before each segment's own, so that ranges
// of equal length take equal time. CTA g's range is each * g + min(g, more) .. .
struct ChunkPlan {
  long long begin, end;       // this CTA's range
  long long each, tiles;      // of a CTA; of a KV head and pass of the chunk it begins in
  long long off;
  long long found_cost;
  int found;                  // the last segment known to begin at or before the range, and the cost before it
  Chunk k;
  int more, chunk, hp, t, at;   // where the range begins: chunk, KV head and pass, segment, position in it
};

__device__ __forceinline__ int chunk_cta_of(const ChunkPlan& p, long long position) {
  const long long big = (p.each + 1) * p.more;   // positions of the CTAs with one more
  return (int)(position < big ? divide(position, p.each + 1) : p.more + divide(position - big, p.each));
}

// Cost of the first t segments.
__device__ __forceinline__ long long cost_before(const ChunkArgs& a, const Chunk& k, int segments, int t) {
  return tiles_before(a.tpt, k.n, k.len, segments, t) + (long long)a.lead * t;
}

// All threads of the CTA; scratch: one int64 per warp.
__device__ __forceinline__ void make_chunk_plan(const ChunkArgs& a, ChunkPlan* plan, long long* scratch) {
  const int least = a.lead + 1;   // of a range: a segment of one tile is not cut
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthreads = blockDim.x;
  const int per = (a.n_chunks + nthreads - 1) / nthreads;
  const int c0 = min(a.n_chunks, tid * per), c1 = min(a.n_chunks, c0 + per);
  const int P = a.hkv * a.passes;
  long long mine = 0, each = 0;
  Chunk k;
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    k = read_chunk(a, c);
    const int segments = chunk_segments(a, k);
    each = cost_before(a, k, segments, segments);
    mine += P * each;
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll 1
  for (int w = 0; w < nthreads / 32; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  const int ctas = total < (long long)least * gridDim.x ? ((int)total + least - 1) / least : (int)gridDim.x;
  const int g = blockIdx.x;
  const long long length = ctas > 0 ? divide(total, ctas) : 0;
  const int more = (int)(total - length * ctas);
  const long long begin = g < ctas ? length * g + min(g, more) : total;
  const long long end = g < ctas ? begin + length + (g < more ? 1 : 0) : total;
  if (tid == 0) {
    plan->begin = begin;
    plan->end = end;
    plan->each = length;
    plan->more = more;
    plan->found = 0;
    plan->found_cost = 0;
  }
  if (begin < end && begin >= before && begin < before + mine) {
    long long at = before;
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      if (per > 1) {
        k = read_chunk(a, c);
        const int segments = chunk_segments(a, k);
        each = cost_before(a, k, segments, segments);
      }
      if (begin < at + P * each) {
        plan->chunk = c;
        plan->off = begin - at;
        plan->tiles = each;
        plan->k = k;
        break;
      }
      at += P * each;
    }
  }
  __syncthreads();
  if (begin >= end) return;
  // the segment: the last one that begins at or before rem, by as many guesses at once as threads
  k = plan->k;
  const int segments = chunk_segments(a, k);
  const long long off = plan->off;
  each = plan->tiles;
  const int hp = (int)divide(off, each);
  const long long rem = off - hp * each;
  int lo = 0, hi = segments;   // within lo .. hi - 1
#pragma unroll 1
  while (hi - lo > 1) {
    const int step = (hi - lo - 1) / nthreads + 1;
    const long long t = lo + (long long)tid * step;
    long long n = 0;
    if (t < hi) {
      n = cost_before(a, k, segments, (int)t);
      if (n <= rem) atomicMax(&plan->found, (int)t);
    }
    __syncthreads();
    lo = plan->found;
    if (t == lo) plan->found_cost = n;
    hi = min(hi, lo + step);
    __syncthreads();
  }
  if (tid == 0) {
    plan->t = lo;
    plan->hp = hp;
    plan->at = (int)(rem - plan->found_cost);
  }
  __syncthreads();
}

// A CTA's way along its range, segment by segment.
struct ChunkWalk {
  Chunk k;
  long long left;                                   // positions of the range not yet taken
  int chunk, segments, hp, t, at, tiles, limit;     // at: position in the segment
  int first, last;                                  // the segment's tiles in this CTA's range

  __device__ __forceinline__ void begin(const ChunkArgs& a, const ChunkPlan& p) {
    chunk = p.chunk;
    k = p.k;
    segments = chunk_segments(a, k);
    hp = p.hp;
    t = p.t;
    at = p.at;
    left = p.end - p.begin;
  }
  // The next segment that has tiles in the range; false: none is left.
  __device__ __forceinline__ bool next(const ChunkArgs& a) {
    while (left > 0) {
      if (at < 0) {   // the segment before is done
        at = 0;
        if (++t == segments) {
          t = 0;
          if (++hp == a.hkv * a.passes) {
            hp = 0;
            do {
              if (++chunk >= a.n_chunks) return false;   // the list ends here
              k = read_chunk(a, chunk);
            } while (k.n == 0);
            segments = chunk_segments(a, k);
          }
        }
      }
      limit = segment_limit(a, k, t);
      tiles = segment_tiles(limit);
      const int end = (int)min((long long)(tiles + a.lead), at + left);
      left -= end - at;
      first = max(0, at - a.lead);
      last = max(0, end - a.lead);
      at = -1;
      if (last > first) return true;
    }
    return false;
  }
};

// KV head and first query head of a KV head and pass.
__device__ __forceinline__ int chunk_kv_head(const ChunkArgs& a, int hp) { return a.passes == 1 ? hp : hp / a.passes; }
__device__ __forceinline__ int chunk_first_head(const ChunkArgs& a, int hp) {
  return a.passes == 1 ? hp * a.group : hp / a.passes * a.group + hp % a.passes * a.hpt;
}

// Row r of block x of a segment: its row of q and o (-1: none), its head and its limit.
struct ChunkRow {
  int64_t m;
  int head, limit;
};
__device__ __forceinline__ ChunkRow chunk_row(const ChunkArgs& a, const Chunk& k, int hp, int t, int x, int r) {
  ChunkRow row;
  const int in = (r * a.hpt_inverse) >> 16, h = r - in * a.hpt;
  const int token = t * a.tpt + x * a.block_tokens + in;
  row.m = -1;
  row.limit = 0;
  row.head = chunk_first_head(a, hp) + h;
  if (in >= a.block_tokens || token >= k.n || (a.passes > 1 && hp % a.passes * a.hpt + h >= a.group)) return row;
  row.m = k.first + token;
  row.limit = max(0, k.len - k.n + 1 + token);
  return row;
}

// A slot's place in the table and in its page.
__device__ __forceinline__ int chunk_page(const ChunkArgs& a, const Chunk& k, int slot) {
  return a.table[(int64_t)k.seq * a.max_pages + (a.page_shift >= 0 ? slot >> a.page_shift : slot / a.page_size)];
}
__device__ __forceinline__ int chunk_in_page(const ChunkArgs& a, int slot) {
  return a.page_shift >= 0 ? slot & (a.page_size - 1) : slot % a.page_size;
}

// Where a segment's part in this CTA's range goes: slot 0 if it began before the range, 1 if it
// begins here and goes on after it. A part is [QR] maxima (log2 units), [QR] sums and the outputs
// as [HD / 4][QR][4], which both the writers' and the join's threads, a row each, touch in whole
// lines.
template <int QR, int HD>
__device__ __forceinline__ float* chunk_part(const ChunkArgs& a, int cta, bool began_before) {
  return a.part + ((int64_t)2 * cta + (began_before ? 0 : 1)) * QR * (HD + 2);
}

// The join of a segment whose first tiles, but not all, are this CTA's, the range's last: it ends
// `left` tiles on.
__device__ __forceinline__ ChunkJoin chunk_join(const ChunkPlan& p, const Chunk& k, int hp, int t, int left) {
  ChunkJoin j;
  j.hp = hp;
  j.t = t;
  j.first = blockIdx.x;
  j.last = chunk_cta_of(p, p.end + left - 1);
  j.k = k;
  return j;
}

// Launchers of the two kernels (cache_chunk_f32.cu, cache_chunk_tc.cu); ctas as planned.
struct Ctx;
int launch_chunk_f32(const Ctx& c, const ChunkArgs& a, int hd, int ctas);
int launch_chunk_tc(const Ctx& c, const ChunkArgs& a, int hd, bool fp8, int ctas);

}  // namespace xmod
