// Work plan of csa2_chunk_attn (and what csa2_attn_mass shares of it): query
// tiles of one request each, a tile's keys in steps, and the whole list of
// (tile, step) pairs cut into equal ranges, one per CTA (or pair of CTAs).
//
// Lengths live on the device, so every CTA derives the same plan from them at
// its start: tiles per request, steps per tile (the keys that the tile's most
// seeing query sees), their total W, and its own range [W c / G, W (c+1) / G).
// A tile that crosses a range's end is split over CTAs along its keys; the
// partial results are joined afterwards.  The cut depends on sizes alone, so
// results do not change from run to run.
#pragma once

#include "common.cuh"

namespace csa2 {

struct DenseArgs {
  csa2_cache cache;
  const int32_t* q_start;   // [batch + 1] queries of each request, or NULL (query i -> request i)
  const int32_t* q_pos;     // [n_queries]
  int n_queries;
  int ratio;                // tokens per entry
  int heads;
  int tile_tokens;          // tokens per query tile
};

constexpr int kMaxDenseBatch = 1024;

// Queries of request b; a range outside [0, n_queries] (or a decreasing one)
// is recorded and the request has none.
__device__ __forceinline__ int queries_of(const DenseArgs& a, int b, int kernel, bool report) {
  if (a.q_start == nullptr) return b < a.n_queries ? 1 : 0;
  const int lo = a.q_start[b], hi = a.q_start[b + 1];
  if (lo < 0 || hi < lo || hi > a.n_queries) {
    if (report) report_error(a.cache.err_word, CSA2_ERR_DEVICE_BOUNDS, kernel, b, hi);
    return 0;
  }
  return hi - lo;
}

// Entries that the query at token position p sees, of n_ctx.
__device__ __forceinline__ int seen_by(int p, int ratio, int n_ctx) {
  if (p < 0) return 0;
  const uint32_t v = (static_cast<uint32_t>(p) + 1u) / static_cast<uint32_t>(ratio);
  return v < static_cast<uint32_t>(n_ctx) ? static_cast<int>(v) : n_ctx;
}

// One query tile: request, first query, tokens, the request's visible length,
// and the entries that any of the tile's queries sees.
struct DenseTile {
  int b, q0, tokens, ctx, keys;
};
// A tile's place: request, and tile inside the request.
struct TilePlace {
  int b, j;
};

struct DensePlan {
  int ctas;                              // CTAs that have work
  long long lo, hi;                      // this CTA's range
  TilePlace start;                       // where it starts: tile ...
  int off;                               // ... and step inside it
};

// Shared memory of the plan (free again once dense_plan has returned and the
// block has synchronised): tiles before each request, context lengths, and
// the threads' partial sums.
template <int kThreads>
struct DensePlanSmem {
  int before[kMaxDenseBatch + 1];
  int ctx[kMaxDenseBatch];
  long long warp_sum[kThreads / 32];
  TilePlace start;
  int off;
};

__device__ __forceinline__ DenseTile dense_tile(const DenseArgs& a, TilePlace p, int n, int ctx) {
  DenseTile d;
  d.b = p.b;
  const int j = p.j * a.tile_tokens;
  d.q0 = (a.q_start ? a.q_start[p.b] : p.b) + j;
  d.tokens = min(a.tile_tokens, n - j);
  d.ctx = ctx;
  int last = -1;                         // the largest position sees the most
#pragma unroll 8
  for (int i = 0; i < d.tokens; ++i) last = max(last, a.q_pos[d.q0 + i]);
  d.keys = seen_by(last, a.ratio, ctx);
  return d;
}
__device__ __forceinline__ DenseTile dense_tile(const DenseArgs& a, TilePlace p) {
  const long long capacity = static_cast<long long>(a.cache.max_pages_per_req) * a.cache.page_size;
  return dense_tile(a, p, queries_of(a, p.b, 0, false), max(0, checked_ctx_len(a.cache, p.b, capacity, 0, false)));
}
// The place after p: the request's next tile, or the first of the next request
// that has queries (there is one while a range is not done).
__device__ __forceinline__ TilePlace next_tile(const DenseArgs& a, TilePlace p) {
  if ((p.j + 1) * a.tile_tokens < queries_of(a, p.b, 0, false)) return TilePlace{p.b, p.j + 1};
  int b = p.b + 1;
  while (b < a.cache.batch && queries_of(a, b, 0, false) == 0) ++b;
  return TilePlace{b, 0};
}

template <int kStep>
__device__ __forceinline__ int dense_steps(const DenseTile& t) {
  return max(1, (t.keys + kStep - 1) / kStep);   // a tile that sees nothing still writes its rows
}

// Starting and ending a tile (queries, first products, output rows) costs about
// as much as three of its steps, so the plan counts kTileCost steps more for
// each, before its own.  A ragged batch (6 requests, up to 333 new tokens x 32
// heads over up to 7,001 entries) by its value, 0 to 4: 419, 314, 257, 245, 247
// us; long prompts and equal requests hardly depend on it.
constexpr int kTileCost = 3;
// The part [first, first + n) of a tile's own steps that lies in a range which
// starts `off` counted steps into the tile and has `left` left; n may be 0.
struct TilePart {
  int counted;                           // of the range's steps
  int first, n;
};
__device__ __forceinline__ TilePart tile_part(int steps, int off, long long left) {
  TilePart t;
  t.counted = static_cast<int>(min(static_cast<long long>(steps + kTileCost - off), left));
  t.first = max(0, off - kTileCost);
  t.n = max(0, off + t.counted - kTileCost - t.first);
  return t;
}

// Every thread of the block calls this.
template <int kThreads, int kStep>
__device__ __forceinline__ DensePlan dense_plan(const DenseArgs& a, DensePlanSmem<kThreads>& S, int cta, int ctas,
                                                int kernel) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long capacity = static_cast<long long>(a.cache.max_pages_per_req) * a.cache.page_size;
  for (int b = tid; b < a.cache.batch; b += kThreads) {
    const int n = queries_of(a, b, kernel, cta == 0);
    S.before[b + 1] = (n + a.tile_tokens - 1) / a.tile_tokens;
    S.ctx[b] = n > 0 ? max(0, checked_ctx_len(a.cache, b, capacity, kernel, cta == 0)) : 0;
  }
  __syncthreads();
  if (warp == 0) {                       // tiles before each request
    int run = 0;
    for (int b0 = 0; b0 < a.cache.batch; b0 += 32) {
      const int b = b0 + lane;
      int v = b < a.cache.batch ? S.before[b + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (b < a.cache.batch) S.before[b + 1] = run + v;
      run += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) S.before[0] = 0;
  }
  __syncthreads();
  DensePlan p;
  // steps of a consecutive part of the tiles per thread
  const int tiles = S.before[a.cache.batch];
  const int per = (tiles + kThreads - 1) / kThreads;
  const int t0 = min(tid * per, tiles), t1 = min(t0 + per, tiles);
  auto place_of = [&](int t) {
    int lo = 0, hi = a.cache.batch;      // before[lo] <= t < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (S.before[mid] <= t) lo = mid;
      else hi = mid;
    }
    return TilePlace{lo, t - S.before[lo]};
  };
  auto steps_of = [&](TilePlace at) {
    const int n = a.q_start ? a.q_start[at.b + 1] - a.q_start[at.b] : 1;
    return dense_steps<kStep>(dense_tile(a, at, n, S.ctx[at.b])) + kTileCost;
  };
  long long mine = 0;
  for (int t = t0; t < t1; ++t) mine += steps_of(place_of(t));
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) S.warp_sum[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += S.warp_sum[w];
    total += S.warp_sum[w];
  }
  p.ctas = static_cast<int>(total < ctas ? total : ctas);
  if (cta < p.ctas) {
    p.lo = total * cta / p.ctas;
    p.hi = total * (cta + 1) / p.ctas;
  } else {
    p.lo = p.hi = total;
  }
  if (p.lo < p.hi && before <= p.lo && p.lo < before + mine) {
    long long at = before;
    for (int t = t0; t < t1; ++t) {
      const TilePlace place = place_of(t);
      const int s = steps_of(place);
      if (p.lo < at + s) {
        S.start = place;
        S.off = static_cast<int>(p.lo - at);
        break;
      }
      at += s;
    }
  }
  __syncthreads();
  p.start = S.start;
  p.off = S.off;
  return p;
}

}  // namespace csa2
