// Work plan of the dense operators (csa2_chunk_attn, csa2_attn_mass): query
// tiles of one request each, a tile's keys in steps, and the whole list of
// (tile, step) pairs cut into equal ranges, one per CTA.
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
  int min_steps;            // a range is at least this long
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
  const long long v = (static_cast<long long>(p) + 1) / ratio;
  return v < n_ctx ? static_cast<int>(v) : n_ctx;
}

// One query tile: request, first query, tokens, and the entries that any of
// its queries sees.
struct DenseTile {
  int b, q0, tokens, keys;
};

struct DensePlan {
  int tiles;                             // of all requests
  int ctas;                              // CTAs that have work
  long long steps;                       // W
  long long lo, hi;                      // this CTA's range
  int tile;                              // where it starts: tile ...
  int off;                               // ... and step inside it
};

// Shared memory of the plan: tiles before each request, context lengths, and
// the partial sums of the threads.
template <int kThreads>
struct DensePlanSmem {
  int before[kMaxDenseBatch + 1];
  int ctx[kMaxDenseBatch];
  long long warp_sum[kThreads / 32];
  long long total;
  int tile, off;
};

template <int kThreads>
__device__ __forceinline__ DenseTile dense_tile(const DenseArgs& a, const DensePlanSmem<kThreads>& S, int t) {
  int lo = 0, hi = a.cache.batch;        // before[lo] <= t < before[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (S.before[mid] <= t) lo = mid;
    else hi = mid;
  }
  DenseTile d;
  d.b = lo;
  const int j = (t - S.before[lo]) * a.tile_tokens;
  const int first = a.q_start ? a.q_start[lo] : lo, n = a.q_start ? a.q_start[lo + 1] - first : 1;
  d.q0 = first + j;
  d.tokens = min(a.tile_tokens, n - j);
  int keys = 0;
  for (int i = 0; i < d.tokens; ++i) keys = max(keys, seen_by(a.q_pos[d.q0 + i], a.ratio, S.ctx[lo]));
  d.keys = keys;
  return d;
}

template <int kStep>
__device__ __forceinline__ int dense_steps(const DenseTile& t) {
  return max(1, (t.keys + kStep - 1) / kStep);   // a tile that sees nothing still writes its rows
}

// Every thread of the block calls this; S is filled and stays valid.
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
  p.tiles = S.before[a.cache.batch];
  // steps of a consecutive part of the tiles per thread
  const int per = (p.tiles + kThreads - 1) / kThreads;
  const int t0 = min(tid * per, p.tiles), t1 = min(t0 + per, p.tiles);
  long long mine = 0;
  for (int t = t0; t < t1; ++t) mine += dense_steps<kStep>(dense_tile(a, S, t));
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
  p.steps = total;
  const long long most = (total + a.min_steps - 1) / a.min_steps;
  p.ctas = static_cast<int>(most < ctas ? most : ctas);
  if (cta < p.ctas) {
    p.lo = total * cta / p.ctas;
    p.hi = total * (cta + 1) / p.ctas;
  } else {
    p.lo = p.hi = total;
  }
  if (p.lo < p.hi && before <= p.lo && p.lo < before + mine) {
    long long at = before;
    for (int t = t0; t < t1; ++t) {
      const int s = dense_steps<kStep>(dense_tile(a, S, t));
      if (p.lo < at + s) {
        S.tile = t;
        S.off = static_cast<int>(p.lo - at);
        break;
      }
      at += s;
    }
  }
  __syncthreads();
  p.tile = S.tile;
  p.off = S.off;
  return p;
}

// What a CTA says of its range, for the launch that joins split tiles.
struct RangeRecord {
  long long lo;          // first step
  long long tile_lo;     // first step of the tile that it starts in
  long long tile_hi;     // behind that tile's last step
  int q0, tokens;        // that tile's queries
  int ctas;              // CTAs that have work
  int pad;
};

}  // namespace csa2
