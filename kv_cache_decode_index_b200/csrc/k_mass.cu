// Attention weight that every cached entry received from the queries of a
// call: mass[b][e] += sum over request b's queries and heads of
// exp(scale q . v_e - lse), with the rows' log-sum-exp given.
//
// A matrix product with a sum over its columns: S^T = V Q^T on tcgen05 over a
// pair of CTAs, M = 256 entries (128 per CTA), N = up to 256 query rows (half
// per CTA), K = 512.  Entries lie in the lanes of tensor memory, so a thread
// sums its entry's weights over the columns by itself.
//   * The query rows of a tile stay in shared memory (128 KB), fp16; the entries
//     stream past them: eight warps dequantise 128 entries per CTA and tile
//     into a ring of two 32 KB pairs of slots.  Entries are 288 bytes each where
//     a query row is 1 KB, so this is the side to stream; for single tokens it
//     is the only one that is long.
//   * With few rows a request the tile is 64 rows (32 per CTA, 32 KB), and packed
//     entries come by bulk copies, two tiles ahead in shared memory: loads into
//     registers kept 36 KB an SM under way, too few for entries from HBM.
//   * The rows' log-sum-exp is taken off by the product itself: one more step of
//     K holds ones for the entries and -lse, in three fp16 parts, for the rows.  It
//     comes last, where the sum is small.  So the epilogue needs nothing per
//     column but a product, exp2 and a sum: factors of each column from shared
//     memory (which the operands keep busy) had it at 52 cycles a column.
//   * One warp of the leader issues the MMAs into two 256-column accumulators;
//     four warps (a lane quarter each) take exp2 and the sums.
// Why a pair: shared memory gives 128 bytes a cycle.  One CTA alone would read
// 128 (operands of M = N = 128) and write 64 (rows); the pair reads 64 and
// writes 32 for each of its CTAs at the full MMA rate.
//
// The work is cut into equal ranges of (row tile, 256 entries) steps, ordered by
// request, part of 8,192 entries, row tile, tile of entries: a pair holds a
// part's sums in shared memory over all row tiles.  Parts that ranges cut are
// joined in a fixed order by a second launch.
//
// 512 tokens x 64 heads of two requests over 16,381 entries (two tokens an entry):
// 0.95 ms for a call by itself, 0.69 of the tensor cores' measured rate, and 1.02 to
// 1.03 ms in calls back to back (0.64), where the power limit lowers the clock; 8
// single tokens x 64 heads over 65,536: 92 us.  What bounds it is the
// dequantisation of a tile's 128 entries a CTA: 5,000 to 7,000 cycles against 4,096
// of products in tiles of 256 rows, 4,700 against 1,500 in tiles of 64.
#include <cuda_bf16.h>

#include "launch.h"
#include "pair_operands.cuh"

namespace csa2 {

namespace {

constexpr int kMEpiWarps = 4, kMDeqWarps = 8, kMMmaWarp = kMEpiWarps + kMDeqWarps;
constexpr int kMThreads = (kMMmaWarp + 1) * 32;   // 416
constexpr int kMKeys = 256;                       // entries of a tile (both CTAs)
constexpr int kMPart = 32;                        // tiles of entries whose sums a pair holds
constexpr int kMSlot = 128 * 128;                 // 128 rows x 64 channels
constexpr int kMStage = 128 * (kKvCodeBytes + kKvScaleBytes);   // 128 packed entries
constexpr int kMAcc = 2;
constexpr int kMaxPairs = 74;                     // ranges of one launch: pairs of CTAs on 148 SMs
constexpr int kBarEpi = 1, kBarDeq = 2;

// Queries are scaled by 2^6 in fp16 while every magnitude of a row tile is below
// 2^9, every log-sum-exp fits and the unit of an accumulator is between 0.01 and 8
// log2 units (scales of 0.002 to 1.4); other tiles ("wide") scale each row by
// itself and take factors and log-sum-exp per column.  Why 8: below fp16's normal
// range a query channel is off by up to 2^-31, which a larger scale, made for
// small queries, would carry into the scores.  Up to it the error of a score is
// below 512 x 2^-31 x 1.4 of the entry's largest channel (1.4 x 2^-22 of it).
constexpr int kMExponent = 8;
constexpr float kMUndo = kRowScale / 64.0f;       // of 2^6 and of the entries' 2^-8
constexpr float kMLargest = 60000.0f;
constexpr float kMUnitLow = 0.01f, kMUnitHigh = 8.0f;

// kMRows: query rows of a tile (both CTAs); kMRing: pairs of slots of entries.
template <int kMRows, int kMRing, int kMStages>
struct __align__(1024) MassSmem {
  uint8_t q[kKvDim / 64][kMRows / 2 * 128];       // B: this CTA's half of the rows, 64 channels a part
  union {
    uint8_t ring[kMRing][2 * kMSlot];             // A: 128 entries, 128 channels a pair
    long long at[kMaxDenseBatch + 1];             // plan, before the first pair is filled: steps before each request
  };
  uint8_t a_ones[128 * 32];                       // the last step of K: A ...
  uint8_t b_lse[128 * 32];                        // ... and B
  uint8_t stage[kMStages * kMStage + 16];         // packed entries on their way: codes, then scales
  float col_scale[2][kMRows];                     // per column: factor of the scores (by turns: the
                                                  // other CTA fills its half of the next one) ...
  float col_lse2[kMRows];                         // ... log2 of the row's sum ...
  int col_lim[kMRows];                            // ... and entries that it sees (0: no row)
  float sum[kMPart * kMKeys / 2];                 // this CTA's entries of the part
  int warp_min[kMEpiWarps];
  float wide[2];                                  // by turns: some row of either CTA needs the wide form
  uint64_t full[kMRing];                          // leader: both CTAs' dequantisation
  uint64_t empty[kMRing];
  uint64_t acc_full[kMAcc];
  uint64_t acc_empty[kMAcc];                      // leader
  uint64_t q_full;                                // leader
  uint64_t scale_full[2];                         // what the other CTA says of its rows has arrived (by turns)
  uint64_t drain;
  uint64_t stage_full[kMStages + 1];
  int stage_row[kMStages + 1];                    // a stage's cache row, -1: not there, -2: no tile
  uint32_t tmem_base;
  int start_b;                                    // the request of the first step, and the steps before it
  long long start_at;
};

// What a pair says of its range, for the joining launch.
struct MassRecord {
  long long lo, part_lo, part_hi;   // first step; first and past-the-last step of the part it starts in
  int b, k0;                        // that part
  int pairs, pad;
};
struct MassWorkspace {
  MassRecord* rec;
  float* part;    // [pairs][2][kMPart * kMKeys]
};
__host__ __device__ inline MassWorkspace split_mass_ws(void* ws) {
  MassWorkspace w;
  w.rec = static_cast<MassRecord*>(ws);
  w.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kMaxPairs * sizeof(MassRecord));
  return w;
}

// A run of steps with one row tile: entries' tiles [kt0, kt1) of the part that
// starts at tile `part` of request b.
struct Run {
  int b, ctx, q0, rows;             // rows: of the whole request
  int part, rt, kt0, kt1;
  long long part_lo, part_hi;       // steps of the whole part
};

template <int kMRows, int kMRing, int kMStages>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMThreads, 1)
    attn_mass_kernel(const DenseArgs a, const __nv_bfloat16* __restrict__ q, float scale, const float* __restrict__ lse,
                     float* __restrict__ mass, void* ws, uint64_t wait_ns) {
  extern __shared__ uint8_t smem_raw[];
  using Smem = MassSmem<kMRows, kMRing, kMStages>;
  static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "shared memory of one CTA");
  constexpr uint32_t kMTmemCols = kMAcc * kMRows;
  constexpr int kMQPart = kMRows / 2 * 128;       // bytes of 64 channels of the rows
  Smem& S = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const csa2_cache& cache = a.cache;
  const MassWorkspace wsp = split_mass_ws(ws);
  const long long capacity = static_cast<long long>(cache.max_pages_per_req) * cache.page_size;

  pdl_launch_dependents();     // the joining launch: it waits for this one's end

  // ---- plan: steps of each request = its tiles of entries x its row tiles ----
  for (int b = tid; b < cache.batch; b += kMThreads) {
    const int n = queries_of(a, b, kKMass, blockIdx.x == 0);
    const int ctx = n > 0 ? max(0, checked_ctx_len(cache, b, capacity, kKMass, blockIdx.x == 0)) : 0;
    S.at[b + 1] = static_cast<long long>((ctx + kMKeys - 1) / kMKeys) *
                  ((static_cast<long long>(n) * a.heads + kMRows - 1) / kMRows);
  }
  if (tid == 0) {
    for (int i = 0; i < kMRing; ++i) {
      mbar_init(&S.full[i], 2 * kMDeqWarps);     // the eight warps of each CTA
      mbar_init(&S.empty[i], 1);
    }
    for (int i = 0; i < kMStages; ++i) mbar_init(&S.stage_full[i], 1);
    for (int i = 0; i < kMAcc; ++i) {
      mbar_init(&S.acc_full[i], 1);
      mbar_init(&S.acc_empty[i], 2 * kMEpiWarps);
    }
    mbar_init(&S.q_full, 2 * kMEpiWarps);
    for (int i = 0; i < 2; ++i) mbar_init(&S.scale_full[i], kMEpiWarps);
    mbar_init(&S.drain, 1);
    S.wide[0] = S.wide[1] = 0.0f;
    fence_barrier_init();
  }
  __syncthreads();
  if (warp == 0) {
    long long run = 0;
    for (int b0 = 0; b0 < cache.batch; b0 += 32) {
      const int b = b0 + lane;
      long long v = b < cache.batch ? S.at[b + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (b < cache.batch) S.at[b + 1] = run + v;
      run += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) S.at[0] = 0;
  } else if (warp == kMMmaWarp) {
    tmem_alloc_pair(&S.tmem_base, kMTmemCols);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync_all();          // both CTAs' barriers are initialised
  const uint32_t tmem = S.tmem_base;
  const long long total = S.at[cache.batch];
  const int used = static_cast<int>(min(total, static_cast<long long>(pairs)));
  const long long lo = pair < used ? total * pair / used : total;
  const long long hi = pair < used ? total * (pair + 1) / used : total;
  if (warp == 0 && lo < hi) {                     // the last request that starts at or before lo
    int at_b = 0;
    for (int b = lane; b < cache.batch; b += 32)
      if (S.at[b] <= lo && S.at[b + 1] > lo) at_b = b;
    at_b = __reduce_max_sync(0xffffffffu, at_b);
    if (lane == 0) S.start_b = at_b, S.start_at = S.at[at_b];
  }
  // the constant operand of the last step of K: ones in three of its 16 channels
  for (int i = tid; i < 128 * 8; i += kMThreads) {
    const int row = i >> 3, word = i & 7;
    const uint32_t v = word == 0 ? 0x3C003C00u : (word == 1 ? 0x00003C00u : 0u);
    *reinterpret_cast<uint32_t*>(S.a_ones + sw32_offset(row, word * 4)) = v;
  }
  fence_proxy_async_smem();
  __syncthreads();             // the plan's tables are read; the ring may be filled

  // Steps of request b, and the run at step pos (place: a request not behind
  // it and the steps before that one).
  struct Walk {
    int b;
    long long at;
  };
  auto steps_of = [&](int b) {
    const int n = queries_of(a, b, kKMass, false);
    const int ctx = n > 0 ? max(0, checked_ctx_len(cache, b, capacity, kKMass, false)) : 0;
    return static_cast<long long>((ctx + kMKeys - 1) / kMKeys) * ((static_cast<long long>(n) * a.heads + kMRows - 1) / kMRows);
  };
  auto run_at = [&](long long pos, Walk& w) {
    Run u;
    for (long long n = steps_of(w.b); w.at + n <= pos; n = steps_of(w.b)) w.at += n, ++w.b;
    const int b = w.b;
    u.b = b;
    u.ctx = cache.ctx_len[b];
    u.q0 = a.q_start ? a.q_start[b] : b;
    u.rows = (a.q_start ? a.q_start[b + 1] - u.q0 : 1) * a.heads;
    const int row_tiles = (u.rows + kMRows - 1) / kMRows, key_tiles = (u.ctx + kMKeys - 1) / kMKeys;
    const long long r = pos - w.at, per = static_cast<long long>(kMPart) * row_tiles;
    u.part = static_cast<int>(r / per) * kMPart;
    const int tiles = min(kMPart, key_tiles - u.part);
    const long long in = r % per;
    u.rt = static_cast<int>(in / tiles);
    u.kt0 = static_cast<int>(in % tiles);
    u.kt1 = static_cast<int>(min(static_cast<long long>(tiles), u.kt0 + (hi - pos)));
    u.part_lo = pos - in;
    u.part_hi = u.part_lo + static_cast<long long>(tiles) * row_tiles;
    return u;
  };
  // Where the run's tiles end for this row tile: it sees nothing behind (every
  // lane of a warp; at most 16 tokens).
  auto seen_end = [&](const Run& u) {
    const int first = (u.rt * kMRows) / a.heads, n = min(kMRows, u.rows - u.rt * kMRows) / a.heads;
    int last = -1;
    if (lane < n) last = a.q_pos[u.q0 + first + lane];
    const int keys = seen_by(__reduce_max_sync(0xffffffffu, last), a.ratio, u.ctx);
    return min(u.kt1, (keys + kMKeys - 1) / kMKeys - u.part);
  };
  auto columns = [&](const Run& u) { return (min(kMRows, u.rows - u.rt * kMRows) + 31) & ~31; };

  if (tid == 0 && rank == 0) {
    MassRecord r = {lo, lo, lo, 0, 0, used, 0};
    if (lo < hi) {
      Walk w = {S.start_b, S.start_at};
      const Run u = run_at(lo, w);
      r.part_lo = u.part_lo;
      r.part_hi = u.part_hi;
      r.b = u.b;
      r.k0 = u.part * kMKeys;
    }
    wsp.rec[pair] = r;
  }

  bool ok = true;
  if (warp < kMEpiWarps) {
    // ================= query rows, exp2 and the sums =================
    const uint32_t q_full = map_rank(smem_u32(&S.q_full), 0);
    const uint32_t tm_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);   // thread: entry tid of this CTA's 128
    const float sign = scale < 0.0f ? -1.0f : 1.0f;
    int item = 0, held_b = -1, held_rt = -1, loads = 0, told = 0, min_lim = 0;
    Walk walk = {S.start_b, S.start_at};
    bool wide = false;
    const float c2 = fabsf(scale) * kLog2e * kMUndo;        // log2 units of an accumulator's unit
    // 16 of the 32 columns of an entry in r (from `o` on)
    auto add_fast = [&](const uint32_t (&r)[32], int o, int c, int key, bool mask, float (&part)[4]) {
      if (!mask) {
#pragma unroll
        for (int j = 0; j < 16; ++j) part[j & 3] += ex2(__uint_as_float(r[o + j]) * c2);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int4 lim = *reinterpret_cast<const int4*>(S.col_lim + c + 4 * j);
          part[0] += key < lim.x ? ex2(__uint_as_float(r[o + 4 * j]) * c2) : 0.0f;
          part[1] += key < lim.y ? ex2(__uint_as_float(r[o + 4 * j + 1]) * c2) : 0.0f;
          part[2] += key < lim.z ? ex2(__uint_as_float(r[o + 4 * j + 2]) * c2) : 0.0f;
          part[3] += key < lim.w ? ex2(__uint_as_float(r[o + 4 * j + 3]) * c2) : 0.0f;
        }
      }
    };
    // the wide form: each column's factor and log2 of its sum
    auto add_wide = [&](const uint32_t (&r)[32], int o, int c, int key, float (&part)[4]) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float p = ex2(fmaf(__uint_as_float(r[o + j]), S.col_scale[loads & 1][c + j], -S.col_lse2[c + j]));
        part[j & 3] += key < S.col_lim[c + j] ? p : 0.0f;
      }
    };
    // Tells the other CTA (its warps wait for all of this CTA's) and hears from
    // it; whether one warp's wait ran out is voted on, so that all four leave.  Two
    // barriers by turns: the other CTA can be at the next exchange before a warp
    // here has looked at this one, and with one barrier that warp would wait for a
    // parity that has gone by.  It cannot be two ahead, since that takes this
    // CTA's arrivals for the next one, which follow the vote.
    auto exchange = [&]() {
      uint64_t* heard = &S.scale_full[told & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive_release_cluster(map_rank(smem_u32(heard), rank ^ 1u));
      ok = mbar_wait_cluster_all(heard, (told >> 1) & 1, wait_ns);
      ok = !named_bar_or(kBarEpi, kMEpiWarps * 32, !ok);
      ++told;
    };
    bool fresh = true;                              // no part is held
    for (long long pos = lo; ok && pos < hi;) {
      const Run u = run_at(pos, walk);
      pos += u.kt1 - u.kt0;
      const int end = seen_end(u), N = columns(u), half = N / 2;
      if (fresh) {
        for (int kt = 0; kt < kMPart; ++kt) S.sum[kt * (kMKeys / 2) + tid] = 0.0f;
        fresh = false;
      }
      if (u.kt0 < end) {
        // every product that read the held rows is done (their accumulators were awaited)
        const bool load = u.b != held_b || u.rt != held_rt;
        if (load) {
          named_bar_sync(kBarEpi, kMEpiWarps * 32);     // the column tables are free
          held_b = u.b;
          held_rt = u.rt;
          const int in_tile = min(kMRows, u.rows - u.rt * kMRows);
          const long long row0 = static_cast<long long>(u.q0) * a.heads + u.rt * kMRows;
          ++loads;
          const int turn = loads & 1;
          if (tid == 0) S.wide[turn ^ 1] = 0.0f;        // (the other CTA writes it after it has heard of this turn)
          // this CTA's half of the rows; the column tables hold both halves
          bool large = !(c2 > kMUnitLow && c2 < kMUnitHigh);
          const int mine = in_tile - static_cast<int>(rank) * half;
          load_query_rows<kMRows / 2, kMEpiWarps, kMExponent>(q, row0 + static_cast<int>(rank) * half, mine, half, sign, S.q[0],
                                                       warp, lane, [&](int, uint32_t top) {
                                                         large = large || top >= (127u + kMExponent + 1) << 7;
                                                       });
          int lowest = 0x7FFFFFFF;
          for (int c = tid; c < N; c += kMEpiWarps * 32) {
            int lim = 0;
            float l = 0.0f;
            if (c < in_tile) {
              lim = seen_by(a.q_pos[u.q0 + (u.rt * kMRows + c) / a.heads], a.ratio, u.ctx);
              l = lse[row0 + c];
              lowest = min(lowest, lim);
            }
            S.col_lim[c] = lim;
            S.col_lse2[c] = l * kLog2e;
            // -lse in the accumulator's unit: three fp16 parts hold an fp32 value
            // whole, or to 2^-25 below 1/2 (columns without a row: far below
            // everything)
            float v = c < in_tile ? (lim > 0 ? -l * (kLog2e / c2) : 0.0f) : -kMLargest;
            if (!(fabsf(v) <= kMLargest)) large = true, v = 0.0f;
            const int r = c - static_cast<int>(rank) * half;
            if (r >= 0 && r < half) {
              const __half h0 = __float2half_rn(v), h1 = __float2half_rn(v - __half2float(h0));
              const __half h2 = __float2half_rn(v - __half2float(h0) - __half2float(h1));
              const uint32_t w0 = __half_as_ushort(h0) | (static_cast<uint32_t>(__half_as_ushort(h1)) << 16);
              *reinterpret_cast<uint4*>(S.b_lse + sw32_offset(r, 0)) = make_uint4(w0, __half_as_ushort(h2), 0u, 0u);
              *reinterpret_cast<uint4*>(S.b_lse + sw32_offset(r, 16)) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          lowest = __reduce_min_sync(0xffffffffu, lowest);
          if (lane == 0) S.warp_min[warp] = lowest;
          if (__any_sync(0xffffffffu, large) && lane == 0) {
            S.wide[turn] = 1.0f;
            st_cluster(map_rank(smem_u32(&S.wide[turn]), rank ^ 1u), 1.0f);
          }
          fence_proxy_async_smem();
          named_bar_sync(kBarEpi, kMEpiWarps * 32);
          min_lim = __reduce_min_sync(0xffffffffu, S.warp_min[lane % kMEpiWarps]);
          exchange();
          if (!ok) break;
          wide = *reinterpret_cast<volatile float*>(&S.wide[turn]) != 0.0f;
          if (wide) {
            // Columns' factors, of both CTAs' rows, and rows scaled by themselves
            float* table = S.col_scale[turn] + rank * half;
            const uint32_t there = map_rank(smem_u32(table), rank ^ 1u);
            load_query_rows<kMRows / 2, kMEpiWarps, kPerRow>(q, row0 + static_cast<int>(rank) * half, mine, half, sign, S.q[0], warp,
                                                      lane, [&](int r, uint32_t top) {
                                                        const float f = query_row_down(top) * fabsf(scale) * kLog2e * kRowScale;
                                                        table[r] = f;
                                                        st_cluster(there + r * 4, f);
                                                      });
            for (int i = tid; i < 128 * 2; i += kMEpiWarps * 32)
              reinterpret_cast<uint4*>(S.b_lse)[i] = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            named_bar_sync(kBarEpi, kMEpiWarps * 32);
            exchange();
            if (!ok) break;
          }
          if (lane == 0) mbar_arrive_cluster(q_full);
        }
      }
      for (int kt = u.kt0; ok && kt < end; ++kt, ++item) {
        const int k0 = (u.part + kt) * kMKeys, key0 = k0 + static_cast<int>(rank) * (kMKeys / 2);
        const int key = key0 + tid;
        int page = -1;                               // of this CTA's entries
        if (key0 < u.ctx) page = cache.page_table[static_cast<long long>(u.b) * cache.max_pages_per_req + key0 / cache.page_size];
        const bool mask = min_lim < min(k0 + kMKeys, u.ctx);
        const int acc = item % kMAcc;
        ok = mbar_wait_all(&S.acc_full[acc], (item / kMAcc) & 1, wait_ns);
        ok = !named_bar_or(kBarEpi, kMEpiWarps * 32, !ok);
        if (!ok) break;
        tc_fence_after();
        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        // Tensor-memory loads of 32 columns run one ahead: each takes about 500
        // cycles next to the MMAs (with 16 the wait for them was most of the time).
        uint32_t r0[32], r1[32];
        const uint32_t from = tm_lane + acc * kMRows;
        auto add = [&](const uint32_t (&r)[32], int c) {
#pragma unroll
          for (int o = 0; o < 32; o += 16) {
            if (wide) add_wide(r, o, c + o, key, part);
            else add_fast(r, o, c + o, key, mask, part);
          }
        };
        tmem_ld_32x32b_x32(from, r0);
#pragma unroll 1
        for (int c = 0; c < N; c += 64) {            // (N is a multiple of 32)
          tmem_ld_wait();
          if (c + 32 < N) tmem_ld_32x32b_x32(from + c + 32, r1);
          add(r0, c);
          if (c + 32 < N) {
            tmem_ld_wait();
            if (c + 64 < N) tmem_ld_32x32b_x32(from + c + 64, r0);
            add(r1, c + 32);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_rank(smem_u32(&S.acc_empty[acc]), 0));
        if (page >= 0 && page < cache.num_pages) S.sum[kt * (kMKeys / 2) + tid] += (part[0] + part[1]) + (part[2] + part[3]);
      }
      // the part's end, or the range's: the entries' weights, or this pair's share of them
      if (ok && (pos >= hi || pos >= u.part_hi)) {
        const bool whole = u.part_lo >= lo && u.part_hi <= hi;
        float* share = wsp.part + (2 * static_cast<size_t>(pair) + (u.part_lo < lo ? 0 : 1)) * (kMPart * kMKeys);
#pragma unroll 4
        for (int kt = 0; kt < kMPart; ++kt) {
          const int in = kt * kMKeys + static_cast<int>(rank) * (kMKeys / 2) + tid, key = u.part * kMKeys + in;
          const float s = S.sum[kt * (kMKeys / 2) + tid];
          if (!whole) share[in] = s;
          else if (key < u.ctx && s != 0.0f) mass[u.b * capacity + key] += s;
        }
        fresh = true;
      }
    }
    if (!ok && lane == 0) report_error(cache.err_word, CSA2_ERR_TIMEOUT, kKMass, static_cast<int>(rank), item);
  } else if (warp < kMEpiWarps + kMDeqWarps) {
    // ================= dequantisation =================
    // All eight warps fill a pair of slots together, so that one pair is filled
    // while the products take the other (with four warps to a pair a slot's
    // filling and its products took turns).  A granule is 32 channels of an
    // entry; lane: keys krow and krow + 64, granule kg of slot ksel of each of
    // a tile's four pairs.  A quarter warp holds 4 entries x 2 neighbouring
    // granules: its 16-byte stores fall into eight different chunks.
    const int krow = (warp - kMEpiWarps) * 8 + ((lane >> 3) & 1) * 4 + (lane & 3), kg = (lane >> 2) & 1, ksel = lane >> 4;
    const int k_code = ksel * 32 + kg * 16, k_sc = ksel * 4 + kg * 2;
    uint4 codes[8];                                  // the lane's granules of the tile in turn: pair, key
    uint32_t sc[8], mask = 0;
    // The page of this CTA's 128 entries is looked up a tile ahead (fetch);
    // row_of_page, half a tile later, gives their first cache row, or -1: not
    // there, or a bad page (recorded).
    struct Place {
      int b, key, page, off;
    };
    auto fetch = [&](int b, int ctx, int tile) {
      Place x;
      x.b = b;
      x.key = tile * kMKeys + static_cast<int>(rank) * (kMKeys / 2);
      const int slot = x.key / cache.page_size;
      x.off = x.key - slot * cache.page_size;
      x.page = -2;
      if (x.key < ctx) x.page = cache.page_table[static_cast<long long>(b) * cache.max_pages_per_req + slot];
      return x;
    };
    auto row_of_page = [&](const Place& x) {
      if (x.page >= 0 && x.page < cache.num_pages) return x.page * cache.page_size + x.off;
      if (x.page != -2) report_error(cache.err_word, CSA2_ERR_DEVICE_BOUNDS, kKMass, x.b, x.key);
      return -1;
    };
    const uint8_t* cp = kMStages > 0 ? S.stage : cache.kv_codes;   // of the tile to be loaded
    const uint8_t* sp = kMStages > 0 ? S.stage : cache.kv_scales;
    uint32_t next_mask = 0;
    auto aim = [&](int base) {
      const long long r = max(base, 0) + krow;       // entries that are not there read row 0 with a scale of 0
      cp = cache.kv_codes + r * kKvCodeBytes + k_code;
      sp = cache.kv_scales + r * kKvScaleBytes + k_sc;
      next_mask = base < 0 ? 0u : 0x7F7Fu;
    };
    auto load = [&](int i) {
      codes[i] = *reinterpret_cast<const uint4*>(cp + (i >> 1) * 64 + (i & 1) * 64 * kKvCodeBytes);
      sc[i] = *reinterpret_cast<const uint16_t*>(sp + (i >> 1) * 8 + (i & 1) * 64 * kKvScaleBytes);
    };
    // The tiles in order: run by run, the visible ones.
    Walk walk = {S.start_b, S.start_at};
    long long pos = lo;
    int tb = 0, tctx = 0, tile = 0, left = 0;        // the tile, its request, and the tiles left of its run
    auto next_tile_of = [&]() {                      // advances to a tile; false at the range's end
      ++tile;
      --left;
      while (left <= 0) {
        if (pos >= hi) return false;
        const Run u = run_at(pos, walk);
        pos += u.kt1 - u.kt0;
        tb = u.b;
        tctx = u.ctx;
        tile = u.part + u.kt0;
        left = seen_end(u) - u.kt0;
      }
      return true;
    };
    int n = 0;                                       // the next pair in the order of all pairs
    // The held granules into the four pairs of slots in turn; their registers
    // then receive those of the tile that is aimed at.
    auto store_tile = [&](bool then_load) {
#pragma unroll
      for (int p = 0; p < 4; ++p, ++n) {
        const int x2 = n % kMRing;
        ok = ok && mbar_wait_all(&S.empty[x2], ((n / kMRing) & 1) ^ 1, wait_ns);
        if (!ok) continue;
        uint8_t* dst = S.ring[x2] + ksel * kMSlot + krow * 128;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint4 o[4];
          dequant_32(codes[2 * p + i], sc[2 * p + i] & mask, o);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(dst + i * 64 * 128 + (((kg * 4 + j) ^ (krow & 7)) << 4)) = o[j];
        }
        if (then_load) load(2 * p), load(2 * p + 1);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_rank(smem_u32(&S.full[x2]), 0));
      }
      mask = next_mask;
    };
    if constexpr (kMStages == 0) {
      bool have = next_tile_of(), more = false;      // a tile is loaded; another one comes after it
      Place ahead = {};
      if (have) {
        aim(row_of_page(fetch(tb, tctx, tile)));
#pragma unroll
        for (int i = 0; i < 8; ++i) load(i);
        mask = next_mask;
        more = next_tile_of();
        if (more) ahead = fetch(tb, tctx, tile);
      }
      while (ok && have) {
        have = more;
        if (more) {
          aim(row_of_page(ahead));
          more = next_tile_of();
          if (more) ahead = fetch(tb, tctx, tile);
        }
        store_tile(true);                            // (at the end the last tile is loaded again)
      }
    } else {
      // The first warp walks over the tiles and has each one's packed rows (128
      // neighbours of one page) copied to a stage, kMStages tiles ahead of the
      // registers; a stage says what it holds, so the other warps need no walk.
      const bool walker = warp == kMEpiWarps;
      const uint64_t policy = l2_policy_evict_first();
      bool more = false;
      Place ahead = {};
      int issued = 0, t = 0;                         // tiles asked for, tiles taken
      auto issue = [&]() {
        const int st = issued++ % kMStages;
        int base = -2;
        if (more) {
          base = row_of_page(ahead);
          more = next_tile_of();
          if (more) ahead = fetch(tb, tctx, tile);
        }
        if (lane == 0) {
          S.stage_row[st] = base;
          if (base >= 0) {
            uint8_t* dst = S.stage + st * kMStage;
            mbar_arrive_expect_tx(&S.stage_full[st], kMStage);
            bulk_load_1d(dst, cache.kv_codes + static_cast<long long>(base) * kKvCodeBytes, 128 * kKvCodeBytes,
                         &S.stage_full[st], policy);
            bulk_load_1d(dst + 128 * kKvCodeBytes, cache.kv_scales + static_cast<long long>(base) * kKvScaleBytes,
                         128 * kKvScaleBytes, &S.stage_full[st], policy);
          } else {
            mbar_arrive(&S.stage_full[st]);
          }
        }
        __syncwarp();
      };
      bool next = false;                             // the tile that is aimed at exists
      auto take = [&]() {
        const int st = t % kMStages;
        ok = mbar_wait_all(&S.stage_full[st], (t / kMStages) & 1, wait_ns);
        const int base = ok ? *reinterpret_cast<volatile int*>(&S.stage_row[st]) : -2;
        next = base != -2;
        next_mask = base < 0 ? 0u : 0x7F7Fu;
        cp = S.stage + st * kMStage + krow * kKvCodeBytes + k_code;
        sp = S.stage + st * kMStage + 128 * kKvCodeBytes + krow * kKvScaleBytes + k_sc;
      };
      auto give = [&]() {                            // every warp has read the stage (or one gave up: all do)
        ok = !named_bar_or(kBarDeq, kMDeqWarps * 32, !ok);
        if (ok) ++t;
        if (ok && walker && next) issue();
      };
      if (walker) {
        more = next_tile_of();
        if (more) ahead = fetch(tb, tctx, tile);
        for (int i = 0; i < kMStages; ++i) issue();
      }
      take();
      if (next) {
#pragma unroll
        for (int i = 0; i < 8; ++i) load(i);
      }
      mask = next_mask;
      bool have = next;
      give();
      while (ok && have) {
        take();
        have = next;
        store_tile(next);
        give();
      }
      // copies that were asked for and not awaited
      if (!ok && walker)
        for (; t < issued; ++t) (void)mbar_wait_all(&S.stage_full[t % kMStages], (t / kMStages) & 1, kWaitLimitNs);
    }
    if (!ok && lane == 0) report_error(cache.err_word, CSA2_ERR_TIMEOUT, kKMass, static_cast<int>(rank), -n);
  } else if (rank == 0) {
    // ================= MMA issuer =================
    const bool issue = elect_one();
    const uint64_t k_desc = sw128_kmajor_desc(smem_u32(S.ring[0])), q_desc = sw128_kmajor_desc(smem_u32(S.q[0]));
    const uint64_t ones_desc = sw32_kmajor_desc(smem_u32(S.a_ones)), lse_desc = sw32_kmajor_desc(smem_u32(S.b_lse));
    Walk walk = {S.start_b, S.start_at};
    int s = 0, item = 0, loads = 0, held_b = -1, held_rt = -1;
    uint32_t phase = 0;
    for (long long pos = lo; ok && pos < hi;) {
      const Run u = run_at(pos, walk);
      pos += u.kt1 - u.kt0;
      const int end = seen_end(u);
      if (u.kt0 >= end) continue;
      if (u.b != held_b || u.rt != held_rt) {
        held_b = u.b;
        held_rt = u.rt;
        ok = mbar_wait_cluster_all(&S.q_full, loads & 1, wait_ns);
        ++loads;
      }
      const uint32_t idesc = idesc_f16_f32(kMKeys, columns(u), false, false);
      for (int kt = u.kt0; ok && kt < end; ++kt, ++item) {
        const int acc = item % kMAcc;
        ok = mbar_wait_cluster_all(&S.acc_empty[acc], ((item / kMAcc) & 1) ^ 1, wait_ns);
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; ok && c < 4; ++c) {
          ok = mbar_wait_cluster_all(&S.full[s], phase, wait_ns);
          if (!ok) break;
          tc_fence_after();
          if (issue) {
            const uint64_t ad = k_desc + s * (2 * kMSlot / 16), bd = q_desc + c * (2 * kMQPart / 16);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_f16_pair(tmem + acc * kMRows, ad + (kk >> 2) * (kMSlot / 16) + (kk & 3) * 2,
                            bd + (kk >> 2) * (kMQPart / 16) + (kk & 3) * 2, idesc, (c | kk) > 0 ? 1u : 0u);
            umma_commit_pair(&S.empty[s]);
            if (c == 3) {
              umma_f16_pair(tmem + acc * kMRows, ones_desc, lse_desc, idesc, 1u);
              umma_commit_pair(&S.acc_full[acc]);
            }
          }
          __syncwarp();
          if (++s == kMRing) {
            s = 0;
            phase ^= 1;
          }
        }
      }
    }
    if (lane == 0 && !ok) report_error(cache.err_word, CSA2_ERR_TIMEOUT, kKMass, -1, item);
    __syncwarp();
    if (issue) umma_commit_pair(&S.drain);
    (void)mbar_wait_all(&S.drain, 0, kWaitLimitNs);
  } else {
    if (lane == 0) (void)mbar_wait(&S.drain, 0, 4 * kWaitLimitNs);   // the leader's last arrival here
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();          // every MMA has completed, no barrier of the other CTA is touched after this
  if (warp == kMMmaWarp) tmem_release_pair(tmem, kMTmemCols);
}

// Joins the parts that ranges cut: block (c, y) takes 256 entries of the part
// that pair c starts inside, if c is the first to do so.
__global__ void __launch_bounds__(kMKeys) attn_mass_join_kernel(const csa2_cache cache, float* __restrict__ mass, void* ws) {
  pdl_wait();
  const MassWorkspace wsp = split_mass_ws(ws);
  const int c = blockIdx.x;
  const MassRecord r = wsp.rec[c];
  if (c >= r.pairs || r.lo == r.part_lo || wsp.rec[c - 1].lo > r.part_lo) return;
  const int in = blockIdx.y * kMKeys + threadIdx.x, key = r.k0 + in;
  // pair c - 1's share comes first, then those of the pairs that start before
  // the part's end (they ascend)
  static_assert(kMaxPairs <= kMKeys, "a thread per pair");
  const int k = threadIdx.x;
  const int end = c + __syncthreads_count(k >= c && k < r.pairs && wsp.rec[min(k, r.pairs - 1)].lo < r.part_hi);
  if (key >= cache.ctx_len[r.b]) return;
  constexpr size_t kShare = kMPart * kMKeys;
  float sum = wsp.part[(2 * static_cast<size_t>(c - 1) + 1) * kShare + in];
#pragma unroll 8
  for (int i = c; i < end; ++i) sum += wsp.part[2 * static_cast<size_t>(i) * kShare + in];
  const long long capacity = static_cast<long long>(cache.max_pages_per_req) * cache.page_size;
  if (sum != 0.0f) mass[r.b * capacity + key] += sum;
}

template <int kMRows, int kMRing, int kMStages>
cudaError_t launch_mass(const DenseArgs& a, const __nv_bfloat16* q, float scale, const float* lse, float* mass, void* ws,
                        int pairs, uint64_t wait_ns, cudaStream_t stream) {
  static ContextMemo attrs;
  const size_t smem = sizeof(MassSmem<kMRows, kMRing, kMStages>) + 1024;
  const cudaError_t e = attrs.once([&] {
    return cudaFuncSetAttribute(attn_mass_kernel<kMRows, kMRing, kMStages>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(smem));
  });
  if (e != cudaSuccess) return e;
  attn_mass_kernel<kMRows, kMRing, kMStages><<<2 * pairs, kMThreads, smem, stream>>>(a, q, scale, lse, mass, ws, wait_ns);
  return cudaGetLastError();
}

}  // namespace

size_t attn_mass_workspace_bytes() {
  return kMaxPairs * (sizeof(MassRecord) + 2 * static_cast<size_t>(kMPart) * kMKeys * sizeof(float));
}

cudaError_t launch_attn_mass(const csa2_cache& cache, int n_queries, const int32_t* q_start, const int32_t* q_pos,
                             int ratio, const uint16_t* q, int H, float scale, const float* lse, float* mass, void* ws,
                             int num_sms, uint64_t wait_ns, cudaStream_t stream) {
  const DenseArgs a = {cache, q_start, q_pos, n_queries, ratio, H, 1};
  const int pairs = min(kMaxPairs, num_sms / 2);
  // At most 64 query rows a request on average (single tokens): tiles of 64 rows,
  // and the room in shared memory for stages of packed entries and a third pair
  // of slots.  One token of 8 requests x 64 heads over 65,536 entries: 91 us, with
  // tiles of 256 rows 104; with 128 rows a request the narrow tiles read the
  // entries twice: 166 us against 121 (8 x 2 tokens x 64 heads over 65,536).  The
  // host knows the average alone.  64 requests of 16,384 entries, 64 tokens x 64
  // heads, narrow / 256 rows: one token each 185 / 208, 30 single tokens and a chunk
  // of 34 in one request 185 / 179, all 64 in one request 173 / 105.
  const bool narrow = static_cast<long long>(n_queries) * H <= 64LL * cache.batch;
  const __nv_bfloat16* q16 = reinterpret_cast<const __nv_bfloat16*>(q);
  cudaError_t e = narrow ? launch_mass<64, 3, 2>(a, q16, scale, lse, mass, ws, pairs, wait_ns, stream)
                         : launch_mass<256, 2, 0>(a, q16, scale, lse, mass, ws, pairs, wait_ns, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pairs, kMPart);
  cfg.blockDim = dim3(kMKeys);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // it waits for the ranges before reading
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_mass_join_kernel, cache, mass, ws);
}

}  // namespace csa2
