// Attention weight that every cached entry received from the queries of a
// call: mass[b][e] += sum over request b's queries and heads of
// exp(scale q . v_e - lse), with the rows' log-sum-exp given.
//
// A matrix product with a sum over its columns: S^T = K Q^T on tcgen05 over a
// pair of CTAs, M = 256 entries (128 per CTA), N = 256 query rows (128 loaded
// by each CTA), bf16 operands (queries as they lie; the dequantised rows are
// exact in bf16: at most 6 significant bits), fp32 sums.  Entries lie in the
// lanes of tensor memory, so a thread sums its entry's weights over the
// columns by itself.
//   * the epilogue warps dequantise 128 entries per CTA into shared memory
//     once per unit; the query rows stream past them;
//   * warp 0: TMA of 64-channel parts of the query rows into a ring; warp 1 of
//     the leader: the MMAs, into one of two 256-column accumulators; warps 2-9:
//     two column halves x four lane quarters, exp2 and the sum.
// Why a pair: one CTA alone would read 128 + 64 bytes of shared memory a cycle
// (operands, and the arriving rows) where it has 128, and every SM would draw
// 64 bytes a cycle from L2; the pair halves both.
// The list of (256 entries, 256 rows) items is cut into equal ranges; cut
// entries' sums are joined in a fixed order by a second launch.
#include <cuda_bf16.h>

#include "attn_tile.cuh"
#include "cta_pair.cuh"
#include "dense_plan.cuh"
#include "launch.h"

namespace csa2 {

namespace {

constexpr int kMKeys = 256;                       // entries per unit (both CTAs)
constexpr int kMRows = 256;                       // query rows per item
constexpr int kMStages = 5;
constexpr int kMEpiWarps = 8;
constexpr int kMThreads = 64 + kMEpiWarps * 32;   // 320
constexpr int kMAcc = 2;
constexpr uint32_t kMTmemCols = kMAcc * kMRows;   // 512
constexpr int kAtomBytes = 128 * 128;             // 128 rows x 64 16-bit channels
constexpr int kBoxRows = 32;                      // rows of one TMA box
constexpr int kMaxPairs = 128;
constexpr int kBarEpi = 1;

struct __align__(1024) MassSmem {
  uint8_t k[kKvDim / 64][kAtomBytes];             // A: this CTA's 128 entries
  uint8_t q[kMStages][kAtomBytes];                // B: this CTA's half of the rows, 64 channels
  float lse2[2][kMRows];                          // log2 of the rows' sums
  int lim[2][kMRows];                             // entries seen by each row (0: no row)
  float red[kMKeys / 2];
  int before[kMaxDenseBatch + 1];                 // units before each request
  long long at[kMaxDenseBatch + 1];               // items before each request
  uint64_t full[kMStages];
  uint64_t empty[kMStages];
  uint64_t acc_full[kMAcc];
  uint64_t acc_empty[kMAcc];
  uint64_t k_full;
  uint64_t drain;
  uint32_t tmem_base;
  volatile int abort_flag;
};

// What a pair says of its range, for the joining launch.
struct MassRecord {
  long long lo, unit_lo, unit_hi;   // first item; first and past-the-last item of the unit it starts in
  int b, k0;                        // that unit
  int pairs, pad;
};

struct MassWorkspace {
  MassRecord* rec;
  float* part;    // [pairs][2][256]
};
__host__ __device__ inline MassWorkspace split_mass_ws(void* ws) {
  MassWorkspace w;
  w.rec = static_cast<MassRecord*>(ws);
  w.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kMaxPairs * sizeof(MassRecord));
  return w;
}

// Entry [k0 + 128 rank, + 128) of request b is there: visible length and page.
__device__ __forceinline__ int page_row(const csa2_cache& c, int b, int key, bool report) {
  const int page = c.page_table[static_cast<long long>(b) * c.max_pages_per_req + key / c.page_size];
  if (page < 0 || page >= c.num_pages) {
    if (report) report_error(c.err_word, CSA2_ERR_DEVICE_BOUNDS, kKMass, b, key);
    return -1;
  }
  return page * c.page_size + key % c.page_size;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMThreads, 1)
    attn_mass_kernel(const DenseArgs a, const __grid_constant__ CUtensorMap q_map, float scale,
                     const float* __restrict__ lse, float* __restrict__ mass, void* ws, uint64_t wait_ns) {
  extern __shared__ uint8_t smem_raw[];
  MassSmem& S = *reinterpret_cast<MassSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const csa2_cache& cache = a.cache;
  const MassWorkspace wsp = split_mass_ws(ws);
  const long long capacity = static_cast<long long>(cache.max_pages_per_req) * cache.page_size;

  // ---- plan: items of each request = (its units of 256 entries) x (its tiles of 256 rows) ----
  for (int b = tid; b < cache.batch; b += kMThreads) {
    const int n = queries_of(a, b, kKMass, blockIdx.x == 0);
    const int ctx = n > 0 ? max(0, checked_ctx_len(cache, b, capacity, kKMass, blockIdx.x == 0)) : 0;
    S.before[b + 1] = ctx;
    S.at[b + 1] = static_cast<long long>((ctx + kMKeys - 1) / kMKeys) *
                  ((static_cast<long long>(n) * a.heads + kMRows - 1) / kMRows);
  }
  if (tid == 0) {
    for (int s = 0; s < kMStages; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], 1);
    }
    for (int i = 0; i < kMAcc; ++i) {
      mbar_init(&S.acc_full[i], 1);
      mbar_init(&S.acc_empty[i], 2 * kMEpiWarps);
    }
    mbar_init(&S.k_full, 2 * kMEpiWarps);
    mbar_init(&S.drain, 1);
    S.abort_flag = 0;
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
  } else if (warp == 1) {
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

  // The range as units: request, entries, and the row tiles [t0, t1) of each.
  struct Unit {
    int b, ctx, k0, t0, t1, tiles, q0, rows;   // rows: of the whole request
  };
  auto unit_at = [&](long long pos, int b) {
    Unit u;
    while (S.at[b + 1] <= pos) ++b;
    u.b = b;
    u.ctx = S.before[b + 1];
    u.q0 = a.q_start ? a.q_start[b] : b;
    const int n = a.q_start ? a.q_start[b + 1] - u.q0 : 1;
    u.rows = n * a.heads;
    u.tiles = (u.rows + kMRows - 1) / kMRows;
    const long long r = pos - S.at[b];
    u.k0 = static_cast<int>(r / u.tiles) * kMKeys;
    u.t0 = static_cast<int>(r % u.tiles);
    u.t1 = static_cast<int>(min(static_cast<long long>(u.tiles), u.t0 + (hi - pos)));
    return u;
  };
  // Whether any row of tile t sees entry k0 or later (every lane of a warp).
  auto tile_seen = [&](const Unit& u, int t) {
    const int first = (t * kMRows) / a.heads, n = min(kMRows, u.rows - t * kMRows) / a.heads;
    int m = 0;
    if (lane < n) m = seen_by(a.q_pos[u.q0 + first + lane], a.ratio, u.ctx);
    return __any_sync(0xffffffffu, m > u.k0);
  };
  // N of the item: its rows, rounded up to 32.
  auto columns = [&](const Unit& u, int t) { return (min(kMRows, u.rows - t * kMRows) + 31) & ~31; };

  if (tid == 0 && rank == 0) {
    MassRecord r = {lo, lo, lo, 0, 0, used, 0};
    if (lo < hi) {
      const Unit u = unit_at(lo, 0);
      r.unit_lo = lo - u.t0;
      r.unit_hi = r.unit_lo + u.tiles;
      r.b = u.b;
      r.k0 = u.k0;
    }
    wsp.rec[pair] = r;
  }

  if (warp == 0) {
    // ================= producer =================
    const uint64_t policy = l2_policy_evict_last();
    int i = 0, b = 0;
    bool ok = true;
    for (long long pos = lo; ok && pos < hi;) {
      const Unit u = unit_at(pos, b);
      b = u.b;
      pos += u.t1 - u.t0;
      for (int t = u.t0; ok && t < u.t1; ++t) {
        if (!tile_seen(u, t)) continue;
        const int N = columns(u, t), half = N / 2;      // a multiple of 16: boxes overrun into the other rows' place
        const int boxes = (half + kBoxRows - 1) / kBoxRows;
        const int row0 = u.q0 * a.heads + t * kMRows + static_cast<int>(rank) * half;
        if (lane == 0) {
          for (int c = 0; c < kKvDim / 64; ++c, ++i) {
            const int s = i % kMStages;
            if (S.abort_flag || !mbar_wait(&S.empty[s], ((i / kMStages) & 1) ^ 1, wait_ns)) {
              ok = false;
              break;
            }
            if (rank == 0) mbar_arrive_expect_tx(&S.full[s], 2 * boxes * kBoxRows * 128);
            const uint32_t bar = map_rank(smem_u32(&S.full[s]), 0);
            for (int x = 0; x < boxes; ++x)
              tma_load_2d_pair(S.q[s] + x * kBoxRows * 128, &q_map, bar, c * 128, row0 + x * kBoxRows, policy);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
    }
    if (lane == 0 && !ok) {
      report_error(cache.err_word, CSA2_ERR_TIMEOUT, kKMass, static_cast<int>(rank), i);
      S.abort_flag = 1;
    }
    // copies still in flight (counted on the leader's barriers)
    if (lane == 0 && rank == 0 && !ok)
      for (int j = i > kMStages ? i - kMStages : 0; j < i; ++j)
        (void)mbar_wait(&S.full[j % kMStages], (j / kMStages) & 1, kWaitLimitNs / 2);
  } else if (warp == 1 && rank == 0) {
    // ================= MMA issuer =================
    const bool issue = elect_one();
    const uint64_t k_desc = sw128_kmajor_desc(smem_u32(S.k[0])), q_desc = sw128_kmajor_desc(smem_u32(S.q[0]));
    int s = 0, item = 0, units = 0, b = 0;      // units: those with an item that is computed
    uint32_t phase = 0;
    bool ok = true;
    for (long long pos = lo; ok && pos < hi;) {
      const Unit u = unit_at(pos, b);
      b = u.b;
      pos += u.t1 - u.t0;
      bool loaded = false;
      for (int t = u.t0; ok && t < u.t1; ++t) {
        if (!tile_seen(u, t)) continue;
        if (!loaded) {
          ok = mbar_wait_cluster_all(&S.k_full, units & 1, wait_ns);
          loaded = true;
          ++units;
        }
        const uint32_t idesc = idesc_f16_f32(kMKeys, columns(u, t), true, false);
        const int acc = item % kMAcc;
        ok = mbar_wait_cluster_all(&S.acc_empty[acc], ((item / kMAcc) & 1) ^ 1, wait_ns) && ok;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; ok && c < kKvDim / 64; ++c) {
          ok = __all_sync(0xffffffffu, S.abort_flag == 0 && mbar_wait(&S.full[s], phase, wait_ns)) != 0;
          if (!ok) break;
          tc_fence_after();
          if (issue) {
            const uint64_t ad = k_desc + c * (kAtomBytes / 16), bd = q_desc + s * (kAtomBytes / 16);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_f16_pair(tmem + acc * kMRows, ad + 2 * kk, bd + 2 * kk, idesc, (c | kk) > 0 ? 1u : 0u);
            umma_commit_pair(&S.empty[s]);
            if (c == kKvDim / 64 - 1) umma_commit_pair(&S.acc_full[acc]);
          }
          __syncwarp();
          if (++s == kMStages) {
            s = 0;
            phase ^= 1;
          }
        }
        ++item;
      }
    }
    if (lane == 0 && !ok) {
      report_error(cache.err_word, CSA2_ERR_TIMEOUT, kKMass, -1, item);
      S.abort_flag = 1;
    }
    __syncwarp();
    if (issue) umma_commit_pair(&S.drain);
    (void)mbar_wait(&S.drain, 0, kWaitLimitNs);
  } else if (warp == 1) {
    if (lane == 0) (void)mbar_wait(&S.drain, 0, 2 * kWaitLimitNs);   // the leader's last arrival here
  } else {
    // ================= dequantisation and epilogue =================
    const int et = tid - 64;                       // 0..255
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const float c2 = scale * kLog2e;
    const uint32_t k_full = map_rank(smem_u32(&S.k_full), 0);
    // The unit's 128 entries of this CTA, dequantised to bf16.  16-byte
    // granules (32 channels): a warp takes 8 rows x 4 granules, so that the
    // 16-byte stores of a quarter warp fall into different banks.
    auto load_keys = [&](int base) {
      for (int it = 0; it < 8; ++it) {
        const int x = it * kMEpiWarps + (warp - 2);             // 64 groups of (8 rows, 4 granules)
        const int row = (x >> 2) * 8 + (lane & 7), g = (x & 3) * 4 + (lane >> 3);
        uint4 hv[4] = {};
        if (base >= 0) {
          const long long r = base + row;
          const uint4 cv = *reinterpret_cast<const uint4*>(cache.kv_codes + r * kKvCodeBytes + g * 16);
          const uint32_t sc = *reinterpret_cast<const uint16_t*>(cache.kv_scales + r * kKvScaleBytes + g * 2);
          dequant16(cv, sc, hv);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&hv[j]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
              const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);   // exact: 6 significant bits
              w[k] = *reinterpret_cast<const uint32_t*>(&h);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int chunk = (g & 1) * 4 + j;
          *reinterpret_cast<uint4*>(S.k[g >> 1] + row * 128 + ((chunk ^ (row & 7)) << 4)) = hv[j];
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(k_full);
    };
    int item = 0, b = 0;
    bool ok = true;
    for (long long pos = lo; ok && pos < hi;) {
      const Unit u = unit_at(pos, b);
      b = u.b;
      pos += u.t1 - u.t0;
      bool loaded = false;
      const int key0 = u.k0 + static_cast<int>(rank) * (kMKeys / 2);
      const int base = key0 < u.ctx ? page_row(cache, u.b, key0, et == 0) : -1;
      const int key = key0 + quarter * 32 + lane;
      float sum = 0.0f;
      for (int t = u.t0; t < u.t1; ++t) {
        // this item's rows: a column per epilogue thread
        const int buf = item & 1;
        const int in_tile = min(kMRows, u.rows - t * kMRows);
        const int first = (t * kMRows) / a.heads, N = columns(u, t);
        int lim = 0;
        float l2 = 0.0f;
        if (et < in_tile) {
          lim = seen_by(a.q_pos[u.q0 + first + et / a.heads], a.ratio, u.ctx);
          l2 = lse[static_cast<long long>(u.q0) * a.heads + t * kMRows + et] * kLog2e;
        }
        const bool any = named_bar_or(kBarEpi, kMEpiWarps * 32, lim > u.k0);
        if (!any) continue;
        if (!loaded) {
          load_keys(base);
          loaded = true;
        }
        S.lse2[buf][et] = l2;
        S.lim[buf][et] = lim;
        const bool mask = named_bar_or(kBarEpi, kMEpiWarps * 32, et < N && lim < min(u.k0 + kMKeys, u.ctx));
        const int acc = item % kMAcc;
        ok = ok && mbar_wait_warp_backoff(&S.acc_full[acc], (item / kMAcc) & 1, wait_ns);
        ++item;
        if (!named_bar_or(kBarEpi, kMEpiWarps * 32, !ok)) {
          tc_fence_after();
          float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          for (int c = half * (kMRows / 2); c < min((half + 1) * (kMRows / 2), N); c += 32) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(tmem + acc * kMRows + (static_cast<uint32_t>(quarter * 32) << 16) + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 l4 = *reinterpret_cast<const float4*>(&S.lse2[buf][c + j]);
              const float lv[4] = {l4.x, l4.y, l4.z, l4.w};
              if (mask) {
                const int4 m4 = *reinterpret_cast<const int4*>(&S.lim[buf][c + j]);
                const int mv[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float p = ex2(fmaf(__uint_as_float(r[j + k]), c2, -lv[k]));
                  part[k] += key < mv[k] ? p : 0.0f;
                }
              } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) part[k] += ex2(fmaf(__uint_as_float(r[j + k]), c2, -lv[k]));
              }
            }
          }
          sum += (part[0] + part[1]) + (part[2] + part[3]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_rank(smem_u32(&S.acc_empty[acc]), 0));
        } else {
          ok = false;
          break;
        }
      }
      // both column halves, then the entry's weight or the pair's part of it
      if (half == 1) S.red[quarter * 32 + lane] = sum;
      named_bar_sync(kBarEpi, kMEpiWarps * 32);
      if (half == 0 && ok) {
        sum += S.red[quarter * 32 + lane];
        if (u.t1 - u.t0 == u.tiles) {
          if (key < u.ctx && base >= 0) mass[u.b * capacity + key] += sum;
        } else {
          wsp.part[(2 * pair + (u.t0 > 0 ? 0 : 1)) * kMKeys + static_cast<int>(rank) * (kMKeys / 2) + quarter * 32 +
                   lane] = base >= 0 ? sum : 0.0f;
        }
      }
      named_bar_sync(kBarEpi, kMEpiWarps * 32);
    }
    if (!ok && lane == 0) {
      report_error(cache.err_word, CSA2_ERR_TIMEOUT, kKMass, static_cast<int>(rank), -item);
      S.abort_flag = 1;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();          // every MMA has completed, no barrier of the other CTA is touched after this
  if (warp == 1) tmem_release_pair(tmem, kMTmemCols);
}

// Joins the units that ranges cut: block c takes the unit that pair c starts
// inside, if c is the first to do so.
__global__ void __launch_bounds__(kMKeys) attn_mass_join_kernel(const csa2_cache cache, float* __restrict__ mass, void* ws) {
  const MassWorkspace wsp = split_mass_ws(ws);
  const int c = blockIdx.x;
  const MassRecord r = wsp.rec[c];
  if (c >= r.pairs || r.lo == r.unit_lo || wsp.rec[c - 1].lo > r.unit_lo) return;
  float sum = wsp.part[(2 * (c - 1) + 1) * kMKeys + threadIdx.x];
  for (int k = c; k < r.pairs && wsp.rec[k].lo < r.unit_hi; ++k) sum += wsp.part[2 * k * kMKeys + threadIdx.x];
  const long long capacity = static_cast<long long>(cache.max_pages_per_req) * cache.page_size;
  const int key = r.k0 + threadIdx.x, ctx = cache.ctx_len[r.b];
  if (key < ctx) mass[r.b * capacity + key] += sum;
}

}  // namespace

size_t attn_mass_workspace_bytes() { return kMaxPairs * (sizeof(MassRecord) + 2 * kMKeys * sizeof(float)); }

cudaError_t launch_attn_mass(const csa2_cache& cache, int n_queries, const int32_t* q_start, const int32_t* q_pos,
                             int ratio, int H, float scale, const float* lse, float* mass, void* ws,
                             const CUtensorMap& q_map, int num_sms, uint64_t wait_ns, cudaStream_t stream) {
  static ContextMemo attrs;
  const size_t smem = sizeof(MassSmem) + 1024;
  cudaError_t e = attrs.once([&] {
    return cudaFuncSetAttribute(attn_mass_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  });
  if (e != cudaSuccess) return e;
  const DenseArgs a = {cache, q_start, q_pos, n_queries, ratio, H, 1, 1};
  const int pairs = min(kMaxPairs, num_sms / 2);
  attn_mass_kernel<<<2 * pairs, kMThreads, smem, stream>>>(a, q_map, scale, lse, mass, ws, wait_ns);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  attn_mass_join_kernel<<<pairs, kMKeys, 0, stream>>>(cache, mass, ws);
  return cudaGetLastError();
}

}  // namespace csa2
