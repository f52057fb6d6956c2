// Eviction by accumulated attention weight: of a request's n entries keep the
// first `sink`, the last `recent`, and of those between the ones with the
// largest weight (ties: the lower index), in order; then move the kept rows to
// other pages.
//
// Selection: one cluster of CTAs per request.  Radix select over the order
// keys of the weights in digits of 11, 11 and 10 bits: every CTA counts its
// part of the entries into shared-memory bins, the CTAs read each other's bins
// (distributed shared memory) and find the same digit; after the third the
// threshold is exact, and the entries on it are taken from the lowest index
// on.  Each warp then counts and emits a consecutive part, so the output is
// sorted without a sort and without atomics whose order could show.  The
// weights are read once into shared memory where a CTA's part fits (up to 163,840
// entries a request), else five times, from L2 after the first: one request of
// 163,840 entries takes 35 us in all, one of 167,936 50 us.
// Moving: a warp per 8 rows, 417 bytes each, all their loads in flight.
#include <cooperative_groups.h>

#include "common.cuh"
#include "launch.h"

namespace csa2 {

namespace {

namespace cg = cooperative_groups;

constexpr int kEThreads = 1024;
constexpr int kEWarps = kEThreads / 32;
constexpr int kECluster = 8;
constexpr int kEBins = 2048;
constexpr int kEKeys = 20480;            // 80 KB: two CTAs per SM
constexpr int kMarkSource = 1 << 30;     // page marks: holds visible entries; below: uses as destination

// Order key of a weight: larger weight, larger key; NaN above everything, and
// -0 like +0.
__device__ __forceinline__ uint32_t weight_key(float f) {
  if (f != f) return 0xFFFFFFFFu;
  return order_key(f + 0.0f);
}

struct EvictSmem {
  uint32_t hist[3][kEBins];
  int warp_a[kEWarps], warp_b[kEWarps];
  int above, digit;          // of the pass's threshold bin
  int gt, eq;                // of this CTA's entries
  uint32_t keys[kEKeys];     // this CTA's order keys, when they fit
};

// Exclusive prefix sums of a and b over the block's threads.
__device__ __forceinline__ int2 block_scan2(int a, int b, EvictSmem& S) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int ua = __shfl_up_sync(0xffffffffu, ia, o), ub = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) ia += ua, ib += ub;
  }
  if (lane == 31) S.warp_a[warp] = ia, S.warp_b[warp] = ib;
  __syncthreads();
  if (warp == 0) {
    const int va = S.warp_a[lane], vb = S.warp_b[lane];
    int xa = va, xb = vb;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int ua = __shfl_up_sync(0xffffffffu, xa, o), ub = __shfl_up_sync(0xffffffffu, xb, o);
      if (lane >= o) xa += ua, xb += ub;
    }
    S.warp_a[lane] = xa - va;
    S.warp_b[lane] = xb - vb;
  }
  __syncthreads();
  return make_int2(S.warp_a[warp] + ia - a, S.warp_b[warp] + ib - b);
}

__global__ void __cluster_dims__(kECluster, 1, 1) __launch_bounds__(kEThreads)
    evict_select_kernel(const csa2_cache cache, const float* __restrict__ mass, int budget, int sink, int recent,
                        const int32_t* __restrict__ dst_pages, int dst_width, int32_t* __restrict__ kept,
                        int32_t* __restrict__ new_len, int32_t* __restrict__ marks) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  EvictSmem& S = *reinterpret_cast<EvictSmem*>(smem_raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int b = blockIdx.x / kECluster;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  const long long capacity = static_cast<long long>(cache.max_pages_per_req) * cache.page_size;
  const int raw = checked_ctx_len(cache, b, capacity, kKEvict, rank == 0 && tid == 0);
  const int n = max(raw, 0);
  const bool cut = n > budget;
  int32_t* out = kept + static_cast<long long>(b) * budget;
  const int all = rank * kEThreads + tid;               // thread of the cluster
  constexpr int kAll = kECluster * kEThreads;

  // pages: those that hold visible entries, and those that will receive some
  const int32_t* src_tab = cache.page_table + static_cast<long long>(b) * cache.max_pages_per_req;
  for (int i = all; i < (n + cache.page_size - 1) / cache.page_size; i += kAll) {
    const int p = src_tab[i];
    if (p >= 0 && p < cache.num_pages) atomicOr(&marks[p], kMarkSource);
  }
  if (cut) {
    for (int i = all; i < (budget + cache.page_size - 1) / cache.page_size; i += kAll) {
      const int p = dst_pages[static_cast<long long>(b) * dst_width + i];
      if (p >= 0 && p < cache.num_pages) atomicAdd(&marks[p], 1);
    }
  }
  if (rank == 0 && tid == 0) new_len[b] = min(n, budget);

  if (!cut) {                                           // (the same for every CTA of the cluster)
    for (int j = all; j < budget; j += kAll) out[j] = j < n ? j : -1;
    return;
  }
  for (int j = all; j < sink; j += kAll) out[j] = j;
  for (int j = all; j < recent; j += kAll) out[budget - recent + j] = n - recent + j;
  const int want = budget - sink - recent;              // of the entries [sink, n - recent): more than that
  if (want == 0) return;

  for (int i = tid; i < 3 * kEBins; i += kEThreads) (&S.hist[0][0])[i] = 0u;
  __syncthreads();
  const int mid = n - recent - sink;
  const int per = (mid + kECluster - 1) / kECluster;
  const int c0 = sink + min(rank * per, mid), c1 = sink + min((rank + 1) * per, mid);
  const int ws = ((per + kEWarps - 1) / kEWarps + 31) & ~31;   // entries per warp
  const int w0 = min(c0 + warp * ws, c1), w1 = min(w0 + ws, c1);
  const float* m = mass + b * capacity;
  const bool cached = per <= kEKeys;
  if (cached) {
#pragma unroll 4
    for (int i = c0 + tid; i < c1; i += kEThreads) S.keys[i - c0] = weight_key(m[i]);
    __syncthreads();
  }
  auto key_of = [&](int i) { return cached ? S.keys[i - c0] : weight_key(m[i]); };

  uint32_t prefix = 0u, mask = 0u;
  int need = want;                                      // still to take among the keys on the prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t digits = pass == 2 ? 1023u : 2047u;
    uint32_t* hist = S.hist[pass];
    // (the hardware adds up the lanes of one bin: weights crowd, entries without any most of all)
#pragma unroll 4
    for (int i = w0 + lane; i < w1; i += 32) {
      const uint32_t k = key_of(i);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & digits], 1u);
    }
    cluster.sync();                                     // every CTA's bins are counted
    // thread t: bins 2047 - 2t and 2046 - 2t of all CTAs, from the top down
    const int hi_bin = kEBins - 1 - 2 * tid;
    int a = 0, c = 0;
#pragma unroll
    for (int r = 0; r < kECluster; ++r) {
      const uint2 two = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(hist, r) + hi_bin - 1);
      a += static_cast<int>(two.y);
      c += static_cast<int>(two.x);
    }
    const int before = block_scan2(a + c, 0, S).x;
    if (before < need && need <= before + a) S.above = before, S.digit = hi_bin;
    else if (before + a < need && need <= before + a + c) S.above = before + a, S.digit = hi_bin - 1;
    __syncthreads();
    need -= S.above;
    prefix |= static_cast<uint32_t>(S.digit) << shift;
    mask |= digits << shift;
    __syncthreads();                                    // S.above is read before the next pass writes it
  }

  // ---- counts of this warp's part: above the threshold, and on it ----
  int gt = 0, eq = 0;
#pragma unroll 4
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t k = key_of(i);
    gt += k > prefix;
    eq += k == prefix;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    gt += __shfl_xor_sync(0xffffffffu, gt, o);
    eq += __shfl_xor_sync(0xffffffffu, eq, o);
  }
  const int2 at = block_scan2(lane == 0 ? gt : 0, lane == 0 ? eq : 0, S);
  int gt_before = __shfl_sync(0xffffffffu, at.x, 0), eq_before = __shfl_sync(0xffffffffu, at.y, 0);
  if (warp == kEWarps - 1 && lane == 0) S.gt = gt_before + gt, S.eq = eq_before + eq;
  cluster.sync();
  for (int r = 0; r < rank; ++r) {
    const EvictSmem* o = cluster.map_shared_rank(&S, r);
    gt_before += o->gt;
    eq_before += o->eq;
  }
#pragma unroll 4
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < w1 ? key_of(i) : 0u;
    const uint32_t g = __ballot_sync(0xffffffffu, i < w1 && k > prefix);
    const uint32_t e = __ballot_sync(0xffffffffu, i < w1 && k == prefix);
    const uint32_t below = (1u << lane) - 1u;
    const int ge = gt_before + __popc(g & below), ee = eq_before + __popc(e & below);
    if ((g >> lane & 1u) || ((e >> lane & 1u) && ee < need)) out[sink + ge + min(ee, need)] = i;
    gt_before += __popc(g);
    eq_before += __popc(e);
  }
  cluster.sync();                                       // the other CTAs have read this one's counts
}

// Cache row of position t of a page table row, or -1 (recorded).
__device__ __forceinline__ int evict_row(const csa2_cache& c, const int32_t* table, int b, int t) {
  const int page = table[t / c.page_size];
  if (page < 0 || page >= c.num_pages) {
    report_error(c.err_word, CSA2_ERR_DEVICE_BOUNDS, kKEvict, b, t);
    return -1;
  }
  return page * c.page_size + t % c.page_size;
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 8;      // rows of one warp

__global__ void __launch_bounds__(kMoveThreads)
    evict_move_kernel(const csa2_cache cache, uint8_t* ik4_codes, uint8_t* ik4_scales, const float* __restrict__ mass,
                      int budget, const int32_t* __restrict__ dst_pages, int dst_width,
                      const int32_t* __restrict__ kept, float* __restrict__ mass_out, const int32_t* __restrict__ marks,
                      int groups) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5);
  const int b = static_cast<int>(w / groups), j0 = static_cast<int>(w % groups) * kMoveRows;
  if (b >= cache.batch) return;
  const long long capacity = static_cast<long long>(cache.max_pages_per_req) * cache.page_size;
  const int n = checked_ctx_len(cache, b, capacity, kKEvict, false);
  if (n <= budget) return;                              // left where it is

  // lanes 0..7: source and destination row of row j0 + lane
  int src = -1, dst = -1, pos = -1;
  const int j = j0 + lane;
  if (lane < kMoveRows && j < budget) {
    pos = kept[static_cast<long long>(b) * budget + j];
    src = evict_row(cache, cache.page_table + static_cast<long long>(b) * cache.max_pages_per_req, b, pos);
    dst = evict_row(cache, dst_pages + static_cast<long long>(b) * dst_width, b, j);
    if (dst >= 0) {
      const int mk = marks[dst / cache.page_size];
      if ((mk & kMarkSource) || (mk & (kMarkSource - 1)) > 1) {   // it holds visible entries, or is given twice
        report_error(cache.err_word, CSA2_ERR_DEVICE_BOUNDS, kKEvict, b, j);
        dst = -1;
      }
    }
  }
  if (mass_out != nullptr && dst >= 0 && src >= 0)
    mass_out[static_cast<long long>(b) * dst_width * cache.page_size + j] = mass[b * capacity + pos];

  // lane -> its 16 bytes of a row: 16 x codes, 2 x scales, 8 x indexer codes, 4 x FP4 indexer codes
  uint8_t* base = nullptr;
  int stride = 0;
  if (lane < 16) base = cache.kv_codes + lane * 16, stride = kKvCodeBytes;
  else if (lane < 18) base = cache.kv_scales + (lane - 16) * 16, stride = kKvScaleBytes;
  else if (lane < 26) base = cache.ik_codes + (lane - 18) * 16, stride = kIndexDim;
  else if (lane >= 28 && ik4_codes != nullptr) base = ik4_codes + (lane - 28) * 16, stride = CSA2_IK4_CODE_BYTES;
  {
    uint4 v[kMoveRows];
    uint32_t x[kMoveRows];
    int s[kMoveRows], d[kMoveRows];
#pragma unroll
    for (int r = 0; r < kMoveRows; ++r) {
      s[r] = __shfl_sync(0xffffffffu, src, r);
      d[r] = __shfl_sync(0xffffffffu, dst, r);
      if (s[r] < 0 || d[r] < 0) continue;
      if (base != nullptr) v[r] = *reinterpret_cast<const uint4*>(base + static_cast<long long>(s[r]) * stride);
      if (lane == 26) x[r] = cache.ik_exp[s[r]];
      if (lane < 2 && ik4_scales != nullptr)
        x[r] = *reinterpret_cast<const uint32_t*>(ik4_scales +
                                                  static_cast<long long>(s[r] / kTile) * CSA2_IK4_TILE_SCALE_BYTES +
                                                  block_scale_offset(s[r] % kTile, lane * 4));
    }
#pragma unroll
    for (int r = 0; r < kMoveRows; ++r) {
      if (s[r] < 0 || d[r] < 0) continue;
      if (base != nullptr) *reinterpret_cast<uint4*>(base + static_cast<long long>(d[r]) * stride) = v[r];
      if (lane == 26) cache.ik_exp[d[r]] = static_cast<uint8_t>(x[r]);
      if (lane < 2 && ik4_scales != nullptr)
        *reinterpret_cast<uint32_t*>(ik4_scales + static_cast<long long>(d[r] / kTile) * CSA2_IK4_TILE_SCALE_BYTES +
                                     block_scale_offset(d[r] % kTile, lane * 4)) = x[r];
    }
  }
}

}  // namespace

size_t evict_workspace_bytes(long long num_pages) { return (static_cast<size_t>(num_pages) * 4 + 15) / 16 * 16; }

cudaError_t launch_evict(const csa2_cache& cache, const csa2_ik4* ik4, const float* mass, int budget, int sink, int recent,
                         const int32_t* dst_pages, int dst_width, int32_t* kept, int32_t* new_len, float* mass_out,
                         void* ws, cudaStream_t stream) {
  static ContextMemo attrs;
  cudaError_t e = attrs.once([&] {
    return cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(sizeof(EvictSmem)));
  });
  if (e != cudaSuccess) return e;
  int32_t* marks = static_cast<int32_t*>(ws);
  e = cudaMemsetAsync(marks, 0, static_cast<size_t>(cache.num_pages) * 4, stream);
  if (e != cudaSuccess) return e;
  evict_select_kernel<<<cache.batch * kECluster, kEThreads, sizeof(EvictSmem), stream>>>(cache, mass, budget, sink, recent,
                                                                                       dst_pages, dst_width, kept, new_len,
                                                                                       marks);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int groups = (budget + kMoveRows - 1) / kMoveRows;
  const long long warps = static_cast<long long>(cache.batch) * groups;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((warps + kMoveThreads / 32 - 1) / (kMoveThreads / 32)));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // it waits for the selection before reading
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel, cache, ik4 ? ik4->codes : nullptr, ik4 ? ik4->scales : nullptr, mass,
                            budget, dst_pages, dst_width, static_cast<const int32_t*>(kept), mass_out,
                            static_cast<const int32_t*>(marks), groups);
}

}  // namespace csa2
