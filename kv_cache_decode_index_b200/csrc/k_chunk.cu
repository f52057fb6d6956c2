// Dense attention of new tokens over the paged FP4 cache (K = V = the
// dequantised 512-channel row, shared by every head):
//   o = sum_e softmax_e(scale q . v_e) v_e   over the entries e that the query sees,
//   lse = log sum_e exp(scale q . v_e),
// on the tensor cores of pairs of CTAs: 128 query rows ((token, head) pairs of
// one request, 64 per CTA) over the keys in tiles of 256.
//
//   S = Q K^T   M = 128 rows, N = 256 keys, K = 512 channels (8 parts of 64)
//   O += P V    M = 128 rows, N = 2 x 256 channels, K = 256 keys (8 parts of 32)
//
// Both products take the dequantised row as operand B, once with the channels
// as K (K-major) and once with the keys as K (MN-major).  tcgen05 over a pair
// has each CTA hold one half of B's N: its 128 keys of the tile for S, its 256
// neighbouring channels of every key for O.  Why a pair with M = 128: 512 output
// channels of 128 rows in fp32 are a whole SM's tensor memory; over a pair they
// take half of each (256 columns), which leaves room for two score tiles (2 x
// 128), and N = 256 keeps the full rate that M = 128 has over a pair (64 cycles
// per MMA of K = 16; N = 128 takes 47, no less than N = 64).
//
// Roles: warps 0-3 softmax (thread = row and half of the tile's keys), warps
// 4-11 dequantisation (packed rows from L2 into registers one half tile ahead,
// fp16 operands into a ring of 16 KB slots), warp 12 of the leader issues the
// MMAs in the order S(0), S(1), O(0), S(2), O(1), ...: the softmax of a tile has
// the time of the next tile's S and of the previous tile's O.
//
// The rows are stored times 2^-8 (an E4M3 code shifted into fp16 is 2^-8 of its
// value; the product with E2M1 stays exact in fp16, subnormals included);
// the scores' factor and the output's carry the 2^8.
// P is held in fp16 relative to a reference 2^7 below the row's maximum, and the
// reference is raised only when a row's new maximum is more than 2^15 above it:
// P stays below 2^15, inside fp16, and O, which lies in tensor memory, is rarely
// rescaled.  The 2^7 are for the other end: weights down to 2^-32 of the largest
// count in P as they do in the fp32 sum.  With a reference at the maximum itself
// they were lost from 2^-25 on: of 262,143 equal entries 17.4 nats below one other,
// all (0.7 % of the weight).  The room costs one subtraction a tile.
//
// 1,024 tokens x 64 heads over 32,768 entries: 3.92 ms for a call by itself, 0.66 of
// the tensor cores' measured rate, and 4.31 ms in calls back to back (0.60), where
// the power limit lowers the clock; one token of 8 requests x 64 heads over 65,536:
// 163 us with the join.  A step of 256 keys takes 6,800 to 7,500 cycles against
// 4,096 of products; what bounds it is the shared-memory pipe (70 % of its
// wavefronts are taken: two dequantised operands, the probabilities, the score
// tiles).
// Taking the maximum and the probabilities in one pass over the score tile, with
// a repeat when a maximum rises, was slower (4.11 ms).
#include <cuda_bf16.h>
#include <stddef.h>

#include "launch.h"
#include "pair_operands.cuh"

namespace csa2 {

namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxPairs = 74;                // ranges of one launch: pairs of CTAs on 148 SMs
constexpr int kPairRows = 128;               // query rows of a tile

// What a pair says of its range, for the launch that joins cut tiles.
struct RangeRecord {
  long long lo;                              // first step
  long long tile_lo, tile_hi;                // the steps of the tile that it starts in, the tile's cost left out
  int q0, tokens;                            // that tile's queries
  int pairs, pad;                            // pairs that have work
};

// Workspace: the records, then two partial results per pair (the tile that
// the range starts inside, the tile that it ends inside): 512 sums of each of
// 128 rows, four channels of all rows together (the writers' lanes are rows),
// then the rows' references (log2) and their sums.
struct ChunkWorkspace {
  RangeRecord* rec;
  float* part;
};
__host__ __device__ inline ChunkWorkspace split_chunk_ws(void* ws) {
  ChunkWorkspace w;
  w.rec = static_cast<RangeRecord*>(ws);
  w.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kMaxPairs * sizeof(RangeRecord));
  return w;
}
static_assert(kMaxPairs * sizeof(RangeRecord) % 16 == 0, "partial results are read 16 bytes at a time");
constexpr size_t kPartialFloats = static_cast<size_t>(kPairRows) * (kKvDim + 2);
// Partial result `which` (0: tile started inside, 1: tile ended inside) of a pair.
__host__ __device__ inline float* partial_of(const ChunkWorkspace& w, int pair, int which) {
  return w.part + (2 * static_cast<size_t>(pair) + which) * kPartialFloats;
}
__host__ __device__ inline int partial_at(int row, int ch) { return ((ch >> 2) * kPairRows + row) * 4 + (ch & 3); }
constexpr int kPartialRef = kPairRows * kKvDim, kPartialSum = kPartialRef + kPairRows;

constexpr int kGSoftWarps = 4, kGDeqWarps = 8;
constexpr int kGThreads = (kGSoftWarps + kGDeqWarps + 1) * 32;   // 416
constexpr int kGKeys = 256;                  // keys of a tile
constexpr int kGRows = 64;                   // query rows of one CTA
constexpr int kGPairs = 4;                   // ring: pairs of slots
constexpr int kSlotBytes = 16384;
constexpr int kPairBytes = 2 * kSlotBytes;
constexpr uint32_t kGTmemCols = 512;
constexpr uint32_t kOCol = 0, kSCol = 256;   // O: 2 x 128 columns; S: 2 buffers of 128
constexpr uint32_t kIdescS = idesc_f16_f32(128, 256, false, false);
constexpr uint32_t kIdescO = idesc_f16_f32(128, 256, false, true);
constexpr int kBarSoft = 1;
constexpr float kBelow = 7.0f;               // log2 units from a row's maximum down to a new reference
constexpr float kRaise = kBelow + 8.0f;      // ... that a maximum may lie above the reference
constexpr int kStageRow = kKvDim * 2 + 16;     // bytes between staged output rows
constexpr float kFar = 1048576.0f;           // 2^20: fp32 values are less than 1/8 apart below it

struct __align__(1024) PairSmem {
  uint8_t q[8][kGRows * 128];                // A of S: 64-channel parts
  uint8_t p[4][kGRows * 128];                // A of O: 64-key parts
  union {
    uint8_t ring[kGPairs][kPairBytes];
    DensePlanSmem<kGThreads> plan;           // before the first pair is filled
  };
  float xchg[2][128];
  float row_scale[kGRows];
  uint64_t full[kGPairs];                    // leader: both CTAs' dequantisation
  uint64_t empty[kGPairs];
  uint64_t s_full[2];
  uint64_t p_full;                           // leader: both CTAs' softmax
  uint64_t o_done;
  uint64_t q_full;                           // leader
  uint64_t drain;
  uint32_t tmem_base;
  volatile int abort_flag;
};
static_assert(sizeof(PairSmem::q) + sizeof(PairSmem::p) >= kGRows * kStageRow, "staged output rows");
static_assert(offsetof(PairSmem, p) == sizeof(PairSmem::q), "P lies behind Q");
static_assert(sizeof(PairSmem) + 1024 <= 227 * 1024, "shared memory of one CTA");

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Bulk copy of a row from shared to global memory (16-byte aligned, a multiple
// of 16 bytes), and the wait for the thread's copies to have read their source.
__device__ __forceinline__ void bulk_store_1d(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// Descriptor of an MN-major operand with the 128-byte swizzle: 64 elements of
// N contiguous per K row (128 bytes), 8-row groups 1024 bytes apart, the next
// 64 elements of N `atom` bytes on.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr, uint32_t atom) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(atom >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGThreads, 1)
    chunk_attn_kernel(const DenseArgs a, const __nv_bfloat16* __restrict__ q, float scale,
                           __nv_bfloat16* __restrict__ out, float* __restrict__ lse, void* ws, uint64_t wait_ns) {
  extern __shared__ uint8_t smem_raw[];
  PairSmem& S = *reinterpret_cast<PairSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1;
  const csa2_cache& cache = a.cache;
  const ChunkWorkspace wsp = split_chunk_ws(ws);
  pdl_launch_dependents();     // the joining launch: it waits for this one's end

  if (tid == 0) {
    for (int s = 0; s < kGPairs; ++s) {
      mbar_init(&S.full[s], 8);                  // four warps of each CTA
      mbar_init(&S.empty[s], 1);
    }
    mbar_init(&S.s_full[0], 1);
    mbar_init(&S.s_full[1], 1);
    mbar_init(&S.p_full, 2 * kGSoftWarps);
    mbar_init(&S.o_done, 1);
    mbar_init(&S.q_full, 2 * kGSoftWarps);
    mbar_init(&S.drain, 1);
    S.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 12) tmem_alloc_pair(&S.tmem_base, kGTmemCols);
  const DensePlan plan = dense_plan<kGThreads, kGKeys>(a, S.plan, pair, gridDim.x >> 1, kKChunk);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync_all();
  const uint32_t tmem = S.tmem_base;
  if (tid == 0 && rank == 0) {
    RangeRecord r = {plan.lo, plan.lo, plan.lo, 0, 0, plan.ctas, 0};
    if (plan.lo < plan.hi) {
      const DenseTile t = dense_tile(a, plan.start);
      r.tile_lo = plan.lo - plan.off + kTileCost;
      r.tile_hi = r.tile_lo + dense_steps<kGKeys>(t);
      r.q0 = t.q0;
      r.tokens = t.tokens;
    }
    wsp.rec[pair] = r;
  }

  if (warp < kGSoftWarps) {
    // ================= softmax =================
    const int row = tid & 63, khalf = tid >> 6;      // row of this CTA, keys khalf*128 .. +127 of the tile
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t p_full = map_rank(smem_u32(&S.p_full), 0), q_full = map_rank(smem_u32(&S.q_full), 0);
    const float sign = scale < 0.0f ? -1.0f : 1.0f;
    int g = 0;                                       // tiles so far
    bool ok = true;
    long long pos = plan.lo;
    int off = plan.off;
    TilePlace place = plan.start;
    while (ok && pos < plan.hi) {
      const DenseTile T = dense_tile(a, place);
      const int steps = dense_steps<kGKeys>(T);
      const TilePart part_of = tile_part(steps, off, plan.hi - pos);
      const int first = part_of.first, seg = part_of.n;
      pos += part_of.counted;
      off = 0;
      if (pos < plan.hi) place = next_tile(a, place);
      if (seg == 0) continue;
      const int rows = T.tokens * a.heads;           // of the pair
      const int own = static_cast<int>(rank) * kGRows + row;
      // (a lane without a row follows the tile's keys: with 0 it would hold its
      // warp to the masked form at every tile)
      const bool real = own < rows;
      const int seen_keys = real ? seen_by(a.q_pos[T.q0 + own / a.heads], a.ratio, T.ctx) : T.keys;
      // A tile's keys of this thread lie on one page; its id is looked up a tile
      // ahead.  Keys under a bad one take no part (the dequantisation records it).
      // The look-up costs a long chunk 0.9 %; one scan of the segment's pages with
      // look-ups only where it finds a bad one cost 1.1 %, and up to 7 % in calls of
      // its own or with its result in shared memory.
      auto page_of = [&](int t) {
        const int key = (first + t) * kGKeys + khalf * 128;
        return key < T.keys ? cache.page_table[static_cast<long long>(T.b) * cache.max_pages_per_req + key / cache.page_size]
                            : 0;
      };
      int page = page_of(0);
      load_query_rows<kGRows, kGSoftWarps, kPerRow>(q, static_cast<long long>(T.q0) * a.heads + static_cast<int>(rank) * kGRows,
                                           rows - static_cast<int>(rank) * kGRows, kGRows, sign, S.q[0], warp, lane,
                                           [&](int r, uint32_t top) {
                                             S.row_scale[r] = fabsf(scale) * query_row_down(top) * kLog2e * kRowScale;
                                           });
      fence_proxy_async_smem();
      named_bar_sync(kBarSoft, kGSoftWarps * 32);
      if (lane == 0) mbar_arrive_cluster(q_full);
      const float c2 = S.row_scale[row];
      float m_ref = -INFINITY, l = 0.0f;

      for (int t = 0; t < seg; ++t, ++g) {
        const int key0 = (first + t) * kGKeys + khalf * 128;
        const int lim = page >= 0 && page < cache.num_pages ? seen_keys : min(seen_keys, key0);
        page = page_of(t + 1);                       // (nothing is read behind the tile's keys)
        const uint32_t s_addr = tmem + lane_base + kSCol + (g & 1) * 128;
        if (!mbar_wait_all(&S.s_full[g & 1], (g >> 1) & 1, wait_ns)) ok = false;
        ok = !named_bar_or(kBarSoft, kGSoftWarps * 32, !ok || S.abort_flag != 0);
        if (!ok) break;
        tc_fence_after();
        const bool masked = __any_sync(0xffffffffu, lim < key0 + 128);
        const bool seen = __any_sync(0xffffffffu, real && lim > key0);   // by any row of this warp
        // tensor-memory loads run one part ahead of the arithmetic
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (seen) {
          uint32_t r[2][32];
          tmem_ld_32x32b_x32(s_addr, r[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_ld_wait();
            if (c < 3) tmem_ld_32x32b_x32(s_addr + (c + 1) * 32, r[(c + 1) & 1]);
            if (masked) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (key0 + c * 32 + j < lim) mx4[j & 3] = fmaxf(mx4[j & 3], __uint_as_float(r[c & 1][j]));
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) mx4[j & 3] = fmaxf(mx4[j & 3], __uint_as_float(r[c & 1][j]));
            }
          }
        }
        float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        S.xchg[g & 1][tid] = mx;
        named_bar_sync(kBarSoft, kGSoftWarps * 32);
        mx = fmaxf(mx, S.xchg[g & 1][tid ^ 64]);
        const float m_new = mx == -INFINITY ? -INFINITY : mx * c2;
        float f = 1.0f;
        // (the difference: above 2^27, where values are 16 apart, m_ref + kRaise can
        // round up to the next one, and probabilities of 2^16 would leave fp16)
        if (m_new - m_ref > kRaise) {
          f = m_ref == -INFINITY ? 0.0f : ex2(m_ref - (m_new - kBelow));
          m_ref = m_new - kBelow;
          l *= f;
        }
        const float ref = m_ref == -INFINITY ? 0.0f : m_ref;
        // Far from 0, s * c2 - ref has to be rounded like ref was.  One of the two
        // factors is 1: the row's bits are those of the plain form unless it is far
        // itself, whatever the warp's other rows are.
        const bool far = !(fabsf(ref) < kFar);
        const float pre = far ? c2 : 1.0f, post = far ? 1.0f : c2;
        const bool careful = __any_sync(0xffffffffu, lim < key0 + 128 || far);
        // the probabilities wait in registers (fp16) for the previous tile's P to be free
        uint32_t h[64];
        if (!seen) {
#pragma unroll
          for (int j = 0; j < 64; ++j) h[j] = 0u;
        } else {
          uint32_t r[2][16];
          float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          tmem_ld_32x32b_x16(s_addr, r[0]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            tmem_ld_wait();
            if (c < 7) tmem_ld_32x32b_x16(s_addr + (c + 1) * 16, r[(c + 1) & 1]);
            if (careful) {
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                const int key = key0 + c * 16 + j;
                const float s0 = __uint_as_float(r[c & 1][j]), s1 = __uint_as_float(r[c & 1][j + 1]);
                const float p0 = key < lim ? ex2(fmaf(__fmul_rn(s0, pre), post, -ref)) : 0.0f;
                const float p1 = key + 1 < lim ? ex2(fmaf(__fmul_rn(s1, pre), post, -ref)) : 0.0f;
                sum[(j >> 1) & 3] += p0 + p1;
                h[c * 8 + (j >> 1)] = pack_half2(p0, p1);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                const float p0 = ex2(fmaf(__uint_as_float(r[c & 1][j]), c2, -ref));
                const float p1 = ex2(fmaf(__uint_as_float(r[c & 1][j + 1]), c2, -ref));
                sum[(j >> 1) & 3] += p0 + p1;
                h[c * 8 + (j >> 1)] = pack_half2(p0, p1);
              }
            }
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        // P and O of the previous tile are free once its product is done
        if (t > 0) {
          if (!mbar_wait_all(&S.o_done, (g - 1) & 1, wait_ns)) ok = false;
          tc_fence_after();
          if (ok && __any_sync(0xffffffffu, f != 1.0f)) {
#pragma unroll 1
            for (int c = 0; c < 256; c += 16) {
              uint32_t r[16];
              tmem_ld_32x32b_x16(tmem + lane_base + kOCol + c, r);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * f);
              tmem_st_32x32b_x16(tmem + lane_base + kOCol + c, r);
            }
            tmem_st_wait();
          }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j)
          *reinterpret_cast<uint4*>(S.p[khalf * 2 + (j >> 3)] + row * 128 + (((j & 7) ^ (row & 7)) << 4)) =
              make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(p_full);
      }
      // ---- the segment's rows (a warp whose wait ran out above comes here too: the four leave together) ----
      ok = ok && mbar_wait_all(&S.o_done, (g - 1) & 1, wait_ns);
      ok = !named_bar_or(kBarSoft, kGSoftWarps * 32, !ok);
      if (!ok) break;
      tc_fence_after();
      S.xchg[g & 1][tid] = l;
      named_bar_sync(kBarSoft, kGSoftWarps * 32);
      l = S.xchg[g & 1][row] + S.xchg[g & 1][row + 64];
      const int pr = own;
      const bool whole = seg == steps;
      const float inv = whole ? (l > 0.0f ? kRowScale / l : (l == 0.0f ? 0.0f : l)) : kRowScale;
      const long long orow = static_cast<long long>(T.q0) * a.heads + pr;
      float* part = partial_of(wsp, pair, first > 0 ? 0 : 1);
      if (whole) {
        // Rows of bf16 into the space of Q and P (every product that read them
        // is done), 16 bytes apart from a multiple of 128 so that the lanes'
        // rows fall into different banks, then one bulk copy a row.
        uint8_t* stage = S.q[0];
#pragma unroll
        for (int c = 0; c < 256; c += 32) {
          uint32_t r[32], h[16];
          tmem_ld_32x32b_x32(tmem + lane_base + kOCol + c, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const __nv_bfloat162 b =
                __floats2bfloat162_rn(__uint_as_float(r[2 * j]) * inv, __uint_as_float(r[2 * j + 1]) * inv);
            h[j] = *reinterpret_cast<const uint32_t*>(&b);
          }
          const int ch = khalf * 256 + c;            // the upper lanes hold the other CTA's channels
          uint4* dst = reinterpret_cast<uint4*>(stage + row * kStageRow + ch * 2);
#pragma unroll
          for (int j = 0; j < 4; ++j) dst[j] = make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
        }
        fence_proxy_async_smem();
        named_bar_sync(kBarSoft, kGSoftWarps * 32);
        if (tid < kGRows && pr < rows) {
          bulk_store_1d(out + orow * kKvDim, stage + row * kStageRow, kKvDim * 2);
          bulk_store_wait_read();
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < 256; c += 32) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(tmem + lane_base + kOCol + c, r);
          tmem_ld_wait();
          if (pr < rows) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<float4*>(part + partial_at(pr, khalf * 256 + c + 4 * j)) = make_float4(__uint_as_float(r[4 * j]) * inv, __uint_as_float(r[4 * j + 1]) * inv,
                                   __uint_as_float(r[4 * j + 2]) * inv, __uint_as_float(r[4 * j + 3]) * inv);
          }
        }
      }
      if (khalf == 0 && pr < rows) {
        if (!whole) {
          part[kPartialRef + pr] = m_ref;
          part[kPartialSum + pr] = l;
        } else if (lse != nullptr) {
          lse[orow] = l == 0.0f ? -INFINITY : (m_ref + log2f(l)) * kLn2;
        }
      }
      tc_fence_before();
      named_bar_sync(kBarSoft, kGSoftWarps * 32);    // Q, the row table and O are free
    }
    if (!ok) {
      if (lane == 0) report_error(cache.err_word, CSA2_ERR_TIMEOUT, kKChunk, static_cast<int>(rank), g);
      S.abort_flag = 1;
    }
  } else if (warp < kGSoftWarps + kGDeqWarps) {
    // ================= dequantisation =================
    // Four warps fill two neighbouring slots (a pair) at a time; group grp
    // takes pairs grp and grp + 2 of a half tile (8 slots).  A pair has to be
    // filled within the time of the five slots before it: with two warps to a
    // pair (all four pairs under way at once) that was the limit.  A granule is
    // 32 channels of a key (16 code bytes).  A warp's load takes 8 keys x 64
    // bytes for K, 4 keys x 128 bytes for V (this CTA's channels are 256
    // neighbours): few cache lines an instruction, which the L1 looks up one by
    // one.  A quarter warp holds 4 keys x 2 neighbouring granules: its 16-byte
    // stores fall into eight different chunks.
    const int dw = warp - kGSoftWarps, grp = dw >> 2, wi = dw & 3;
    // K: keys krow + 32 i, granule kg of slot ksel of the pair
    const int krow = wi * 8 + ((lane >> 3) & 1) * 4 + (lane & 3), kg = (lane >> 2) & 1, ksel = lane >> 4;
    // V: keys vkey + 16 i of the pair's 64, granule vg of this CTA's 8
    const int vkey = wi * 4 + (lane & 3), vg = (lane >> 3) * 2 + ((lane >> 2) & 1);
    const int k_code = (2 * grp + ksel) * 32 + kg * 16, k_sc = (2 * grp + ksel) * 4 + kg * 2;
    const int v_code = static_cast<int>(rank) * 128 + vg * 16, v_sc = static_cast<int>(rank) * 16 + vg * 2;
    const uint32_t k_dst = krow * 128, v_dst = (vg >> 1) * 4096 + vkey * 128;
    const int k_c = kg * 4, v_c = (vg & 1) * 4;

    // The pages of a tile's two blocks of 128 keys are looked up a tile ahead:
    // fetch reads the table, resolve (half a tile later) turns the entries into
    // first cache rows, or -1: not seen by the tile, or a bad page (recorded).
    struct Blocks {
      int page[2], off[2];
    };
    struct Rows {
      int row[2];
    };
    auto fetch = [&](const DenseTile& T, int tile) {
      Blocks x;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int key = tile * kGKeys + b * 128;
        const int slot = key / cache.page_size;
        x.page[b] = -2;
        x.off[b] = key - slot * cache.page_size;
        if (key < T.keys)
          x.page[b] = cache.page_table[static_cast<long long>(T.b) * cache.max_pages_per_req + slot];
      }
      return x;
    };
    auto resolve = [&](const DenseTile& T, int tile, const Blocks& x) {
      Rows r;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const bool seen = tile * kGKeys + b * 128 < T.keys, good = x.page[b] >= 0 && x.page[b] < cache.num_pages;
        if (seen && !good) report_error(cache.err_word, CSA2_ERR_DEVICE_BOUNDS, kKChunk, T.b, tile * kGKeys + b * 128);
        r.row[b] = seen && good ? x.page[b] * cache.page_size + x.off[b] : -1;
      }
      return r;
    };
    // Where a lane's 2 x 4 granules of a half tile lie: the codes and scales of
    // each pair's first one, and the keys between two of a pair.  Keys that are
    // not there read row 0 and a scale of 0 (mask): no branch lies between two
    // granules, so their conversions overlap.
    struct Half {
      const uint8_t *codes[2], *scales[2];
      uint32_t mask[2];
      int step;
    };
    auto half_k = [&](const Rows& rows) {
      const int base = rank == 0 ? rows.row[0] : rows.row[1];
      const long long r = max(base, 0) + krow;
      const uint32_t mask = base < 0 ? 0u : 0x7F7Fu;
      const uint8_t *c = cache.kv_codes + r * kKvCodeBytes + k_code, *x = cache.kv_scales + r * kKvScaleBytes + k_sc;
      return Half{{c, c + 128}, {x, x + 16}, {mask, mask}, 32};
    };
    auto half_v = [&](const Rows& rows) {
      Half h;
#pragma unroll
      for (int b = 0; b < 2; ++b) {                  // a pair's 64 keys lie in one block of 128
        const long long r = max(rows.row[b], 0) + grp * 64 + vkey;
        h.codes[b] = cache.kv_codes + r * kKvCodeBytes + v_code;
        h.scales[b] = cache.kv_scales + r * kKvScaleBytes + v_sc;
        h.mask[b] = rows.row[b] < 0 ? 0u : 0x7F7Fu;
      }
      h.step = 16;
      return h;
    };
    uint4 codes[8];                                  // the lane's granules of the half tile in turn
    uint32_t sc[8], mask[2];                         // (the mask is applied at use: here it would wait for the load)
    auto load = [&](const Half& h, int i) {
      codes[i] = *reinterpret_cast<const uint4*>(h.codes[i >> 2] + (i & 3) * h.step * kKvCodeBytes);
      sc[i] = *reinterpret_cast<const uint16_t*>(h.scales[i >> 2] + (i & 3) * h.step * kKvScaleBytes);
      mask[i >> 2] = h.mask[i >> 2];
    };
    int n = grp;                                     // this group's next pair in the order of all pairs
    bool ok = true;
    // Granules 4 p .. 4 p + 3 into a pair of slots; their registers then receive
    // those of the next half tile.
    auto store_pair = [&](int p, bool keys, const Half& next) {
      const int x4 = n % kGPairs;
      ok = ok && mbar_wait_all(&S.empty[x4], ((n / kGPairs) & 1) ^ 1, wait_ns);
      n += 2;
      if (ok) {
        uint8_t *d0, *d1;                            // of granules 4 p, 4 p + 1 and of 4 p + 2, 4 p + 3
        if (keys) {
          d0 = S.ring[x4] + ksel * kSlotBytes + k_dst;
          d1 = d0 + 64 * 128;
        } else {
          d0 = S.ring[x4] + v_dst;
          d1 = d0 + kSlotBytes;
        }
        const uint32_t step = keys ? 32 * 128 : 16 * 128;
        const int c0 = keys ? k_c : v_c, x = keys ? krow & 7 : vkey & 7;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 o[4];
          dequant_32(codes[4 * p + i], sc[4 * p + i] & mask[p], o);
          uint8_t* dst = (i < 2 ? d0 : d1) + (i & 1) * step;
#pragma unroll
          for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(dst + (((c0 + j) ^ x) << 4)) = o[j];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) load(next, 4 * p + i);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_rank(smem_u32(&S.full[x4]), 0));
      }
    };
    auto store_half = [&](bool keys, const Half& next) {
      store_pair(0, keys, next);
      store_pair(1, keys, next);
    };

    long long pos = plan.lo;
    int off = plan.off;
    // the order of the MMAs: K(0), then K(t), V(t - 1), and V of the last tile
    TilePlace place = plan.start;
    DenseTile T = {};
    int first = 0, seg = 0;                          // the tile's steps in this range
    auto next_part = [&]() {                         // advances to a tile with steps in the range, if there is one
      for (seg = 0; seg == 0 && pos < plan.hi; off = 0) {
        T = dense_tile(a, place);
        const TilePart x = tile_part(dense_steps<kGKeys>(T), off, plan.hi - pos);
        first = x.first;
        seg = x.n;
        pos += x.counted;
        if (pos < plan.hi) place = next_tile(a, place);
      }
    };
    Rows cur = {{-1, -1}};                           // of the tile whose K comes next
    next_part();
    if (seg > 0) {
      cur = resolve(T, first, fetch(T, first));
      const Half head = half_k(cur);
#pragma unroll
      for (int i = 0; i < 8; ++i) load(head, i);
    }
    while (ok && seg > 0) {
      Rows prev = cur;
      for (int t = 0; ok && t < seg; ++t) {
        const Blocks ahead = fetch(T, first + t + 1);  // (nothing is read behind the tile's keys)
        if (t > 0) store_half(true, half_v(prev));
        else store_half(true, seg > 1 ? half_k(resolve(T, first + 1, ahead)) : half_v(cur));
        const Rows next = resolve(T, first + t + 1, ahead);
        if (t > 0) store_half(false, t + 1 < seg ? half_k(next) : half_v(cur));
        prev = cur;
        cur = next;
      }
      next_part();
      if (seg > 0) {
        cur = resolve(T, first, fetch(T, first));
        store_half(false, half_k(cur));
      } else {
        store_half(false, half_v(prev));             // (nothing comes after it: loaded once more)
      }
    }
    if (!ok && lane == 0) {
      report_error(cache.err_word, CSA2_ERR_TIMEOUT, kKChunk, static_cast<int>(rank), -n);
      S.abort_flag = 1;
    }
  } else if (rank == 0) {
    // ================= MMA issuer =================
    const bool issue = elect_one();
    const uint64_t q_desc = sw128_kmajor_desc(smem_u32(S.q[0])), p_desc = sw128_kmajor_desc(smem_u32(S.p[0]));
    const uint64_t k_desc = sw128_kmajor_desc(smem_u32(S.ring[0]));
    const uint64_t v_desc = sw128_mnmajor_desc(smem_u32(S.ring[0]), 4096);
    int s = 0, g = 0, segs = 0;                      // pair of slots in turn and its phase
    uint32_t phase = 0;
    bool ok = true;
    auto pair_ready = [&]() {
      ok = mbar_wait_cluster_all(&S.full[s], phase, wait_ns);
      tc_fence_after();
      return ok;
    };
    auto next_pair = [&]() {
      __syncwarp();
      if (++s == kGPairs) {
        s = 0;
        phase ^= 1;
      }
    };
    auto scores = [&](int buf) {
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        if (!pair_ready()) return;
        if (issue) {
          const uint64_t ad = q_desc + c * (2 * kGRows * 128 / 16), bd = k_desc + s * (kPairBytes / 16);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_f16_pair(tmem + kSCol + buf * 128, ad + (kk >> 2) * (kGRows * 128 / 16) + (kk & 3) * 2,
                          bd + (kk >> 2) * (kSlotBytes / 16) + (kk & 3) * 2, kIdescS, (c | kk) > 0 ? 1u : 0u);
          umma_commit_pair(&S.empty[s]);
          if (c == 3) umma_commit_pair(&S.s_full[buf]);
        }
        next_pair();
      }
    };
    auto output = [&](int tile, bool first) {        // tile: running number
      ok = mbar_wait_cluster_all(&S.p_full, tile & 1, wait_ns);
      tc_fence_after();
#pragma unroll 1
      for (int j = 0; ok && j < 4; ++j) {
        if (!pair_ready()) return;
        if (issue) {
          const uint64_t ad = p_desc + j * (kGRows * 128 / 16), bd = v_desc + s * (kPairBytes / 16);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)             // 16 of the pair's 64 keys
#pragma unroll
            for (int x = 0; x < 2; ++x)
              umma_f16_pair(tmem + kOCol + x * 128, ad + 2 * kk,
                            bd + (kk >> 1) * (kSlotBytes / 16) + (kk & 1) * (2048 / 16) + x * (8192 / 16), kIdescO,
                            first && (j | kk) == 0 ? 0u : 1u);
          umma_commit_pair(&S.empty[s]);
          if (j == 3) umma_commit_pair(&S.o_done);
        }
        next_pair();
      }
    };
    TilePlace place = plan.start;
    long long pos = plan.lo;
    int off = plan.off;
    for (; ok && pos < plan.hi; off = 0) {
      const TilePart x = tile_part(dense_steps<kGKeys>(dense_tile(a, place)), off, plan.hi - pos);
      const int seg = x.n;
      pos += x.counted;
      if (pos < plan.hi) place = next_tile(a, place);
      if (seg == 0) continue;
      ok = mbar_wait_cluster_all(&S.q_full, segs & 1, wait_ns);
      ++segs;
      tc_fence_after();
      for (int t = 0; ok && t < seg; ++t, ++g) {
        scores(g & 1);
        if (ok && t > 0) output(g - 1, t == 1);
      }
      if (ok) output(g - 1, seg == 1);
    }
    if (lane == 0 && !ok) {
      report_error(cache.err_word, CSA2_ERR_TIMEOUT, kKChunk, -1, g);
      S.abort_flag = 1;
    }
    __syncwarp();
    if (issue) umma_commit_pair(&S.drain);           // the lane that issued: its commits track its own operations
    (void)mbar_wait_all(&S.drain, 0, kWaitLimitNs);
  } else {
    if (lane == 0) (void)mbar_wait(&S.drain, 0, 4 * kWaitLimitNs);   // the leader's last arrival here
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();          // every MMA has completed, no barrier of the other CTA is touched after this
  if (warp == 12) tmem_release_pair(tmem, kGTmemCols);
}

// Joins the tiles that ranges cut: block (c, x, y) takes 32 rows and 64
// channels of the tile that range c starts inside, if c is the first to do so.
// A lane is a row, a warp 8 channels.
constexpr int kJoinRows = 32, kJoinChannels = 64, kJoinWarps = 8;

__global__ void __launch_bounds__(kJoinWarps * 32)
    chunk_join_kernel(int heads, __nv_bfloat16* __restrict__ out, float* __restrict__ lse, void* ws) {
  __shared__ float factor[kMaxPairs][kJoinRows], total[kMaxPairs][kJoinRows], red[kJoinWarps][kJoinRows];
  static_assert(kMaxPairs <= kJoinWarps * 32, "a thread per range");
  pdl_wait();
  const ChunkWorkspace wsp = split_chunk_ws(ws);
  const int c = blockIdx.x;
  const RangeRecord r = wsp.rec[c];
  if (c >= r.pairs || r.lo <= r.tile_lo || wsp.rec[c - 1].lo > r.tile_lo) return;
  if (static_cast<int>(blockIdx.z) * kJoinRows >= r.tokens * heads) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.z * kJoinRows + lane;
  const int ch = blockIdx.y * kJoinChannels + warp * 8;
  // parts of the tile: its head is range c - 1's, which ended (or also began)
  // with it, then those of the ranges that start before its end (they ascend)
  const int k = threadIdx.x;
  const int parts = 1 + __syncthreads_count(k >= c && k < r.pairs && wsp.rec[min(k, r.pairs - 1)].lo < r.tile_hi);
  auto part_of = [&](int i) { return partial_of(wsp, c - 1 + i, i == 0 ? 1 : 0); };
  // the rows' references and sums: the warps share the parts, so that all of a row's
  // loads are in flight together
  float m = -INFINITY;
#pragma unroll 4
  for (int i = warp; i < parts; i += kJoinWarps) {
    const float* part = part_of(i);
    factor[i][lane] = part[kPartialRef + row];       // (rows that are not there: never used)
    total[i][lane] = part[kPartialSum + row];
    m = fmaxf(m, factor[i][lane]);
  }
  red[warp][lane] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, red[w][lane]);
  const float ref = m == -INFINITY ? 0.0f : m;
  for (int i = warp; i < parts; i += kJoinWarps) factor[i][lane] = exp2f(factor[i][lane] - ref);
  __syncthreads();
  float l = 0.0f, o[8] = {};
#pragma unroll 8
  for (int i = 0; i < parts; ++i) {
    const float* part = part_of(i);
    const float f = factor[i][lane];
    l = fmaf(total[i][lane], f, l);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 v = *reinterpret_cast<const float4*>(part + partial_at(row, ch + 4 * h));
      o[4 * h] = fmaf(v.x, f, o[4 * h]);
      o[4 * h + 1] = fmaf(v.y, f, o[4 * h + 1]);
      o[4 * h + 2] = fmaf(v.z, f, o[4 * h + 2]);
      o[4 * h + 3] = fmaf(v.w, f, o[4 * h + 3]);
    }
  }
  if (row >= r.tokens * heads) return;
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
  const long long orow = static_cast<long long>(r.q0) * heads + row;
  uint32_t pk[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * h] * inv, o[2 * h + 1] * inv);
    pk[h] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(out + orow * kKvDim + ch) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
  if (lse != nullptr && ch == 0) lse[orow] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

size_t chunk_attn_workspace_bytes() {
  return kMaxPairs * (sizeof(RangeRecord) + 2 * kPartialFloats * sizeof(float));
}

cudaError_t launch_chunk_attn(const csa2_cache& cache, int n_queries, const int32_t* q_start, const int32_t* q_pos,
                              int ratio, const uint16_t* q, int H, float scale, uint16_t* out, float* lse, void* ws,
                              int num_sms, uint64_t wait_ns, cudaStream_t stream) {
  static ContextMemo attrs;
  const size_t smem = sizeof(PairSmem) + 1024;
  cudaError_t e = attrs.once([&] {
    return cudaFuncSetAttribute(chunk_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  });
  if (e != cudaSuccess) return e;
  const DenseArgs a = {cache, q_start, q_pos, n_queries, ratio, H, kPairRows / H};
  const int pairs = min(kMaxPairs, num_sms / 2);
  __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(out);
  chunk_attn_kernel<<<2 * pairs, kGThreads, smem, stream>>>(a, reinterpret_cast<const __nv_bfloat16*>(q), scale, o, lse, ws,
                                                            wait_ns);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pairs, kKvDim / kJoinChannels, kPairRows / kJoinRows);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // it waits for the ranges before reading
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_join_kernel, H, o, lse, ws);
}

}  // namespace csa2
