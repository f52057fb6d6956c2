// Dense attention of new tokens over the paged FP4 cache (K = V = the
// dequantised 512-channel row, shared by every head):
//   o = sum_e softmax_e(scale q . v_e) v_e   over the entries e that the query sees,
//   lse = log sum_e exp(scale q . v_e).
//
// Rows of a tile are (token, head) pairs of one request.  One pass over the
// keys in steps of 64 with the running maximum and sum of the softmax; the
// packed rows are copied one step ahead (cp.async), dequantised once in shared
// memory (exact in fp16) and used as K and as V.  Products on mma.sync
// m16n8k16 with fp32 sums; the probabilities are rounded to fp16 for P V (2^-12
// relative each, an eighth of the bf16 output's own rounding), their sum is
// taken in fp32 before that rounding.
// Long contexts with few rows are cut along the keys (dense_plan.cuh); a
// second launch joins the partial results.
#include <cuda_bf16.h>

#include "attn_tile.cuh"
#include "chunk_join.cuh"
#include "launch.h"

namespace csa2 {

namespace {

constexpr int kCThreads = 256;
constexpr int kCWarps = kCThreads / 32;
constexpr int kDimsPerWarp = kKvDim / kCWarps;   // 64 output channels per warp in P V
template <int MR>
struct ChunkSmem {
  static constexpr int HT = MR / 16;
  static constexpr int KG = kCWarps / HT;      // key groups in S
  static constexpr int KW = kChunk / KG;       // keys per warp in S
  static constexpr int NT = KW / 8;
  uint8_t q[MR * kRowBytes];
  uint8_t kv[kChunk * kRowBytes];
  uint8_t raw[kChunk * kKvCodeBytes];
  uint8_t raw_scale[kChunk * kKvScaleBytes];
  uint8_t p[MR * kPRowBytes];
  float red_max[KG][MR];
  float red_sum[KG][MR];
  float qscale[MR];
  int lim[MR];                                 // entries seen by each row
  DensePlanSmem<kCThreads> plan;
};

template <int MR>
__global__ void __launch_bounds__(kCThreads, MR == 16 ? 2 : 1)
    chunk_attn_kernel(const DenseArgs a, const __nv_bfloat16* __restrict__ q, float softmax_scale,
                      __nv_bfloat16* __restrict__ out, float* __restrict__ lse, void* ws) {
  using L = ChunkSmem<MR>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  L& S = *reinterpret_cast<L*>(smem_raw);
  const uint32_t q_sh = smem_u32(S.q), kv_sh = smem_u32(S.kv), p_sh = smem_u32(S.p);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ht = warp % L::HT, kg = warp / L::HT;
  const csa2_cache& cache = a.cache;
  const ChunkWorkspace wsp = split_chunk_ws(ws);

  const DensePlan plan = dense_plan<kCThreads, kChunk>(a, S.plan, blockIdx.x, gridDim.x, kKChunk);
  if (tid == 0) write_range_record<kChunk>(a, plan, &wsp.rec[blockIdx.x]);

  const int r0 = lane >> 2;
  const int h0 = ht * 16 + r0, h1 = h0 + 8;
  long long pos = plan.lo;
  int off = plan.off;
  TilePlace place = plan.start;
  while (pos < plan.hi) {
    const DenseTile T = dense_tile(a, place);
    const int steps = dense_steps<kChunk>(T);
    const int seg = static_cast<int>(min(static_cast<long long>(steps - off), plan.hi - pos));
    pos += seg;
    const int rows = T.tokens * a.heads;
    const int key_begin = off * kChunk, key_end = min(T.keys, (off + seg) * kChunk);
    const int32_t* ptab = cache.page_table + static_cast<long long>(T.b) * cache.max_pages_per_req;

    // rows of the page of step c, or -1 (recorded): its entries are left out
    auto first_row = [&](int c) {
      const int page = ptab[c / cache.page_size];
      if (page < 0 || page >= cache.num_pages) {
        if (tid == 0) report_error(cache.err_word, CSA2_ERR_DEVICE_BOUNDS, kKChunk, T.b, c);
        return -1;
      }
      return page * cache.page_size + c % cache.page_size;
    };
    auto issue = [&](int c) {
      const int row = first_row(c);
      if (row >= 0) {
        const int nk = min(kChunk, key_end - c);
        for (int g = tid; g < nk * kRowGran; g += kCThreads) {
          const int r = g / kRowGran, part = g - r * kRowGran;
          if (part < kCodeGran)
            cp_async16(smem_u32(S.raw) + r * kKvCodeBytes + ((part ^ (r & 7)) << 4),
                       cache.kv_codes + static_cast<long long>(row + r) * kKvCodeBytes + part * 16);
          else
            cp_async16(smem_u32(S.raw_scale) + r * kKvScaleBytes + (part - kCodeGran) * 16,
                       cache.kv_scales + static_cast<long long>(row + r) * kKvScaleBytes + (part - kCodeGran) * 16);
        }
      }
      cp_async_commit();
      return row >= 0;
    };

    __syncthreads();   // the previous tile's shared memory is free
    bool ok = key_begin < key_end ? issue(key_begin) : false;
    // queries -> fp16 with a power-of-two scale per row (bf16's 8 bits are
    // kept whole; the row's largest value comes to lie in [2^14, 2^15))
    for (int r = warp; r < MR; r += kCWarps) {
      uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
      if (r < rows) {
        const uint4* src =
            reinterpret_cast<const uint4*>(q + (static_cast<long long>(T.q0) * a.heads + r) * kKvDim) + lane * 2;
        v0 = src[0];
        v1 = src[1];
      }
      const uint32_t wv[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
      float f[16], amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[2 * i] = __uint_as_float(wv[i] << 16);
        f[2 * i + 1] = __uint_as_float(wv[i] & 0xFFFF0000u);
        amax = fmaxf(amax, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      int E = static_cast<int>((__float_as_uint(amax) >> 23) & 0xFF) - 127;
      if (amax == 0.0f) E = 14;
      E = max(E, -100);
      const float up = exp2i(14 - E), down = exp2i(E - 14);
      uint32_t hv[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) hv[i] = pack_half2(f[2 * i] * up, f[2 * i + 1] * up);
      *reinterpret_cast<uint4*>(S.q + swz(r, 2 * lane)) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
      *reinterpret_cast<uint4*>(S.q + swz(r, 2 * lane + 1)) = make_uint4(hv[4], hv[5], hv[6], hv[7]);
      if (lane == 0) {
        S.qscale[r] = softmax_scale * down * kLog2e;
        S.lim[r] = r < rows ? seen_by(a.q_pos[T.q0 + r / a.heads], a.ratio, T.ctx) : 0;
      }
    }

    float o_acc[L::HT][kDimsPerWarp / 8][4];
#pragma unroll
    for (int t = 0; t < L::HT; ++t)
#pragma unroll
      for (int i = 0; i < kDimsPerWarp / 8; ++i) o_acc[t][i][0] = o_acc[t][i][1] = o_acc[t][i][2] = o_acc[t][i][3] = 0.0f;
    float m_run[L::HT][2], l_run[L::HT][2];
#pragma unroll
    for (int t = 0; t < L::HT; ++t) m_run[t][0] = m_run[t][1] = -INFINITY, l_run[t][0] = l_run[t][1] = 0.0f;

    for (int c0 = key_begin; c0 < key_end; c0 += kChunk) {
      const int nk = ok ? min(kChunk, key_end - c0) : 0;
      cp_async_wait_all();
      __syncthreads();   // staged rows visible; the previous step's products are done
      {
        const int row = tid & (kChunk - 1), part = tid / kChunk;   // channels 128*part .. 128*part + 127 of the row
        if (row < nk) {
          const uint8_t* rc = S.raw + row * kKvCodeBytes;
          const uint2 sp = *reinterpret_cast<const uint2*>(S.raw_scale + row * kKvScaleBytes + part * 8);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 cv = *reinterpret_cast<const uint4*>(rc + (((4 * part + j) ^ (row & 7)) << 4));
            uint4 hv[4];
            dequant16(cv, j < 2 ? (sp.x >> (16 * j)) : (sp.y >> (16 * (j - 2))), hv);
#pragma unroll
            for (int c = 0; c < 4; ++c) *reinterpret_cast<uint4*>(S.kv + swz(row, part * 16 + j * 4 + c)) = hv[c];
          }
        } else {
#pragma unroll
          for (int c = 0; c < 16; ++c) *reinterpret_cast<uint4*>(S.kv + swz(row, part * 16 + c)) = make_uint4(0, 0, 0, 0);
        }
      }
      __syncthreads();
      if (c0 + kChunk < key_end) ok = issue(c0 + kChunk);

      // ---- S = Q K^T: 16 rows x KW keys per warp ----
      float s[L::NT][4];
#pragma unroll
      for (int j = 0; j < L::NT; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.0f;
      const int key0 = kg * L::KW;
#pragma unroll 4
      for (int ks = 0; ks < kKvDim / 16; ++ks) {
        uint32_t a0, a1, a2, a3;
        ldsm_x4(q_sh + swz(ht * 16 + (lane & 15), ks * 2 + (lane >> 4)), a0, a1, a2, a3);
        if constexpr (L::NT == 1) {
          uint32_t b0, b1;
          ldsm_x2(kv_sh + swz(key0 + (lane & 7), ks * 2 + ((lane >> 3) & 1)), b0, b1);
          mma_f16(s[0], a0, a1, a2, a3, b0, b1);
        } else {
#pragma unroll
          for (int np = 0; np < L::NT / 2; ++np) {
            const int mi = lane >> 3;
            uint32_t b0, b1, b2, b3;
            ldsm_x4(kv_sh + swz(key0 + np * 16 + (mi >> 1) * 8 + (lane & 7), ks * 2 + (mi & 1)), b0, b1, b2, b3);
            mma_f16(s[2 * np], a0, a1, a2, a3, b0, b1);
            mma_f16(s[2 * np + 1], a0, a1, a2, a3, b2, b3);
          }
        }
      }

      // ---- running maximum and sum (log2 domain) over the key groups ----
      const float sc0 = S.qscale[h0], sc1 = S.qscale[h1];
      const int lim0 = min(S.lim[h0], c0 + nk), lim1 = min(S.lim[h1], c0 + nk);
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int j = 0; j < L::NT; ++j) {
        const int key = c0 + key0 + j * 8 + 2 * (lane & 3);
        s[j][0] = key < lim0 ? s[j][0] * sc0 : -INFINITY;
        s[j][1] = key + 1 < lim0 ? s[j][1] * sc0 : -INFINITY;
        s[j][2] = key < lim1 ? s[j][2] * sc1 : -INFINITY;
        s[j][3] = key + 1 < lim1 ? s[j][3] * sc1 : -INFINITY;
        mx0 = fmaxf(mx0, fmaxf(s[j][0], s[j][1]));
        mx1 = fmaxf(mx1, fmaxf(s[j][2], s[j][3]));
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
      }
      if ((lane & 3) == 0) {
        S.red_max[kg][h0] = mx0;
        S.red_max[kg][h1] = mx1;
      }
      __syncthreads();
      float mn0 = m_run[0][0], mn1 = m_run[0][1];
#pragma unroll
      for (int t = 1; t < L::HT; ++t)
        if (t == ht) mn0 = m_run[t][0], mn1 = m_run[t][1];
#pragma unroll
      for (int g = 0; g < L::KG; ++g) {
        mn0 = fmaxf(mn0, S.red_max[g][h0]);
        mn1 = fmaxf(mn1, S.red_max[g][h1]);
      }
      const float ref0 = mn0 == -INFINITY ? 0.0f : mn0, ref1 = mn1 == -INFINITY ? 0.0f : mn1;
      float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
      for (int j = 0; j < L::NT; ++j) {
        const float p0 = exp2f(s[j][0] - ref0), p1 = exp2f(s[j][1] - ref0);
        const float p2 = exp2f(s[j][2] - ref1), p3 = exp2f(s[j][3] - ref1);
        sum0 += p0 + p1;
        sum1 += p2 + p3;
        const int col = key0 + j * 8 + 2 * (lane & 3);
        const uint32_t within = (col & 7) * 2;
        *reinterpret_cast<uint32_t*>(S.p + pswz(h0, col >> 3) + within) = pack_half2(p0, p1);
        *reinterpret_cast<uint32_t*>(S.p + pswz(h1, col >> 3) + within) = pack_half2(p2, p3);
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        sum0 += __shfl_xor_sync(0xffffffffu, sum0, o);
        sum1 += __shfl_xor_sync(0xffffffffu, sum1, o);
      }
      if ((lane & 3) == 0) {
        S.red_sum[kg][h0] = sum0;
        S.red_sum[kg][h1] = sum1;
      }
      __syncthreads();
#pragma unroll
      for (int t = 0; t < L::HT; ++t) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int row = t * 16 + r0 + 8 * hf;
          float mn = m_run[t][hf], tot = 0.0f;
#pragma unroll
          for (int g = 0; g < L::KG; ++g) {
            mn = fmaxf(mn, S.red_max[g][row]);
            tot += S.red_sum[g][row];
          }
          const float ref = mn == -INFINITY ? 0.0f : mn;
          const float corr = exp2f(m_run[t][hf] - ref);
          l_run[t][hf] = l_run[t][hf] * corr + tot;
          m_run[t][hf] = mn;
#pragma unroll
          for (int i = 0; i < kDimsPerWarp / 8; ++i) {
            o_acc[t][i][2 * hf] *= corr;
            o_acc[t][i][2 * hf + 1] *= corr;
          }
        }
      }

      // ---- O += P V: every row x this warp's 64 channels ----
#pragma unroll
      for (int kk = 0; kk < kChunk / 16; ++kk) {
        uint32_t pa[L::HT][4];
#pragma unroll
        for (int t = 0; t < L::HT; ++t)
          ldsm_x4(p_sh + pswz(t * 16 + (lane & 15), kk * 2 + (lane >> 4)), pa[t][0], pa[t][1], pa[t][2], pa[t][3]);
#pragma unroll
        for (int np = 0; np < kDimsPerWarp / 16; ++np) {
          const int mi = lane >> 3;
          const int dchunk = (warp * kDimsPerWarp) / 8 + np * 2 + (mi >> 1);
          uint32_t b0, b1, b2, b3;
          ldsm_x4_t(kv_sh + swz(kk * 16 + (mi & 1) * 8 + (lane & 7), dchunk), b0, b1, b2, b3);
#pragma unroll
          for (int t = 0; t < L::HT; ++t) {
            mma_f16(o_acc[t][2 * np], pa[t][0], pa[t][1], pa[t][2], pa[t][3], b0, b1);
            mma_f16(o_acc[t][2 * np + 1], pa[t][0], pa[t][1], pa[t][2], pa[t][3], b2, b3);
          }
        }
      }
    }
    cp_async_wait_all();

    // ---- the whole tile: its rows; a part of it: the partial sums ----
    if (seg == steps) {
#pragma unroll
      for (int t = 0; t < L::HT; ++t)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int row = t * 16 + r0 + 8 * hf;
          if (row >= rows) continue;
          const long long orow = static_cast<long long>(T.q0) * a.heads + row;
          const float l = l_run[t][hf], inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
          uint32_t* dst = reinterpret_cast<uint32_t*>(out + orow * kKvDim + warp * kDimsPerWarp + 2 * (lane & 3));
#pragma unroll
          for (int i = 0; i < kDimsPerWarp / 8; ++i) {
            const __nv_bfloat162 h =
                __floats2bfloat162_rn(o_acc[t][i][2 * hf] * inv, o_acc[t][i][2 * hf + 1] * inv);
            dst[i * 4] = *reinterpret_cast<const uint32_t*>(&h);
          }
          if (lse != nullptr && warp == 0 && (lane & 3) == 0)
            lse[orow] = l == 0.0f ? -INFINITY : (m_run[t][hf] + log2f(l)) * kLn2;
        }
    } else {
      float* part = partial_of(wsp, blockIdx.x, off > 0 ? 0 : 1, MR);
#pragma unroll
      for (int t = 0; t < L::HT; ++t)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int row = t * 16 + r0 + 8 * hf;
          if (row >= rows) continue;
#pragma unroll
          for (int i = 0; i < kDimsPerWarp / 8; ++i)
            *reinterpret_cast<float2*>(part + partial_at(row, warp * kDimsPerWarp + 2 * (lane & 3) + i * 8, MR)) =
                make_float2(o_acc[t][i][2 * hf], o_acc[t][i][2 * hf + 1]);
          if (warp == 0 && (lane & 3) == 0) {
            part[MR * kKvDim + row] = m_run[t][hf];
            part[MR * (kKvDim + 1) + row] = l_run[t][hf];
          }
        }
    }
    if (pos < plan.hi) place = next_tile(a, place);
    off = 0;
  }
}

// Joins the tiles that ranges cut: block (c, x, y) takes 32 rows and 64
// channels of the tile that range c starts inside, if c is the first to do so.
// A lane is a row, a warp 8 channels.
constexpr int kJoinRows = 32, kJoinChannels = 64;

__global__ void __launch_bounds__(256)
    chunk_join_kernel(int heads, int tile_rows, __nv_bfloat16* __restrict__ out, float* __restrict__ lse, void* ws) {
  const ChunkWorkspace wsp = split_chunk_ws(ws);
  const int c = blockIdx.x;
  const RangeRecord r = wsp.rec[c];
  if (c >= r.ctas || r.lo == r.tile_lo || wsp.rec[c - 1].lo > r.tile_lo) return;
  const int row = blockIdx.z * kJoinRows + (threadIdx.x & 31);
  const int ch = blockIdx.y * kJoinChannels + (threadIdx.x >> 5) * 8;
  int last = c;                          // the last range with a part of the tile, 32 records at a look
  for (bool more = true; more;) {
    const int k = last + 1 + (threadIdx.x & 31);
    const uint32_t in = __ballot_sync(0xffffffffu, k < r.ctas && wsp.rec[min(k, r.ctas - 1)].lo < r.tile_hi);
    last += __popc(in);                  // (the records' starts ascend)
    more = in == 0xffffffffu;
  }
  if (row >= r.tokens * heads) return;
  // the tile's head came from range c - 1, which ended (or also began) with it
  float M = -INFINITY;
#pragma unroll 8
  for (int k = c - 1; k <= last; ++k) M = fmaxf(M, partial_of(wsp, k, k < c ? 1 : 0, tile_rows)[tile_rows * kKvDim + row]);
  const float ref = M == -INFINITY ? 0.0f : M;
  float l = 0.0f, o[8] = {};
#pragma unroll 8
  for (int k = c - 1; k <= last; ++k) {
    const float* part = partial_of(wsp, k, k < c ? 1 : 0, tile_rows);
    const float f = exp2f(part[tile_rows * kKvDim + row] - ref);
    l = fmaf(part[tile_rows * (kKvDim + 1) + row], f, l);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 v = *reinterpret_cast<const float4*>(part + partial_at(row, ch + 4 * h, tile_rows));
      o[4 * h] = fmaf(v.x, f, o[4 * h]);
      o[4 * h + 1] = fmaf(v.y, f, o[4 * h + 1]);
      o[4 * h + 2] = fmaf(v.z, f, o[4 * h + 2]);
      o[4 * h + 3] = fmaf(v.w, f, o[4 * h + 3]);
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
  const long long orow = static_cast<long long>(r.q0) * heads + row;
  uint32_t pk[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * h] * inv, o[2 * h + 1] * inv);
    pk[h] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(out + orow * kKvDim + ch) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
  if (lse != nullptr && ch == 0) lse[orow] = l == 0.0f ? -INFINITY : (M + log2f(l)) * kLn2;
}

template <int MR>
cudaError_t launch_chunk(const DenseArgs& a, const uint16_t* q, float scale, uint16_t* out, float* lse, void* ws,
                         int num_sms, cudaStream_t stream) {
  static ContextMemo attrs;
  const size_t smem = sizeof(ChunkSmem<MR>);
  cudaError_t e = attrs.once([&] {
    return cudaFuncSetAttribute(chunk_attn_kernel<MR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(smem));
  });
  if (e != cudaSuccess) return e;
  const int ctas = min(kMaxRanges, num_sms * (MR == 16 ? 2 : 1));
  chunk_attn_kernel<MR><<<ctas, kCThreads, smem, stream>>>(a, reinterpret_cast<const __nv_bfloat16*>(q), scale,
                                                           reinterpret_cast<__nv_bfloat16*>(out), lse, ws);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_chunk_join(a.heads, MR, ctas, out, lse, ws, stream);
}

}  // namespace

cudaError_t launch_chunk_join(int heads, int tile_rows, int ranges, uint16_t* out, float* lse, void* ws,
                              cudaStream_t stream) {
  chunk_join_kernel<<<dim3(ranges, kKvDim / kJoinChannels, (tile_rows + kJoinRows - 1) / kJoinRows), 256, 0, stream>>>(
      heads, tile_rows, reinterpret_cast<__nv_bfloat16*>(out), lse, ws);
  return cudaGetLastError();
}

size_t chunk_attn_workspace_bytes() {
  return kMaxRanges * sizeof(RangeRecord) + static_cast<size_t>(kWsRows) * (kKvDim + 2) * sizeof(float);
}

cudaError_t launch_chunk_attn(const csa2_cache& cache, int n_queries, const int32_t* q_start, const int32_t* q_pos,
                              int ratio, const uint16_t* q, int H, float scale, uint16_t* out, float* lse, void* ws,
                              int num_sms, uint64_t wait_ns, cudaStream_t stream) {
  DenseArgs a = {cache, q_start, q_pos, n_queries, ratio, H, 1, 2};
  if (true) {
    a.tile_tokens = 128 / H;
    a.min_steps = 1;
    return launch_chunk_attn_pair(a, q, scale, out, lse, ws, num_sms, wait_ns, stream);
  }
  // One token per tile while requests have about one each; more tokens share a
  // tile of 64 rows otherwise.
  const bool single = n_queries <= cache.batch;
  a.tile_tokens = single ? 1 : 64 / H;
  switch (a.tile_tokens * H) {
    case 16: return launch_chunk<16>(a, q, scale, out, lse, ws, num_sms, stream);
    case 32: return launch_chunk<32>(a, q, scale, out, lse, ws, num_sms, stream);
    default: return launch_chunk<64>(a, q, scale, out, lse, ws, num_sms, stream);
  }
}

}  // namespace csa2
