// Per-head RMS norm with the position rotation in the same pass, for queries
// (norm_rope_kernel) and, fused with quantise-on-append, for new cache rows
// (norm_rope_append_kernel).
//
//   y = x * w / sqrt(mean(x^2) + eps), then on the last `rot` channels, pair i:
//   (u, v) -> (u cos a - v sin a, u sin a + v cos a),  a = pos * freq_i.
//
// The angle is formed in float64: pos * freq_i in fp32 is off by 2^-25 of
// itself, 0.03 radians at position 10^6 for the fastest pair.
#include <cuda_bf16.h>

#include "append_row.cuh"
#include "launch.h"

namespace csa2 {

namespace {

constexpr int kNThreads = 256;
constexpr int kNWarps = kNThreads / 32;

// Eight consecutive elements as fp32.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// cos and sin of pos * freq: the angle in float64, reduced to [-pi, pi] by a
// two-part 2 pi, then fp32 (|angle| <= pi rounded to fp32: off by <= 1.2e-7).
__device__ __forceinline__ float2 turn_of(int pos, double freq) {
  constexpr double kTwoPi = 6.283185307179586, kTwoPiLow = 2.4492935982947064e-16;
  const double a = static_cast<double>(pos) * freq;
  const double k = rint(a * 0.15915494309189535);
  const float r = static_cast<float>(fma(-k, kTwoPiLow, fma(-k, kTwoPi, a)));
  float2 t;
  sincosf(r, &t.y, &t.x);
  return t;
}

// A row of D elements is D / 8 chunks of 8; a group of G lanes holds a row,
// lane g its chunks g and (D = 512) g + 32.
template <int D, int R, typename Tin, typename Tout>
__global__ void __launch_bounds__(kNThreads)
    norm_rope_kernel(int n_rows, int heads, const Tin* x, long long x_stride, const float* __restrict__ weight,
                     float eps, const double* __restrict__ freqs, int rot, int interleaved,
                     const int32_t* __restrict__ pos, Tout* out, int tokens_per_block, int heads_per_block) {
  constexpr int kChunks = D / 8;
  constexpr int G = kChunks < 32 ? kChunks : 32;       // lanes per row
  constexpr int C = kChunks / G;                       // chunks per lane
  constexpr int RPW = 32 / G;                          // rows a warp holds at once
  extern __shared__ float2 turns[];                    // [tokens_per_block][rot / 2]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane % G;
  const int half = rot / 2, lo = D - rot;
  const int t0 = blockIdx.x * tokens_per_block, h0 = blockIdx.y * heads_per_block;
  const int nh = min(heads_per_block, heads - h0);
  const int rows = min(tokens_per_block, n_rows - t0) * nh;

  // the rows first: they do not wait for the angles
  float v[R][C][8];
  int tok[R], head[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = (i * kNWarps + warp) * RPW + lane / G;
    tok[i] = r < rows ? r / nh : -1;
    head[i] = r < rows ? h0 + r % nh : 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (tok[i] >= 0) {
        load8(x + static_cast<long long>(t0 + tok[i]) * x_stride + static_cast<long long>(head[i]) * D + (g + c * G) * 8,
              v[i][c]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][c][k] = 0.0f;
      }
    }
  }
  float w[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (weight != nullptr) {
      load8(weight + (g + c * G) * 8, w[c]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) w[c][k] = 1.0f;
    }
  }
  const int nt = min(tokens_per_block, n_rows - t0);
  for (int i = threadIdx.x; i < nt * half; i += kNThreads) turns[i] = turn_of(pos[t0 + i / half], freqs[i % half]);
  __syncthreads();

#pragma unroll
  for (int i = 0; i < R; ++i) {
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(v[i][c][k], v[i][c][k], ss);
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    float inv;
    if (ss <= 1e37f) {
      inv = 1.0f / sqrtf(ss * (1.0f / D) + eps);
    } else {
      inv = 0.0f;
    }
    // Squares that leave fp32's range: the row times 2^-70 (every lane of the
    // warp takes part; the sum of 512 squares is then below 2^126).
    if (__any_sync(0xffffffffu, !(ss <= 1e37f))) {
      constexpr float kDown = 8.470329472543003e-22f;   // 2^-70
      float s2 = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float d = v[i][c][k] * kDown;
          s2 = fmaf(d, d, s2);
        }
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) s2 += __shfl_xor_sync(0xffffffffu, s2, o);
      if (!(ss <= 1e37f)) {
        inv = 1.0f / sqrtf(s2 * (1.0f / D));            // eps <= 1 is nothing next to a mean above 1e34
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int k = 0; k < 8; ++k) v[i][c][k] *= kDown;
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][c][k] = v[i][c][k] * inv * w[c][k];

    if (rot > 0) {
      const float2* tt = turns + max(tok[i], 0) * half;
      if (interleaved) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int ch = (g + c * G) * 8 - lo;          // first rotated channel of the chunk, if any
          if (ch >= 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 t = tt[ch / 2 + k];
              const float u = v[i][c][2 * k], z = v[i][c][2 * k + 1];
              v[i][c][2 * k] = u * t.x - z * t.y;
              v[i][c][2 * k + 1] = u * t.y + z * t.x;
            }
          }
        }
      } else {
        // the partner chunk is rot / 16 chunks away (rot is a multiple of
        // 32: whole chunks), in another lane or in this lane's other chunk
        float p[C][8];
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int ch = (g + c * G) * 8 - lo;
          const int other = g + c * G + (ch < half ? half / 8 : -(half / 8));
          const int src = ch >= 0 ? other : 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            p[c][k] = __shfl_sync(0xffffffffu, v[i][0][k], src % G, G);
            if (C > 1) {
              const float q = __shfl_sync(0xffffffffu, v[i][C - 1][k], src % G, G);
              if (src >= G) p[c][k] = q;
            }
          }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int ch = (g + c * G) * 8 - lo;
          if (ch >= 0) {
            const bool first = ch < half;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float2 t = tt[(first ? ch : ch - half) + k];
              v[i][c][k] = first ? v[i][c][k] * t.x - p[c][k] * t.y : p[c][k] * t.y + v[i][c][k] * t.x;
            }
          }
        }
      }
    }
    if (tok[i] >= 0) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        store8(out + (static_cast<long long>(t0 + tok[i]) * heads + head[i]) * D + (g + c * G) * 8, v[i][c]);
    }
  }
}

// New cache rows: one warp per row, lane l holding main-KV channels 16l .. 16l+15
// and indexer elements 4l .. 4l+3 (the layout of quantize_store).  Everything
// up to the rounding to fp32 is float64, so that the stored codes are those of
// the formula itself: an fp32 norm, off by 1e-7, would move values across the
// FP4 and FP8 borders.
__device__ __forceinline__ double warp_sum(double s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

struct RopeArg {
  const double* freqs;
  int rot;
};

// Rotates N consecutive channels first .. first + N - 1 of a row of D held by
// this lane (N * 32 = D); tt: the row's (cos, sin) table in shared memory.
template <int N, int D>
__device__ __forceinline__ void rotate_lane(double (&y)[N], int lane, int rot, bool interleaved,
                                            const double2* tt) {
  const int half = rot / 2, ch = lane * N - (D - rot);
  if (interleaved) {
    if (ch >= 0) {
#pragma unroll
      for (int k = 0; k < N / 2; ++k) {
        const double2 t = tt[ch / 2 + k];
        const double u = y[2 * k], v = y[2 * k + 1];
        y[2 * k] = u * t.x - v * t.y;
        y[2 * k + 1] = u * t.y + v * t.x;
      }
    }
  } else {
    const bool first = ch < half;
    const int src = ch >= 0 ? lane + (first ? half / N : -(half / N)) : lane;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const double p = __shfl_sync(0xffffffffu, y[k], src);
      if (ch >= 0) {
        const double2 t = tt[(first ? ch : ch - half) + k];
        y[k] = first ? y[k] * t.x - p * t.y : p * t.y + y[k] * t.x;
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(128)
    norm_rope_append_kernel(csa2_cache cache, uint8_t* ik4_codes, uint8_t* ik4_scales, int n_rows, const T* kv,
                            long long kv_stride, const T* ik, long long ik_stride, const float* kv_weight,
                            const float* ik_weight, double eps, RopeArg kv_rope, RopeArg ik_rope, int kv_inter,
                            int ik_inter, const int32_t* rope_pos, const int32_t* req, const int32_t* pos) {
  extern __shared__ double2 turn_tab[];               // per warp: [kv_rot / 2] then [ik_rot / 2]
  const int wib = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.x * (blockDim.x >> 5) + wib;
  if (i >= n_rows) return;
  const long long row = row_of(cache, req ? req[i] : i, pos[i], lane);
  if (row < 0) return;
  float x[16], k4[4];
  {
    float a[8], b[8];
    load8(kv + i * kv_stride + lane * 16, a);
    load8(kv + i * kv_stride + lane * 16 + 8, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = a[j], x[8 + j] = b[j];
    const T* kp = ik + i * ik_stride + lane * 4;
    if constexpr (sizeof(T) == 2) {
      const uint2 r = *reinterpret_cast<const uint2*>(kp);
      k4[0] = __uint_as_float(r.x << 16);
      k4[1] = __uint_as_float(r.x & 0xFFFF0000u);
      k4[2] = __uint_as_float(r.y << 16);
      k4[3] = __uint_as_float(r.y & 0xFFFF0000u);
    } else {
      const float4 r = *reinterpret_cast<const float4*>(kp);
      k4[0] = r.x; k4[1] = r.y; k4[2] = r.z; k4[3] = r.w;
    }
  }
  // angles of this row, spread over the lanes
  double2* tkv = turn_tab + wib * ((kv_rope.rot + ik_rope.rot) / 2);
  const bool same = kv_rope.freqs == ik_rope.freqs && kv_rope.rot == ik_rope.rot;
  double2* tik = same ? tkv : tkv + kv_rope.rot / 2;
  const double p = static_cast<double>(rope_pos ? rope_pos[i] : pos[i]);
  for (int f = lane; f < kv_rope.rot / 2; f += 32) {
    double2 t;
    sincos(p * kv_rope.freqs[f], &t.y, &t.x);
    tkv[f] = t;
  }
  if (!same)
    for (int f = lane; f < ik_rope.rot / 2; f += 32) {
      double2 t;
      sincos(p * ik_rope.freqs[f], &t.y, &t.x);
      tik[f] = t;
    }
  __syncwarp();

  double y[16], z[4], s = 0.0, sk = 0.0;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    y[j] = static_cast<double>(x[j]);
    s = fma(y[j], y[j], s);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    z[j] = static_cast<double>(k4[j]);
    sk = fma(z[j], z[j], sk);
  }
  const double inv = 1.0 / sqrt(warp_sum(s) * (1.0 / kKvDim) + eps);
  const double invk = 1.0 / sqrt(warp_sum(sk) * (1.0 / kIndexDim) + eps);
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    y[j] *= inv;
    if (kv_weight) y[j] *= static_cast<double>(kv_weight[lane * 16 + j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    z[j] *= invk;
    if (ik_weight) z[j] *= static_cast<double>(ik_weight[lane * 4 + j]);
  }
  if (kv_rope.rot > 0) rotate_lane<16, kKvDim>(y, lane, kv_rope.rot, kv_inter != 0, tkv);
  if (ik_rope.rot > 0) rotate_lane<4, kIndexDim>(z, lane, ik_rope.rot, ik_inter != 0, tik);
#pragma unroll
  for (int j = 0; j < 16; ++j) x[j] = __double2float_rn(y[j]);
  const float4 k = make_float4(__double2float_rn(z[0]), __double2float_rn(z[1]), __double2float_rn(z[2]),
                               __double2float_rn(z[3]));
  quantize_store(cache, row, x, k, lane);
  if (ik4_codes != nullptr) store_ik4(ik4_codes, ik4_scales, row, k, lane);
}

template <int D, int R, typename Tin, typename Tout>
cudaError_t launch_nr(int n_rows, int heads, const void* x, long long x_stride, const float* weight, float eps,
                      const csa2_rope& rope, const int32_t* pos, void* out, cudaStream_t stream) {
  constexpr int kRows = kNWarps * (D == 128 ? 2 : 1) * R;   // rows per block
  const int heads_per_block = heads < kRows ? heads : kRows;
  const int tokens_per_block = heads < kRows ? kRows / heads : 1;
  const dim3 grid((n_rows + tokens_per_block - 1) / tokens_per_block, (heads + heads_per_block - 1) / heads_per_block);
  const size_t smem = static_cast<size_t>(tokens_per_block) * (rope.rot / 2) * sizeof(float2);
  norm_rope_kernel<D, R, Tin, Tout><<<grid, kNThreads, smem, stream>>>(
      n_rows, heads, static_cast<const Tin*>(x), x_stride, weight, eps, rope.freqs, rope.rot, rope.interleaved, pos,
      static_cast<Tout*>(out), tokens_per_block, heads_per_block);
  return cudaGetLastError();
}

template <int D, int R>
cudaError_t launch_nr_types(int n_rows, int heads, const void* x, csa2_dtype xt, long long x_stride,
                            const float* weight, float eps, const csa2_rope& rope, const int32_t* pos, void* out,
                            csa2_dtype ot, cudaStream_t stream) {
  if (xt == CSA2_BF16)
    return ot == CSA2_BF16 ? launch_nr<D, R, __nv_bfloat16, __nv_bfloat16>(n_rows, heads, x, x_stride, weight, eps, rope, pos, out, stream)
                           : launch_nr<D, R, __nv_bfloat16, float>(n_rows, heads, x, x_stride, weight, eps, rope, pos, out, stream);
  return ot == CSA2_BF16 ? launch_nr<D, R, float, __nv_bfloat16>(n_rows, heads, x, x_stride, weight, eps, rope, pos, out, stream)
                         : launch_nr<D, R, float, float>(n_rows, heads, x, x_stride, weight, eps, rope, pos, out, stream);
}

}  // namespace

cudaError_t launch_norm_rope(int n_rows, int heads, int dim, const void* x, csa2_dtype x_type, long long x_stride,
                             const float* weight, float eps, const csa2_rope& rope, const int32_t* pos, void* out,
                             csa2_dtype out_type, cudaStream_t stream) {
  if (dim == 128)
    return launch_nr_types<128, 1>(n_rows, heads, x, x_type, x_stride, weight, eps, rope, pos, out, out_type, stream);
  return launch_nr_types<512, 1>(n_rows, heads, x, x_type, x_stride, weight, eps, rope, pos, out, out_type, stream);
}

cudaError_t launch_norm_rope_append(const csa2_cache& cache, const csa2_ik4* ik4, int n_rows, csa2_dtype type,
                                    const void* kv, long long kv_stride, const void* ik, long long ik_stride,
                                    const float* kv_weight, const float* ik_weight, float eps,
                                    const csa2_rope& kv_rope, const csa2_rope& ik_rope, const int32_t* rope_pos,
                                    const int32_t* req, const int32_t* pos, cudaStream_t stream) {
  constexpr int kWarps = 4;
  const unsigned blocks = static_cast<unsigned>((n_rows + kWarps - 1) / kWarps);
  const size_t smem = static_cast<size_t>(kWarps) * ((kv_rope.rot + ik_rope.rot) / 2) * sizeof(double2);
  const RopeArg kr = {kv_rope.freqs, kv_rope.rot}, ir = {ik_rope.freqs, ik_rope.rot};
  uint8_t* c4 = ik4 ? ik4->codes : nullptr;
  uint8_t* s4 = ik4 ? ik4->scales : nullptr;
  if (type == CSA2_BF16)
    norm_rope_append_kernel<__nv_bfloat16><<<blocks, kWarps * 32, smem, stream>>>(
        cache, c4, s4, n_rows, static_cast<const __nv_bfloat16*>(kv), kv_stride, static_cast<const __nv_bfloat16*>(ik),
        ik_stride, kv_weight, ik_weight, eps, kr, ir, kv_rope.interleaved, ik_rope.interleaved, rope_pos, req, pos);
  else
    norm_rope_append_kernel<float><<<blocks, kWarps * 32, smem, stream>>>(
        cache, c4, s4, n_rows, static_cast<const float*>(kv), kv_stride, static_cast<const float*>(ik), ik_stride,
        kv_weight, ik_weight, eps, kr, ir, kv_rope.interleaved, ik_rope.interleaved, rope_pos, req, pos);
  return cudaGetLastError();
}

}  // namespace csa2
