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

// Four consecutive elements as fp32.
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 r = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                     __uint_as_float(r.y & 0xFFFF0000u));
}
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

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

// A row of D elements is D / 8 units of two groups of 4 channels; G lanes hold
// a row, lane g its units g and (D = 512) g + 32.  A unit of the rotated part
// holds whole pairs: the groups are 8 neighbours when pairs are interleaved or
// nothing is rotated there, and 4 channels with their partners rot / 2 further
// on otherwise.  So the rotation needs no exchange between lanes; with 8
// neighbours a lane and shuffles to the partners the kernel took 32 instructions
// an element, and twice the time.
// Bound by memory: the row is read and written once.
template <int D, int R, typename Tin, typename Tout>
__global__ void __launch_bounds__(kNThreads, D == 128 ? 5 : 4)
    norm_rope_kernel(int n_rows, int heads, const Tin* x, long long x_stride, const float* __restrict__ weight,
                     float eps, const double* __restrict__ freqs, int rot, int interleaved,
                     const int32_t* __restrict__ pos, Tout* out, int tokens_per_block, int heads_per_block) {
  constexpr int kUnits = D / 8;
  constexpr int G = kUnits < 32 ? kUnits : 32;         // lanes per row
  constexpr int C = kUnits / G;                        // units per lane
  constexpr int RPW = 32 / G;                          // rows a warp holds at once
  extern __shared__ float4 turn_pairs[];               // [tokens_per_block][rot / 4] two (cos, sin) each
  float2* turns = reinterpret_cast<float2*>(turn_pairs);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane % G;
  const int half = rot / 2, lo = D - rot;
  const int t0 = blockIdx.x * tokens_per_block, h0 = blockIdx.y * heads_per_block;
  const int nh = min(heads_per_block, heads - h0), nt = min(tokens_per_block, n_rows - t0);
  const int rows = nt * nh;

  // the lane's channels, the same in every row
  int ca[C], cb[C], turn[C];                           // turn: its first pair, or -1
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int u = g + c * G;
    ca[c] = u * 8;
    cb[c] = u * 8 + 4;
    turn[c] = -1;
    if (u * 8 >= lo) {
      turn[c] = (u * 8 - lo) / 2;
      if (!interleaved) ca[c] = lo + turn[c], cb[c] = lo + half + turn[c];
    }
  }

  // the rows first: they do not wait for the angles
  float4 va[R][C], vb[R][C];
  int tok[R], head[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = (i * kNWarps + warp) * RPW + lane / G;
    tok[i] = tokens_per_block == 1 ? 0 : r / nh;
    head[i] = h0 + (tokens_per_block == 1 ? r : r % nh);
    if (r >= rows) tok[i] = -1;
    const Tin* src = x + static_cast<long long>(t0 + max(tok[i], 0)) * x_stride + (tok[i] < 0 ? h0 : head[i]) * D;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      va[i][c] = load4(src + ca[c]);                   // (lanes without a row read the block's first again)
      vb[i][c] = load4(src + cb[c]);
    }
  }
  float4 wa[C], wb[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    wa[c] = wb[c] = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    if (weight != nullptr) wa[c] = load4(weight + ca[c]), wb[c] = load4(weight + cb[c]);
  }
  for (int i = threadIdx.x; i < nt * half; i += kNThreads) turns[i] = turn_of(pos[t0 + i / half], freqs[i % half]);
  __syncthreads();

#pragma unroll
  for (int i = 0; i < R; ++i) {
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float4 a = va[i][c], b = vb[i][c];
      ss = fmaf(a.x, a.x, fmaf(a.y, a.y, fmaf(a.z, a.z, fmaf(a.w, a.w, ss))));
      ss = fmaf(b.x, b.x, fmaf(b.y, b.y, fmaf(b.z, b.z, fmaf(b.w, b.w, ss))));
    }
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    float inv = rsqrtf(fmaf(ss, 1.0f / D, eps));
    // Squares that leave fp32's range: the row times 2^-70 (every lane of the
    // warp takes part; the sum of 512 squares is then below 2^126).
    if (__any_sync(0xffffffffu, !(ss <= 1e37f))) {
      constexpr float kDown = 8.470329472543003e-22f;   // 2^-70
      const bool big = !(ss <= 1e37f);
      const float down = big ? kDown : 1.0f;
      float s2 = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float4 &a = va[i][c], &b = vb[i][c];
        a.x *= down; a.y *= down; a.z *= down; a.w *= down;
        b.x *= down; b.y *= down; b.z *= down; b.w *= down;
        s2 = fmaf(a.x, a.x, fmaf(a.y, a.y, fmaf(a.z, a.z, fmaf(a.w, a.w, s2))));
        s2 = fmaf(b.x, b.x, fmaf(b.y, b.y, fmaf(b.z, b.z, fmaf(b.w, b.w, s2))));
      }
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) s2 += __shfl_xor_sync(0xffffffffu, s2, o);
      if (big) inv = rsqrtf(s2 * (1.0f / D));           // eps <= 1 is nothing next to a mean above 1e34
    }
    Tout* dst = out + (static_cast<long long>(t0 + max(tok[i], 0)) * heads + head[i]) * D;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float4 a = va[i][c], b = vb[i][c];
      a.x *= inv * wa[c].x; a.y *= inv * wa[c].y; a.z *= inv * wa[c].z; a.w *= inv * wa[c].w;
      b.x *= inv * wb[c].x; b.y *= inv * wb[c].y; b.z *= inv * wb[c].z; b.w *= inv * wb[c].w;
      if (turn[c] >= 0) {
        const float4* tt = reinterpret_cast<const float4*>(turns + max(tok[i], 0) * half + turn[c]);
        const float4 p = tt[0], q = tt[1];              // (cos, sin) of four pairs
        if (interleaved) {
          a = make_float4(a.x * p.x - a.y * p.y, a.x * p.y + a.y * p.x, a.z * p.z - a.w * p.w, a.z * p.w + a.w * p.z);
          b = make_float4(b.x * q.x - b.y * q.y, b.x * q.y + b.y * q.x, b.z * q.z - b.w * q.w, b.z * q.w + b.w * q.z);
        } else {
          const float4 u = a, v = b;
          a = make_float4(u.x * p.x - v.x * p.y, u.y * p.z - v.y * p.w, u.z * q.x - v.z * q.y, u.w * q.z - v.w * q.w);
          b = make_float4(u.x * p.y + v.x * p.x, u.y * p.w + v.y * p.z, u.z * q.y + v.z * q.x, u.w * q.w + v.w * q.z);
        }
      }
      if (tok[i] >= 0) {
        store4(dst + ca[c], a);
        store4(dst + cb[c], b);
      }
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
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 v = load4(kv + i * kv_stride + lane * 16 + 4 * j);
      x[4 * j] = v.x; x[4 * j + 1] = v.y; x[4 * j + 2] = v.z; x[4 * j + 3] = v.w;
    }
    const float4 r = load4(ik + i * ik_stride + lane * 4);
    k4[0] = r.x; k4[1] = r.y; k4[2] = r.z; k4[3] = r.w;
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
  // Rows a warp holds at once: two where there are rows enough to fill the GPU
  // with such blocks, else one.
  const bool many = static_cast<long long>(n_rows) * heads * dim >= (1LL << 22);
  if (dim == 128)
    return many ? launch_nr_types<128, 2>(n_rows, heads, x, x_type, x_stride, weight, eps, rope, pos, out, out_type, stream)
                : launch_nr_types<128, 1>(n_rows, heads, x, x_type, x_stride, weight, eps, rope, pos, out, out_type, stream);
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
