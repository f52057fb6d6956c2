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
// and indexer elements 4l .. 4l+3 (the layout of quantize_store).
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
struct AppendArgs {
  csa2_cache cache;
  uint8_t *ik4_codes, *ik4_scales;
  int n_rows;
  const T *kv, *ik;
  long long kv_stride, ik_stride;
  const float *kv_weight, *ik_weight;
  double eps;
  RopeArg kv_rope, ik_rope;
  int kv_inter, ik_inter;
  const int32_t *rope_pos, *req, *pos;
};

// Row i in float64, as it is defined, into cache row `row`; tab: shared memory
// for (rot + rot) / 2 (cos, sin) pairs of this warp.
template <typename T>
__device__ __noinline__ void append_exact(const AppendArgs<T>& a, int i, long long row, int lane, double2* tab) {
  float x[16], k4[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 v = load4(a.kv + i * a.kv_stride + lane * 16 + 4 * j);
    x[4 * j] = v.x; x[4 * j + 1] = v.y; x[4 * j + 2] = v.z; x[4 * j + 3] = v.w;
  }
  const float4 r = load4(a.ik + i * a.ik_stride + lane * 4);
  k4[0] = r.x; k4[1] = r.y; k4[2] = r.z; k4[3] = r.w;
  double2 *tkv = tab, *tik = tab + a.kv_rope.rot / 2;
  const double p = static_cast<double>(a.rope_pos ? a.rope_pos[i] : a.pos[i]);
  __syncwarp();
  for (int f = lane; f < a.kv_rope.rot / 2; f += 32) sincos(p * a.kv_rope.freqs[f], &tkv[f].y, &tkv[f].x);
  for (int f = lane; f < a.ik_rope.rot / 2; f += 32) sincos(p * a.ik_rope.freqs[f], &tik[f].y, &tik[f].x);
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
  const double inv = 1.0 / sqrt(warp_sum(s) * (1.0 / kKvDim) + a.eps);
  const double invk = 1.0 / sqrt(warp_sum(sk) * (1.0 / kIndexDim) + a.eps);
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    y[j] *= inv;
    if (a.kv_weight) y[j] *= static_cast<double>(a.kv_weight[lane * 16 + j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    z[j] *= invk;
    if (a.ik_weight) z[j] *= static_cast<double>(a.ik_weight[lane * 4 + j]);
  }
  if (a.kv_rope.rot > 0) rotate_lane<16, kKvDim>(y, lane, a.kv_rope.rot, a.kv_inter != 0, tkv);
  if (a.ik_rope.rot > 0) rotate_lane<4, kIndexDim>(z, lane, a.ik_rope.rot, a.ik_inter != 0, tik);
#pragma unroll
  for (int j = 0; j < 16; ++j) x[j] = __double2float_rn(y[j]);
  const float4 k = make_float4(__double2float_rn(z[0]), __double2float_rn(z[1]), __double2float_rn(z[2]),
                               __double2float_rn(z[3]));
  quantize_store(a.cache, row, x, k, lane);
  if (a.ik4_codes != nullptr) store_ik4(a.ik4_codes, a.ik4_scales, row, k, lane);
}

// fp32 form of a lane's N channels of a row of D: y = x * inv * w, rotated, and
// a bound of |y - its exact value| for each.  fp32 errors, in 2^-24: the sum of
// squares 16 terms a lane and 5 steps (21, halved by the root), eps and mean 2,
// rsqrtf 4, products 2; the rotation's cos and sin 5.2 and its product and sum
// 2, of |u| + |v|: below 26.  64 (2^-18) are allowed for; the rounding to fp32 of
// the exact value is one of them.
constexpr float kAppendErr = 3.814697265625e-06f;   // 2^-18
template <int N, int D>
__device__ __forceinline__ void rotate_fast(float (&y)[N], float (&err)[N], int lane, int rot, bool interleaved,
                                            const float2* tt) {
  const int half = rot / 2, ch = lane * N - (D - rot);
#pragma unroll
  for (int k = 0; k < N; ++k) err[k] = fabsf(y[k]);
  if (rot > 0) {
    if (interleaved) {
      if (ch >= 0) {
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
          const float2 t = tt[ch / 2 + k];
          const float u = y[2 * k], v = y[2 * k + 1];
          y[2 * k] = u * t.x - v * t.y;
          y[2 * k + 1] = u * t.y + v * t.x;
          err[2 * k] = err[2 * k + 1] = fabsf(u) + fabsf(v);
        }
      }
    } else {
      const bool first = ch < half;
      const int src = ch >= 0 ? lane + (first ? half / N : -(half / N)) : lane;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float p = __shfl_sync(0xffffffffu, y[k], src);
        if (ch >= 0) {
          const float2 t = tt[(first ? ch : ch - half) + k];
          err[k] = fabsf(y[k]) + fabsf(p);
          y[k] = first ? y[k] * t.x - p * t.y : p * t.y + y[k] * t.x;
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < N; ++k) err[k] *= kAppendErr;
}

// Eight E2M1 codes of v / s (r: about 1 / s), -0 as +0.
__device__ __forceinline__ uint32_t e2m1x8(const float* v, float r) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t b;
    asm("{\n\t.reg .b8 c;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n\t"
        "cvt.u32.u8 %0, c;\n\t}"
        : "=r"(b)
        : "f"(v[2 * i + 1] * r), "f"(v[2 * i] * r));
    w |= b << (8 * i);
  }
  const uint32_t some = ((w & 0x77777777u) + 0x77777777u) & 0x88888888u;   // sign bits of codes that are not 0
  return w & (some | 0x77777777u);
}

// The stored codes are those of the float64 formula rounded once to fp32: an
// fp32 norm, off by 1e-7, would now and then move a value across an FP4 or FP8
// border.  float64 for every row is slow (conversions run at an eighth of the
// fp32 rate: 63 us for 32,765 rows), and rarely needed: the quantisation is
// monotone, so when y - err and y + err, the ends of the interval that holds
// the exact value, give the same scales, exponents and codes, these are the
// exact value's.  Rows where they differ (about one in 60), and rows outside
// fp32's comfortable range, take append_exact.
template <typename T>
__global__ void __launch_bounds__(128, 6) norm_rope_append_kernel(const __grid_constant__ AppendArgs<T> a) {
  extern __shared__ double2 turn_tab[];               // per warp: (kv rot + ik rot) / 2 entries
  const int wib = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.x * (blockDim.x >> 5) + wib;
  if (i >= a.n_rows) return;
  float y[16], z[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 v = load4(a.kv + i * a.kv_stride + lane * 16 + 4 * j);
    y[4 * j] = v.x; y[4 * j + 1] = v.y; y[4 * j + 2] = v.z; y[4 * j + 3] = v.w;
  }
  {
    const float4 v = load4(a.ik + i * a.ik_stride + lane * 4);
    z[0] = v.x; z[1] = v.y; z[2] = v.z; z[3] = v.w;
  }
  const long long row = row_of(a.cache, a.req ? a.req[i] : i, a.pos[i], lane);
  // angles of this row, spread over the lanes
  double2* tab = turn_tab + wib * ((a.kv_rope.rot + a.ik_rope.rot) / 2);
  float2 *tkv = reinterpret_cast<float2*>(tab), *tik = tkv;
  const int rope_pos = a.rope_pos ? a.rope_pos[i] : a.pos[i];
  for (int f = lane; f < a.kv_rope.rot / 2; f += 32) tkv[f] = turn_of(rope_pos, a.kv_rope.freqs[f]);
  if (a.kv_rope.freqs != a.ik_rope.freqs || a.kv_rope.rot != a.ik_rope.rot) {
    tik = tkv + a.kv_rope.rot / 2;
    for (int f = lane; f < a.ik_rope.rot / 2; f += 32) tik[f] = turn_of(rope_pos, a.ik_rope.freqs[f]);
  }
  __syncwarp();
  if (row < 0) return;

  float s = 0.0f, sk = 0.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j) s = fmaf(y[j], y[j], s);
#pragma unroll
  for (int j = 0; j < 4; ++j) sk = fmaf(z[j], z[j], sk);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    sk += __shfl_xor_sync(0xffffffffu, sk, o);
  }
  const float eps = static_cast<float>(a.eps);
  const float inv = rsqrtf(fmaf(s, 1.0f / kKvDim, eps)), invk = rsqrtf(fmaf(sk, 1.0f / kIndexDim, eps));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float4 w = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    if (a.kv_weight) w = load4(a.kv_weight + lane * 16 + 4 * j);
    y[4 * j] *= inv * w.x; y[4 * j + 1] *= inv * w.y; y[4 * j + 2] *= inv * w.z; y[4 * j + 3] *= inv * w.w;
  }
  {
    float4 w = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    if (a.ik_weight) w = load4(a.ik_weight + lane * 4);
    z[0] *= invk * w.x; z[1] *= invk * w.y; z[2] *= invk * w.z; z[3] *= invk * w.w;
  }
  float ey[16], ez[4];
  rotate_fast<16, kKvDim>(y, ey, lane, a.kv_rope.rot, a.kv_inter != 0, tkv);
  rotate_fast<4, kIndexDim>(z, ez, lane, a.ik_rope.rot, a.ik_inter != 0, tik);

  // main KV: both ends' scale and codes
  float lo16[16], hi16[16], amax_lo = 0.0f, amax_hi = 0.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    amax_lo = fmaxf(amax_lo, fabsf(y[j]) - ey[j]);
    amax_hi = fmaxf(amax_hi, fabsf(y[j]) + ey[j]);
    lo16[j] = y[j] - ey[j];
    hi16[j] = y[j] + ey[j];
  }
  PackedRow p;
  p.kv_scale = e4m3_code_of_sixth(amax_hi);
  bool sure = p.kv_scale == e4m3_code_of_sixth(amax_lo);
  p.kv = make_uint2(0u, 0u);
  if (p.kv_scale != 0u) {
    const float r = 1.0f / e4m3_value(p.kv_scale);   // off by 2^-24, as is its product: within err's reserve
    p.kv = make_uint2(e2m1x8(lo16, r), e2m1x8(lo16 + 8, r));
    sure = sure && p.kv.x == e2m1x8(hi16, r) && p.kv.y == e2m1x8(hi16 + 8, r);
  }
  // indexer key
  float km_lo = 0.0f, km_hi = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    km_lo = fmaxf(km_lo, fabsf(z[j]) - ez[j]);
    km_hi = fmaxf(km_hi, fabsf(z[j]) + ez[j]);
  }
  float group_lo = km_lo, group_hi = km_hi;          // of 16 elements (4 lanes), for the FP4 form
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    km_lo = fmaxf(km_lo, __shfl_xor_sync(0xffffffffu, km_lo, o));
    km_hi = fmaxf(km_hi, __shfl_xor_sync(0xffffffffu, km_hi, o));
    if (o == 2) group_lo = km_lo, group_hi = km_hi;
  }
  p.ik_exp = indexer_exponent(km_hi);
  sure = sure && p.ik_exp == indexer_exponent(fmaxf(km_lo, 0.0f));
  const float two = exp2i(-p.ik_exp);
  p.ik = e4m3x2((z[0] - ez[0]) * two, (z[1] - ez[1]) * two) | (e4m3x2((z[2] - ez[2]) * two, (z[3] - ez[3]) * two) << 16);
  sure = sure && p.ik == (e4m3x2((z[0] + ez[0]) * two, (z[1] + ez[1]) * two) |
                          (e4m3x2((z[2] + ez[2]) * two, (z[3] + ez[3]) * two) << 16));
  uint32_t c4 = 0u, s4 = 0u;
  if (a.ik4_codes != nullptr) {
    s4 = e4m3_code_of_sixth(group_hi);
    sure = sure && s4 == e4m3_code_of_sixth(group_lo);
    if (s4 != 0u) {
      const float r = 1.0f / e4m3_value(s4);
      const float v[8] = {z[0] - ez[0], z[1] - ez[1], z[2] - ez[2], z[3] - ez[3],
                          z[0] + ez[0], z[1] + ez[1], z[2] + ez[2], z[3] + ez[3]};
      const uint32_t both = e2m1x8(v, r);
      c4 = both & 0xFFFFu;
      sure = sure && c4 == both >> 16;
    }
  }
  // squares that fp32 may have lost, large values, and anything that is not
  // finite (a weight or an angle may be the cause; the maxima above drop a NaN)
  float size = 0.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j) size += ey[j];
#pragma unroll
  for (int j = 0; j < 4; ++j) size += ez[j];
  const bool usual = s <= 1e30f && sk <= 1e30f && (s >= 1e-20f || s == 0.0f) && (sk >= 1e-20f || sk == 0.0f) &&
                     size <= 1e24f;
  if (__all_sync(0xffffffffu, sure && usual)) {
    store_row(a.cache, row, p, lane);
    if (a.ik4_codes != nullptr) store_ik4_codes(a.ik4_codes, a.ik4_scales, row, c4, s4, lane);
  } else {
    append_exact(a, i, row, lane, tab);
  }
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
  // with such blocks, else one.  Measured with 32 heads x 128 channels, bf16 to
  // fp32, two rows / one: 8 tokens 2.8 / 2.4 us, 256 tokens 3.4 / 3.4, 512 tokens
  // 4.4 / 5.1, 8,192 tokens 42 / 51.  Rows of 512 channels go one at a time: two take
  // more than the 64 registers that four blocks an SM leave.  64 heads, bf16 to bf16,
  // two rows (with those spills) / one: 8 tokens 9.2 / 7.2 us, 512 tokens 23.6 / 23.5,
  // 2,048 tokens 67 / 69, 8,191 tokens 241 / 255 (memory alone: 164).
  const bool many = static_cast<long long>(n_rows) * heads * dim >= (1LL << 21);
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
  if (type == CSA2_BF16) {
    using T = __nv_bfloat16;
    norm_rope_append_kernel<T><<<blocks, kWarps * 32, smem, stream>>>(
        AppendArgs<T>{cache, c4, s4, n_rows, static_cast<const T*>(kv), static_cast<const T*>(ik), kv_stride, ik_stride,
                      kv_weight, ik_weight, eps, kr, ir, kv_rope.interleaved, ik_rope.interleaved, rope_pos, req, pos});
  } else {
    norm_rope_append_kernel<float><<<blocks, kWarps * 32, smem, stream>>>(
        AppendArgs<float>{cache, c4, s4, n_rows, static_cast<const float*>(kv), static_cast<const float*>(ik), kv_stride,
                          ik_stride, kv_weight, ik_weight, eps, kr, ir, kv_rope.interleaved, ik_rope.interleaved, rope_pos,
                          req, pos});
  }
  return cudaGetLastError();
}

}  // namespace csa2
