// Operands of the dense kernels over CTA pairs (csa2_chunk_attn,
// csa2_attn_mass): cache rows dequantised to fp16, query rows converted to it.
#pragma once

#include <cuda_bf16.h>

#include "attn_tile.cuh"
#include "cta_pair.cuh"
#include "dense_plan.cuh"

namespace csa2 {

constexpr float kRowScale = 256.0f;          // stored rows are 2^-8 of their value

// 32 channels of a packed row (16 code bytes, two scale codes below 0x80 in the
// low half of `sc`) -> four 16-byte chunks of fp16, each value times 2^-8.  Any
// scale code gives finite values (rows that nobody sees may hold any bytes).
__device__ __forceinline__ void dequant_32(uint4 codes, uint32_t sc, uint4 (&out)[4]) {
  const uint32_t b0 = (sc & 0xFFu) << 7, b1 = (sc >> 8) << 7;
  const uint32_t s0 = b0 | (b0 << 16), s1 = b1 | (b1 << 16);
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w[i]));
    const uint32_t s = i < 2 ? s0 : s1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&h[k]), *reinterpret_cast<const __half2*>(&s));
      h[k] = *reinterpret_cast<const uint32_t*>(&v);
    }
    out[i] = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

// The factor that undoes the power-of-two scale of a query row whose largest
// bf16 magnitude has the bits `top`.
__device__ __forceinline__ int query_row_exponent(uint32_t top) {
  return top == 0u ? 14 : max(static_cast<int>(top >> 7) - 127, -100);
}
__device__ __forceinline__ float query_row_down(uint32_t top) { return exp2i(query_row_exponent(top) - 14); }

// Query rows first .. first + kRows - 1 of q (bf16 [..][512]) as a K-major
// operand in 64-channel parts of kRows rows at `dst`: fp16 with a power-of-two
// scale per row (bf16's 8 bits are kept whole; the row's largest value comes to
// lie in [2^14, 2^15)), or 2^(14 - kExponent) for every row, eight rows' loads
// in flight per warp.  Rows from `valid` on are zeros; rows from `limit` on are
// left out.  seen(row, top) is called by one lane with the bits of the row's
// largest magnitude.
constexpr int kPerRow = 1000;
template <int kRows, int kWarps, int kExponent, class Seen>
__device__ __forceinline__ void load_query_rows(const __nv_bfloat16* __restrict__ q, long long first, int valid, int limit,
                                                float sign, uint8_t* dst, int warp, int lane, Seen seen) {
#pragma unroll 1
  for (int r0 = warp; r0 < limit; r0 += 8 * kWarps) {
    uint4 v[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + i * kWarps;
      v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
      if (r < valid) {
        const uint4* src = reinterpret_cast<const uint4*>(q + (first + r) * kKvDim) + lane * 2;
        v[i][0] = src[0];
        v[i][1] = src[1];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + i * kWarps;
      if (r >= limit) break;
      const uint32_t wv[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
      uint32_t top = 0;                          // exponent and mantissa of the largest magnitude (the bits order like it)
#pragma unroll
      for (int k = 0; k < 8; ++k) top = max(top, max(wv[k] & 0x7FFFu, (wv[k] >> 16) & 0x7FFFu));
      top = __reduce_max_sync(0xffffffffu, top);
      const float up = exp2i(14 - (kExponent == kPerRow ? query_row_exponent(top) : kExponent)) * sign;
      uint32_t hv[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        hv[k] = pack_half2(__uint_as_float(wv[k] << 16) * up, __uint_as_float(wv[k] & 0xFFFF0000u) * up);
      // lane: channels 16*lane .. +15: part lane / 4, chunks 2*(lane % 4), +1
      uint8_t* at = dst + (lane >> 2) * (kRows * 128) + r * 128;
      const int c0 = 2 * (lane & 3);
      *reinterpret_cast<uint4*>(at + ((c0 ^ (r & 7)) << 4)) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
      *reinterpret_cast<uint4*>(at + (((c0 + 1) ^ (r & 7)) << 4)) = make_uint4(hv[4], hv[5], hv[6], hv[7]);
      if (lane == 0) seen(r, top);
    }
  }
}

}  // namespace csa2
