// Pieces of the attention kernels on mma.sync tiles: swizzled fp16 rows in
// shared memory, fragment loads, the fp16 MMA, asynchronous copies and the
// FP4 -> fp16 conversion of packed main-KV rows.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include "fp4.cuh"

namespace csa2 {

constexpr int kChunk = 64;                   // keys per chunk
constexpr int kRowBytes = kKvDim * 2;        // fp16 row: 1024 B
constexpr int kPRowBytes = kChunk * 2;       // fp16 row of P: 128 B
constexpr int kCodeGran = kKvCodeBytes / 16;                    // 16-byte granules of a packed row's codes
constexpr int kRowGran = (kKvCodeBytes + kKvScaleBytes) / 16;   // ... of codes + scales
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint32_t swz(uint32_t row, uint32_t chunk) {   // 16-byte chunk of a 1 KB row
  return row * kRowBytes + ((chunk ^ (row & 7u)) << 4);
}
__device__ __forceinline__ uint32_t pswz(uint32_t row, uint32_t chunk) {  // 16-byte chunk of a 128 B row of P
  return row * kPRowBytes + ((chunk ^ (row & 7u)) << 4);
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x2(uint32_t addr, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 2^x (results below 2^-126 are 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cp.async (LSU path, no tensor map): 16 bytes global -> shared, completion
// tracked per thread by commit groups.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// Two E2M1 codes (low nibble = even channel) -> f16x2, low half = even channel.
__device__ __forceinline__ uint32_t e2m1x2_half2(uint32_t byte) {
  const __half2_raw r = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(byte & 0xFFu), __NV_E2M1);
  return static_cast<uint32_t>(r.x) | (static_cast<uint32_t>(r.y) << 16);
}

// Dequantise 16 code bytes (32 channels, 2 scale groups) into 4 fp16 chunks.
__device__ __forceinline__ void dequant16(uint4 codes, uint32_t s01, uint4 (&out)[4]) {
  const uint32_t sc0 = e4m3_half_bits(s01 & 0xFFu), sc1 = e4m3_half_bits((s01 >> 8) & 0xFFu);
  const __half2 s0 = __halves2half2(__ushort_as_half(sc0), __ushort_as_half(sc0));
  const __half2 s1 = __halves2half2(__ushort_as_half(sc1), __ushort_as_half(sc1));
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t h[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t pair = e2m1x2_half2(w[i >> 2] >> (8 * (i & 3)));
    __half2 v = *reinterpret_cast<const __half2*>(&pair);
    v = __hmul2(v, i < 8 ? s0 : s1);   // exact: <= 5 significant bits, inside fp16's normal range
    h[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) out[c] = make_uint4(h[4 * c], h[4 * c + 1], h[4 * c + 2], h[4 * c + 3]);
}

}  // namespace csa2
