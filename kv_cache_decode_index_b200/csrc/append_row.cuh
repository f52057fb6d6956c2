// One new cache row held by a warp: its slot, and its quantisation and store
// (csa2_append_kv, csa2_compress_append, csa2_norm_rope_append).
#pragma once

#include "fp4.cuh"

namespace csa2 {

// Cache row of position t of request b, or -1 (error recorded) when the
// request, the position or its page is out of range.
__device__ __forceinline__ long long row_of(const csa2_cache& cache, int b, int t, int lane) {
  const long long capacity = static_cast<long long>(cache.max_pages_per_req) * cache.page_size;
  if (b < 0 || b >= cache.batch || t < 0 || t >= capacity) {
    if (lane == 0) report_error(cache.err_word, CSA2_ERR_DEVICE_BOUNDS, kKAppend, b, t);
    return -1;
  }
  const int page = cache.page_table[static_cast<long long>(b) * cache.max_pages_per_req + t / cache.page_size];
  if (page < 0 || page >= cache.num_pages) {
    if (lane == 0) report_error(cache.err_word, CSA2_ERR_DEVICE_BOUNDS, kKAppend, b, t);
    return -1;
  }
  return static_cast<long long>(page) * cache.page_size + t % cache.page_size;
}

// What a lane stores of a row: 16 E2M1 codes (8 bytes) and their scale code, 4
// E4M3 indexer codes and the row's exponent.
struct PackedRow {
  uint2 kv;
  uint32_t kv_scale;
  uint32_t ik;
  int ik_exp;
};
__device__ __forceinline__ void store_row(const csa2_cache& cache, long long row, const PackedRow& p, int lane) {
  reinterpret_cast<uint2*>(cache.kv_codes + row * kKvCodeBytes)[lane] = p.kv;
  cache.kv_scales[row * kKvScaleBytes + lane] = static_cast<uint8_t>(p.kv_scale);
  reinterpret_cast<uint32_t*>(cache.ik_codes + row * kIndexDim)[lane] = p.ik;
  if (lane == 0) cache.ik_exp[row] = static_cast<uint8_t>(p.ik_exp + 127);
}

// Quantise one row held by a warp and store it: x = main-KV channels
// 16*lane .. 16*lane+15, k = indexer-K elements 4*lane .. 4*lane+3.
__device__ __forceinline__ void quantize_store(const csa2_cache& cache, long long row, const float (&x)[16], float4 k,
                                               int lane) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
  const uint32_t sc = e4m3_code_of_sixth(amax);
  const float s = e4m3_value(sc);
  uint32_t lo = 0, hi = 0;
  if (s > 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t byte = e2m1_code(x[2 * i], s) | (e2m1_code(x[2 * i + 1], s) << 4);
      if (i < 4) lo |= byte << (8 * i);
      else hi |= byte << (8 * (i - 4));
    }
  }

  float km = fmaxf(fmaxf(fabsf(k.x), fabsf(k.y)), fmaxf(fabsf(k.z), fabsf(k.w)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) km = fmaxf(km, __shfl_xor_sync(0xffffffffu, km, o));
  const int e = indexer_exponent(km);
  const float inv = exp2i(-e);
  const uint32_t codes = e4m3x2(k.x * inv, k.y * inv) | (e4m3x2(k.z * inv, k.w * inv) << 16);
  store_row(cache, row, PackedRow{make_uint2(lo, hi), sc, codes, e}, lane);
}

// Quantise one indexer key held by a warp (k = elements 4*lane .. 4*lane+3)
// to the FP4 indexer format and store it in row `row`.
__device__ __forceinline__ void store_ik4_codes(uint8_t* codes, uint8_t* scales, long long row, uint32_t c, uint32_t sc,
                                                int lane) {
  reinterpret_cast<uint16_t*>(codes + row * CSA2_IK4_CODE_BYTES)[lane] = static_cast<uint16_t>(c);
  if ((lane & 3) == 0)
    scales[(row / kTile) * CSA2_IK4_TILE_SCALE_BYTES +
           block_scale_offset(static_cast<uint32_t>(row % kTile), lane >> 2)] = static_cast<uint8_t>(sc);
}
__device__ __forceinline__ void store_ik4(uint8_t* codes, uint8_t* scales, long long row, float4 k, int lane) {
  uint32_t sc;
  const uint32_t c = fp4_row_lane(k, &sc);
  store_ik4_codes(codes, scales, row, c, sc, lane);
}

}  // namespace csa2
