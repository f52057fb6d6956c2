// What the two kernels of csa2_chunk_attn share: the workspace of cut tiles
// and the launch that joins them.
#pragma once

#include "dense_plan.cuh"

namespace csa2 {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxRanges = 296;                  // ranges of one launch: two CTAs on each of 148 SMs
constexpr int kWsRows = kMaxRanges * 2 * 64;     // rows of partial results: two tiles per range

// The ranges' records, then two partial results per range (the tile that the
// range starts inside, the tile that it ends inside): 512 sums of each of `rows`
// rows, four channels of all rows together (the writers' lanes are rows), then
// the rows' maxima (log2) and their sums.
struct ChunkWorkspace {
  RangeRecord* rec;
  float* part;
};
__host__ __device__ inline ChunkWorkspace split_chunk_ws(void* ws) {
  ChunkWorkspace w;
  w.rec = static_cast<RangeRecord*>(ws);
  w.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kMaxRanges * sizeof(RangeRecord));
  return w;
}
// Partial result `which` (0: tile started inside, 1: tile ended inside) of a range.
__host__ __device__ inline float* partial_of(const ChunkWorkspace& w, int range, int which, int rows) {
  return w.part + (2 * static_cast<size_t>(range) + which) * (static_cast<size_t>(rows) * (kKvDim + 2));
}

// Where channel ch of a row lies in a partial result.
__host__ __device__ inline int partial_at(int row, int ch, int rows) { return ((ch >> 2) * rows + row) * 4 + (ch & 3); }

template <int kStep>
__device__ __forceinline__ void write_range_record(const DenseArgs& a, const DensePlan& plan, RangeRecord* rec) {
  RangeRecord r = {plan.lo, plan.lo, plan.lo, 0, 0, plan.ctas, 0};
  if (plan.lo < plan.hi) {
    const DenseTile t = dense_tile(a, plan.start);
    r.tile_lo = plan.lo - plan.off;
    r.tile_hi = r.tile_lo + dense_steps<kStep>(t);
    r.q0 = t.q0;
    r.tokens = t.tokens;
  }
  *rec = r;
}

cudaError_t launch_chunk_join(int heads, int tile_rows, int ranges, uint16_t* out, float* lse, void* ws,
                              cudaStream_t stream);
cudaError_t launch_chunk_attn_pair(const DenseArgs& a, const uint16_t* q, float scale, uint16_t* out, float* lse, void* ws,
                                   int num_sms, uint64_t wait_ns, cudaStream_t stream);

}  // namespace csa2
