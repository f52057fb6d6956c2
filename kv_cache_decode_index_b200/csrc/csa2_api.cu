// C ABI of libcsa2.so (declared in include/csa2.h and include/csa2_ops.h): host-side validation,
// TMA tensor maps, launches.  No allocation, no synchronisation except in
// csa2_get_error.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>

#include "common.cuh"
#include "launch.h"

namespace {

thread_local char g_msg[512] = "";

csa2_status fail(csa2_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return s;
}

csa2_status cuda_fail(cudaError_t e, const char* what) {
  return fail(CSA2_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int kMaxBatch = 1024;
constexpr int kMaxK = 4096;
constexpr int kMaxPool = 4096;
constexpr long long kMaxFlatPositions = 65536;        // Top-k without a pool
constexpr long long kMaxPoolSelectBlocks = 16LL * 16384;
constexpr int kMaxPrefillQueries = 1 << 20;

uint64_t g_wait_limit_ns = csa2::kWaitLimitNs;

// Device properties, cached per device ordinal.
struct DeviceInfo {
  int sms = 0;
  int major = 0;
};
std::mutex g_dev_mu;
DeviceInfo g_dev[64];

csa2_status device_info(DeviceInfo* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= 64) return fail(CSA2_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
  std::lock_guard<std::mutex> lk(g_dev_mu);
  if (g_dev[dev].sms == 0) {
    int sms = 0, major = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
    g_dev[dev].sms = sms;
    g_dev[dev].major = major;
  }
  *out = g_dev[dev];
  if (out->major != 10) return fail(CSA2_ERR_UNSUPPORTED, "needs an sm_100 (B200-class) device, found sm_%d", out->major * 10);
  return CSA2_OK;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point.
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

csa2_status encode_rows_map(void* base, long long rows, int row_bytes, int box_rows, CUtensorMapSwizzle swizzle,
                            CUtensorMap* map);

csa2_status encode_ik_map(const csa2_cache* c, int box_rows, CUtensorMap* map) {
  return encode_rows_map(c->ik_codes, static_cast<long long>(c->num_pages) * c->page_size, csa2::kIndexDim, box_rows,
                         CU_TENSOR_MAP_SWIZZLE_128B, map);
}

// 2-D map over `rows` rows of `row_bytes` bytes (uint8), box of box_rows
// full rows.
csa2_status encode_rows_map(void* base, long long rows, int row_bytes, int box_rows, CUtensorMapSwizzle swizzle,
                            CUtensorMap* map) {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
  });
  if (fn == nullptr) return fail(CSA2_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(row_bytes), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(CSA2_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return CSA2_OK;
}

csa2_status check_ik4(const csa2_ik4* ik4) {
  if (ik4 == nullptr || ik4->codes == nullptr || ik4->scales == nullptr || !aligned(ik4->codes, 16) ||
      !aligned(ik4->scales, 16))
    return fail(CSA2_ERR_ARG, "ik4, ik4.codes and ik4.scales must be set and 16-byte aligned");
  return CSA2_OK;
}

long long capacity_of(const csa2_cache* c) {
  return static_cast<long long>(c->max_pages_per_req) * c->page_size;
}

csa2_status check_cache(const csa2_cache* c, bool need_kv, bool need_ik) {
  if (c == nullptr) return fail(CSA2_ERR_ARG, "cache is NULL");
  if (c->page_table == nullptr || c->ctx_len == nullptr || c->err_word == nullptr)
    return fail(CSA2_ERR_ARG, "cache.page_table, ctx_len and err_word must be set");
  if (c->batch < 1 || c->batch > kMaxBatch) return fail(CSA2_ERR_SHAPE, "batch %d outside [1, %d]", c->batch, kMaxBatch);
  if (c->page_size <= 0 || c->page_size % csa2::kTile != 0)
    return fail(CSA2_ERR_SHAPE, "page_size %d must be a positive multiple of 128", c->page_size);
  if (c->num_pages < 1 || c->max_pages_per_req < 1)
    return fail(CSA2_ERR_SHAPE, "num_pages and max_pages_per_req must be >= 1");
  if (static_cast<long long>(c->num_pages) * c->page_size >= (1LL << 31))
    return fail(CSA2_ERR_SHAPE, "num_pages * page_size must stay below 2^31 rows");
  if (capacity_of(c) >= (1LL << 31)) return fail(CSA2_ERR_SHAPE, "max_pages_per_req * page_size must stay below 2^31");
  if (need_kv && (c->kv_codes == nullptr || c->kv_scales == nullptr || !aligned(c->kv_codes, 16) ||
                  !aligned(c->kv_scales, 16)))
    return fail(CSA2_ERR_ARG, "kv_codes and kv_scales must be set and 16-byte aligned");
  if (need_ik && (c->ik_codes == nullptr || c->ik_exp == nullptr || !aligned(c->ik_codes, 16) ||
                  !aligned(c->ik_exp, 16)))
    return fail(CSA2_ERR_ARG, "ik_codes and ik_exp must be set and 16-byte aligned");
  return CSA2_OK;
}

#define CSA2_TRY(expr)                 \
  do {                                 \
    const csa2_status s_ = (expr);     \
    if (s_ != CSA2_OK) return s_;      \
  } while (0)

constexpr int kMaxNormHeads = 4096;
constexpr int kMaxDenseQueries = 1 << 20;
constexpr long long kMaxOpsCapacity = 1 << 30;   // entries a request: positions plus a page or a tile stay in 32 bits

csa2_status check_dtype(csa2_dtype t) {
  return t == CSA2_BF16 || t == CSA2_F32 ? CSA2_OK : fail(CSA2_ERR_ARG, "unknown element type %d", static_cast<int>(t));
}

csa2_status check_rope(const csa2_rope* r, int dim, const char* name) {
  if (r == nullptr) return fail(CSA2_ERR_ARG, "%s must be set", name);
  if (r->rot < 0 || r->rot > dim || r->rot % 32 != 0)
    return fail(CSA2_ERR_SHAPE, "%s.rot %d must be a multiple of 32 in [0, %d]", name, r->rot, dim);
  if (r->rot > 0 && (r->freqs == nullptr || !aligned(r->freqs, 8)))
    return fail(CSA2_ERR_ARG, "%s.freqs must be set and 8-byte aligned", name);
  return CSA2_OK;
}

csa2_status check_eps(float eps) {   // also refuses NaN
  if (!(eps >= 1e-12f && eps <= 1.0f)) return fail(CSA2_ERR_SHAPE, "eps %g outside [1e-12, 1]", static_cast<double>(eps));
  return CSA2_OK;
}

csa2_status check_stride(long long stride, long long width, csa2_dtype t, const char* name) {
  if (stride < width || stride % (t == CSA2_BF16 ? 8 : 4) != 0)
    return fail(CSA2_ERR_SHAPE, "%s %lld must be at least %lld elements and a multiple of 16 bytes", name, stride, width);
  return CSA2_OK;
}

csa2_status check_ops_capacity(const csa2_cache* c) {
  if (capacity_of(c) > kMaxOpsCapacity)
    return fail(CSA2_ERR_SHAPE, "max_pages_per_req * page_size must be at most 2^30 here");
  return CSA2_OK;
}

// What the dense operators (chunk_attn, attn_mass) share.
csa2_status check_dense(const csa2_cache* c, int n_queries, const int32_t* q_start, int ratio, int H, float scale) {
  CSA2_TRY(check_cache(c, true, false));
  CSA2_TRY(check_ops_capacity(c));
  if (n_queries < 0 || n_queries > kMaxDenseQueries)
    return fail(CSA2_ERR_SHAPE, "n_queries %d outside [0, %d]", n_queries, kMaxDenseQueries);
  if (q_start == nullptr && n_queries > c->batch)
    return fail(CSA2_ERR_SHAPE, "without q_start, n_queries (%d) must not exceed batch (%d)", n_queries, c->batch);
  if (ratio < 1) return fail(CSA2_ERR_SHAPE, "ratio %d < 1", ratio);
  if (H != 16 && H != 32 && H != 64) return fail(CSA2_ERR_SHAPE, "H %d not in {16, 32, 64}", H);
  if (!std::isfinite(scale)) return fail(CSA2_ERR_ARG, "scale must be finite");
  return CSA2_OK;
}

// Whether [a, a + a_bytes) and [b, b + b_bytes) meet.
bool overlap(const void* a, unsigned long long a_bytes, const void* b, unsigned long long b_bytes) {
  const unsigned long long x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a_bytes > 0 && b_bytes > 0 && x < y + b_bytes && y < x + a_bytes;
}
// An argument's bytes.
struct Range {
  const char* name;
  const void* at;
  unsigned long long bytes;
};

csa2_status check_workspace(const void* ws, size_t bytes, size_t need, const char* fn) {
  if (ws == nullptr || !aligned(ws, 16)) return fail(CSA2_ERR_ARG, "workspace must be set and 16-byte aligned");
  if (bytes < need) return fail(CSA2_ERR_SHAPE, "workspace_bytes %zu < %zu (%s)", bytes, need, fn);
  return CSA2_OK;
}

csa2_status sparse_attn_impl(const csa2_cache* cache, int32_t n_layers, int32_t n_queries, const int32_t* q_req,
                             const int32_t* const* topk, int32_t k, const uint16_t* const* q, int32_t H, float scale,
                             uint16_t* const* out, void* stream, void* workspace = nullptr,
                             size_t workspace_bytes = 0) {
  CSA2_TRY(check_cache(cache, true, false));
  if (n_layers < 1 || n_layers > CSA2_ATTN_MAX_LAYERS)
    return fail(CSA2_ERR_SHAPE, "n_layers %d outside [1, %d]", n_layers, CSA2_ATTN_MAX_LAYERS);
  if (n_queries < 0) return fail(CSA2_ERR_SHAPE, "n_queries %d < 0", n_queries);
  if (n_queries == 0) return CSA2_OK;
  if (q_req == nullptr && n_queries > cache->batch)
    return fail(CSA2_ERR_SHAPE, "without q_req, n_queries (%d) must not exceed batch (%d)", n_queries, cache->batch);
  if (H != 16 && H != 32 && H != 64) return fail(CSA2_ERR_SHAPE, "H %d not in {16, 32, 64}", H);
  if (k < 1 || k > kMaxK) return fail(CSA2_ERR_SHAPE, "k %d outside [1, %d]", k, kMaxK);
  if (static_cast<long long>(n_layers) * n_queries * 4 >= (1LL << 31))
    return fail(CSA2_ERR_SHAPE, "n_layers * n_queries too large");
  if (topk == nullptr || q == nullptr || out == nullptr) return fail(CSA2_ERR_ARG, "topk, q and out must be set");
  for (int l = 0; l < n_layers; ++l)
    if (topk[l] == nullptr || q[l] == nullptr || out[l] == nullptr || !aligned(q[l], 16) || !aligned(out[l], 16))
      return fail(CSA2_ERR_ARG, "layer %d: topk, q and out (16-byte aligned) must be set", l);
  if (workspace != nullptr) {
    if (!aligned(workspace, 16)) return fail(CSA2_ERR_ARG, "workspace must be 16-byte aligned");
    const size_t need = csa2::attn_workspace_bytes(n_layers, n_queries, H);
    if (workspace_bytes < need)
      return fail(CSA2_ERR_SHAPE, "workspace_bytes %zu < %zu (csa2_attn_workspace_bytes)", workspace_bytes, need);
  }
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  const cudaError_t e = csa2::launch_sparse_attn(*cache, n_layers, n_queries, q_req, topk, k, q, H, scale, out,
                                                 static_cast<cudaStream_t>(stream), nullptr, nullptr, nullptr, 0,
                                                 workspace);
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "sparse_attn launch");
}

}  // namespace

extern "C" {

csa2_status csa2_append_kv(const csa2_cache* cache, int32_t n_rows, const float* kv_new, const float* ik_new,
                           const int32_t* req, const int32_t* pos, void* stream) {
  CSA2_TRY(check_cache(cache, true, true));
  if (n_rows < 0) return fail(CSA2_ERR_SHAPE, "n_rows %d < 0", n_rows);
  if (n_rows == 0) return CSA2_OK;
  if (kv_new == nullptr || ik_new == nullptr || pos == nullptr || !aligned(kv_new, 16) || !aligned(ik_new, 16))
    return fail(CSA2_ERR_ARG, "kv_new, ik_new (16-byte aligned) and pos must be set");
  if (req == nullptr && n_rows > cache->batch)
    return fail(CSA2_ERR_SHAPE, "without req, n_rows (%d) must not exceed batch (%d)", n_rows, cache->batch);
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  const cudaError_t e = csa2::launch_append(*cache, n_rows, kv_new, ik_new, req, pos, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "append_kv launch");
}

csa2_status csa2_compress_append(const csa2_cache* cache, int32_t n_entries, int32_t m, const float* kv_tok,
                                 const float* ik_tok, const int32_t* req, const int32_t* pos, void* stream) {
  CSA2_TRY(check_cache(cache, true, true));
  if (n_entries < 0) return fail(CSA2_ERR_SHAPE, "n_entries %d < 0", n_entries);
  if (m != 1 && m != 2 && m != 4 && m != 8) return fail(CSA2_ERR_SHAPE, "m %d not in {1, 2, 4, 8}", m);
  if (n_entries == 0) return CSA2_OK;
  if (kv_tok == nullptr || ik_tok == nullptr || pos == nullptr || !aligned(kv_tok, 16) || !aligned(ik_tok, 16))
    return fail(CSA2_ERR_ARG, "kv_tok, ik_tok (16-byte aligned) and pos must be set");
  if (static_cast<long long>(n_entries) * m >= (1LL << 31))
    return fail(CSA2_ERR_SHAPE, "n_entries * m must stay below 2^31");
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  const cudaError_t e = csa2::launch_compress_append(*cache, n_entries, m, kv_tok, ik_tok, req, pos,
                                                     static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "compress_append launch");
}

csa2_status csa2_index_full(const csa2_cache* cache, const float* q, const float* w, float* blockmax, float* scores,
                            uint32_t* hist, void* stream) {
  CSA2_TRY(check_cache(cache, false, true));
  if (q == nullptr || w == nullptr || blockmax == nullptr || !aligned(q, 16))
    return fail(CSA2_ERR_ARG, "q (16-byte aligned), w and blockmax must be set");
  if (hist != nullptr && !aligned(hist, 16)) return fail(CSA2_ERR_ARG, "hist must be 16-byte aligned");
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  // With pages of whole 256-position units, one TMA box covers a unit.
  const int whole_units = cache->page_size % (2 * csa2::kTile) == 0;
  CUtensorMap map;
  CSA2_TRY(encode_ik_map(cache, whole_units ? 2 * csa2::kTile : csa2::kTile, &map));
  const cudaError_t e = csa2::launch_index_full(*cache, q, w, blockmax, scores, hist, map, whole_units, d.sms,
                                                g_wait_limit_ns,
                                                static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "index_full launch");
}

csa2_status csa2_append_ik4(const csa2_cache* cache, const csa2_ik4* ik4, int32_t n_rows, const float* ik_new,
                            const int32_t* req, const int32_t* pos, void* stream) {
  CSA2_TRY(check_cache(cache, false, false));
  CSA2_TRY(check_ik4(ik4));
  if (n_rows < 0) return fail(CSA2_ERR_SHAPE, "n_rows %d < 0", n_rows);
  if (n_rows == 0) return CSA2_OK;
  if (ik_new == nullptr || pos == nullptr || !aligned(ik_new, 16))
    return fail(CSA2_ERR_ARG, "ik_new (16-byte aligned) and pos must be set");
  if (req == nullptr && n_rows > cache->batch)
    return fail(CSA2_ERR_SHAPE, "without req, n_rows (%d) must not exceed batch (%d)", n_rows, cache->batch);
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  const cudaError_t e = csa2::launch_append_ik4(*cache, ik4->codes, ik4->scales, n_rows, ik_new, req, pos,
                                                static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "append_ik4 launch");
}

csa2_status csa2_index_full_fp4(const csa2_cache* cache, const csa2_ik4* ik4, const float* q, const float* w,
                                float* blockmax, float* scores, uint32_t* hist, void* stream) {
  CSA2_TRY(check_cache(cache, false, false));
  CSA2_TRY(check_ik4(ik4));
  if (q == nullptr || w == nullptr || blockmax == nullptr || !aligned(q, 16))
    return fail(CSA2_ERR_ARG, "q (16-byte aligned), w and blockmax must be set");
  if (hist != nullptr && !aligned(hist, 16)) return fail(CSA2_ERR_ARG, "hist must be 16-byte aligned");
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  const int whole_units = cache->page_size % (2 * csa2::kTile) == 0;   // one TMA box per unit
  CUtensorMap map;
  CSA2_TRY(encode_rows_map(ik4->codes, static_cast<long long>(cache->num_pages) * cache->page_size,
                           CSA2_IK4_CODE_BYTES, whole_units ? 2 * csa2::kTile : csa2::kTile,
                           CU_TENSOR_MAP_SWIZZLE_64B, &map));
  const cudaError_t e = csa2::launch_index_full_fp4(*cache, ik4->scales, q, w, blockmax, scores, hist, map,
                                                    whole_units, d.sms, g_wait_limit_ns,
                                                    static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "index_full_fp4 launch");
}

csa2_status csa2_pool_select(const csa2_cache* cache, const float* blockmax, uint32_t* hist, int32_t pool_blocks,
                             int32_t* pool, void* stream) {
  CSA2_TRY(check_cache(cache, false, false));
  if (blockmax == nullptr || pool == nullptr) return fail(CSA2_ERR_ARG, "blockmax and pool must be set");
  if (hist != nullptr && !aligned(hist, 16)) return fail(CSA2_ERR_ARG, "hist must be 16-byte aligned");
  if (pool_blocks < 1 || pool_blocks > kMaxPool)
    return fail(CSA2_ERR_SHAPE, "pool_blocks %d outside [1, %d]", pool_blocks, kMaxPool);
  const long long nblk = (capacity_of(cache) + csa2::kBlock - 1) / csa2::kBlock;
  if (nblk > kMaxPoolSelectBlocks)
    return fail(CSA2_ERR_SHAPE, "request capacity %lld positions exceeds the pool-select limit of %lld",
                capacity_of(cache), kMaxPoolSelectBlocks * csa2::kBlock);
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  // Without a histogram the radix passes scan every key: 16 CTAs above
  // 524,288 positions halve the keys per CTA.  With one, the passes only
  // touch the keys of the threshold's bin, and 8 CTAs (up to 16,384 keys
  // each) halve the cost of each pass's exchange instead.
  const long long per_cta = 16384;
  const int cluster = (nblk <= 4LL * per_cta || (hist != nullptr && nblk <= 8LL * per_cta)) ? 8 : 16;
  const cudaError_t e = csa2::launch_pool_select(*cache, blockmax, hist, pool_blocks, pool, cluster,
                                                 static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "pool_select launch");
}

csa2_status csa2_reindex(const csa2_cache* cache, csa2_mode mode, const int32_t* pool, int32_t pool_blocks,
                         const float* q, const float* w, const float* full_scores, const int32_t* prev_topk,
                         int32_t k, int32_t* topk, void* stream) {
  CSA2_TRY(check_cache(cache, false, mode != CSA2_REUSE));
  if (k < 1 || k > kMaxK) return fail(CSA2_ERR_SHAPE, "k %d outside [1, %d]", k, kMaxK);
  if (topk == nullptr) return fail(CSA2_ERR_ARG, "topk must be set");
  if (mode != CSA2_FULL && mode != CSA2_REINDEX && mode != CSA2_REUSE)
    return fail(CSA2_ERR_ARG, "unknown mode %d", static_cast<int>(mode));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (mode == CSA2_REUSE) {
    if (prev_topk == nullptr) return fail(CSA2_ERR_ARG, "REUSE needs prev_topk");
    if (prev_topk == topk) return CSA2_OK;
    DeviceInfo d;
    CSA2_TRY(device_info(&d));
    const cudaError_t e = csa2::launch_copy_topk(prev_topk, topk, static_cast<long long>(cache->batch) * k, s);
    return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "reuse copy launch");
  }
  const float* stored = mode == CSA2_FULL ? full_scores : nullptr;
  if (stored == nullptr && (q == nullptr || w == nullptr || !aligned(q, 16)))
    return fail(CSA2_ERR_ARG, "re-scoring needs q (16-byte aligned) and w");
  int max_blocks;
  if (pool != nullptr) {
    if (pool_blocks < 1 || pool_blocks > kMaxPool)
      return fail(CSA2_ERR_SHAPE, "pool_blocks %d outside [1, %d]", pool_blocks, kMaxPool);
    max_blocks = (pool_blocks + csa2::kReindexPoolCluster - 1) / csa2::kReindexPoolCluster;
  } else {
    if (capacity_of(cache) > kMaxFlatPositions)
      return fail(CSA2_ERR_SHAPE, "Top-k without a pool supports request capacity <= %lld positions (got %lld)",
                  kMaxFlatPositions, capacity_of(cache));
    const long long nblk = (capacity_of(cache) + csa2::kBlock - 1) / csa2::kBlock;
    max_blocks = static_cast<int>((nblk + 7) / 8);
  }
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  CUtensorMap map;
  CSA2_TRY(encode_ik_map(cache, csa2::kBlock, &map));
  const cudaError_t e = csa2::launch_reindex(*cache, pool, pool_blocks, q, w, stored, k, topk, map, max_blocks,
                                             g_wait_limit_ns, s);
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "reindex launch");
}

size_t csa2_reindex_layers_workspace_bytes(int32_t batch, int32_t n_layers, int32_t pool_blocks) {
  return csa2::rescore_workspace_bytes(batch, n_layers, pool_blocks);
}

static csa2_status reindex_layers_impl(const csa2_cache* cache, const csa2_ik4* ik4, int32_t n_layers, const int32_t* pool,
                                int32_t pool_blocks, const float* const* q, const float* const* w, int32_t k,
                                int32_t* const* topk, void* workspace, size_t workspace_bytes, void* stream) {
  CSA2_TRY(check_cache(cache, false, ik4 == nullptr));
  if (ik4 != nullptr) CSA2_TRY(check_ik4(ik4));
  const int max_layers = ik4 != nullptr ? 4 : CSA2_MAX_SCORE_LAYERS;
  if (n_layers < 1 || n_layers > max_layers)
    return fail(CSA2_ERR_SHAPE, "n_layers %d outside [1, %d]", n_layers, max_layers);
  if (pool_blocks < 1 || pool_blocks > kMaxPool)
    return fail(CSA2_ERR_SHAPE, "pool_blocks %d outside [1, %d]", pool_blocks, kMaxPool);
  if (k < 1 || k > kMaxK) return fail(CSA2_ERR_SHAPE, "k %d outside [1, %d]", k, kMaxK);
  if (pool == nullptr || q == nullptr || w == nullptr || topk == nullptr)
    return fail(CSA2_ERR_ARG, "pool, q, w and topk must be set");
  for (int l = 0; l < n_layers; ++l)
    if (q[l] == nullptr || w[l] == nullptr || topk[l] == nullptr || !aligned(q[l], 16))
      return fail(CSA2_ERR_ARG, "layer %d: q (16-byte aligned), w and topk must be set", l);
  if (workspace == nullptr || !aligned(workspace, 16))
    return fail(CSA2_ERR_ARG, "workspace must be set and 16-byte aligned");
  const size_t need = csa2::rescore_workspace_bytes(cache->batch, n_layers, pool_blocks);
  if (workspace_bytes < need)
    return fail(CSA2_ERR_SHAPE, "workspace_bytes %zu < %zu (csa2_reindex_layers_workspace_bytes)", workspace_bytes,
                need);
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  CUtensorMap map;
  if (ik4 != nullptr)
    CSA2_TRY(encode_rows_map(ik4->codes, static_cast<long long>(cache->num_pages) * cache->page_size,
                             CSA2_IK4_CODE_BYTES, csa2::kBlock, CU_TENSOR_MAP_SWIZZLE_64B, &map));
  else
    CSA2_TRY(encode_ik_map(cache, csa2::kBlock, &map));
  const cudaError_t e =
      csa2::launch_rescore_layers(*cache, ik4 != nullptr ? ik4->scales : nullptr, n_layers, pool, pool_blocks, q, w, k,
                                  topk, workspace, map, d.sms, g_wait_limit_ns, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "reindex_layers launch");
}

csa2_status csa2_reindex_layers(const csa2_cache* cache, int32_t n_layers, const int32_t* pool, int32_t pool_blocks,
                                const float* const* q, const float* const* w, int32_t k, int32_t* const* topk,
                                void* workspace, size_t workspace_bytes, void* stream) {
  return reindex_layers_impl(cache, nullptr, n_layers, pool, pool_blocks, q, w, k, topk, workspace, workspace_bytes,
                             stream);
}

csa2_status csa2_reindex_layers_fp4(const csa2_cache* cache, const csa2_ik4* ik4, int32_t n_layers,
                                    const int32_t* pool, int32_t pool_blocks, const float* const* q,
                                    const float* const* w, int32_t k, int32_t* const* topk, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  if (ik4 == nullptr) return fail(CSA2_ERR_ARG, "ik4 must be set");
  return reindex_layers_impl(cache, ik4, n_layers, pool, pool_blocks, q, w, k, topk, workspace, workspace_bytes,
                             stream);
}

csa2_status csa2_pool_candidates(const csa2_cache* shard, const float* blockmax, const int32_t* pool,
                                 int32_t pool_blocks, int32_t block_offset, float* values, int32_t* ids,
                                 void* stream) {
  CSA2_TRY(check_cache(shard, false, false));
  if (blockmax == nullptr || pool == nullptr || values == nullptr || ids == nullptr)
    return fail(CSA2_ERR_ARG, "blockmax, pool, values and ids must be set");
  if (pool_blocks < 1 || pool_blocks > kMaxPool)
    return fail(CSA2_ERR_SHAPE, "pool_blocks %d outside [1, %d]", pool_blocks, kMaxPool);
  if (block_offset < 0 ||
      static_cast<long long>(block_offset) + (capacity_of(shard) + csa2::kBlock - 1) / csa2::kBlock >= (1LL << 31))
    return fail(CSA2_ERR_SHAPE, "block_offset %d: global block ids must lie in [0, 2^31)", block_offset);
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  const cudaError_t e = csa2::launch_pool_candidates(*shard, blockmax, pool, pool_blocks, block_offset, values, ids,
                                                     static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "pool_candidates launch");
}

csa2_status csa2_pool_merge(int32_t n_shards, int32_t batch, int32_t pool_blocks, const float* values,
                            const int32_t* ids, int32_t* pool, void* stream) {
  if (n_shards < 1 || n_shards > CSA2_MAX_SHARDS)
    return fail(CSA2_ERR_SHAPE, "n_shards %d outside [1, %d]", n_shards, CSA2_MAX_SHARDS);
  if (batch < 1 || batch > kMaxBatch) return fail(CSA2_ERR_SHAPE, "batch %d outside [1, %d]", batch, kMaxBatch);
  if (pool_blocks < 1 || pool_blocks > kMaxPool)
    return fail(CSA2_ERR_SHAPE, "pool_blocks %d outside [1, %d]", pool_blocks, kMaxPool);
  if (static_cast<long long>(n_shards) * pool_blocks > 32768)
    return fail(CSA2_ERR_SHAPE, "n_shards * pool_blocks = %lld exceeds 32768 candidates",
                static_cast<long long>(n_shards) * pool_blocks);
  if (values == nullptr || ids == nullptr || pool == nullptr)
    return fail(CSA2_ERR_ARG, "values, ids and pool must be set");
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  const cudaError_t e =
      csa2::launch_pool_merge(n_shards, batch, pool_blocks, values, ids, pool, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "pool_merge launch");
}

csa2_status csa2_sparse_attn(const csa2_cache* cache, int32_t n_queries, const int32_t* q_req, const int32_t* topk,
                             int32_t k, const uint16_t* q, int32_t H, float scale, uint16_t* out, void* stream) {
  const uint16_t* qs[1] = {q};
  uint16_t* os[1] = {out};
  const int32_t* ts[1] = {topk};
  return sparse_attn_impl(cache, 1, n_queries, q_req, ts, k, qs, H, scale, os, stream);
}

csa2_status csa2_swa_append(const csa2_cache* cache, int32_t window, uint8_t* swa_codes, uint8_t* swa_exp,
                            int32_t n_rows, const float* x, const int32_t* req, const int32_t* pos, void* stream) {
  CSA2_TRY(check_cache(cache, false, false));
  if (window < 1 || window > CSA2_SWA_MAX_WINDOW)
    return fail(CSA2_ERR_SHAPE, "window %d outside [1, %d]", window, CSA2_SWA_MAX_WINDOW);
  if (n_rows < 0) return fail(CSA2_ERR_SHAPE, "n_rows %d < 0", n_rows);
  if (n_rows == 0) return CSA2_OK;
  if (swa_codes == nullptr || swa_exp == nullptr || x == nullptr || pos == nullptr || !aligned(swa_codes, 16) ||
      !aligned(x, 16))
    return fail(CSA2_ERR_ARG, "swa_codes (16-byte aligned), swa_exp, x (16-byte aligned) and pos must be set");
  if (req == nullptr && n_rows > cache->batch)
    return fail(CSA2_ERR_SHAPE, "without req, n_rows (%d) must not exceed batch (%d)", n_rows, cache->batch);
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  const cudaError_t e = csa2::launch_swa_append(*cache, window, swa_codes, swa_exp, n_rows, x, req, pos,
                                                static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "swa_append launch");
}

csa2_status csa2_sparse_attn_swa(const csa2_cache* cache, int32_t n_queries, const int32_t* q_req,
                                 const int32_t* topk, int32_t k, const uint8_t* swa_codes, const uint8_t* swa_exp,
                                 int32_t window, const int32_t* q_pos, const uint16_t* q, int32_t H, float scale,
                                 uint16_t* out, void* stream) {
  CSA2_TRY(check_cache(cache, true, false));
  if (window < 1 || window > CSA2_SWA_MAX_WINDOW)
    return fail(CSA2_ERR_SHAPE, "window %d outside [1, %d]", window, CSA2_SWA_MAX_WINDOW);
  if (swa_codes == nullptr || swa_exp == nullptr || q_pos == nullptr || !aligned(swa_codes, 16))
    return fail(CSA2_ERR_ARG, "swa_codes (16-byte aligned), swa_exp and q_pos must be set");
  if (n_queries < 0) return fail(CSA2_ERR_SHAPE, "n_queries %d < 0", n_queries);
  if (n_queries == 0) return CSA2_OK;
  if (q_req == nullptr && n_queries > cache->batch)
    return fail(CSA2_ERR_SHAPE, "without q_req, n_queries (%d) must not exceed batch (%d)", n_queries, cache->batch);
  if (H != 16 && H != 32 && H != 64) return fail(CSA2_ERR_SHAPE, "H %d not in {16, 32, 64}", H);
  if (k < 1 || k > kMaxK) return fail(CSA2_ERR_SHAPE, "k %d outside [1, %d]", k, kMaxK);
  if (topk == nullptr || q == nullptr || out == nullptr || !aligned(q, 16) || !aligned(out, 16))
    return fail(CSA2_ERR_ARG, "topk, q and out (16-byte aligned) must be set");
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  const uint16_t* qs[1] = {q};
  uint16_t* os[1] = {out};
  const int32_t* ts[1] = {topk};
  const cudaError_t e = csa2::launch_sparse_attn(*cache, 1, n_queries, q_req, ts, k, qs, H, scale, os,
                                                 static_cast<cudaStream_t>(stream), swa_codes, swa_exp, q_pos,
                                                 window);
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "sparse_attn_swa launch");
}

csa2_status csa2_sparse_attn_layers(const csa2_cache* cache, int32_t n_layers, int32_t n_queries,
                                    const int32_t* q_req, const int32_t* const* topk, int32_t k, const uint16_t* const* q,
                                    int32_t H, float scale, uint16_t* const* out, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  return sparse_attn_impl(cache, n_layers, n_queries, q_req, topk, k, q, H, scale, out, stream, workspace,
                          workspace_bytes);
}

size_t csa2_attn_workspace_bytes(int32_t n_layers, int32_t n_queries, int32_t H) {
  if (n_layers < 0 || n_queries < 0 || H < 0) return 0;
  return csa2::attn_workspace_bytes(n_layers, n_queries, H);
}

size_t csa2_prefill_workspace_bytes(int32_t n_queries) { return csa2::prefill_workspace_bytes(n_queries); }

csa2_status csa2_prefill_index(const csa2_cache* cache, int32_t req, int32_t n_queries, const int32_t* q_pos,
                               int32_t ratio, const float* q, const float* w, int32_t k, int32_t* topk,
                               void* workspace, size_t workspace_bytes, void* stream) {
  CSA2_TRY(check_cache(cache, false, true));
  if (req < 0 || req >= cache->batch) return fail(CSA2_ERR_SHAPE, "req %d outside [0, %d)", req, cache->batch);
  if (n_queries < 0 || n_queries > kMaxPrefillQueries)
    return fail(CSA2_ERR_SHAPE, "n_queries %d outside [0, %d]", n_queries, kMaxPrefillQueries);
  if (n_queries == 0) return CSA2_OK;
  if (ratio < 1) return fail(CSA2_ERR_SHAPE, "ratio %d < 1", ratio);
  if (k < 1 || k > CSA2_PREFILL_MAX_K) return fail(CSA2_ERR_SHAPE, "k %d outside [1, %d]", k, CSA2_PREFILL_MAX_K);
  if (q_pos == nullptr || q == nullptr || w == nullptr || topk == nullptr || !aligned(q, 16))
    return fail(CSA2_ERR_ARG, "q_pos, q (16-byte aligned), w and topk must be set");
  if (workspace == nullptr || !aligned(workspace, 16))
    return fail(CSA2_ERR_ARG, "workspace must be set and 16-byte aligned");
  if (workspace_bytes < csa2::prefill_workspace_bytes(n_queries))
    return fail(CSA2_ERR_SHAPE, "workspace of %zu bytes, %zu needed", workspace_bytes,
                csa2::prefill_workspace_bytes(n_queries));
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  CUtensorMap map;
  CSA2_TRY(encode_ik_map(cache, csa2::kTile, &map));
  const cudaError_t e = csa2::launch_prefill_index(*cache, req, n_queries, q_pos, ratio, q, w, k, topk, workspace,
                                                   map, g_wait_limit_ns, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "prefill_index launch");
}

csa2_status csa2_prefill_index_static(const csa2_cache* cache, int32_t req, int32_t n_queries,
                                      const int32_t* q_pos, int32_t ratio, const float* q, const float* w,
                                      int32_t k, int32_t* topk, void* stream) {
  if (n_queries > CSA2_PREFILL_STATIC_MAX_QUERIES)
    return fail(CSA2_ERR_SHAPE, "n_queries %d above the static scratch limit of %d", n_queries,
                CSA2_PREFILL_STATIC_MAX_QUERIES);
  if (n_queries <= 0) return csa2_prefill_index(cache, req, n_queries, q_pos, ratio, q, w, k, topk, nullptr, 0, stream);
  // the host-side checks of csa2_prefill_index, before the device is touched
  CSA2_TRY(check_cache(cache, false, true));
  if (req < 0 || req >= cache->batch) return fail(CSA2_ERR_SHAPE, "req %d outside [0, %d)", req, cache->batch);
  if (ratio < 1) return fail(CSA2_ERR_SHAPE, "ratio %d < 1", ratio);
  if (k < 1 || k > CSA2_PREFILL_MAX_K) return fail(CSA2_ERR_SHAPE, "k %d outside [1, %d]", k, CSA2_PREFILL_MAX_K);
  if (q_pos == nullptr || q == nullptr || w == nullptr || topk == nullptr || !aligned(q, 16))
    return fail(CSA2_ERR_ARG, "q_pos, q (16-byte aligned), w and topk must be set");
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  void* scratch = nullptr;
  const cudaError_t e = csa2::static_prefill_scratch(&scratch);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(prefill scratch)");
  return csa2_prefill_index(cache, req, n_queries, q_pos, ratio, q, w, k, topk, scratch,
                            csa2::prefill_workspace_bytes(n_queries), stream);
}

csa2_status csa2_norm_rope(int32_t n_rows, int32_t heads, int32_t dim, const void* x, csa2_dtype x_type,
                           int64_t x_stride, const float* weight, float eps, const csa2_rope* rope,
                           const int32_t* pos, void* out, csa2_dtype out_type, void* stream) {
  if (n_rows < 0) return fail(CSA2_ERR_SHAPE, "n_rows %d < 0", n_rows);
  if (dim != csa2::kIndexDim && dim != csa2::kKvDim) return fail(CSA2_ERR_SHAPE, "dim %d not in {128, 512}", dim);
  if (heads < 1 || heads > kMaxNormHeads) return fail(CSA2_ERR_SHAPE, "heads %d outside [1, %d]", heads, kMaxNormHeads);
  CSA2_TRY(check_dtype(x_type));
  CSA2_TRY(check_dtype(out_type));
  CSA2_TRY(check_rope(rope, dim, "rope"));
  CSA2_TRY(check_eps(eps));
  CSA2_TRY(check_stride(x_stride, static_cast<long long>(heads) * dim, x_type, "x_stride"));
  if (n_rows == 0) return CSA2_OK;
  if (x == nullptr || out == nullptr || pos == nullptr || !aligned(x, 16) || !aligned(out, 16) || !aligned(weight, 16))
    return fail(CSA2_ERR_ARG, "x, out (16-byte aligned) and pos must be set, weight 16-byte aligned");
  const unsigned long long row = static_cast<unsigned long long>(heads) * dim, xs = x_type == CSA2_BF16 ? 2 : 4;
  const bool in_place = out == x && out_type == x_type && (n_rows == 1 || static_cast<unsigned long long>(x_stride) == row);
  if (!in_place && overlap(x, ((n_rows - 1ull) * x_stride + row) * xs, out, n_rows * row * (out_type == CSA2_BF16 ? 2 : 4)))
    return fail(CSA2_ERR_ARG, "out overlaps x without being x");
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  const cudaError_t e = csa2::launch_norm_rope(n_rows, heads, dim, x, x_type, x_stride, weight, eps, *rope, pos, out,
                                               out_type, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "norm_rope launch");
}

csa2_status csa2_norm_rope_append(const csa2_cache* cache, const csa2_ik4* ik4, int32_t n_rows, csa2_dtype type,
                                  const void* kv, int64_t kv_stride, const void* ik, int64_t ik_stride,
                                  const float* kv_weight, const float* ik_weight, float eps,
                                  const csa2_rope* kv_rope, const csa2_rope* ik_rope, const int32_t* rope_pos,
                                  const int32_t* req, const int32_t* pos, void* stream) {
  CSA2_TRY(check_cache(cache, true, true));
  if (ik4 != nullptr) CSA2_TRY(check_ik4(ik4));
  if (n_rows < 0) return fail(CSA2_ERR_SHAPE, "n_rows %d < 0", n_rows);
  CSA2_TRY(check_dtype(type));
  CSA2_TRY(check_rope(kv_rope, csa2::kKvDim, "kv_rope"));
  CSA2_TRY(check_rope(ik_rope, csa2::kIndexDim, "ik_rope"));
  CSA2_TRY(check_eps(eps));
  CSA2_TRY(check_stride(kv_stride, csa2::kKvDim, type, "kv_stride"));
  CSA2_TRY(check_stride(ik_stride, csa2::kIndexDim, type, "ik_stride"));
  if (n_rows == 0) return CSA2_OK;
  if (kv == nullptr || ik == nullptr || pos == nullptr || !aligned(kv, 16) || !aligned(ik, 16) ||
      !aligned(kv_weight, 16) || !aligned(ik_weight, 16))
    return fail(CSA2_ERR_ARG, "kv, ik (16-byte aligned) and pos must be set, the weights 16-byte aligned");
  if (req == nullptr && n_rows > cache->batch)
    return fail(CSA2_ERR_SHAPE, "without req, n_rows (%d) must not exceed batch (%d)", n_rows, cache->batch);
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  const cudaError_t e = csa2::launch_norm_rope_append(*cache, ik4, n_rows, type, kv, kv_stride, ik, ik_stride, kv_weight,
                                                      ik_weight, eps, *kv_rope, *ik_rope, rope_pos, req, pos,
                                                      static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "norm_rope_append launch");
}

size_t csa2_chunk_attn_workspace_bytes(int32_t batch, int32_t n_queries, int32_t H) {
  if (batch < 1 || n_queries < 1 || H < 1) return 0;
  return csa2::chunk_attn_workspace_bytes();
}

csa2_status csa2_chunk_attn(const csa2_cache* cache, int32_t n_queries, const int32_t* q_start, const int32_t* q_pos,
                            int32_t ratio, const uint16_t* q, int32_t H, float scale, uint16_t* out, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream) {
  CSA2_TRY(check_dense(cache, n_queries, q_start, ratio, H, scale));
  if (n_queries == 0) return CSA2_OK;
  if (q_pos == nullptr || q == nullptr || out == nullptr || !aligned(q, 16) || !aligned(out, 16))
    return fail(CSA2_ERR_ARG, "q_pos, q and out (16-byte aligned) must be set");
  CSA2_TRY(check_workspace(workspace, workspace_bytes, csa2_chunk_attn_workspace_bytes(cache->batch, n_queries, H),
                           "csa2_chunk_attn_workspace_bytes"));
  const unsigned long long bytes = 2ull * n_queries * H * csa2::kKvDim;
  if (overlap(q, bytes, out, bytes)) return fail(CSA2_ERR_ARG, "out overlaps q");
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  const cudaError_t e = csa2::launch_chunk_attn(*cache, n_queries, q_start, q_pos, ratio, q, H, scale, out, lse, workspace,
                                                d.sms, g_wait_limit_ns, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "chunk_attn launch");
}

size_t csa2_attn_mass_workspace_bytes(int32_t batch, int32_t n_queries, int32_t H) {
  if (batch < 1 || n_queries < 1 || H < 1) return 0;
  return csa2::attn_mass_workspace_bytes();
}

csa2_status csa2_attn_mass(const csa2_cache* cache, int32_t n_queries, const int32_t* q_start, const int32_t* q_pos,
                           int32_t ratio, const uint16_t* q, int32_t H, float scale, const float* lse, float* mass,
                           void* workspace, size_t workspace_bytes, void* stream) {
  CSA2_TRY(check_dense(cache, n_queries, q_start, ratio, H, scale));
  if (n_queries == 0) return CSA2_OK;
  if (q_pos == nullptr || q == nullptr || lse == nullptr || mass == nullptr || !aligned(q, 16))
    return fail(CSA2_ERR_ARG, "q_pos, q (16-byte aligned), lse and mass must be set");
  CSA2_TRY(check_workspace(workspace, workspace_bytes, csa2_attn_mass_workspace_bytes(cache->batch, n_queries, H),
                           "csa2_attn_mass_workspace_bytes"));
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  const cudaError_t e = csa2::launch_attn_mass(*cache, n_queries, q_start, q_pos, ratio, q, H, scale, lse, mass, workspace,
                                               d.sms, g_wait_limit_ns, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "attn_mass launch");
}

size_t csa2_evict_workspace_bytes(int32_t num_pages) {
  return num_pages < 1 ? 0 : csa2::evict_workspace_bytes(num_pages);
}

csa2_status csa2_evict(const csa2_cache* cache, const csa2_ik4* ik4, const float* mass, int32_t budget, int32_t sink,
                       int32_t recent, const int32_t* dst_pages, int32_t dst_width, int32_t* kept, int32_t* new_len,
                       float* mass_out, void* workspace, size_t workspace_bytes, void* stream) {
  CSA2_TRY(check_cache(cache, true, true));
  if (ik4 != nullptr) CSA2_TRY(check_ik4(ik4));
  CSA2_TRY(check_ops_capacity(cache));
  if (budget < 1 || budget > kMaxOpsCapacity) return fail(CSA2_ERR_SHAPE, "budget %d outside [1, 2^30]", budget);
  if (sink < 0 || recent < 0 || static_cast<long long>(sink) + recent > budget)
    return fail(CSA2_ERR_SHAPE, "sink %d and recent %d must be >= 0 and together at most the budget (%d)", sink, recent, budget);
  if (dst_width < 1 || static_cast<long long>(dst_width) * cache->page_size < budget)
    return fail(CSA2_ERR_SHAPE, "dst_width %d pages hold fewer than budget (%d) rows", dst_width, budget);
  if (static_cast<long long>(cache->batch) * budget >= (1LL << 31))
    return fail(CSA2_ERR_SHAPE, "batch * budget must stay below 2^31");
  if (mass == nullptr || dst_pages == nullptr || kept == nullptr || new_len == nullptr)
    return fail(CSA2_ERR_ARG, "mass, dst_pages, kept and new_len must be set");
  if (dst_pages == cache->page_table) return fail(CSA2_ERR_ARG, "dst_pages must not be the cache's page table");
  CSA2_TRY(check_workspace(workspace, workspace_bytes, csa2_evict_workspace_bytes(cache->num_pages),
                           "csa2_evict_workspace_bytes"));
  // what is written meets nothing that is read, nor one another
  const unsigned long long B = cache->batch, capacity = capacity_of(cache);
  const Range written[] = {{"kept", kept, 4 * B * budget},
                           {"new_len", new_len, 4 * B},
                           {"mass_out", mass_out, mass_out ? 4 * B * dst_width * cache->page_size : 0},
                           {"workspace", workspace, csa2_evict_workspace_bytes(cache->num_pages)}};
  const Range read[] = {{"mass", mass, 4 * B * capacity},
                        {"dst_pages", dst_pages, 4 * B * dst_width},
                        {"page_table", cache->page_table, 4 * B * cache->max_pages_per_req},
                        {"ctx_len", cache->ctx_len, 4 * B}};
  for (const Range& w : written) {
    for (const Range& r : read)
      if (overlap(w.at, w.bytes, r.at, r.bytes)) return fail(CSA2_ERR_ARG, "%s overlaps %s", w.name, r.name);
    for (const Range& o : written)
      if (&o != &w && overlap(w.at, w.bytes, o.at, o.bytes)) return fail(CSA2_ERR_ARG, "%s overlaps %s", w.name, o.name);
  }
  DeviceInfo d;
  CSA2_TRY(device_info(&d));
  const cudaError_t e = csa2::launch_evict(*cache, ik4, mass, budget, sink, recent, dst_pages, dst_width, kept, new_len,
                                           mass_out, workspace, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CSA2_OK : cuda_fail(e, "evict launch");
}

csa2_status csa2_get_error(const csa2_cache* cache, int32_t* out, void* stream) {
  if (cache == nullptr || cache->err_word == nullptr || out == nullptr)
    return fail(CSA2_ERR_ARG, "cache, cache.err_word and out must be set");
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  e = cudaMemcpy(out, cache->err_word, 4 * sizeof(int32_t), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpy(err_word)");
  return static_cast<csa2_status>(out[0]);
}

const char* csa2_status_string(csa2_status s) {
  switch (s) {
    case CSA2_OK: return "ok";
    case CSA2_ERR_ARG: return "invalid argument";
    case CSA2_ERR_SHAPE: return "unsupported shape";
    case CSA2_ERR_CUDA: return "CUDA runtime error";
    case CSA2_ERR_DEVICE_BOUNDS: return "out-of-range page or position found on the device";
    case CSA2_ERR_TIMEOUT: return "a pipeline wait on the device gave up";
    case CSA2_ERR_UNSUPPORTED: return "unsupported device or feature";
  }
  return "unknown status";
}

const char* csa2_last_error_message(void) { return g_msg; }

void csa2_set_wait_limit_ns(uint64_t ns) { g_wait_limit_ns = ns; }

}  // extern "C"
