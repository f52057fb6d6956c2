/*
 * csa2_ops.h -- C ABI of libcsa2.so, the operators around the paged cache of
 * csa2.h: what turns a layer's projections into rotated queries and cache
 * rows, dense attention of new tokens over the whole cache, and the eviction
 * of entries by the attention weight that they have received.
 *
 * The conventions of csa2.h hold: device pointers owned by the caller, host
 * validation before any launch, no allocation or synchronisation, work
 * enqueued on `stream`, data-dependent violations recorded in
 * cache->err_word and never trapping.  csa2_chunk_attn, csa2_attn_mass and
 * csa2_evict take caches of up to 2^30 entries a request (max_pages_per_req *
 * page_size).
 */
#ifndef CSA2_OPS_H
#define CSA2_OPS_H

#include "csa2.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of an argument that may have either. */
typedef enum { CSA2_BF16 = 0, CSA2_F32 = 1 } csa2_dtype;

/*
 * Rotation of the LAST `rot` channels of a row of dim channels by its
 * position: pair i is turned by the angle pos * freqs[i],
 *   (u, v) -> (u cos - v sin, u sin + v cos).
 * The pairs are channels (dim - rot + 2i, dim - rot + 2i + 1) when
 * interleaved != 0, else (dim - rot + i, dim - rot/2 + i).  Angles are formed
 * in float64: in fp32 the angle of position 10^6 is off by up to 0.03.
 *   freqs  float64 [rot / 2] device, radians per position (8-byte aligned;
 *          NULL when rot == 0)
 *   rot    0 .. dim, a multiple of 32
 */
typedef struct csa2_rope {
  const double* freqs;
  int32_t rot;
  int32_t interleaved;
} csa2_rope;

/*
 * csa2_norm_rope -- RMS norm of every head and rotation, in one pass:
 *   y = x * weight / sqrt(mean(x^2) + eps), then the rotation above.
 * fp32 arithmetic (angles float64), one rounding to the output's type.
 *   n_rows    tokens (0 does nothing);  heads >= 1;  dim 128 or 512
 *   x         [n_rows] rows of `heads` x `dim` elements of x_type (16-byte
 *             aligned); consecutive rows are x_stride elements apart
 *             (x_stride >= heads * dim and a multiple of 16 bytes)
 *   weight    float [dim], the same for every head, or NULL (ones); 16-byte
 *             aligned
 *   eps       in [1e-12, 1]
 *   pos       int32 [n_rows] position of each row (any value)
 *   out       [n_rows][heads][dim] of out_type, contiguous, 16-byte aligned.
 *             It may be x itself when the type and the layout are the same;
 *             any other overlap with x is refused.
 * A row that holds a NaN or an infinity follows the formula (NaN where the
 * value is not finite, 0 or NaN elsewhere).
 */
CSA2_API csa2_status csa2_norm_rope(int32_t n_rows, int32_t heads, int32_t dim, const void* x, csa2_dtype x_type,
                                    int64_t x_stride, const float* weight, float eps, const csa2_rope* rope,
                                    const int32_t* pos, void* out, csa2_dtype out_type, void* stream);

/*
 * csa2_norm_rope_append -- norm, rotation and quantise-on-append of new cache
 * rows in one pass: main-KV row kv[i] (512) and indexer key ik[i] (128) are
 * normed (each over its own row) and rotated in float64, rounded once to
 * fp32, and stored exactly as csa2_append_kv stores fp32 rows; with ik4 the
 * indexer key is also stored as csa2_append_ik4 stores it.
 *   kv, ik     rows of `type` elements (16-byte aligned), kv_stride and
 *              ik_stride elements apart (multiples of 16 bytes): they may be
 *              slices of one projection's output
 *   kv_weight  float [512] or NULL, ik_weight float [128] or NULL (16-byte
 *              aligned);  eps in [1e-12, 1]
 *   kv_rope, ik_rope  the rotation of each kind of row
 *   rope_pos   int32 [n_rows] positions for the rotation; NULL: pos (after
 *              an eviction a token's slot is no longer its position)
 *   req, pos   as csa2_append_kv: the slot of each row.  No two rows of one
 *              call may have the same slot.
 * ctx_len is not modified.  Device errors as csa2_append_kv.
 */
CSA2_API csa2_status csa2_norm_rope_append(const csa2_cache* cache, const csa2_ik4* ik4, int32_t n_rows,
                                           csa2_dtype type, const void* kv, int64_t kv_stride, const void* ik,
                                           int64_t ik_stride, const float* kv_weight, const float* ik_weight,
                                           float eps, const csa2_rope* kv_rope, const csa2_rope* ik_rope,
                                           const int32_t* rope_pos, const int32_t* req, const int32_t* pos,
                                           void* stream);

/*
 * csa2_chunk_attn -- dense attention of new tokens over the paged cache
 * (K = V = the dequantised main-KV row, one for all heads):
 *   out = sum_e softmax_e(scale q . v_e) v_e,  lse = ln sum_e exp(scale q . v_e)
 * over the entries e that the query sees: e < min(ctx_len[b],
 * floor((q_pos + 1) / ratio)), the causal rule of csa2_prefill_index.  The new
 * tokens' own rows are appended first; ctx_len counts them.  A query that sees
 * nothing has out = 0 and lse = -inf.
 *   q_start  int32 [batch + 1]: request b's queries are rows q_start[b] ..
 *            q_start[b + 1] - 1 (ascending; 0 .. any number of them).  Rows
 *            from q_start[batch] on (a padded batch) are left untouched.  NULL:
 *            query i belongs to request i (n_queries <= batch), one new token
 *            each.
 *   q_pos    int32 [n_queries] token position of each query (negative: sees
 *            nothing; any order)
 *   ratio    tokens per entry, >= 1
 *   q, out   bf16 [n_queries][H][512], 16-byte aligned; H in {16, 32, 64}.
 *            An out that overlaps q is refused
 *   lse      float [n_queries][H] or NULL
 *   n_queries <= 2^20
 *   workspace  at least csa2_chunk_attn_workspace_bytes bytes, 16-byte
 *            aligned; its contents on entry do not matter.  Two calls in
 *            flight at once must not share it.
 * Dequantised rows are exact in fp16; scores, softmax and sums are fp32, the
 * probabilities are rounded to fp16 for the product with V (by 2^-11 of
 * themselves, or by 2^-32 of the row's largest where they are below 2^-21 of it).
 * Long contexts are cut along the keys by a plan made of the lengths alone: the
 * same lengths give the same bits.
 * Device errors: a page id outside [0, num_pages) under a visible entry
 * (CSA2_ERR_DEVICE_BOUNDS; its entries are left out, as if the query did not
 * see them), a q_start that decreases or leaves [0, n_queries] (the request has
 * no queries), a ctx_len outside [0, capacity] (its queries see nothing); a
 * pipeline wait that runs out -> CSA2_ERR_TIMEOUT (out and lse are then
 * undefined; see csa2_set_wait_limit_ns).
 */
CSA2_API size_t csa2_chunk_attn_workspace_bytes(int32_t batch, int32_t n_queries, int32_t H);
CSA2_API csa2_status csa2_chunk_attn(const csa2_cache* cache, int32_t n_queries, const int32_t* q_start,
                                     const int32_t* q_pos, int32_t ratio, const uint16_t* q, int32_t H, float scale,
                                     uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                                     void* stream);

/*
 * csa2_attn_mass -- the attention weight that every cached entry received:
 *   mass[b][e] += sum over request b's queries i and heads h of
 *                 exp(scale q_ih . v_e - lse_ih)
 * over the entries each query sees (the rule of csa2_chunk_attn); an entry's
 * weights of one call sum to at most (queries) x H.  With ratio, q_start,
 * q_pos, q, H and scale as csa2_chunk_attn took them and the lse it wrote.
 *   mass     float [batch][capacity], added to (zero it once); entries that no
 *            query of the call sees are untouched
 *   workspace  at least csa2_attn_mass_workspace_bytes bytes, as above
 * fp32 sums in an order fixed by the sizes and lengths.  Device errors as
 * csa2_chunk_attn; a pipeline wait that runs out -> CSA2_ERR_TIMEOUT (mass is
 * then undefined).
 */
CSA2_API size_t csa2_attn_mass_workspace_bytes(int32_t batch, int32_t n_queries, int32_t H);
CSA2_API csa2_status csa2_attn_mass(const csa2_cache* cache, int32_t n_queries, const int32_t* q_start,
                                    const int32_t* q_pos, int32_t ratio, const uint16_t* q, int32_t H, float scale,
                                    const float* lse, float* mass, void* workspace, size_t workspace_bytes,
                                    void* stream);

/*
 * csa2_evict -- keep `budget` entries of every longer request and move them to
 * other pages.  Of a request's n = ctx_len entries the first `sink`, the last
 * `recent` and, of those between, the (budget - sink - recent) with the largest
 * mass are kept (ties: the lower index; a NaN counts as the largest, -0 as 0),
 * in their old order: the new cache is the old one without the others.
 * Requests with n <= budget are left where they are.
 *   mass       float [batch][capacity] (from csa2_attn_mass)
 *   budget     1 .. 2^30; sink, recent >= 0, sink + recent <= budget
 *   dst_pages  int32 [batch][dst_width]: the pages that receive a request's
 *              rows (dst_width * page_size >= budget; entries of requests that
 *              are left alone are not read).  They must be free: a page that
 *              holds visible entries of any request, or is given twice, is a
 *              violation and receives nothing.  Pages that requests share
 *              stay as they are.
 *   kept       int32 [batch][budget] out: kept positions, ascending, -1 padded
 *   new_len    int32 [batch] out: min(n, budget)
 *   mass_out   float [batch][dst_width * page_size] or NULL: the kept entries'
 *              mass (requests that are moved, their first `budget` values)
 *   ik4        the FP4 indexer keys to move with the rows, or NULL
 *   workspace  at least csa2_evict_workspace_bytes bytes, 16-byte aligned
 * kept, new_len, mass_out and the workspace overlap neither mass, dst_pages, the
 * page table or ctx_len nor one another (refused).  ctx_len and the page table
 * are not modified: the caller continues with dst_pages and new_len for the
 * requests that were moved and frees their old pages.
 * Device errors: CSA2_ERR_DEVICE_BOUNDS for a bad page (the row is not moved)
 * or ctx_len (the request counts as empty).
 */
CSA2_API size_t csa2_evict_workspace_bytes(int32_t num_pages);
CSA2_API csa2_status csa2_evict(const csa2_cache* cache, const csa2_ik4* ik4, const float* mass, int32_t budget,
                                int32_t sink, int32_t recent, const int32_t* dst_pages, int32_t dst_width,
                                int32_t* kept, int32_t* new_len, float* mass_out, void* workspace,
                                size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CSA2_OPS_H */
