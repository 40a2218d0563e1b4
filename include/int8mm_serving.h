/*
 * int8mm_serving.h -- C ABI of the serving operators that stand beside the
 * decomposed int8 matmul of int8mm.h in a decode step on MI355X (gfx950):
 *
 *   - products of a few rows with 4-bit weights and group scales (int4_*);
 *   - a paged key-value cache in float16, bfloat16 or int8: writing and
 *     reading rows (kv_append, kv_gather), one new token's attention over it
 *     (kv_attention), and the upkeep of its pages (kv_pages_*).
 *
 * The conventions of int8mm.h hold for every entry point here: device
 * pointers owned by the caller, nothing allocated, no host synchronisation,
 * all work enqueued on `stream`, argument checks on the host before anything
 * is enqueued, status codes INT8MM_*, capture in a HIP graph allowed (only
 * kernel launches are recorded and no workspace content is kept between
 * calls).  Indexes that live on the device (page ids, row ids, positions,
 * lengths) are bounds-checked by the kernels: an entry out of range is
 * skipped, as described for each call, and never dereferenced.
 *
 * Limits (ESHAPE beyond): table_rows <= 2^30, table_width * page_size <= 2^30,
 * 1024 kv heads, 65536 query heads, 4096 layers, 2^30 bytes for a page's keys
 * in 16 bits; 2^28 - 32 tokens for a kv_append or kv_gather, B * q_heads <
 * 2^24 for a kv_attention, 16384 rows or pairs for a kv_pages_reserve or _fork,
 * 2^23 rows for a kv_pages_free, 2^30 pairs for a kv_pages_copy.
 */
#ifndef INT8MM_SERVING_H
#define INT8MM_SERVING_H

#include "int8mm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the serving operators. */
#define INT8MM_F16 0
#define INT8MM_BF16 1
#define INT8MM_I8 2 /* caches only */

/* ------------------------------------------------------- 4-bit weights --
 *
 *   Y[m][n] = sum_g s[n][g] * sum_{k in group g} X[m][k] * (q[n][k] - z[n][g])
 *             (+ bias[n]),  rounded once,
 *
 * q the 4-bit codes 0..15, groups of `group` consecutive k (the last one may
 * be shorter), s one float16 scale and z one zero point 0..15 per group and
 * output channel; without zero points z = 8.  Sums are held in fp32.
 *
 * The prepared weight.  Codes are stored in tiles of 16 output channels x 128
 * k (1 KiB), the order in which one wave feeds them to the matrix cores with
 * one 16-byte load a lane: tile (n/16, k/128) at ((n/16)*ceil(K/128) + k/128)
 * * 1024; inside it the dword at 16*l + 4*j (l = 0..63, j = 0..3) holds, for
 * channel l%16 of the tile, the codes of k = 32*j + 8*(l/16) + e, e = 0..7, at
 * bits 4*p(e), p = {0,4,1,5,2,6,3,7}.  Padding rows and columns hold code 8.
 * Group parameters: per tile and channel one entry for each sub-group of
 * min(group, 128) k: a float16 scale, or with zero points a pair of float16
 * (scale, 1024 + z), laid out [n/16][k/128][n%16][sub-group].  A group wider
 * than 128 repeats its entry for every tile it covers.
 */
#define INT4_MAX_K (1 << 20)
#define INT4_MAX_N (1 << 24)
#define INT4_MAX_M (1 << 21)

/* Bytes of the prepared codes, and of the prepared group parameters; -1 for
 * an invalid shape or group.  group: 32, 64, or a multiple of 128. */
INT8MM_API int64_t int4_weight_bytes(int64_t N, int64_t K);
INT8MM_API int64_t int4_param_bytes(int64_t N, int64_t K, int64_t group, int zeros);

/*
 * int4_pack_weight -- already-quantized codes into the prepared form.
 *   codes  [N][K] uint8, values 0..15 (higher bits are ignored).
 *   scales [N][ceil(K/group)] float16; zeros the same shape, uint8 0..15
 *          (higher bits are ignored), or NULL.
 *   Wq     int4_weight_bytes(N, K) bytes out; params int4_param_bytes(N, K,
 *          group, zeros != NULL) bytes out; both 16-byte aligned.
 * N == 0 or K == 0: nothing to do.
 * Errors: EINVAL (null or misaligned pointer), ESHAPE (dimensions, group), EHIP.
 */
INT8MM_API int int4_pack_weight(const uint8_t* codes, int64_t N, int64_t K, int64_t group,
                                const int8mm_half* scales, const uint8_t* zeros, void* Wq,
                                void* params, hipStream_t stream);

/*
 * int4_prepare_weight -- quantizes W [N][K] (dtype INT8MM_F16 or INT8MM_BF16)
 * per output channel and group, and packs it.
 *   symmetric: s = fp16(max|w| / 7), q = clamp(rne(w / s), -8, 7) + 8.
 *   zeros:     lo = min(w, 0), hi = max(w, 0), s = fp16((hi - lo) / 15),
 *              z = clamp(rne(-lo / s), 0, 15), q = clamp(rne(w / s) + z, 0, 15).
 * A scale beyond float16's range is stored as its largest finite value; a
 * group whose scale rounds to 0 gets codes equal to its zero point (8 or z = 0).
 * Finite W.  Errors as int4_pack_weight, EINVAL for another dtype.
 */
INT8MM_API int int4_prepare_weight(const void* W, int dtype, int64_t N, int64_t K, int64_t group,
                                   int zeros, void* Wq, void* params, hipStream_t stream);

/* Bytes of workspace int4_linear needs (256-byte aligned; 0: none) for more
 * than 16 rows, or for rows that are not 16-byte aligned or not a multiple of
 * 8 long; other calls may pass NULL. */
INT8MM_API size_t int4_linear_workspace_size(int64_t M, int64_t K, int64_t N);

/*
 * int4_linear -- the product above.
 *   X    [M][K], dtype INT8MM_F16 or INT8MM_BF16, rows ldx elements apart
 *        (ldx >= K); Y [M][N] and bias [N] (or NULL) of the same dtype.
 *   Wq, params, group, zeros: a prepared weight.
 * Meant for the few rows of a decode step: rows are taken 64 at a time, and
 * each 64 read the weight once.  An infinity or NaN in X (or in a scale) makes
 * what depends on it infinite or NaN, which of the two is unspecified, and
 * nothing else.  In bfloat16 rows finite numbers of 2^113 or more may do the
 * same: the sums are formed with codes 128 larger, and the rest comes off them.
 * M == 0 or N == 0: nothing to do.  K == 0: Y = bias, or 0.  Errors: EINVAL,
 * ESHAPE, EWORKSPACE, EHIP.
 */
INT8MM_API int int4_linear(const void* X, int dtype, int64_t M, int64_t K, int64_t ldx,
                           const void* Wq, const void* params, int64_t N, int64_t group, int zeros,
                           const void* bias, void* Y, void* workspace, size_t workspace_bytes,
                           hipStream_t stream);

/* ------------------------------------------------------ key-value pages --
 *
 * A page holds page_size tokens of all kv heads of one layer.  Keys are
 * [head][token][dim], so that a token's key is one contiguous row; values are
 * [head][dim][token], so that the 8 or 16 consecutive tokens a matrix
 * instruction contracts over are one 16-byte load.  An int8 cache holds codes
 * in [-127, 127] and, per head and token, a = max |x| over the token's dims:
 * a code c stands for c * a / 127 (the convention of the int8 matmul's scales).
 *
 * A sequence is a row of `table` ([*][table_width] page ids) with its number
 * of tokens in lengths[row]; token t of it sits in page table[row][t /
 * page_size] at t % page_size.  refcount[page] counts the rows that hold the
 * page; 0 means free.
 */
typedef struct int8mm_kv {
  void* k;        /* [layers][num_pages][kv_heads][page_size][head_dim] */
  void* v;        /* [layers][num_pages][kv_heads][head_dim][page_size] */
  float* k_scale; /* [layers][num_pages][kv_heads][page_size], INT8MM_I8 only */
  float* v_scale;
  /* distances in elements; the dims of one page are contiguous */
  int64_t k_layer_stride, v_layer_stride, ks_layer_stride, vs_layer_stride;
  int64_t k_page_stride, v_page_stride, ks_page_stride, vs_page_stride;
  int32_t layers;    /* 1 for the calls that work on one layer */
  int32_t num_pages;
  int32_t kv_heads;
  int32_t page_size; /* a power of two, 16 .. 1024 */
  int32_t head_dim;  /* a multiple of 16, 16 .. 256 */
  int32_t dtype;     /* INT8MM_F16, INT8MM_BF16 or INT8MM_I8 */
} int8mm_kv;

#define INT8MM_KV_MAX_PAGES (1 << 22)
#define INT8MM_KV_MAX_PAGE_SIZE 1024
#define INT8MM_KV_MAX_HEAD_DIM 256

/*
 * kv_append -- writes T tokens' keys and values into their pages (quantized
 * for an int8 cache: a = max |x|, code = clamp(rne(127 x / a), -127, 127)).
 *   k, v      [T][kv_heads][head_dim] of `dtype` (F16 or BF16; the cache's own
 *             type unless that is I8), token and head distances in elements.
 *   rows, positions [T] int32: token i goes to position positions[i] of the
 *             sequence in table row rows[i].
 * A token whose row (0 .. table_rows-1), position (0 .. table_width *
 * page_size - 1) or page id is out of range is skipped.  Two tokens of one
 * call for the same place: what it then holds is unspecified.  An int8
 * cache takes finite values; a token with an infinity or NaN reads back as
 * NaN in some or all places.  Errors: EINVAL, ESHAPE, EHIP.
 */
INT8MM_API int kv_append(const void* k, const void* v, int dtype, int64_t T,
                         int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                         int64_t v_head_stride, const int8mm_kv* kv, const int32_t* table,
                         int64_t table_rows, int64_t table_width, const int32_t* rows,
                         const int32_t* positions, hipStream_t stream);

/*
 * kv_gather -- the reverse: the keys and values of T (row, position) places
 * as contiguous rows k, v [T][kv_heads][head_dim] of `dtype` (the cache's own
 * type; F16 or BF16, rounded once, for an int8 cache).  A place out of range
 * gives zeros.  Arguments and errors as kv_append.
 */
INT8MM_API int kv_gather(void* k, void* v, int dtype, int64_t T, const int8mm_kv* kv,
                         const int32_t* table, int64_t table_rows, int64_t table_width,
                         const int32_t* rows, const int32_t* positions, hipStream_t stream);

/* Bytes of workspace kv_attention needs for these sizes (256-byte aligned;
 * 0: none, the workspace may be NULL).  max_len: see kv_attention. */
INT8MM_API size_t kv_attention_workspace_size(int64_t B, int64_t q_heads, int64_t kv_heads,
                                              int64_t head_dim, int64_t max_len);

/*
 * kv_attention -- the attention of one new token per sequence over its pages.
 * With L = lengths[row], lo = window > 0 ? max(0, L - window) : 0, query head
 * h reading kv head h / (q_heads / kv_heads):
 *
 *   s[t] = scale * q[b][h] . k[t]       (softcap c > 0: c * tanh(s / c))
 *   out[b][h] = sum_{lo <= t < L} softmax(s)[t] * v[t],  rounded once
 *   lse[b][h] = log sum_{lo <= t < L} exp(s[t])          (fp32, optional)
 *
 *   q     [B][q_heads][head_dim] of `dtype` (F16 or BF16; the cache's own type
 *         unless that is I8), batch and head distances in elements; 16-byte
 *         aligned rows.  out [B][q_heads][head_dim] contiguous.
 *   rows  [B] int32: the table row and length of each batch entry, or NULL for
 *         0 .. B-1.
 *   max_len: an upper bound on the lengths known to the host (the work is
 *         split by it); a longer sequence is read up to max_len tokens only.
 * No visible token (L <= 0, a row out of range, scores that are all -inf):
 * out 0, lse -inf.  Tokens in pages whose id is out of range are not visible.
 * What the pages hold outside [lo, L) does not matter, NaN included; inside
 * it, infinities and NaN propagate.  Sums, maxima and scores are fp32.
 * Where max_len is above 256 (and the window, if there is one, above 193), the
 * places at which sequences are cut into parts go by the head counts, B,
 * max_len and the lengths of all rows of the call, so another sequence's length
 * may change how this one's sums are rounded.  What other sequences hold never
 * does, and the same call gives the same bits again.
 * Errors: EINVAL, ESHAPE, EWORKSPACE, EHIP.
 */
INT8MM_API int kv_attention(const void* q, int dtype, int64_t B, int64_t q_heads,
                            int64_t q_batch_stride, int64_t q_head_stride, const int8mm_kv* kv,
                            const int32_t* table, int64_t table_rows, int64_t table_width,
                            const int32_t* lengths, const int32_t* rows, int64_t max_len,
                            float scale, int64_t window, float softcap, void* out, float* lse,
                            void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Workspace of kv_pages_reserve, kv_pages_fork and kv_pages_compact for a
 * pool of num_pages and n rows or pairs (256-byte aligned). */
INT8MM_API size_t kv_pages_workspace_size(int64_t num_pages, int64_t n);

/* Per-row results of kv_pages_reserve and kv_pages_fork (on the device). */
#define INT8MM_KV_DONE 0
#define INT8MM_KV_NO_PAGES 1 /* not enough free pages: the row is unchanged */
#define INT8MM_KV_BAD_ROW 2  /* a row out of range, in use, or named twice */

/*
 * kv_pages_copy -- copies n whole pages, every layer: page dst[i] becomes a
 * copy of page src[i].  A pair with an id out of range is skipped.  No page
 * may be the destination of two pairs, or the destination of one and the
 * source of another (unspecified contents otherwise).
 */
INT8MM_API int kv_pages_copy(const int8mm_kv* kv, const int32_t* src, const int32_t* dst,
                             int64_t n, hipStream_t stream);

/*
 * kv_pages_reserve -- grows n sequences to new_lengths[i] tokens: row rows[i]
 * gets the pages it lacks, lowest free ids first, in the order of i, and its
 * length is set.  (kv_append then writes the tokens.)  A length below the
 * present one, beyond the table's width or a row named twice is BAD_ROW (the
 * first naming counts).  When the pages run out, the rows from the first that
 * does not fit on get NO_PAGES, also those that would fit by themselves;
 * rows that need no page are DONE.  status [n] int32 out.
 */
INT8MM_API int kv_pages_reserve(int32_t num_pages, int32_t page_size, int32_t* table,
                                int64_t table_rows, int64_t table_width, int32_t* lengths,
                                int32_t* refcount, const int32_t* rows,
                                const int32_t* new_lengths, int64_t n, int32_t* status,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * kv_pages_fork -- children[i] becomes a sequence with the tokens of
 * parents[i]: whole pages are shared (counted once more), a partly filled
 * last page is copied (all layers) into the lowest free page, in the order
 * of i.  A child must be an empty row (length 0), named once and no pair's
 * parent (BAD_ROW otherwise).  status [n] int32 out, NO_PAGES as above.
 */
INT8MM_API int kv_pages_fork(const int8mm_kv* kv, int32_t* table, int64_t table_rows,
                             int64_t table_width, int32_t* lengths, int32_t* refcount,
                             const int32_t* parents, const int32_t* children, int64_t n,
                             int32_t* status, void* workspace, size_t workspace_bytes,
                             hipStream_t stream);

/*
 * kv_pages_free -- the n sequences' pages are counted down (0: free again),
 * their table rows set to -1 and their lengths to 0.  Rows out of range are
 * skipped; a row named twice is freed once.
 */
INT8MM_API int kv_pages_free(int32_t num_pages, int32_t* table, int64_t table_rows,
                             int64_t table_width, int32_t* lengths, int32_t* refcount,
                             const int32_t* rows, int64_t n, hipStream_t stream);

/*
 * kv_pages_compact -- makes the pool dense: with n_live pages in use, the
 * i-th used page at or above n_live moves (all layers) to the i-th free page
 * below it, and every table entry follows.  refcount_out and table_out may be
 * refcount and table (in place) or other arrays; entries out of range become
 * -1.  n_live [1] int32 out.
 */
INT8MM_API int kv_pages_compact(const int8mm_kv* kv, const int32_t* table, int32_t* table_out,
                                int64_t table_rows, int64_t table_width, const int32_t* refcount,
                                int32_t* refcount_out, int32_t* n_live, void* workspace,
                                size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* INT8MM_SERVING_H */
