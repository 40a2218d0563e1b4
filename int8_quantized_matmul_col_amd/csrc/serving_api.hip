// C ABI of the serving operators (include/int8mm_serving.h): argument checks,
// workspace carving and launches.  Host code only; nothing is allocated and
// the host never waits on the device.
#include <math.h>

#include "int8mm_serving.h"
#include "serving_launch.h"

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxCount = (int64_t)1 << 30;  // int32 indexing in the kernels
constexpr int64_t kMaxNamed = 16384;             // rows or pairs of one reserve or fork
// a launch holds fewer than 2^32 threads
constexpr int64_t kMaxTokens = (((int64_t)1 << 32) - 1) / i8mm::kKvRowsThreads * i8mm::kKvRowsTokens;
static_assert(kMaxTokens == ((int64_t)1 << 28) - 32, "the limit that the header states");
constexpr int64_t kMaxFreed = (int64_t)1 << 23;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }
int status_of(hipError_t e) { return e == hipSuccess ? INT8MM_OK : i8mm::record_hip_error(e); }

// ------------------------------------------------------------ 4-bit weights

bool int4_shape(int64_t N, int64_t K) {
  return N >= 0 && K >= 0 && K <= INT4_MAX_K && N <= INT4_MAX_N;
}
bool int4_group(int64_t group) {
  return group == 32 || group == 64 || (group >= 128 && group % 128 == 0 && group <= INT4_MAX_K);
}

// ---------------------------------------------------------- key-value pages

// Shape, type and alignment of a cache.  `layered`: the layer strides count.
int check_kv(const int8mm_kv* kv, bool layered) {
  if (kv == nullptr) return INT8MM_EINVAL;
  if (kv->dtype != INT8MM_F16 && kv->dtype != INT8MM_BF16 && kv->dtype != INT8MM_I8) return INT8MM_EINVAL;
  const int64_t ps = kv->page_size, D = kv->head_dim, H = kv->kv_heads;
  if (ps < 16 || ps > INT8MM_KV_MAX_PAGE_SIZE || (ps & (ps - 1)) != 0) return INT8MM_ESHAPE;
  if (D < 16 || D > INT8MM_KV_MAX_HEAD_DIM || D % 16 != 0) return INT8MM_ESHAPE;
  if (H < 1 || H > 1024 || kv->layers < 1 || kv->layers > 4096) return INT8MM_ESHAPE;
  if (kv->num_pages < 0 || kv->num_pages > INT8MM_KV_MAX_PAGES) return INT8MM_ESHAPE;
  // a page's bytes fit 32 bits: 1024 heads * 1024 tokens * 256 dims * 2 would not
  if (H * ps * D * 2 > kMaxCount) return INT8MM_ESHAPE;
  if (kv->num_pages == 0) return INT8MM_OK;
  const bool i8 = kv->dtype == INT8MM_I8;
  if (kv->k == nullptr || kv->v == nullptr) return INT8MM_EINVAL;
  if (i8 && (kv->k_scale == nullptr || kv->v_scale == nullptr)) return INT8MM_EINVAL;
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || (i8 && (!aligned(kv->k_scale, 16) || !aligned(kv->v_scale, 16))))
    return INT8MM_EINVAL;
  // distances keep every page on 16 bytes and pages apart
  const int64_t unit = i8 ? 16 : 8, data = H * ps * D, scales = H * ps;
  auto strides = [&](int64_t page, int64_t layer, int64_t size, int64_t u) {
    return page >= size && page % u == 0 && (!layered || kv->layers == 1 || (layer >= size && layer % u == 0));
  };
  if (!strides(kv->k_page_stride, kv->k_layer_stride, data, unit) ||
      !strides(kv->v_page_stride, kv->v_layer_stride, data, unit))
    return INT8MM_EINVAL;
  if (i8 && (!strides(kv->ks_page_stride, kv->ks_layer_stride, scales, 4) ||
             !strides(kv->vs_page_stride, kv->vs_layer_stride, scales, 4)))
    return INT8MM_EINVAL;
  return INT8MM_OK;
}

// The type of the rows beside a cache.
bool row_type(int dtype, const int8mm_kv* kv) {
  return dtype == INT8MM_F16 || dtype == INT8MM_BF16 ? kv->dtype == INT8MM_I8 || kv->dtype == dtype : false;
}

bool table_shape(int64_t rows, int64_t width, int64_t page_size) {
  // token positions, and sums of two of them, fit int32
  return rows >= 0 && rows <= kMaxCount && width >= 0 && width <= kMaxCount &&
         width * page_size <= kMaxCount;
}

bool workspace_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws != nullptr && aligned(ws, kAlign) && have >= need);
}

struct AttentionSizes {
  size_t part_ml = 0, cuts = 0, total = 0;
};
AttentionSizes attention_sizes(int64_t B, int64_t groups, int64_t tile_heads, int64_t D, int parts) {
  AttentionSizes z;
  if (parts > 0) {
    const size_t n = (size_t)groups * parts * 2 * tile_heads;
    z.part_ml = align_up(n * D * 4);
    z.cuts = z.part_ml + align_up(n * 2 * 4);
    z.total = z.cuts + align_up((size_t)B * 8);
  }
  return z;
}
int64_t tile_heads(int64_t q_heads, int64_t kv_heads) {
  const int64_t group = q_heads / kv_heads;
  return group < i8mm::kKvHeadTile ? group : i8mm::kKvHeadTile;
}
int64_t head_groups(int64_t q_heads, int64_t kv_heads) {
  const int64_t group = q_heads / kv_heads;
  return kv_heads * ((group + i8mm::kKvHeadTile - 1) / i8mm::kKvHeadTile);
}

}  // namespace

extern "C" {

INT8MM_API int64_t int4_weight_bytes(int64_t N, int64_t K) {
  if (!int4_shape(N, K)) return -1;
  return i8mm::int4_padded_rows(N) / 16 * i8mm::int4_tiles_k(K) * i8mm::kInt4TileBytes;
}

INT8MM_API int64_t int4_param_bytes(int64_t N, int64_t K, int64_t group, int zeros) {
  if (!int4_shape(N, K) || !int4_group(group)) return -1;
  const int64_t per = 4 / i8mm::int4_group_steps(group);
  return i8mm::int4_padded_rows(N) * i8mm::int4_tiles_k(K) * per * (zeros ? 4 : 2);
}

INT8MM_API int int4_pack_weight(const uint8_t* codes, int64_t N, int64_t K, int64_t group,
                                const int8mm_half* scales, const uint8_t* zeros, void* Wq,
                                void* params, hipStream_t stream) {
  if (!int4_shape(N, K) || !int4_group(group)) return INT8MM_ESHAPE;
  if (N == 0 || K == 0) return INT8MM_OK;
  if (codes == nullptr || scales == nullptr || Wq == nullptr || params == nullptr) return INT8MM_EINVAL;
  if (!aligned(scales, 2) || !aligned(Wq, 16) || !aligned(params, 16)) return INT8MM_EINVAL;
  return status_of(i8mm::launch_int4_pack(codes, N, K, group, scales, zeros,
                                          static_cast<uint32_t*>(Wq),
                                          static_cast<uint16_t*>(params), stream));
}

INT8MM_API int int4_prepare_weight(const void* W, int dtype, int64_t N, int64_t K, int64_t group,
                                   int zeros, void* Wq, void* params, hipStream_t stream) {
  if (dtype != INT8MM_F16 && dtype != INT8MM_BF16) return INT8MM_EINVAL;
  if (!int4_shape(N, K) || !int4_group(group)) return INT8MM_ESHAPE;
  if (N == 0 || K == 0) return INT8MM_OK;
  if (W == nullptr || Wq == nullptr || params == nullptr) return INT8MM_EINVAL;
  if (!aligned(W, 2) || !aligned(Wq, 16) || !aligned(params, 16)) return INT8MM_EINVAL;
  return status_of(i8mm::launch_int4_prepare(static_cast<const uint16_t*>(W), dtype == INT8MM_BF16,
                                             N, K, group, zeros != 0, static_cast<uint32_t*>(Wq),
                                             static_cast<uint16_t*>(params), stream));
}

INT8MM_API size_t int4_linear_workspace_size(int64_t M, int64_t K, int64_t N) {
  if (!int4_shape(N, K) || M < 0 || M > INT4_MAX_M) return 0;
  if (M == 0 || K == 0 || N == 0) return 0;
  const int parts = i8mm::int4_k_parts(M, K, N);
  return parts > 1 ? align_up((size_t)parts * M * N * 4) : 0;
}

INT8MM_API int int4_linear(const void* X, int dtype, int64_t M, int64_t K, int64_t ldx,
                           const void* Wq, const void* params, int64_t N, int64_t group, int zeros,
                           const void* bias, void* Y, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  if (dtype != INT8MM_F16 && dtype != INT8MM_BF16) return INT8MM_EINVAL;
  if (!int4_shape(N, K) || !int4_group(group) || M < 0 || M > INT4_MAX_M) return INT8MM_ESHAPE;
  if (M == 0 || N == 0) return INT8MM_OK;
  if (ldx < K) return INT8MM_ESHAPE;
  if (Y == nullptr || (K > 0 && (X == nullptr || Wq == nullptr || params == nullptr))) return INT8MM_EINVAL;
  if (!aligned(X, 2) || !aligned(Y, 2) || !aligned(bias, 2) || !aligned(Wq, 16) || !aligned(params, 16))
    return INT8MM_EINVAL;
  i8mm::Int4Args a{};
  a.X = static_cast<const uint16_t*>(X);
  if (K > 0 && !i8mm::int4_few_rows(a.X, M, K, ldx) &&
      !workspace_ok(workspace, workspace_bytes, int4_linear_workspace_size(M, K, N)))
    return INT8MM_EWORKSPACE;
  a.Wq = static_cast<const uint8_t*>(Wq);
  a.params = static_cast<const uint8_t*>(params);
  a.bias = static_cast<const uint16_t*>(bias);
  a.Y = static_cast<uint16_t*>(Y);
  a.part = static_cast<float*>(workspace);
  a.ldx = ldx;
  a.M = (int)M;
  a.K = (int)K;
  a.N = (int)N;
  return status_of(i8mm::launch_int4_linear(a, dtype == INT8MM_BF16, group, zeros != 0, stream));
}

INT8MM_API int kv_append(const void* k, const void* v, int dtype, int64_t T,
                         int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                         int64_t v_head_stride, const int8mm_kv* kv, const int32_t* table,
                         int64_t table_rows, int64_t table_width, const int32_t* rows,
                         const int32_t* positions, hipStream_t stream) {
  const int st = check_kv(kv, false);
  if (st != INT8MM_OK) return st;
  if (!row_type(dtype, kv)) return INT8MM_EINVAL;
  if (T < 0 || T > kMaxTokens || !table_shape(table_rows, table_width, kv->page_size)) return INT8MM_ESHAPE;
  if (T == 0 || kv->num_pages == 0) return INT8MM_OK;
  if (k == nullptr || v == nullptr || rows == nullptr || positions == nullptr) return INT8MM_EINVAL;
  if (table == nullptr && table_rows > 0 && table_width > 0) return INT8MM_EINVAL;
  if (!aligned(k, 2) || !aligned(v, 2) || !aligned(table, 4) || !aligned(rows, 4) || !aligned(positions, 4))
    return INT8MM_EINVAL;
  return status_of(i8mm::launch_kv_append(
      static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), dtype == INT8MM_BF16,
      (int)T, k_token_stride, k_head_stride, v_token_stride, v_head_stride, *kv, table,
      (int)table_rows, (int)table_width, rows, positions, stream));
}

INT8MM_API int kv_gather(void* k, void* v, int dtype, int64_t T, const int8mm_kv* kv,
                         const int32_t* table, int64_t table_rows, int64_t table_width,
                         const int32_t* rows, const int32_t* positions, hipStream_t stream) {
  const int st = check_kv(kv, false);
  if (st != INT8MM_OK) return st;
  if (!row_type(dtype, kv)) return INT8MM_EINVAL;
  if (T < 0 || T > kMaxTokens || !table_shape(table_rows, table_width, kv->page_size)) return INT8MM_ESHAPE;
  if (T == 0) return INT8MM_OK;
  if (k == nullptr || v == nullptr || rows == nullptr || positions == nullptr) return INT8MM_EINVAL;
  if (table == nullptr && table_rows > 0 && table_width > 0) return INT8MM_EINVAL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(table, 4) || !aligned(rows, 4) || !aligned(positions, 4))
    return INT8MM_EINVAL;
  return status_of(i8mm::launch_kv_gather(static_cast<uint16_t*>(k), static_cast<uint16_t*>(v),
                                          dtype == INT8MM_BF16, (int)T, *kv, table,
                                          (int)table_rows, (int)table_width, rows, positions,
                                          stream));
}

INT8MM_API size_t kv_attention_workspace_size(int64_t B, int64_t q_heads, int64_t kv_heads,
                                              int64_t head_dim, int64_t max_len) {
  if (B < 0 || B > kMaxCount || kv_heads < 1 || q_heads < 1 || q_heads % kv_heads != 0 ||
      q_heads > 65536 || head_dim < 16 || head_dim > INT8MM_KV_MAX_HEAD_DIM || max_len < 0 ||
      max_len >= ((int64_t)1 << 31))
    return 0;
  const int64_t groups = head_groups(q_heads, kv_heads);
  return attention_sizes(B, groups, tile_heads(q_heads, kv_heads), head_dim,
                         i8mm::kv_attention_parts(B, groups, max_len, 0)).total;
}

INT8MM_API int kv_attention(const void* q, int dtype, int64_t B, int64_t q_heads,
                            int64_t q_batch_stride, int64_t q_head_stride, const int8mm_kv* kv,
                            const int32_t* table, int64_t table_rows, int64_t table_width,
                            const int32_t* lengths, const int32_t* rows, int64_t max_len,
                            float scale, int64_t window, float softcap, void* out, float* lse,
                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int st = check_kv(kv, false);
  if (st != INT8MM_OK) return st;
  if (!row_type(dtype, kv)) return INT8MM_EINVAL;
  if (B < 0 || q_heads < 1 || q_heads > 65536 || q_heads % kv->kv_heads != 0 ||
      B > kMaxCount || B * q_heads >= ((int64_t)1 << 24) || max_len < 0 || max_len >= ((int64_t)1 << 31) || window < 0 ||
      !table_shape(table_rows, table_width, kv->page_size))
    return INT8MM_ESHAPE;
  if (!isfinite(scale) || !isfinite(softcap) || softcap < 0.0f) return INT8MM_EINVAL;
  if (B == 0) return INT8MM_OK;
  if (q == nullptr || out == nullptr || lengths == nullptr) return INT8MM_EINVAL;
  if (table == nullptr && table_rows > 0 && table_width > 0) return INT8MM_EINVAL;
  if (!aligned(q, 16) || q_batch_stride % 8 != 0 || q_head_stride % 8 != 0 || !aligned(out, 2) ||
      !aligned(lse, 4) || !aligned(table, 4) || !aligned(lengths, 4) || !aligned(rows, 4))
    return INT8MM_EINVAL;
  // what a sequence can show at most, which the split goes by
  int64_t most = table_width * kv->page_size;
  if (most > max_len) most = max_len;
  // units of 128 tokens are counted in 32 bits
  if (B * (most / 128 + 2) > kMaxCount) return INT8MM_ESHAPE;
  const int64_t groups = head_groups(q_heads, kv->kv_heads);
  i8mm::KvAttentionArgs a{};
  if (groups > 65535) return INT8MM_ESHAPE;
  a.parts = i8mm::kv_attention_parts(B, groups, most, window);
  a.tile_heads = (int)tile_heads(q_heads, kv->kv_heads);
  const AttentionSizes z = attention_sizes(B, groups, a.tile_heads, kv->head_dim, a.parts);
  if (!workspace_ok(workspace, workspace_bytes, z.total)) return INT8MM_EWORKSPACE;
  a.q = static_cast<const uint16_t*>(q);
  a.q_batch_stride = q_batch_stride;
  a.q_head_stride = q_head_stride;
  a.table = table;
  a.lengths = lengths;
  a.rows = rows;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + z.part_ml);
  a.cuts = reinterpret_cast<int2*>(static_cast<char*>(workspace) + z.cuts);
  a.B = (int)B;
  a.q_heads = (int)q_heads;
  a.group = (int)(q_heads / kv->kv_heads);
  a.table_rows = (int)table_rows;
  a.table_width = (int)table_width;
  a.max_len = (int)max_len;
  a.scale = scale;
  a.softcap = softcap;
  a.window = window;
  return status_of(i8mm::launch_kv_attention(a, dtype == INT8MM_BF16, *kv, stream));
}

INT8MM_API size_t kv_pages_workspace_size(int64_t num_pages, int64_t n) {
  if (num_pages < 0 || num_pages > INT8MM_KV_MAX_PAGES || n < 0 || n > kMaxNamed) return 0;
  return i8mm::kv_pages_workspace(num_pages, n);
}

INT8MM_API int kv_pages_copy(const int8mm_kv* kv, const int32_t* src, const int32_t* dst,
                             int64_t n, hipStream_t stream) {
  const int st = check_kv(kv, true);
  if (st != INT8MM_OK) return st;
  if (n < 0 || n > kMaxCount) return INT8MM_ESHAPE;
  if (n == 0 || kv->num_pages == 0) return INT8MM_OK;
  if (src == nullptr || dst == nullptr || !aligned(src, 4) || !aligned(dst, 4)) return INT8MM_EINVAL;
  return status_of(i8mm::launch_kv_pages_copy(*kv, src, dst, (int)n, stream));
}

INT8MM_API int kv_pages_reserve(int32_t num_pages, int32_t page_size, int32_t* table,
                                int64_t table_rows, int64_t table_width, int32_t* lengths,
                                int32_t* refcount, const int32_t* rows,
                                const int32_t* new_lengths, int64_t n, int32_t* status,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (num_pages < 0 || num_pages > INT8MM_KV_MAX_PAGES || page_size < 16 ||
      page_size > INT8MM_KV_MAX_PAGE_SIZE || (page_size & (page_size - 1)) != 0)
    return INT8MM_ESHAPE;
  if (n < 0 || n > kMaxNamed || !table_shape(table_rows, table_width, page_size)) return INT8MM_ESHAPE;
  if (n == 0) return INT8MM_OK;
  if (table == nullptr || lengths == nullptr || rows == nullptr || new_lengths == nullptr ||
      status == nullptr || (refcount == nullptr && num_pages > 0))
    return INT8MM_EINVAL;
  if (!aligned(table, 4) || !aligned(lengths, 4) || !aligned(refcount, 4) || !aligned(rows, 4) ||
      !aligned(new_lengths, 4) || !aligned(status, 4))
    return INT8MM_EINVAL;
  if (!workspace_ok(workspace, workspace_bytes, i8mm::kv_pages_workspace(num_pages, n))) return INT8MM_EWORKSPACE;
  return status_of(i8mm::launch_kv_pages_reserve(num_pages, page_size, table, (int)table_rows,
                                                 (int)table_width, lengths, refcount, rows,
                                                 new_lengths, (int)n, status, workspace, stream));
}

INT8MM_API int kv_pages_fork(const int8mm_kv* kv, int32_t* table, int64_t table_rows,
                             int64_t table_width, int32_t* lengths, int32_t* refcount,
                             const int32_t* parents, const int32_t* children, int64_t n,
                             int32_t* status, void* workspace, size_t workspace_bytes,
                             hipStream_t stream) {
  const int st = check_kv(kv, true);
  if (st != INT8MM_OK) return st;
  if (n < 0 || n > kMaxNamed || !table_shape(table_rows, table_width, kv->page_size)) return INT8MM_ESHAPE;
  if (n == 0) return INT8MM_OK;
  if (table == nullptr || lengths == nullptr || parents == nullptr || children == nullptr ||
      status == nullptr || (refcount == nullptr && kv->num_pages > 0))
    return INT8MM_EINVAL;
  if (!aligned(table, 4) || !aligned(lengths, 4) || !aligned(refcount, 4) || !aligned(parents, 4) ||
      !aligned(children, 4) || !aligned(status, 4))
    return INT8MM_EINVAL;
  if (!workspace_ok(workspace, workspace_bytes, i8mm::kv_pages_workspace(kv->num_pages, n)))
    return INT8MM_EWORKSPACE;
  return status_of(i8mm::launch_kv_pages_fork(*kv, table, (int)table_rows, (int)table_width,
                                              lengths, refcount, parents, children, (int)n, status,
                                              workspace, stream));
}

INT8MM_API int kv_pages_free(int32_t num_pages, int32_t* table, int64_t table_rows,
                             int64_t table_width, int32_t* lengths, int32_t* refcount,
                             const int32_t* rows, int64_t n, hipStream_t stream) {
  if (num_pages < 0 || num_pages > INT8MM_KV_MAX_PAGES) return INT8MM_ESHAPE;
  if (n < 0 || n > kMaxFreed || !table_shape(table_rows, table_width, 1)) return INT8MM_ESHAPE;
  if (n == 0) return INT8MM_OK;
  if (table == nullptr || lengths == nullptr || rows == nullptr || (refcount == nullptr && num_pages > 0))
    return INT8MM_EINVAL;
  if (!aligned(table, 4) || !aligned(lengths, 4) || !aligned(refcount, 4) || !aligned(rows, 4))
    return INT8MM_EINVAL;
  return status_of(i8mm::launch_kv_pages_free(num_pages, table, (int)table_rows, (int)table_width,
                                              lengths, refcount, rows, (int)n, stream));
}

INT8MM_API int kv_pages_compact(const int8mm_kv* kv, const int32_t* table, int32_t* table_out,
                                int64_t table_rows, int64_t table_width, const int32_t* refcount,
                                int32_t* refcount_out, int32_t* n_live, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  const int st = check_kv(kv, true);
  if (st != INT8MM_OK) return st;
  if (!table_shape(table_rows, table_width, kv->page_size)) return INT8MM_ESHAPE;
  if (n_live == nullptr || !aligned(n_live, 4)) return INT8MM_EINVAL;
  if (kv->num_pages > 0 && (refcount == nullptr || refcount_out == nullptr)) return INT8MM_EINVAL;
  if (table_rows * table_width > 0 && (table == nullptr || table_out == nullptr)) return INT8MM_EINVAL;
  if (!aligned(table, 4) || !aligned(table_out, 4) || !aligned(refcount, 4) || !aligned(refcount_out, 4))
    return INT8MM_EINVAL;
  if (!workspace_ok(workspace, workspace_bytes, i8mm::kv_pages_workspace(kv->num_pages, 0)))
    return INT8MM_EWORKSPACE;
  return status_of(i8mm::launch_kv_pages_compact(*kv, table, table_out, (int)table_rows,
                                                 (int)table_width, refcount, refcount_out, n_live,
                                                 workspace, stream));
}

}  // extern "C"
