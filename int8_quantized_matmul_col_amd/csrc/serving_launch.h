// Host-side launchers of the serving kernels (internal; the C ABI is
// include/int8mm_serving.h).  Arguments are validated by serving_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "int8mm_serving.h"

namespace i8mm {

// ---- 4-bit weights: tiles of 16 channels x 128 k, 1 KiB each
constexpr int kInt4TileK = 128;
constexpr int kInt4TileBytes = 1024;
inline int64_t int4_padded_rows(int64_t N) { return (N + 15) / 16 * 16; }
inline int64_t int4_tiles_k(int64_t K) { return (K + kInt4TileK - 1) / kInt4TileK; }
// 32-k steps of a tile that share one parameter entry
inline int int4_group_steps(int64_t group) { return group >= 128 ? 4 : (int)(group / 32); }

hipError_t launch_int4_pack(const uint8_t* codes, int64_t N, int64_t K, int64_t group,
                            const uint16_t* scales, const uint8_t* zeros, uint32_t* Wq,
                            uint16_t* params, hipStream_t s);
hipError_t launch_int4_prepare(const uint16_t* W, bool bf16, int64_t N, int64_t K, int64_t group,
                               bool zeros, uint32_t* Wq, uint16_t* params, hipStream_t s);
struct Int4Args {
  const uint16_t* X;
  const uint8_t* Wq;
  const uint8_t* params;
  const uint16_t* bias;
  uint16_t* Y;
  float* part;  // [int4_k_parts][M][N] if that is more than one
  int64_t ldx;
  int M, K, N;
};
hipError_t launch_int4_linear(const Int4Args& a, bool bf16, int64_t group, bool zeros,
                              hipStream_t s);
// Whether the kernel for up to 16 aligned rows takes them; it needs no
// workspace.  The other splits K into int4_k_parts.
bool int4_few_rows(const uint16_t* X, int64_t M, int64_t K, int64_t ldx);
int int4_k_parts(int64_t M, int64_t K, int64_t N);

// ---- key-value pages
// Tokens, and the most threads, of a workgroup that writes or reads rows.
constexpr int kKvRowsTokens = 32, kKvRowsThreads = 512;
hipError_t launch_kv_append(const uint16_t* k, const uint16_t* v, bool bf16, int T, int64_t kts,
                            int64_t khs, int64_t vts, int64_t vhs, const int8mm_kv& kv,
                            const int32_t* table, int table_rows, int table_width,
                            const int32_t* rows, const int32_t* positions, hipStream_t s);
hipError_t launch_kv_gather(uint16_t* k, uint16_t* v, bool bf16, int T, const int8mm_kv& kv,
                            const int32_t* table, int table_rows, int table_width,
                            const int32_t* rows, const int32_t* positions, hipStream_t s);

// Workgroups that share the batch's tokens evenly for every group of up to 16
// query heads (a second kernel joins sequences that were cut); 0: one
// workgroup for each sequence.  max_len, window: bounds of what one shows.
int kv_attention_parts(int64_t B, int64_t head_groups, int64_t max_len, int64_t window);
// Query heads of one kv head that one wave's matrix tile holds.
constexpr int kKvHeadTile = 16;

struct KvAttentionArgs {
  const uint16_t* q;
  int64_t q_batch_stride, q_head_stride;
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* rows;
  uint16_t* out;
  float* lse;
  float* part_o;   // [head groups][parts][2][tile_heads][head_dim]
  float* part_ml;  // [head groups][parts][2][tile_heads][2]
  int2* cuts;      // [B], where each sequence was cut
  int B, q_heads, group, table_rows, table_width, max_len;  // group: query heads per kv head
  float scale, softcap;
  int64_t window;
  int parts;       // kv_attention_parts
  int tile_heads;  // min(group, kKvHeadTile)
  // A part of a larger sum: tokens before `first` are not taken, and sequences
  // that were not cut go to whole_o [B][q_heads][head_dim] and whole_ml
  // [B][q_heads][2] as the cut ones' parts do, not to out.
  int first;
  float* whole_o;
  float* whole_ml;
};
hipError_t launch_kv_attention(const KvAttentionArgs& a, bool bf16, const int8mm_kv& kv,
                               hipStream_t s);

// ---- queries and keys by their positions
struct QkRopeArgs {
  const uint16_t* q;
  const uint16_t* k;
  uint16_t* q_out;
  uint16_t* k_out;
  const uint16_t* q_weight;  // or null: no norm
  const uint16_t* k_weight;
  const int32_t* positions;
  const uint64_t* turns;
  int64_t q_token, q_head, k_token, k_head, qo_token, qo_head, ko_token, ko_head;  // elements
  int T, q_heads, k_heads, D, rot;
  bool interleaved;
  float factor, eps, inv_dim;
};
hipError_t launch_rope_prepare(const double* inv_freq, int n, uint64_t* turns, hipStream_t s);
hipError_t launch_qk_rope(const QkRopeArgs& a, bool bf16, hipStream_t s);

// ---- the next tokens
constexpr int kSampleChunk = 8192;    // logits of a workgroup
constexpr int kSampleBins = 456;      // 64-bit words that it leaves
constexpr int kSampleMaxChunks = 192;  // of a row, three a lane of a wave
struct SampleHead {
  float top;  // the chunk's maximum
  int first;  // greedy: the first index that has it
  int last;   // the last bin with a token, -1: none
  int bad;    // an infinity or NaN
  double mass;  // of a row without filters, below the chunk's maximum's bin
};
struct SampleArgs {
  const void* logits;
  int64_t row_stride;
  const float* u;
  const float* temperature;  // or null: the one of all rows
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  float temperature_all, top_p_all, min_p_all;
  int32_t top_k_all;
  int32_t* tokens;
  SampleHead* heads;  // [B][S]
  uint64_t* bins;     // [B][S][kSampleBins]
  int B, V, S;
};
// Chunks of a row of V logits that begins anywhere within 16 bytes.
inline int sample_chunks(int64_t V) { return V == 0 ? 0 : (int)((V + 7 + kSampleChunk - 1) / kSampleChunk); }
hipError_t launch_sample(const SampleArgs& a, int dtype, hipStream_t s);

// A prefix that all sequences share: cut into pieces, its rows (a kv head's
// queries of all sequences) padded to tiles.
struct KvSharedPlan {
  int64_t pieces, piece_len, rows_padded;
  int64_t most_pieces;  // grows with prefix_len
};
KvSharedPlan kv_shared_plan(int64_t B, int64_t group, int64_t kv_heads, int64_t head_dim,
                            int64_t prefix_len);
struct KvSharedArgs {
  KvAttentionArgs own;  // the tokens behind the prefix
  const int32_t* prefix_pages;
  float* part_o;   // [kv_heads][pieces][rows_padded][head_dim]
  float* part_ml;  // [kv_heads][pieces][rows_padded][2]
  int prefix_len, pieces, piece_len, rows_padded;
};
hipError_t launch_kv_shared(const KvSharedArgs& a, bool bf16, const int8mm_kv& kv, hipStream_t s);

size_t kv_pages_workspace(int64_t num_pages, int64_t n);
hipError_t launch_kv_pages_copy(const int8mm_kv& kv, const int32_t* src, const int32_t* dst, int n,
                                hipStream_t s);
hipError_t launch_kv_pages_reserve(int num_pages, int page_size, int32_t* table, int table_rows,
                                   int table_width, int32_t* lengths, int32_t* refcount,
                                   const int32_t* rows, const int32_t* new_lengths, int n,
                                   int32_t* status, void* ws, hipStream_t s);
hipError_t launch_kv_pages_extend(int num_pages, int page_size, int32_t* table, int table_rows,
                                  int table_width, int32_t* lengths, int32_t* refcount,
                                  const int32_t* rows, const int32_t* counts, int n, int total,
                                  int32_t* status, int32_t* starts, int32_t* token_rows,
                                  int32_t* positions, void* ws, hipStream_t s);
hipError_t launch_kv_pages_fork(const int8mm_kv& kv, int32_t* table, int table_rows,
                                int table_width, int32_t* lengths, int32_t* refcount,
                                const int32_t* parents, const int32_t* children, int n,
                                int32_t* status, void* ws, hipStream_t s);
hipError_t launch_kv_pages_free(int num_pages, int32_t* table, int table_rows, int table_width,
                                int32_t* lengths, int32_t* refcount, const int32_t* rows, int n,
                                hipStream_t s);
hipError_t launch_kv_pages_compact(const int8mm_kv& kv, const int32_t* table, int32_t* table_out,
                                   int table_rows, int table_width, const int32_t* refcount,
                                   int32_t* refcount_out, int32_t* n_live, void* ws,
                                   hipStream_t s);

// Records a HIP error for int8mm_last_hip_error and returns INT8MM_EHIP
// (api.hip, shared by both ABI files).
int record_hip_error(hipError_t e);

}  // namespace i8mm
