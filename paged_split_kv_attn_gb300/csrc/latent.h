// latent.h -- arguments and launchers of the latent-cache kernels and of the
// draft verification (not installed).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pskv {

struct LatentPrepArgs {
  const void *x;           // bf16 [n][x_token]: latent columns, then the key's rotated ones
  long long x_token;
  int n;
  int dc;                  // latent columns
  float eps;
  int adjacent;            // pairs (2i, 2i + 1) instead of (i, i + 32)
  const float *w;          // [dc] or null (1)
  const float *rope_cos;   // [max_pos][32]
  const float *rope_sin;
  int max_pos;
  int num_q_heads;         // 0: no queries
  const void *q;           // bf16, strides in elements
  long long q_token, q_head;
  void *q_out;
  long long q_out_token, q_out_head;
  const int32_t *row_of, *pos_of, *first_pos;  // first_pos may be null
  const int32_t *page_tables;
  int table_stride;
  const int32_t *pages_of_row;
  int batch;
  void *pool;              // bf16 [num_pages][page_size][dc + 64]
  long long num_pages;
  int page_size;
  void *dense;             // bf16 [n][dc + 64] or null
  int32_t *status;
};

// Absorbed attention: pieces of rows, blocks of 128 query columns.
struct LatentAttnArgs {
  const void *q;               // bf16 [B][T][Hq][dc + 64]
  const void *pool;            // bf16 [num_pages][page_size][dc + 64]
  const int32_t *page_tables;  // [B][table_stride]
  const int32_t *seq_lens;     // [B]
  int32_t *status;
  // partials of groups of 32 query columns (null: one piece a row): m (log2 units) and l
  // [B][groups][num_splits][32], o [B][groups][num_splits][dc / 4][32] float4; then the tiles per
  // piece, for the merge
  float *ws_m, *ws_l, *ws_o;
  int32_t *ws_tiles;
  void *out;                   // [B][T][Hq][dc] of out_dtype
  int out_dtype;
  long long num_pages;
  int table_stride, page_size;
  int batch, num_tokens, num_q_heads;
  int num_splits;              // most pieces of a row
  int tiles_per_piece;
  int clusters;                // CTA pairs to launch
  float scale_log2;
  const unsigned long long *tree_mask;  // [B][T] window tokens each token sees, or null: causal
};

struct ExpandedAttnArgs {
  const void *q;        // bf16 [total_q][H][192]
  const void *kv;       // bf16 [total_k][H][256]
  const void *k_rot;    // bf16 [total_k][k_rot_token], 64 columns used
  long long k_rot_token;
  const int32_t *cu_q, *cu_k;  // [B + 1]
  int batch, num_heads;
  int total_q, total_k;
  long long blocks;     // of 256 queries of a row, over all rows
  float scale_log2;
  void *out;            // [total_q][H][128] of out_dtype
  int out_dtype;
  int32_t *status;
};

struct VerifyArgs {
  const void *target;   // [B][T + 1][V]
  const void *draft;    // [B][T][V] or null
  int dtype;
  const int32_t *drafts;      // [B][T]
  const int32_t *num_drafts;  // [B] or null
  const float *u;             // [B][T + 1]
  int batch, max_drafts, vocab;
  int32_t *tokens;            // [B][T + 1]
  int32_t *accepted;          // [B]
  int32_t *status;
};

cudaError_t launch_latent_prep(const LatentPrepArgs &a, cudaStream_t s);
cudaError_t launch_attn_latent(const LatentAttnArgs &a, int dc, cudaStream_t s);
cudaError_t launch_merge_latent(const LatentAttnArgs &a, int dc, cudaStream_t s);
cudaError_t launch_attn_expanded(const ExpandedAttnArgs &a, cudaStream_t s);
cudaError_t launch_verify_drafts(const VerifyArgs &a, cudaStream_t s);

}  // namespace pskv
