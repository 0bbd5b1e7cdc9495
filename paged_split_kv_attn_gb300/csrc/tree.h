// tree.h -- arguments and launchers of the sampling, drafted-tree and forked-row kernels (not installed).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pskv.h"

namespace pskv {

struct SampleArgs {
  const void *logits;         // row r at logits + r * logits_row (elements)
  long long logits_row;
  int dtype;
  int rows, per_request;      // rows, and rows that share one request's filters
  int vocab;
  const float *temperature;   // [requests] each, or null
  const int32_t *top_k;
  const float *top_p;
  const float *min_p;
  const float *u;             // [rows] or null
  int32_t *tokens;            // [rows] or null
  void *probs;                // [rows][vocab] or null
  int probs_dtype;
  int32_t *status;
};

struct VerifyTreeArgs {
  const int32_t *drafts;      // [B][T]
  const unsigned long long *tree_mask;
  const int32_t *sampled;
  int batch, num_tokens;
  int32_t *tokens, *path;     // [B][T]
  int32_t *kept;              // [B]
  int32_t *status;
};

// The pools of layers of one description.
struct Pools {
  void *k[PSKV_MAX_LAYOUTS];
  void *v[PSKV_MAX_LAYOUTS];  // null for latent rows
  int count;
  int heads, page_size;
  int k_vecs, v_vecs;         // 16-byte vectors of a row of one head (v 0 for latent rows)
  long long num_pages;
  int32_t *status;
};

struct KeepArgs {
  const int32_t *page_tables;  // [B][table_stride]
  int table_stride;
  const int32_t *seq_lens;     // [B]
  const int32_t *path;         // [B][T]
  const int32_t *kept;         // [B]
  int batch, num_tokens;
  int32_t *new_lens;           // [B]
};

struct ForkArgs {
  const int32_t *src, *dst, *new_pages;  // [n]
  int n;
  int32_t *page_tables;        // [B][table_stride]
  int table_stride;
  int32_t *seq_lens, *pages_of_row;
  int batch;
};

cudaError_t launch_sample(const SampleArgs &a, int sms, cudaStream_t s);
cudaError_t launch_verify_tree(const VerifyTreeArgs &a, cudaStream_t s);
cudaError_t launch_keep(const KeepArgs &a, const Pools &p, cudaStream_t s);
cudaError_t launch_fork(const ForkArgs &a, const Pools &p, cudaStream_t s);

}  // namespace pskv
