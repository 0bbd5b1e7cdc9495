// pskv_plan.h -- host-only planning and argument checks (no CUDA calls).
//
// Kept free of CUDA so it can be compiled and tested on any host, including
// under the address and undefined-behaviour sanitizers.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "pskv.h"

struct pskv_layout {
  pskv_layout_desc d;
  int elem_size;    // bytes per element
  int k_row_bytes;  // bytes of one stored key row of one head
  int v_row_bytes;  // bytes of one value row of one head
};

namespace pskv {

// Byte offsets of the workspace sections (each 256-byte aligned): the
// partials only (the merge keeps its group states on chip).
struct WorkspacePlan {
  size_t m_off, l_off, o_off;  // partials: m, l [rows][P], o [rows][P][dv]
  size_t total;
  int groups;  // ng = ceil(P / group)
};

int check_layout_desc(const pskv_layout_desc *d);

// Sizes of the decode workspace for `splits` partitions (merged in groups of `group`).
int plan_workspace(int64_t batch, int64_t num_q_heads, int64_t head_dim_v, int64_t splits,
                   int64_t group, WorkspacePlan *out);

// Checks the host lengths: each in [min_len, table_stride * page_size].
int check_lengths(const pskv_layout *layout, int32_t batch, int32_t table_stride,
                  const int32_t *seq_lens_host, int32_t min_len = 1);

// Automatic split count for `slots` CTA slots (SMs x CTAs per SM), filling
// fill32 / 32 of them.  Byte-bound calls (the split-format single-token decode
// on the tensor-core kernel) fill 27/32: with a few SMs running one CTA
// instead of two the stream still saturates HBM, and fewer, longer pieces
// spend less on each CTA's start and on the merge (measured on GB300 over
// 10.6K-163K keys: 64 pieces of a 304-slot grid beat 76 by 1-3.5 % per call).
// Calls with more arithmetic per byte (folded rows, verify windows, prefill)
// fill every slot.
constexpr int kFillBytes32 = 27;
// Key partitions for the tensor-memory prefill kernel: `units` blocks of 128
// query columns (x KV heads x rows) over `slots` concurrent units (SMs, or SM
// pairs at head dim 512), each block holding up to max_tiles 64-key tiles.
// Splits the keys only when the blocks alone leave slots idle: P = ceil(slots /
// units), at most 32 and at least 4 tiles per partition; with a wave or more
// of blocks, P = 1 (a block's fixed costs and the merge outweigh balancing the
// last wave).
int plan_tc_splits(int64_t units, int slots, int64_t max_tiles);
// Partitions per (row, KV head) for the key-major verify kernel: `units`
// (KV heads x rows) CTAs per partition over `slots` SMs, rows of at most
// max_tiles 128-key tiles.  One wave: P = floor(slots / units), at least 1,
// at most max_tiles / 2 (two tiles per partition) and PSKV_MAX_SPLITS.
int plan_verify_splits(int64_t units, int slots, int64_t max_tiles);
// decode_attn_latent's pieces: each row's tiles of kLatentTile keys are cut into
// pieces of tiles_per_piece, one per CTA pair (`clusters` run at a time) and block of
// 128 query columns (`blocks` of them).  The automatic size is the one of the lowest
// estimate among one piece a row and the smallest pieces that take one to four waves: waves
// x (a piece's start and end, about kLatentPieceTiles tiles of 512 values, + its tiles), and the
// merge, about kLatentMergeTiles, where a row has several.  Given num_splits, the longest
// row's tiles are cut into that many.  Against every split count it is within 5 % of the best on
// rows of 1,000 to 40,000 keys in batches of 1 to 64 (1 x 1,000 keys: one piece 18.7 us, eight
// 10.5; 40 x 1,500: one 28.5, two 41.3).
constexpr int kLatentTile = 128;
constexpr double kLatentPieceTiles = 3.0;
constexpr double kLatentMergeTiles = 2.5;
struct LatentPlan {
  int tiles_per_piece, splits, clusters;  // splits: most pieces of a row
};
LatentPlan plan_latent(int clusters, int head_dim_v, int32_t batch, const int32_t *seq_lens_host, int64_t blocks,
                       int32_t num_splits);
// No plan of `batch` rows with up to `longest` keys has more pieces of a row than this.  (The pieces do
// not grow with the lengths: a batch of even rows that fills the pairs is left whole, and one
// long row between short ones is cut.)
int latent_most_splits(int clusters, int32_t batch, int64_t longest, int64_t blocks, int32_t num_splits);
// kv_fork_rows' blocks.  A block compares its forks with the n of the call.  Up to kFewForks of them it has one piece of a
// fork's page (2,048 forks of 16-row pages in four layers: 31 us, by the rule below 38; 4,096: 72 and 62; 16,384: 716 and
// 220).  Then a piece more (`pieces` of them, all layers) for every kForkScan forks of the call, about as long as a
// piece's copy takes; where a block has all of a fork's pieces, up to kForksTogether forks.
constexpr int kFewForks = 2048;
constexpr int kForkScan = 1024;
constexpr int kForksTogether = 8;
struct ForkBlocks {
  int pieces, forks;  // of a block (several forks: all pieces of each)
};
ForkBlocks fork_blocks(int32_t n, int64_t pieces);
int plan_splits(int slots, int32_t batch, int32_t num_kv_heads, const int32_t *seq_lens_host,
                int fill32 = 32);

// Checks host copies of an append's rows against the leases.
int check_append_host(const pskv_layout *layout, int32_t n, int32_t table_stride, int32_t batch,
                      const int32_t *row_of, const int32_t *pos_of, const int32_t *pages_of_row);

// Which partial kernel family serves (dtype, head_dim_v, group, format); -1 if none.
enum { kKernelMma = 0, kKernelSimt = 1 };
int pick_kernel(int kv_dtype, int head_dim, int group, int format = PSKV_FORMAT_SPLIT);

}  // namespace pskv
