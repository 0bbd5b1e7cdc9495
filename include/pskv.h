/*
 * pskv.h -- paged split-KV GQA attention for single-token decode on GB300
 * (sm_103a).  C ABI: plain pointers and sizes, no C++ or framework types.
 *
 * The operation (sources are web pages, cited by title and section):
 *   For every table row b and query head h, with G = num_q_heads / num_kv_heads
 *   query heads per KV head and kv head g = h / G,
 *     out[b][h][:] = sum_i softmax_i(scale * q[b][h] . k_i) * v_i
 *   over the keys i of row b, where key i lives in page page_tables[b][i / ps]
 *   at row i % ps ("TensorFold #1619 ... caches in pages of the core pool",
 *   description "Paged"; "Parked D512 fused split-KV decode design" (gem),
 *   "Fixed production shape": exact dense attention, 32 q heads over 4 KV
 *   heads, D = 512).
 *   It is computed split-KV: the keys of a row are cut into partitions, each
 *   produces an online-softmax partial (running max m, sum l, unnormalised
 *   numerator o), and the partials are merged in two levels by the exact
 *   rescaling identity m = max(ma, mb), l = la e^(ma-m) + lb e^(mb-m),
 *   o = oa e^(ma-m) + ob e^(mb-m), then out = o / l (gem design, introduction
 *   and "Candidate ownership and storage"; pegainfer #1055 "decode the global
 *   family through a generated split-KV kernel...", Description).
 *   The windowed variant masks keys below a window lower bound (pegainfer
 *   #1057 "serve the sliding family through generated kernels...",
 *   Description).
 *
 * Conventions for every entry point:
 *   - Device pointers are CUDA device memory of the current device; host
 *     pointers are ordinary host memory.  The caller owns all memory; the
 *     library never allocates device memory and never synchronizes a stream.
 *   - Work is enqueued on `stream` (NULL = the legacy default stream) and is
 *     asynchronous; a return of PSKV_OK means it was enqueued.
 *   - Every call returns a status code (PSKV_OK or a negative PSKV_ERR_*).
 *     Host-visible arguments are checked before anything is enqueued; on an
 *     error nothing is enqueued.  Device-side faults (a bad page id, a length
 *     out of range) never trap: the kernel skips the bad access and ORs a
 *     PSKV_FAULT_* bit into the layout's status word, which the caller reads.
 *   - bf16 data is IEEE bfloat16 (1-8-7), f32 is IEEE binary32.
 */
#ifndef PSKV_H
#define PSKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same types as cudaStream_t / cudaEvent_t, declared without CUDA headers. */
typedef struct CUstream_st *pskv_stream_t;
typedef struct CUevent_st *pskv_event_t;

/* ---- status codes --------------------------------------------------------- */
#define PSKV_OK 0
#define PSKV_ERR_INVALID_ARG (-1)          /* a null pointer, a bad size or value */
#define PSKV_ERR_UNSUPPORTED (-2)          /* a shape or format this build refuses */
#define PSKV_ERR_OVERFLOW (-3)             /* a size product overflows size_t */
#define PSKV_ERR_WORKSPACE_TOO_SMALL (-4)
#define PSKV_ERR_PAST_PAGES (-5)           /* an append position past its row's pages */
#define PSKV_ERR_CUDA (-6)                 /* a CUDA runtime call failed */

/* ---- element types and pool formats ---------------------------------------- */
#define PSKV_DTYPE_F32 0
#define PSKV_DTYPE_BF16 1

#define PSKV_FORMAT_SPLIT 0   /* K and V rows kept whole, one region each */
#define PSKV_FORMAT_FOLDED 1  /* K keeps only its first head_dim_v/4 columns (pegainfer #1055's
                                 640-column row at head dim 512), V in full; bf16 only */
#define PSKV_FORMAT_LATENT 2  /* one region: a latent vector and one rotated key per token, shared by
                                 all query heads; bf16 only */

/* ---- which columns the rotation of kv_prep_append_latent pairs ----------------- */
#define PSKV_PAIRS_HALVES 0    /* (i, i + 32) */
#define PSKV_PAIRS_ADJACENT 1  /* (2i, 2i + 1) */

/* ---- device fault bits, ORed into status[0] of the layout's status word ------ */
#define PSKV_FAULT_BAD_PAGE 1u      /* a table entry outside [0, num_pages): that tile or row skipped */
#define PSKV_FAULT_PAST_PAGES 2u    /* an append past its row's pages: that row skipped */
#define PSKV_FAULT_BAD_LENGTH 4u    /* a device length outside [tokens, table_stride * page_size]: clamped */
#define PSKV_FAULT_WAIT_TIMEOUT 8u  /* a bounded wait on a copy expired: the partition was dropped */
#define PSKV_FAULT_EMPTY_ROW 16u    /* a row had no attended key: its output was written as zeros */
#define PSKV_FAULT_BAD_STATE 32u    /* merge input with m = -inf but l != 0, or a NaN m; a sampled row whose filters' border
                                       was not found in the passes that it may take: treated as empty */
#define PSKV_FAULT_BAD_POSITION 64u /* a prep token whose rotation position is outside the table: skipped */
#define PSKV_FAULT_BAD_MASK 128u    /* a tree mask without its own bit or with a later one: later bits ignored */
#define PSKV_FAULT_BAD_TOKEN 256u   /* a drafted token outside the vocabulary: refused like any other */
#define PSKV_FAULT_BAD_ROW 512u     /* a fork's row outside the batch, or one it may not write: that fork skipped */
#define PSKV_FAULT_BAD_PATH 1024u   /* a path that does not go up through its window: that row left as it was */

/* ---- limits ---------------------------------------------------------------- */
#define PSKV_MAX_SPLITS 1024       /* most partitions one decode call may use */
#define PSKV_AUTO_MAX_SPLITS 256   /* most partitions the automatic plan picks */
#define PSKV_MERGE_GROUP 16        /* partials folded per level-1 group of the merge */
#define PSKV_KEY_TILE 16           /* keys per kernel tile; partitions are whole tiles */
#define PSKV_MAX_WINDOW_TOKENS 64  /* query tokens per row of decode_attn_multirow */
#define PSKV_LATENT_ROT 64         /* rotated columns of a latent row (and of its queries) */
#define PSKV_LATENT_MAX_HEADS 128  /* query heads of decode_attn_latent */
#define PSKV_EXPANDED_NOPE 128     /* unrotated columns of an expanded query or key */
#define PSKV_EXPANDED_V 128        /* columns of an expanded value */
#define PSKV_MAX_LAYOUTS 128       /* layouts (layers) of one kv_keep_tokens or kv_fork_rows call */
#define PSKV_MAX_VOCAB 4194304     /* tokens of a row of sample_tokens */
#define PSKV_MAX_SAMPLED 16777216  /* rows (requests * tokens_per_request) of one sample_tokens call */
#define PSKV_MAX_TREES 1048576     /* rows of one verify_tree call */
#define PSKV_MAX_KEPT_ROWS 65535   /* rows of one kv_keep_tokens call */
#define PSKV_MAX_FORKS 65535       /* forks of one kv_fork_rows call */

/* Description of one paged KV pool.
 *
 * k_pool / v_pool are the pool's K region and V region (TensorFold #1619,
 * "Paged": per layer a K region, then a V region; page p is rows
 * [ps*p, ps*(p+1)) of each).  Within a page the rows are head-major, so
 * element (page, kv_head, row, d) of a region is at
 *     ((page * num_kv_heads + kv_head) * page_size + row) * head_dim + d.
 * This keeps one head's keys of a page contiguous (a design choice of this
 * library; the pages do not fix the order inside a page).
 *
 * status: device int32[4] the caller zeroes; kernels OR PSKV_FAULT_* bits into
 * status[0].  May be NULL (faults are then skipped silently).
 * The format is fixed for the pool's life (pegainfer #1055, Description).
 *
 * Folded format (pegainfer #1055, Description: the folded row holds K only
 * where the rotation touches it, V in full, and the prep folds K's norm
 * weight into the query): the K region keeps the first head_dim_v/4 columns
 * of each key (the rotated quarter), the V region all head_dim_v; queries
 * are head_dim_v wide and the score of key i is
 *     scale * (q[0:Dr] . k_i[0:Dr] + q[Dr:Dv] . v_i[Dr:Dv]),  Dr = Dv/4,
 * i.e. the key is taken to equal V outside the rotated quarter once the norm
 * weight sits in q (this library's reading of the page).
 *
 * Latent format: a token keeps one row of head_dim_v + PSKV_LATENT_ROT columns,
 * its normalised latent vector c (head_dim_v columns) and one rotated key r,
 * which every query head shares (num_kv_heads = 1).  k_pool holds the rows,
 * [num_pages][page_size][head_dim_k]; v_pool is NULL: the values are the rows'
 * first head_dim_v columns.  Written by kv_prep_append_latent, read by
 * decode_attn_latent and decode_attn_latent_tree, moved by kv_keep_tokens and kv_fork_rows; every
 * other call refuses the format (UNSUPPORTED). */
typedef struct pskv_layout_desc {
  int64_t num_pages;   /* pages in each region, >= 1 */
  int32_t page_size;   /* keys per page: a multiple of PSKV_KEY_TILE */
  int32_t num_kv_heads;
  int32_t head_dim_k;  /* stored K columns: head_dim_v (split), head_dim_v / 4 (folded) or
                          head_dim_v + PSKV_LATENT_ROT (latent) */
  int32_t head_dim_v;  /* 256 or 512 */
  int32_t kv_dtype;    /* PSKV_DTYPE_F32 or PSKV_DTYPE_BF16 (queries use the same type) */
  int32_t format;      /* PSKV_FORMAT_SPLIT, PSKV_FORMAT_FOLDED or PSKV_FORMAT_LATENT */
  void *k_pool;        /* device, 16-byte aligned */
  void *v_pool;        /* device, 16-byte aligned (latent: NULL) */
  int32_t *status;     /* device int32[4] or NULL */
} pskv_layout_desc;

/* Opaque handle: holds a copy of the description (host memory only). */
typedef struct pskv_layout pskv_layout;

/* Optional per-call settings; pass NULL (or zeroed fields) for the defaults.
 *
 * append_k / append_v / append_pages (single-token decode_attn_splitkv and
 * decode_attn_windowed only): the step's new K/V row of each table row, its
 * key seq_lens[b] - 1, is written into its page by the decode itself, as
 * kv_append_rows would write it (same bits, same checks and fault bits:
 * PSKV_FAULT_PAST_PAGES, PSKV_FAULT_BAD_PAGE) -- TensorFold #1619, "Writes"
 * and "Leasing"; pegainfer #1055, Description (the row written where it is
 * produced).  The CTA whose partition holds that key copies the row before it
 * loads the tile, so the call takes two launches (partial kernel, merge)
 * instead of an append launch plus those two.
 *   append_k      device [batch][num_kv_heads][head_dim_k] of the pool's dtype, 16-byte aligned
 *   append_v      device [batch][num_kv_heads][head_dim_v], 16-byte aligned
 *   append_pages  device int32[batch]: pages leased to each row */
typedef struct pskv_decode_opts {
  int32_t merge_group;        /* partials per level-1 merge group, 1..PSKV_MERGE_GROUP; 0 = PSKV_MERGE_GROUP */
  pskv_event_t partial_begin; /* if not NULL, recorded on the stream just before the partial kernel */
  pskv_event_t partial_end;   /* if not NULL, recorded on the stream just after the partial kernel */
  const void *append_k;       /* the step's new K rows, or NULL (no append) */
  const void *append_v;       /* the step's new V rows */
  const int32_t *append_pages; /* pages leased per row */
} pskv_decode_opts;

/* Validate `desc` and make a layout handle.  Touches no device.
 * Errors: INVALID_ARG (null pointers, sizes < 1, misaligned pools,
 * page_size not a multiple of PSKV_KEY_TILE, unknown format), UNSUPPORTED
 * (head_dim_v not 256/512; split with head_dim_k != head_dim_v; folded with
 * head_dim_k != head_dim_v / 4 or an f32 pool; latent with head_dim_k !=
 * head_dim_v + PSKV_LATENT_ROT, num_kv_heads != 1 or an f32 pool). */
int paged_kv_layout_create(const pskv_layout_desc *desc, pskv_layout **out);

/* Free a handle (NULL is ignored).  The pools are the caller's. */
void paged_kv_layout_destroy(pskv_layout *layout);

/* Append n new rows into the pool, bit for bit (TensorFold #1619, "Writes":
 * rows copied into the pages keep the linear cache's bits).
 *   k_new, v_new     device [n][num_kv_heads][head_dim_k] and [n][num_kv_heads][head_dim_v],
 *                    the pool's dtype, 16-byte aligned
 *   row_of, pos_of   device int32[n]: table row and key position of each new row
 *   page_tables      device int32[batch][table_stride]
 *   pages_of_row     device int32[batch]: pages row b holds (its lease)
 *   row_of_host, pos_of_host, pages_of_row_host: optional host copies of the
 *     same arrays (all three or none).  When given they are checked before
 *     launch and a position at or past pages_of_row[row] * page_size refuses
 *     the whole call with PSKV_ERR_PAST_PAGES (TensorFold #1619, "Leasing":
 *     rows past a slot's pages are refused), nothing enqueued.  Without them
 *     the kernel checks each row and skips a bad one, setting
 *     PSKV_FAULT_PAST_PAGES or PSKV_FAULT_BAD_PAGE.
 * (row, pos) pairs must be distinct within one call. */
int kv_append_rows(const pskv_layout *layout, const void *k_new, const void *v_new,
                   const int32_t *row_of, const int32_t *pos_of, int32_t n,
                   const int32_t *page_tables, int32_t table_stride,
                   const int32_t *pages_of_row, int32_t batch,
                   const int32_t *row_of_host, const int32_t *pos_of_host,
                   const int32_t *pages_of_row_host, pskv_stream_t stream);

/* Rotation and normalisation parameters of kv_prep_append. */
typedef struct pskv_prep_desc {
  int32_t rot_dims;       /* leading columns of each head row rotated: even, 0..head_dim */
  float eps;              /* added to the mean square before the square root */
  const float *w_q;       /* device float[head_dim], 16-byte aligned: query norm
                             multiplier, or NULL (1) */
  const float *w_k;       /* device float[head_dim], 16-byte aligned: key norm
                             multiplier, or NULL (1); required for a folded pool */
  const float *rope_cos;  /* device float[max_pos][rot_dims / 2] */
  const float *rope_sin;  /* device float[max_pos][rot_dims / 2] */
  int32_t max_pos;        /* rows of the tables */
} pskv_prep_desc;

/* K/V prep with the page write fused in (pegainfer #1055, Description: the
 * hd512 prep writes the split or the folded row and folds K's norm weight
 * into the query; pegainfer #1057, Description: elementwise preps with one RMS
 * reduction per head row; TensorFold #1619, "Writes" and "Leasing").  For
 * each new token t (n of them) it takes the projection row
 *   x          device bf16 [n][x_stride], 16-byte aligned, x_stride a multiple of 8;
 *              the query band starts at column q_col (num_q_heads head rows of
 *              head_dim), the key band at k_col and the value band at v_col
 *              (num_kv_heads head rows each); columns multiples of 8
 * and computes per head row r of head_dim columns
 *   r' = r / sqrt(mean(r^2) + eps) * w        (w = w_q for q, w_k for K, 1 for V)
 * then, for q and K, turns the first rot_dims columns as pairs (i, i + rot/2):
 *   r''[i] = a cos - b sin,  r''[i + rot/2] = b cos + a sin
 * with (a, b) = (r'[i], r'[i + rot/2]) and cos, sin = table row p, column i,
 * p = first_pos[row_of[t]] + pos_of[t] (first_pos NULL: 0).  K (its first
 * head_dim_k columns: all of them in a split pool, the rotated quarter in a
 * folded one) and V go straight into page slot pos_of[t] of table row
 * row_of[t], as kv_append_rows would place them; the prepared query goes to
 *   q_out      device bf16 [n][num_q_heads][head_dim], 16-byte aligned
 * and, for a folded pool, its columns past rot_dims are further multiplied by
 * w_k, which makes q_out the folded query decode_attn_* expect.  A folded pool
 * needs rot_dims == head_dim_k, k_col == v_col (K and V from one projection)
 * and w_k.  Values are computed in f32 and rounded to nearest even bf16.
 * Checks, the host copies and the device fault bits are those of
 * kv_append_rows, plus PSKV_FAULT_BAD_POSITION for a table row p outside
 * [0, max_pos) (that token is skipped).  bf16 pools only.
 * Errors: INVALID_ARG, UNSUPPORTED, PAST_PAGES (from the host copies), CUDA. */
int kv_prep_append(const pskv_layout *layout, const pskv_prep_desc *prep, const void *x,
                   int64_t x_stride, int32_t q_col, int32_t k_col, int32_t v_col, int32_t n,
                   int32_t num_q_heads, const int32_t *row_of, const int32_t *pos_of,
                   const int32_t *first_pos, const int32_t *page_tables, int32_t table_stride,
                   const int32_t *pages_of_row, int32_t batch, const int32_t *row_of_host,
                   const int32_t *pos_of_host, const int32_t *pages_of_row_host, void *q_out,
                   pskv_stream_t stream);

/* Split-KV decode: one query token per row.
 *   q              device [batch][num_q_heads][head_dim_v], the pool's dtype (for a
 *                  folded pool, the folded query: see pskv_layout_desc)
 *   page_tables    device int32[batch][table_stride]; entries past a row's
 *                  pages are never read
 *   seq_lens_host  host int32[batch]: keys per row, each in [1, table_stride * page_size];
 *                  the plan (split count, grid) is made from these
 *   seq_lens       device int32[batch]: the same lengths, read by the kernels
 *   scale          score scale (e.g. 1/sqrt(head_dim)); no softcap
 *   num_splits     partitions per (row, KV head): 1..PSKV_MAX_SPLITS, or 0 for
 *                  the automatic plan (pskv_plan_splits).  Keys are cut into
 *                  tiles of PSKV_KEY_TILE; partition p of a row takes tiles
 *                  [p*c, (p+1)*c) of its attended tiles, c = ceil(tiles / num_splits);
 *                  trailing partitions may be empty.
 *   workspace      device scratch of at least decode_attn_workspace_bytes(...)
 *                  bytes, 256-byte aligned (NULL is fine with num_splits = 1 on
 *                  a bf16 pool with 1/2/4/8 query heads per KV head: the one
 *                  partition then writes the output itself and no merge runs).
 *                  Otherwise, on return its head holds the partials: float
 *                  m[batch][num_q_heads][P], then (at the next 256-byte
 *                  boundary) float l[...][P], then float
 *                  o[batch][num_q_heads][P][head_dim] (m in units of the scaled
 *                  score; o of a partition with m = -inf is left unwritten).
 *   out            device [batch][num_q_heads][head_dim] of out_dtype
 *                  (PSKV_DTYPE_BF16, round to nearest even, or PSKV_DTYPE_F32)
 * The result is run-to-run deterministic for a fixed split count.
 * Errors: INVALID_ARG, UNSUPPORTED (num_q_heads % num_kv_heads != 0, or a
 * query-group size this build has no kernel for: bf16 takes 1/2/4/8 query heads
 * per KV head (and 16 at head dim 256, split only), f32 takes 1/2/4/8 (16 at
 * head dim 256)), WORKSPACE_TOO_SMALL, CUDA. */
int decode_attn_splitkv(const pskv_layout *layout, const void *q, const int32_t *page_tables,
                        int32_t table_stride, const int32_t *seq_lens_host,
                        const int32_t *seq_lens, int32_t batch, int32_t num_q_heads, float scale,
                        int32_t num_splits, void *workspace, size_t workspace_bytes, void *out,
                        int32_t out_dtype, const pskv_decode_opts *opts, pskv_stream_t stream);

/* Windowed split-KV decode (pegainfer #1057, Description: the resident pages
 * hold up to a page more than the window and those keys are masked).  As
 * decode_attn_splitkv, plus:
 *   first_pos   device int32[batch]: key i of row b has position first_pos[b] + i
 *   window_lo   device int32[batch]: key i is attended iff its position >= window_lo[b]
 * Keys below the bound are neither loaded nor used; partitions cover only the
 * tiles from the one holding the first attended key.  A row whose bound
 * excludes every key gets zeros and PSKV_FAULT_EMPTY_ROW. */
int decode_attn_windowed(const pskv_layout *layout, const void *q, const int32_t *page_tables,
                         int32_t table_stride, const int32_t *seq_lens_host,
                         const int32_t *seq_lens, const int32_t *first_pos,
                         const int32_t *window_lo, int32_t batch, int32_t num_q_heads,
                         float scale, int32_t num_splits, void *workspace,
                         size_t workspace_bytes, void *out, int32_t out_dtype,
                         const pskv_decode_opts *opts, pskv_stream_t stream);

/* Multi-row split-KV decode: num_tokens query tokens per row, the row's last
 * num_tokens keys (a verify window; TensorFold #1619, description "Reads" and
 * the review thread: drafted verify windows and tree-attention rows read
 * their keys through the page table).  Token t of row b sits at key
 * seq_lens[b] - num_tokens + t and attends keys [0, seq_lens[b] - num_tokens + t]
 * (causal inside the window).  As decode_attn_splitkv, except:
 *   q           device [batch][num_tokens][num_q_heads][head_dim_v]
 *   out         device [batch][num_tokens][num_q_heads][head_dim_v] of out_dtype
 *   num_tokens  1..PSKV_MAX_WINDOW_TOKENS.  The window's query columns per KV
 *               head (query heads per KV head x num_tokens) are served 8 per
 *               CTA when they fit in 8, else 16 per CTA, the CTAs of one
 *               partition reading the same keys (the later ones mostly from L2);
 *               on bf16 split pools of head dim 256 or 512, 17 to 64 columns
 *               by the key-major tensor-memory kernel when the longest row
 *               has at least 8,192 keys (128 keys per tile as the MMA's M,
 *               the columns as its N, one CTA per partition streaming the
 *               keys once), and otherwise from 40 columns on by the
 *               query-major tensor-memory kernel, 128 columns per CTA (pair)
 *   seq_lens    every length at least num_tokens
 *   workspace   decode_attn_workspace_bytes(batch * num_tokens, num_q_heads, ...)
 *               bytes; its partials are laid out as for batch * num_tokens rows
 *               (row b * num_tokens + t)
 * bf16 pools with 1/2/4/8 query heads per KV head (any power of two up to
 * 128 when the window has more than 16 columns on a split pool); no key window.
 * num_tokens = 1 gives decode_attn_splitkv's bits.
 * Errors: INVALID_ARG (also a host length below num_tokens), UNSUPPORTED,
 * WORKSPACE_TOO_SMALL, CUDA. */
int decode_attn_multirow(const pskv_layout *layout, const void *q, const int32_t *page_tables,
                         int32_t table_stride, const int32_t *seq_lens_host,
                         const int32_t *seq_lens, int32_t batch, int32_t num_tokens,
                         int32_t num_q_heads, float scale, int32_t num_splits, void *workspace,
                         size_t workspace_bytes, void *out, int32_t out_dtype,
                         const pskv_decode_opts *opts, pskv_stream_t stream);

/* Tree attention over a drafted window read through the page table
 * (TensorFold #1619, description "Reads" and review thread: tree-attention
 * rows read their keys from a page table, next to drafted verify windows).
 * The window's num_tokens drafted tokens are row b's last keys (already
 * appended), ordered so that every token comes after its ancestors.  Token t
 * sits at key w0 + t, w0 = seq_lens[b] - num_tokens, and attends every key
 * before the window and the window keys w0 + j, j <= t, whose bit j is set in
 * its mask.  As decode_attn_multirow, except:
 *   tree_mask   device uint64[batch][num_tokens]: bit j of the mask of token t
 *               of row b marks window token j as visible to it; a valid mask
 *               holds bit t (the token itself) and no bit above t.  A mask
 *               without bit t or with a later bit sets PSKV_FAULT_BAD_MASK
 *               (the later bits are ignored; the token attends what the
 *               remaining bits and the prefix give it)
 * A chain (the mask of token t = bits 0..t) gives decode_attn_multirow's
 * causal window.  Routing as for decode_attn_multirow, except that windows
 * the query-major tensor-memory kernel would take run on the split-KV
 * kernels instead: bf16 (or folded) pools with 1/2/4/8 query heads per KV
 * head, 8 or 16 columns per CTA; on bf16 split pools of head dim 256 or 512,
 * 17 to 64 columns per KV head on the key-major kernel when the longest row
 * has at least 8,192 keys (there also with 16 to 64 query heads per KV head).
 * Errors: INVALID_ARG (also a host length below num_tokens, a null mask),
 * UNSUPPORTED, WORKSPACE_TOO_SMALL, CUDA. */
int decode_attn_tree(const pskv_layout *layout, const void *q, const int32_t *page_tables,
                     int32_t table_stride, const int32_t *seq_lens_host, const int32_t *seq_lens,
                     const uint64_t *tree_mask, int32_t batch, int32_t num_tokens,
                     int32_t num_q_heads, float scale, int32_t num_splits, void *workspace,
                     size_t workspace_bytes, void *out, int32_t out_dtype,
                     const pskv_decode_opts *opts, pskv_stream_t stream);

/* Paged prefill over variable-length chunks (pegainfer #1057, Description:
 * the sliding family's prompt rows read through a windowed varlen kernel
 * with a window lower bound; pegainfer #1055, Description: a generated
 * prefill beside the split-KV decode).  Row b's new tokens are its last
 * T_b = cu_q[b+1] - cu_q[b] keys, already in the pool (kv_append_rows or
 * kv_prep_append); token t sits at key own = seq_lens[b] - T_b + t and
 * attends keys [lo, own], lo = max(0, own - window + 1) when window > 0, else
 * 0.  As decode_attn_multirow, except:
 *   q            device [cu_q[batch]][num_q_heads][head_dim_v] (packed rows)
 *   cu_q_host    host int32[batch + 1]: 0, then non-decreasing, T_b <= seq_lens[b]
 *   cu_q         device int32[batch + 1]: the same offsets, read by the kernels
 *                (rows outside [0, cu_q_host[batch]] are never addressed)
 *   window       keys a token sees, itself included; 0 = all earlier keys
 *   out          device [cu_q[batch]][num_q_heads][head_dim_v] of out_dtype
 *   workspace    decode_attn_workspace_bytes(cu_q[batch], num_q_heads, ...)
 *                bytes; NULL is fine when the plan has one partition (the
 *                automatic plan for long chunks): each CTA then writes its
 *                normalised output directly and no merge runs
 * Split-format bf16 pools of head dim 256 or 512 run on the tensor-memory
 * kernel: a CTA (head dim 512: a cluster of two, each holding half of the
 * head dim) serves 128 query columns (query heads of a KV head x tokens) of
 * one row, for 1, 2, 4, ..., 128 query heads per KV head; its keys are those
 * its tokens see.  Folded bf16 pools run 16 columns per CTA on the split-KV
 * kernels, with 1/2/4/8 query heads per KV head.  Other pools: UNSUPPORTED.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE_TOO_SMALL, CUDA. */
int prefill_attn_paged(const pskv_layout *layout, const void *q, const int32_t *cu_q_host,
                       const int32_t *cu_q, const int32_t *page_tables, int32_t table_stride,
                       const int32_t *seq_lens_host, const int32_t *seq_lens, int32_t batch,
                       int32_t num_q_heads, int32_t window, float scale, int32_t num_splits,
                       void *workspace, size_t workspace_bytes, void *out, int32_t out_dtype,
                       const pskv_decode_opts *opts, pskv_stream_t stream);

/* ---- the latent cache --------------------------------------------------------
 *
 * Latent attention keeps one latent vector c and one rotated key r a token
 * instead of keys and values per head.  Head h's key is [U_h c, r] and its
 * value W_h c for up-projections U_h, W_h.  In the absorbed form the query is
 * taken through U_h^T once, q_h = [U_h^T qn_h, qr_h], so that the score of key i
 * is scale * q_h . [c_i, r_i] and the output sum_i softmax_i c_i, taken through
 * W_h afterwards by the caller (decode_attn_latent reads the cache alone).  In
 * the expanded form keys and values are formed for every head first
 * (prefill_attn_expanded): fewer operations for long chunks.  Both forms give
 * the same attention. */

/* Parameters of kv_prep_append_latent. */
typedef struct pskv_latent_prep_desc {
  float eps;              /* added to the mean square before the square root, >= 0 */
  int32_t pairs;          /* PSKV_PAIRS_HALVES or PSKV_PAIRS_ADJACENT */
  const float *w;         /* device float[head_dim_v], 16-byte aligned: the latent's norm
                             multiplier, or NULL (1) */
  const float *rope_cos;  /* device float[max_pos][PSKV_LATENT_ROT / 2], 16-byte aligned */
  const float *rope_sin;  /* the same */
  int32_t max_pos;        /* rows of the tables */
  int32_t num_q_heads;    /* query heads to rotate, 0 = none */
  const void *q;          /* device bf16, the queries' rotated columns: PSKV_LATENT_ROT of head h
                             of token t at q + t * q_token + h * q_head (elements) */
  int64_t q_token, q_head;
  void *q_out;            /* where they go, same form (q_out = q with equal strides: in place) */
  int64_t q_out_token, q_out_head;
} pskv_latent_prep_desc;

/* The prep and page write of a latent pool (kv_prep_append's place there).
 * For each new token t (n of them) it takes the down-projection's row
 *   x          device bf16, head_dim_v latent columns then PSKV_LATENT_ROT key columns at
 *              x + t * x_token (elements); 16-byte aligned, x_token a multiple of 8
 * and forms c' = c / sqrt(mean(c^2) + eps) * w and r', r turned by the angle of
 * position p = first_pos[row_of[t]] + pos_of[t] (first_pos NULL: 0): for each
 * pair (a, b), number i, with cos and sin = table row p, column i,
 *   a' = a cos - b sin,  b' = b cos + a sin.
 * [c', r'] goes into page slot pos_of[t] of table row row_of[t], and also to
 * dense + t * head_dim_k (bf16, 16-byte aligned) unless dense is NULL (the
 * up-projection's input and the rotated keys of prefill_attn_expanded).  The
 * queries' rotated columns are turned by the same angle.  q, q_out: 16-byte
 * aligned, strides multiples of 8.  Computed in f32, rounded once to nearest
 * even bf16.  A row that is refused (its page, lease or position) writes
 * nothing at all.  Checks, host copies and fault bits are those of
 * kv_prep_append; (row, pos) pairs must be distinct within one call.
 * Errors: INVALID_ARG, UNSUPPORTED (not a latent pool), PAST_PAGES, CUDA. */
int kv_prep_append_latent(const pskv_layout *layout, const pskv_latent_prep_desc *prep,
                          const void *x, int64_t x_token, int32_t n, const int32_t *row_of,
                          const int32_t *pos_of, const int32_t *first_pos,
                          const int32_t *page_tables, int32_t table_stride,
                          const int32_t *pages_of_row, int32_t batch, const int32_t *row_of_host,
                          const int32_t *pos_of_host, const int32_t *pages_of_row_host,
                          void *dense, pskv_stream_t stream);

/* Absorbed attention over a latent pool, num_tokens query tokens per row: the
 * row's last num_tokens keys, causal inside the window, as for
 * decode_attn_multirow (num_tokens = 1: single-token decode).  As there, except:
 *   q            device bf16 [batch][num_tokens][num_q_heads][head_dim_k]
 *   out          device [batch][num_tokens][num_q_heads][head_dim_v] of out_dtype
 *   num_q_heads  1..PSKV_LATENT_MAX_HEADS (any number)
 *   num_tokens   1..PSKV_MAX_WINDOW_TOKENS
 *   seq_lens     each at least num_tokens, or 0: a row of a padded batch, whose
 *                outputs are zeros (no fault bit); table_stride * page_size at most 2^31 - 129
 *   num_splits   0: chosen from the host lengths; else pieces of whole 128-key tiles,
 *                this many at most for the longest row (shorter rows have fewer)
 *   workspace    decode_attn_latent_workspace_bytes(...) bytes of these lengths, or
 *                decode_attn_latent_workspace_bound(...), 16-byte aligned
 *                (NULL is fine where that is 0); its contents are this call's own (the
 *                pieces are folded in one level: opts->merge_group is only checked)
 * Keys that a token does not attend take no part, whatever their scores; those of the
 * row's own later tokens have to hold finite values (they share its tiles), and
 * slots behind the row's last key may hold anything.
 * The softmax weights meet the values as bf16 when the output is bf16 (their
 * rounding adds to the output about what its own rounding does), as a bf16
 * pair when it is f32; scores, maxima, sums and outputs accumulate in f32.
 * The result is run-to-run deterministic for a fixed split count.
 * Errors: INVALID_ARG, UNSUPPORTED (not a latent pool, an appending option, more
 * than 2^31 - 1 pool rows), WORKSPACE_TOO_SMALL, CUDA. */
int decode_attn_latent(const pskv_layout *layout, const void *q, const int32_t *page_tables,
                       int32_t table_stride, const int32_t *seq_lens_host,
                       const int32_t *seq_lens, int32_t batch, int32_t num_tokens,
                       int32_t num_q_heads, float scale, int32_t num_splits, void *workspace,
                       size_t workspace_bytes, void *out, int32_t out_dtype,
                       const pskv_decode_opts *opts, pskv_stream_t stream);

/* The workspace a decode_attn_latent call needs under its plan (0 when one
 * partition writes the output directly).  It does not grow with the lengths: even rows that
 * fill the GPU are left whole and need none, one long row between short ones is cut.
 * Nothing is enqueued. */
int decode_attn_latent_workspace_bytes(const pskv_layout *layout, const int32_t *seq_lens_host,
                                       int32_t table_stride, int32_t batch, int32_t num_tokens,
                                       int32_t num_q_heads, int32_t num_splits, size_t *bytes);

/* A workspace that every decode_attn_latent call with this num_splits can use that has up to
 * max_batch rows, up to max_tokens tokens a row and no length above max_len (what a serving loop
 * sizes once). */
int decode_attn_latent_workspace_bound(const pskv_layout *layout, int32_t max_len,
                                       int32_t max_batch, int32_t max_tokens,
                                       int32_t num_q_heads, int32_t num_splits, size_t *bytes);

/* Tree attention over a drafted window of a latent pool: decode_attn_latent with the masks of
 * decode_attn_tree.  Token t of row b attends every key before the window (the row's last
 * num_tokens keys) and the window keys whose bits its mask holds.
 *   tree_mask   device uint64[batch][num_tokens], 8-byte aligned, as for decode_attn_tree: a valid mask
 *               holds bit t (the token itself) and no bit above t; one without bit t or
 *               with a later bit sets PSKV_FAULT_BAD_MASK (the later bits are ignored, the token
 *               attends what is left; with nothing left its output is zeros and
 *               PSKV_FAULT_EMPTY_ROW is set)
 * A chain (the mask of token t = bits 0..t) gives decode_attn_latent's bits.  All else, the workspace
 * with its sizes included, is decode_attn_latent's; every token's key in a row's own window
 * has to hold finite values.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE_TOO_SMALL, CUDA. */
int decode_attn_latent_tree(const pskv_layout *layout, const void *q, const int32_t *page_tables,
                            int32_t table_stride, const int32_t *seq_lens_host,
                            const int32_t *seq_lens, const uint64_t *tree_mask, int32_t batch,
                            int32_t num_tokens, int32_t num_q_heads, float scale,
                            int32_t num_splits, void *workspace, size_t workspace_bytes, void *out,
                            int32_t out_dtype, const pskv_decode_opts *opts, pskv_stream_t stream);

/* Expanded latent attention of variable-length chunks: row b's queries are
 * rows [cu_q[b], cu_q[b+1]) of q, its keys rows [cu_k[b], cu_k[b+1]) of kv and
 * k_rot; the queries are the row's last keys (as many keys as queries at
 * least), each attending keys up to its own.
 *   q       device bf16 [total_q][num_heads][PSKV_EXPANDED_NOPE + PSKV_LATENT_ROT]
 *   kv      device bf16 [total_k][num_heads][PSKV_EXPANDED_NOPE + PSKV_EXPANDED_V]: the
 *           up-projection's rows, a head's key columns then its value columns
 *   k_rot   device bf16, the rotated keys (all heads share them): token j's
 *           PSKV_LATENT_ROT columns at k_rot + j * k_rot_token (elements, a multiple of 8)
 *   cu_q_host, cu_k_host  host int32[batch + 1]: 0, then non-decreasing
 *   cu_q, cu_k            device int32[batch + 1]: the same, read by the kernel (rows
 *                         outside the host totals are never addressed)
 *   out     device [total_q][num_heads][PSKV_EXPANDED_V] of out_dtype
 * All 16-byte aligned.  The score of query i and key j is scale * (qn_i . kn_j
 * + qr_i . r_j).  The weights' precision is decode_attn_latent's, and so is what
 * keys that are not attended may hold.  Device offsets that are not such offsets
 * within the host totals raise PSKV_FAULT_BAD_LENGTH in status (device int32[4] or
 * NULL), and those rows are left out; so do rows that take more blocks of 256 queries
 * than the host's, and blocks past that count are left out.  No workspace.
 * Errors: INVALID_ARG (also a row with more queries than keys), CUDA. */
int prefill_attn_expanded(const void *q, const void *kv, const void *k_rot, int64_t k_rot_token,
                          const int32_t *cu_q_host, const int32_t *cu_q, const int32_t *cu_k_host,
                          const int32_t *cu_k, int32_t batch, int32_t num_heads, float scale,
                          void *out, int32_t out_dtype, int32_t *status, pskv_stream_t stream);

/* Verification of a drafted chain against the target's probabilities (what
 * follows the verify windows of decode_attn_multirow and decode_attn_latent:
 * speculative sampling, whose output has the target's distribution).  Row b has
 * drafts x_0 .. x_{d-1}, d = num_drafts[b].  With p_t the target's distribution
 * at draft t, q_t the draft's and u_t given uniform numbers, draft t stands
 * while every earlier one stood and u_t * q_t(x_t) < p_t(x_t).  With a drafts
 * standing, one more token comes from the weights
 *   r(v) = max(p_a(v) - q_a(v), 0)  when a < d,   r = p_a  when a = d
 * (when these are all 0: r = p_a): the lowest v with sum_{w <= v} r(w) >
 * u_D * sum r, D = max_drafts.  Products and comparisons are exact, and the sums
 * are of probabilities rounded to the nearest multiple of 2^-60, whole numbers,
 * so the result does not depend on their order.
 *   target_probs  device [batch][max_drafts + 1][vocab] of dtype (F32 or BF16)
 *   draft_probs   device [batch][max_drafts][vocab] of dtype, or NULL: the draft
 *                 has no distribution, q_t is 1 at x_t and 0 elsewhere
 *   drafts        device int32[batch][max_drafts]
 *   num_drafts    device int32[batch], 0..max_drafts each, or NULL (max_drafts)
 *   u             device float[batch][max_drafts + 1], in [0, 1)
 *   tokens        device int32[batch][max_drafts + 1]: the standing drafts, the drawn
 *                 token, then -1
 *   accepted      device int32[batch]: drafts standing
 *   status        device int32[4] fault word or NULL
 * max_drafts 0..PSKV_MAX_WINDOW_TOKENS (drafts may be NULL when 0).  Values
 * outside [0, 1] count as the nearer end, NaN as 0.  A draft outside the vocabulary does not stand
 * (PSKV_FAULT_BAD_TOKEN); a count outside its range is clamped
 * (PSKV_FAULT_BAD_LENGTH); a row without any weight draws -1
 * (PSKV_FAULT_EMPTY_ROW).  No workspace.  Errors: INVALID_ARG, CUDA. */
int verify_drafts(const void *target_probs, const void *draft_probs, int32_t dtype,
                  const int32_t *drafts, const int32_t *num_drafts, const float *u, int32_t batch,
                  int32_t max_drafts, int32_t vocab, int32_t *tokens, int32_t *accepted,
                  int32_t *status, pskv_stream_t stream);

/* Filters of sample_tokens: one value a request each, or NULL (off for all). */
typedef struct pskv_sample_desc {
  const float *temperature; /* device float[requests]: logits are divided by it; one that is not above
                               0 (0, NaN, or so small that its reciprocal is not finite) takes the
                               likeliest token.  NULL: 1 */
  const int32_t *top_k;     /* device int32[requests]: tokens kept; below 1 or from vocab on: all */
  const float *top_p;       /* device float[requests]: share of the weight kept; 1 and above, or NaN: all */
  const float *min_p;       /* device float[requests]: least weight, of the likeliest token's; 0 and below,
                               or NaN: all; above 1 counts as 1 */
} pskv_sample_desc;

/* Sampling from logits: a token from a given uniform number, the filtered distribution, or both
 * (what verify_drafts takes as target_probs or draft_probs).  For a row l of logits with M its
 * largest (NaN counts as -inf):
 *   x(v) = (l(v) - M) * (1 / temperature), each step rounded to f32 (0 where l(v) = M)
 *   w(v) = expf(x(v)), W(v) = w(v) rounded to the nearest multiple of 2^-40 (ties to the even one)
 * Tokens are ordered by x, the largest first, equal ones by index.  top_k keeps the first k of
 * them.  Of these, with S their sum of W, top_p keeps the ones whose predecessors sum to less than
 * floor(top_p * S) (in units of 2^-40), and always the first.  Of these, min_p keeps the ones with
 * w(v) >= min_p.  With S the sum of W over what is kept,
 *   token = the lowest kept v with sum_{w <= v} W(w) > floor(u * S),   probs(v) = W(v) / S, 0 elsewhere.
 * Products and sums are exact, so the token does not depend on how the work is split.
 *   logits        device, dtype (F32 or BF16): row r (of requests * tokens_per_request) begins at
 *                 logits + r * logits_row (elements, >= vocab); only the first vocab of a row are read
 *   filters       or NULL (no filter, temperature 1)
 *   u             device float[rows] in [0, 1) (values outside count as the nearer end, NaN as 0), or NULL:
 *                 no token is drawn
 *   tokens        device int32[rows], or NULL when u is
 *   probs         device [rows][vocab] of probs_dtype (F32 or BF16), or NULL
 *   status        device int32[4] fault word or NULL
 * A row without any finite or +inf logit gives token -1, zeros and PSKV_FAULT_EMPTY_ROW; several logits
 * of +inf share the weight.  (The search for a border is bounded, far above what any row is known to take; one that
 * would pass the bound gives token -1, zeros and PSKV_FAULT_BAD_STATE.)  vocab
 * 1..PSKV_MAX_VOCAB, requests and tokens_per_request 1 at least, their product PSKV_MAX_SAMPLED at most.  No workspace.  Errors: INVALID_ARG (also neither tokens
 * nor probs asked for, or these not apart from each other and from what is read), CUDA. */
int sample_tokens(const void *logits, int32_t dtype, int64_t logits_row, int32_t requests,
                  int32_t tokens_per_request, int32_t vocab, const pskv_sample_desc *filters,
                  const float *u, int32_t *tokens, void *probs, int32_t probs_dtype,
                  int32_t *status, pskv_stream_t stream);

/* The path of a drafted tree that stands, given the target's own token behind each window token
 * (sample_tokens on the window's logits; what follows decode_attn_tree and decode_attn_latent_tree).
 * The window's token 0 is no draft: it stands.  The parent of token t > 0 is the highest bit below t
 * of its mask (none: it never stands); t stands if its parent does, drafts[t] = sampled[parent] >= 0, and no
 * lower token with the same parent has the same draft.  So the tokens that stand are one path, and the
 * text goes on with what the target says along it.
 *   drafts     device int32[batch][num_tokens]: the window's tokens (drafts[0] is not looked at)
 *   tree_mask  device uint64[batch][num_tokens], 8-byte aligned, as for decode_attn_tree (same faults)
 *   sampled    device int32[batch][num_tokens]
 *   tokens     device int32[batch][num_tokens]: sampled[path[0]], sampled[path[1]], ..., then -1
 *   path       device int32[batch][num_tokens]: the standing tokens' places, going up, then -1
 *   kept       device int32[batch]: how many stand (1 at least)
 *   status     device int32[4] fault word or NULL
 * batch 1..PSKV_MAX_TREES, num_tokens 1..PSKV_MAX_WINDOW_TOKENS.  No workspace.  Errors: INVALID_ARG (also outputs that are not apart
 * from each other and from what is read), CUDA. */
int verify_tree(const int32_t *drafts, const uint64_t *tree_mask, const int32_t *sampled,
                int32_t batch, int32_t num_tokens, int32_t *tokens, int32_t *path, int32_t *kept,
                int32_t *status, pskv_stream_t stream);

/* Keep some of each row's last num_tokens keys (a drafted window's standing path) and drop the
 * others: key w0 + path[b][i] of row b becomes key w0 + i for i < kept[b], w0 = seq_lens[b] -
 * num_tokens, in the pools of all the layouts (layers that share the page tables), bit for bit, and the
 * row's new length is w0 + kept[b].
 *   layouts    host array of num_layouts (1..PSKV_MAX_LAYOUTS) layouts of one description but for
 *              their pools, which share no memory, and status words; any format.  Faults go to the
 *              first one's status word
 *   path       device int32[batch][num_tokens]: path[b][0 .. kept[b]) goes up, within [0, num_tokens);
 *              the rest is not looked at.  Else PSKV_FAULT_BAD_PATH
 *   kept       device int32[batch], 0..num_tokens each (else PSKV_FAULT_BAD_PATH)
 *   seq_lens   device int32[batch]: each at least num_tokens, or 0 (a padded batch's row: nothing is
 *              done, its new length is 0), table_stride * page_size at most; else PSKV_FAULT_BAD_LENGTH
 *   new_lens   device int32[batch]; not one of the arrays read
 * A row refused (these, or a page id outside the pool: PSKV_FAULT_BAD_PAGE) keeps its rows and its
 * length.  The window's pages must belong to the row alone (kv_fork_rows' last pages do).  batch
 * 1..PSKV_MAX_KEPT_ROWS, num_tokens 1..PSKV_MAX_WINDOW_TOKENS.  Errors: INVALID_ARG (also layouts that differ or share memory), UNSUPPORTED (pages of more
 * than 16 GB), CUDA. */
int kv_keep_tokens(const pskv_layout *const *layouts, int32_t num_layouts,
                   const int32_t *page_tables, int32_t table_stride, const int32_t *seq_lens,
                   const int32_t *path, const int32_t *kept, int32_t batch, int32_t num_tokens,
                   int32_t *new_lens, pskv_stream_t stream);

/* Rows that continue another row's keys: for each fork i, table row dst[i] becomes a copy of row src[i].
 * Whole pages are shared (their ids are copied); the page that the keys end in, when they end
 * inside one, is copied (its seq_lens % page_size first rows, all heads, all layouts) into page
 * new_pages[i], so that both rows go on in pages of their own.  Then seq_lens[dst] =
 * seq_lens[src] and pages_of_row[dst] = the pages that hold keys; table entries past these are left as they are.
 * Who holds which page, and when one is free again, is the caller's to count.
 *   layouts       as for kv_keep_tokens
 *   src, dst      device int32[n]: rows of the tables.  A dst that is out of range or that another fork of
 *                 the call has as its src or dst, or equals its own src, is refused
 *                 (PSKV_FAULT_BAD_ROW), and so is a src out of range
 *   new_pages     device int32[n]: pages no row holds, distinct; not looked at where the keys fill their pages
 *   page_tables   device int32[batch][table_stride], read and written; seq_lens, pages_of_row device
 *                 int32[batch], too; these three apart from each other and from src, dst and new_pages
 * A fork is also refused for a length outside [0, table_stride * page_size] (PSKV_FAULT_BAD_LENGTH), a lease
 * of fewer pages than its keys need or of more than table_stride (PSKV_FAULT_PAST_PAGES), or a page to copy from or to that is outside the
 * pool or the same (PSKV_FAULT_BAD_PAGE).  A refused fork writes nothing.  n 0..PSKV_MAX_FORKS (each is
 * compared with all others: 65,535 forks take 1.5 ms beside what they copy).
 * Errors: INVALID_ARG (also layouts that differ or share memory), UNSUPPORTED (pages of more than 16 GB), CUDA. */
int kv_fork_rows(const pskv_layout *const *layouts, int32_t num_layouts, const int32_t *src,
                 const int32_t *dst, const int32_t *new_pages, int32_t n, int32_t *page_tables,
                 int32_t table_stride, int32_t *seq_lens, int32_t *pages_of_row, int32_t batch,
                 pskv_stream_t stream);

/* Merge P partials per row in two levels by the exact rescaling identity and
 * normalise (gem design, "Candidate ownership and storage"; pegainfer #1055,
 * Description).  One launch: level 1 folds each group of merge_group partials
 * into a group state held in shared memory (never into the inputs), level 2
 * folds a row's group states; both in index order.
 *   m, l         device float[rows][num_splits]; m in units of the scaled score
 *   o            device float[rows][num_splits][head_dim_v], 16-byte aligned
 *   head_dim_v   a multiple of 4
 *   out          device [rows][head_dim_v] of out_dtype
 *   workspace    not used (the group states stay on chip): NULL and 0 are fine
 *   status       device int32[4] fault word or NULL
 * The empty state is (m = -inf, l = 0); its o is never used (it may be
 * uninitialised); merging an empty state changes nothing.  At most 64 groups
 * per row (num_splits <= 64 * merge_group). */
int merge_partials(const float *m, const float *l, const float *o, int32_t rows,
                   int32_t num_splits, int32_t head_dim_v, void *out, int32_t out_dtype,
                   void *workspace, size_t workspace_bytes, int32_t *status,
                   const pskv_decode_opts *opts, pskv_stream_t stream);

/* Scratch bytes a decode call needs for `num_splits` partitions (0 = enough
 * for any automatic plan).  Host-only.  Errors: INVALID_ARG, OVERFLOW. */
int decode_attn_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t head_dim_v,
                                int32_t num_splits, size_t *bytes);

/* Scratch bytes merge_partials needs: 0 in this build.  Host-only. */
int merge_partials_workspace_bytes(int32_t rows, int32_t num_splits, int32_t head_dim_v,
                                   size_t *bytes);

/* The partial buffer's byte contract (gem design, "Candidate ownership and
 * storage"): maxima batch*num_q_heads*P*4 bytes, denominators the same,
 * numerators batch*num_q_heads*P*head_dim_v*4; every product checked for
 * overflow.  Host-only.  Any output pointer may be NULL. */
int pskv_partial_scratch_bytes(int64_t batch, int64_t num_q_heads, int64_t head_dim_v,
                               int64_t num_splits, size_t *maxima, size_t *denominators,
                               size_t *numerators, size_t *total);

/* The split count the automatic plan picks for these lengths on the current
 * device (num_splits = 0 in a decode call).  It reads the device's SM count
 * and how many CTAs of the serving kernel fit on an SM; no kernel runs.  The
 * plan aims for one wave of CTAs: for one row, floor(slots / num_kv_heads)
 * partitions (slots = SMs x CTAs per SM); for a batch, enough partitions that
 * the longest row's pieces carry about half a slot's fair share of all
 * tiles.  It depends on the lengths only, never on a window bound. */
int pskv_plan_splits(const pskv_layout *layout, int32_t batch, int32_t num_q_heads,
                     const int32_t *seq_lens_host, int32_t *num_splits);

/* The workspace a prefill_attn_paged call needs under its plan.  A sizing
 * helper: the pages give the workspace only as the partial buffer's byte
 * contract (gem design, "Candidate ownership and storage"), which this
 * applies to the plan's split count.  The same
 * arguments' host-visible parts (cu_q_host, seq_lens_host, table_stride,
 * batch, num_q_heads, window, num_splits, 0 = automatic) are checked and
 * planned exactly as the call does, and *bytes receives the bytes its
 * partials take, or 0 when the plan has one partition (each CTA writes its
 * output directly and no workspace is read).  Nothing is enqueued.  The
 * answer depends on the device (its SM count) for automatic plans.
 * Errors: as prefill_attn_paged's host-side checks. */
int prefill_attn_workspace_bytes(const pskv_layout *layout, const int32_t *cu_q_host,
                                 const int32_t *seq_lens_host, int32_t table_stride,
                                 int32_t batch, int32_t num_q_heads, int32_t window,
                                 int32_t num_splits, size_t *bytes);

/* The workspace a decode_attn_multirow (tree = 0) or decode_attn_tree
 * (tree = 1) call needs under its plan, with the same meaning as
 * prefill_attn_workspace_bytes (the same sizing helper, no passage of its
 * own); the two calls can route a window to different kernels, so the flag
 * selects whose plan. */
int decode_attn_multirow_workspace_bytes(const pskv_layout *layout, const int32_t *seq_lens_host,
                                         int32_t table_stride, int32_t batch, int32_t num_tokens,
                                         int32_t num_q_heads, int32_t tree, int32_t num_splits,
                                         size_t *bytes);

/* Bytes of the scratch array that decode_attn_splitkv_static uses (16 MiB). */
#define PSKV_STATIC_SCRATCH_BYTES (16 * 1024 * 1024)

/* decode_attn_splitkv for callers that cannot allocate device memory.
 * No passage of the source pages corresponds to this entry point: it exists
 * for callers that have no way to obtain a workspace (code that must not call
 * cudaMalloc, such as a host callback, a real-time or signal-safe path, or a
 * plugin whose host framework owns every device allocation).
 * It takes the arguments of decode_attn_splitkv except the workspace and the
 * options, and uses instead a scratch array of PSKV_STATIC_SCRATCH_BYTES
 * compiled into the library (held on every GPU that loads the library until
 * the process exits).  It allocates nothing and frees nothing.
 *   - num_splits = 0 picks the automatic plan, lowered to the largest split
 *     count whose workspace (decode_attn_workspace_bytes) fits the array;
 *     an explicit count whose workspace does not fit is refused with
 *     PSKV_ERR_WORKSPACE_TOO_SMALL before anything is enqueued.
 *   - The first call on a device looks up the array's device address (with
 *     that device current) and keeps it; make that first call before any
 *     stream capture on the device.  The kept address is not looked up
 *     again: calling this entry point after cudaDeviceReset on that device
 *     is not supported.
 *   - All calls share the array.  Calls that may run at the same time on the
 *     GPU (other streams or host threads without ordering) overwrite each
 *     other's partials: order them.  Nothing in the array needs clearing;
 *     every call writes what it reads. */
int decode_attn_splitkv_static(const pskv_layout *layout, const void *q,
                               const int32_t *page_tables, int32_t table_stride,
                               const int32_t *seq_lens_host, const int32_t *seq_lens,
                               int32_t batch, int32_t num_q_heads, float scale,
                               int32_t num_splits, void *out, int32_t out_dtype,
                               pskv_stream_t stream);

/* Read the layout's fault word: copies status[0] to *flags after all work
 * already enqueued on `stream`, and optionally clears it for the next calls.
 * This call synchronizes the stream (the only one that does).  A layout made
 * without a status word reads as 0.  Errors: INVALID_ARG, CUDA. */
int pskv_check_flags(const pskv_layout *layout, int32_t clear, pskv_stream_t stream,
                     uint32_t *flags);

/* Static text for a status code. */
const char *pskv_strerror(int status);

/* Text of the last CUDA error seen by this thread (empty if none). */
const char *pskv_last_cuda_error(void);

/* Number of kernels this library has launched in this process. */
uint64_t pskv_kernel_launches(void);

/* Library version: major * 10000 + minor * 100 + patch. */
int pskv_version(void);

#ifdef __cplusplus
}
#endif
#endif /* PSKV_H */
