// cache_rows.cu -- rows of a paged cache moved together (kv_keep_tokens) and
// continued by others (kv_fork_rows), in the pools of all layers by one launch.
//
// Both move 16-byte vectors as they are: a stored row of one head is k_vecs vectors in the K region
// and v_vecs in the V region, and a token's row of one layer heads * (k_vecs + v_vecs) of them
// (8 KB at head dim 512 with four KV heads, 1,152 bytes of a latent row).
//
// Measured, calls one after the other: kv_keep_tokens of 32 windows of 16 tokens over four layers (head dim 512, four
// KV heads) 3.1 us for 6.6 MB; of one latent window of 8 2.1 us.  kv_fork_rows of 64 forks of 16 rows over four layers (571 MB)
// 86 us, 6.6 TB/s or 97 % of a plain copy's rate; one latent row's three forks 2.9 us.
#include "pskv_internal.cuh"
#include "tree.h"

namespace pskv {

namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 8;  // loads of a thread in flight

// Vector u of a token's row: the address of its place in a page-row `at` = page * heads * page_size + row.
struct Column {
  uint4 *base;
  int vecs;
  __device__ Column(const Pools &p, int layer, int u) {
    const int k_all = p.heads * p.k_vecs;
    const bool is_k = u < k_all;
    vecs = is_k ? p.k_vecs : p.v_vecs;
    const int e = is_k ? u : u - k_all, head = e / vecs;
    base = static_cast<uint4 *>(is_k ? p.k[layer] : p.v[layer]) + (size_t)head * p.page_size * vecs + (e - head * vecs);
  }
  __device__ uint4 *at(long long row) const { return base + row * vecs; }
};

// Pieces of a page's rows of one head.
__host__ __device__ int pieces(int vecs, int page_size) {
  return (vecs * page_size + kThreads * kAhead - 1) / (kThreads * kAhead);
}

}  // namespace

// Grid (blocks of vectors, rows, layers).  Every block checks its row alike, so that a row is
// refused as a whole; the first one reports it and writes the new length.  The call is three dependent loads (length
// and path, page ids, rows) behind its launch.
// A thread takes one vector of every token, eight of them in flight: the places go up and path[i] >= i, so
// what a step writes lies below everything that later ones read.
__global__ void __launch_bounds__(kThreads) pskv_keep_tokens(const KeepArgs a, const __grid_constant__ Pools p) {
  __shared__ long long from[PSKV_MAX_WINDOW_TOKENS], to[PSKV_MAX_WINDOW_TOKENS];
  const int b = blockIdx.y, i = threadIdx.x, T = a.num_tokens;
  const bool first = blockIdx.x == 0 && blockIdx.z == 0;
  pdl_wait();
  pdl_launch_dependents();
  const int len = a.seq_lens[b], kept = a.kept[b], w0 = len - T;
  if (len == 0) {
    if (first && i == 0) a.new_lens[b] = 0;
    return;
  }
  uint32_t fault = 0;
  if (len < T || (long long)len > (long long)a.table_stride * p.page_size) fault = PSKV_FAULT_BAD_LENGTH;
  if (kept < 0 || kept > T) fault |= PSKV_FAULT_BAD_PATH;
  if (!fault && i < kept) {
    const int at = a.path[(size_t)b * T + i], before = i > 0 ? a.path[(size_t)b * T + i - 1] : -1;
    if (at <= before || at >= T || at < i) {
      fault = PSKV_FAULT_BAD_PATH;
    } else {
      const int32_t *table = a.page_tables + (size_t)b * a.table_stride;
      const int s = (w0 + at) / p.page_size, d = (w0 + i) / p.page_size;
      const int sp = table[s], dp = table[d];
      if (sp < 0 || sp >= p.num_pages || dp < 0 || dp >= p.num_pages) fault = PSKV_FAULT_BAD_PAGE;
      from[i] = (long long)sp * p.heads * p.page_size + (w0 + at - s * p.page_size);
      to[i] = (long long)dp * p.heads * p.page_size + (w0 + i - d * p.page_size);
    }
  }
  if (__syncthreads_or(fault != 0)) {
    if (first && fault) raise_fault(p.status, fault);
    if (first && i == 0) a.new_lens[b] = len;
    return;
  }
  if (first && i == 0) a.new_lens[b] = w0 + kept;
  const int u = blockIdx.x * kThreads + i;
  if (u >= p.heads * (p.k_vecs + p.v_vecs)) return;
  const Column col(p, blockIdx.z, u);
  for (int t0 = 0; t0 < kept; t0 += kAhead) {
    uint4 x[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (t0 + k < kept && from[t0 + k] != to[t0 + k]) x[k] = *col.at(from[t0 + k]);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (t0 + k < kept && from[t0 + k] != to[t0 + k]) *col.at(to[t0 + k]) = x[k];
  }
}

// Grid (pieces of a page, forks, layers): a piece is kThreads * kAhead vectors of one region's head, whose rows lie
// one after another (a block of one column of every row, as above, wrote short runs: 111 instead of 86 us).  As above, every block checks its fork alike; the first one reports, and writes the row's table,
// length and lease.  Sources are rows that no fork of the call writes.
__global__ void __launch_bounds__(kThreads) pskv_fork_rows(const ForkArgs a, const __grid_constant__ Pools p) {
  const int f = blockIdx.y, i = threadIdx.x;
  const bool first = blockIdx.x == 0 && blockIdx.z == 0;
  pdl_wait();
  pdl_launch_dependents();
  const int src = a.src[f], dst = a.dst[f];
  uint32_t fault = 0;
  if (src < 0 || src >= a.batch || dst < 0 || dst >= a.batch || src == dst) fault = PSKV_FAULT_BAD_ROW;
  for (int k = i; k < a.n; k += kThreads)
    if (k != f && (a.dst[k] == dst || a.src[k] == dst)) fault = PSKV_FAULT_BAD_ROW;
  if (__syncthreads_or(fault != 0)) {
    if (first && fault) raise_fault(p.status, fault);
    return;
  }
  const int len = a.seq_lens[src], lease = a.pages_of_row[src];
  if (len < 0 || (long long)len > (long long)a.table_stride * p.page_size) {
    if (first && i == 0) raise_fault(p.status, PSKV_FAULT_BAD_LENGTH);
    return;
  }
  const int whole = len / p.page_size, rest = len - whole * p.page_size, pages = whole + (rest > 0);
  if (lease < pages || lease > a.table_stride) {
    if (first && i == 0) raise_fault(p.status, PSKV_FAULT_PAST_PAGES);
    return;
  }
  const int32_t *from = a.page_tables + (size_t)src * a.table_stride;
  int old_page = 0, new_page = 0;
  if (rest > 0) {
    old_page = from[whole];
    new_page = a.new_pages[f];
    if (old_page < 0 || old_page >= p.num_pages || new_page < 0 || new_page >= p.num_pages || old_page == new_page) {
      if (first && i == 0) raise_fault(p.status, PSKV_FAULT_BAD_PAGE);
      return;
    }
  }
  if (first) {
    int32_t *table = a.page_tables + (size_t)dst * a.table_stride;
    for (int s = i; s < whole; s += kThreads) table[s] = from[s];
    if (i == 0) {
      if (rest > 0) table[whole] = new_page;
      a.seq_lens[dst] = len;
      a.pages_of_row[dst] = pages;
    }
  }
  // this block's piece: of a K head, or behind these of a V head
  const int k_pieces = pieces(p.k_vecs, p.page_size), v_pieces = pieces(p.v_vecs, p.page_size);
  const bool is_k = (int)blockIdx.x < p.heads * k_pieces;
  const int x = is_k ? blockIdx.x : blockIdx.x - p.heads * k_pieces, each = is_k ? k_pieces : v_pieces;
  const int head = x / each, vecs = is_k ? p.k_vecs : p.v_vecs, run = rest * vecs;
  const int u0 = (x - head * each) * kThreads * kAhead + i;
  uint4 *pool = static_cast<uint4 *>(is_k ? p.k[blockIdx.z] : p.v[blockIdx.z]);
  const uint4 *old_run = pool + ((size_t)old_page * p.heads + head) * p.page_size * vecs;
  uint4 *new_run = pool + ((size_t)new_page * p.heads + head) * p.page_size * vecs;
  uint4 q[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (u0 + k * kThreads < run) q[k] = old_run[u0 + k * kThreads];
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (u0 + k * kThreads < run) new_run[u0 + k * kThreads] = q[k];
}

cudaError_t launch_keep(const KeepArgs &a, const Pools &p, cudaStream_t s) {
  const int vecs = p.heads * (p.k_vecs + p.v_vecs);
  const dim3 grid((unsigned)((vecs + kThreads - 1) / kThreads), (unsigned)a.batch, (unsigned)p.count);
  return launch_pdl(pskv_keep_tokens, grid, dim3(kThreads), 0, s, a, p);
}

cudaError_t launch_fork(const ForkArgs &a, const Pools &p, cudaStream_t s) {
  const dim3 grid((unsigned)(p.heads * (pieces(p.k_vecs, p.page_size) + pieces(p.v_vecs, p.page_size))),
                  (unsigned)a.n, (unsigned)p.count);
  return launch_pdl(pskv_fork_rows, grid, dim3(kThreads), 0, s, a, p);
}

}  // namespace pskv
