// cache_rows.cu -- rows of a paged cache moved together (kv_keep_tokens) and
// continued by others (kv_fork_rows), in the pools of all layers by one launch.
//
// Both move 16-byte vectors as they are: a stored row of one head is k_vecs vectors in the K region
// and v_vecs in the V region, and a token's row of one layer heads * (k_vecs + v_vecs) of them
// (8 KB at head dim 512 with four KV heads, 1,152 bytes of a latent row).
//
// Measured, calls one after the other: kv_keep_tokens of 32 windows of 16 tokens over four layers (head dim 512, four
// KV heads) 3.1 us for 6.6 MB; of one latent window of 8 2.1 us.  kv_fork_rows of 64 forks of 16 rows over four layers (571 MB)
// 86 us, 6.6 TB/s or 97 % of a plain copy's rate; one latent row's three forks 2.9 us; 65,535 forks 1.5 ms beside their copies.
#include "pskv_internal.cuh"
#include "pskv_plan.h"
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

// ---- forks

namespace {

// One fork: from where its row goes on, and the page its last keys are copied from and to.
struct Fork {
  int src, dst, len, whole, rest, old_page, new_page;

  // Its rows exist.  (Not yet: that no other fork of the call has dst.)
  __device__ bool names_rows(const ForkArgs &a, int f) {
    src = a.src[f];
    dst = a.dst[f];
    return src >= 0 && src < a.batch && dst >= 0 && dst < a.batch && src != dst;
  }
  // What it is refused for beside its rows, or 0.
  __device__ uint32_t look(const ForkArgs &a, const Pools &p, int f) {
    len = a.seq_lens[src];
    const int lease = a.pages_of_row[src];
    if (len < 0 || (long long)len > (long long)a.table_stride * p.page_size) return PSKV_FAULT_BAD_LENGTH;
    whole = len / p.page_size;
    rest = len - whole * p.page_size;
    if (lease < whole + (rest > 0) || lease > a.table_stride) return PSKV_FAULT_PAST_PAGES;
    old_page = new_page = 0;
    if (rest == 0) return 0;
    old_page = a.page_tables[(size_t)src * a.table_stride + whole];
    new_page = a.new_pages[f];
    return old_page < 0 || old_page >= p.num_pages || new_page < 0 || new_page >= p.num_pages || old_page == new_page
               ? PSKV_FAULT_BAD_PAGE
               : 0;
  }
  // The row's table, length and lease, by a block.
  __device__ void write_row(const ForkArgs &a, int i) const {
    const int32_t *from = a.page_tables + (size_t)src * a.table_stride;
    int32_t *table = a.page_tables + (size_t)dst * a.table_stride;
    for (int s = i; s < whole; s += kThreads) table[s] = from[s];
    if (i == 0) {
      if (rest > 0) table[whole] = new_page;
      a.seq_lens[dst] = len;
      a.pages_of_row[dst] = whole + (rest > 0);
    }
  }
  // Piece x of a layer's page, K heads before V heads: kThreads * kAhead vectors of one head's rows, which lie one after
  // another (a block of one column of every row, as above, wrote short runs: 111 instead of 86 us).
  __device__ void copy(const Pools &p, int layer, int x, int i) const {
    const int k_pieces = pieces(p.k_vecs, p.page_size), v_pieces = pieces(p.v_vecs, p.page_size);
    const bool is_k = x < p.heads * k_pieces;
    const int y = is_k ? x : x - p.heads * k_pieces, each = is_k ? k_pieces : v_pieces;
    const int head = y / each, vecs = is_k ? p.k_vecs : p.v_vecs, run = rest * vecs;
    const int u0 = (y - head * each) * kThreads * kAhead + i;
    uint4 *pool = static_cast<uint4 *>(is_k ? p.k[layer] : p.v[layer]);
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
};

}  // namespace

// Grid (pieces of a layer's page, forks, layers).  As above, every block checks its fork alike; the first one
// reports, and writes the row's table, length and lease.  Sources are rows that no fork of the call writes.
__global__ void __launch_bounds__(kThreads) pskv_fork_rows(const ForkArgs a, const __grid_constant__ Pools p) {
  const int f = blockIdx.y, i = threadIdx.x;
  const bool first = blockIdx.x == 0 && blockIdx.z == 0;
  pdl_wait();
  pdl_launch_dependents();
  Fork fork;
  uint32_t fault = fork.names_rows(a, f) ? 0 : PSKV_FAULT_BAD_ROW;
  for (int k = i; k < a.n; k += kThreads)
    if (k != f && (a.dst[k] == fork.dst || a.src[k] == fork.dst)) fault = PSKV_FAULT_BAD_ROW;
  if (__syncthreads_or(fault != 0)) {
    if (first && fault) raise_fault(p.status, fault);
    return;
  }
  fault = fork.look(a, p, f);
  if (fault) {
    if (first && i == 0) raise_fault(p.status, fault);
    return;
  }
  if (first) fork.write_row(a, i);
  fork.copy(p, blockIdx.z, blockIdx.x, i);
}

// The same for many forks.  Each is compared with all others, so that a block for each piece reads the call's n forks n *
// pieces times: 59.7 ms for 65,535 forks of 16-row pages in eight layers, 7.6 in one.  Here a block takes more pieces (of any
// layer) as n goes up, then several forks with all of theirs, which it compares at once: 1.6 and 1.5.
// Grid (blocks of a fork's pieces, groups of forks).
__global__ void __launch_bounds__(kThreads) pskv_fork_many(const ForkArgs a, const __grid_constant__ Pools p, int all_pieces,
                                                           const ForkBlocks of) {
  __shared__ uint32_t found[kThreads / 32];
  const int f0 = blockIdx.y * of.forks, i = threadIdx.x;
  const int x0 = blockIdx.x * of.pieces, x1 = min(x0 + of.pieces, all_pieces), of_layer = all_pieces / p.count;
  const bool first = blockIdx.x == 0;
  pdl_wait();
  pdl_launch_dependents();
  if (!first) {  // (of one fork) nothing to copy, nothing to compare
    Fork fork;
    if (!fork.names_rows(a, f0) || fork.look(a, p, f0) || fork.rest == 0) return;
  }
  int rows[kForksTogether];
#pragma unroll
  for (int g = 0; g < kForksTogether; ++g) rows[g] = g < of.forks && f0 + g < a.n ? a.dst[f0 + g] : -1;
  uint32_t taken = 0;  // bit g: another fork has the row of fork f0 + g (or that fork reads it itself)
#pragma unroll 2
  for (int k = i; k < a.n; k += kThreads) {
    const int s = a.src[k], d = a.dst[k];
#pragma unroll
    for (int g = 0; g < kForksTogether; ++g) taken |= (uint32_t)(s == rows[g] || (d == rows[g] && k != f0 + g)) << g;
  }
  taken = __reduce_or_sync(0xffffffffu, taken);
  if ((i & 31) == 0) found[i >> 5] = taken;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) taken |= found[w];
#pragma unroll 1
  for (int g = 0; g < of.forks && f0 + g < a.n; ++g) {
    Fork fork;
    uint32_t fault = fork.names_rows(a, f0 + g) && !((taken >> g) & 1u) ? 0 : PSKV_FAULT_BAD_ROW;
    if (!fault) fault = fork.look(a, p, f0 + g);
    if (fault) {
      if (first && i == 0) raise_fault(p.status, fault);
      continue;
    }
    if (first) fork.write_row(a, i);
    int layer = x0 / of_layer, x = x0 - layer * of_layer;
#pragma unroll 1
    for (int k = fork.rest > 0 ? x0 : x1; k < x1; ++k) {
      fork.copy(p, layer, x, i);
      if (++x == of_layer) x = 0, ++layer;
    }
  }
}

cudaError_t launch_keep(const KeepArgs &a, const Pools &p, cudaStream_t s) {
  const int vecs = p.heads * (p.k_vecs + p.v_vecs);
  const dim3 grid((unsigned)((vecs + kThreads - 1) / kThreads), (unsigned)a.batch, (unsigned)p.count);
  return launch_pdl(pskv_keep_tokens, grid, dim3(kThreads), 0, s, a, p);
}

cudaError_t launch_fork(const ForkArgs &a, const Pools &p, cudaStream_t s) {
  const int of_layer = p.heads * (pieces(p.k_vecs, p.page_size) + pieces(p.v_vecs, p.page_size)), all = p.count * of_layer;
  if (a.n <= kFewForks)
    return launch_pdl(pskv_fork_rows, dim3((unsigned)of_layer, (unsigned)a.n, (unsigned)p.count), dim3(kThreads), 0, s, a, p);
  const ForkBlocks b = fork_blocks(a.n, all);
  const dim3 grid((unsigned)((all + b.pieces - 1) / b.pieces), (unsigned)((a.n + b.forks - 1) / b.forks));
  return launch_pdl(pskv_fork_many, grid, dim3(kThreads), 0, s, a, p, all, b);
}

}  // namespace pskv
