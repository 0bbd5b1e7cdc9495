// attn_latent.cu -- absorbed attention over a paged latent pool on a pair of CTAs.
//
// For every query column (token t, head h) of a row: s_i = scale * q . row_i over
// the dc + 64 columns of a cached row, o = sum_i softmax(s)_i row_i[0:dc].  All
// heads share the rows, so a block of 128 query columns meets each cached row once:
// per key 2 * 128 * (2 dc + 64) operations against 2 (dc + 64) bytes.
//
// A cluster of two CTAs takes 128 columns of one row and a piece of its keys, as one
// tcgen05 product of M = 128 over the pair (cta_group::2): CTA r holds columns
// 64 r .. + 63 of Q (dc + 64 wide) in shared memory, and of O (64 x dc in f32: 256
// tensor-memory columns, half of the lanes holding half of the columns each),
// which one CTA alone could not hold beside the scores (128 x 512 f32 fill its tensor
// memory).  Per tile j of 128 keys:
//   S = Q K^T     N = 128 keys, CTA r brings the tile's keys 64 r .. + 63
//   softmax       a row's 128 scores lie in four threads (halves by lane, halves of these by
//                 warp group), which mask them and exchange their maxima; the reference
//                 maximum moves only past a slack of 8 (log2 units), so O is rarely
//                 rescaled; P goes to shared memory as bf16 (f32 output: a hi + lo pair)
//   O += P V      per half of the keys and 256 columns: CTA r brings columns
//                 128 r .. + 127 of them, 64 keys
// A product of M = 128 over a pair runs at the full rate of both SMs from N = 128 on
// (measured: 32 cycles per K = 16 step at N = 128 and 64 at N = 256; 25 instead of 16
// at N = 64, where reading the operands binds; M = 64 on one CTA runs at half rate).
// The two products want a row in different CTAs (scores: by key, values: by column),
// so a CTA copies both shares: 1.9x of a row's bytes from L2, each byte once from
// HBM (a prefetch into L2 some tiles ahead only slowed the copies down, warm or cold).  K
// moves in chunks of a few 64-column slabs and V in chunks of 64 keys, through rings of their
// own with their own copy warps and issuing warps, so a chunk's place is refilled as soon as
// its products are done, and S(j + 1) runs while the softmax works on tile j.  Measured at dc = 512:
// a tile costs a pair 1.42 us until 56 pairs run (the rings' turnaround), 1.97 us with all
// 76, which is 5.7 TB/s of cached rows; a call costs 7.5 to 10 us beside its tiles (one
// row of 40,002 keys, 32 heads: 63 pieces of five tiles and the merge, 19.8 us).
//
// A row's keys are cut into pieces of `tiles_per_piece` tiles, one piece per cluster
// (pskv_plan.cpp picks the size that fills the clusters in one wave).  A row of one
// piece is written at once; longer ones leave f32 partials (m, l, O) in groups of 32 query
// columns, [group][piece][column / 4][32] float4, which a warp writes from its registers
// and pskv_merge_latent reads back in whole 512-byte lines (through shared memory and
// row-wise bulk copies the same bytes took 3 us more).
//
// A drafted tree (kTree) differs in what a column sees of the window's keys: its limit is the window's first key, and
// the token's mask, shifted to a thread's 32 keys, says which of the later ones.  Only tiles in which a key is not
// seen take the branch that masks, the same ones that a causal window takes: a chain gives the same bits, and the
// time is the window's (1 x 8 tokens x 40,002 keys, 32 heads: 30 us; 4 rows x 16 tokens of up to 10,602: 44 us).
//
// P is rounded to bf16 when the output is (the weights' rounding then adds about
// what the output's own does; the sum takes the rounded weights, so a lone key gives
// its row exactly); maxima, sums, O and partials are f32.
// Every wait is bounded; on expiry the CTA flags PSKV_FAULT_WAIT_TIMEOUT, lets
// what it issued finish and frees its tensor memory.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math_constants.h>

#include <atomic>

#include "latent.h"
#include "pskv_internal.cuh"
#include "pskv_plan.h"
#include "tc_common.cuh"
#include "tc_ops.cuh"
#include "tc_pair.cuh"

namespace pskv {

namespace {

using tc::elect_one;
using tc::ex2;
using tc::PageCache;

constexpr int kKeys = kLatentTile;  // keys per tile (128)
constexpr int kHalf = kKeys / 2;   // of which each CTA brings half to the scores
constexpr int kRows = 64;          // query columns per CTA (128 per pair)
// warps: 0 score products, 1 value products, 2 Q's copies, 3, 12 and 13 K copies,
// 14 and 15 V copies, 4-11 softmax (two groups of four; warp w reads tensor-memory lanes 32 (w % 4) ..)
constexpr int kThreads = 512;
constexpr int kSoftWarps = 8;
constexpr int kTmemCols = 512;
constexpr int kOCol = 0;           // O: DC / 2 columns
constexpr int kSCol = 256;         // score region r at kSCol + 64 r
constexpr float kSlack = 8.f;
constexpr int kInfo = 8;           // tile records in flight: K runs at most 2 tiles ahead of S, S 2 ahead of the softmax
constexpr int kSlab = kHalf * 128;  // 64 rows (of Q, K, V or P) of 64 columns: 8 KB

template <int DC, bool kLo>
struct Lay {
  static constexpr int kSlabs = DC / 64 + 1;             // 64-column slabs of a row
  static constexpr int kChunkSlabs = DC == 512 ? 3 : 5;  // of them in a K chunk
  static constexpr int kChunks = kSlabs / kChunkSlabs;   // K chunks per tile
  static constexpr int kBlocks = DC / 256;               // 256-column blocks of O
  static constexpr int kQBytes = kSlabs * kSlab;
  static constexpr int kKBytes = kChunkSlabs * kSlab;
  static constexpr int kVBytes = 2 * kBlocks * kSlab;    // 64 keys of this CTA's columns
  static constexpr int kRingK = DC == 512 && !kLo ? 3 : 2;
  static constexpr int kRingV = DC == 512 ? 2 : 4;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kQBytes;
  static constexpr int kOffV = kOffK + kRingK * kKBytes;
  static constexpr int kOffP = kOffV + kRingV * kVBytes;  // P: half h at h * kSlab; the lo part behind
  static constexpr int kOffBar = kOffP + (kLo ? 4 : 2) * kSlab;
  // O on its way out: rows padded by 16 bytes against bank conflicts, over the rings and P
  static constexpr int kStagePitch = DC * 4 + 16;
  static_assert(kOffK + kRows * kStagePitch <= kOffBar, "staging");
  // barrier slots
  static constexpr int kFullK = 0;                       // (even CTA) both CTAs' K landed
  static constexpr int kFullV = kFullK + kRingK;         // (even CTA) both CTAs' V landed
  static constexpr int kEmptyK = kFullV + kRingV;        // the scores of the chunk done
  static constexpr int kEmptyV = kEmptyK + kRingK;       // the values of the chunk done
  static constexpr int kSFull = kEmptyV + kRingV;        // [2] S of region r done
  static constexpr int kSFree = kSFull + 2;              // [2] (even CTA) region r read in both CTAs
  static constexpr int kPFull = kSFree + 2;              // (even CTA) P written in both CTAs
  static constexpr int kPvDone = kPFull + 1;             // [2] the values of half h of a tile done
  static constexpr int kInfoFull = kPvDone + 2;          // [8] a tile's record written
  static constexpr int kQFull = kInfoFull + kInfo;       // (even CTA) both CTAs' Q landed
  static constexpr int kQFree = kQFull + 1;              // the piece's score products done
  static constexpr int kOut = kQFree + 1;                // this CTA's O has left the rings
  static constexpr int kRagged = kOut + 1;               // [2] this CTA's V of a chunk that is not whole
  static constexpr int kDrainS = kRagged + 2;            // every product done
  static constexpr int kDrainV = kDrainS + 1;
  static constexpr int kNumBars = kDrainV + 1;
  static constexpr int kOffInfo = (kOffBar + kNumBars * 8 + 15) & ~15;
  static constexpr int kOffRed = kOffInfo + kInfo * 8;   // float[2][4][64] maxima (then sums)
  static constexpr int kOffSlot = kOffRed + 2 * 4 * kRows * 4;
  static constexpr int kOffAbort = kOffSlot + 4;
  static constexpr int kUsed = kOffAbort + 4;
  // + alignment of the dynamic base, as far as a CTA's limit leaves room (the base is in fact
  // aligned; the kernel checks)
  static constexpr int kSmemBytes = kUsed + 1024 < 232448 ? kUsed + 1024 : 232448;
  static_assert(kUsed <= 232448, "shared memory per CTA");
  static_assert(kSlabs % kChunkSlabs == 0, "whole chunks");
  static constexpr uint32_t kIdescS = tc::instr_desc(2 * kRows, kKeys, false, false);
  static constexpr uint32_t kIdescPV = tc::instr_desc(2 * kRows, 256, false, true);
};

// Bit c of `bad` marks a 16-key group of the tile whose page id lies outside the pool (not loaded).
struct TileInfo {
  uint32_t bad, pad;
};

// One piece of the work, the same in every thread of both CTAs.
struct Piece {
  int b, cb, p, count;  // row, block of 128 columns, piece of the row's `count`
  int len;              // the row's keys
  int t0, n;            // tiles [t0, t0 + n)
};

__device__ __forceinline__ int tiles_of(int len) { return (len + kKeys - 1) / kKeys; }

// Lengths as the kernels use them: clamped into the table, `bad` where that changes one or a row
// is shorter than its window.
__device__ __forceinline__ int usable_len(const LatentAttnArgs &a, int b, bool *bad) {
  const long long cap = (long long)a.table_stride * a.page_size, len = a.seq_lens[b];
  *bad = len < 0 || len > cap || (len > 0 && len < a.num_tokens);
  return (int)(len < 0 ? 0 : (len > cap ? cap : len));
}

// The rows' lengths as this lane holds them (up to 32 rows; longer batches are read again).
struct Rows {
  int len;  // of row `lane`, 0 past the batch
  int q;    // tiles per piece
};

// Tiles per piece: the plan's, or more if a device length outgrew the planned ones (at
// most num_splits pieces a row).  Every warp computes it alike.
__device__ __forceinline__ Rows read_rows(const LatentAttnArgs &a, int lane, bool report) {
  int most = 0;
  bool any_bad = false;
  Rows r;
  r.len = 0;
  for (int b = lane; b < a.batch; b += 32) {
    bool bad;
    const int len = usable_len(a, b, &bad);
    if (b < 32) r.len = len;
    most = max(most, tiles_of(len));
    any_bad |= bad;
  }
  if (report && any_bad) raise_fault(a.status, PSKV_FAULT_BAD_LENGTH);
  most = __reduce_max_sync(0xffffffffu, most);
  r.q = a.tiles_per_piece;
  if ((long long)r.q * a.num_splits < most) r.q = (most + a.num_splits - 1) / a.num_splits;
  return r;
}

// Piece u in the order (row, piece, block of columns), the last fastest; false past the end.
__device__ __forceinline__ bool find_piece(const LatentAttnArgs &a, int u, const Rows &r, int lane,
                                           Piece &pc) {
  const int blocks = (a.num_tokens * a.num_q_heads + 127) / 128;
  const int unit = blocks == 1 ? u : u / blocks;
  if (a.batch == 1) {
    pc.b = 0;
    pc.cb = u - unit * blocks;
    pc.len = tc2::uniform(r.len);
    const int tiles = tiles_of(pc.len);
    pc.count = max(1, (tiles + r.q - 1) / r.q);
    pc.p = unit;
    pc.t0 = min(unit * r.q, tiles);
    pc.n = min(pc.t0 + r.q, tiles) - pc.t0;
    return unit < pc.count;
  }
  int base = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    bool bad;
    const int len = b0 == 0 ? r.len : (b0 + lane < a.batch ? usable_len(a, b0 + lane, &bad) : 0);
    const int n = b0 + lane < a.batch ? max(1, (tiles_of(len) + r.q - 1) / r.q) : 0;
    int incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, base + incl > unit);
    if (past) {
      const int l = __ffs(past) - 1;
      pc.b = b0 + l;
      pc.cb = u - unit * blocks;
      pc.len = tc2::uniform(__shfl_sync(0xffffffffu, len, l));
      pc.count = tc2::uniform(__shfl_sync(0xffffffffu, n, l));
      pc.p = tc2::uniform(unit - base - __shfl_sync(0xffffffffu, incl - n, l));
      const int tiles = tiles_of(pc.len);
      pc.t0 = min(pc.p * r.q, tiles);
      pc.n = min(pc.t0 + r.q, tiles) - pc.t0;
      return true;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

struct Maps {
  CUtensorMap q, k, v;
};

// Where a tile's keys lie: the table slot and the row in its page, stepped from tile to tile
// without a division.
struct Place {
  int slot, row;
  __device__ Place(int key, int page_size) : slot(key / page_size) { row = key - slot * page_size; }
  __device__ void step(int keys, int page_size) {
    row += keys;
    while (row >= page_size) {
      row -= page_size;
      ++slot;
    }
  }
};

// A copy warp (all lanes converged; one elected lane issues) of one CTA: the
// scores' share of each tile (keys 64 r .. + 63, all columns, in chunks of slabs) or
// the values' (in chunks of 64 keys, all the CTA's columns).  A copy costs its issuing warp ~365
// cycles whatever its size (measured: 8 KB a copy 23 bytes a cycle and warp, 24 KB 67; the
// SM's own limit is 85 to 118), so chunks are single copies of 24 and 32 KB, and the
// chunks of a ring are dealt out to several warps, each with stages of its own.
template <int DC, bool kLo, bool kV>
struct Loader {
  using L = Lay<DC, kLo>;
  static constexpr int kRing = kV ? L::kRingV : L::kRingK;
  static constexpr int kWarps = kV ? 2 : L::kRingK;      // warps the chunks are dealt to
  static constexpr int kChunks = kV ? 2 : L::kChunks;    // chunks per tile
  static_assert(kRing % kWarps == 0, "a stage belongs to one warp");
  const LatentAttnArgs &a;
  const CUtensorMap *map;
  unsigned char *sm;
  uint64_t *bars;
  volatile int *abort_flag;
  uint32_t rank;
  int lane;
  bool lead;
  bool whole;  // pages of whole half tiles: boxes of 64 rows (else of 16)
  PageCache pages;
  int which;                 // of the kWarps
  int seq = 0, ragged = 0;   // chunks of all warps, chunks of this one landed on kRagged, over all pieces

  __device__ Loader(const LatentAttnArgs &a_, const CUtensorMap *m, unsigned char *sm_,
                    uint64_t *bars_, volatile int *ab, uint32_t rank_, bool lead_, int which_,
                    const PageCache &pages_)
      : a(a_), map(m), sm(sm_), bars(bars_), abort_flag(ab), rank(rank_), lead(lead_), pages(pages_),
        which(which_) {
    lane = threadIdx.x & 31;
    whole = a.page_size % kHalf == 0;
  }

  // Pool rows of a tile's boxes (whole: two of 64 rows; else eight of 16); -1: not loaded.
  // `left`: the row's keys from the tile's first on.
  __device__ uint32_t find(const int32_t *tbl, int n_slots, int left, Place at, int (&ys)[8]) {
    uint32_t bad = 0;
    if (whole) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ys[i] = -1;
        if (i * kHalf >= left) break;
        const int page = pages.get(tbl, at.slot, n_slots, lane);
        if (page < 0 || (long long)page >= a.num_pages)
          bad |= 0xFu << (4 * i);
        else
          ys[i] = page * a.page_size + at.row;
        at.step(kHalf, a.page_size);
      }
      return bad;
    }
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      int y = -1;
      if (16 * i < left) {
        const int page = pages.get(tbl, at.slot, n_slots, lane);
        if (page < 0 || (long long)page >= a.num_pages)
          bad |= 1u << i;
        else
          y = page * a.page_size + at.row;
      }
      at.step(16, a.page_size);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k == i) ys[k] = y;
    }
    return bad;
  }

  __device__ bool free_stage(int st) {
    return seq < kRing || tc::all_wait(bars + (kV ? L::kEmptyV : L::kEmptyK) + st,
                                        (seq / kRing - 1) & 1, abort_flag, a.status);
  }

  __device__ bool run(const Piece &pc) {
    if (a.batch > 1) pages.base = -1;  // another row's table
    const int32_t *tbl = a.page_tables + (size_t)pc.b * a.table_stride;
    const int n_slots = (pc.len - 1) / a.page_size + 1;
    Place at(pc.t0 * kKeys, a.page_size);
    for (int j = 0; j < pc.n; ++j) {
      const int left = pc.len - (pc.t0 + j) * kKeys;
      int ys[8];
      const uint32_t bad = find(tbl, n_slots, left, at, ys);
      at.step(kKeys, a.page_size);
#pragma unroll 1
      for (int c = 0; c < kChunks; ++c, ++seq) {
        if (seq % kWarps != which) continue;
        if (!free_stage(seq % kRing)) return false;
        if (kV)
          load_v(c, min(left, kKeys), ys, bad);
        else
          load_k(c, ys, bad);
      }
    }
    return true;
  }

  __device__ void load_k(int c, const int (&ys)[8], uint32_t bad) {
    // rows behind the row's end (inside a page) may come along: their scores are masked
    const int st = seq % kRing;
    const uint32_t dst = smem_u32(sm + L::kOffK + st * L::kKBytes);
    const uint32_t bar = tc2::map_to(smem_u32(bars + L::kFullK + st), 0);
    uint32_t rows = 0;  // both CTAs'
    if (whole)
      rows = (ys[0] >= 0 ? kHalf : 0) + (ys[1] >= 0 ? kHalf : 0);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) rows += ys[i] >= 0 ? 16 : 0;
    tc2::expect_tx(bars + L::kFullK + st, rows * 128 * L::kChunkSlabs, lead && rank == 0);
    if (whole) {
      const int y = rank == 0 ? ys[0] : ys[1];
      tc2::tma_load_3d(dst, map, 0, y, c * L::kChunkSlabs, bar, lead && y >= 0);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int y = rank == 0 ? ys[i] : ys[4 + i];
        for (int s = 0; s < L::kChunkSlabs; ++s)
          tc2::tma_load_3d(dst + s * kSlab + i * 16 * 128, map, 0, y, c * L::kChunkSlabs + s, bar,
                           lead && y >= 0);
      }
    }
    if (c == 0 && lead) {
      const int tile = seq / kChunks;
      if (bad && rank == 0) raise_fault(a.status, PSKV_FAULT_BAD_PAGE);
      reinterpret_cast<TileInfo *>(sm + L::kOffInfo)[tile % kInfo].bad = bad;
      mbar_arrive(bars + L::kInfoFull + tile % kInfo);
    }
    __syncwarp();
  }

  __device__ void load_v(int h, int vhi, const int (&ys)[8], uint32_t bad) {
    const int st = seq % kRing;
    unsigned char *stage = sm + L::kOffV + st * L::kVBytes;
    const uint32_t dst = smem_u32(stage);
    uint64_t *own_full = bars + L::kFullV + st;
    const uint32_t full = tc2::map_to(smem_u32(own_full), 0);
    const uint32_t hbad = (bad >> (4 * h)) & 0xFu;
    const bool plain = vhi >= (h + 1) * kHalf && hbad == 0;
    // a chunk with rows that must not be met lands on a barrier of this CTA first; one
    // without any key is passed on as it is and not met at all
    const bool dead = vhi <= h * kHalf;
    uint64_t *rag = bars + L::kRagged + which;
    const uint32_t bar = plain ? full : smem_u32(rag);
    if (!dead) {
      uint32_t rows = 0;
      if (whole)
        rows = (h == 0 ? ys[0] : ys[1]) >= 0 ? kHalf : 0;
      else
#pragma unroll
        for (int i = 0; i < 4; ++i) rows += (h == 0 ? ys[i] : ys[4 + i]) >= 0 ? 16 : 0;
      const uint32_t bytes = rows * 256 * L::kBlocks;
      if (!plain)
        tc2::expect_tx(rag, bytes, lead);
      else
        tc2::expect_tx(own_full, 2 * bytes, lead && rank == 0);
      if (whole) {
        const int y = h == 0 ? ys[0] : ys[1];
        tc2::tma_load_4d(dst, map, 0, y, 2 * (int)rank, 0, bar, lead && y >= 0);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int y = h == 0 ? ys[i] : ys[4 + i];
          for (int s = 0; s < 2 * L::kBlocks; ++s)
            tc2::tma_load_4d(dst + s * kSlab + i * 16 * 128, map, 0, y, 2 * (int)rank + (s & 1),
                             s >> 1, bar, lead && y >= 0);
        }
      }
    }
    if (!plain && !dead) {
      // rows behind the end or of skipped groups may hold anything and meet P = 0: zero them
      __syncwarp();
      if (!mbar_wait(rag, ragged & 1)) {  // (given up on, the chunk is passed on all the same)
        *abort_flag = 1;
        raise_fault(a.status, PSKV_FAULT_WAIT_TIMEOUT);
      }
      ++ragged;
      for (int e = lane; e < kHalf * 16 * L::kBlocks; e += 32) {
        const int row = e & (kHalf - 1), piece = e >> 6;
        if (row + h * kHalf >= vhi || ((hbad >> (row >> 4)) & 1u))
          *reinterpret_cast<uint4 *>(stage + (piece >> 3) * kSlab + row * 128 + (piece & 7) * 16) =
              make_uint4(0, 0, 0, 0);
      }
      tc::fence_smem_for_async();
      __syncwarp();
    }
    if (!plain && lead && rank == 0) mbar_arrive(own_full);  // in place of the copies' count
    if (plain || dead)
      tc2::arrive_pair(full, lead);
    else
      tc2::arrive_pair_release(full, lead);
    __syncwarp();
  }

  // Wait (bounded) for the last copies into each stage, of both CTAs (their count is the even CTA's).
  __device__ void drain() {
    if (rank != 0) return;
    for (int s = max(0, seq - kRing); s < seq; ++s)
      if (s % kWarps == which) mbar_wait(bars + (kV ? L::kFullV : L::kFullK) + s % kRing, (s / kRing) & 1);
  }

  // All of the cluster's pieces.
  __device__ void run_all(const Rows &rows, int first, int step) {
    int k = 0;
    Piece pc;
    for (int u = first; find_piece(a, u, rows, lane, pc); u += step) {
      if (pc.n == 0) continue;
      // the last piece's O may be leaving through the rings
      if (k > 0 && !tc::all_wait(bars + L::kOut, (k - 1) & 1, abort_flag, a.status)) break;
      ++k;
      if (!run(pc)) break;
    }
    drain();
  }
};

}  // namespace

template <int DC, bool kLo, bool kTree>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    pskv_attn_latent(const LatentAttnArgs a, const __grid_constant__ Maps maps) {
  using L = Lay<DC, kLo>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *sm = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::kOffBar);
  uint32_t *slot = reinterpret_cast<uint32_t *>(sm + L::kOffSlot);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + L::kOffAbort);
  const int warp = tc2::uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rank = tc2::cluster_rank();
  const bool lead = elect_one();  // one thread of each warp
  if (sm + L::kUsed > smem_raw + L::kSmemBytes) {  // (never seen) no room for the alignment
    raise_fault(a.status, PSKV_FAULT_WAIT_TIMEOUT);
    return;
  }
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

  // set up before the previous kernel's results are waited for
  if (warp == 1) {
    if (lane == 0) {
      tc2::prefetch_map(&maps.q);
      tc2::prefetch_map(&maps.k);
      for (int s = 0; s < L::kRingK; ++s) {
        mbar_init(&bars[L::kFullK + s], 1);
        mbar_init(&bars[L::kEmptyK + s], 1);
      }
      for (int s = 0; s < L::kRingV; ++s) {
        mbar_init(&bars[L::kFullV + s], 3);  // the expected bytes, and a word from either V copy warp
        mbar_init(&bars[L::kEmptyV + s], 1);
      }
      for (int r = 0; r < 2; ++r) {
        mbar_init(&bars[L::kSFull + r], 1);
        mbar_init(&bars[L::kSFree + r], 2 * kSoftWarps);  // the softmax warps of both CTAs
        mbar_init(&bars[L::kRagged + r], 1);
        mbar_init(&bars[L::kPvDone + r], 1);
      }
      mbar_init(&bars[L::kPFull], 2 * kSoftWarps);
      for (int k = 0; k < kInfo; ++k) mbar_init(&bars[L::kInfoFull + k], 1);
      mbar_init(&bars[L::kQFull], 1);
      mbar_init(&bars[L::kQFree], 1);
      mbar_init(&bars[L::kOut], kSoftWarps);
      mbar_init(&bars[L::kDrainS], 1);
      mbar_init(&bars[L::kDrainV], 1);
      *abort_flag = 0;
      mbar_fence_init();
    }
    __syncwarp();
  } else if (warp == 0) {
    tc2::alloc(slot, kTmemCols);
  } else if (warp == 14 && lane == 0) {
    tc2::prefetch_map(&maps.v);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc2::cluster_sync();  // both CTAs' barriers are set up
  tc::fence_after_sync();
  const uint32_t tmem = *slot;
  auto wait = [&](int s, uint32_t parity) {
    return tc::all_wait(bars + s, parity, abort_flag, a.status);
  };
  auto wait_pair = [&](int s, uint32_t parity) {  // for what the other CTA's threads and copies bring
    return tc2::all_wait(bars + s, parity, abort_flag, a.status);
  };
  // a single row's copy warps read its page ids beside its length, not behind it (0.2 us)
  PageCache pages;
  if (a.batch == 1)
    pages.base = (int)((long long)(first / ((a.num_tokens * a.num_q_heads + 127) / 128)) *
                       a.tiles_per_piece * kKeys / a.page_size);
  pdl_wait();
  pdl_launch_dependents();
  if (a.batch == 1 && (warp == 3 || warp >= 12))
    pages.val = pages.base + lane < a.table_stride ? __ldg(a.page_tables + pages.base + lane) : -1;
  const Rows rows = read_rows(a, lane, blockIdx.x == 0 && warp == 0);
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.ws_tiles) *a.ws_tiles = rows.q;  // for the merge
  Piece pc;

  if (warp == 0 && rank == 0) {
    // ---- the score products (all lanes alike, one issues)
    bool ok = true;
    int seq = 0, g = 0, k = 0;  // chunks, tiles, pieces so far
    const uint32_t q0 = smem_u32(sm + L::kOffQ), k0 = smem_u32(sm + L::kOffK);
    for (int u = first; ok && find_piece(a, u, rows, lane, pc); u += step) {
      if (pc.n == 0) continue;
      ok = wait_pair(L::kQFull, k & 1);
      ++k;
      for (int j = 0; ok && j < pc.n; ++j, ++g) {
        const int r = g & 1;
        if (g >= 2) ok = wait_pair(L::kSFree + r, (g / 2 - 1) & 1);
#pragma unroll 1
        for (int c = 0; ok && c < L::kChunks; ++c, ++seq) {
          const int st = seq % L::kRingK;
          ok = wait_pair(L::kFullK + st, (seq / L::kRingK) & 1);
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t kc = k0 + st * L::kKBytes, qc = q0 + c * L::kKBytes;
#pragma unroll
          for (int kk = 0; kk < 4 * L::kChunkSlabs; ++kk) {
            const uint32_t at = (kk >> 2) * kSlab + (kk & 3) * 32;
            tc2::mma(tmem + kSCol + kHalf * r, tc::smem_desc(qc + at, 16, 1024),
                     tc::smem_desc(kc + at, 16, 1024), L::kIdescS, c > 0 || kk > 0, lead);
          }
          tc2::commit_both(bars + L::kEmptyK + st, lead);
        }
        if (ok) tc2::commit_both(bars + L::kSFull + r, lead);
      }
      tc2::commit_both(bars + L::kQFree, lead);
    }
    tc2::commit_both(bars + L::kDrainS, lead);
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    // ---- the value products
    bool ok = true;
    int g = 0;
    const uint32_t p0 = smem_u32(sm + L::kOffP), v0 = smem_u32(sm + L::kOffV);
    for (int u = first; ok && find_piece(a, u, rows, lane, pc); u += step)
      for (int j = 0; ok && j < pc.n; ++j, ++g) {
        const bool both = pc.len - (pc.t0 + j) * kKeys > kHalf;  // keys in the second half
        ok = wait_pair(L::kPFull, g & 1);
#pragma unroll 1
        for (int h = 0; ok && h < 2; ++h) {
          const int sq = 2 * g + h, st = sq % L::kRingV;
          ok = wait_pair(L::kFullV + st, (sq / L::kRingV) & 1);
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t vc = v0 + st * L::kVBytes;
          if (h == 0 || both)
#pragma unroll
            for (int nb = 0; nb < L::kBlocks; ++nb)
#pragma unroll
              for (int part = 0; part < (kLo ? 2 : 1); ++part)
#pragma unroll
                for (int kk = 0; kk < kHalf / 16; ++kk)
                  tc2::mma(tmem + kOCol + 128 * nb,
                           tc::smem_desc(p0 + (2 * part + h) * kSlab + kk * 32, 16, 1024),
                           tc::smem_desc(vc + 2 * nb * kSlab + kk * 2048, kSlab, 1024), L::kIdescPV,
                           j > 0 || h > 0 || part > 0 || kk > 0, lead);
          tc2::commit_both(bars + L::kEmptyV + st, lead);
          tc2::commit_both(bars + L::kPvDone + h, lead);
        }
      }
    tc2::commit_both(bars + L::kDrainV, lead);
    __syncwarp();
  } else if (warp == 2) {
    // ---- Q of every piece (this CTA's 64 columns; behind the row's last column: other rows' or zeros)
    int k = 0;
    const int cols = a.num_tokens * a.num_q_heads;
    for (int u = first; find_piece(a, u, rows, lane, pc); u += step) {
      if (pc.n == 0) continue;
      if (k > 0 && !wait(L::kQFree, (k - 1) & 1)) break;
      tc2::expect_tx(bars + L::kQFull, 2 * L::kQBytes, lead && rank == 0);
      tc2::tma_load_3d(smem_u32(sm + L::kOffQ), &maps.q, 0,
                       pc.b * cols + pc.cb * 128 + (int)rank * kRows, 0,
                       tc2::map_to(smem_u32(bars + L::kQFull), 0), lead);
      __syncwarp();
      ++k;
    }
    if (rank == 0 && k > 0) mbar_wait(bars + L::kQFull, (k - 1) & 1);
  } else if (warp == 3 || warp == 12 || warp == 13) {
    const int which = warp == 3 ? 0 : warp - 11;
    if (which < L::kRingK)
      Loader<DC, kLo, false>(a, &maps.k, sm, bars, abort_flag, rank, lead, which, pages).run_all(rows, first, step);
  } else if (warp >= 14) {
    Loader<DC, kLo, true>(a, &maps.v, sm, bars, abort_flag, rank, lead, warp - 14, pages).run_all(rows, first, step);
  } else if (warp >= 4 && warp <= 11) {
    // ---- the softmax: thread (row i, keys 64 kh + 32 gr .. + 31 of the tile).  The loops never
    // leave early (the four warps of a row's threads meet every tile); after a failed wait
    // results are not written.
    const int w = warp & 3, gr = (warp - 4) >> 2, i = (32 * w + lane) & (kRows - 1), kh = w >> 1;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * w) << 16);
    float *red = reinterpret_cast<float *>(sm + L::kOffRed);
    const TileInfo *info = reinterpret_cast<const TileInfo *>(sm + L::kOffInfo);
    const float sc = a.scale_log2;
    const uint32_t s_free = tc2::map_to(smem_u32(bars + L::kSFree), 0);
    const uint32_t p_full = tc2::map_to(smem_u32(bars + L::kPFull), 0);
    const int cols = a.num_tokens * a.num_q_heads;
    bool ok = true;
    int g = 0;      // tiles so far
    int meets = 0;  // meetings so far: their buffers alternate
    for (int u = first; find_piece(a, u, rows, lane, pc); u += step) {
      const int col0 = pc.cb * 128 + (int)rank * kRows, col = col0 + i;
      const size_t row0 = (size_t)pc.b * cols + col0;
      if (pc.n == 0) {  // a row without keys (of one piece): zeros
        const int es = a.out_dtype == PSKV_DTYPE_BF16 ? 2 : 4;
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<char *>(a.out) + (row0 + i) * DC * es);
        if (col < cols)
          for (int e = 2 * gr + kh; e < DC * es / 16; e += 4) dst[e] = make_uint4(0, 0, 0, 0);
        __syncwarp();  // (the next piece's tensor-memory loads want the warp together)
        continue;
      }
      // keys below lim are seen (columns behind the last, whose results go nowhere, see all: a
      // warp of theirs would mask every tile for nothing)
      // (of a drafted tree: the keys before the window, and in it what the token's mask holds)
      const int token = col / a.num_q_heads, w0 = pc.len - a.num_tokens;
      const int lim = col < cols ? (kTree ? w0 : w0 + token + 1) : pc.len;
      unsigned long long sees = 0;
      if (kTree && col < cols) {
        const unsigned long long mask = a.tree_mask[(size_t)pc.b * a.num_tokens + token], own = 1ull << token;
        sees = mask & (own | (own - 1));
        if (sees != mask || !(mask & own)) raise_fault(a.status, PSKV_FAULT_BAD_MASK);
      }
      __syncwarp();
      float m = -CUDART_INF_F, l = 0.f;
      for (int j = 0; j < pc.n; ++j, ++g, ++meets) {
        const int r = g & 1;
        ok = ok && wait(L::kSFull + r, (g >> 1) & 1);
        ok = ok && wait(L::kInfoFull + g % kInfo, (g / kInfo) & 1);
        const uint32_t bad = (info[g % kInfo].bad >> (4 * kh + 2 * gr)) & 3u;
        tc::fence_after_sync();
        uint32_t v[32];
        tc::ld32(lane_base + kSCol + kHalf * r + 32 * gr, v);
        tc::wait_ld();
        tc::reg_fence(v);
        tc::fence_before_sync();
        __syncwarp();
        float x[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) x[c] = __uint_as_float(v[c]);
        // scores in log2 units are mul * x: whole tiles leave the product to the exponent's
        // multiply-add, others (and scales that are not positive) take it before the mask (by
        // selection: rows never loaded may hold anything)
        const int key0 = (pc.t0 + j) * kKeys + kHalf * kh + 32 * gr;
        float mul = sc;
        bool some = key0 + 32 > lim;  // of these keys are not seen
        uint32_t vis = ~0u;           // (a tree's) bit c: key0 + c is seen, before the window or by the mask
        if constexpr (kTree) {
          const int d = key0 - lim;
          if (some) vis = d >= 64 ? 0u : d >= 0 ? (uint32_t)(sees >> d) : (uint32_t)(sees << -d) | ((1u << -d) - 1u);
          some = vis != ~0u;
        }
        if (__any_sync(0xffffffffu, some || bad != 0 || !(sc > 0.f))) {
          mul = 1.f;
          if constexpr (kTree) {
            if (bad & 1u) vis &= 0xffff0000u;
            if (bad & 2u) vis &= 0x0000ffffu;
#pragma unroll
            for (int c = 0; c < 32; ++c) x[c] = (vis >> c) & 1u ? x[c] * sc : -CUDART_INF_F;
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              x[c] = key0 + c < lim && !((bad >> (c >> 4)) & 1u) ? x[c] * sc : -CUDART_INF_F;
          }
        }
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < 32; ++c) mx[c & 3] = fmaxf(mx[c & 3], x[c]);
        float *mine = red + (meets & 1) * 4 * kRows + i;
        mine[(2 * kh + gr) * kRows] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * mul;
        asm volatile("bar.sync %0, 128;" ::"r"(1 + (w & 1)) : "memory");
        const float mt = fmaxf(fmaxf(mine[0], mine[kRows]), fmaxf(mine[2 * kRows], mine[3 * kRows]));
        float alpha = 1.f;
        bool rescale = false;
        if (mt > m + kSlack) {
          rescale = m != -CUDART_INF_F;  // with m = -inf the row's O and l are still 0
          alpha = rescale ? ex2(m - mt) : 1.f;
          l *= alpha;
          m = mt;
        }
        const float off = m == -CUDART_INF_F ? 0.f : -m;
        uint32_t hi[16], lo[kLo ? 16 : 1];
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float p0 = ex2(fmaf(x[2 * e], mul, off)), p1 = ex2(fmaf(x[2 * e + 1], mul, off));
          hi[e] = pack_bf16x2(p0, p1);
          if (kLo) {
            lo[e] = pack_bf16x2(p0 - bf16_lo(hi[e]), p1 - bf16_hi(hi[e]));
            s0 += p0;
            s1 += p1;
          } else {
            s0 += bf16_lo(hi[e]);
            s1 += bf16_hi(hi[e]);
          }
        }
        l += s0 + s1;
        // half kh of P is free once its values of the last tile are done
        if (g >= 1) ok = ok && wait(L::kPvDone + kh, (g - 1) & 1);
        unsigned char *prow = sm + L::kOffP + kh * kSlab + i * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int at = ((4 * gr + c) ^ (i & 7)) << 4;
          *reinterpret_cast<uint4 *>(prow + at) =
              make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
          if constexpr (kLo)
            *reinterpret_cast<uint4 *>(prow + 2 * kSlab + at) =
                make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
        }
        if (__any_sync(0xffffffffu, rescale)) {
          ok = ok && wait(L::kPvDone + 1, (g - 1) & 1);  // (and with the second half the first)
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = gr * (DC / 128); c < (gr + 1) * (DC / 128); ++c) {
            uint32_t o[32];
            tc::ld32(lane_base + kOCol + 32 * c, o);
            tc::wait_ld();
            tc::reg_fence(o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tc::st32(lane_base + kOCol + 32 * c, o);
            tc::wait_st();
          }
        }
        tc::fence_smem_for_async();
        tc::fence_before_sync();
        __syncwarp();
        tc2::arrive_pair_release(p_full, lead);
        // S(j + 2) may take the region: not earlier, as the tensor pipe takes products in order
        // and scores that are not needed yet would hold up this tile's values
        tc2::arrive_pair(s_free + 8 * r, lead);
      }
      // ---- the row's sum over its four threads, then its columns: this thread's are
      // 128 kh + [0, 128) of one 256 (DC = 256: half of them)
      float *sums = red + (meets & 1) * 4 * kRows + i;
      ++meets;
      sums[(2 * kh + gr) * kRows] = l;
      asm volatile("bar.sync %0, 128;" ::"r"(1 + (w & 1)) : "memory");
      l = (sums[0] + sums[kRows]) + (sums[2 * kRows] + sums[3 * kRows]);
      ok = ok && wait(L::kPvDone + 1, (g - 1) & 1);
      tc::fence_after_sync();
      const bool empty = m == -CUDART_INF_F;
      if (pc.count > 1) {
        // a partial: [column / 4][32 query columns] of this warp's group of 32
        const int groups = (cols + 31) / 32, group = col0 / 32 + (w & 1);
        if (ok && group < groups) {
          const size_t at = ((size_t)pc.b * groups + group) * a.num_splits + pc.p;
          const uint64_t keep = make_evict_last_policy();
          float4 *dst = reinterpret_cast<float4 *>(a.ws_o) + at * (DC / 4 * 32) + lane;
#pragma unroll 2
          for (int c = gr * (DC / 128); c < (gr + 1) * (DC / 128); ++c) {
            uint32_t o[32];
            tc::ld32(lane_base + kOCol + 32 * c, o);
            tc::wait_ld();
            tc::reg_fence(o);
            const int d4 = 64 * (c >> 2) + 32 * kh + 8 * (c & 3);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              st_keep(dst + (d4 + k) * 32,
                      make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                  __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3])),
                      keep);
          }
          if (kh == 0 && gr == 0) {
            a.ws_m[at * 32 + lane] = m;
            a.ws_l[at * 32 + lane] = l;
          }
        }
      } else {
        // final rows, put together in the drained rings so that they leave in whole lines
        const float mul = empty ? 0.f : 1.f / l;
        const bool bf16_rows = a.out_dtype == PSKV_DTYPE_BF16;
        const int bytes = bf16_rows ? DC * 2 : DC * 4, pitch = bytes + 16;
        unsigned char *stage = sm + L::kOffK;
#pragma unroll 1
        for (int c = gr * (DC / 128); c < (gr + 1) * (DC / 128); ++c) {
          uint32_t o[32];
          tc::ld32(lane_base + kOCol + 32 * c, o);
          tc::wait_ld();
          tc::reg_fence(o);
          const int d = 256 * (c >> 2) + 128 * kh + 32 * (c & 3);
          float f[32];  // (a column that met no key may hold anything: zeros by selection)
#pragma unroll
          for (int k = 0; k < 32; ++k) f[k] = empty ? 0.f : __uint_as_float(o[k]) * mul;
          if (bf16_rows) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4 *>(stage + i * pitch + 2 * d + 16 * k) =
                  make_uint4(pack_bf16x2(f[8 * k], f[8 * k + 1]),
                             pack_bf16x2(f[8 * k + 2], f[8 * k + 3]),
                             pack_bf16x2(f[8 * k + 4], f[8 * k + 5]),
                             pack_bf16x2(f[8 * k + 6], f[8 * k + 7]));
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<float4 *>(stage + i * pitch + 4 * d + 16 * k) =
                  make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
          }
        }
        if (ok && empty && col < cols && kh == 0 && gr == 0) raise_fault(a.status, PSKV_FAULT_EMPTY_ROW);
        asm volatile("bar.sync 3, 256;" ::: "memory");
        if (ok)
          for (int r = warp - 4; r < kRows && col0 + r < cols; r += kSoftWarps)
            for (int e = 16 * lane; e < bytes; e += 512)
              *reinterpret_cast<uint4 *>(static_cast<char *>(a.out) + (row0 + r) * bytes + e) =
                  *reinterpret_cast<const uint4 *>(stage + r * pitch + e);
        tc::fence_smem_for_async();  // these accesses before the next piece's copies
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + L::kOut);
    }
  }
  // every product done (both CTAs learn it; every copy has landed) before the memory is released
  if (warp == 0) mbar_wait(bars + L::kDrainS, 0);
  if (warp == 1) mbar_wait(bars + L::kDrainV, 0);
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc2::cluster_sync();
  if (warp == 0) {
    tc::fence_after_sync();
    tc2::dealloc(tmem, kTmemCols);
  }
}

// Folds the pieces of a row (those longer than one piece; the others are final):
//   M = max m_p,  l = sum l_p 2^(m_p - M),  out = sum O_p 2^(m_p - M) / l,
// the exact rescaling identity, in index order within each of kLanes interleaved
// states and then over these, so the result is deterministic.  A block takes a group of 32 query
// columns and 16 of their output columns: a warp reads four output columns of all 32 as one
// 512-byte line.  Bound by the partials' bytes (L2) and its three dependent loads.
template <int DC, int kLanes>
__global__ void __launch_bounds__(128 * kLanes) pskv_merge_latent(const LatentAttnArgs a) {
  __shared__ float m_s[kLanes][32], l_s[kLanes][32];
  __shared__ float4 o_s[kLanes][4][32];
  const int i = threadIdx.x & 31, f = (threadIdx.x >> 5) & 3, s = threadIdx.x >> 7;
  const int cols = a.num_tokens * a.num_q_heads, groups = (cols + 31) / 32;
  const int b = blockIdx.x / groups, group = blockIdx.x - b * groups;
  pdl_wait();
  pdl_launch_dependents();
  bool bad;
  const int q = *a.ws_tiles, len = usable_len(a, b, &bad);
  const int count = (tiles_of(len) + q - 1) / q;
  if (count <= 1) return;
  const size_t at = (size_t)blockIdx.x * a.num_splits;
  const float *m = a.ws_m + at * 32 + i, *l = a.ws_l + at * 32 + i;
  const float4 *o = reinterpret_cast<const float4 *>(a.ws_o) +
                    (at * (DC / 4) + blockIdx.y * 4 + f) * 32 + i;
  constexpr int kMany = kLanes == 8 ? 5 : 8;  // pieces a lane loads at once (registers)
  float M = -CUDART_INF_F, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = s; p0 < count; p0 += kMany * kLanes) {
    float mp[kMany], lp[kMany];
    float4 v[kMany];
#pragma unroll
    for (int k = 0; k < kMany; ++k) {
      const int p = p0 + k * kLanes;
      mp[k] = -CUDART_INF_F;
      if (p < count) {
        mp[k] = m[p * 32];
        lp[k] = l[p * 32];
        v[k] = __ldcs(o + (size_t)p * (DC / 4 * 32));
      }
    }
    float top = M;
#pragma unroll
    for (int k = 0; k < kMany; ++k) top = fmaxf(top, mp[k]);
    if (top == -CUDART_INF_F) continue;
    const float w0 = exp2f(M - top);
    L *= w0;
    acc.x *= w0;
    acc.y *= w0;
    acc.z *= w0;
    acc.w *= w0;
    M = top;
#pragma unroll
    for (int k = 0; k < kMany; ++k)
      if (mp[k] != -CUDART_INF_F) {  // an empty piece's O is never used
        const float w = exp2f(mp[k] - top);
        L = fmaf(lp[k], w, L);
        acc.x = fmaf(v[k].x, w, acc.x);
        acc.y = fmaf(v[k].y, w, acc.y);
        acc.z = fmaf(v[k].z, w, acc.z);
        acc.w = fmaf(v[k].w, w, acc.w);
      }
  }
  o_s[s][f][i] = acc;
  if (f == 0) {
    m_s[s][i] = M;
    l_s[s][i] = L;
  }
  __syncthreads();
  // thread (column i, four output columns f): 32 bytes of a row from four neighbouring threads
  if (threadIdx.x >= 128) return;
  const int r = threadIdx.x >> 2, k4 = threadIdx.x & 3, col = group * 32 + r;
  if (col >= cols) return;
  float top = -CUDART_INF_F, sum = 0.f;
#pragma unroll
  for (int k = 0; k < kLanes; ++k) top = fmaxf(top, m_s[k][r]);
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kLanes; ++k)
    if (m_s[k][r] != -CUDART_INF_F) {
      const float w = exp2f(m_s[k][r] - top);
      const float4 v = o_s[k][k4][r];
      sum = fmaf(l_s[k][r], w, sum);
      acc.x = fmaf(v.x, w, acc.x);
      acc.y = fmaf(v.y, w, acc.y);
      acc.z = fmaf(v.z, w, acc.z);
      acc.w = fmaf(v.w, w, acc.w);
    }
  const bool empty = top == -CUDART_INF_F;
  if (empty && k4 == 0 && blockIdx.y == 0) raise_fault(a.status, PSKV_FAULT_EMPTY_ROW);
  const float inv = empty ? 0.f : 1.f / sum;
  const size_t dst = ((size_t)b * cols + col) * (DC / 4) + blockIdx.y * 4 + k4;
  if (a.out_dtype == PSKV_DTYPE_BF16)
    static_cast<uint2 *>(a.out)[dst] =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  else
    static_cast<float4 *>(a.out)[dst] = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
}

namespace {

template <int DC, bool kLo, bool kTree>
cudaError_t launch(const LatentAttnArgs &a, cudaStream_t s) {
  using L = Lay<DC, kLo>;
  static std::atomic<bool> attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(dev >= 0 && dev < 64 && attr_set[dev])) {
    e = cudaFuncSetAttribute(pskv_attn_latent<DC, kLo, kTree>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             L::kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const bool whole = a.page_size % kHalf == 0;
  const long long cols = (long long)a.num_tokens * a.num_q_heads;
  Maps maps;
  if (!tc2::make_slab_map(&maps.q, a.q, a.batch * cols, DC + 64, kRows, L::kSlabs) ||
      !tc2::make_slab_map(&maps.k, a.pool, a.num_pages * a.page_size, DC + 64, whole ? kHalf : 16,
                          whole ? L::kChunkSlabs : 1) ||
      !tc2::make_block_map(&maps.v, a.pool, a.num_pages * a.page_size, DC + 64, DC / 256,
                           whole ? kHalf : 16, whole ? 2 : 1, whole ? DC / 256 : 1))
    return cudaErrorInvalidValue;
  return launch_pdl(pskv_attn_latent<DC, kLo, kTree>, dim3(2 * (unsigned)a.clusters), dim3(kThreads),
                    L::kSmemBytes, s, a, maps);
}

}  // namespace

cudaError_t launch_attn_latent(const LatentAttnArgs &a, int dc, cudaStream_t s) {
  const bool lo = a.out_dtype == PSKV_DTYPE_F32, tree = a.tree_mask != nullptr;
  if (dc == 512 && tree) return lo ? launch<512, true, true>(a, s) : launch<512, false, true>(a, s);
  if (dc == 256 && tree) return lo ? launch<256, true, true>(a, s) : launch<256, false, true>(a, s);
  if (dc == 512) return lo ? launch<512, true, false>(a, s) : launch<512, false, false>(a, s);
  if (dc == 256) return lo ? launch<256, true, false>(a, s) : launch<256, false, false>(a, s);
  return cudaErrorInvalidValue;
}

cudaError_t launch_merge_latent(const LatentAttnArgs &a, int dc, cudaStream_t s) {
  const int groups = (a.num_tokens * a.num_q_heads + 31) / 32;
  const dim3 grid((unsigned)(a.batch * groups), dc / 16);
  // eight states a block for many pieces (a lane then loads its share at once), two for few
  const bool many = a.num_splits > 16;
  if (dc == 512)
    return many ? launch_pdl(pskv_merge_latent<512, 8>, grid, dim3(1024), 0, s, a)
                : launch_pdl(pskv_merge_latent<512, 2>, grid, dim3(256), 0, s, a);
  if (dc == 256)
    return many ? launch_pdl(pskv_merge_latent<256, 8>, grid, dim3(1024), 0, s, a)
                : launch_pdl(pskv_merge_latent<256, 2>, grid, dim3(256), 0, s, a);
  return cudaErrorInvalidValue;
}

}  // namespace pskv
