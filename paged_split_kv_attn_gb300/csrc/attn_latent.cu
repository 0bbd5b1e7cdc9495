// attn_latent.cu -- absorbed attention over a paged latent pool on a pair of CTAs.
//
// For every query column (token t, head h) of a row: s_i = scale * q . row_i over
// the dc + 64 columns of a cached row, o = sum_i softmax(s)_i row_i[0:dc].  All
// heads share the rows, so a block of 128 query columns meets each cached row once:
// per key 2 * 128 * (2 dc + 64) operations against 2 (dc + 64) bytes.
//
// A cluster of two CTAs takes 128 columns of one row and a partition of its keys,
// as one tcgen05 product of M = 128 over the pair (cta_group::2): CTA r holds
// columns 64 r .. + 63 of Q (dc + 64 wide) in shared memory, and of O (64 x dc
// in f32: 256 tensor-memory columns, half of the lanes holding half of the
// columns each), which one CTA alone could not hold beside the scores (128 x 512 f32
// fill its tensor memory).  Per tile j of 64 keys:
//   S = Q K^T     N = 64 keys, CTA r brings the tile's keys 32 r .. + 31
//   softmax       thread (row i, half of the keys) masks its 32 scores; the two threads
//                 of a row exchange their maxima; the reference maximum moves only
//                 past a slack of 8 (log2 units), so O is rarely rescaled; P goes
//                 to shared memory as bf16 (f32 output: a hi + lo pair)
//   O += P V      per 256 columns: CTA r brings columns 128 r .. + 127 of each, all 64 keys
// The two products want a row in different CTAs (scores: by key, values: by column),
// so a CTA copies both shares: 1.9x of a row's bytes from L2, each byte once from
// HBM (the copies of the scores' share run ahead by a prefetch into L2).  Each of
// the rings has its own copy warp and its own issuing warp in the even CTA, so
// S(j + 1) runs while the softmax works on tile j.
//
// P is rounded to bf16 when the output is (the weights' rounding then adds about
// what the output's own does; the sum takes the rounded weights, so a lone key gives
// its row exactly); maxima, sums, O and partials are f32.
// Every wait is bounded; on expiry the CTA flags PSKV_FAULT_WAIT_TIMEOUT, lets
// what it issued finish and frees its tensor memory.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math_constants.h>

#include "latent.h"
#include "pskv_internal.cuh"
#include "tc_common.cuh"
#include "tc_ops.cuh"
#include "tc_pair.cuh"

namespace pskv {

namespace {

using tc::elect_one;
using tc::ex2;
using tc::PageCache;

constexpr int kKeys = 64;        // keys per tile
constexpr int kHalfKeys = 32;    // of which each CTA brings half to the scores
constexpr int kRows = 64;        // query columns per CTA (128 per pair)
constexpr int kThreads = 256;    // warps: 0 S, 1 K copies, 2-5 softmax, 6 V copies, 7 PV
constexpr int kTmemCols = 512;
constexpr int kOCol = 0;         // O: DC / 2 columns
constexpr int kSCol = 256;       // score region r at kSCol + 32 r
constexpr float kSlack = 8.f;
constexpr int kInfo = 8;         // tile records in flight: K runs kStages ahead of S, S two ahead of the softmax
constexpr int kAhead = 4;        // tiles the L2 prefetch runs ahead of the copies

template <int DC, bool kLo>
struct Lay {
  static constexpr int kSlabs = DC / 64 + 1;             // 64-column slabs of a row
  static constexpr int kQSlab = kRows * 128;             // 8 KB
  static constexpr int kKSlab = kHalfKeys * 128;         // 4 KB
  static constexpr int kVSlab = kKeys * 128;             // 8 KB
  static constexpr int kBlocks = DC / 256;               // value products per tile
  static constexpr int kVSlabs = 2 * kBlocks;            // this CTA's value slabs
  static constexpr int kQBytes = kSlabs * kQSlab;
  static constexpr int kKBytes = kSlabs * kKSlab;
  static constexpr int kVBytes = kVSlabs * kVSlab;
  static constexpr int kPBytes = kRows * 128;            // a tile's P (hi or lo)
  static constexpr int kPBufs = kLo ? 1 : 2;
  static constexpr int kStages = DC == 512 ? 2 : 4;      // of K and of V
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kQBytes;
  static constexpr int kOffV = kOffK + kStages * kKBytes;
  static constexpr int kOffP = kOffV + kStages * kVBytes;
  // barrier slots
  static constexpr int kFullK = 0;                       // (even CTA) both CTAs' K landed
  static constexpr int kFullV = kFullK + kStages;        // (even CTA) both CTAs' V landed
  static constexpr int kEmptyK = kFullV + kStages;       // S of the stage's tile done
  static constexpr int kEmptyV = kEmptyK + kStages;      // PV of the stage's tile done
  static constexpr int kSFull = kEmptyV + kStages;       // [2] S of region r done
  static constexpr int kSFree = kSFull + 2;              // [2] (even CTA) region r read in both CTAs
  static constexpr int kPFull = kSFree + 2;              // [2] (even CTA) P written in both CTAs
  static constexpr int kPvDone = kPFull + 2;             // [2] PV of the P buffer's tile done
  static constexpr int kInfoFull = kPvDone + 2;          // [8] a tile's record written
  static constexpr int kQFull = kInfoFull + kInfo;       // (even CTA) both CTAs' Q landed
  static constexpr int kRagged = kQFull + 1;             // this CTA's V of a tile that is not whole
  static constexpr int kDrainS = kRagged + 1;
  static constexpr int kDrainV = kDrainS + 1;
  static constexpr int kNumBars = kDrainV + 1;
  static constexpr int kOffBar = kOffP + (kLo ? 2 : kPBufs) * kPBytes;
  static constexpr int kOffInfo = (kOffBar + kNumBars * 8 + 15) & ~15;
  static constexpr int kOffRed = kOffInfo + kInfo * 16;  // float[2][2][64] maxima (then sums)
  static constexpr int kOffSlot = kOffRed + 2 * 2 * kRows * 4;
  static constexpr int kOffAbort = kOffSlot + 4;
  static constexpr int kSmemBytes = kOffAbort + 4 + 1024;  // + alignment of the dynamic base
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
  static_assert(kInfo >= kStages + 2, "tile records");
  static_assert(kQSlab % 1024 == 0 && kKSlab % 1024 == 0 && kOffP % 1024 == 0, "swizzle atoms");
  static constexpr uint32_t kIdescS = tc::instr_desc(2 * kRows, kKeys, false, false);
  static constexpr uint32_t kIdescPV = tc::instr_desc(2 * kRows, 256, false, true);
};

// Rows [0, vhi) of the tile hold keys of the partition; bit c of `bad` marks a
// 16-key group whose page id lies outside the pool (not loaded).
struct TileInfo {
  int vhi;
  uint32_t bad;
  int pad[2];
};

// The pair's share of the work, the same in every thread of both CTAs.
struct Plan {
  int b, cb, p;    // row, block of 128 columns, partition
  int cols, len;   // the row's query columns and keys
  int t0, n;       // tiles [t0, t0 + n)
  bool ok;
};

__device__ __forceinline__ Plan make_plan(const LatentAttnArgs &a) {
  Plan pl;
  const int blocks = (a.num_tokens * a.num_q_heads + 127) / 128;
  const int x = blockIdx.x >> 1;
  pl.cb = x % blocks;
  pl.p = x / blocks;
  pl.b = blockIdx.y;
  pl.cols = a.num_tokens * a.num_q_heads;
  const long long cap = (long long)a.table_stride * a.page_size;
  long long len = a.seq_lens[pl.b];
  pl.ok = !(len < 0 || len > cap || (len > 0 && len < a.num_tokens));
  len = len < 0 ? 0 : (len > cap ? cap : len);
  pl.len = (int)len;
  const int tiles = (pl.len + kKeys - 1) / kKeys, per = (tiles + a.num_splits - 1) / a.num_splits;
  pl.t0 = min(pl.p * per, tiles);
  pl.n = min(pl.t0 + per, tiles) - pl.t0;
  return pl;
}

struct Maps {
  CUtensorMap q, k, v;
};

// A copy warp (all lanes converged; one elected lane issues) of one CTA: the
// scores' share of each tile (keys 32 r .. + 31, all columns) or the values' (all
// keys, the CTA's columns).
template <int DC, bool kLo, bool kV>
struct Loader {
  using L = Lay<DC, kLo>;
  static constexpr int kBoxes = kKeys / 16;
  const LatentAttnArgs &a;
  const Plan &pl;
  const CUtensorMap *map;
  unsigned char *sm;
  uint64_t *bars;
  volatile int *abort_flag;
  uint32_t rank;
  int lane, n_slots;
  bool whole;  // pages of whole tiles: one box of all slabs (else 16 rows of a slab each)
  PageCache pages;
  int issued = 0, ragged = 0;  // tiles begun; of them landed on kRagged

  __device__ Loader(const LatentAttnArgs &a_, const Plan &pl_, const CUtensorMap *m,
                    unsigned char *sm_, uint64_t *bars_, volatile int *ab, uint32_t rank_)
      : a(a_), pl(pl_), map(m), sm(sm_), bars(bars_), abort_flag(ab), rank(rank_) {
    lane = threadIdx.x & 31;
    n_slots = (pl.len + a.page_size - 1) / a.page_size;
    whole = a.page_size % kKeys == 0;
  }

  // Pool rows of the tile's 16-key groups (whole pages: of the tile, in ys[0]); -1: not loaded.
  __device__ void find(int j, int (&ys)[kBoxes], TileInfo &inf) {
    const int32_t *tbl = a.page_tables + (size_t)pl.b * a.table_stride;
    const int key0 = (pl.t0 + j) * kKeys;
    inf.vhi = min(kKeys, pl.len - key0);
    inf.bad = 0;
    const int step = whole ? kKeys : 16;
#pragma unroll
    for (int i = 0; i < kBoxes; ++i) {
      ys[i] = -1;
      if (i * step >= inf.vhi) continue;
      const int key = key0 + i * step;
      const int page = pages.get(tbl, key / a.page_size, n_slots, lane);
      if (page < 0 || (long long)page >= a.num_pages)
        inf.bad |= whole ? 0xFu : 1u << i;
      else
        ys[i] = page * a.page_size + key % a.page_size;
    }
  }

  __device__ bool wait(int slot, uint32_t parity) {
    return tc2::warp_wait(bars + slot, parity, abort_flag, a.status);
  }

  __device__ void run() {
    for (int j = 0; j < pl.n; ++j) {
      const int st = j % L::kStages;
      if (j >= L::kStages &&
          !wait((kV ? L::kEmptyV : L::kEmptyK) + st, ((j / L::kStages) - 1) & 1))
        return;
      int ys[kBoxes];
      TileInfo inf;
      find(j, ys, inf);
      issued = j + 1;
      if (kV)
        load_v(j, st, ys, inf);
      else
        load_k(j, st, ys, inf);
    }
  }

  // Wait (bounded) for the last copies into each stage, of both CTAs (their count is the even CTA's).
  __device__ void drain() {
    if (rank != 0) return;
    for (int j = max(0, issued - L::kStages); j < issued; ++j)
      mbar_wait(bars + (kV ? L::kFullV : L::kFullK) + j % L::kStages, (j / L::kStages) & 1);
  }

  __device__ void load_k(int j, int st, const int (&ys)[kBoxes], const TileInfo &inf) {
    const uint32_t dst = smem_u32(sm + L::kOffK + st * L::kKBytes);
    const uint32_t bar = tc2::map_to(smem_u32(bars + L::kFullK + st), 0);
    if (elect_one()) {
      if (inf.bad && rank == 0) raise_fault(a.status, PSKV_FAULT_BAD_PAGE);
      TileInfo &t = *reinterpret_cast<TileInfo *>(sm + L::kOffInfo + (j % kInfo) * 16);
      t.vhi = inf.vhi;
      t.bad = inf.bad;
      mbar_arrive(bars + L::kInfoFull + j % kInfo);
      if (whole) {
        // both CTAs' 32 rows, whatever of them lies behind the row's end (inside the page)
        if (rank == 0) mbar_arrive_expect_tx(bars + L::kFullK + st, ys[0] < 0 ? 0 : 2 * L::kKBytes);
        if (ys[0] >= 0) tc2::tma_load_3d(dst, map, 0, ys[0] + kHalfKeys * (int)rank, 0, bar);
      } else {
        int loaded = 0;
#pragma unroll
        for (int i = 0; i < kBoxes; ++i) loaded += ys[i] >= 0;
        if (rank == 0) mbar_arrive_expect_tx(bars + L::kFullK + st, loaded * L::kSlabs * 16 * 128);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int y = rank == 0 ? ys[i] : ys[i + 2];
          if (y < 0) continue;
          for (int s = 0; s < L::kSlabs; ++s)
            tc2::tma_load_3d(dst + s * L::kKSlab + i * 16 * 128, map, 0, y, s, bar);
        }
      }
    }
    __syncwarp();
    if (whole && j + kAhead < pl.n) {  // the same share of a later tile into L2
      const int key = (pl.t0 + j + kAhead) * kKeys;
      const int page = pages.get(a.page_tables + (size_t)pl.b * a.table_stride, key / a.page_size,
                                 n_slots, lane);
      if (page >= 0 && (long long)page < a.num_pages && elect_one())
        tc2::tma_prefetch_3d(map, 0, page * a.page_size + key % a.page_size + kHalfKeys * (int)rank, 0);
      __syncwarp();
    }
  }

  // Value slab s of this CTA: columns of block s / 2, 128 rank + 64 (s % 2).
  __device__ int slab_of(int s) { return 4 * (s >> 1) + 2 * (int)rank + (s & 1); }

  __device__ void load_v(int j, int st, const int (&ys)[kBoxes], const TileInfo &inf) {
    unsigned char *stage = sm + L::kOffV + st * L::kVBytes;
    const uint32_t dst = smem_u32(stage);
    const uint32_t full = tc2::map_to(smem_u32(bars + L::kFullV + st), 0);
    const bool plain = inf.vhi == kKeys && inf.bad == 0;
    int loaded = 0;
#pragma unroll
    for (int i = 0; i < kBoxes; ++i) loaded += ys[i] >= 0;
    const uint32_t bytes = (uint32_t)(loaded * (whole ? kKeys : 16) * 128 * L::kVSlabs);
    // a tile with rows that must not be met lands on a barrier of this CTA first
    const uint32_t bar = plain ? full : smem_u32(bars + L::kRagged);
    if (elect_one()) {
      if (plain) {
        if (rank == 0) mbar_arrive_expect_tx(bars + L::kFullV + st, 2 * bytes);
      } else {
        mbar_arrive_expect_tx(bars + L::kRagged, bytes);
      }
      if (whole) {
        if (ys[0] >= 0)
#pragma unroll
          for (int k = 0; k < L::kBlocks; ++k)
            tc2::tma_load_3d(dst + 2 * k * L::kVSlab, map, 0, ys[0], 4 * k + 2 * (int)rank, bar);
      } else {
#pragma unroll
        for (int i = 0; i < kBoxes; ++i)
          if (ys[i] >= 0)
            for (int s = 0; s < L::kVSlabs; ++s)
              tc2::tma_load_3d(dst + s * L::kVSlab + i * 16 * 128, map, 0, ys[i], slab_of(s), bar);
      }
    }
    __syncwarp();
    if (!plain) {
      // rows behind the end or of skipped groups may hold anything and meet P = 0: zero them
      mbar_wait(bars + L::kRagged, ragged & 1);  // (bounded; landed or given up on, the tile is passed on)
      ++ragged;
      for (int e = lane; e < kKeys * L::kVSlabs * 8; e += 32) {
        const int row = e & (kKeys - 1), piece = e >> 6;
        if (row >= inf.vhi || ((inf.bad >> (row >> 4)) & 1u))
          *reinterpret_cast<uint4 *>(stage + (piece >> 3) * L::kVSlab + row * 128 +
                                     (piece & 7) * 16) = make_uint4(0, 0, 0, 0);
      }
      tc::fence_smem_for_async();
      __syncwarp();
    }
    if (lane == 0) tc2::arrive_cluster(full);
    if (!plain && rank == 0 && lane == 0) mbar_arrive(bars + L::kFullV + st);  // in place of the copies' count
  }
};

}  // namespace

template <int DC, bool kLo>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    pskv_attn_latent(const LatentAttnArgs a, const __grid_constant__ Maps maps) {
  using L = Lay<DC, kLo>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *sm = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::kOffBar);
  uint32_t *slot = reinterpret_cast<uint32_t *>(sm + L::kOffSlot);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + L::kOffAbort);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc2::cluster_rank();

  pdl_wait();
  pdl_launch_dependents();
  const Plan pl = make_plan(a);
  if (!pl.ok && threadIdx.x == 0 && blockIdx.x == 0) raise_fault(a.status, PSKV_FAULT_BAD_LENGTH);
  const int w = warp & 3, i = (32 * w + lane) & (kRows - 1), kh = w >> 1;  // softmax thread: row, half
  const int col = pl.cb * 128 + (int)rank * kRows + i;
  const size_t row = (size_t)pl.b * pl.cols + col, part = row * a.num_splits + pl.p;
  if (pl.n <= 0) {  // (both CTAs leave here together) the empty state, or zeros
    if (warp < 2 || warp > 5 || col >= pl.cols) return;
    if (a.direct) {
      if (pl.len > 0 && kh == 0) raise_fault(a.status, PSKV_FAULT_EMPTY_ROW);
      const int es = a.out_dtype == PSKV_DTYPE_BF16 ? 2 : 4;
      uint4 *dst = reinterpret_cast<uint4 *>(static_cast<char *>(a.out) + row * DC * es);
      for (int e = kh; e < DC * es / 16; e += 2) dst[e] = make_uint4(0, 0, 0, 0);
    } else if (kh == 0) {
      a.ws_m[part] = -CUDART_INF_F;
      a.ws_l[part] = 0.f;
    }
    return;
  }

  if (warp == 1) {
    if (lane == 0) {
      for (int s = 0; s < L::kStages; ++s) {
        mbar_init(&bars[L::kFullK + s], 1);
        mbar_init(&bars[L::kFullV + s], 3);  // the expected bytes, and a word from either V copy warp
        mbar_init(&bars[L::kEmptyK + s], 1);
        mbar_init(&bars[L::kEmptyV + s], 1);
      }
      for (int r = 0; r < 2; ++r) {
        mbar_init(&bars[L::kSFull + r], 1);
        mbar_init(&bars[L::kSFree + r], 8);  // four softmax warps in each CTA
        mbar_init(&bars[L::kPFull + r], 8);
        mbar_init(&bars[L::kPvDone + r], 1);
      }
      for (int k = 0; k < kInfo; ++k) mbar_init(&bars[L::kInfoFull + k], 1);
      mbar_init(&bars[L::kQFull], 1);
      mbar_init(&bars[L::kRagged], 1);
      mbar_init(&bars[L::kDrainS], 1);
      mbar_init(&bars[L::kDrainV], 1);
      *abort_flag = 0;
      mbar_fence_init();
    }
    __syncwarp();
  } else if (warp == 0) {
    tc2::alloc(slot, kTmemCols);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc2::cluster_sync();  // both CTAs' barriers are set up
  tc::fence_after_sync();
  const uint32_t tmem = *slot;
  auto wait = [&](int s, uint32_t parity) {
    return tc2::warp_wait(bars + s, parity, abort_flag, a.status);
  };

  if (warp == 0 && rank == 0) {
    // ---- the score products
    bool ok = wait(L::kQFull, 0);
    const uint32_t q0 = smem_u32(sm + L::kOffQ);
    for (int j = 0; ok && j < pl.n; ++j) {
      const int st = j % L::kStages, r = j & 1;
      ok = wait(L::kFullK + st, (j / L::kStages) & 1) &&
           (j < 2 || wait(L::kSFree + r, ((j - 2) >> 1) & 1));
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t k0 = smem_u32(sm + L::kOffK + st * L::kKBytes);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4 * L::kSlabs; ++kk)
          tc2::mma(tmem + kSCol + kHalfKeys * r,
                   tc::smem_desc(q0 + (kk >> 2) * L::kQSlab + (kk & 3) * 32, 16, 1024),
                   tc::smem_desc(k0 + (kk >> 2) * L::kKSlab + (kk & 3) * 32, 16, 1024), L::kIdescS,
                   kk > 0);
        tc2::commit_both(bars + L::kSFull + r);
        tc2::commit_both(bars + L::kEmptyK + st);
      }
      __syncwarp();
    }
    if (elect_one()) tc2::commit_both(bars + L::kDrainS);
    __syncwarp();
  } else if (warp == 7 && rank == 0) {
    // ---- the value products
    bool ok = true;
    for (int j = 0; ok && j < pl.n; ++j) {
      const int st = j % L::kStages, pb = j % L::kPBufs;
      ok = wait(L::kPFull + pb, (j / L::kPBufs) & 1) && wait(L::kFullV + st, (j / L::kStages) & 1);
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t v0 = smem_u32(sm + L::kOffV + st * L::kVBytes);
      const uint32_t p0 = smem_u32(sm + L::kOffP + pb * L::kPBytes);
      if (elect_one()) {
#pragma unroll
        for (int nb = 0; nb < L::kBlocks; ++nb)
#pragma unroll
          for (int part_ = 0; part_ < (kLo ? 2 : 1); ++part_)
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              tc2::mma(tmem + kOCol + 128 * nb,
                       tc::smem_desc(p0 + part_ * L::kPBytes + kk * 32, 16, 1024),
                       tc::smem_desc(v0 + 2 * nb * L::kVSlab + kk * 2048, L::kVSlab, 1024),
                       L::kIdescPV, j > 0 || part_ > 0 || kk > 0);
        tc2::commit_both(bars + L::kPvDone + pb);
        tc2::commit_both(bars + L::kEmptyV + st);
      }
      __syncwarp();
    }
    if (elect_one()) tc2::commit_both(bars + L::kDrainV);
    __syncwarp();
  } else if (warp == 1) {
    // ---- Q (this CTA's 64 columns; behind the row's last column: other rows' or zeros), then K
    if (elect_one()) {
      if (rank == 0) mbar_arrive_expect_tx(bars + L::kQFull, 2 * L::kQBytes);
      tc2::tma_load_3d(smem_u32(sm + L::kOffQ), &maps.q, 0,
                       pl.b * pl.cols + pl.cb * 128 + (int)rank * kRows, 0,
                       tc2::map_to(smem_u32(bars + L::kQFull), 0));
    }
    __syncwarp();
    Loader<DC, kLo, false> ld(a, pl, &maps.k, sm, bars, abort_flag, rank);
    ld.run();
    ld.drain();
    if (rank == 0) mbar_wait(bars + L::kQFull, 0);
  } else if (warp == 6) {
    Loader<DC, kLo, true> ld(a, pl, &maps.v, sm, bars, abort_flag, rank);
    ld.run();
    ld.drain();
  } else if (warp >= 2 && warp <= 5) {
    // ---- the softmax: thread (row i, keys 32 kh .. + 31 of the tile).  The loop never
    // leaves early (the two warps of a row's halves meet every tile); after a failed wait its
    // results are not written.
    const uint32_t lane_base = tmem + ((uint32_t)(32 * w) << 16);
    float *red = reinterpret_cast<float *>(sm + L::kOffRed);
    const int t = col / a.num_q_heads;
    const int lim = col < pl.cols ? pl.len - a.num_tokens + t + 1 : 0;  // keys below lim are seen
    const float sc = a.scale_log2;
    const uint32_t s_free = tc2::map_to(smem_u32(bars + L::kSFree), 0);
    const uint32_t p_full = tc2::map_to(smem_u32(bars + L::kPFull), 0);
    float m = -CUDART_INF_F, l = 0.f;
    bool ok = true;
    for (int j = 0; j < pl.n; ++j) {
      const int r = j & 1, pb = j % L::kPBufs;
      ok = ok && wait(L::kSFull + r, (j >> 1) & 1);
      ok = ok && wait(L::kInfoFull + j % kInfo, (j / kInfo) & 1);
      const TileInfo inf = *reinterpret_cast<const TileInfo *>(sm + L::kOffInfo + (j % kInfo) * 16);
      tc::fence_after_sync();
      uint32_t v[32];
      tc::ld32(lane_base + kSCol + kHalfKeys * r, v);
      tc::wait_ld();
      tc::reg_fence(v);
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc2::arrive_cluster(s_free + 8 * r);
      const int key0 = (pl.t0 + j) * kKeys + kHalfKeys * kh;
      float x[32];
#pragma unroll
      for (int c = 0; c < 32; ++c) x[c] = __uint_as_float(v[c]) * sc;
      if (key0 + 32 > lim || inf.bad != 0) {  // (by selection: rows never loaded may hold anything)
        const uint32_t bad = inf.bad >> (2 * kh);
#pragma unroll
        for (int c = 0; c < 32; ++c)
          x[c] = key0 + c < lim && !((bad >> (c >> 4)) & 1u) ? x[c] : -CUDART_INF_F;
      }
      float mt = x[0];
#pragma unroll
      for (int c = 1; c < 32; ++c) mt = fmaxf(mt, x[c]);
      float *mine = red + (j & 1) * 2 * kRows;
      mine[kh * kRows + i] = mt;
      asm volatile("bar.sync %0, 64;" ::"r"(1 + (w & 1)) : "memory");
      mt = fmaxf(mt, mine[(kh ^ 1) * kRows + i]);
      float alpha = 1.f;
      bool rescale = false;
      if (mt > m + kSlack) {
        rescale = m != -CUDART_INF_F;  // with m = -inf the row's O and l are still 0
        alpha = rescale ? ex2(m - mt) : 1.f;
        l *= alpha;
        m = mt;
      }
      const float u = m == -CUDART_INF_F ? 0.f : m;
      uint32_t hi[16], lo[16];
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float p0 = ex2(x[2 * e] - u), p1 = ex2(x[2 * e + 1] - u);
        hi[e] = pack_bf16x2(p0, p1);
        if (kLo) {
          lo[e] = pack_bf16x2(p0 - bf16_lo(hi[e]), p1 - bf16_hi(hi[e]));
          sum += p0 + p1;
        } else {
          sum += bf16_lo(hi[e]) + bf16_hi(hi[e]);
        }
      }
      l += sum;
      // the P buffer is free once the values of tile j - kPBufs are done
      if (j >= L::kPBufs) ok = ok && wait(L::kPvDone + pb, (j / L::kPBufs - 1) & 1);
      unsigned char *prow = sm + L::kOffP + pb * L::kPBytes + i * 128;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int at = ((4 * kh + c) ^ (i & 7)) << 4;
        *reinterpret_cast<uint4 *>(prow + at) =
            make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
        if (kLo)
          *reinterpret_cast<uint4 *>(prow + L::kPBytes + at) =
              make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
      }
      if (__any_sync(0xffffffffu, rescale)) {
        ok = ok && wait(L::kPvDone + (j - 1) % L::kPBufs, ((j - 1) / L::kPBufs) & 1);
        tc::fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < DC / 64; ++c) {
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
      if (lane == 0) tc2::arrive_cluster(p_full + 8 * pb);
    }
    // ---- the row's sum over both halves, and its columns: 128 kh + [0, 128) of every 256
    float *sums = red + (pl.n & 1) * 2 * kRows;
    sums[kh * kRows + i] = l;
    asm volatile("bar.sync %0, 64;" ::"r"(1 + (w & 1)) : "memory");
    l = sums[i] + sums[kRows + i];
    ok = ok && wait(L::kPvDone + (pl.n - 1) % L::kPBufs, ((pl.n - 1) / L::kPBufs) & 1);
    if (ok) {
      tc::fence_after_sync();
      const bool real = col < pl.cols, empty = m == -CUDART_INF_F;
      const float inv = empty ? 0.f : 1.f / l;
      const uint64_t keep = make_evict_last_policy();
#pragma unroll 1
      for (int c = 0; c < DC / 64; ++c) {
        uint32_t o[32];
        tc::ld32(lane_base + kOCol + 32 * c, o);
        tc::wait_ld();
        tc::reg_fence(o);
        if (!real) continue;
        const int d = 256 * (c >> 2) + 128 * kh + 32 * (c & 3);
        if (!a.direct) {
          float4 *dst = reinterpret_cast<float4 *>(a.ws_o + part * DC + d);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            st_keep(dst + q,
                    make_float4(__uint_as_float(o[4 * q]), __uint_as_float(o[4 * q + 1]),
                                __uint_as_float(o[4 * q + 2]), __uint_as_float(o[4 * q + 3])),
                    keep);
        } else if (a.out_dtype == PSKV_DTYPE_BF16) {
          uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + row * DC + d);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[e] = empty ? 0u
                           : pack_bf16x2(__uint_as_float(o[8 * q + 2 * e]) * inv,
                                         __uint_as_float(o[8 * q + 2 * e + 1]) * inv);
            dst[q] = make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else {
          float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + row * DC + d);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            dst[q] = empty ? make_float4(0.f, 0.f, 0.f, 0.f)
                           : make_float4(__uint_as_float(o[4 * q]) * inv,
                                         __uint_as_float(o[4 * q + 1]) * inv,
                                         __uint_as_float(o[4 * q + 2]) * inv,
                                         __uint_as_float(o[4 * q + 3]) * inv);
        }
      }
      if (real && kh == 0) {
        if (a.direct) {
          if (empty) raise_fault(a.status, PSKV_FAULT_EMPTY_ROW);
        } else {
          a.ws_m[part] = empty ? -CUDART_INF_F : m * kLn2;
          a.ws_l[part] = l;
        }
      }
    }
  }
  // every product done (both CTAs learn it; every copy has landed) before the memory is released
  if (warp == 0) mbar_wait(bars + L::kDrainS, 0);
  if (warp == 7) mbar_wait(bars + L::kDrainV, 0);
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc2::cluster_sync();
  if (warp == 0) {
    tc::fence_after_sync();
    tc2::dealloc(tmem, kTmemCols);
  }
}

namespace {

template <int DC, bool kLo>
cudaError_t launch(const LatentAttnArgs &a, cudaStream_t s) {
  using L = Lay<DC, kLo>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(dev >= 0 && dev < 64 && attr_set[dev])) {
    e = cudaFuncSetAttribute(pskv_attn_latent<DC, kLo>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             L::kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const bool whole = a.page_size % kKeys == 0;
  const long long cols = (long long)a.num_tokens * a.num_q_heads;
  Maps maps;
  if (!tc2::make_slab_map(&maps.q, a.q, a.batch * cols, DC + 64, kRows, L::kSlabs) ||
      !tc2::make_slab_map(&maps.k, a.pool, a.num_pages * a.page_size, DC + 64,
                          whole ? kHalfKeys : 16, whole ? L::kSlabs : 1) ||
      !tc2::make_slab_map(&maps.v, a.pool, a.num_pages * a.page_size, DC + 64, whole ? kKeys : 16,
                          whole ? 2 : 1))
    return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(2 * ((cols + 127) / 128) * a.num_splits), a.batch);
  return launch_pdl(pskv_attn_latent<DC, kLo>, grid, dim3(kThreads), L::kSmemBytes, s, a, maps);
}

}  // namespace

cudaError_t launch_attn_latent(const LatentAttnArgs &a, int dc, cudaStream_t s) {
  const bool lo = a.out_dtype == PSKV_DTYPE_F32;
  if (dc == 512) return lo ? launch<512, true>(a, s) : launch<512, false>(a, s);
  if (dc == 256) return lo ? launch<256, true>(a, s) : launch<256, false>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace pskv
