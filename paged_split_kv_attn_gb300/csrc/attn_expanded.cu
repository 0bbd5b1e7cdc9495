// attn_expanded.cu -- expanded latent attention of variable-length chunks on pairs
// of CTAs.
//
// Per row, head h and query i: s_ij = scale * (qn_i . kn_j + qr_i . r_j) over the keys
// j up to the query's own, o_i = sum_j softmax(s_i)_j v_j; 192 score columns (the rotated
// 64 shared by all heads) and 128 value columns.  2 * (192 + 128) operations a (query, key)
// pair and head: compute-bound from a few hundred tokens on.
//
// A cluster of two CTAs takes 256 queries of one head, CTA r queries 128 r .. + 127, as
// tcgen05 products of M = 256 over the pair (cta_group::2), and walks the keys in tiles of 128:
//   S = Q K^T   CTA r brings keys 64 r .. + 63 (12 products of K = 16)
//   O += P V    CTA r brings value columns 64 r .. + 63 (8 products), P from tensor memory
// so a tile is copied once for 256 queries, half by each CTA (40 KB a CTA), and each CTA's
// tensor memory has room for two score regions beside P and its own O:
// S [0, 256), P [256, 384) (two of bf16 pairs; f32 output: one hi and one lo), O [384, 512).
// S(j + 1) runs while the softmax works on tile j.  (One CTA with two blocks of 128 queries has no
// room for that: sharing one score region between the blocks took 5,500 cycles for the same
// 2 * 256 * 128 pairs that two tiles take 3,150 for.)
//
// Resident clusters take one block of queries after another: while a block runs, the next is asked
// for (cluster launch control), and its first copies and scores run behind the last softmax.
// Launching a cluster a block cost 8,500 cycles a block (one prompt of 4,096 tokens and 32 heads:
// 138.7 us against 120.8).  Up to 32 rows the longest blocks are given out first.
//
// A query's 128 scores lie in two threads, which mask them and exchange their maxima; the reference
// maximum moves only past a slack of 8 (log2 units), so O is rarely rescaled.
//
// Per tile the tensor pipe works (12 + 8) * 64 = 1,280 cycles, and the softmax takes 1,500: 512
// of the special-function unit (4 cycles a warp's exponent), as many of single-issue
// operations, and the latencies of the barriers between them.  Measured for that prompt: 113.4 us
// replayed back to back (1.51 PFLOP/s), 126.5 as one call among others (1.36); of 117.8 before the
// last step 103 were left without the exponents and 108 with a third of the score products.
// Other splits of the softmax were no faster: four threads a query 120.6, one thread with
// the next tile's scores in flight 131, two warps on alternate tiles 133 us.
//
// P is rounded to bf16 when the output is (it adds about what the output's own
// rounding does; f32 output: a bf16 pair), everything else is f32.  Every wait is bounded; on
// expiry the CTA flags PSKV_FAULT_WAIT_TIMEOUT, lets what it issued finish and
// frees its tensor memory.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math_constants.h>

#include <atomic>

#include "latent.h"
#include "pskv_internal.cuh"
#include "tc_common.cuh"
#include "tc_ops.cuh"
#include "tc_pair.cuh"

namespace pskv {

namespace {

using tc::elect_one;
using tc::ex2;

constexpr int kRows = 128;             // queries per CTA
constexpr int kKeys = 128;             // keys per tile
constexpr int kHalf = 64;              // of which each CTA brings half to the scores
constexpr int kQSlabs = 3;             // 64-column slabs of a query or key
constexpr int kDv = PSKV_EXPANDED_V;
constexpr int kQSlab = kRows * 128;    // 16 KB
constexpr int kKSlab = kHalf * 128;    // 8 KB
constexpr int kQBytes = kQSlabs * kQSlab, kKBytes = kQSlabs * kKSlab;
constexpr int kVBytes = kKeys * 128;   // this CTA's 64 value columns
constexpr int kRing = 4;               // tiles in flight, of K and of V
constexpr int kSplit = 2;              // softmax threads of a query
constexpr int kSoftWarps = 4 * kSplit;
constexpr int kCols = kKeys / kSplit;  // scores (and output columns) a thread
constexpr int kScores = kSoftWarps, kValues = kScores + 1, kKeyCopies = kScores + 2, kValueCopies = kScores + 3;
constexpr int kThreads = 32 * (kSoftWarps + 4);
constexpr int kTmemCols = 512;
constexpr float kSlack = 8.f;
constexpr int kSCol = 0, kPCol = 256, kOCol = 384;

constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + kQBytes;
constexpr int kOffV = kOffK + kRing * kKBytes;
constexpr int kOffBar = kOffV + kRing * kVBytes;
enum : int {
  kFullK = 0,                // [4] (even CTA) both CTAs' K landed
  kFullV = kFullK + kRing,   // [4] (even CTA) both CTAs' V landed
  kEmptyK = kFullV + kRing,  // [4] the tile's scores done
  kEmptyV = kEmptyK + kRing,  // [4] the tile's values done
  kQFull = kEmptyV + kRing,  // (even CTA) both CTAs' queries landed
  kQFree = kQFull + 1,       // the block's scores done
  kSFull = kQFree + 1,       // [2] scores of region r in
  kSFree = kSFull + 2,       // [2] (even CTA) region r read in both CTAs
  kPFull = kSFree + 2,       // [2] (even CTA) P written in both CTAs
  kPvDone = kPFull + 2,      // [2] the values of P's tile done
  kRagged = kPvDone + 2,     // this CTA's V of the tile with the row's end
  kWorkFull = kRagged + 1,   // [2] the block's numbers written
  kWorkFree = kWorkFull + 2,  // [2] and read by all warps
  kReply = kWorkFree + 2,    // the answer to a request for a block landed
  kReplyRead = kReply + 1,   // (even CTA) and was read in both CTAs
  kDrainS = kReplyRead + 1,  // all products done
  kDrainV = kDrainS + 1,
  kNumBars = kDrainV + 1
};
constexpr int kOffWork = (kOffBar + kNumBars * 8 + 15) & ~15;  // Work[2]
constexpr int kOffReply = kOffWork + 2 * 32;                   // 16 bytes
constexpr int kOffRed = kOffReply + 16;        // float[2][kSplit][128] maxima (then sums)
constexpr int kOffSlot = kOffRed + 2 * kSplit * kRows * 4;
constexpr int kOffAbort = kOffSlot + 4;
constexpr int kUsed = kOffAbort + 4;
// the launch asks for what there is of the 1,023 bytes that the base's alignment could take
constexpr int kSmemBytes = kUsed + 1024 < 232448 ? kUsed + 1024 : 232448;
static_assert(kUsed <= 232448, "shared memory per CTA");
constexpr int kReaders = 3 + kSoftWarps;  // warps that read a block's numbers

constexpr uint32_t kIdescS = tc::instr_desc(2 * kRows, kKeys, false, false);
constexpr uint32_t kIdescPV = tc::instr_desc(2 * kRows, kDv, false, true);

struct Maps {
  CUtensorMap q, k, v, rot;
};

// A block of 2 * kRows queries of one head, as its CTAs' warps take it up.
struct __align__(16) Work {
  int q0, k0, nq, nk;  // the row's first query and key, its queries and keys
  int h, t0, n, more;  // head, the block's first query in the row, tiles (0: nothing to do); 0: the end
};
static_assert(sizeof(Work) == 32, "two 16-byte words");

// The rows' blocks in the order in which they are given out (whole warp).  Up to 32 rows, a lane
// each: by their number of tiles, the longest first, so that the last to run are short (block
// c of a row has before / 256 + c pairs of tiles, its level; the k-th block's level is found
// by bisection over the count of blocks above).  More rows: one after the other, each
// from its last block on (six ragged chunks of 332 to 517 queries: 51.7 us against 45.2).
struct Blocks {
  int base = 0;       // first row held
  int skipped = 0;    // blocks of the rows before
  int q0, k0, nq, nk, blocks, level;
  bool bad = false;

  __device__ void load(const ExpandedAttnArgs &a, int first, int lane) {
    base = first;
    q0 = k0 = nq = nk = blocks = level = 0;
    bad = false;
    const int b = first + lane;
    if (b >= a.batch) return;
    const int qa = a.cu_q[b], qb = a.cu_q[b + 1], ka = a.cu_k[b], kb = a.cu_k[b + 1];
    bad = qa < 0 || qb < qa || qb > a.total_q || ka < 0 || kb < ka || kb > a.total_k ||
          kb - ka < qb - qa;
    if (bad) return;  // (the row is left out)
    q0 = qa;
    k0 = ka;
    nq = qb - qa;
    nk = kb - ka;
    blocks = (nq + 2 * kRows - 1) / (2 * kRows);
    level = (nk - nq) / (2 * kRows);
  }
  __device__ int held() const { return (int)__reduce_add_sync(0xffffffffu, (uint32_t)blocks); }

  // Block number k's row as a lane, and its first query in the row; -1: there is none.
  __device__ int find(const ExpandedAttnArgs &a, int k, int lane, int &t0) {
    int row, c;
    if (a.batch <= 32) {
      int lo = 0, hi = (int)__reduce_max_sync(0xffffffffu, (uint32_t)(blocks ? level + blocks : 0));
      auto above = [&](int l) {  // blocks of level l and more
        return (int)__reduce_add_sync(0xffffffffu, (uint32_t)min(blocks, max(0, level + blocks - l)));
      };
      if (k >= held()) return -1;
      while (hi - lo > 1) {  // above(lo) > k >= above(hi)
        const int mid = (lo + hi) >> 1;
        if (above(mid) > k)
          lo = mid;
        else
          hi = mid;
      }
      const int left = k - above(hi);
      const bool in = level <= lo && lo < level + blocks;
      const uint32_t rows = __ballot_sync(0xffffffffu, in);
      row = __ffs(__ballot_sync(0xffffffffu, in && __popc(rows & ((1u << lane) - 1)) == left)) - 1;
      c = lo - __shfl_sync(0xffffffffu, level, row);
    } else {
      if (k < skipped) {
        skipped = 0;
        load(a, 0, lane);
      }
      int sum = held();
      while (k - skipped >= sum) {
        if (base + 32 >= a.batch) return -1;
        skipped += sum;
        load(a, base + 32, lane);
        sum = held();
      }
      int incl = blocks;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
      }
      row = __ffs(__ballot_sync(0xffffffffu, incl > k - skipped)) - 1;
      c = __shfl_sync(0xffffffffu, incl, row) - 1 - (k - skipped);
    }
    t0 = c * 2 * kRows;
    return row;
  }
};

// Whether any thread of a query's warps says so, told to all of them (named barrier `id`).
__device__ __forceinline__ bool any_of(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %3, 0;\n\t"
      "barrier.cta.red.or.aligned.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "n"(32 * kSplit), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

// Lane i of four neighbours has piece k of row i in y[k] and gets piece i of row k.
__device__ __forceinline__ void transpose4(uint32_t (&y)[4][4], int lane) {
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    const bool upper = lane & d;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (!(k & d))
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t give = upper ? y[k][e] : y[k + d][e];
          const uint32_t got = __shfl_xor_sync(0xffffffffu, give, d);
          if (upper)
            y[k][e] = got;
          else
            y[k + d][e] = got;
        }
  }
}

// Ask for a cluster of the grid that has not started, in both CTAs' shared memory, counted
// on both's barriers (one thread of the pair).
__device__ __forceinline__ void ask_for_cluster(uint32_t reply, uint32_t bar, bool lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes"
      ".multicast::cluster::all.b128 [%0], [%1];\n\t}" ::"r"(reply),
      "r"(bar), "r"((uint32_t)lead)
      : "memory");
}
// The answer: that cluster's first blockIdx.x, or -1 when none is left.
__device__ __forceinline__ int cluster_given(uint32_t reply) {
  uint32_t x, got;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %1, 1, 0, p;\n\tmov.u32 %0, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}"
      : "=&r"(x), "=&r"(got)
      : "r"(reply)
      : "memory");
  return got ? (int)x : -1;
}

}  // namespace

template <bool kLo>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    pskv_attn_expanded(const ExpandedAttnArgs a, const __grid_constant__ Maps maps) {
  constexpr int kPBufs = kLo ? 1 : 2;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *sm = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  if (sm + kUsed > smem_raw + kSmemBytes) {  // (never seen) no room for the alignment
    if (threadIdx.x == 0) raise_fault(a.status, PSKV_FAULT_WAIT_TIMEOUT);
    return;
  }
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + kOffBar);
  uint32_t *slot = reinterpret_cast<uint32_t *>(sm + kOffSlot);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + kOffAbort);
  const int warp = tc2::uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rank = tc2::cluster_rank();
  const bool lead = elect_one();  // one thread of each warp
  if (warp == kKeyCopies) {
    if (lane == 0) {
      for (int s = 0; s < kRing; ++s) {
        mbar_init(&bars[kFullK + s], 1);
        mbar_init(&bars[kFullV + s], 3);  // the expected bytes, and a word from either V copy warp
        mbar_init(&bars[kEmptyK + s], 1);
        mbar_init(&bars[kEmptyV + s], 1);
      }
      mbar_init(&bars[kQFull], 1);
      mbar_init(&bars[kQFree], 1);
      for (int r = 0; r < 2; ++r) {
        mbar_init(&bars[kSFull + r], 1);
        mbar_init(&bars[kSFree + r], 2 * kSoftWarps);
        mbar_init(&bars[kPFull + r], 2 * kSoftWarps);
        mbar_init(&bars[kPvDone + r], 1);
        mbar_init(&bars[kWorkFull + r], 1);
        mbar_init(&bars[kWorkFree + r], kReaders);
      }
      mbar_init(&bars[kReply], 1);
      mbar_init(&bars[kReplyRead], 2);
      mbar_init(&bars[kRagged], 1);
      mbar_init(&bars[kDrainS], 1);
      mbar_init(&bars[kDrainV], 1);
      *abort_flag = 0;
      mbar_fence_init();
    }
    __syncwarp();
    tc2::prefetch_map(&maps.q);
    tc2::prefetch_map(&maps.k);
    tc2::prefetch_map(&maps.rot);
  } else if (warp == kScores) {
    tc2::alloc(slot, kTmemCols);
  }
  pdl_wait();
  pdl_launch_dependents();
  Blocks rows;
  if (warp == kKeyCopies) {
    rows.load(a, 0, lane);
    if (blockIdx.x == 0) {
      // offsets that the host copies do not allow: those rows, or the blocks past the grid's, are
      // left out
      bool bad = __any_sync(0xffffffffu, rows.bad);
      long long blocks = rows.held();
      for (int b = 32; b < a.batch; b += 32) {
        rows.load(a, b, lane);
        bad = bad || __any_sync(0xffffffffu, rows.bad);
        blocks += rows.held();
      }
      if ((bad || blocks > gridDim.x / (2 * a.num_heads)) && lead) raise_fault(a.status, PSKV_FAULT_BAD_LENGTH);
      if (a.batch > 32) rows.load(a, 0, lane);
    }
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
  // The numbers of this CTA's block number i; false: a wait failed.
  Work *works = reinterpret_cast<Work *>(sm + kOffWork);
  auto next = [&](int i, Work &w) {
    const int s = i & 1;
    if (!wait(kWorkFull + s, (i >> 1) & 1)) return false;
    const int4 x = reinterpret_cast<const int4 *>(works + s)[0];
    const int4 y = reinterpret_cast<const int4 *>(works + s)[1];
    __syncwarp();
    if (lead) mbar_arrive(bars + kWorkFree + s);
    w = Work{x.x, x.y, x.z, x.w, y.x, y.y, tc2::uniform(y.z), tc2::uniform(y.w)};
    return true;
  };

  // g counts a CTA's tiles over all its blocks: rings, regions and parities go by it
  if (warp >= kSoftWarps) {
    if (warp == kScores) {
      // ---- the score products (all lanes alike, one of the even CTA's issues)
      bool ok = true;
      const uint32_t q = smem_u32(sm + kOffQ), k = smem_u32(sm + kOffK);
      Work w;
      for (int i = 0, g = 0, nb = 0; ok; ++i) {
        ok = next(i, w);
        if (!ok || !w.more) break;
        if (rank != 0 || w.n == 0) continue;
        ok = wait_pair(kQFull, nb++ & 1);
        for (int j = 0; ok && j < w.n; ++j, ++g) {
          const int st = g % kRing, r = g & 1;
          ok = wait_pair(kFullK + st, (g / kRing) & 1) && (g < 2 || wait_pair(kSFree + r, (g / 2 - 1) & 1));
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t kt = k + st * kKBytes;
#pragma unroll
          for (int kk = 0; kk < 4 * kQSlabs; ++kk)
            tc2::mma(tmem + kSCol + kKeys * r,
                     tc::smem_desc(q + (kk >> 2) * kQSlab + (kk & 3) * 32, 16, 1024),
                     tc::smem_desc(kt + (kk >> 2) * kKSlab + (kk & 3) * 32, 16, 1024), kIdescS, kk > 0,
                     lead);
          tc2::commit_both(bars + kSFull + r, lead);
          tc2::commit_both(bars + kEmptyK + st, lead);
        }
        tc2::commit_both(bars + kQFree, lead);
      }
      if (rank == 0) tc2::commit_both(bars + kDrainS, lead);
      __syncwarp();
    } else if (warp == kValues) {
      // ---- the value products
      bool ok = true;
      const uint32_t v = smem_u32(sm + kOffV);
      Work w;
      for (int i = 0, g = 0; ok; ++i) {
        ok = next(i, w);
        if (!ok || !w.more) break;
        if (rank != 0) continue;
        for (int j = 0; ok && j < w.n; ++j, ++g) {
          const int st = g % kRing, pb = g % kPBufs;
          ok = wait_pair(kFullV + st, (g / kRing) & 1) && wait_pair(kPFull + pb, (g / kPBufs) & 1);
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t vt = v + st * kVBytes;
#pragma unroll
          for (int part = 0; part < (kLo ? 2 : 1); ++part)
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              tc2::mma_ts(tmem + kOCol, tmem + kPCol + 64 * (pb + part) + 8 * kk,
                          tc::smem_desc(vt + kk * 2048, kVBytes, 1024), kIdescPV,
                          j > 0 || part > 0 || kk > 0, lead);
          tc2::commit_both(bars + kPvDone + (g & 1), lead);
          tc2::commit_both(bars + kEmptyV + st, lead);
        }
      }
      if (rank == 0) tc2::commit_both(bars + kDrainV, lead);
      __syncwarp();
    } else if (warp == kKeyCopies) {
      // ---- the blocks; Q (queries behind the row's last: other rows' or zeros), then K: this
      // CTA's half.  The next block is asked for when one begins and looked at behind its copies.
      const uint32_t reply = smem_u32(sm + kOffReply);
      int x = blockIdx.x, g = 0, nb = 0, i = 0;
      bool ok = true, asked = false;
      for (;; ++i) {
        Work w{};
        w.more = x >= 0;
        if (x >= 0) {
          const int pair = x >> 1;
          w.h = pair % a.num_heads;
          const int row = rows.find(a, pair / a.num_heads, lane, w.t0);
          if (row >= 0) {
            w.q0 = __shfl_sync(0xffffffffu, rows.q0, row);
            w.k0 = __shfl_sync(0xffffffffu, rows.k0, row);
            w.nq = __shfl_sync(0xffffffffu, rows.nq, row);
            w.nk = __shfl_sync(0xffffffffu, rows.nk, row);
            // tiles up to the last own key
            w.n = (w.nk - w.nq + min(w.nq, w.t0 + 2 * kRows) + kKeys - 1) / kKeys;
          }
        }
        ok = i < 2 || wait(kWorkFree + (i & 1), (i / 2 - 1) & 1);
        if (!ok) break;
        if (lane == 0) works[i & 1] = w;
        __syncwarp();
        if (lead) mbar_arrive(bars + kWorkFull + (i & 1));
        if (!w.more) break;
        if (rank == 0) {
          ok = i == 0 || wait_pair(kReplyRead, (i - 1) & 1);
          if (!ok) break;
          ask_for_cluster(reply, smem_u32(bars + kReply), lead);
        }
        tc2::expect_tx(bars + kReply, 16, lead);
        asked = true;
        if (w.n > 0) {
          ok = nb == 0 || wait(kQFree, (nb - 1) & 1);
          if (!ok) break;
          ++nb;
          tc2::expect_tx(bars + kQFull, 2 * kQBytes, lead && rank == 0);
          tc2::tma_load_3d(smem_u32(sm + kOffQ), &maps.q, 0, w.q0 + w.t0 + (int)rank * kRows, kQSlabs * w.h,
                           tc2::map_to(smem_u32(bars + kQFull), 0), lead);
        }
        for (int j = 0; j < w.n; ++j, ++g) {
          const int st = g % kRing;
          ok = g < kRing || wait(kEmptyK + st, (g / kRing - 1) & 1);
          if (!ok) break;
          const uint32_t dst = smem_u32(sm + kOffK + st * kKBytes);
          const uint32_t bar = tc2::map_to(smem_u32(bars + kFullK + st), 0);
          const int y = w.k0 + j * kKeys + kHalf * (int)rank;
          tc2::expect_tx(bars + kFullK + st, 2 * kKBytes, lead && rank == 0);
          tc2::tma_load_3d(dst, &maps.k, 0, y, 4 * w.h, bar, lead);
          tc2::tma_load_3d(dst + 2 * kKSlab, &maps.rot, 0, y, 0, bar, lead);
        }
        if (!ok) break;
        ok = wait(kReply, i & 1);
        if (!ok) break;
        asked = false;
        x = cluster_given(reply);
        __syncwarp();
        tc::fence_smem_for_async();  // read before the next answer lands
        tc2::arrive_pair_release(tc2::map_to(smem_u32(bars + kReplyRead), 0), lead);
      }
      // every copy of both CTAs landed before they leave (their count is the even CTA's)
      if (asked) mbar_wait(bars + kReply, i & 1);
      if (rank == 0) {
        for (int s = max(0, g - kRing); s < g; ++s) mbar_wait(bars + kFullK + s % kRing, (s / kRing) & 1);
        if (nb > 0) mbar_wait(bars + kQFull, (nb - 1) & 1);
      }
      __syncwarp();
    } else if (warp == kValueCopies) {
      // ---- V: this CTA's 64 columns of every tile.  The tile with the row's last key: rows
      // behind it are another row's and meet P = 0, so they are zeroed first.
      bool ok = true;
      Work w;
      int g = 0, seen = 0;
      for (int i = 0; ok; ++i) {
        ok = next(i, w);
        if (!ok || !w.more) break;
        const bool ragged = w.n * kKeys > w.nk;
        for (int j = 0; ok && j < w.n; ++j, ++g) {
          const int st = g % kRing;
          ok = g < kRing || wait(kEmptyV + st, (g / kRing - 1) & 1);
          if (!ok) break;
          const uint32_t full = tc2::map_to(smem_u32(bars + kFullV + st), 0);
          unsigned char *dst = sm + kOffV + st * kVBytes;
          const bool whole = !(ragged && j == w.n - 1);
          if (!whole)
            tc2::expect_tx(bars + kRagged, kVBytes, lead);
          else
            tc2::expect_tx(bars + kFullV + st, 2 * kVBytes, lead && rank == 0);
          tc2::tma_load_3d(smem_u32(dst), &maps.v, 0, w.k0 + j * kKeys, 4 * w.h + 2 + (int)rank,
                           whole ? full : smem_u32(bars + kRagged), lead);
          if (!whole) {
            ok = wait(kRagged, seen & 1);
            if (!ok) {
              mbar_wait(bars + kRagged, seen & 1);
              break;
            }
            ++seen;
            const int left = w.nk - j * kKeys;
            for (int e = lane; e < (kKeys - left) * 8; e += 32)
              *reinterpret_cast<uint4 *>(dst + (left + (e >> 3)) * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
            tc::fence_smem_for_async();
            __syncwarp();
            if (rank == 0 && lead) mbar_arrive(bars + kFullV + st);  // in place of the copies' count
          }
          if (whole)
            tc2::arrive_pair(full, lead);
          else
            tc2::arrive_pair_release(full, lead);
        }
      }
      __syncwarp();
      if (rank == 0)
        for (int s = max(0, g - kRing); s < g; ++s) mbar_wait(bars + kFullV + s % kRing, (s / kRing) & 1);
      __syncwarp();
    }
  } else {
    // ---- the softmax: thread (query, keys kCols part .. of the tile; at the end, as many output
    // columns).  A block's loop never leaves early (the warps of a query's threads meet every
    // tile); after a failed wait nothing is written, and all leave before the next block.
    const int w4 = warp & 3, part = warp >> 2, row = 32 * w4 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * w4) << 16);
    // scores in log2 units are mul * f; scales that are not positive are taken before the mask
    const float sc = a.scale_log2, mul = sc > 0.f ? sc : 1.f;
    float *red = reinterpret_cast<float *>(sm + kOffRed) + row;
    const uint32_t s_free = tc2::map_to(smem_u32(bars + kSFree), 0);
    const uint32_t p_full = tc2::map_to(smem_u32(bars + kPFull), 0);
    auto wait = [&](int s, uint32_t parity) {  // (one vote, not one a poll)
      if (__all_sync(0xffffffffu, mbar_wait(bars + s, parity))) return true;
      *abort_flag = 1;
      raise_fault(a.status, PSKV_FAULT_WAIT_TIMEOUT);
      return false;
    };
    auto values_done = [&](int tile) { return wait(kPvDone + (tile & 1), (tile >> 1) & 1); };
    bool ok = true;
    Work w;
    for (int i = 0, g = 0;; ++i) {
      ok = ok && next(i, w);
      if (any_of(1 + w4, !ok) || !w.more) break;
      if (w.n == 0) continue;
      const int t = w.t0 + (int)rank * kRows + row;
      // keys below lim are seen (queries behind the last, whose results go nowhere, see all: a
      // warp of theirs would mask every tile for nothing)
      const int lim = t < w.nq ? w.nk - w.nq + t + 1 : w.nk;
      const int all_see = (int)__reduce_min_sync(0xffffffffu, (uint32_t)lim);
      float m = -CUDART_INF_F, l = 0.f;
      for (int j = 0; j < w.n; ++j, ++g) {
        const int r = g & 1, pb = g % kPBufs;
        ok = ok && wait(kSFull + r, (g >> 1) & 1);
        tc::fence_after_sync();
        uint32_t f[kCols / 32][32];
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c)
          tc::ld32(lane_base + kSCol + kKeys * r + kCols * part + 32 * c, f[c]);
        tc::wait_ld();
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) tc::reg_fence(f[c]);
        tc::fence_before_sync();
        __syncwarp();
        tc2::arrive_pair(s_free + 8 * r, lead);
        // P's buffer of tile g - 2 (the f32 form's one buffer is waited for below)
        if (g >= 2) ok = ok && values_done(g - 2);
        tc::fence_after_sync();
        const int key0 = j * kKeys + kCols * part;
        if (key0 + kCols > all_see || !(sc > 0.f)) {
          const int seen = lim - key0;  // of this thread's keys
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            float x = __uint_as_float(f[c >> 5][c & 31]);
            if (!(sc > 0.f)) x *= sc;
            f[c >> 5][c & 31] = c < seen ? __float_as_uint(x) : 0xff800000u;
          }
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const float x = __uint_as_float(f[c >> 5][c & 31]);
          mx[c & 3] = c < 4 ? x : fmaxf(mx[c & 3], x);
        }
        float *all = red + r * kSplit * kRows;
        all[part * kRows] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * mul;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + w4), "n"(32 * kSplit) : "memory");
        float mt = all[0];
#pragma unroll
        for (int c = 1; c < kSplit; ++c) mt = fmaxf(mt, all[c * kRows]);
        float alpha = 1.f;
        bool rescale = false;
        if (mt > m + kSlack) {
          rescale = m != -CUDART_INF_F;  // with m = -inf the row's O and l are still 0
          alpha = rescale ? ex2(m - mt) : 1.f;
          l *= alpha;
          m = mt;
        }
        const float off = m == -CUDART_INF_F ? 0.f : -m;
        const uint32_t weights = lane_base + kPCol + 64 * pb + kCols / 2 * part;
        uint32_t hi[kCols / 32][16], lo[kLo ? kCols / 32 : 1][16];
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float p0 = ex2(fmaf(__uint_as_float(f[c][2 * e]), mul, off));
            const float p1 = ex2(fmaf(__uint_as_float(f[c][2 * e + 1]), mul, off));
            const uint32_t p = pack_bf16x2(p0, p1);
            hi[c][e] = p;
            if constexpr (kLo) lo[c][e] = pack_bf16x2(p0 - bf16_lo(p), p1 - bf16_hi(p));
            s0 += p0;
            s1 += p1;
          }
          if constexpr (!kLo) tc::st16(weights + 16 * c, hi[c]);
        }
        l += s0 + s1;
        if (__any_sync(0xffffffffu, rescale)) {
          ok = ok && values_done(g - 1);
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < kCols / 32; ++c) {
            uint32_t o[32];
            tc::ld32(lane_base + kOCol + kCols * part + 32 * c, o);
            tc::wait_ld();
            tc::reg_fence(o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tc::st32(lane_base + kOCol + kCols * part + 32 * c, o);
          }
        }
        if constexpr (kLo) {
          if (g >= 1) ok = ok && values_done(g - 1);
          tc::fence_after_sync();
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) {
            tc::st16(weights + 16 * c, hi[c]);
            tc::st16(weights + 64 + 16 * c, lo[c]);
          }
        }
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        tc2::arrive_pair(p_full + 8 * pb, lead);
      }
      // ---- the sum over the query's threads, then O / l
      float *sums = red + (g & 1) * kSplit * kRows;
      sums[part * kRows] = l;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + w4), "n"(32 * kSplit) : "memory");
      l = sums[0];
#pragma unroll
      for (int c = 1; c < kSplit; ++c) l += sums[c * kRows];
      if (g > 1) ok = ok && values_done(g - 2);
      ok = ok && values_done(g - 1);
      tc::fence_after_sync();
      const float inv = m == -CUDART_INF_F ? 0.f : 1.f / l;
      uint32_t o[kCols / 32][32];
#pragma unroll
      for (int c = 0; c < kCols / 32; ++c) tc::ld32(lane_base + kOCol + kCols * part + 32 * c, o[c]);
      tc::wait_ld();
#pragma unroll
      for (int c = 0; c < kCols / 32; ++c) tc::reg_fence(o[c]);
      tc::fence_before_sync();  // (the next block's first P tells the tensor core that O is read)
      // 64 bytes a row and pass; four lanes exchange their 16-byte pieces so that the four write one
      // row's (lanes storing their own rows took 3,000 cycles a block)
      const int first = w.t0 + (int)rank * kRows + 32 * w4 + (lane & ~3);
#pragma unroll
      for (int pass = 0; pass < kCols / (kLo ? 16 : 32); ++pass) {
        uint32_t y[4][4];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          if constexpr (kLo)
            y[k >> 2][k & 3] = __float_as_uint(__uint_as_float(o[pass >> 1][16 * (pass & 1) + k]) * inv);
          else
            y[k >> 2][k & 3] = pack_bf16x2(__uint_as_float(o[kLo ? 0 : pass][2 * k]) * inv,
                                           __uint_as_float(o[kLo ? 0 : pass][2 * k + 1]) * inv);
        }
        transpose4(y, lane);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (ok && first + k < w.nq)
            *reinterpret_cast<uint4 *>(
                static_cast<unsigned char *>(a.out) +
                (((size_t)(w.q0 + first + k) * a.num_heads + w.h) * kDv + kCols * part) * (kLo ? 4 : 2) +
                64 * pass + 16 * (lane & 3)) = make_uint4(y[k][0], y[k][1], y[k][2], y[k][3]);
      }
    }
  }
  // every product done (both CTAs learn it; every copy has landed) before the memory is released
  if (warp == kScores) mbar_wait(bars + kDrainS, 0);
  if (warp == kValues) mbar_wait(bars + kDrainV, 0);
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc2::cluster_sync();
  if (warp == kScores) {
    tc::fence_after_sync();
    tc2::dealloc(tmem, kTmemCols);
  }
}

namespace {

// Rows of `pitch` bytes as (64, rows, slabs): a box of box_rows rows and box_slabs slabs.
bool make_map(CUtensorMap *m, const void *base, long long rows, long long pitch, int slabs,
              int box_rows, int box_slabs) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tc::encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)slabs};
  const cuuint64_t strides[2] = {(cuuint64_t)pitch, 128};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_slabs};
  const cuuint32_t elem[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
             elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kLo>
cudaError_t launch(const ExpandedAttnArgs &a, cudaStream_t s) {
  static std::atomic<bool> attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(dev >= 0 && dev < 64 && attr_set[dev])) {
    e = cudaFuncSetAttribute(pskv_attn_expanded<kLo>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const long long h = a.num_heads;
  Maps maps;
  if (!make_map(&maps.q, a.q, a.total_q, h * kQSlabs * 128, (int)h * kQSlabs, kRows, kQSlabs) ||
      !make_map(&maps.k, a.kv, a.total_k, h * 512, (int)h * 4, kHalf, 2) ||
      !make_map(&maps.v, a.kv, a.total_k, h * 512, (int)h * 4, kKeys, 1) ||
      !make_map(&maps.rot, a.k_rot, a.total_k, a.k_rot_token * 2, 1, kHalf, 1))
    return cudaErrorInvalidValue;
  return launch_pdl(pskv_attn_expanded<kLo>,
                    dim3((unsigned)(2 * h * a.blocks)),
                    dim3(kThreads), kSmemBytes, s, a, maps);
}

}  // namespace

cudaError_t launch_attn_expanded(const ExpandedAttnArgs &a, cudaStream_t s) {
  return a.out_dtype == PSKV_DTYPE_F32 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace pskv
