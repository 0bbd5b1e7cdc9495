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
// S(j + 1) runs while the softmax works on tile j.  Per tile the pipe works (12 + 8) * 64 = 1,280
// cycles on both SMs.  (One CTA with two blocks of 128 queries has no room for that: sharing one
// score region between the blocks took 5,500 cycles for the same 2 * 256 * 128 pairs
// that now take two tiles.)
// A row's 128 scores lie in two threads (halves of the keys by warp group), which
// mask them and exchange their maxima; the reference maximum moves only past a slack of
// 8 (log2 units), so O is rarely rescaled.
//
// P is rounded to bf16 when the output is (it adds about what the output's own
// rounding does; f32 output: a bf16 pair), everything else is f32.  Every wait is bounded; on
// expiry the CTA flags PSKV_FAULT_WAIT_TIMEOUT, lets what it issued finish and
// frees its tensor memory.
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
constexpr int kThreads = 384;          // warps: 0 S, 1 PV, 2 Q and K copies, 3 V copies, 4-11 softmax
constexpr int kSoftWarps = 8;
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
  kSFull = kQFull + 1,       // [2] scores of region r in
  kSFree = kSFull + 2,       // [2] (even CTA) region r read in both CTAs
  kPFull = kSFree + 2,       // [2] (even CTA) P written in both CTAs
  kPvDone = kPFull + 2,      // [2] the values of P's tile done
  kRagged = kPvDone + 2,     // this CTA's V of the tile with the row's end
  kDrainS = kRagged + 1,
  kDrainV = kDrainS + 1,
  kNumBars = kDrainV + 1
};
constexpr int kOffRed = kOffBar + kNumBars * 8;          // float[2][2][128] maxima (then sums)
constexpr int kOffSlot = kOffRed + 2 * 2 * kRows * 4;
constexpr int kOffAbort = kOffSlot + 4;
constexpr int kSmemBytes = kOffAbort + 4 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

constexpr uint32_t kIdescS = tc::instr_desc(2 * kRows, kKeys, false, false);
constexpr uint32_t kIdescPV = tc::instr_desc(2 * kRows, kDv, false, true);

struct Maps {
  CUtensorMap q, k, v, rot;
};

}  // namespace

template <bool kLo>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    pskv_attn_expanded(const ExpandedAttnArgs a, const __grid_constant__ Maps maps) {
  constexpr int kPBufs = kLo ? 1 : 2;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *sm = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + kOffBar);
  uint32_t *slot = reinterpret_cast<uint32_t *>(sm + kOffSlot);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + kOffAbort);
  const int warp = tc2::uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rank = tc2::cluster_rank();
  const bool lead = elect_one();  // one thread of each warp
  const int h = blockIdx.x >> 1, b = blockIdx.z;

  pdl_wait();
  pdl_launch_dependents();
  const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
  const int nq = q1 - q0, nk = k1 - k0;
  // offsets that the host copies do not allow: the row is left out (by both CTAs)
  if (q0 < 0 || q1 < q0 || q1 > a.total_q || k0 < 0 || k1 < k0 || k1 > a.total_k || nk < nq ||
      nq > (long long)gridDim.y * 2 * kRows) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
      raise_fault(a.status, PSKV_FAULT_BAD_LENGTH);
    return;
  }
  // later queries see more keys: they go first
  const int blocks = (nq + 2 * kRows - 1) / (2 * kRows);
  if ((int)blockIdx.y >= blocks) return;
  const int t0 = (blocks - 1 - (int)blockIdx.y) * 2 * kRows;  // the pair's first query in the row
  const int before = nk - nq;                                 // keys before the row's first query
  const int n = (before + min(nq, t0 + 2 * kRows) + kKeys - 1) / kKeys;  // tiles up to the last own key

  if (warp == 2) {
    if (lane == 0) {
      for (int s = 0; s < kRing; ++s) {
        mbar_init(&bars[kFullK + s], 1);
        mbar_init(&bars[kFullV + s], 3);  // the expected bytes, and a word from either V copy warp
        mbar_init(&bars[kEmptyK + s], 1);
        mbar_init(&bars[kEmptyV + s], 1);
      }
      mbar_init(&bars[kQFull], 1);
      for (int r = 0; r < 2; ++r) {
        mbar_init(&bars[kSFull + r], 1);
        mbar_init(&bars[kSFree + r], 2 * kSoftWarps);
        mbar_init(&bars[kPFull + r], 2 * kSoftWarps);
        mbar_init(&bars[kPvDone + r], 1);
      }
      mbar_init(&bars[kRagged], 1);
      mbar_init(&bars[kDrainS], 1);
      mbar_init(&bars[kDrainV], 1);
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
    return tc::all_wait(bars + s, parity, abort_flag, a.status);
  };

  if (warp == 0) {
    if (rank == 0) {
      // ---- the score products (all lanes alike, one issues)
      bool ok = wait(kQFull, 0);
      const uint32_t q = smem_u32(sm + kOffQ), k = smem_u32(sm + kOffK);
      for (int j = 0; ok && j < n; ++j) {
        const int st = j % kRing, r = j & 1;
        ok = wait(kFullK + st, (j / kRing) & 1) && (j < 2 || wait(kSFree + r, (j / 2 - 1) & 1));
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
      tc2::commit_both(bars + kDrainS, lead);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      // ---- the value products
      bool ok = true;
      const uint32_t v = smem_u32(sm + kOffV);
      for (int j = 0; ok && j < n; ++j) {
        const int st = j % kRing, pb = j % kPBufs;
        ok = wait(kFullV + st, (j / kRing) & 1) && wait(kPFull + pb, (j / kPBufs) & 1);
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
        tc2::commit_both(bars + kPvDone + pb, lead);
        tc2::commit_both(bars + kEmptyV + st, lead);
      }
      tc2::commit_both(bars + kDrainV, lead);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---- Q (queries behind the row's last: other rows' or zeros), then K: this CTA's half
    tc2::expect_tx(bars + kQFull, 2 * kQBytes, lead && rank == 0);
    tc2::tma_load_3d(smem_u32(sm + kOffQ), &maps.q, 0, q0 + t0 + (int)rank * kRows, kQSlabs * h,
                     tc2::map_to(smem_u32(bars + kQFull), 0), lead);
    int j = 0;
    for (; j < n; ++j) {
      const int st = j % kRing;
      if (j >= kRing && !wait(kEmptyK + st, (j / kRing - 1) & 1)) break;
      const uint32_t dst = smem_u32(sm + kOffK + st * kKBytes);
      const uint32_t bar = tc2::map_to(smem_u32(bars + kFullK + st), 0);
      const int y = k0 + j * kKeys + kHalf * (int)rank;
      tc2::expect_tx(bars + kFullK + st, 2 * kKBytes, lead && rank == 0);
      tc2::tma_load_3d(dst, &maps.k, 0, y, 4 * h, bar, lead);
      tc2::tma_load_3d(dst + 2 * kKSlab, &maps.rot, 0, y, 0, bar, lead);
    }
    // every copy of both CTAs landed before they leave (their count is the even CTA's)
    if (rank == 0) {
      for (int s = max(0, j - kRing); s < j; ++s) mbar_wait(bars + kFullK + s % kRing, (s / kRing) & 1);
      mbar_wait(bars + kQFull, 0);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ---- V: this CTA's 64 columns of every tile.  The tile with the row's last key: rows
    // behind it are another row's and meet P = 0, so they are zeroed first.
    const bool ragged = n * kKeys > nk;
    const int last = n - 1;
    int j = 0;
    for (; j < n; ++j) {
      const int st = j % kRing;
      if (j >= kRing && !wait(kEmptyV + st, (j / kRing - 1) & 1)) break;
      const uint32_t full = tc2::map_to(smem_u32(bars + kFullV + st), 0);
      const bool whole = !(ragged && j == last);
      if (!whole)
        tc2::expect_tx(bars + kRagged, kVBytes, lead);
      else
        tc2::expect_tx(bars + kFullV + st, 2 * kVBytes, lead && rank == 0);
      tc2::tma_load_3d(smem_u32(sm + kOffV + st * kVBytes), &maps.v, 0, k0 + j * kKeys,
                       4 * h + 2 + (int)rank, whole ? full : smem_u32(bars + kRagged), lead);
      tc2::arrive_pair(full, lead && whole);
    }
    __syncwarp();
    if (ragged && j == n) mbar_wait(bars + kRagged, 0);  // (bounded)
    if (rank == 0)
      for (int s = max(0, j - kRing); s < j; ++s)
        if (!(ragged && s == last)) mbar_wait(bars + kFullV + s % kRing, (s / kRing) & 1);
    __syncwarp();
    if (ragged) {
      const int st = last % kRing, left = nk - last * kKeys;
      unsigned char *dst = sm + kOffV + st * kVBytes;
      for (int e = lane; e < (kKeys - left) * 8; e += 32)
        *reinterpret_cast<uint4 *>(dst + (left + (e >> 3)) * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
      tc::fence_smem_for_async();
      __syncwarp();
      if (rank == 0 && lead) mbar_arrive(bars + kFullV + st);  // in place of the copies' count
      tc2::arrive_pair(tc2::map_to(smem_u32(bars + kFullV + st), 0), lead);
    }
  } else {
    // ---- the softmax: thread (query i, keys 64 gr .. + 63 of the tile).  The loop never leaves
    // early (the two warps of a query's threads meet every tile); after a failed wait nothing
    // is written.
    const int w = warp & 3, gr = (warp - 4) >> 2, i = 32 * w + lane;
    const int t = t0 + (int)rank * kRows + i;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * w) << 16);
    const int lim = t < nq ? before + t + 1 : 0;  // keys below lim are seen
    const float sc = a.scale_log2;
    float *red = reinterpret_cast<float *>(sm + kOffRed);
    const uint32_t s_free = tc2::map_to(smem_u32(bars + kSFree), 0);
    const uint32_t p_full = tc2::map_to(smem_u32(bars + kPFull), 0);
    float m = -CUDART_INF_F, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int r = j & 1, pb = j % kPBufs;
      ok = ok && wait(kSFull + r, (j >> 1) & 1);
      tc::fence_after_sync();
      uint32_t va[32], vb[32];
      tc::ld32(lane_base + kSCol + kKeys * r + kHalf * gr, va);
      tc::ld32(lane_base + kSCol + kKeys * r + kHalf * gr + 32, vb);
      tc::wait_ld();
      tc::reg_fence(va);
      tc::reg_fence(vb);
      tc::fence_before_sync();
      __syncwarp();
      tc2::arrive_pair(s_free + 8 * r, lead);
      float f[kHalf];
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        f[c] = __uint_as_float(va[c]);
        f[32 + c] = __uint_as_float(vb[c]);
      }
      const int key0 = j * kKeys + kHalf * gr;
      // scores in log2 units are mul * f: whole tiles leave the product to the exponent's
      // multiply-add, others (and scales that are not positive) take it before the mask
      float mul = sc;
      if (__any_sync(0xffffffffu, key0 + kHalf > lim || !(sc > 0.f))) {
        mul = 1.f;
#pragma unroll
        for (int c = 0; c < kHalf; ++c) f[c] = key0 + c < lim ? f[c] * sc : -CUDART_INF_F;
      }
      float mx[4] = {f[0], f[1], f[2], f[3]};
#pragma unroll
      for (int c = 4; c < kHalf; ++c) mx[c & 3] = fmaxf(mx[c & 3], f[c]);
      float *mine = red + r * 2 * kRows + i;
      float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * mul;
      mine[gr * kRows] = mt;
      asm volatile("bar.sync %0, 64;" ::"r"(1 + w) : "memory");
      mt = fmaxf(mt, mine[(gr ^ 1) * kRows]);
      float alpha = 1.f;
      bool rescale = false;
      if (mt > m + kSlack) {
        rescale = m != -CUDART_INF_F;  // with m = -inf the row's O and l are still 0
        alpha = rescale ? ex2(m - mt) : 1.f;
        l *= alpha;
        m = mt;
      }
      const float off = m == -CUDART_INF_F ? 0.f : -m;
      uint32_t hi[32], lo[kLo ? 32 : 1];
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const float p0 = ex2(fmaf(f[2 * e], mul, off)), p1 = ex2(fmaf(f[2 * e + 1], mul, off));
        hi[e] = pack_bf16x2(p0, p1);
        if constexpr (kLo) lo[e] = pack_bf16x2(p0 - bf16_lo(hi[e]), p1 - bf16_hi(hi[e]));
        s0 += p0;
        s1 += p1;
      }
      l += s0 + s1;
      // P's buffer is free once the values of tile j - kPBufs are done
      if (j >= kPBufs) ok = ok && wait(kPvDone + pb, (j / kPBufs - 1) & 1);
      if (__any_sync(0xffffffffu, rescale)) {
        ok = ok && wait(kPvDone + (j - 1) % kPBufs, ((j - 1) / kPBufs) & 1);
        tc::fence_after_sync();
#pragma unroll 1
        for (int c = 2 * gr; c < 2 * gr + 2; ++c) {
          uint32_t o[32];
          tc::ld32(lane_base + kOCol + 32 * c, o);
          tc::wait_ld();
          tc::reg_fence(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
          tc::st32(lane_base + kOCol + 32 * c, o);
        }
      }
      tc::fence_after_sync();
      tc::st32(lane_base + kPCol + 64 * pb + 32 * gr, hi);
      if constexpr (kLo) tc::st32(lane_base + kPCol + 64 + 32 * gr, lo);
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      tc2::arrive_pair(p_full + 8 * pb, lead);
    }
    // ---- the sum over both threads, then O / l, put together in the queries' place and the K
    // ring (their products are done) so that rows leave in whole lines
    float *sums = red + (n & 1) * 2 * kRows + i;
    sums[gr * kRows] = l;
    asm volatile("bar.sync %0, 64;" ::"r"(1 + w) : "memory");
    l = sums[0] + sums[kRows];
    ok = ok && wait(kPvDone + (n - 1) % kPBufs, ((n - 1) / kPBufs) & 1);
    tc::fence_after_sync();
    const float inv = m == -CUDART_INF_F ? 0.f : 1.f / l;
    constexpr int kBytes = kDv * (kLo ? 4 : 2), kPitch = kBytes + 16;
    static_assert(kRows * kPitch <= kOffV, "staging");
    unsigned char *stage = sm + kOffQ + 32 * w * kPitch;
#pragma unroll 1
    for (int c = 2 * gr; c < 2 * gr + 2; ++c) {
      uint32_t o[32];
      tc::ld32(lane_base + kOCol + 32 * c, o);
      tc::wait_ld();
      tc::reg_fence(o);
      uint4 *dst = reinterpret_cast<uint4 *>(stage + lane * kPitch + c * (kLo ? 128 : 64));
      float y[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) y[k] = __uint_as_float(o[k]) * inv;
      if constexpr (kLo) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          reinterpret_cast<float4 *>(dst)[k] = make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          dst[k] = make_uint4(pack_bf16x2(y[8 * k], y[8 * k + 1]), pack_bf16x2(y[8 * k + 2], y[8 * k + 3]),
                              pack_bf16x2(y[8 * k + 4], y[8 * k + 5]), pack_bf16x2(y[8 * k + 6], y[8 * k + 7]));
      }
    }
    asm volatile("bar.sync %0, 64;" ::"r"(1 + w) : "memory");
    constexpr int kPieces = kBytes / 16;  // per row
    const int first = t0 + (int)rank * kRows + 32 * w;
    if (ok)
      for (int e = 32 * gr + lane; e < 32 * kPieces; e += 64) {
        const int r = e / kPieces, piece = e % kPieces;
        if (first + r < nq)
          reinterpret_cast<uint4 *>(a.out)[((size_t)(q0 + first + r) * a.num_heads + h) * kPieces + piece] =
              *reinterpret_cast<const uint4 *>(stage + r * kPitch + piece * 16);
      }
  }
  // every product done (both CTAs learn it; every copy has landed) before the memory is released
  if (warp == 0) mbar_wait(bars + kDrainS, 0);
  if (warp == 1) mbar_wait(bars + kDrainV, 0);
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
  static bool attr_set[64] = {};
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
                    dim3(2 * a.num_heads, (a.max_q + 2 * kRows - 1) / (2 * kRows), a.batch),
                    dim3(kThreads), kSmemBytes, s, a, maps);
}

}  // namespace

cudaError_t launch_attn_expanded(const ExpandedAttnArgs &a, cudaStream_t s) {
  return a.out_dtype == PSKV_DTYPE_F32 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace pskv
