// attn_expanded.cu -- expanded latent attention of variable-length chunks on the
// fifth-generation tensor cores.
//
// Per row, head h and query i: s_ij = scale * (qn_i . kn_j + qr_i . r_j) over the keys
// j up to the query's own, o_i = sum_j softmax(s_i)_j v_j; 192 score columns (the rotated
// 64 shared by all heads) and 128 value columns.  2 * (192 + 128) operations a (query, key)
// pair and head: compute-bound from a few hundred tokens on.
//
// A CTA takes 256 queries of one head as two blocks A and B of 128 (the MMAs' M; f32 output:
// one block) and walks the keys in tiles of 128.  Tensor memory, 512 columns: one score
// region of 128 that both blocks use in turn, a P region of 64 for each (bf16 pairs, the
// MMAs' A operand) and O, 128 f32 columns each.  The tensor pipe's order is
//   S_A(j)  PV_B(j-1)  S_B(j)  PV_A(j)  S_A(j+1) ...
// so that while a block's scores are read into registers the other block's values run, and
// every product waits only for something issued a whole product earlier.  (Two score
// regions with P over them would make S_x(j+1) wait for PV_x(j) itself.)  Per tile
// of both blocks the pipe works 2 * (12 + 8) * 64 = 2,560 cycles (S from shared memory, PV with A
// from tensor memory, both at the full rate).
// One softmax thread per query: it reads its 128 scores, masks them, moves the
// reference maximum only past a slack of 8 (log2 units) and writes P.  K and V come
// in 64-column slabs of 128 rows (16 KB): K (two unrotated slabs and the rotated one a tile)
// through a ring of four, V (both slabs in one copy) through one of two tiles.  The products
// and the copies are each issued by a single thread that runs its whole loop (with a
// whole-warp wait and an election per slab the same products took three times as long to issue
// as to run).
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

namespace pskv {

namespace {

using tc::elect_one;
using tc::ex2;

constexpr int kRows = 128;             // queries per block (MMA M)
constexpr int kKeys = 128;             // keys per tile
constexpr int kQSlabs = 3;             // 64-column slabs of a query or key
constexpr int kSlab = 128 * 128;       // 128 rows of 64 columns: 16 KB
constexpr int kRingK = 4;              // K slabs in flight (three a tile)
constexpr int kRingV = 2;              // V tiles in flight (two slabs)
constexpr int kDv = PSKV_EXPANDED_V;
constexpr int kThreads = 384;          // warps: 0 MMA, 1 Q and K copies, 2 V copies, 4-7 softmax A, 8-11 B
constexpr int kTmemCols = 512;
constexpr float kSlack = 8.f;
// tensor memory: S, then P of the blocks (f32 output: hi and lo of the one), then O
constexpr int kSCol = 0, kPCol = 128, kOCol = 256;

constexpr int kOffQ = 0;                             // block x at x * 3 slabs
constexpr int kOffK = kOffQ + 2 * kQSlabs * kSlab;
constexpr int kOffV = kOffK + kRingK * kSlab;
constexpr int kOffBar = kOffV + kRingV * 2 * kSlab;
enum : int {
  kFullK = 0,                // [4] slab landed
  kFullV = kFullK + kRingK,  // [2] tile landed
  kEmptyK = kFullV + kRingV,  // [4] its products done
  kEmptyV = kEmptyK + kRingK,  // [2]
  kQFull = kEmptyV + kRingV,  // [2] block x's queries landed
  kSFull = kQFull + 2,       // [2] block x's scores in
  kSFree = kSFull + 2,       // the score region read
  kPFull = kSFree + 1,       // [2] block x's P written
  kPvDone = kPFull + 2,      // [2] block x's values done
  kRagged = kPvDone + 2,     // V of the tile with the row's end
  kDrain = kRagged + 1,
  kNumBars = kDrain + 1
};
constexpr int kOffSlot = kOffBar + kNumBars * 8;
constexpr int kOffAbort = kOffSlot + 4;
constexpr int kSmemBytes = kOffAbort + 4 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

constexpr uint32_t kIdescS = tc::instr_desc(kRows, kKeys, false, false);
constexpr uint32_t kIdescPV = tc::instr_desc(kRows, kDv, false, true);

struct Maps {
  CUtensorMap q, k, v, rot;
};

// The CTA's share, the same in every thread.
struct Plan {
  int q0, nq, k0, nk;  // the row's first query and key, and how many
  int t0;              // the CTA's first query in the row
  int n[2];            // key tiles of each block
  int tiles;           // of either
};

__device__ __forceinline__ int tiles_below(int keys) { return keys > 0 ? (keys + kKeys - 1) / kKeys : 0; }

}  // namespace

template <bool kLo>
__global__ void __launch_bounds__(kThreads, 1)
    pskv_attn_expanded(const ExpandedAttnArgs a, const __grid_constant__ Maps maps) {
  constexpr int kBlocks = kLo ? 1 : 2;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *sm = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + kOffBar);
  uint32_t *slot = reinterpret_cast<uint32_t *>(sm + kOffSlot);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + kOffAbort);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x, b = blockIdx.z;

  pdl_wait();
  pdl_launch_dependents();
  Plan pl;
  pl.q0 = a.cu_q[b];
  pl.k0 = a.cu_k[b];
  const int q1 = a.cu_q[b + 1], k1 = a.cu_k[b + 1];
  pl.nq = q1 - pl.q0;
  pl.nk = k1 - pl.k0;
  constexpr int per = kBlocks * kRows;
  // offsets that the host copies do not allow: the row is left out
  if (pl.q0 < 0 || q1 < pl.q0 || q1 > a.total_q || pl.k0 < 0 || k1 < pl.k0 || k1 > a.total_k ||
      pl.nk < pl.nq || pl.nq > (long long)gridDim.y * per) {
    if (h == 0 && blockIdx.y == 0 && threadIdx.x == 0) raise_fault(a.status, PSKV_FAULT_BAD_LENGTH);
    return;
  }
  // later queries see more keys: they go first
  const int blocks = (pl.nq + per - 1) / per;
  if ((int)blockIdx.y >= blocks) return;
  pl.t0 = (blocks - 1 - (int)blockIdx.y) * per;

  if (warp == 1) {
    if (lane == 0) {
      for (int s = 0; s < kQFull; ++s) mbar_init(&bars[s], 1);  // full and empty
      for (int x = 0; x < 2; ++x) {
        mbar_init(&bars[kQFull + x], 1);
        mbar_init(&bars[kSFull + x], 1);
        mbar_init(&bars[kPFull + x], 4);
        mbar_init(&bars[kPvDone + x], 1);
      }
      mbar_init(&bars[kSFree], 4);
      mbar_init(&bars[kRagged], 1);
      mbar_init(&bars[kDrain], 1);
      *abort_flag = 0;
      mbar_fence_init();
    }
    __syncwarp();
  } else if (warp == 0) {
    tc::alloc(slot, kTmemCols);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *slot;
  auto wait = [&](int s, uint32_t parity) {
    return tc::all_wait(bars + s, parity, abort_flag, a.status);
  };
  auto wait1 = [&](int s, uint32_t parity) {
    return tc::one_wait(bars + s, parity, abort_flag, a.status);
  };

  // queries [t0, t0 + 128 kBlocks) of the row; key tiles up to each block's last own key
  const int before = pl.nk - pl.nq;  // keys before the row's first query
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int t = pl.t0 + x * kRows;
    pl.n[x] = x < kBlocks && t < pl.nq ? tiles_below(before + min(pl.nq, t + kRows)) : 0;
  }
  pl.tiles = max(pl.n[0], pl.n[1]);

  if (warp == 0) {
    if (elect_one()) {
      // ---- the products
      bool ok = true;
      int s_ops = 0;  // score products so far: the region is free once the last one's scores are read
      const uint32_t q0 = smem_u32(sm + kOffQ), k0 = smem_u32(sm + kOffK), v0 = smem_u32(sm + kOffV);
      auto scores = [&](int x, int j) {
        if (s_ops > 0) ok = ok && wait1(kSFree, (s_ops - 1) & 1);
        if (j == 0) ok = ok && wait1(kQFull + x, 0);
        ++s_ops;
        const bool frees = x == 1 || j >= pl.n[1];  // the tile's last scores
#pragma unroll
        for (int c = 0; c < kQSlabs; ++c) {
          const int s = kQSlabs * j + c, st = s % kRingK;
          ok = ok && wait1(kFullK + st, (s / kRingK) & 1);
          if (!ok) return;
          tc::fence_after_sync();
          const uint32_t q = q0 + (x * kQSlabs + c) * kSlab, k = k0 + st * kSlab;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc::mma(tmem + kSCol, tc::smem_desc(q + kk * 32, 16, 1024),
                    tc::smem_desc(k + kk * 32, 16, 1024), kIdescS, c > 0 || kk > 0);
          if (frees) tc::commit(bars + kEmptyK + st);
        }
        tc::commit(bars + kSFull + x);
      };
      auto values = [&](int x, int j) {
        const int st = j % kRingV;
        ok = ok && wait1(kPFull + x, j & 1) && wait1(kFullV + st, (j / kRingV) & 1);
        if (!ok) return;
        tc::fence_after_sync();
        const uint32_t v = v0 + st * 2 * kSlab;
#pragma unroll
        for (int part = 0; part < (kLo ? 2 : 1); ++part)
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            tc::mma_ts(tmem + kOCol + kDv * x, tmem + kPCol + 64 * (x + part) + 8 * kk,
                       tc::smem_desc(v + kk * 2048, kSlab, 1024), kIdescPV,
                       j > 0 || part > 0 || kk > 0);
        if (x == 1 || j >= pl.n[1]) tc::commit(bars + kEmptyV + st);
        tc::commit(bars + kPvDone + x);
      };
      if (pl.n[1] == 0) {  // one block: its next scores go ahead of its values
        for (int j = 0; ok && j <= pl.tiles; ++j) {
          if (j < pl.tiles) scores(0, j);
          if (j > 0) values(0, j - 1);
        }
      } else {
        for (int j = 0; ok && j <= pl.tiles; ++j) {
          if (j < pl.n[0]) scores(0, j);
          if (j > 0 && j - 1 < pl.n[1]) values(1, j - 1);
          if (j < pl.n[1]) scores(1, j);
          if (j < pl.n[0]) values(0, j);
        }
      }
      tc::commit(bars + kDrain);
      mbar_wait(bars + kDrain, 0);  // every product done before the memory is released
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      // ---- Q, and K's slabs
#pragma unroll
      for (int x = 0; x < kBlocks; ++x)
        if (pl.n[x] > 0) {
          mbar_arrive_expect_tx(bars + kQFull + x, kQSlabs * kSlab);
          tc::tma_load_3d(sm + kOffQ + x * kQSlabs * kSlab, &maps.q, 0, pl.q0 + pl.t0 + x * kRows,
                          kQSlabs * h, bars + kQFull + x);
        }
      int s = 0;
      bool ok = true;
      for (int j = 0; ok && j < pl.tiles; ++j)
#pragma unroll
        for (int c = 0; c < kQSlabs; ++c) {
          const int st = s % kRingK;
          if (s >= kRingK) ok = ok && wait1(kEmptyK + st, (s / kRingK - 1) & 1);
          if (!ok) break;
          uint64_t *bar = bars + kFullK + st;
          unsigned char *dst = sm + kOffK + st * kSlab;
          mbar_arrive_expect_tx(bar, kSlab);
          if (c < 2)
            tc::tma_load_3d(dst, &maps.k, 0, pl.k0 + j * kKeys, 4 * h + c, bar);
          else
            tc::tma_load_3d(dst, &maps.rot, 0, pl.k0 + j * kKeys, 0, bar);
          ++s;
        }
      // every copy landed before the CTA leaves
      for (int r = max(0, s - kRingK); r < s; ++r) mbar_wait(bars + kFullK + r % kRingK, (r / kRingK) & 1);
#pragma unroll
      for (int x = 0; x < kBlocks; ++x)
        if (pl.n[x] > 0) mbar_wait(bars + kQFull + x, 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---- V's tiles.  The one with the row's last key: rows behind it are another row's and
    // meet P = 0, so they are zeroed first.
    const bool ragged = pl.tiles * kKeys > pl.nk;
    const int last = pl.tiles - 1, left = pl.nk - last * kKeys;
    if (elect_one()) {
      int j = 0;
      for (; j < pl.tiles; ++j) {
        const int st = j % kRingV;
        if (j >= kRingV && !wait1(kEmptyV + st, (j / kRingV - 1) & 1)) break;
        uint64_t *bar = bars + (ragged && j == last ? (int)kRagged : kFullV + st);
        mbar_arrive_expect_tx(bar, 2 * kSlab);
        tc::tma_load_3d(sm + kOffV + st * 2 * kSlab, &maps.v, 0, pl.k0 + j * kKeys, 4 * h + 2, bar);
      }
      if (ragged && j == pl.tiles) mbar_wait(bars + kRagged, 0);  // (bounded)
      for (int r = max(0, j - kRingV); r < j; ++r)  // every copy landed before the CTA leaves
        if (!(ragged && r == last)) mbar_wait(bars + kFullV + r % kRingV, (r / kRingV) & 1);
    }
    __syncwarp();
    if (ragged) {
      unsigned char *dst = sm + kOffV + (last % kRingV) * 2 * kSlab;
      for (int e = lane; e < (kKeys - left) * 16; e += 32)
        *reinterpret_cast<uint4 *>(dst + ((e >> 3) & 1) * kSlab + (left + (e >> 4)) * 128 + (e & 7) * 16) =
            make_uint4(0, 0, 0, 0);
      tc::fence_smem_for_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + kFullV + last % kRingV);
    }
  } else if (warp >= 4 && (warp - 4) / 4 < kBlocks) {
    // ---- the softmax: one thread per query
    const int x = (warp - 4) >> 2, w = warp & 3, i = 32 * w + lane;
    const int t = pl.t0 + x * kRows + i;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * w) << 16);
    const int lim = t < pl.nq ? before + t + 1 : 0;  // keys below lim are seen
    const float sc = a.scale_log2;
    float m = -CUDART_INF_F, l = 0.f;
    bool ok = true;
    for (int j = 0; ok && j < pl.n[x]; ++j) {
      if (!(ok = wait(kSFull + x, j & 1))) break;
      tc::fence_after_sync();
      uint32_t v[4][32];
#pragma unroll
      for (int q = 0; q < 4; ++q) tc::ld32(lane_base + kSCol + 32 * q, v[q]);
      tc::wait_ld();
#pragma unroll
      for (int q = 0; q < 4; ++q) tc::reg_fence(v[q]);
      float f[kKeys];
#pragma unroll
      for (int c = 0; c < kKeys; ++c) f[c] = __uint_as_float(v[c >> 5][c & 31]);
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + kSFree);
      const int key0 = j * kKeys;
      // scores in log2 units are mul * f: whole tiles leave the product to the exponent's
      // multiply-add, others (and scales that are not positive) take it before the mask
      float mul = sc;
      if (key0 + kKeys > lim || !(sc > 0.f)) {
        mul = 1.f;
#pragma unroll
        for (int c = 0; c < kKeys; ++c) f[c] = key0 + c < lim ? f[c] * sc : -CUDART_INF_F;
      }
      float mx[4] = {f[0], f[1], f[2], f[3]};
#pragma unroll
      for (int c = 4; c < kKeys; ++c) mx[c & 3] = fmaxf(mx[c & 3], f[c]);
      const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * mul;
      float alpha = 1.f;
      bool rescale = false;
      if (mt > m + kSlack) {
        rescale = m != -CUDART_INF_F;  // with m = -inf the row's O and l are still 0
        alpha = rescale ? ex2(m - mt) : 1.f;
        l *= alpha;
        m = mt;
      }
      // P's region is free, and O may be rescaled, once the last tile's values are done
      if (j > 0 && !(ok = wait(kPvDone + x, (j - 1) & 1))) break;
      tc::fence_after_sync();
      if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
        for (int c = 0; c < kDv / 32; ++c) {
          uint32_t o[32];
          tc::ld32(lane_base + kOCol + kDv * x + 32 * c, o);
          tc::wait_ld();
          tc::reg_fence(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
          tc::st32(lane_base + kOCol + kDv * x + 32 * c, o);
        }
      }
      const float off = m == -CUDART_INF_F ? 0.f : -m;
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t hi[32], lo[kLo ? 32 : 1];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float p0 = ex2(fmaf(f[64 * q + 2 * e], mul, off));
          const float p1 = ex2(fmaf(f[64 * q + 2 * e + 1], mul, off));
          hi[e] = pack_bf16x2(p0, p1);
          if constexpr (kLo) lo[e] = pack_bf16x2(p0 - bf16_lo(hi[e]), p1 - bf16_hi(hi[e]));
          s0 += p0;
          s1 += p1;
        }
        tc::st32(lane_base + kPCol + 64 * x + 32 * q, hi);
        if constexpr (kLo) tc::st32(lane_base + kPCol + 64 + 32 * q, lo);
      }
      l += s0 + s1;
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + kPFull + x);
    }
    // ---- O / l, put together in the queries' place (their products are done) by warps, each
    // its own 32 rows, so that they leave in whole lines
    if (pl.n[x] > 0) ok = ok && wait(kPvDone + x, (pl.n[x] - 1) & 1);
    if (ok && pl.n[x] > 0) {
      tc::fence_after_sync();
      const float inv = m == -CUDART_INF_F ? 0.f : 1.f / l;
      constexpr int kBytes = kDv * (kLo ? 4 : 2), kPitch = kBytes + 16;
      unsigned char *stage = sm + kOffQ + x * kQSlabs * kSlab + 32 * w * kPitch;
      static_assert(kRows * kPitch <= (kLo ? 2 : 1) * kQSlabs * kSlab, "staging");
#pragma unroll 1
      for (int c = 0; c < kDv / 32; ++c) {
        uint32_t o[32];
        tc::ld32(lane_base + kOCol + kDv * x + 32 * c, o);
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
      __syncwarp();
      constexpr int kPieces = kBytes / 16;  // per row
      const int first = pl.t0 + x * kRows + 32 * w;
      for (int e = lane; e < 32 * kPieces; e += 32) {
        const int r = e / kPieces, piece = e % kPieces;
        if (first + r < pl.nq)
          reinterpret_cast<uint4 *>(a.out)[((size_t)(pl.q0 + first + r) * a.num_heads + h) * kPieces + piece] =
              *reinterpret_cast<const uint4 *>(stage + r * kPitch + piece * 16);
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::dealloc(tmem, kTmemCols);
  }
}

namespace {

// Rows of `pitch` bytes as (64, rows, slabs): a box of 128 rows and box_slabs slabs.
bool make_map(CUtensorMap *m, const void *base, long long rows, long long pitch, int slabs,
              int box_slabs) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tc::encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)slabs};
  const cuuint64_t strides[2] = {(cuuint64_t)pitch, 128};
  const cuuint32_t box[3] = {64, 128, (cuuint32_t)box_slabs};
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
  if (!make_map(&maps.q, a.q, a.total_q, h * kQSlabs * 128, (int)h * kQSlabs, kQSlabs) ||
      !make_map(&maps.k, a.kv, a.total_k, h * 512, (int)h * 4, 1) ||
      !make_map(&maps.v, a.kv, a.total_k, h * 512, (int)h * 4, 2) ||
      !make_map(&maps.rot, a.k_rot, a.total_k, a.k_rot_token * 2, 1, 1))
    return cudaErrorInvalidValue;
  const int per = (kLo ? 1 : 2) * kRows;
  return launch_pdl(pskv_attn_expanded<kLo>, dim3(a.num_heads, (a.max_q + per - 1) / per, a.batch),
                    dim3(kThreads), kSmemBytes, s, a, maps);
}

}  // namespace

cudaError_t launch_attn_expanded(const ExpandedAttnArgs &a, cudaStream_t s) {
  return a.out_dtype == PSKV_DTYPE_F32 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace pskv
