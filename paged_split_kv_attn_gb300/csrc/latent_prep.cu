// latent_prep.cu -- the prep of a latent pool with the page write fused in.
//
// Per token: the latent c becomes c / sqrt(mean(c^2) + eps) * w, the key's 64
// columns turn by the token's position, both go straight into the token's page
// slot (and into a dense copy when one is asked for); the query heads' 64
// rotated columns turn by the same angle.  No sum but the one of squares, formed
// in a fixed order (each lane over its columns, then a butterfly), in f32;
// each value is rounded once, when it is stored.
//
// Bound by bytes for a prompt chunk and by the chain of dependent loads (row
// and key -> page and angle -> store) for a decode step, so every load that
// does not wait for another is issued first.  One warp writes a token's row
// (lane l: 16-byte pieces l, l + 32 of the latent; lanes 0-7 a piece of the
// rotated key each); the queries take a warp for sixteen heads (8 lanes of 16 bytes
// a head, four heads at a time, all loaded before the chain of page and angle loads is
// waited for: with four heads a warp a chunk of 8,168 tokens under 32 heads took 30.5 us,
// bound by that chain; with 72 registers a thread and blocks of eight warps 18.5, with 64
// and four 15.7, 6.2 TB/s, or 20.9 from memory), so a pair (i, i + 32) lies in two lanes,
// four apart, and a pair (2i, 2i + 1) inside one lane.
#include "latent.h"
#include "pskv_internal.cuh"

namespace pskv {

namespace {

constexpr int kWarps = 4;
constexpr int kBlocksPerSm = 8;  // 64 registers a thread, 32 warps an SM
constexpr int kRot = PSKV_LATENT_ROT;
constexpr int kHeadSteps = 4;                  // four heads at a time
constexpr int kHeadsPerWarp = 4 * kHeadSteps;

__device__ __forceinline__ void unpack8(const uint4 x, float (&f)[8]) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(u[i]);
    f[2 * i + 1] = bf16_hi(u[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// The angles that piece `piece` (8 of the 64 columns) needs, at table row `at`:
// halves: columns 8 (piece % 4) .. + 7; adjacent: 4 piece .. + 3 (the rest unused).
struct Angles {
  float c[8], s[8];
};

__device__ __forceinline__ void load_angles(Angles &g, const LatentPrepArgs &a, int pos, int piece) {
  const size_t at = (size_t)pos * (kRot / 2);
  const int first = a.adjacent ? 4 * piece : 8 * (piece & 3);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (k == 1 && a.adjacent) break;
    const float4 c = __ldg(reinterpret_cast<const float4 *>(a.rope_cos + at + first) + k);
    const float4 s = __ldg(reinterpret_cast<const float4 *>(a.rope_sin + at + first) + k);
    g.c[4 * k] = c.x; g.c[4 * k + 1] = c.y; g.c[4 * k + 2] = c.z; g.c[4 * k + 3] = c.w;
    g.s[4 * k] = s.x; g.s[4 * k + 1] = s.y; g.s[4 * k + 2] = s.z; g.s[4 * k + 3] = s.w;
  }
}

// Turn the 64 columns that 8 neighbouring lanes hold (8 each); every lane of the warp calls.
__device__ __forceinline__ uint4 turn(const uint4 x, const Angles &g, bool adjacent, int piece) {
  float f[8], y[8];
  unpack8(x, f);
  if (adjacent) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = f[2 * i] * g.c[i] - f[2 * i + 1] * g.s[i];
      y[2 * i + 1] = f[2 * i + 1] * g.c[i] + f[2 * i] * g.s[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, f[i], 4);
      y[i] = piece < 4 ? f[i] * g.c[i] - other * g.s[i] : f[i] * g.c[i] + other * g.s[i];
    }
  }
  return pack8(y);
}

}  // namespace

template <int DC>
__global__ void __launch_bounds__(kWarps * 32, kBlocksPerSm) pskv_latent_prep(const LatentPrepArgs a) {
  constexpr int kPieces = DC / 256;  // 16-byte pieces of the latent per lane
  const int lane = threadIdx.x & 31, piece = lane & 7;
  const int slots = 1 + (a.num_q_heads + kHeadsPerWarp - 1) / kHeadsPerWarp;
  const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  pdl_wait();
  pdl_launch_dependents();
  if (item >= (long long)a.n * slots) return;
  const int t = (int)(item / slots), s = (int)(item % slots);
  const int b = a.row_of[t], key = a.pos_of[t];
  uint4 c[kPieces], r = make_uint4(0, 0, 0, 0), rq[kHeadSteps];
  float4 w[kPieces][2];
  const int head = (s - 1) * kHeadsPerWarp + (lane >> 3);  // then every fourth
  const bool mine = lane < 8;  // (s = 0) this lane holds a piece of the key to turn
  if (s == 0) {
    const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) +
                                                     (size_t)t * (size_t)a.x_token);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      c[k] = x[lane + 32 * k];
      if (a.w) {
        w[k][0] = __ldg(reinterpret_cast<const float4 *>(a.w) + 2 * (lane + 32 * k));
        w[k][1] = __ldg(reinterpret_cast<const float4 *>(a.w) + 2 * (lane + 32 * k) + 1);
      } else {
        w[k][0] = w[k][1] = make_float4(1.f, 1.f, 1.f, 1.f);
      }
    }
    if (mine) r = x[DC / 8 + lane];
  } else {
#pragma unroll
    for (int k = 0; k < kHeadSteps; ++k)
      rq[k] = head + 4 * k < a.num_q_heads
                  ? *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) +
                                                     (size_t)t * (size_t)a.q_token +
                                                     (size_t)(head + 4 * k) * (size_t)a.q_head + 8 * piece)
                  : make_uint4(0, 0, 0, 0);
  }
  // the token's place, checked the same way by all its warps: a refused row writes nothing
  uint32_t fault = 0;
  int page = -1, pos = 0;
  if (b < 0 || b >= a.batch || key < 0) {
    fault = PSKV_FAULT_PAST_PAGES;
  } else {
    const int lease = a.pages_of_row[b];
    const long long slot = key / a.page_size;
    page = slot < a.table_stride ? a.page_tables[(size_t)b * a.table_stride + slot] : -1;
    const long long p = (long long)key + (a.first_pos ? a.first_pos[b] : 0);
    if (p < 0 || p >= a.max_pos)
      fault = PSKV_FAULT_BAD_POSITION;
    else if (lease < 0 || lease > a.table_stride || (long long)key >= (long long)lease * a.page_size)
      fault = PSKV_FAULT_PAST_PAGES;
    else if (page < 0 || (long long)page >= a.num_pages)
      fault = PSKV_FAULT_BAD_PAGE;
    pos = (int)p;
  }
  if (fault) {
    if (s == 0 && lane == 0) raise_fault(a.status, fault);
    return;
  }
  Angles g;
  load_angles(g, a, pos, piece);
  if (s > 0) {
#pragma unroll
    for (int k = 0; k < kHeadSteps; ++k) {
      const uint4 y = turn(rq[k], g, a.adjacent != 0, piece);
      if (head + 4 * k < a.num_q_heads)
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.q_out) +
                                   (size_t)t * (size_t)a.q_out_token +
                                   (size_t)(head + 4 * k) * (size_t)a.q_out_head + 8 * piece) = y;
    }
    return;
  }
  r = turn(r, g, a.adjacent != 0, piece);
  float f[kPieces][8], ss = 0.f;
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    unpack8(c[k], f[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(f[k][e], f[k][e], ss);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  const float inv = 1.f / sqrtf(ss / (float)DC + a.eps);
  const size_t row = (size_t)page * a.page_size + key % a.page_size;
  uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.pool) + row * (DC + kRot));
  uint4 *den = a.dense ? reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.dense) +
                                                   (size_t)t * (DC + kRot))
                       : nullptr;
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    const float m[8] = {w[k][0].x, w[k][0].y, w[k][0].z, w[k][0].w,
                        w[k][1].x, w[k][1].y, w[k][1].z, w[k][1].w};
#pragma unroll
    for (int e = 0; e < 8; ++e) f[k][e] = f[k][e] * inv * m[e];
    const uint4 y = pack8(f[k]);
    dst[lane + 32 * k] = y;
    if (den) den[lane + 32 * k] = y;
  }
  if (mine) {
    dst[DC / 8 + lane] = r;
    if (den) den[DC / 8 + lane] = r;
  }
}

cudaError_t launch_latent_prep(const LatentPrepArgs &a, cudaStream_t s) {
  const long long items =
      (long long)a.n * (1 + (a.num_q_heads + kHeadsPerWarp - 1) / kHeadsPerWarp);
  const long long blocks = (items + kWarps - 1) / kWarps;
  if (blocks <= 0) return cudaSuccess;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (a.dc == 512)
    return launch_pdl(pskv_latent_prep<512>, dim3((unsigned)blocks), dim3(kWarps * 32), 0, s, a);
  if (a.dc == 256)
    return launch_pdl(pskv_latent_prep<256>, dim3((unsigned)blocks), dim3(kWarps * 32), 0, s, a);
  return cudaErrorInvalidValue;
}

}  // namespace pskv
