// attn_latent.cu -- absorbed attention over a paged latent pool.
//
// A first, simple kernel: one warp per (row, query column, partition) walks its
// keys with a running maximum and sum; lane l holds columns 64 i + 2 l, + 1.
#include <math_constants.h>

#include "latent.h"
#include "pskv_internal.cuh"

namespace pskv {

template <int DC>
__global__ void __launch_bounds__(128) pskv_attn_latent(const LatentAttnArgs a) {
  constexpr int D = DC + PSKV_LATENT_ROT, kC = D / 64, kV = DC / 64;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const int cols = a.num_tokens * a.num_q_heads;
  const int col = blockIdx.x * 4 + (threadIdx.x >> 5), p = blockIdx.y, b = blockIdx.z;
  if (col >= cols) return;
  const long long cap = (long long)a.table_stride * a.page_size;
  long long len = a.seq_lens[b];
  if (len < 0 || len > cap || (len > 0 && len < a.num_tokens)) {
    if (col == 0 && p == 0 && lane == 0) raise_fault(a.status, PSKV_FAULT_BAD_LENGTH);
    len = len < 0 ? 0 : (len > cap ? cap : len);
  }
  const int t = col / a.num_q_heads;
  const int tiles = (int)((len + 63) / 64), per = (tiles + a.num_splits - 1) / a.num_splits;
  const int k_lo = min(p * per, tiles) * 64;
  const int k_hi = (int)min((long long)min(p * per + per, tiles) * 64, len - a.num_tokens + t + 1);
  const size_t row = (size_t)b * cols + col;
  const uint32_t *q = reinterpret_cast<const uint32_t *>(a.q) + row * (D / 2) + lane;
  float qf[kC][2], o[kV][2], m = -CUDART_INF_F, l = 0.f;
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    qf[i][0] = bf16_lo(q[32 * i]);
    qf[i][1] = bf16_hi(q[32 * i]);
  }
#pragma unroll
  for (int i = 0; i < kV; ++i) o[i][0] = o[i][1] = 0.f;
  const int32_t *tbl = a.page_tables + (size_t)b * a.table_stride;
  for (int key = k_lo; key < k_hi; ++key) {
    const int page = tbl[key / a.page_size];
    if (page < 0 || (long long)page >= a.num_pages) {
      if (lane == 0) raise_fault(a.status, PSKV_FAULT_BAD_PAGE);
      continue;
    }
    const uint32_t *k = reinterpret_cast<const uint32_t *>(a.pool) +
                        ((size_t)page * a.page_size + key % a.page_size) * (D / 2) + lane;
    uint32_t x[kC];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      x[i] = k[32 * i];
      s = fmaf(qf[i][0], bf16_lo(x[i]), fmaf(qf[i][1], bf16_hi(x[i]), s));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= a.scale_log2;
    if (s > m) {
      const float f = exp2f(m - s);
      l *= f;
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        o[i][0] *= f;
        o[i][1] *= f;
      }
      m = s;
    }
    const float w = exp2f(s - m);
    l += w;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      o[i][0] = fmaf(w, bf16_lo(x[i]), o[i][0]);
      o[i][1] = fmaf(w, bf16_hi(x[i]), o[i][1]);
    }
  }
  const bool empty = m == -CUDART_INF_F;
  if (!a.direct) {
    const size_t at = row * a.num_splits + p;
    if (lane == 0) {
      a.ws_m[at] = empty ? m : m * kLn2;
      a.ws_l[at] = l;
    }
#pragma unroll
    for (int i = 0; i < kV; ++i)
      reinterpret_cast<float2 *>(a.ws_o + at * DC)[32 * i + lane] = make_float2(o[i][0], o[i][1]);
    return;
  }
  if (empty && len > 0 && lane == 0) raise_fault(a.status, PSKV_FAULT_EMPTY_ROW);
  const float inv = empty ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const float y0 = o[i][0] * inv, y1 = o[i][1] * inv;
    if (a.out_dtype == PSKV_DTYPE_BF16)
      (static_cast<uint32_t *>(a.out) + row * (DC / 2))[32 * i + lane] = pack_bf16x2(y0, y1);
    else
      reinterpret_cast<float2 *>(static_cast<float *>(a.out) + row * DC)[32 * i + lane] =
          make_float2(y0, y1);
  }
}

cudaError_t launch_attn_latent(const LatentAttnArgs &a, int dc, cudaStream_t s) {
  const dim3 grid((a.num_tokens * a.num_q_heads + 3) / 4, a.num_splits, a.batch);
  if (dc == 512) return launch_pdl(pskv_attn_latent<512>, grid, dim3(128), 0, s, a);
  if (dc == 256) return launch_pdl(pskv_attn_latent<256>, grid, dim3(128), 0, s, a);
  return cudaErrorInvalidValue;
}

}  // namespace pskv
