// attn_expanded.cu -- expanded latent attention of variable-length chunks.
//
// A first, simple kernel: one warp per (row, token, head) walks the keys up to
// the token's own with a running maximum and sum; lane l holds columns 64 i + 2 l, + 1.
#include <math_constants.h>

#include "latent.h"
#include "pskv_internal.cuh"

namespace pskv {

__global__ void __launch_bounds__(128) pskv_attn_expanded(const ExpandedAttnArgs a) {
  constexpr int kQ = PSKV_EXPANDED_NOPE + PSKV_LATENT_ROT, kKV = PSKV_EXPANDED_NOPE + PSKV_EXPANDED_V;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5), h = blockIdx.y, b = blockIdx.z;
  const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
  if (q0 < 0 || q1 < q0 || q1 > a.total_q || k0 < 0 || k1 > a.total_k || k1 - k0 < q1 - q0) {
    if (t == 0 && h == 0 && lane == 0) raise_fault(a.status, PSKV_FAULT_BAD_LENGTH);
    return;
  }
  if (t >= q1 - q0) return;
  const size_t row = (size_t)(q0 + t) * a.num_heads + h;
  const uint32_t *q = static_cast<const uint32_t *>(a.q) + row * (kQ / 2) + lane;
  float qf[3][2], o[2][2] = {}, m = -CUDART_INF_F, l = 0.f;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    qf[i][0] = bf16_lo(q[32 * i]);
    qf[i][1] = bf16_hi(q[32 * i]);
  }
  const int n = (k1 - k0) - (q1 - q0) + t + 1;
  for (int j = 0; j < n; ++j) {
    const uint32_t *kv = static_cast<const uint32_t *>(a.kv) +
                         ((size_t)(k0 + j) * a.num_heads + h) * (kKV / 2) + lane;
    const uint32_t r = *(reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(a.k_rot) +
                                                            (size_t)(k0 + j) * a.k_rot_token) + lane);
    const uint32_t x0 = kv[0], x1 = kv[32], v0 = kv[64], v1 = kv[96];
    float s = qf[0][0] * bf16_lo(x0) + qf[0][1] * bf16_hi(x0) + qf[1][0] * bf16_lo(x1) +
              qf[1][1] * bf16_hi(x1) + qf[2][0] * bf16_lo(r) + qf[2][1] * bf16_hi(r);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
    l = l * f + w;
    o[0][0] = o[0][0] * f + w * bf16_lo(v0);
    o[0][1] = o[0][1] * f + w * bf16_hi(v0);
    o[1][0] = o[1][0] * f + w * bf16_lo(v1);
    o[1][1] = o[1][1] * f + w * bf16_hi(v1);
    m = mn;
  }
  const float inv = 1.f / l;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float y0 = o[i][0] * inv, y1 = o[i][1] * inv;
    if (a.out_dtype == PSKV_DTYPE_BF16)
      (static_cast<uint32_t *>(a.out) + row * (PSKV_EXPANDED_V / 2))[32 * i + lane] =
          pack_bf16x2(y0, y1);
    else
      reinterpret_cast<float2 *>(static_cast<float *>(a.out) + row * PSKV_EXPANDED_V)[32 * i + lane] =
          make_float2(y0, y1);
  }
}

cudaError_t launch_attn_expanded(const ExpandedAttnArgs &a, cudaStream_t s) {
  return launch_pdl(pskv_attn_expanded, dim3((a.max_q + 3) / 4, a.num_heads, a.batch), dim3(128), 0,
                    s, a);
}

}  // namespace pskv
