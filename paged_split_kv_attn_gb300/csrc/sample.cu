// sample.cu -- sampling from logits with temperature, top-k, top-p and min-p.
//
// For a row l with largest value M: x = (l - M) / T in f32 steps, w = expf(x), W = w rounded to the
// nearest multiple of 2^-40.  Tokens are ordered by x, then by index; what the filters keep is a
// first part of that order (and w >= min_p), so it is given by a border: every x above the border's,
// and of those equal to it the ones up to some index.  The border is found digit by digit of the bits of |x|
// (which go up as x falls), from counts (top-k) or sums (top-p) of each digit's tokens.
// W are whole numbers and their sums exact, so nothing depends on the order of the work.
#include <limits.h>
#include <math_constants.h>

#include "pskv_internal.cuh"
#include "tree.h"

namespace pskv {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr uint32_t kNever = 0x7f800000u;  // |x| of a token without weight: infinity's bits
constexpr float kOne = 1099511627776.f;   // 2^40

template <typename T>
__device__ __forceinline__ float logit(T x) {
  float f;
  if constexpr (sizeof(T) == 2)
    f = __uint_as_float((uint32_t)x << 16);
  else
    f = x;
  return f == f ? f : -CUDART_INF_F;
}

// The bits of |x| for a logit, M the row's largest and inv = 1 / T.
__device__ __forceinline__ uint32_t depth(float l, float M, float inv) {
  const float x = l == M ? 0.f : __fmul_rn(__fsub_rn(l, M), inv);
  return x == x ? __float_as_uint(x) & 0x7fffffffu : kNever;
}
__device__ __forceinline__ float weight(uint32_t d) { return expf(-__uint_as_float(d)); }
__device__ __forceinline__ uint64_t whole(float w) { return (uint64_t)__float2ll_rn(w * kOne); }

// floor(x * s) for x in [0, 1) and s below 2^63.
__device__ __forceinline__ uint64_t share(float x, uint64_t s) {
  if (!(x > 0.f)) return 0;
  const uint32_t bits = __float_as_uint(x), e = bits >> 23;
  const uint64_t m = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
  const int shift = 150 - (int)(e ? e : 1);
  return shift >= 128 ? 0 : (uint64_t)(((unsigned __int128)s * m) >> shift);
}

struct Shared {
  uint32_t count[kBins];
  unsigned long long sum[kBins];
  unsigned long long part[kWarps];
  float top[kWarps];
  int index[kWarps];
};

template <typename T>
struct Row {
  const T *l;
  int vocab, lo, hi;  // this warp's part [lo, hi)
  float M, inv;
  uint32_t border;    // kept: depth below it, or equal and index <= last
  int last;
  float least;        // and weight at least this
  __device__ uint32_t at(int v) const { return depth(logit(l[v]), M, inv); }
  __device__ bool inside(uint32_t d, int v) const { return d < border || (d == border && v <= last); }
  __device__ uint64_t kept(int v) const {
    const uint32_t d = at(v);
    if (!inside(d, v)) return 0;
    const float w = weight(d);
    return w >= least ? whole(w) : 0;
  }
};

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long x) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// Move the border to the last token of the order's first part: the `limit` first ones (by_sum false), or
// the shortest part whose sum is at least `limit`.  Returns the sum of that part.
template <typename T>
__device__ uint64_t find_border(Row<T> &r, Shared &sh, bool by_sum, uint64_t limit) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t prefix = 0;
  int shift = 31;
  uint64_t many = 0, sum = 0;  // tokens and weight before the digits found so far
  while (shift > 0) {
    const int width = shift > 20 ? 11 : 10, below = shift - width;
    for (int i = tid; i < kBins; i += kThreads) sh.count[i] = 0, sh.sum[i] = 0;
    __syncthreads();
    for (int v = r.lo + lane; v < r.hi; v += 32) {
      const uint32_t d = r.at(v);
      if ((d >> shift) != prefix || !r.inside(d, v)) continue;
      const uint32_t digit = (d >> below) & ((1u << width) - 1);
      atomicAdd(&sh.count[digit], 1u);
      atomicAdd(&sh.sum[digit], (unsigned long long)whole(weight(d)));
    }
    __syncthreads();
    uint32_t digit = 0;  // every thread alike
    for (; digit < kBins - 1; ++digit) {
      if (by_sum ? sum + sh.sum[digit] >= limit : many + sh.count[digit] >= limit) break;
      sum += sh.sum[digit];
      many += sh.count[digit];
    }
    prefix = (prefix << width) | digit;
    shift = below;
    __syncthreads();
  }
  // how many of the equal ones
  const uint64_t w = whole(weight(prefix));
  const uint64_t ties = by_sum ? (limit - sum + w - 1) / w : limit - many;
  // and the index of the last of them
  uint32_t mine = 0;
  for (int v0 = r.lo; v0 < r.hi; v0 += 32)
    mine += __popc(__ballot_sync(0xffffffffu, v0 + lane < r.hi && r.at(v0 + lane) == prefix));
  if (lane == 0) sh.part[warp] = mine;
  __syncthreads();
  uint64_t before = 0;
  for (int k = 0; k < warp; ++k) before += sh.part[k];
  if (before < ties && ties <= before + mine)
    for (int v0 = r.lo; v0 < r.hi; v0 += 32) {
      const bool eq = v0 + lane < r.hi && r.at(v0 + lane) == prefix;
      const uint32_t all = __ballot_sync(0xffffffffu, eq);
      if (eq && before + __popc(all & ((2u << lane) - 1)) == ties) sh.index[0] = v0 + lane;
      before += __popc(all);
    }
  __syncthreads();
  r.border = prefix;
  r.last = sh.index[0];
  __syncthreads();
  return sum + ties * w;
}

}  // namespace

template <typename T>
__global__ void __launch_bounds__(kThreads) pskv_sample(const SampleArgs a) {
  __shared__ Shared sh;
  const int row = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_launch_dependents();
  const int req = row / a.per_request;
  Row<T> r;
  r.l = static_cast<const T *>(a.logits) + row * a.logits_row;
  r.vocab = a.vocab;
  const int seg = (a.vocab + kWarps - 1) / kWarps;
  r.lo = min(warp * seg, a.vocab);
  r.hi = min(r.lo + seg, a.vocab);
  // ---- the largest logit, lowest index first
  float top = -CUDART_INF_F;
  int at = INT_MAX;
  for (int v = r.lo + lane; v < r.hi; v += 32) {
    const float l = logit(r.l[v]);
    if (l > top) top = l, at = v;
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, top, m);
    const int i = __shfl_xor_sync(0xffffffffu, at, m);
    if (o > top || (o == top && i < at)) top = o, at = i;
  }
  if (lane == 0) sh.top[warp] = top, sh.index[warp] = at;
  __syncthreads();
  top = sh.top[0], at = sh.index[0];
  for (int k = 1; k < kWarps; ++k)
    if (sh.top[k] > top) top = sh.top[k], at = sh.index[k];
  __syncthreads();
  const bool empty = top == -CUDART_INF_F;
  r.M = top;
  const float heat = a.temperature ? a.temperature[req] : 1.f;
  r.inv = __fdiv_rn(1.f, heat);
  const bool greedy = !(heat > 0.f) || r.inv == CUDART_INF_F;
  if (greedy) r.inv = 1.f;
  r.border = greedy ? 0 : kNever;
  r.last = greedy ? at : INT_MAX;
  const float least = a.min_p ? a.min_p[req] : 0.f;
  r.least = least > 0.f ? fminf(least, 1.f) : 0.f;
  if (!empty && !greedy) {
    const int k = a.top_k ? a.top_k[req] : 0;
    const float p = a.top_p ? a.top_p[req] : 1.f;
    const bool some = k > 0 && k < a.vocab;
    uint64_t sum = 0;
    if (some) sum = find_border(r, sh, false, (uint64_t)k);
    if (p < 1.f) {
      if (!some) {
        for (int v = r.lo + lane; v < r.hi; v += 32) sum += whole(weight(r.at(v)));
        sum = warp_sum(sum);
        if (lane == 0) sh.part[warp] = sum;
        __syncthreads();
        sum = 0;
        for (int i = 0; i < kWarps; ++i) sum += sh.part[i];
        __syncthreads();
      }
      const uint64_t limit = share(p, sum);
      find_border(r, sh, true, limit > 0 ? limit : 1);
    }
  }
  // ---- the draw
  unsigned long long mine = 0;
  if (!empty)
    for (int v = r.lo + lane; v < r.hi; v += 32) mine += r.kept(v);
  mine = warp_sum(mine);
  if (lane == 0) sh.part[warp] = mine;
  __syncthreads();
  uint64_t total = 0, before = 0;
  for (int k = 0; k < kWarps; ++k) {
    if (k < warp) before += sh.part[k];
    total += sh.part[k];
  }
  if (a.u) {
    if (empty) {
      if (tid == 0) a.tokens[row] = -1;
    } else {
      const float u = a.u[row];
      const uint64_t thr = u >= 1.f ? total - 1 : share(u, total);
      if (before <= thr && thr < before + mine) {
        uint64_t run = before;
        for (int v0 = r.lo; v0 < r.hi; v0 += 32) {
          const uint64_t w = v0 + lane < r.hi ? r.kept(v0 + lane) : 0;
          uint64_t incl = w;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const unsigned long long y = __shfl_up_sync(0xffffffffu, (unsigned long long)incl, d);
            if (lane >= d) incl += y;
          }
          if (run + incl - w <= thr && thr < run + incl) a.tokens[row] = v0 + lane;
          run += __shfl_sync(0xffffffffu, (unsigned long long)incl, 31);
        }
      }
    }
  }
  if (empty && tid == 0) raise_fault(a.status, PSKV_FAULT_EMPTY_ROW);
  if (a.probs) {
    // W / S: W has at most 24 significant bits; 1 / S as a float pair
    const double inv = empty ? 0.0 : 1.0 / (double)total;
    const float hi = (float)inv, lo = (float)(inv - (double)hi);
    const size_t out = (size_t)row * a.vocab;
    for (int v = r.lo + lane; v < r.hi; v += 32) {
      const float w = empty ? 0.f : (float)r.kept(v);
      const float p = fmaf(w, hi, w * lo);
      if (a.probs_dtype == PSKV_DTYPE_BF16)
        static_cast<__nv_bfloat16 *>(a.probs)[out + v] = __float2bfloat16_rn(p);
      else
        static_cast<float *>(a.probs)[out + v] = p;
    }
  }
}

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t s) {
  const dim3 grid((unsigned)a.rows), block(kThreads);
  return a.dtype == PSKV_DTYPE_BF16 ? launch_pdl(pskv_sample<uint16_t>, grid, block, 0, s, a)
                                    : launch_pdl(pskv_sample<float>, grid, block, 0, s, a);
}

}  // namespace pskv
