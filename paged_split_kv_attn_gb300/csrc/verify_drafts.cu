// verify_drafts.cu -- speculative sampling's verification of a drafted chain.
//
// A draft x_t stands while u_t q_t(x_t) < p_t(x_t); behind the standing ones a
// token is drawn from r = max(p - q, 0) (or from p when all stood) by inverting
// the running sum of r at u S, S = sum r.  Only the rows p and q of that one
// place are read whole, once: the call is bound by those bytes, or for a few rows
// by its chain of loads.
//
// The draw has to be the same however the sum is split, so the weights are whole
// numbers: a probability in [0, 1] is taken as the nearest multiple of 2^-60 (exact from 2^-37
// up; ties to the even one), and sums are 128-bit integers, whose order does not matter.
// u is a 24-bit integer times a power of two, so floor(u S) is exact as well.  The multiple
// comes as three signed 20-bit digits, each read off the low bits of a float add to
// 1.5 * 2^3, whose last place is 2^-20, with the exact remainder carried to the next
// (7 floating operations; shifting the mantissa into place took 12 integer ones, which run at
// half the rate).
//
// One cluster of eight CTAs takes a row: warp W of its 64 sums the W-th piece of the
// vocabulary and writes its sum into every CTA's shared memory (distributed shared
// memory); after one cluster barrier every warp knows all 64 sums and with them
// the piece that holds the drawn token, whose CTA goes over it once more (from L2).
// A CTA's shared memory may be written only once the CTA has started: all arrive on the
// cluster's barrier as they start and wait for it before the first remote store, behind the
// sums' loads.
// No workspace, no second launch, no atomics but fault bits.
//
// Measured: 64 rows of 131,072 f32 (67 MB of p and q) 18.2 us with the rows in L2, 22.9 from
// memory (2.9 TB/s); one row of 32,001 bf16, which is the chain launch, drafts, rows, barrier,
// rows again, 6.2 us, and about the same chain stands before and behind the large call's
// stream.  Eight CTAs of eight warps: sixteen CTAs 25.6 and 6.2 us, four of sixteen warps 18.6
// and 7.1.
#include <type_traits>

#include "latent.h"
#include "pskv_internal.cuh"

namespace pskv {

namespace {

using u128 = unsigned __int128;

constexpr int kCluster = 8;
constexpr int kWarps = 8;
constexpr int kPieces = kCluster * kWarps;

// The digits of a probability p (NaN and below 0 as 0, above 1 as 1), p * 2^60 rounded =
// (x - K) * 2^40 + (y - K) * 2^20 + (z - K), K the bits of 12.0f.
struct Digits {
  int x, y, z;
  __device__ explicit Digits(float p) {
    const float s = __saturatef(p);
    const float t1 = s + 12.f, r1 = s - (t1 - 12.f);
    const float t2 = fmaf(r1, 0x1p20f, 12.f), r2 = fmaf(t2 - 12.f, -0x1p-20f, r1);
    const float t3 = fmaf(r2, 0x1p40f, 12.f);
    x = __float_as_int(t1);
    y = __float_as_int(t2);
    z = __float_as_int(t3);
  }
};
constexpr int kTwelve = 0x41400000;

__device__ __forceinline__ uint64_t fixed_point(float p) {
  const Digits d(p);
  return (uint64_t)(((long long)(d.x - kTwelve) << 40) + ((long long)(d.y - kTwelve) << 20) +
                    (d.z - kTwelve));
}

// The row being drawn from.
template <typename T>
struct Weights {
  const T *p, *q;  // q null: nothing taken off but 1 at `point` (-1: nothing)
  int point;

  __device__ static float value(T x) {
    if constexpr (sizeof(T) == 2)
      return __uint_as_float((uint32_t)x << 16);
    else
      return x;
  }
  __device__ uint64_t at(int v, T pv, T qv) const {
    const uint64_t a = fixed_point(value(pv));
    const uint64_t b = q ? fixed_point(value(qv)) : (v == point ? 1ull << 60 : 0);
    return a > b ? a - b : 0;
  }
  __device__ uint64_t at(int v) const { return at(v, p[v], q ? q[v] : T(0)); }
};

__device__ __forceinline__ u128 shfl_xor_128(u128 x, int m) {
  const uint64_t lo = __shfl_xor_sync(0xffffffffu, (unsigned long long)x, m);
  const uint64_t hi = __shfl_xor_sync(0xffffffffu, (unsigned long long)(x >> 64), m);
  return ((u128)hi << 64) | lo;
}
__device__ __forceinline__ u128 shfl_up_128(u128 x, int d) {
  const uint64_t lo = __shfl_up_sync(0xffffffffu, (unsigned long long)x, d);
  const uint64_t hi = __shfl_up_sync(0xffffffffu, (unsigned long long)(x >> 64), d);
  return ((u128)hi << 64) | lo;
}
__device__ __forceinline__ u128 shfl_128(u128 x, int l) {
  const uint64_t lo = __shfl_sync(0xffffffffu, (unsigned long long)x, l);
  const uint64_t hi = __shfl_sync(0xffffffffu, (unsigned long long)(x >> 64), l);
  return ((u128)hi << 64) | lo;
}
__device__ __forceinline__ u128 warp_sum(u128 x) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) x += shfl_xor_128(x, m);
  return x;
}
__device__ __forceinline__ u128 warp_scan(u128 x, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const u128 y = shfl_up_128(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// floor(u * sum), below sum: u in [0, 1) exactly, anything else the nearer end.
__device__ __forceinline__ u128 threshold(float u, u128 sum) {
  if (!(u > 0.f)) return 0;
  if (u >= 1.f) return sum - 1;
  const uint32_t bits = __float_as_uint(u), e = bits >> 23;
  const uint32_t m = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
  const int shift = 150 - (int)(e ? e : 1);
  return shift >= 128 ? (u128)0 : (sum * m) >> shift;
}

// A running sum of weights by digits: 2^20 * kFlush stays below 2^31 in each.
struct Sum {
  static constexpr int kFlush = 1024;  // weights between carries
  int x = 0, y = 0, z = 0, n = 0;
  __int128 total = 0;
  __device__ void add(const Digits &p) {
    x += p.x - kTwelve;
    y += p.y - kTwelve;
    z += p.z - kTwelve;
  }
  // Add p - q where p > q.
  __device__ void add_excess(const Digits &p, const Digits &q, bool more) {
    if (more) {
      x += p.x - q.x;
      y += p.y - q.y;
      z += p.z - q.z;
    }
  }
  __device__ void carry() {
    total += (((__int128)x) << 40) + (((long long)y) << 20) + z;
    x = y = z = n = 0;
  }
  // (called after `count` more weights, which divides kFlush)
  __device__ void counted(int count) {
    if ((n += count) == kFlush) carry();
  }
  __device__ u128 value() {
    carry();
    return (u128)total;
  }
};

// The sum over [lo, hi), 16 bytes a lane and step where both rows are aligned.
template <typename T, bool kVec>
__device__ __forceinline__ u128 sum_range(const Weights<T> &w, int lo, int hi, int lane) {
  using Load = typename std::conditional<kVec, uint4, T>::type;
  constexpr int kN = sizeof(Load) / sizeof(T);  // values a lane takes at once
  constexpr int kDepth = kVec ? 4 : 8;          // loads of each row in flight
  Sum sum;
  auto row = [](const T *p, int v) {
    if constexpr (kVec)
      return __ldg(reinterpret_cast<const uint4 *>(p + v));
    else
      return p[v];
  };
  const Load none = Load{};
  for (int v0 = lo + kN * lane; v0 < hi; v0 += 32 * kN * kDepth) {
    Load pl[kDepth], ql[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) pl[d] = v0 + 32 * kN * d < hi ? row(w.p, v0 + 32 * kN * d) : none;
    if (w.q) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) ql[d] = v0 + 32 * kN * d < hi ? row(w.q, v0 + 32 * kN * d) : none;
#pragma unroll
      for (int d = 0; d < kDepth; ++d)
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const float pv = Weights<T>::value(reinterpret_cast<const T *>(&pl[d])[e]);
          const float qv = Weights<T>::value(reinterpret_cast<const T *>(&ql[d])[e]);
          // (clamped values: a NaN counts as 0)
          sum.add_excess(Digits(pv), Digits(qv), __saturatef(pv) > __saturatef(qv));
        }
    } else {
#pragma unroll
      for (int d = 0; d < kDepth; ++d)
#pragma unroll
        for (int e = 0; e < kN; ++e)
          sum.add(Digits(Weights<T>::value(reinterpret_cast<const T *>(&pl[d])[e])));
    }
    sum.counted(kN * kDepth);
  }
  u128 total = warp_sum(sum.value());
  // the guessed token has no weight left (1 is taken off): what was counted for it goes again
  if (!w.q && w.point >= lo && w.point < hi) total -= fixed_point(Weights<T>::value(w.p[w.point]));
  return total;
}

__device__ __forceinline__ uint32_t rank_in_cluster() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void store_remote(uint64_t *p, uint32_t rank, u128 x) {
  asm volatile(
      "{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.v2.u64 [a], {%2, %3};\n\t}" ::"r"(smem_u32(p)),
      "r"(rank), "l"((uint64_t)x), "l"((uint64_t)(x >> 64))
      : "memory");
}
__device__ __forceinline__ void cluster_arrive_started() {  // nothing written yet: no release
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace

template <typename T, bool kVec>
__global__ void __launch_bounds__(kWarps * 32) pskv_verify_drafts(const VerifyArgs a) {
  __shared__ __align__(16) uint64_t piece_sum[2][kPieces][2];  // (low, high) of each piece; second try
  __shared__ __align__(16) uint64_t part_sum[kWarps][2];
  const int b = blockIdx.x / kCluster, rank = (int)rank_in_cluster();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T_ = a.max_drafts, V = a.vocab;
  cluster_arrive_started();
  pdl_wait();
  pdl_launch_dependents();
  // ---- which drafts stand (every warp for itself)
  int d = a.num_drafts ? a.num_drafts[b] : T_;
  const bool bad_count = d < 0 || d > T_;
  d = min(max(d, 0), T_);
  const T *target = static_cast<const T *>(a.target) + (size_t)b * (T_ + 1) * V;
  const T *draft = a.draft ? static_cast<const T *>(a.draft) + (size_t)b * T_ * V : nullptr;
  const int32_t *drafts = a.drafts + (size_t)b * T_;
  const float *u = a.u + (size_t)b * (T_ + 1);
  int taken = 0;
  bool bad_token = false;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int t = lane + 32 * half;
    bool stands = false;
    if (t < d) {
      const int x = drafts[t];
      if (x >= 0 && x < V) {
        // f32 products in f64 and comparisons of values in [0, 1] are exact; the
        // clamping is the one of the weights
        const float p = Weights<T>::value(target[(size_t)t * V + x]);
        const float q = draft ? Weights<T>::value(draft[(size_t)t * V + x]) : 1.f;
        const float ut = u[t];
        const double uc = !(ut > 0.f) ? 0.0 : (ut >= 1.f ? 1.0 : (double)ut);
        const double qc = !(q > 0.f) ? 0.0 : (q >= 1.f ? 1.0 : (double)q);
        const double pc = !(p > 0.f) ? 0.0 : (p >= 1.f ? 1.0 : (double)p);
        stands = uc * qc < pc;
      } else {
        bad_token = true;
      }
    }
    const uint32_t yes = __ballot_sync(0xffffffffu, stands);
    if (taken == 32 * half) taken += __ffs(~yes) ? __ffs(~yes) - 1 : 32;
  }
  Weights<T> w;
  w.p = target + (size_t)taken * V;
  w.q = taken < d && draft ? draft + (size_t)taken * V : nullptr;
  w.point = taken < d && !draft ? drafts[taken] : -1;
  const bool less = taken < d;  // something is taken off
  // ---- the pieces' sums
  const int seg = ((V + kPieces - 1) / kPieces + 7) & ~7;
  const int W = rank * kWarps + warp;
  u128 before = 0, total = 0;
  int tries = 0;
  for (;; ++tries) {
    const int lo = (int)min((long long)W * seg, (long long)V);
    const int hi = (int)min((long long)(W + 1) * seg, (long long)V);
    const u128 own = sum_range<T, kVec>(w, lo, hi, lane);
    if (tries == 0) {
      __syncwarp();
      cluster_wait();  // and so have the others
    }
    if (lane < kCluster) store_remote(piece_sum[tries][W], lane, own);
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    const uint64_t(*ps)[2] = piece_sum[tries];
    constexpr int kEach = kPieces / 32;  // pieces a lane looks at
    u128 part[kEach], four = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      part[k] = ((u128)ps[kEach * lane + k][1] << 64) | ps[kEach * lane + k][0];
      four += part[k];
    }
    const u128 incl = warp_scan(four, lane);
    total = shfl_128(incl, 31);
    if (total != 0) {
      // the piece where the running sum first passes the threshold
      const u128 thr = threshold(u[T_], total);
      const uint32_t past = __ballot_sync(0xffffffffu, incl > thr);
      const int l = __ffs(past) - 1;  // some lane: thr < total
      u128 left = thr - (incl - four);  // (meant in lane l)
      int k = 0;
#pragma unroll
      for (int e = 0; e < kEach; ++e)
        if (e == k && part[e] <= left) {
          left -= part[e];
          k = e + 1;
        }
      const int hit = __shfl_sync(0xffffffffu, kEach * lane + k, l);
      before = shfl_128(left, l);  // what is left to pass inside the piece
      if (hit / kWarps != rank) return;

      // ---- the CTA that holds it: an eighth of the piece a warp
      const int p0 = hit * seg, p1 = (int)min((long long)p0 + seg, (long long)V);
      const int sub = ((p1 - p0 + kWarps - 1) / kWarps + 7) & ~7;
      const int s_lo = min(p0 + warp * sub, p1), s_hi = min(s_lo + sub, p1);
      const u128 mine = sum_range<T, kVec>(w, s_lo, s_hi, lane);
      if (lane == 0) {
        part_sum[warp][0] = (uint64_t)mine;
        part_sum[warp][1] = (uint64_t)(mine >> 64);
      }
      __syncthreads();
      u128 at = 0;
      for (int k = 0; k < warp; ++k) at += ((u128)part_sum[k][1] << 64) | part_sum[k][0];
      if (before < at || before >= at + mine) return;
      // eight neighbouring tokens a lane: one scan finds the lane, which finds the token
      u128 rest = before - at;
      int token = -1;
      for (int v0 = s_lo; token < 0 && v0 < s_hi; v0 += 32 * 8) {
        uint64_t x[8];
        u128 own8 = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int v = v0 + 8 * lane + e;
          x[e] = v < s_hi ? w.at(v) : 0;
          own8 += x[e];
        }
        const u128 incl8 = warp_scan(own8, lane);
        const uint32_t over = __ballot_sync(0xffffffffu, incl8 > rest);
        if (over) {
          const int l8 = __ffs(over) - 1;
          u128 left = rest - (incl8 - own8);  // (meant in lane l8)
          int e8 = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e == e8 && x[e] <= left) {
              left -= x[e];
              e8 = e + 1;
            }
          token = __shfl_sync(0xffffffffu, v0 + 8 * lane + e8, l8);
        } else {
          rest -= shfl_128(incl8, 31);
        }
      }
      for (int t = lane; t <= T_; t += 32)
        a.tokens[(size_t)b * (T_ + 1) + t] = t < taken ? drafts[t] : (t == taken ? token : -1);
      if (lane == 0) {
        a.accepted[b] = taken;
        if (bad_count) raise_fault(a.status, PSKV_FAULT_BAD_LENGTH);
      }
      if (bad_token) raise_fault(a.status, PSKV_FAULT_BAD_TOKEN);
      return;
    }
    if (tries == 1 || !less) break;
    w.q = nullptr;  // nothing is left of p: the draw is from p itself
    w.point = -1;
  }
  // ---- no weight at all
  if (W != 0) return;
  for (int t = lane; t <= T_; t += 32)
    a.tokens[(size_t)b * (T_ + 1) + t] = t < taken ? drafts[t] : -1;
  if (lane == 0) {
    a.accepted[b] = taken;
    raise_fault(a.status, PSKV_FAULT_EMPTY_ROW | (bad_count ? PSKV_FAULT_BAD_LENGTH : 0u));
  }
  if (bad_token) raise_fault(a.status, PSKV_FAULT_BAD_TOKEN);
}

namespace {

template <typename T, bool kVec>
cudaError_t launch(const VerifyArgs &a, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.batch * kCluster);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, pskv_verify_drafts<T, kVec>, a);
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs &a, cudaStream_t s) {
  const int size = a.dtype == PSKV_DTYPE_BF16 ? 2 : 4;
  // 16-byte loads need every row on a 16-byte boundary
  const bool vec = ((reinterpret_cast<uintptr_t>(a.target) | reinterpret_cast<uintptr_t>(a.draft)) & 15u) == 0 &&
                   (long long)a.vocab * size % 16 == 0;
  if (size == 2) return vec ? launch<uint16_t, true>(a, s) : launch<uint16_t, false>(a, s);
  return vec ? launch<float, true>(a, s) : launch<float, false>(a, s);
}

}  // namespace pskv
