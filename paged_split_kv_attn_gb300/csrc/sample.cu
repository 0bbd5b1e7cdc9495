// sample.cu -- sampling from logits with temperature, top-k, top-p and min-p.
//
// For a row l with largest value M: x = (l - M) / T in f32 steps, w = expf(x), W = w rounded to the
// nearest multiple of 2^-40.  Tokens are ordered by x, then by index; what top-k and top-p keep is a
// first part of that order, so it is given by a border: the last token kept, (|x|, index).
// W are whole numbers and sums 64-bit integers, so nothing depends on how the work is split.
//
// A cluster of up to eight CTAs takes a row, each warp a piece of the vocabulary.  The row is
// read from memory once, for M; the later passes find it in L1 and L2 (staged in shared memory, fewer
// CTAs fit on an SM: 64 rows of 131,072 would take two waves).
//   1  M, and the largest logit of each of a piece's 32 chunks: later passes leave out chunks below what they look for
//   2  the sum of W, and a histogram of |x| in steps of 1/64 (counts: a shared-memory atomic a token,
//      beside the exponentials)
//   3  the bin that holds the border: by the counts (top-k), or by the bins' estimated weight (top-p).
//      If all tokens up to that bin's end fit in a list, they are listed, and all that is left
//      (top-k's border, top-p's, the draw) is found in the list by every CTA for itself.  Else the pass
//      sums W exactly over what lies before the bin and lists the bin alone; an estimate that was off shows in the
//      exact sum, and another bin is tried from there.  A bin that does not fit is cut into
//      2,048 finer ones, down to a single |x|, whose tokens' border is a matter of counting
//   4  the drawn token's piece again, and the probabilities where they are asked for.
// Between passes the warps' results cross the cluster through distributed shared memory, one barrier each.
// A token in a list is found by 256 bins of its key (|x|'s bits, then the index) at a time.
#include <float.h>
#include <limits.h>
#include <math_constants.h>

#include "pskv_internal.cuh"
#include "tree.h"

namespace pskv {

namespace {

using u64 = unsigned long long;

constexpr int kMaxCluster = 8;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxPieces = kMaxCluster * kWarps;
constexpr int kPerSm = 4;        // CTAs an SM holds (registers)
constexpr int kBins = 2048;
constexpr int kList = 1024;      // listed tokens of a cluster
constexpr int kEach = 8;         // elements a lane takes in a step
constexpr int kStep = 32 * kEach;
constexpr int kQueue = 32 + 4 * 32;
constexpr float kDeepest = 31.98f;        // what lies deeper has no weight: expf(-31.98) is under 2^-46
constexpr uint32_t kDeep = 0x41ffd70au;   // its bits

// |x| of a logit, up to kDeepest (NaN and -inf: that), M the row's largest and inv = 1 / T.  (M = +inf: its
// tokens have 0, all others kDeepest, by the largest finite number as M and inv = +inf.)
__device__ __forceinline__ float depth_of(float l, float M, float inv) {
  return fabsf(fminf(fmaxf(__fmul_rn(__fsub_rn(l, M), inv), -kDeepest), 0.f));
}
// Its bits, which go up as x falls.
__device__ __forceinline__ uint32_t depth(float l, float M, float inv) { return __float_as_uint(depth_of(l, M, inv)); }
__device__ __forceinline__ float weight(uint32_t d) { return expf(-__uint_as_float(d)); }

// W = hi * 2^20 + lo by two float adds whose last place is 2^-20: hi the nearest multiple, lo of the exact rest.
constexpr uint32_t kTwelve = 0x41400000u;
struct Digits {
  uint32_t hi, lo;  // plus kTwelve each
  __device__ explicit Digits(float w) {
    const float t1 = w + 12.f, rest = w - (t1 - 12.f), t2 = fmaf(rest, 0x1p20f, 12.f);
    hi = __float_as_uint(t1);
    lo = __float_as_uint(t2);
  }
};
__device__ __forceinline__ u64 whole(float w) {
  const Digits g(w);
  return ((u64)(g.hi - kTwelve) << 20) + (u64)(long long)(int)(g.lo - kTwelve);
}

// A sum of W by digits: carried before 2^11 of them have been added.
struct Sum {
  uint32_t hi = 0, lo = 0;
  u64 total = 0;
  __device__ void add(float w) {
    const Digits g(w);
    hi += g.hi - kTwelve;
    lo += g.lo - kTwelve;
  }
  __device__ void carry() {
    total += ((u64)hi << 20) + (u64)(long long)(int)lo;
    hi = lo = 0;
  }
};

// floor(x * s) for x in [0, 1) and s below 2^63.
__device__ __forceinline__ u64 share(float x, u64 s) {
  if (!(x > 0.f)) return 0;
  const uint32_t bits = __float_as_uint(x), e = bits >> 23;
  const u64 m = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
  const int shift = 150 - (int)(e ? e : 1);
  return shift >= 128 ? 0 : (u64)(((unsigned __int128)s * m) >> shift);
}

__device__ __forceinline__ u64 warp_sum(u64 x) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}
__device__ __forceinline__ u64 warp_scan(u64 x, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// The largest of the lanes' floats (none of them NaN), as integers of the same order.
__device__ __forceinline__ float warp_max(float x) {
  const int i = __float_as_int(x), m = __reduce_max_sync(0xffffffffu, i ^ ((i >> 31) & 0x7fffffff));
  return __int_as_float(m ^ ((m >> 31) & 0x7fffffff));
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t remote(const void *p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void store_remote(uint32_t at, u64 x) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(x) : "memory");
}
__device__ __forceinline__ void store_remote(uint32_t at, uint32_t x) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}
__device__ __forceinline__ uint32_t load_remote_word(uint32_t at) {
  uint32_t x;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ uint2 load_remote(uint32_t at) {
  uint2 x;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ void cluster_arrive_started() {  // nothing written yet: no release
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  cluster_wait();
}

struct Shared {
  union {
    uint32_t hist[kBins];          // this CTA's counts
    uint2 all[kList];              // the cluster's listed tokens, once the counts are read
  };
  uint32_t total[kBins];           // the cluster's counts
  uint2 list[kList];               // this CTA's listed tokens (|x|'s bits, index)
  union {
    u64 all_w[kList];              // W of `all`
    float queue[kWarps][kQueue];   // |x| of tokens before the bin, before their weights are formed
  };
  u64 post[2][3][kMaxPieces];      // what the pieces' warps told last, and before that
  uint32_t border[2];
  u64 scan_s[kWarps];
  uint32_t scan_n[kWarps];
  float scan_e[kWarps];
  int listed, bin;
  uint32_t before_n;
  float before_e;
  uint32_t sub_n[kThreads], sub_hi[kThreads], sub_lo[kThreads];  // a list's bins: tokens, W by 20-bit digits
  int first_of[kMaxCluster + 1];   // where a CTA's listed tokens lie in `all`
  int sub_bin, few_n;
  u64 sub_before_s;
  uint32_t sub_before_n, sub_count;
  int few[32];
};

// A row as a warp sees it: elements at `base`, 16-byte aligned, of which [skip, end) are the row.
template <typename T>
struct Row {
  const T *base;
  int skip, end;
  int lo, hi;         // this warp's piece, whole vectors (but for the last one's end)
  int per_chunk;      // steps of a chunk
  float chunk_top;    // lane c: the largest logit of chunk c
  float M, inv;
  uint32_t border;    // kept: |x| above the border's, or equal and index up to `last`
  uint32_t last;
  float least;        // and weight at least this

  static constexpr int kN = 16 / sizeof(T);      // elements of a vector
  static constexpr int kVecs = kEach / kN;
  __device__ static float value(T x) {
    if constexpr (sizeof(T) == 2)
      return __uint_as_float((uint32_t)x << 16);
    else
      return x;
  }
  __device__ bool inside(uint32_t d, uint32_t v) const { return d < border || (d == border && v <= last); }
  __device__ float kept(uint32_t d, int v) const {  // weight, 0 where it is not kept
    if (!inside(d, (uint32_t)v)) return 0.f;
    const float w = weight(d);
    return w >= least ? w : 0.f;
  }
  // A lane's vectors of the step at i0: raw, and what a guarded one could not read.
  // Logits of a step's elements [i0, b): those that are not the row's or behind b: -inf.
  __device__ void load(int i0, int b, int lane, float (&x)[kEach]) const {
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int i = i0 + (32 * k + lane) * kN;
      if (i >= skip && i + kN <= b) {
        const uint4 q = __ldg(reinterpret_cast<const uint4 *>(base + i));
#pragma unroll
        for (int e = 0; e < kN; ++e) x[k * kN + e] = value(reinterpret_cast<const T *>(&q)[e]);
      } else {
#pragma unroll
        for (int e = 0; e < kN; ++e)
          x[k * kN + e] = i + e >= skip && i + e < b ? value(base[i + e]) : -CUDART_INF_F;
      }
    }
  }
  // The index of element j of a lane's step at i0.
  __device__ int index(int i0, int j, int lane) const { return i0 + (32 * (j / kN) + lane) * kN + j % kN - skip; }

  // The first step from s on whose chunk is alive.
  __device__ int next(int s, int steps, uint32_t alive) const {
    while (s < steps && !((alive >> (s / per_chunk)) & 1u)) ++s;
    return s;
  }
  // f(logit, index) for this piece's elements in live chunks, one step's loads ahead; g(whether the step is
  // done) after every four.
  template <typename F, typename G>
  __device__ void each(uint32_t alive, int lane, F f, G g) const {
    const int steps = (hi - lo + kStep - 1) / kStep;
    int s = next(0, steps, alive);
    float x[kEach], y[kEach];
    if (s < steps) load(lo + s * kStep, hi, lane, y);
    while (s < steps) {
#pragma unroll
      for (int j = 0; j < kEach; ++j) x[j] = y[j];
      const int at = lo + s * kStep;
      s = next(s + 1, steps, alive);
      if (s < steps) load(lo + s * kStep, hi, lane, y);
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        f(x[j], index(at, j, lane));
        if (j % 4 == 3) g(j == kEach - 1);
      }
    }
  }
  // The chunks that have tokens with |x|'s bits below d.
  __device__ uint32_t alive(uint32_t d) const { return __ballot_sync(0xffffffffu, depth(chunk_top, M, inv) < d); }
};

// A level of bins.  The first: |x| to the nearest 1/64, up to 2,047; finer ones: |x|'s bits d in [lo, hi), bin
// (d - lo) >> shift.
struct Level {
  uint32_t lo, hi;
  int shift;  // -1: the first level
  __device__ static int first_bin(uint32_t d) {
    return (int)(__float_as_uint(__uint_as_float(d) + 131072.f) - 0x48000000u);  // (a last place of 1/64)
  }
  __device__ uint32_t begin(int b) const {
    if (shift >= 0) return min((uint32_t)b << shift, hi - lo) + lo;
    // halfway goes to the even bin
    return b == 0 ? 0u : b == kBins ? kDeep + 1 : __float_as_uint(((float)b - 0.5f) * 0x1p-6f) + (b & 1);
  }
  // an estimate of a bin's weights: the middle's
  __device__ float middle(int b) const {
    return shift < 0 ? expf((float)b * -0x1p-6f) : weight(min(lo + ((uint32_t)b << shift) + ((1u << shift) >> 1), hi));
  }
};

template <typename T>
struct Sampler {
  const SampleArgs &a;
  Shared &sh;
  Row<T> r;
  int cluster, rank, warp, lane, piece, pieces;
  int turn = 0;  // exchanges so far: their buffers alternate
  bool coarse = true;  // sh.total has the first level's counts

  // Tell the cluster up to three numbers of this piece; afterwards all of them are in post.
  template <int kNumbers>
  __device__ void exchange(u64 x, u64 y = 0, u64 z = 0) {
    u64(*p)[kMaxPieces] = sh.post[turn & 1];
    if (lane < cluster) {
      store_remote(remote(&p[0][piece], lane), x);
      if (kNumbers > 1) store_remote(remote(&p[1][piece], lane), y);
      if (kNumbers > 2) store_remote(remote(&p[2][piece], lane), z);
    }
    ++turn;
    cluster_barrier();
  }
  __device__ u64 posted(int k, int i) const { return i < pieces ? sh.post[(turn - 1) & 1][k][i] : 0; }
  // Sums of number k of the last exchange over all pieces, and over those before this one.
  __device__ u64 told(int k) const { return warp_sum(posted(k, lane) + posted(k, lane + 32)); }
  __device__ u64 told_before(int k) const {
    return warp_sum((lane < piece ? posted(k, lane) : 0) + (lane + 32 < piece ? posted(k, lane + 32) : 0));
  }

  // The cluster's counts of each bin, from the CTAs' (each sums a share of them and hands it to all).
  __device__ void add_up() {
    const int share_of = kBins / cluster;
    for (int i = threadIdx.x; i < share_of; i += kThreads) {
      const int b = rank * share_of + i;
      uint32_t n = 0, x[kMaxCluster];
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) x[c] = c < cluster ? load_remote_word(remote(&sh.hist[b], c)) : 0;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) n += x[c];
      for (int c = 0; c < cluster; ++c) store_remote(remote(&sh.total[b], c), n);
    }
    cluster_barrier();
  }

  // The bin at which the running count reaches `many`, or (by_sum) the running estimate e0 + w times all bins'
  // estimate over `all_w`; within [first, last].  sh.before_n and sh.before_e: what lies before it.
  __device__ int seek(const Level &lv, bool by_sum, u64 many, float e0, float w, u64 all_w, int first, int last) {
    constexpr int kMine = kBins / kThreads;
    const int b0 = threadIdx.x * kMine;
    uint32_t n[kMine], n_all = 0;
    float m[kMine], e_all = 0.f;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      n[k] = sh.total[b0 + k];
      m[k] = n[k] ? (float)n[k] * lv.middle(b0 + k) : 0.f;
      n_all += n[k];
      e_all += m[k];
    }
    uint32_t n_run = n_all;
    float e_run = e_all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, n_run, d);
      const float z = __shfl_up_sync(0xffffffffu, e_run, d);
      if (lane >= d) n_run += y, e_run += z;
    }
    if (lane == 31) sh.scan_n[warp] = n_run, sh.scan_e[warp] = e_run;
    if (threadIdx.x == 0) sh.bin = last;
    __syncthreads();
    n_run -= n_all;
    e_run -= e_all;
    float everything = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      if (k < warp) n_run += sh.scan_n[k], e_run += sh.scan_e[k];
      everything += sh.scan_e[k];
    }
    const float e = e0 + w * (everything / (float)all_w);
    const uint32_t n_at = n_run;
    const float e_at = e_run;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      n_run += n[k];
      e_run += m[k];
      if (n[k] && (by_sum ? e_run >= e : n_run >= many)) {
        atomicMin(&sh.bin, max(b0 + k, first));
        break;
      }
    }
    __syncthreads();
    const int bin = sh.bin;
    n_run = n_at;
    e_run = e_at;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      if (b0 + k == bin) sh.before_n = n_run, sh.before_e = e_run;
      n_run += n[k];
      e_run += m[k];
    }
    __syncthreads();
    return bin;
  }

  // ---- lists

  // Append this piece's tokens with |x|'s bits in [from, to), inside the border, to the CTA's list.
  __device__ void append(uint32_t d, int v) {
    const int at = atomicAdd(&sh.listed, 1);
    if (at < kList) sh.list[at] = make_uint2(d, (uint32_t)v);
  }

  // All CTAs' lists in one (number 2 of the last exchange: each piece's tokens): returns how many.
  __device__ int gather() {
    int n = 0, incl;
    if (lane < cluster)
#pragma unroll
      for (int i = 0; i < kWarps; ++i) n += (int)posted(2, lane * kWarps + i);
    incl = n;
#pragma unroll
    for (int d = 1; d < kMaxCluster; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += y;
    }
    const int all = __shfl_sync(0xffffffffu, incl, kMaxCluster - 1);
    if (warp == 0 && lane < kMaxCluster) sh.first_of[lane] = incl - n;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kList / kThreads; ++k) {
      const int i = threadIdx.x + k * kThreads;
      if (i < all) {
        int c = 0;
        while (c + 1 < cluster && sh.first_of[c + 1] <= i) ++c;
        const uint2 q = load_remote(remote(&sh.list[i - sh.first_of[c]], c));
        sh.all[i] = q;
        sh.all_w[i] = whole(weight(q.x));
      }
    }
    __syncthreads();
    return all;
  }

  // Of the list's n tokens that lie inside the border (and weigh `least`), in their order (or by index), the one at
  // which their running number (or the sum of their W) reaches `target`.  base: what the sum begins with; `with`:
  // the sum up to that token, it included (by number: left as it is).  [lo, lo + 2^bits): where its key lies.
  __device__ uint2 pick(int n, bool by_index, bool by_sum, u64 target, u64 base, uint32_t lo, int bits, u64 &with) {
    u64 before_n = 0, before_s = base;
    uint32_t fixed = 0;      // |x|'s bits, once these are down to one value
    bool on_v = by_index, tied = false;
    auto in = [&](int i, uint2 &q, uint32_t &key) {
      q = sh.all[i];
      key = on_v ? q.y : q.x;
      return r.inside(q.x, q.y) && (!tied || q.x == fixed) && !(r.least > 0.f && weight(q.x) < r.least);
    };
    int shift = max(0, bits - 8);
    for (;;) {
      sh.sub_n[threadIdx.x] = sh.sub_hi[threadIdx.x] = sh.sub_lo[threadIdx.x] = 0;
      if (threadIdx.x == 0) sh.sub_bin = kThreads - 1, sh.few_n = 0, sh.sub_count = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < n; i += kThreads) {
        uint2 q;
        uint32_t key;
        if (in(i, q, key) && key - lo < (256u << shift)) {
          const uint32_t b = (key - lo) >> shift;
          atomicAdd(&sh.sub_n[b], 1u);
          if (by_sum) {  // (64-bit atomics on one word hold each other up; a digit's sums stay below 2^31)
            atomicAdd(&sh.sub_hi[b], (uint32_t)(sh.all_w[i] >> 20));
            atomicAdd(&sh.sub_lo[b], (uint32_t)sh.all_w[i] & 0xfffffu);
          }
        }
      }
      __syncthreads();
      const uint32_t my_n = sh.sub_n[threadIdx.x];
      const u64 my_s = ((u64)sh.sub_hi[threadIdx.x] << 20) + sh.sub_lo[threadIdx.x];
      uint32_t n_run = my_n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, n_run, d);
        if (lane >= d) n_run += y;
      }
      u64 s_run = by_sum ? warp_scan(my_s, lane) : 0;
      if (lane == 31) sh.scan_n[warp] = n_run, sh.scan_s[warp] = s_run;
      __syncthreads();
      s_run += before_s;
      for (int k = 0; k < warp; ++k) n_run += sh.scan_n[k], s_run += sh.scan_s[k];
      const u64 at = by_sum ? s_run : before_n + n_run, was = by_sum ? s_run - my_s : before_n + n_run - my_n;
      if (was < target && target <= at) {
        sh.sub_bin = threadIdx.x;
        sh.sub_before_n = n_run - my_n;
        sh.sub_before_s = s_run - my_s;
        sh.sub_count = my_n;
      }
      __syncthreads();
      const int count = (int)sh.sub_count;
      before_n += sh.sub_before_n;
      before_s = sh.sub_before_s;
      lo += (uint32_t)sh.sub_bin << shift;
      if (count <= 32) break;
      if (shift == 0) {  // many of one |x|: by index
        fixed = lo;
        tied = on_v = true;
        lo = 0;
        shift = 14;
      } else {
        shift = max(0, shift - 8);
      }
      __syncthreads();
    }
    // a few: ranked in every warp's lanes
    for (int i = threadIdx.x; i < n; i += kThreads) {
      uint2 q;
      uint32_t key;
      if (in(i, q, key) && key - lo < (1u << shift)) sh.few[atomicAdd(&sh.few_n, 1) & 31] = i;
    }
    __syncthreads();
    const int count = min(sh.few_n, 32), mine = lane < count ? sh.few[lane] : 0;
    const uint2 q = sh.all[mine];
    const u64 w = sh.all_w[mine];
    u64 sum = before_s + w, place = before_n + 1;
    for (int k = 0; k < count; ++k) {
      const uint32_t d = __shfl_sync(0xffffffffu, q.x, k), v = __shfl_sync(0xffffffffu, q.y, k);
      const u64 o = __shfl_sync(0xffffffffu, w, k);
      if (by_index ? v < q.y : d < q.x || (d == q.x && v < q.y)) sum += o, ++place;
    }
    const bool hit = lane < count && (by_sum ? sum - w < target && target <= sum : place == target);
    const uint32_t who = __ballot_sync(0xffffffffu, hit);
    const int l = who ? __ffs(who) - 1 : 0;
    if (by_sum) with = __shfl_sync(0xffffffffu, sum, l);
    const uint2 found = make_uint2(__shfl_sync(0xffffffffu, q.x, l), __shfl_sync(0xffffffffu, q.y, l));
    __syncthreads();
    return found;
  }

  // The sum of W of the list's tokens that lie inside the border (and weigh `least`), and of this piece's alone.
  __device__ u64 list_sum(int n, u64 &mine) {
    u64 x = 0, y = 0;
    for (int j = lane; j < n; j += 32) {
      const uint2 q = sh.all[j];
      if (!r.inside(q.x, q.y) || (r.least > 0.f && weight(q.x) < r.least)) continue;
      const int at = (int)q.y + r.skip;
      x += sh.all_w[j];
      if (at >= r.lo && at < r.hi) y += sh.all_w[j];
    }
    mine = warp_sum(y);
    return warp_sum(x);
  }

  // The border among tokens of one |x| (bits d): the first `ties` of them stay.
  __device__ void rank_ties(uint32_t d, u64 ties, u64 before_here, u64 here) {
    if (before_here < ties && ties <= before_here + here) {
      u64 run = before_here;
      for (int i = r.lo; i < r.hi; i += 32) {
        const int at = i + lane;
        const bool eq = at >= r.skip && at < r.hi && r.inside(d, (uint32_t)(at - r.skip)) &&
                        depth(Row<T>::value(r.base[at]), r.M, r.inv) == d;
        uint32_t who = __ballot_sync(0xffffffffu, eq);
        if (ties <= run + __popc(who)) {
          while (++run < ties) who &= who - 1;
          if (lane < cluster) store_remote(remote(&sh.border[1], lane), (uint32_t)(i + __ffs(who) - 1 - r.skip));
          break;
        }
        run += __popc(who);
      }
    }
    cluster_barrier();
    r.border = d;
    r.last = sh.border[1];
  }

  // The level's counts, of the tokens with |x|'s bits in [from, to).
  __device__ void count(const Level &lv, uint32_t from, uint32_t to) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh.hist[i] = 0;
    __syncthreads();
    r.each(r.alive(to), lane, [&](float l, int) {
      const uint32_t d = depth(l, r.M, r.inv);
      if (d - from < to - from) {
        const int b = lv.shift < 0 ? Level::first_bin(d) : (int)((d - from) >> lv.shift);
        atomicAdd(&sh.hist[b], 1u);
      }
    }, [](bool) {});
    cluster_barrier();
    add_up();
  }

  // Move the border to the last token of the order's first part: the `limit` first ones (by_sum false), or the
  // shortest part whose W sum to `limit` at least (1 .. their sum); S: the sum of all W.  sum: that part's, mine:
  // this piece's share of it.  Returns how many tokens are listed when the list holds all of that part (sum and
  // mine then say nothing where the border is not moved), else 0.
  __device__ int find_border(bool by_sum, u64 limit, u64 S, u64 &sum, u64 &mine) {
    Level lv{0u, 0u, -1};
    int first = 0, last = kBins - 1, tries = 0;
    if (!coarse) count(lv, 0u, kDeep + 1);
    coarse = true;
    int bin = seek(lv, by_sum, limit, 0.f, (float)limit, S, first, last);
    u64 skipped = 0;  // tokens before the level's first bin
    for (;;) {
      if (!by_sum && lv.shift < 0 && bin == kBins - 1) return 0;  // nothing with weight is left out
      const uint32_t to = lv.begin(bin + 1);
      const u64 before = skipped + sh.before_n;
      const float e_before = sh.before_e;
      // the whole first part is listed where it fits
      const bool whole_part = before + sh.total[bin] <= kList;
      const uint32_t from = whole_part ? 0u : lv.begin(bin);
      // ---- exact sums, and the bin's tokens
      if (threadIdx.x == 0) sh.listed = 0;
      __syncthreads();
      Sum above, within;
      uint32_t n = 0;
      int queued = 0;
      float *queue = sh.queue[warp];
      r.each(r.alive(to), lane, [&](float l, int v) {
        const float x = depth_of(l, r.M, r.inv);
        const uint32_t d = __float_as_uint(x);
        // tokens before the bin are packed first: mostly few of a warp's are
        const uint32_t who = __ballot_sync(0xffffffffu, d < from);
        if (d < from) queue[queued + __popc(who & ((1u << lane) - 1))] = x;
        queued += __popc(who);
        if (d - from < to - from && r.inside(d, (uint32_t)v)) {
          within.add(weight(d));
          ++n;
          append(d, v);
        }
      }, [&](bool) {
        __syncwarp();
        while (queued >= 32) above.add(expf(-queue[(queued -= 32) + lane]));
        __syncwarp();
        above.carry();
        within.carry();
      });
      if (lane < queued) above.add(expf(-queue[lane]));
      above.carry();
      const u64 above_here = warp_sum(above.total), here = __reduce_add_sync(0xffffffffu, n);
      exchange<3>(above_here, warp_sum(within.total), here);
      const u64 A = told(0), B = told(1), N = told(2);
      if (by_sum && !(A < limit && limit <= A + B)) {
        // the estimate was off: on from the exact sum, after some tries by halves
        if (A >= limit)
          last = bin - 1;
        else
          first = bin + 1;
        if (first > last) return 0;  // (cannot be)
        if (++tries < 5) {
          // (of a whole part the sum ends at the bin's end)
          const float off = A >= limit ? -(float)(A - limit) : whole_part ? (float)(limit - B) : (float)(limit - A);
          bin = seek(lv, true, 0, e_before, off, S, first, last);
        } else {
          const int middle = (first + last) / 2;
          bin = seek(lv, true, 0, 0.f, 0.f, S, middle, middle);
        }
        continue;
      }
      if (N <= kList) {
        const int listed = gather();
        const uint2 b = pick(listed, false, by_sum, by_sum ? limit : limit - (whole_part ? 0 : before), A, from,
                             32 - __clz((int)(to - from - 1) | 255), sum);
        r.border = b.x;
        r.last = b.y;
        sum = A + list_sum(listed, mine);
        mine += above_here;
        return whole_part ? listed : 0;
      }
      if (to - from == 1) {
        const u64 w = whole(weight(from)), ties = by_sum ? (limit - A + w - 1) / w : limit - before;
        const u64 N_before = told_before(2);
        rank_ties(from, ties, N_before, here);
        sum = A + ties * w;
        mine = above_here + (ties > N_before ? min(ties - N_before, here) : 0) * w;
        return 0;
      }
      // ---- finer bins
      skipped = before;
      lv = Level{from, to, max(0, 21 - __clz((int)(to - from - 1)))};
      coarse = false;
      count(lv, from, to);
      first = tries = 0;
      last = (int)((to - 1 - from) >> lv.shift);
      S = B > 0 ? B : 1;  // (without what top-k left out: a first guess that this puts off is tried again)
      bin = seek(lv, by_sum, limit - skipped, 0.f, by_sum ? (float)(limit - A) : 0.f, S, first, last);
    }
  }
};

}  // namespace

template <typename T>
__global__ void __launch_bounds__(kThreads, kPerSm) pskv_sample(const SampleArgs a, const int cluster) {
  __shared__ Shared sh;
  Sampler<T> s{a, sh};
  Row<T> &r = s.r;
  s.cluster = cluster;
  s.rank = (int)cluster_rank();
  s.warp = threadIdx.x >> 5;
  s.lane = threadIdx.x & 31;
  s.pieces = cluster * kWarps;
  s.piece = s.rank * kWarps + s.warp;
  const int row = blockIdx.x / cluster, lane = s.lane, warp = s.warp;
  cluster_arrive_started();
  pdl_wait();
  pdl_launch_dependents();
  // ---- the row's pieces, from the 16-byte boundary before it
  const T *l = static_cast<const T *>(a.logits) + row * a.logits_row;
  r.skip = (int)((reinterpret_cast<uintptr_t>(l) & 15) / sizeof(T));
  r.base = l - r.skip;
  r.end = r.skip + a.vocab;
  constexpr int kN = Row<T>::kN;
  const int seg = ((r.end + s.pieces - 1) / s.pieces + kN - 1) / kN * kN;
  r.lo = min(s.piece * seg, r.end);
  r.hi = min(r.lo + seg, r.end);
  r.per_chunk = max(1, (seg + 32 * kStep - 1) / (32 * kStep));
  const int req = row / a.per_request;
  float heat = a.temperature ? a.temperature[req] : 1.f, p = a.top_p ? a.top_p[req] : 1.f;
  float least = a.min_p ? a.min_p[req] : 0.f;
  int k = a.top_k ? a.top_k[req] : 0;
  const float u = a.u ? a.u[row] : 0.f;
  // ---- M
  r.chunk_top = -CUDART_INF_F;
  {
    float chunk = -CUDART_INF_F;
    int left = r.per_chunk, c = 0;
    r.each(~0u, lane, [&](float x, int) { chunk = fmaxf(chunk, x); }, [&](bool done) {
      if (!done || --left > 0) return;
      chunk = warp_max(chunk);
      if (lane == c) r.chunk_top = chunk;
      chunk = -CUDART_INF_F;
      left = r.per_chunk;
      ++c;
    });
    if (left < r.per_chunk) {
      chunk = warp_max(chunk);
      if (lane == c) r.chunk_top = chunk;
    }
  }
  float top = warp_max(r.chunk_top);
  __syncwarp();
  cluster_wait();  // the others have started too
  // (the settings are the ones that the first piece read: the CTAs go the same way whoever writes to them meanwhile)
  s.template exchange<3>((u64)__float_as_uint(top), (u64)__float_as_uint(heat) << 32 | __float_as_uint(p),
                         (u64)__float_as_uint(least) << 32 | (uint32_t)k);
  const u64 *tops = sh.post[0][0];
  heat = __uint_as_float((uint32_t)(sh.post[0][1][0] >> 32));
  p = __uint_as_float((uint32_t)sh.post[0][1][0]);
  least = __uint_as_float((uint32_t)(sh.post[0][2][0] >> 32));
  k = (int)(uint32_t)sh.post[0][2][0];
  if (lane < s.pieces) top = fmaxf(top, __uint_as_float((uint32_t)tops[lane]));
  if (lane + 32 < s.pieces) top = fmaxf(top, __uint_as_float((uint32_t)tops[lane + 32]));
  top = warp_max(top);
  const bool empty = top == -CUDART_INF_F;
  if (empty && s.rank == 0 && threadIdx.x == 0) {
    if (a.tokens) a.tokens[row] = -1;
    raise_fault(a.status, PSKV_FAULT_EMPTY_ROW);
  }
  const bool endless = top == CUDART_INF_F;
  r.M = endless ? FLT_MAX : top;
  r.inv = __fdiv_rn(1.f, heat);
  r.border = kDeep;
  r.last = UINT_MAX;
  r.least = least > 0.f ? fminf(least, 1.f) : 0.f;
  u64 total = 1;
  int listed = 0;  // the list's tokens, where it holds all that is kept
  if (empty) {
    r.border = r.last = 0;
  } else if (!(heat > 0.f) || r.inv == CUDART_INF_F) {
    // ---- the likeliest token, the lowest index of M
    r.inv = endless ? CUDART_INF_F : 1.f;
    uint32_t at = UINT_MAX;
    r.each(r.alive(1u), lane, [&](float x, int v) { at = x == top ? min(at, (uint32_t)v) : at; }, [](bool) {});
    s.template exchange<1>((u64)__reduce_min_sync(0xffffffffu, at));
    const u64 *ats = sh.post[1][0];
    if (lane < s.pieces) at = min(at, (uint32_t)ats[lane]);
    if (lane + 32 < s.pieces) at = min(at, (uint32_t)ats[lane + 32]);
    at = __reduce_min_sync(0xffffffffu, at);
    r.border = 0;
    r.last = at;
    total = 1ull << 40;
    if (a.tokens && s.rank == 0 && threadIdx.x == 0) a.tokens[row] = (int)at;
  } else {
    const bool some = k > 0 && k < a.vocab, part = p < 1.f, filters = some || part;
    if (endless) r.inv = CUDART_INF_F;
    // ---- the sum of W, and where the tokens lie
    if (filters) {
      for (int i = threadIdx.x; i < kBins; i += kThreads) sh.hist[i] = 0;
      __syncthreads();
    }
    Sum all;
    r.each(~0u, lane, [&](float x, int) {
      const uint32_t d = depth(x, r.M, r.inv);
      const float w = weight(d);
      if (filters) {
        all.add(w);
        atomicAdd(&sh.hist[Level::first_bin(d)], 1u);
      } else {
        all.add(w >= r.least ? w : 0.f);
      }
    }, [&](bool done) { if (done) all.carry(); });
    u64 mine = warp_sum(all.total);
    s.template exchange<1>(mine);
    total = s.told(0);
    if (filters) {
      s.add_up();
      const u64 S = total;
      const float least_w = r.least;  // (min_p comes last)
      r.least = 0.f;
      if (some) listed = s.find_border(false, (u64)k, S, total, mine);
      if (part) {
        const u64 limit = max(share(p, total), 1ull);
        if (listed) {
          const uint2 b = s.pick(listed, false, true, limit, 0, 0u, 31, total);
          r.border = b.x;
          r.last = b.y;
        } else {
          listed = s.find_border(true, limit, S, total, mine);
        }
      }
      r.least = least_w;
      if (listed) {
        if (r.least > 0.f) total = s.list_sum(listed, mine);
      } else {
        if (r.least > 0.f) {
          Sum kept;
          r.each(r.alive(r.border + 1), lane, [&](float x, int v) { kept.add(r.kept(depth(x, r.M, r.inv), v)); },
                 [&](bool done) { if (done) kept.carry(); });
          mine = warp_sum(kept.total);
        }
        s.template exchange<1>(mine);
        total = s.told(0);
      }
    }
    // ---- the draw: where the running sum passes u's share
    const u64 thr = u >= 1.f ? total - 1 : share(u, total);
    if (a.tokens && listed) {
      u64 with;
      const uint2 t = s.pick(listed, true, true, thr + 1, 0, 0u, 22, with);
      if (s.rank == 0 && threadIdx.x == 0) a.tokens[row] = (int)t.y;
    } else if (a.tokens) {
      const u64 before = s.told_before(0);
      if (threadIdx.x == 0) sh.bin = -1;
      __syncthreads();
      if (lane == 0 && before <= thr && thr < before + mine) {
        sh.bin = s.piece;
        sh.sub_before_s = thr - before;
      }
      __syncthreads();
      const int hit = sh.bin;
      if (hit >= 0) {
        // its CTA: an eighth a warp
        const u64 left = sh.sub_before_s;
        const int p0 = min(hit * seg, r.end), p1 = min(p0 + seg, r.end);
        const int sub = ((p1 - p0 + kWarps - 1) / kWarps + kN - 1) / kN * kN;
        r.lo = min(p0 + warp * sub, p1);
        r.hi = min(r.lo + sub, p1);
        r.per_chunk = INT_MAX;
        Sum kept;
        r.each(1u, lane, [&](float x, int v) { kept.add(r.kept(depth(x, r.M, r.inv), v)); }, [&](bool done) { if (done) kept.carry(); });
        const u64 own = warp_sum(kept.total);
        if (lane == 0) sh.scan_s[warp] = own;
        __syncthreads();
        u64 at = 0;
        for (int i = 0; i < warp; ++i) at += sh.scan_s[i];
        if (at <= left && left < at + own) {
          for (int i0 = r.lo; i0 < r.hi && at <= left; i0 += 32 * kN) {
            const int i = i0 + lane * kN;
            u64 w[kN], w_all = 0;
#pragma unroll
            for (int e = 0; e < kN; ++e) {
              const bool real = i + e >= r.skip && i + e < r.hi;
              const float x = real ? Row<T>::value(r.base[i + e]) : -CUDART_INF_F;
              w[e] = real ? whole(r.kept(depth(x, r.M, r.inv), i + e - r.skip)) : 0;
              w_all += w[e];
            }
            const u64 incl = at + warp_scan(w_all, lane);
            u64 run = incl - w_all;
#pragma unroll
            for (int e = 0; e < kN; ++e) {
              if (run <= left && left < run + w[e]) a.tokens[row] = i + e - r.skip;
              run += w[e];
            }
            at = __shfl_sync(0xffffffffu, incl, 31);
          }
        }
        r.lo = min(s.piece * seg, r.end);
        r.hi = min(r.lo + seg, r.end);
      }
    }
  }
  if (a.probs) {
    // W / S, W being floats: 1 / S as a float pair
    const double inv = 1.0 / (double)total;
    const float hi = (float)inv, lo = (float)(inv - (double)hi);
    const size_t out = (size_t)row * a.vocab;
    auto put = [&](int v, float w) {
      const float q = fmaf(w, hi, w * lo);
      if (a.probs_dtype == PSKV_DTYPE_BF16)
        static_cast<__nv_bfloat16 *>(a.probs)[out + v] = __float2bfloat16_rn(q);
      else
        static_cast<float *>(a.probs)[out + v] = q;
    };
    for (int i = max(r.lo, r.skip) + lane; i < r.hi; i += 32) {
      const int v = i - r.skip;
      float w = 0.f;
      if (!empty && !listed) {
        const uint32_t d = depth(Row<T>::value(r.base[i]), r.M, r.inv);
        if (r.inside(d, (uint32_t)v)) w = (float)whole(r.kept(d, v));
      }
      put(v, w);
    }
    __syncwarp();
    for (int j = lane; j < listed; j += 32) {
      const uint2 q = sh.all[j];
      const int i = (int)q.y + r.skip;
      if (i >= r.lo && i < r.hi) put((int)q.y, (float)whole(r.kept(q.x, (int)q.y)));
    }
  }
}

namespace {

template <typename T>
cudaError_t launch(const SampleArgs &a, int cluster, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.rows * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, pskv_sample<T>, a, cluster);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, int sms, cudaStream_t s) {
  // the largest cluster with which all rows run at once
  int cluster = kMaxCluster;
  while (cluster > 1 && (long long)a.rows * cluster > (long long)kPerSm * sms) cluster /= 2;
  return a.dtype == PSKV_DTYPE_BF16 ? launch<uint16_t>(a, cluster, s) : launch<float>(a, cluster, s);
}

}  // namespace pskv
