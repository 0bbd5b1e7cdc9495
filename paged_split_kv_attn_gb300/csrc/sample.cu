// sample.cu -- sampling from logits with temperature, top-k, top-p and min-p.
//
// For a row l with largest value M: x = (l - M) / T in f32 steps, w = expf(x), W = w rounded to the
// nearest multiple of 2^-40.  Tokens are ordered by x, then by index; what top-k and top-p keep is a
// first part of that order, so it is given by a border: the last token kept, (|x|, index).
// W are whole numbers and sums 64-bit integers, so nothing depends on how the work is split.
//
// A cluster of up to eight CTAs takes a row, each warp a piece of the vocabulary.  The row is
// read from memory once, for M; the later passes find it in L1 and L2 (staged in shared memory, fewer
// CTAs fit on an SM: 64 rows of 131,072 would take two waves).  Passes:
//   1  M
//   2  the sum of W, and a histogram of |x| by its leading bits (256 bins an octave from 2^-3 to 2^5:
//      counts only, a shared-memory atomic a token, beside the exponentials)
//   3  the bin that holds the border: from the counts (top-k), or by the bins' estimated weight
//      (top-p).  The pass sums W exactly over what lies before the bin and lists the bin's own tokens.
//      An estimate that was off shows in the exact sum, and the next bin is tried from there
//   -  the bin's tokens (some hundred) are ranked against each other.  More than fit in the list: the
//      bin is cut into 2,048 finer ones (pass 2's counts again, for its tokens alone), down to a
//      single |x|, whose tokens' border is a matter of counting
//   4  the drawn token's piece again, and the probabilities where they are asked for.
// Between passes the warps' results cross the cluster through distributed shared memory, one barrier each.
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
constexpr uint32_t kFirst = 0x3e000000u >> 15;  // the first level's bin 1: |x| from 2^-3, by its 17 leading bits

// The bits of |x| for a logit, M the row's largest and inv = 1 / T: they go up as x falls.  No weight: infinity's.
__device__ __forceinline__ uint32_t depth(float l, float M, float inv) {
  const float x = __fmul_rn(__fsub_rn(l, M), inv);
  return l == M ? 0u : __float_as_uint(fminf(fabsf(x), CUDART_INF_F));  // (a NaN: infinity)
}
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
  uint2 list[kList];               // this CTA's listed tokens (|x|'s bits, index): kList / cluster of them at most
  u64 all_w[kList];                // their W
  u64 post[2][3][kMaxPieces];      // what the pieces' warps told last, and before that
  uint32_t border[2];
  u64 border_sum;
  u64 part[kWarps];
  uint32_t scan_n[kWarps];
  float scan_e[kWarps];
  int listed, bin;
  uint32_t before_n;
  float before_e;
};

// A row as a warp sees it: elements at `base`, 16-byte aligned, of which [skip, skip + vocab) are the row.
template <typename T>
struct Row {
  const T *base;
  int skip, end;      // the row's elements
  int lo, hi;         // this warp's piece, whole vectors (but for the last one's end)
  float M, inv;
  uint32_t border;    // kept: |x| above the border's, or equal and index up to `last`
  uint32_t last;
  float least;        // and weight at least this

  static constexpr int kN = 16 / sizeof(T);  // elements of a vector
  __device__ static float value(T x) {
    if constexpr (sizeof(T) == 2)
      return __uint_as_float((uint32_t)x << 16);
    else
      return x;
  }
  __device__ bool inside(uint32_t d, int v) const { return d < border || (d == border && (uint32_t)v <= last); }
  __device__ float kept(uint32_t d, int v) const {  // weight, 0 where it is not kept
    if (!inside(d, v)) return 0.f;
    const float w = weight(d);
    return w >= least ? w : 0.f;
  }
  // Logits of a vector's elements; those that are not the row's: -inf.
  __device__ void load(int i, float (&x)[kN]) const {
    if (i >= skip && i + kN <= end) {
      const uint4 q = __ldg(reinterpret_cast<const uint4 *>(base + i));
#pragma unroll
      for (int e = 0; e < kN; ++e) x[e] = value(reinterpret_cast<const T *>(&q)[e]);
    } else {
#pragma unroll
      for (int e = 0; e < kN; ++e) x[e] = i + e >= skip && i + e < end ? value(base[i + e]) : -CUDART_INF_F;
    }
  }
  // f(logit, index) for the elements [a, b) (a at a vector), kDepth vectors of a lane in flight; g() after each step.
  template <int kDepth, typename F, typename G>
  __device__ void each(int a, int b, int lane, F f, G g) const {
    for (int i0 = a; i0 < b; i0 += 32 * kN * kDepth) {
      float x[kDepth][kN];
#pragma unroll
      for (int k = 0; k < kDepth; ++k) {
        const int i = i0 + (32 * k + lane) * kN;
        if (i < b)
          load(i, x[k]);
        else
#pragma unroll
          for (int e = 0; e < kN; ++e) x[k][e] = -CUDART_INF_F;
      }
#pragma unroll
      for (int k = 0; k < kDepth; ++k)
#pragma unroll
        for (int e = 0; e < kN; ++e) f(x[k][e], i0 + (32 * k + lane) * kN + e - skip);
      g();
    }
  }
};

// A level of bins: |x|'s bits d in [lo, hi) belong to bin (d - lo) >> shift; the first level's bins are kFirst's.
struct Level {
  uint32_t lo, hi;
  int shift;  // 0..20, or -1: the first level
  __device__ int bin(uint32_t d) const {
    return shift < 0 ? min(max((int)(d >> 15) - (int)kFirst + 1, 0), kBins - 1) : (int)((d - lo) >> shift);
  }
  __device__ uint32_t begin(int b) const {
    return shift < 0 ? (b == 0 ? 0u : (kFirst + b - 1) << 15) : min((uint32_t)b << shift, hi - lo) + lo;
  }
  // an estimate of a bin's weights: the middle's
  __device__ float middle(int b) const {
    const uint32_t a = begin(b), z = begin(b + 1);
    return weight(a == 0 ? __float_as_uint(0.5f * __uint_as_float(z)) : a + (z - a) / 2);
  }
};

template <typename T>
struct Sampler {
  const SampleArgs &a;
  Shared &sh;
  Row<T> r;
  int cluster, rank, warp, lane, piece, pieces;
  int turn = 0;  // exchanges so far: their buffers alternate

  // Tell the cluster up to three numbers of this piece; afterwards `told(k)` holds everybody's.
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
  // Sums of number k of the last exchange over all pieces, and over those before this one.
  __device__ void told(int k, u64 &all, u64 &before) const {
    const u64 *p = sh.post[(turn - 1) & 1][k];
    const u64 x0 = lane < pieces ? p[lane] : 0, x1 = lane + 32 < pieces ? p[lane + 32] : 0;
    all = warp_sum(x0 + x1);
    before = warp_sum((lane < piece ? x0 : 0) + (lane + 32 < piece ? x1 : 0));
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
    constexpr int kEach = kBins / kThreads;
    const int b0 = threadIdx.x * kEach;
    uint32_t n[kEach], n_all = 0;
    float m[kEach], e_all = 0.f;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
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
    for (int k = 0; k < kWarps; ++k) {
      if (k < warp) n_run += sh.scan_n[k], e_run += sh.scan_e[k];
      everything += sh.scan_e[k];
    }
    const float e = e0 + w * (everything / (float)all_w);
    const uint32_t n_at = n_run;
    const float e_at = e_run;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
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
    for (int k = 0; k < kEach; ++k) {
      if (b0 + k == bin) sh.before_n = n_run, sh.before_e = e_run;
      n_run += n[k];
      e_run += m[k];
    }
    __syncthreads();
    return bin;
  }

  // Tokens that CTA c listed in the last pass.
  __device__ int listed(int c) const {
    const u64 *counts = sh.post[(turn - 1) & 1][2];
    int n = 0;
    for (int i = 0; i < kWarps; ++i) n += (int)counts[c * kWarps + i];
    return n;
  }

  // The border among the listed tokens (A: the sum before them, `before` tokens): each CTA ranks its own against all.
  __device__ void rank_listed(bool by_sum, u64 limit, u64 A, u64 before, u64 above_here, u64 &part_sum, u64 &mine) {
    int all = 0, first = 0;
    for (int c = 0; c < cluster; ++c) {
      const int n = listed(c);
      if (c == rank) first = all;
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint2 q = load_remote(remote(&sh.list[i], c));
        sh.all[all + i] = q;
        sh.all_w[all + i] = whole(weight(q.x));
      }
      all += n;
    }
    __syncthreads();
    const int own = listed(rank);
    for (int j = first + warp; j < first + own; j += kWarps) {
      const uint2 q = sh.all[j];
      u64 w = 0;
      uint32_t n = 0;
      for (int i = lane; i < all; i += 32) {
        const uint2 o = sh.all[i];
        const bool less = o.x < q.x || (o.x == q.x && o.y < q.y);
        n += less;
        w += less ? sh.all_w[i] : 0;
      }
      w = A + warp_sum(w);
      n = __reduce_add_sync(0xffffffffu, n);
      const u64 with = w + sh.all_w[j];
      if ((by_sum ? w < limit && limit <= with : before + n + 1 == limit) && lane < cluster) {
        store_remote(remote(&sh.border[0], lane), q.x);
        store_remote(remote(&sh.border[1], lane), q.y);
        store_remote(remote(&sh.border_sum, lane), with);
      }
    }
    cluster_barrier();
    r.border = sh.border[0];
    r.last = sh.border[1];
    part_sum = sh.border_sum;
    u64 x = 0;
    for (int j = first + lane; j < first + own; j += 32) {
      const uint2 q = sh.all[j];
      const int at = (int)q.y + r.skip;
      if (at >= r.lo && at < r.hi && r.inside(q.x, (int)q.y)) x += sh.all_w[j];
    }
    mine = above_here + warp_sum(x);
  }

  // The border among tokens of one |x| (bits d): the first `ties` of them stay.
  __device__ void rank_ties(uint32_t d, u64 ties, u64 before_here, u64 here) {
    if (before_here < ties && ties <= before_here + here) {
      u64 run = before_here;
      for (int i = r.lo; i < r.hi; i += 32) {
        const int at = i + lane;
        const bool eq = at >= r.skip && at < r.hi && r.inside(d, at - r.skip) &&
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

  // Move the border to the last token of the order's first part: the `limit` first ones (by_sum false), or the
  // shortest part whose W sum to `limit` at least (1 .. their sum); S: the sum of all W.  part_sum: that part's sum,
  // mine: this piece's share of it.  False: nothing with weight is left out, the border stays.
  __device__ bool find_border(bool by_sum, u64 limit, u64 S, u64 &part_sum, u64 &mine) {
    Level lv{0u, 0u, -1};
    int first = 0, last = kBins - 1, tries = 0;
    int bin = seek(lv, by_sum, limit, 0.f, (float)limit, S, first, last);
    u64 skipped = 0;  // tokens before the level's first bin
    for (;;) {
      if (!by_sum && lv.shift < 0 && bin == kBins - 1) return false;
      const uint32_t from = lv.begin(bin), to = lv.begin(bin + 1);
      const u64 before = skipped + sh.before_n;
      const float e_before = sh.before_e;
      // ---- exact sums, and the bin's tokens
      if (threadIdx.x == 0) sh.listed = 0;
      __syncthreads();
      const int room = kList / cluster;
      Sum above, within;
      uint32_t n = 0;
      r.template each<2>(r.lo, r.hi, lane, [&](float l, int v) {
        const uint32_t d = depth(l, r.M, r.inv);
        if (d < from) above.add(weight(d));
        if (d - from < to - from && r.inside(d, v)) {
          within.add(weight(d));
          ++n;
          const int at = atomicAdd(&sh.listed, 1);
          if (at < room) sh.list[at] = make_uint2(d, (uint32_t)v);
        }
      }, [&] { above.carry(), within.carry(); });
      const u64 above_here = warp_sum(above.total), here = __reduce_add_sync(0xffffffffu, n);
      exchange<3>(above_here, warp_sum(within.total), here);
      u64 A, B, N, N_before, other;
      told(0, A, other);
      told(1, B, other);
      told(2, N, N_before);
      if (by_sum && !(A < limit && limit <= A + B)) {
        // the estimate was off: on from the exact sum, after some tries by halves
        if (A >= limit)
          last = bin - 1;
        else
          first = bin + 1;
        if (first > last) return false;  // (cannot be)
        if (++tries < 5) {
          const float off = A >= limit ? -(float)(A - limit) : (float)(limit - A);
          bin = seek(lv, true, 0, e_before, off, S, first, last);
        } else {
          const int middle = (first + last) / 2;
          bin = seek(lv, true, 0, 0.f, 0.f, S, middle, middle);
        }
        continue;
      }
      bool fits = true;
      for (int c = 0; c < cluster; ++c) fits &= listed(c) <= room;
      if (fits) {
        rank_listed(by_sum, limit, A, before, above_here, part_sum, mine);
        return true;
      }
      if (to - from == 1) {
        const u64 w = whole(weight(from)), ties = by_sum ? (limit - A + w - 1) / w : limit - before;
        rank_ties(from, ties, N_before, here);
        part_sum = A + ties * w;
        mine = above_here + (ties > N_before ? min(ties - N_before, here) : 0) * w;
        return true;
      }
      // ---- finer bins
      skipped = before;
      lv = Level{from, to, max(0, 21 - __clz((int)(to - from - 1)))};
      for (int i = threadIdx.x; i < kBins; i += kThreads) sh.hist[i] = 0;
      __syncthreads();
      r.template each<2>(r.lo, r.hi, lane, [&](float l, int v) {
        const uint32_t d = depth(l, r.M, r.inv);
        if (d - from < to - from) atomicAdd(&sh.hist[lv.bin(d)], 1u);
      }, [] {});
      cluster_barrier();
      add_up();
      first = tries = 0;
      last = lv.bin(to - 1);
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
  const int req = row / a.per_request;
  float heat = a.temperature ? a.temperature[req] : 1.f, p = a.top_p ? a.top_p[req] : 1.f;
  float least = a.min_p ? a.min_p[req] : 0.f;
  int k = a.top_k ? a.top_k[req] : 0;
  const float u = a.u ? a.u[row] : 0.f;
  // ---- M
  float top = -CUDART_INF_F;
  r.template each<4>(r.lo, r.hi, lane, [&](float x, int) { top = fmaxf(top, x); }, [] {});
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
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
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
  const bool empty = top == -CUDART_INF_F;
  if (empty && s.rank == 0 && threadIdx.x == 0) {
    if (a.tokens) a.tokens[row] = -1;
    raise_fault(a.status, PSKV_FAULT_EMPTY_ROW);
  }
  r.M = top;
  r.inv = __fdiv_rn(1.f, heat);
  r.border = 0x7f800000u;
  r.last = UINT_MAX;
  r.least = least > 0.f ? fminf(least, 1.f) : 0.f;
  u64 total = 1;
  if (empty) {
  } else if (!(heat > 0.f) || r.inv == CUDART_INF_F) {
    // ---- the likeliest token, the lowest index of M
    r.inv = 1.f;
    uint32_t at = UINT_MAX;
    r.template each<2>(r.lo, r.hi, lane, [&](float x, int v) { at = x == top ? min(at, (uint32_t)v) : at; }, [] {});
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
    // ---- the sum of W, and where the tokens lie
    if (filters) {
      for (int i = threadIdx.x; i < kBins; i += kThreads) sh.hist[i] = 0;
      __syncthreads();
    }
    const Level coarse{0u, 0u, -1};
    Sum sum;
    if (filters)
      r.template each<2>(r.lo, r.hi, lane, [&](float x, int) {
        const uint32_t d = depth(x, r.M, r.inv);
        sum.add(weight(d));
        const int b = coarse.bin(d);
        if (b < kBins - 1) atomicAdd(&sh.hist[b], 1u);  // (behind lies no weight)
      }, [&] { sum.carry(); });
    else
      r.template each<2>(r.lo, r.hi, lane, [&](float x, int) {
        const float w = weight(depth(x, r.M, r.inv));
        sum.add(w >= r.least ? w : 0.f);
      }, [&] { sum.carry(); });
    u64 mine = warp_sum(sum.total), before;
    s.template exchange<1>(mine);
    s.told(0, total, before);
    if (filters) {
      s.add_up();
      const u64 S = total;
      if (some) s.find_border(false, (u64)k, S, total, mine);
      if (part) s.find_border(true, max(share(p, total), 1ull), S, total, mine);
      if (r.least > 0.f) {
        Sum kept;
        r.template each<2>(r.lo, r.hi, lane, [&](float x, int v) { kept.add(r.kept(depth(x, r.M, r.inv), v)); },
                           [&] { kept.carry(); });
        mine = warp_sum(kept.total);
      }
      s.template exchange<1>(mine);
      s.told(0, total, before);
    }
    // ---- the draw: the piece in which the running sum passes u's share
    if (a.tokens) {
      const u64 thr = u >= 1.f ? total - 1 : share(u, total);
      if (threadIdx.x == 0) sh.bin = -1;
      __syncthreads();
      if (lane == 0 && before <= thr && thr < before + mine) {
        sh.bin = s.piece;
        sh.border_sum = thr - before;
      }
      __syncthreads();
      const int hit = sh.bin;
      if (hit >= 0) {
        // its CTA: an eighth a warp
        const u64 left = sh.border_sum;
        const int p0 = min(hit * seg, r.end), p1 = min(p0 + seg, r.end);
        const int sub = ((p1 - p0 + kWarps - 1) / kWarps + kN - 1) / kN * kN;
        const int s0 = min(p0 + warp * sub, p1), s1 = min(s0 + sub, p1);
        Sum kept;
        r.template each<1>(s0, s1, lane, [&](float x, int v) { kept.add(r.kept(depth(x, r.M, r.inv), v)); },
                           [&] { kept.carry(); });
        const u64 own = warp_sum(kept.total);
        if (lane == 0) sh.part[warp] = own;
        __syncthreads();
        u64 at = 0;
        for (int i = 0; i < warp; ++i) at += sh.part[i];
        if (at <= left && left < at + own) {
          for (int i0 = s0; i0 < s1; i0 += 32 * kN) {
            float x[kN];
            u64 w[kN], w_all = 0;
            const int i = i0 + lane * kN;
            if (i < s1) r.load(i, x);
#pragma unroll
            for (int e = 0; e < kN; ++e) {
              w[e] = i < s1 ? whole(r.kept(depth(x[e], r.M, r.inv), i + e - r.skip)) : 0;
              w_all += w[e];
            }
            const u64 incl = at + warp_scan(w_all, lane);
            u64 run = incl - w_all;
            if (run <= left && left < incl) {
#pragma unroll
              for (int e = 0; e < kN; ++e) {
                if (run <= left && left < run + w[e]) a.tokens[row] = i + e - r.skip;
                run += w[e];
              }
            }
            at = __shfl_sync(0xffffffffu, incl, 31);
            if (at > left) break;
          }
        }
      }
    }
  }
  if (a.probs) {
    // W / S, W being floats: 1 / S as a float pair
    const double inv = empty ? 0.0 : 1.0 / (double)total;
    const float hi = (float)inv, lo = (float)(inv - (double)hi);
    const size_t out = (size_t)row * a.vocab;
    for (int i = max(r.lo, r.skip) + lane; i < r.hi; i += 32) {
      const int v = i - r.skip;
      float w = 0.f;
      if (!empty) {
        const uint32_t d = depth(Row<T>::value(r.base[i]), r.M, r.inv);
        if (r.inside(d, v)) w = (float)whole(r.kept(d, v));
      }
      const float q = fmaf(w, hi, w * lo);
      if (a.probs_dtype == PSKV_DTYPE_BF16)
        static_cast<__nv_bfloat16 *>(a.probs)[out + v] = __float2bfloat16_rn(q);
      else
        static_cast<float *>(a.probs)[out + v] = q;
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
