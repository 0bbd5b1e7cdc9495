// sample.cu -- sampling from logits with temperature, top-k, top-p and min-p.
//
// For a row l with largest value M: x = (l - M) / T in f32 steps, w = expf(x), W = w rounded to the
// nearest multiple of 2^-40.  Tokens are ordered by x, then by index; what top-k and top-p keep is a
// first part of that order, so it is given by a border: the last token kept, (|x|, index).
// W are whole numbers and sums 64-bit integers, so nothing depends on how the work is split.
//
// A cluster of up to eight CTAs takes a row, each warp a piece of the vocabulary.  The row is
// read from memory once, for M; later passes find it in shared memory where the pieces fit (rows few or short), else
// in L1 and L2 (64 rows of 131,072 f32 staged in shared memory would take two waves).
//   1  M, and the largest logit of each of a piece's 32 chunks: later passes leave out chunks below what they look for
//   2  the sum of W, and a histogram of |x| in steps of 1/64 (counts: a shared-memory atomic a token,
//      beside the exponentials)
//   3  the bin that holds the border: by the counts (top-k), or by the bins' estimated weight (top-p); each CTA
//      adds up a share of the bins and tells all, which then find the border alike.  The pass sums W exactly over what
//      lies before the bin and lists the bin's own tokens; or, where they are few enough, all tokens up to the bin's
//      end.  An estimate that was off shows in the exact sums, and another bin is tried from there.  A bin that does not
//      fit the list is cut into 2,048 finer ones, down to a single |x|, whose tokens' border is a matter of counting.
//      The listed tokens go to the first CTA, by index.  It finds the border among them (up to 64: each compared
//      with all; more: 256 bins of a token's key at a time, |x|'s bits, then the index).  Where they are all
//      that is kept, it finds top-p's border and draws from them, too, and the other CTAs are done
//   4  else the drawn token's piece again; and the probabilities where they are asked for.
// Between passes the warps' results cross the cluster through distributed shared memory, one barrier each.
//
// What bounds it (device time, calls one after the other; stages by clock readings in each row's first CTA).  Without top-k and
// top-p (64 x 131,072 f32 16.4 us, 2.0 TB/s; 256 x 32,001 16.7) reading and computing take turns, as all rows are resident and
// begin at once: M 3.4 us, the exponentials and their sums 5.7, two exchanges 3.9, the draw 0.9 to 1.9, launch and start 2;
// 40 warp instructions for 32 tokens over the whole call, issue slots 44 % busy.
// top-p over weights that are spread out (64 x 131,072: 40.3 us): M 3.5, sum and histogram 7.2, the list's pass with its
// exponentials again 7.5; eight cluster barriers with their exchanges 14, under 1 us each where nothing is late and nothing is
// to be sent; bins, list and border sought 5.7; the draw 1.  One row of 32,001 with top-k, top-p and min-p
// (12.7 us) is that chain alone, and the first fetch of its code: hence loops that are not unrolled wherever speed
// does not count (134 -> 97 KB of code at the time: 64 x 131,072 49 -> 45 us, a row 16 -> 15).
// Temperature 0 seeks M's lowest index token by token: 64 x 131,072 17.2 us, 600 rows (one CTA each) 278 against 148 of a draw.
#include <float.h>
#include <limits.h>
#include <math_constants.h>

#include <algorithm>
#include <atomic>

#include "pskv_internal.cuh"
#include "sample_search.h"
#include "tree.h"

namespace pskv {

namespace {

using namespace border;

constexpr int kMaxCluster = 8;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxPieces = kMaxCluster * kWarps;
constexpr int kPerSm = 4;        // CTAs an SM holds (registers)
constexpr int kSmShared = 228 << 10;  // shared memory of an SM, and what a CTA may ask for beside its own 42 KB
constexpr int kMostStaged = 180 << 10;
constexpr int kOwn = kBins / kThreads;
constexpr int kWarpList = kList / kWarps;  // listed tokens of a warp
constexpr int kFew = kThreads / 4;         // of a list whose tokens are compared with each other
constexpr int kEach = 8;         // elements a lane takes in a step
constexpr int kStep = 32 * kEach;

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
__device__ __forceinline__ u64 whole_weight(float w) {
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

// The sum of the lanes' numbers, by 24-bit digits.
__device__ __forceinline__ u64 warp_sum(u64 x) {
  const uint32_t a = __reduce_add_sync(0xffffffffu, (uint32_t)x & 0xffffffu);
  const uint32_t b = __reduce_add_sync(0xffffffffu, (uint32_t)(x >> 24) & 0xffffffu);
  const uint32_t c = __reduce_add_sync(0xffffffffu, (uint32_t)(x >> 48));
  return a + ((u64)b << 24) + ((u64)c << 48);
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
__device__ __forceinline__ u64 load_remote(uint32_t at) {
  u64 x;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(x) : "r"(at) : "memory");
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
    alignas(8) uint32_t hist[kBins];  // this CTA's counts
    uint2 all[kList];              // the first CTA: the cluster's listed tokens (|x|'s bits, index)
  };
  u64 all_w[kList];                // W of `all`
  alignas(8) uint32_t counts[kBins];  // the cluster's
  u64 at[kThreads + 1];            // counts and estimates before each thread's bins, and of all
  uint2 list[kWarps][kWarpList];   // listed tokens
  u64 post[2][3][kMaxPieces];      // what the pieces' warps told last, and before that
  u64 taken[4];                    // first bin, what lies before it, last bin, what lies up to its end
  u64 result[2];                   // the border, the sum up to it
  Search q;
  u64 scan_s[kWarps];
  uint32_t sub_n[kThreads], sub_hi[kThreads], sub_lo[kThreads];  // a list's bins: tokens, W by 20-bit digits
  int sub_bin, few_n, hit;
  u64 sub_before_s;
  uint32_t sub_before_n, sub_count;
  int few[32];
};

extern __shared__ uint4 staged[];  // a CTA's pieces, where they fit, and a step

// A row as a warp sees it: elements at `base`, 16-byte aligned, of which [skip, end) are the row.
template <typename T, bool kStaged>
struct Row {
  const T *base;
  int origin;         // of the CTA's pieces: where `staged` begins
  int skip, end;
  int lo, hi;         // this warp's piece, whole steps (but for the last one's end)
  int chunk_log;      // steps of a chunk: 2^chunk_log
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
  __device__ float kept(uint32_t d, uint32_t v) const {  // weight, 0 where it is not kept
    if (!inside(d, v)) return 0.f;
    const float w = weight(d);
    return w >= least ? w : 0.f;
  }
  // Logits of a step's elements [i0, b): those that are not the row's or behind b: -inf.  fetch: from memory; load:
  // from where the first pass has put them.
  __device__ void fetch(int i0, int b, int lane, float (&x)[kEach]) const {
    if (i0 >= skip && i0 + kStep <= b) {
      const uint4 *p = reinterpret_cast<const uint4 *>(base + i0) + lane;
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        const uint4 q = __ldg(p + 32 * k);
#pragma unroll
        for (int e = 0; e < kN; ++e) x[k * kN + e] = value(reinterpret_cast<const T *>(&q)[e]);
      }
    } else {
      const int i = i0 + lane * kN;
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int at = i + 32 * kN * (j / kN) + j % kN;
        const float v = value(base[min(max(at, skip), end - 1)]);
        x[j] = at >= skip && at < b ? v : -CUDART_INF_F;
      }
    }
  }
  __device__ void put(int i0, int lane, const float (&x)[kEach]) const {
    uint4 *p = staged + (i0 - origin) / kN + lane;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      uint4 q;
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        if constexpr (sizeof(T) == 2)
          reinterpret_cast<T *>(&q)[e] = (T)(__float_as_uint(x[k * kN + e]) >> 16);
        else
          reinterpret_cast<T *>(&q)[e] = x[k * kN + e];
      }
      p[32 * k] = q;
    }
  }
  __device__ void load(int i0, int b, int lane, float (&x)[kEach]) const {
    if constexpr (!kStaged) {
      fetch(i0, b, lane, x);
    } else {
      const uint4 *p = staged + (i0 - origin) / kN + lane;
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        const uint4 q = p[32 * k];
#pragma unroll
        for (int e = 0; e < kN; ++e) x[k * kN + e] = value(reinterpret_cast<const T *>(&q)[e]);
      }
      if (i0 + kStep > b)
#pragma unroll
        for (int j = 0; j < kEach; ++j)
          if (i0 + (32 * (j / kN) + lane) * kN + j % kN >= b) x[j] = -CUDART_INF_F;
    }
  }
  __device__ float at(int i) const {
    if constexpr (kStaged) return value(reinterpret_cast<const T *>(staged)[i - origin]);
    return value(base[i]);
  }
  // Element k of a lane's step (its registers cannot be indexed).
  __device__ static float element(const float (&x)[kEach], int k) {
    float l = x[0];
#pragma unroll
    for (int i = 1; i < kEach; ++i) l = i == k ? x[i] : l;
    return l;
  }
  // The index of element j of a lane's step at i0.
  __device__ int index(int i0, int j, int lane) const { return i0 + (32 * (j / kN) + lane) * kN + j % kN - skip; }

  // The first step from s on whose chunk is alive.
  __device__ int next(int s, int steps, uint32_t alive) const {
#pragma unroll 1
    while (s < steps && !((alive >> (s >> chunk_log)) & 1u)) ++s;
    return s;
  }
  // f(logit) for this piece's elements in live chunks; g(the step's place, its logits) after each step.  (The next
  // step's loads ahead of it were no faster: an SM's other warps cover them, and the registers spill.)
  template <bool kFirst = false, typename F, typename G>
  __device__ void each(uint32_t alive, F f, G g) const {
    const int steps = (hi - lo + kStep - 1) / kStep, lane = threadIdx.x & 31;
#pragma unroll 1
    for (int s = next(0, steps, alive); s < steps; s = next(s + 1, steps, alive)) {
      float x[kEach];
      const int at = lo + s * kStep;
      if constexpr (kFirst)
        fetch(at, hi, lane, x);
      else
        load(at, hi, lane, x);
      if constexpr (kFirst && kStaged) put(at, lane, x);
#pragma unroll
      for (int j = 0; j < kEach; ++j) f(x[j]);
      g(at, x);
    }
  }
  // f(bits of |x|, index) for the elements [a, b), a lane's one after another: where speed does not count.
  template <typename F>
  __device__ void each_slowly(int a, int b, int lane, F f) const {
#pragma unroll 1
    for (int i = max(a, skip) + lane; i < b; i += 32) f(depth(at(i), M, inv), (uint32_t)(i - skip));
  }
  // The chunks that have tokens with |x|'s bits below d.
  __device__ uint32_t alive(uint32_t d) const { return __ballot_sync(0xffffffffu, depth(chunk_top, M, inv) < d); }
};

template <typename T, bool kStaged>
struct Sampler {
  using R = Row<T, kStaged>;
  const SampleArgs &a;
  Shared &sh;
  R r;
  int cluster, rank, warp, lane, piece, pieces;
  int turn = 0;         // exchanges so far: their buffers alternate
  enum { kCounted, kReduced, kGone } first_level = kCounted;  // its counts in sh.hist; its shares added up; neither
  uint32_t n = 0;       // this warp's listed tokens

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

  // ---- bins

  // Counts of q's level in sh.hist, of the tokens with |x|'s bits in [from, to).
  __device__ void count() {
    const Search &q = sh.q;
#pragma unroll 1
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh.hist[i] = 0;
    __syncthreads();
    const uint32_t from = q.from, to = q.to;
    const Level lv = q.lv;
    r.each(r.alive(to), [&](float l) {
      const uint32_t d = depth(l, r.M, r.inv);
      if (d - from < to - from) atomicAdd(&sh.hist[lv.bin(d)], 1u);
    }, [&](int, const float(&)[kEach]) {});
    cluster_barrier();
  }

  // The cluster's counts, to every CTA: each adds up a share of the bins.  Then, alike in all of them, what lies before
  // each thread's bins.
  __device__ void reduce() {
    const int pairs = kBins / 2 / cluster;  // whole warps of them
#pragma unroll 1
    for (int i = threadIdx.x; i < pairs; i += kThreads) {
      const int b = 2 * (rank * pairs + i);
      u64 x[kMaxCluster], c = 0;  // (a count is below 2^23)
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) x[r] = r < cluster ? load_remote(remote(&sh.hist[b], r)) : 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) c += x[r];
#pragma unroll 1
      for (int r = 0; r < cluster; ++r) store_remote(remote(&sh.counts[b], r), c);
      u64 sum = sh.q.lv.both(b, (uint32_t)c) + sh.q.lv.both(b + 1, (uint32_t)(c >> 32));
      // a thread's own bins, in four lanes here
#pragma unroll
      for (int d = 1; d < kOwn / 2; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
#pragma unroll 1
      for (int r = lane & (kOwn / 2 - 1); r < cluster; r += kOwn / 2) store_remote(remote(&sh.at[b / kOwn], r), sum);
    }
    cluster_barrier();
    const u64 mine = sh.at[threadIdx.x];
    u64 run = warp_scan(mine, lane);
    if (lane == 31) sh.scan_s[warp] = run;
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < warp; ++i) run += sh.scan_s[i];
    sh.at[threadIdx.x] = run - mine;
    if (threadIdx.x == kThreads - 1) sh.at[kThreads] = run;
    __syncthreads();
  }

  // Takes the bins that may hold the border: the one at which the running count reaches q.many, or (by_sum) those at
  // which the running estimate may pass q.e0 and what q.w (a sum of W) makes, give or take q.slack of that; of the bins
  // in question.  Every CTA finds the same ones.
  __device__ void seek() {
    const Search &q = sh.q;
    u64 target[2];
    q.aim(sh.at[kThreads], target[0], target[1]);
    const int lowest = q.lowest(), highest = q.highest(), b0 = threadIdx.x * kOwn;
    auto here = [&](u64 t, int b, int to, u64 before, u64 until) { return q.holds(t, b, to, before, until, lowest, highest); };
    const u64 run = sh.at[threadIdx.x], end = sh.at[threadIdx.x + 1];
    // (its bins a lane each)
#pragma unroll 1
    for (uint32_t who = __ballot_sync(0xffffffffu, here(target[0], b0, b0 + kOwn - 1, run, end) ||
                                                       here(target[1], b0, b0 + kOwn - 1, run, end));
         who; who &= who - 1) {
      const int l = __ffs(who) - 1, b = (warp * 32 + l) * kOwn + (lane & (kOwn - 1));
      const u64 x = lane < kOwn ? q.lv.both(b, sh.counts[b]) : 0, to = __shfl_sync(0xffffffffu, run, l) + warp_scan(x, lane);
      if (lane < kOwn) {
        if (here(target[0], b, b, to - x, to)) sh.taken[0] = (u64)b, sh.taken[1] = to - x;
        if (here(target[1], b, b, to - x, to)) sh.taken[2] = (u64)b, sh.taken[3] = to;
      }
    }
    __syncthreads();
  }

  // ---- lists (of the first CTA)

  // Of the list's tokens that lie inside the border, in their order, the one at which their running number (or the
  // sum of their W) reaches `target`.  base: the number (sum) before those with |x|'s bits lo; [lo, lo + 2^bits):
  // where its own lie; bits -1: anywhere, in steps of 1/8 first.
  __device__ uint2 pick(int listed, bool by_sum, u64 target, u64 base, uint32_t lo, int bits) {
    u64 before_n = by_sum ? 0 : base, before_s = by_sum ? base : 0;
    uint32_t fixed = 0;      // |x|'s bits, once these are down to one value
    bool tied = false, eighths = bits < 0;
    auto in = [&](int i, uint2 &q, uint32_t &key) {
      q = sh.all[i];
      key = tied ? q.y : q.x;
      return r.inside(q.x, q.y) && (!tied || q.x == fixed);
    };
    uint32_t width = 0;      // of the last level's bin
    int shift = max(0, bits - 8);
#pragma unroll 1
    for (int level = 0; level < 16; ++level) {  // (five of |x| and three of the index at most)
      sh.sub_n[threadIdx.x] = sh.sub_hi[threadIdx.x] = sh.sub_lo[threadIdx.x] = 0;
      if (threadIdx.x == 0) sh.sub_bin = kThreads - 1, sh.few_n = 0, sh.sub_count = 0;
      __syncthreads();
#pragma unroll 1
      for (int i = threadIdx.x; i < listed; i += kThreads) {
        uint2 q;
        uint32_t key;
        if (in(i, q, key) && (eighths || key - lo < (256u << shift))) {
          const uint32_t b = eighths ? (uint32_t)(__uint_as_float(key) * 8.f) : (key - lo) >> shift;
          atomicAdd(&sh.sub_n[b], 1u);
          // (64-bit atomics on one word hold each other up; a digit's sums stay below 2^31)
          atomicAdd(&sh.sub_hi[b], (uint32_t)(sh.all_w[i] >> 20));
          atomicAdd(&sh.sub_lo[b], (uint32_t)sh.all_w[i] & 0xfffffu);
        }
      }
      __syncthreads();
      const uint32_t my_n = sh.sub_n[threadIdx.x];
      const u64 my_s = ((u64)sh.sub_hi[threadIdx.x] << 20) + sh.sub_lo[threadIdx.x];
      u64 run = warp_scan(by_sum ? my_s : (u64)my_n, lane);
      if (lane == 31) sh.scan_s[warp] = run;
      __syncthreads();
      run += by_sum ? before_s : before_n;
#pragma unroll 1
      for (int k = 0; k < warp; ++k) run += sh.scan_s[k];
      const u64 was = run - (by_sum ? my_s : (u64)my_n);
      if (was < target && target <= run) {
        sh.sub_bin = threadIdx.x;
        sh.sub_before_s = was;
        sh.sub_count = my_n;
      }
      __syncthreads();
      const int count = (int)sh.sub_count;
      (by_sum ? before_s : before_n) = sh.sub_before_s;
      if (eighths) {
        lo = __float_as_uint((float)sh.sub_bin * 0.125f);
        width = __float_as_uint((float)(sh.sub_bin + 1) * 0.125f) - lo;
        shift = 32 - __clz((int)(width - 1));
        eighths = false;
      } else {
        lo += (uint32_t)sh.sub_bin << shift;
        width = 1u << shift;
      }
      if (count <= 32) break;
      if (shift == 0) {  // many of one |x|: by index
        fixed = lo;
        tied = true;
        lo = 0;
        shift = 14;
      } else {
        shift = max(0, shift - 8);
      }
      __syncthreads();
    }
    // a few: ranked in every warp's lanes
#pragma unroll 1
    for (int i = threadIdx.x; i < listed; i += kThreads) {
      uint2 q;
      uint32_t key;
      if (in(i, q, key) && key - lo < width) sh.few[atomicAdd(&sh.few_n, 1) & 31] = i;
    }
    __syncthreads();
    const int count = min(sh.few_n, 32), mine = lane < count ? sh.few[lane] : 0;
    const uint2 q = sh.all[mine];
    const u64 w = sh.all_w[mine];
    u64 sum = before_s + w, place = before_n + 1;
#pragma unroll 1
    for (int k = 0; k < count; ++k) {
      const uint32_t d = __shfl_sync(0xffffffffu, q.x, k), v = __shfl_sync(0xffffffffu, q.y, k);
      const u64 o = __shfl_sync(0xffffffffu, w, k);
      if (d < q.x || (d == q.x && v < q.y)) sum += o, ++place;
    }
    const bool hit = lane < count && (by_sum ? sum - w < target && target <= sum : place == target);
    const uint32_t who = __ballot_sync(0xffffffffu, hit);
    const int l = who ? __ffs(who) - 1 : 0;
    const uint2 found = make_uint2(__shfl_sync(0xffffffffu, q.x, l), __shfl_sync(0xffffffffu, q.y, l));
    __syncthreads();
    return found;
  }

  // The same where the list is short and its tokens are all that counts (`before` the number, or the sum, before them):
  // four threads compare each with all.  sum: that of the list's W up to that token.
  __device__ uint2 pick_few(int listed, bool by_sum, u64 target, u64 before, u64 &sum) {
    const int i = threadIdx.x >> 2;
    const uint2 q = sh.all[i];  // (a place behind the list is no hit)
    u64 w = 0;
    uint32_t place = 0;
#pragma unroll 4
    for (int j = threadIdx.x & 3; j < listed; j += 4) {
      const uint2 o = sh.all[j];
      const u64 x = sh.all_w[j];
      const bool before_it = r.inside(o.x, o.y) & (o.x < q.x || (o.x == q.x && o.y <= q.y));
      w += before_it ? x : 0;
      place += before_it;
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      w += __shfl_xor_sync(0xffffffffu, w, d);
      place += __shfl_xor_sync(0xffffffffu, place, d);
    }
    if (i < listed && r.inside(q.x, q.y) &&
        (by_sum ? before + w - sh.all_w[i] < target && target <= before + w : before + place == target) &&
        (threadIdx.x & 3) == 0) {
      sh.taken[0] = (u64)q.x << 32 | q.y;
      sh.taken[1] = w;
    }
    __syncthreads();
    sum = sh.taken[1];
    const u64 found = sh.taken[0];
    __syncthreads();
    return make_uint2((uint32_t)(found >> 32), (uint32_t)found);
  }

  // The first of the list's tokens that are kept at which the sum of their W passes `left`.
  __device__ void draw(int listed, u64 left, int32_t *token) {
    const int each = (listed + kThreads - 1) / kThreads, j0 = threadIdx.x * each;
    auto w_of = [&](int j) {
      if (j >= listed) return (u64)0;
      const uint2 q = sh.all[j];
      return r.kept(q.x, q.y) > 0.f ? sh.all_w[j] : 0;
    };
    u64 own = 0;
#pragma unroll 1
    for (int j = 0; j < each; ++j) own += w_of(j0 + j);
    u64 run = warp_scan(own, lane);
    if (lane == 31) sh.scan_s[warp] = run;
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < warp; ++i) run += sh.scan_s[i];
    if (left < run && run - own <= left) {
      run -= own;
#pragma unroll 1
      for (int j = j0; j < j0 + each; ++j) {
        run += w_of(j);
        if (left < run) {
          *token = (int)sh.all[j].y;
          break;
        }
      }
    }
  }

  // The sum of W of the list's tokens that lie inside the border (and weigh `least`), with |x|'s bits below d.
  __device__ u64 list_sum(int listed, uint32_t d) {
    u64 x = 0;
#pragma unroll 1
    for (int j = threadIdx.x; j < listed; j += kThreads) {
      const uint2 q = sh.all[j];
      if (q.x < d && r.inside(q.x, q.y) && !(r.least > 0.f && weight(q.x) < r.least)) x += sh.all_w[j];
    }
    x = warp_sum(x);
    if (lane == 0) sh.scan_s[warp] = x;
    __syncthreads();
    x = warp_sum(lane < kWarps ? sh.scan_s[lane] : 0);
    __syncthreads();
    return x;
  }

  // Lists this piece's tokens with |x|'s bits in [from, to), by index; the sum of W of those before.
  __device__ u64 list_pass(uint32_t from, uint32_t to) {
    uint2 *list = sh.list[warp];
    Sum above;
    uint32_t marked = 0;  // bit j: element j of the lane's step is to be listed
    int j = 0;
    n = 0;
    r.each(r.alive(to), [&](float l) {
      const uint32_t d = depth(l, r.M, r.inv);
      const float w = weight(d);  // (without a branch: in most warps some lane has a token before the bins)
      above.add(d < from ? w : 0.f);
      marked |= (uint32_t)(d - from < to - from) << j++;
    }, [&](int at, const float(&x)[kEach]) {
      above.carry();
      j = 0;
      if (to > r.border) {  // (a border among tokens of one |x| is one of indices, too)
#pragma unroll 1
        for (uint32_t m = marked; m; m &= m - 1) {
          const int k = __ffs(m) - 1;
          if (!r.inside(depth(R::element(x, k), r.M, r.inv), (uint32_t)r.index(at, k, lane))) marked &= ~(m & -m);
        }
      }
      if (n > kWarpList) {  // (too many already)
        n += __reduce_add_sync(0xffffffffu, (uint32_t)__popc(marked));
      } else if (__any_sync(0xffffffffu, marked)) {
        // in the order of their indices: a lane's vector behind the lanes' before it (16 bits of a count each)
        uint32_t here = 0;
#pragma unroll
        for (int v = 0; v < R::kVecs; ++v) here |= __popc(marked >> (v * R::kN) & ((1u << R::kN) - 1)) << (16 * v);
        uint32_t incl = here;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += y;
        }
        const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
        uint32_t place = n + (incl - here & 0xffffu), next = n + (all & 0xffffu) + (incl - here >> 16);
#pragma unroll 1
        for (uint32_t m = marked; m; m &= m - 1) {
          const int k = __ffs(m) - 1;
          if (k >= R::kN) place = next, next += 1;
          if (place < kWarpList)
            list[place] = make_uint2(depth(R::element(x, k), r.M, r.inv), (uint32_t)r.index(at, k, lane));
          ++place;
        }
        n += (all & 0xffffu) + (all >> 16);
      }
      marked = 0;
    });
    return warp_sum(above.total);
  }

  // The border among tokens of one |x| (bits d): the first `ties` of them stay.
  __device__ void rank_ties(uint32_t d, u64 ties, u64 before_here, u64 here) {
    if (before_here < ties && ties <= before_here + here) {
      u64 run = before_here;
#pragma unroll 1
      for (int i = r.lo; i < r.hi; i += 32) {
        const int at = i + lane;
        const bool eq = at >= r.skip && at < r.hi && r.inside(d, (uint32_t)(at - r.skip)) &&
                        depth(r.at(at), r.M, r.inv) == d;
        uint32_t who = __ballot_sync(0xffffffffu, eq);
        if (ties <= run + __popc(who)) {
#pragma unroll 1
          while (++run < ties) who &= who - 1;
          if (lane < cluster)
            store_remote(remote(&sh.result[0], lane), (u64)d << 32 | (uint32_t)(i + __ffs(who) - 1 - r.skip));
          break;
        }
        run += __popc(who);
      }
    }
    cluster_barrier();
    r.border = d;
    r.last = (uint32_t)sh.result[0];
  }

  // Move the border to the last token of the order's first part: the `limit` first ones (by_sum false), or the
  // shortest part whose W sum to `limit` at least (1 .. their sum); S: the sum of all W.  sum: that part's, mine:
  // this piece's share of it.  listed: how many tokens are listed where the list holds all that lies inside the
  // border, else 0, before and after: then only the first CTA moves its border, and knows sum.
  // Where nothing with weight would be left out the border, sum and mine stay.  sum 0: the border was not found.
  // (One loop with each step in it once: the code is long, and it is fetched from memory when a call is the first.)
  __device__ void find_border(bool by_sum, u64 limit, u64 S, u64 &sum, u64 &mine, int &listed) {
    Search &q = sh.q;
    const bool lead = threadIdx.x == 0;
    u64 A = 0, above_here = 0, start = 0;
    uint32_t lo = 0;
    int bits = -1;
    if (!listed) {
      if (lead) q.start(by_sum, limit, S, first_level != kGone, first_level == kReduced);
      first_level = kReduced;
      __syncthreads();
    }
    // A pass ends the search, goes to a level of one of its level's bins (up to three times), or narrows what it looks at
    // within it: [first, last] in halves from the third wrong guess on, or once to one bin or to the bins alone
#pragma unroll 1
    for (int pass = 0; !listed; ++pass) {
      if (pass == kMostPasses) {
        sum = 0;
        return;
      }
      if (!q.counted) count();
      if (!q.reduced) reduce();
      seek();
      if (q.none(sh.taken)) {  // (asked first: among the bins below one row took 0.5 us longer)
        __syncthreads();  // (the next search writes to q)
        return;
      }
      const Bins t = q.bins(sh.taken);
      __syncthreads();
      if (lead) q.take(t, sh.taken);
      if (t.wide) {
        __syncthreads();
        continue;
      }
      // ---- the exact sum of what lies before the bins, and their tokens
      const uint2 *list = sh.list[warp];
      above_here = list_pass(t.from, t.to);
      __syncwarp();
      // their own sum
      u64 within = 0;
      if (q.by_sum) {
        if (n <= kWarpList)
#pragma unroll 1
          for (int i = lane; i < (int)n; i += 32) within += whole_weight(weight(list[i].x));
        else
          r.each_slowly(r.lo, r.hi, lane, [&](uint32_t d, uint32_t v) {
            if (d - t.from < t.to - t.from && r.inside(d, v)) within += whole_weight(weight(d));
          });
        within = warp_sum(within);
      }
      exchange<3>(above_here, (u64)n, within);
      A = told(0);
      const u64 N = told(1), N_before = told_before(1), B = told(2);
      const bool missed = q.low(A) || q.high(A, B);
      const bool fits = N <= kList && !__any_sync(0xffffffffu, posted(1, lane) > kWarpList || posted(1, lane + 32) > kWarpList);
      if (!missed && fits) {
        // to the first CTA
#pragma unroll 1
        for (int i = lane; i < (int)n; i += 32) {
          const uint2 x = list[i];
          store_remote(remote(&sh.all[N_before + i], 0), (u64)x.y << 32 | x.x);
          store_remote(remote(&sh.all_w[N_before + i], 0), whole_weight(weight(x.x)));
        }
        listed = (int)N;
        lo = t.begin;
        bits = 32 - __clz((int)(t.to - t.begin - 1) | 255);
        start = q.by_sum ? A : q.before;
        cluster_barrier();
        break;
      }
      if (!missed && t.to - t.from == 1) {
        const u64 W = whole_weight(weight(t.from)), stay = q.by_sum ? (q.limit - A + W - 1) / W : q.limit - q.before;
        first_level = q.lv.shift < 0 ? kReduced : kGone;
        rank_ties(t.from, stay, N_before, n);  // (ends with a barrier, after which q may be written to)
        sum = A + stay * W;
        mine = above_here + (stay > N_before ? min(stay - N_before, (u64)n) : 0) * W;
        return;
      }
      __syncthreads();
      if (lead) q.narrow(t, A, B);
      __syncthreads();
      first_level = q.lv.shift < 0 ? kReduced : kGone;
    }
    // ---- the border among the listed tokens
    if (rank == 0) {
      uint2 b;
      if (listed <= kFew) {
        b = pick_few(listed, by_sum, limit, q.whole ? 0 : start, sum);
        sum += A;
      } else {
        if (bits >= 0 && q.whole && by_sum) {  // (what lies before the bins: by weight it is summed up here)
          start = list_sum(listed, lo);
          if (start >= limit) lo = 0, start = 0, bits = -1;
        }
        b = pick(listed, by_sum, limit, start, lo, bits);
      }
      r.border = b.x;
      r.last = b.y;
      if (listed > kFew) sum = A + list_sum(listed, UINT_MAX);
      if (!q.whole && warp == 0 && lane < cluster) {
        store_remote(remote(&sh.result[0], lane), (u64)b.x << 32 | b.y);
        store_remote(remote(&sh.result[1], lane), sum);
      }
    }
    if (q.whole) return;
    listed = 0;
    cluster_barrier();
    r.border = (uint32_t)(sh.result[0] >> 32);
    r.last = (uint32_t)sh.result[0];
    sum = sh.result[1];
    u64 x = 0;
#pragma unroll 1
    for (int i = lane; i < (int)n; i += 32) {
      const uint2 t = sh.list[warp][i];
      if (r.inside(t.x, t.y)) x += whole_weight(weight(t.x));
    }
    mine = above_here + warp_sum(x);
  }
};

}  // namespace

template <typename T, bool kStaged>
__global__ void __launch_bounds__(kThreads, kPerSm) pskv_sample(const SampleArgs a, const int cluster,
                                                                     const bool beside) {
  __shared__ Shared sh;
  Sampler<T, kStaged> s{a, sh};
  using R = Row<T, kStaged>;
  R &r = s.r;
  s.cluster = cluster;
  s.rank = (int)cluster_rank();
  s.warp = threadIdx.x >> 5;
  s.lane = threadIdx.x & 31;
  s.pieces = cluster * kWarps;
  s.piece = s.rank * kWarps + s.warp;
  const int row = blockIdx.x / cluster, lane = s.lane, warp = s.warp;
  cluster_arrive_started();
  pdl_wait();
  if (beside) pdl_launch_dependents();
  // ---- the row's pieces, from the 16-byte boundary before it
  const T *l = static_cast<const T *>(a.logits) + row * a.logits_row;
  r.skip = (int)((reinterpret_cast<uintptr_t>(l) & 15) / sizeof(T));
  r.base = l - r.skip;
  r.end = r.skip + a.vocab;
  constexpr int kN = R::kN;
  const int seg = ((r.end + s.pieces - 1) / s.pieces + kStep - 1) / kStep * kStep;
  r.origin = s.rank * kWarps * seg;
  r.lo = min(s.piece * seg, r.end);
  r.hi = min(r.lo + seg, r.end);
  r.chunk_log = max(0, 32 - __clz(max(seg - 1, 0) / (32 * kStep)));  // at most 32 chunks
  const int req = row / a.per_request;
  float heat = a.temperature ? a.temperature[req] : 1.f, p = a.top_p ? a.top_p[req] : 1.f;
  float least = a.min_p ? a.min_p[req] : 0.f;
  int k = a.top_k ? a.top_k[req] : 0;
  // ---- M
  r.chunk_top = -CUDART_INF_F;
  {
    float chunk = -CUDART_INF_F;
    r.template each<true>(~0u, [&](float x) { chunk = fmaxf(chunk, x); }, [&](int at, const float(&)[kEach]) {
      const int step = (at - r.lo) / kStep + 1;
      if (step & ((1 << r.chunk_log) - 1) && at + kStep < r.hi) return;
      chunk = warp_max(chunk);
      if (lane == (step - 1) >> r.chunk_log) r.chunk_top = chunk;
      chunk = -CUDART_INF_F;
    });
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
  const bool empty = top == -CUDART_INF_F, endless = top == CUDART_INF_F;
  if (empty && s.rank == 0 && threadIdx.x == 0) {
    if (a.tokens) a.tokens[row] = -1;
    raise_fault(a.status, PSKV_FAULT_EMPTY_ROW);
  }
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
    if (r.alive(1u))
#pragma unroll 1
      for (int i = max(r.lo, r.skip) + lane; i < r.hi && at == UINT_MAX; i += 32)
        if (r.at(i) == top) at = (uint32_t)(i - r.skip);
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
    if (endless) r.inv = CUDART_INF_F;
    const bool some = k > 0 && k < a.vocab, part = p < 1.f, filters = some || part;
    // ---- the sum of W, and where the tokens lie
    if (filters) {
#pragma unroll 1
      for (int i = threadIdx.x; i < kBins; i += kThreads) sh.hist[i] = 0;
      __syncthreads();
    }
    const Level first{0u, 0u, -1};
    const float least_w = r.least;
    if (filters) r.least = 0.f;  // (min_p comes last)
    Sum all;
    r.each(~0u, [&](float x) {
      const uint32_t d = depth(x, r.M, r.inv);
      const float w = weight(d);
      all.add(w >= r.least ? w : 0.f);
      if (filters) atomicAdd(&sh.hist[first.bin(d)], 1u);
    }, [&](int, const float(&)[kEach]) { all.carry(); });
    u64 mine = warp_sum(all.total);
    s.template exchange<1>(mine);
    total = s.told(0);
    if (filters) {
      const u64 S = total;
#pragma unroll 1
      for (int by_sum = some ? 0 : 1; by_sum < (part ? 2 : 1) && total; ++by_sum)
        if (!listed || s.rank == 0)
          s.find_border(by_sum, by_sum ? max(share(p, total), 1ull) : (u64)k, S, total, mine, listed);
      r.least = least_w;
      if (!total) {
        // (as of an empty row, nothing is kept: no piece has a share)
        total = 1;
        mine = 0;
        r.least = 2.f;
        if (s.rank == 0 && threadIdx.x == 0) {
          if (a.tokens) a.tokens[row] = -1;
          raise_fault(a.status, PSKV_FAULT_BAD_STATE);
        }
      } else if (listed) {
        if (r.least > 0.f && s.rank == 0) total = s.list_sum(listed, UINT_MAX);
      } else {
        // (where the border's weight is above it, so are all: expf is right to 2^-22)
        if (r.least > 0.f && weight(r.border) < r.least * 1.000001f) {
          Sum some;
          uint32_t tied = 0;  // bit j: element j of the lane's step is as deep as the border
          int j = 0;
          mine = 0;
          r.each(r.alive(r.border + 1), [&](float x) {
            const uint32_t d = depth(x, r.M, r.inv);
            const float w = weight(d);
            some.add(d < r.border && w >= r.least ? w : 0.f);
            tied |= (uint32_t)(d == r.border) << j++;
          }, [&](int at, const float(&)[kEach]) {
            some.carry();
            j = 0;
#pragma unroll 1
            for (; tied; tied &= tied - 1)
              mine += whole_weight(r.kept(r.border, (uint32_t)r.index(at, __ffs(tied) - 1, lane)));
          });
          mine = warp_sum(mine + some.total);
        }
        s.template exchange<1>(mine);
        total = s.told(0);
      }
    }
    pdl_launch_dependents();
    // ---- the draw: where the running sum passes u's share
    if (listed) {
      if (s.rank == 0 && a.tokens) {
        const float u = a.u[row];
        s.draw(listed, u >= 1.f ? total - 1 : share(u, total), a.tokens + row);
      }
      if (!a.probs) return;
      if (s.rank == 0 && warp == 0 && lane < cluster) {
        store_remote(remote(&sh.result[0], lane), (u64)r.border << 32 | r.last);
        store_remote(remote(&sh.result[1], lane), total);
      }
      cluster_barrier();
      r.border = (uint32_t)(sh.result[0] >> 32);
      r.last = (uint32_t)sh.result[0];
      total = sh.result[1];
    } else if (a.tokens) {
      const float u = a.u[row];
      const u64 thr = u >= 1.f ? total - 1 : share(u, total), before = s.told_before(0);
      if (threadIdx.x == 0) sh.hit = -1;
      __syncthreads();
      if (lane == 0 && before <= thr && thr < before + mine) {
        sh.hit = s.piece;
        sh.sub_before_s = thr - before;
      }
      __syncthreads();
      if (sh.hit >= 0) {
        // its CTA: an eighth a warp
        const u64 left = sh.sub_before_s;
        const int p0 = min(sh.hit * seg, r.end), p1 = min(p0 + seg, r.end);
        const int sub = ((p1 - p0 + kWarps - 1) / kWarps + kN - 1) / kN * kN;
        const int s0 = min(p0 + warp * sub, p1), s1 = min(s0 + sub, p1);
        // (a vector's elements lie one after another, then the next lane's: sums of each vector of a lane)
        constexpr int kVecs = R::kVecs;
        u64 own = 0, part[kVecs] = {};
        float x[kEach];
        auto weigh = [&](int at, int j) {
          return whole_weight(r.kept(depth(R::element(x, j), r.M, r.inv), (uint32_t)r.index(at, j, lane)));
        };
        auto sums = [&](int at) {
          r.load(at, s1, lane, x);
#pragma unroll
          for (int k = 0; k < kVecs; ++k) part[k] = 0;
#pragma unroll 1
          for (int j = 0; j < kEach; ++j) {
            const u64 w = weigh(at, j);
#pragma unroll
            for (int k = 0; k < kVecs; ++k) part[k] += j / kN == k ? w : 0;
          }
        };
#pragma unroll 1
        for (int at = s0; at < s1; at += kStep) {
          sums(at);
#pragma unroll
          for (int k = 0; k < kVecs; ++k) own += part[k];
        }
        own = warp_sum(own);
        if (lane == 0) sh.scan_s[warp] = own;
        __syncthreads();
        u64 run = 0;
#pragma unroll 1
        for (int i = 0; i < warp; ++i) run += sh.scan_s[i];
        if (run <= left && left < run + own) {
#pragma unroll 1
          for (int at = s0; at < s1 && run <= left; at += kStep) {
            if (sub > kStep) sums(at);
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
              const u64 incl = run + warp_scan(part[k], lane);
              u64 before_it = incl - part[k];
              if (before_it <= left && left < incl) {
#pragma unroll 1
                for (int j = k * kN; j < (k + 1) * kN; ++j) {
                  before_it += weigh(at, j);
                  if (left < before_it) {
                    a.tokens[row] = r.index(at, j, lane);
                    break;
                  }
                }
              }
              run = __shfl_sync(0xffffffffu, incl, 31);
            }
          }
        }
      }
    }
  }
  if (a.probs) {
    // W / S, W being floats: 1 / S as a float pair.  A step's values go through shared memory, so that they leave in
    // whole lines wherever the row begins
    const double inv = 1.0 / (double)total;
    const float hi = (float)inv, lo = (float)(inv - (double)hi);
    const size_t out = (size_t)row * a.vocab;
    auto put = [&](int v, float q) {
      if (a.probs_dtype == PSKV_DTYPE_BF16)
        static_cast<__nv_bfloat16 *>(a.probs)[out + v] = __float2bfloat16_rn(q);
      else
        static_cast<float *>(a.probs)[out + v] = q;
    };
    auto share_of = [&](float w) {
      const float W = rintf(w * 0x1p40f);
      return fmaf(W, hi, W * lo);
    };
    const uint32_t alive = empty || listed ? 0 : r.alive(r.border + 1);
    float *stage = reinterpret_cast<float *>(sh.list[warp]);  // (of a listed row nothing is staged)
    static_assert(sizeof sh.list[0] >= kStep * sizeof(float), "room for a step");
#pragma unroll 1
    for (int s0 = r.lo, step = 0; s0 < r.hi; s0 += kStep, ++step) {
      const bool live = (alive >> (step >> r.chunk_log)) & 1u;
      if (live) {
        float x[kEach];
        r.load(s0, r.hi, lane, x);
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          const int at = 32 * kN * (j / kN) + lane * kN + j % kN;
          stage[at] = share_of(r.kept(depth(x[j], r.M, r.inv), (uint32_t)(s0 + at - r.skip)));
        }
        __syncwarp();
      }
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int at = s0 + 32 * j + lane;
        if (at >= r.skip && at < r.hi) put(at - r.skip, live ? stage[32 * j + lane] : 0.f);
      }
      __syncwarp();
    }
    if (listed)
#pragma unroll 1
      for (int i = lane; i < (int)s.n; i += 32) {
        const uint2 t = sh.list[warp][i];
        const float w = r.kept(t.x, t.y);
        if (w > 0.f) put((int)t.y, share_of(w));
      }
  }

}

namespace {

template <typename T, bool kStaged>
cudaError_t launch(const SampleArgs &a, int cluster, bool beside, size_t bytes, cudaStream_t s) {
  if (kStaged) {
    static std::atomic<bool> allowed[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!(dev >= 0 && dev < 64 && allowed[dev])) {
      e = cudaFuncSetAttribute(pskv_sample<T, kStaged>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostStaged);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) allowed[dev] = true;
    }
  }
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
  cfg.dynamicSmemBytes = kStaged ? bytes : 0;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, pskv_sample<T, kStaged>, a, cluster, beside);
}

template <typename T>
cudaError_t launch(const SampleArgs &a, int cluster, int sms, cudaStream_t s) {
  // A CTA's pieces stay in shared memory where all CTAs run at once all the same: at three or more an SM with an eighth
  // of the places to spare, else half of them, as clusters do not fill every group of SMs (80 rows of 32,001 bf16, 17 KB:
  // 33 -> 28 us; one of 131,072 f32, 66 KB: 9.8 -> 8.8; but 16 of these, 128 CTAs of one or two an SM: 11.2 -> 15.3).
  const long long seg = ((a.vocab + 16 / (int)sizeof(T) - 1 + cluster * kWarps - 1) / (cluster * kWarps) + kStep - 1) / kStep * kStep;
  const long long bytes = (kWarps * seg + kStep) * (long long)sizeof(T), ctas = (long long)a.rows * cluster;
  const long long fit = bytes <= kMostStaged ? std::min<long long>(kPerSm, kSmShared / ((long long)sizeof(Shared) + bytes + 1024)) : 0;
  const bool staged = fit >= 3 ? ctas + ctas / 8 <= fit * sms : fit > 0 && 2 * ctas <= sms;
  // The next grid may start beside this one where both fit; else its CTAs would take what places there are, unevenly
  // (40 rows of 131,072 bf16 one call after the other: 16.7 -> 14.2 us; but 32, where both fit: 12.1 -> 13.5)
  const bool beside = 2 * ctas <= (staged ? fit : kPerSm) * sms;
  return staged ? launch<T, true>(a, cluster, beside, (size_t)bytes, s) : launch<T, false>(a, cluster, beside, 0, s);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, int sms, cudaStream_t s) {
  // the largest cluster with which all rows run at once
  int cluster = kMaxCluster;
#pragma unroll 1
  while (cluster > 1 && (long long)a.rows * cluster > (long long)kPerSm * sms) cluster /= 2;
  return a.dtype == PSKV_DTYPE_BF16 ? launch<uint16_t>(a, cluster, sms, s) : launch<float>(a, cluster, sms, s);
}

}  // namespace pskv
