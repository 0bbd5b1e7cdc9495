// sample_search.h -- the search for a border of sample_tokens: where it stands, which bins it takes next, and how it goes
// on from what a pass over them has found.  Whole numbers and a few floats, compiled for the kernel and, by
// tests/test_sample_search.py, for the host, where rows of every kind go through it and its passes are counted.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PSKV_SEARCH __host__ __device__ __forceinline__
#else
#define PSKV_SEARCH inline
#endif
#ifndef __CUDA_ARCH__
#include <cmath>
#include <cstring>
#endif

namespace pskv {
namespace border {

using u64 = unsigned long long;

constexpr int kBins = 2048;
constexpr int kList = 1024;      // listed tokens of a cluster
constexpr int kCountBits = 23;   // of a number that holds a count (up to 2^22) and an estimate (up to 2^40)
constexpr uint32_t kCountMask = (1u << kCountBits) - 1;
constexpr float kSlack = 2.5e-4f;  // of an estimated sum: half a bin's width off in some of the likeliest tokens
constexpr float kDeepest = 31.98f;        // what lies deeper has no weight: expf(-31.98) is under 2^-46
constexpr uint32_t kDeep = 0x41ffd70au;   // its bits

// Passes that a search may take; a row that is not done by then counts as empty, with a fault.  (Of 240,000 rows of every
// kind none took more than 34.)
#ifndef PSKV_SAMPLE_PASSES
#define PSKV_SAMPLE_PASSES 256
#endif
constexpr int kMostPasses = PSKV_SAMPLE_PASSES;

#ifdef __CUDA_ARCH__
PSKV_SEARCH uint32_t bits_of(float x) { return __float_as_uint(x); }
PSKV_SEARCH float float_of(uint32_t x) { return __uint_as_float(x); }
PSKV_SEARCH u64 nearest(float x) { return __float2ull_rn(x); }
PSKV_SEARCH int leading_zeros(uint32_t x) { return __clz((int)x); }
PSKV_SEARCH float exp_of(float x) { return expf(x); }
PSKV_SEARCH uint32_t smaller(uint32_t a, uint32_t b) { return min(a, b); }
PSKV_SEARCH float larger(float a, float b) { return fmaxf(a, b); }
PSKV_SEARCH float size_of(float x) { return fabsf(x); }
#else
PSKV_SEARCH uint32_t bits_of(float x) {
  uint32_t u;
  std::memcpy(&u, &x, 4);
  return u;
}
PSKV_SEARCH float float_of(uint32_t u) {
  float x;
  std::memcpy(&x, &u, 4);
  return x;
}
PSKV_SEARCH u64 nearest(float x) { return (u64)std::llrint((double)x); }
PSKV_SEARCH int leading_zeros(uint32_t x) { return x ? __builtin_clz(x) : 32; }
PSKV_SEARCH float exp_of(float x) { return (float)std::exp((double)x); }
PSKV_SEARCH uint32_t smaller(uint32_t a, uint32_t b) { return a < b ? a : b; }
PSKV_SEARCH float larger(float a, float b) { return a > b ? a : b; }
PSKV_SEARCH float size_of(float x) { return std::fabs(x); }
#endif

// A level of bins.  The first: |x| to the nearest 1/64, up to 2,047; finer ones: |x|'s bits d in [lo, hi), bin
// (d - lo) >> shift.
struct Level {
  uint32_t lo, hi;
  int shift;  // -1: the first level
  PSKV_SEARCH int bin(uint32_t d) const {
    // (a float add whose last place is 1/64)
    return shift < 0 ? (int)(bits_of(float_of(d) + 131072.f) - 0x48000000u) : (int)((d - lo) >> shift);
  }
  PSKV_SEARCH uint32_t begin(int b) const {
    if (shift >= 0) return smaller((uint32_t)b << shift, hi - lo) + lo;
    // halfway goes to the even bin
    return b == 0 ? 0u : b == kBins ? kDeep + 1 : bits_of(((float)b - 0.5f) * 0x1p-6f) + (b & 1);
  }
  // n tokens of a bin and an estimate of their weights, the middle's, in units of 2^-18: both in one number.  (Running
  // sums of whole numbers go up from bin to bin, whoever forms them in what order.)
  PSKV_SEARCH u64 both(int b, uint32_t n) const {
    const float x = shift < 0 ? (float)b * 0x1p-6f
                              : float_of(smaller(lo + ((uint32_t)b << shift) + ((1u << shift) >> 1), hi));
    return n ? nearest((float)n * exp_of(-x) * 0x1p18f) << kCountBits | n : 0;
  }
};

// Bins that may hold the border.
struct Bins {
  int first, last;
  uint32_t before_n, until_n;  // tokens of the level before the first one, and up to the last one's end
  bool whole;                  // the whole first part is to be listed, as it may fit
  bool wide;                   // more than a list holds, from a guess with slack: guess again without
  uint32_t begin, from, to;    // |x|'s bits: where the bins begin, what is listed
};

// Where the search stands (the same in all CTAs; in shared memory, as the passes over the logits need the registers).
// Written by one thread between barriers.
struct Search {
  Level lv;
  bool by_sum;             // the border is one of weight, not of number
  bool counted, reduced;   // the level's counts are in, and its shares added up
  bool whole;              // the list is to hold all of the first part
  bool spread;             // and may (no warp has yet had more tokens of it than its list holds)
  int first, last, tries;  // bins in question
  u64 limit, many;         // the border's sum or number, and its number within the level
  u64 S;                   // the sum of the level's W
  u64 skipped, before;     // tokens before the level's first bin, and before the taken ones
  u64 e_before, e_until;   // the estimates before these and up to their end
  float e0, w, slack;      // the estimate looked for: e0 and what the weight w makes, give or take slack of that
  uint32_t from, to;       // |x|'s bits of the taken bins

  PSKV_SEARCH void start(bool sum, u64 lim, u64 all, bool counts_in, bool added_up) {
    lv = Level{0u, 0u, -1};
    by_sum = sum;
    counted = counts_in;
    reduced = added_up;
    first = tries = 0;
    spread = true;
    last = kBins - 1;
    limit = many = lim;
    S = all;
    skipped = 0;
    e0 = 0.f;
    w = (float)lim;
    slack = kSlack;
    from = 0;
    to = kDeep + 1;
  }

  // What of a running number (counts and estimates) the border is looked for by.
  PSKV_SEARCH u64 number(u64 x) const { return by_sum ? x >> kCountBits : x & kCountMask; }

  // The running numbers between which the border may lie; all: the level's.
  PSKV_SEARCH void aim(u64 all, u64 &least, u64 &most) const {
    least = most = many;
    if (!by_sum) return;
    // (an estimate's unit is 2^22 of W's; within a hundredth of that the level's own ratio is better: else it has
    // tokens that top-k left out)
    float unit = (float)(all >> kCountBits) / (float)S;
    if (!(size_of(unit * 0x1p22f - 1.f) <= 0.01f)) unit = 0x1p-22f;
    const float part = w * unit, e = e0 + part, give = size_of(part) * slack;
    least = nearest(larger(e - give, 1.f));
    most = nearest(larger(e + give, 1.f));
  }

  // The bins in question: from the third wrong guess on the middle one.
  PSKV_SEARCH int lowest() const { return tries < 3 ? first : (first + last) / 2; }
  PSKV_SEARCH int highest() const { return tries < 3 ? last : (first + last) / 2; }
  // A bin (or bins b .. to) within [lo, hi] holds a target: running numbers before and up to its end.
  PSKV_SEARCH bool holds(u64 target, int b, int to, u64 before, u64 until, int lo, int hi) const {
    return to >= lo && b <= hi && (b <= lo || number(before) < target) && (to >= hi || number(until) >= target);
  }

  // taken: the first bin, what lies before it, the last bin, what lies up to its end.
  // The border lies behind all that has weight.
  PSKV_SEARCH bool none(const u64 *taken) const { return !by_sum && lv.shift < 0 && (int)taken[0] == kBins - 1; }
  PSKV_SEARCH Bins bins(const u64 *taken) const {
    Bins t;
    t.first = (int)taken[0];
    t.last = (int)taken[2];
    t.before_n = (uint32_t)taken[1] & kCountMask;
    t.until_n = (uint32_t)taken[3] & kCountMask;
    // the whole first part is listed where it fits
    t.whole = spread && skipped + t.until_n <= kList;
    t.wide = !t.whole && t.first < t.last && t.until_n - t.before_n > kList && slack > 0.f;
    t.begin = lv.begin(t.first);
    t.from = t.whole ? 0u : t.begin;
    t.to = lv.begin(t.last + 1);
    return t;
  }
  PSKV_SEARCH void take(const Bins &t, const u64 *taken) {
    counted = reduced = true;
    whole = t.whole;
    before = skipped + t.before_n;
    e_before = taken[1] >> kCountBits;
    e_until = taken[3] >> kCountBits;
    from = t.from;
    to = t.to;
    if (t.wide) slack = 0.f;
  }

  // The border lies before the taken bins, or behind them.  A: the exact sum before what is listed; B: of that.
  PSKV_SEARCH bool low(u64 A) const { return by_sum && A >= limit; }
  PSKV_SEARCH bool high(u64 A, u64 B) const { return by_sum && A + B < limit; }

  // On from a pass that has not ended the search.
  PSKV_SEARCH void narrow(const Bins &t, u64 A, u64 B) {
    if (low(A) || high(A, B)) {
      // the estimate was off: on from the exact sum and the estimate of the same place (of a whole part: its end)
      if (low(A)) {
        last = t.first > 0 ? t.first - 1 : 0;
        w = -(float)(A - limit);
      } else {
        first = t.last + 1 < kBins ? t.last + 1 : kBins - 1;
        w = (float)(limit - (whole ? B : A));
      }
      e0 = (float)(high(A, B) && whole ? e_until : e_before);
      slack = 8 * kSlack;
      ++tries;
    } else if (whole) {
      // (a warp has too many of them, as where a mask leaves a run of tokens: the bins' own, then)
      spread = false;
    } else if (t.first < t.last) {
      // (they may be all of the level: the one bin of the estimate, then)
      slack = 0.f;
    } else {
      // finer bins
      const int z = 21 - leading_zeros(t.to - t.from - 1);
      skipped = before;
      lv = Level{t.from, t.to, z > 0 ? z : 0};
      counted = reduced = false;
      first = tries = 0;
      last = (int)((t.to - 1 - t.from) >> lv.shift);
      many = limit - before;
      e0 = 0.f;
      w = by_sum ? (float)(limit - A) : 0.f;
      S = B > 0 ? B : 1;
      slack = kSlack;
    }
  }
};

}  // namespace border
}  // namespace pskv
