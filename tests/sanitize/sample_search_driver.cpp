// Takes rows of every kind through sample_tokens' search for a border (sample_search.h), the kernel's passes restated by
// plain loops: the border is the definition's, what a wrong guess goes on from lies where the exact sum ends, and the
// search ends in few passes.  Built and run by tests/test_sample_search.py; returns non-zero on a failed check.
//   sample_search_driver ROWS: prints how many rows took how many passes
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <numeric>
#include <random>
#include <vector>

#include "sample_search.h"

using namespace pskv::border;

namespace {

constexpr int kMost = 48;  // passes of a search
static_assert(kMost < kMostPasses, "the kernel's own bound is not reached");
constexpr int kWarpList = kList / 8, kStep = 256;

u64 whole_weight(uint32_t d) { return (u64)std::nearbyint((double)exp_of(-float_of(d)) * 0x1p40); }

struct Row {
  std::vector<uint32_t> d;  // |x|'s bits
  std::vector<u64> W;
  std::vector<int> order;   // by |x|, then by index
  int piece;                // elements of a warp
  uint32_t border = kDeep, last = UINT32_MAX;
  bool inside(int i) const { return d[i] < border || (d[i] == border && (uint32_t)i <= last); }
};

int fail(const char *what, const Row &r, bool by_sum, u64 limit) {
  std::fprintf(stderr, "%s: %zu tokens, %s %llu\n", what, r.d.size(), by_sum ? "sum" : "number", limit);
  return -1;
}

// The border moved as find_border does; how many passes that took, below 0: a check failed.
int find(Row &r, bool by_sum, u64 limit, u64 S) {
  Search q;
  q.start(by_sum, limit, S, false, false);
  std::vector<u64> run(kBins + 1);
  const int n = (int)r.d.size();
  for (int pass = 1;; ++pass) {
    if (pass > kMost) return fail("too many passes", r, by_sum, limit);
    if (!q.counted) {
      std::vector<uint32_t> counts(kBins);
      for (uint32_t d : r.d)
        if (d - q.from < q.to - q.from) {
          const int b = q.lv.bin(d);
          if (b < 0 || b >= kBins || d < q.lv.begin(b) || d >= q.lv.begin(b + 1)) return fail("a token outside its bin", r, by_sum, limit);
          ++counts[b];
        }
      for (int b = 0; b < kBins; ++b) run[b + 1] = run[b] + q.lv.both(b, counts[b]);
    }
    u64 target[2], taken[4];
    q.aim(run[kBins], target[0], target[1]);
    int hits[2] = {0, 0};
    for (int b = 0; b < kBins; ++b)
      for (int k = 0; k < 2; ++k)
        if (q.holds(target[k], b, b, run[b], run[b + 1], q.lowest(), q.highest())) {
          taken[2 * k] = (u64)b;
          taken[2 * k + 1] = run[b + k];
          ++hits[k];
        }
    if (hits[0] != 1 || hits[1] != 1) return fail("not one bin", r, by_sum, limit);
    if (q.none(taken)) return pass;
    const Bins t = q.bins(taken);
    q.take(t, taken);
    if (t.wide) continue;
    u64 A = 0, B = 0, N = 0;
    bool fits = true;
    std::vector<int> list;
    for (int p = 0; p < n; p += r.piece) {
      u64 mine = 0;
      for (int i = p; i < std::min(n, p + r.piece); ++i) {
        if (r.d[i] < t.from) A += r.W[i];
        if (r.d[i] - t.from < t.to - t.from && r.inside(i)) {
          ++mine;
          B += r.W[i];
          list.push_back(i);
        }
      }
      N += mine;
      fits &= mine <= (u64)kWarpList;
    }
    fits &= N <= (u64)kList;
    const bool low = q.low(A), high = q.high(A, B);
    if (!low && !high && (fits || t.to - t.from == 1)) {
      std::sort(list.begin(), list.end(), [&](int a, int b) { return r.d[a] != r.d[b] ? r.d[a] < r.d[b] : a < b; });
      u64 at = by_sum ? A : t.whole ? 0 : q.before;
      for (int i : list) {
        at += by_sum ? r.W[i] : 1;
        if (at >= limit) {
          r.border = r.d[i];
          r.last = (uint32_t)i;
          return pass;
        }
      }
      return fail("a border behind the list", r, by_sum, limit);
    }
    q.narrow(t, A, B);
    if (high) {
      // what is missing lies behind the place up to which the sum is exact
      u64 least, most;
      q.aim(run[kBins], least, most);
      const u64 reached = t.whole ? taken[3] >> kCountBits : taken[1] >> kCountBits;
      if ((double)most < (double)reached * (1 - 0x1p-22)) return fail("a guess before what is known to be short", r, by_sum, limit);
    }
  }
}

struct Random {
  std::mt19937_64 g;
  explicit Random(u64 seed) : g(seed) {}
  int below(int n) { return (int)(g() % (u64)n); }
  float u() { return (float)((double)(g() >> 11) * 0x1p-53); }
  float normal() {
    double s = 0;
    for (int i = 0; i < 12; ++i) s += (double)(g() >> 11) * 0x1p-53;
    return (float)(s - 6);
  }
  template <typename T>
  T one(std::initializer_list<T> v) { return v.begin()[below((int)v.size())]; }
};

std::vector<float> logits(Random &g, int n) {
  std::vector<float> l((size_t)n);
  const int kind = g.below(12);
  const float a = g.one({0.001f, 0.1f, 1.f, 2.5f, 6.f, 30.f}), q = g.one({1.f, 4.f, 64.f, 512.f}), c = g.one({1e-5f, 1e-3f, 0.01f, 0.3f});
  const float part = g.one({.01f, .1f, .5f}), base = g.one({0.f, 8.999f, 5.f, -3.f}), deep = g.one({1.f, 3.f, 7.f, 12.f});
  const int few = g.one({2, 5, 300});
  float sum = 0;
  for (int i = 0; i < n; ++i) {
    switch (kind) {
      case 0: l[i] = g.normal() * a; break;
      case 1: l[i] = std::nearbyint(g.normal() * 3 * q) / q; break;
      case 2: l[i] = 1.5f; break;
      case 3: l[i] = g.u() < part ? 9.f : base; break;
      case 4: l[i] = -(float)i * c; break;
      case 5: l[i] = (float)i * std::min(c, 0.01f); break;
      case 6: l[i] = -std::log(1.f + (float)i) * (0.5f + part); break;
      case 7: l[i] = g.normal(); break;
      case 8: l[i] = 3.f + (float)g.below(few) * 0x1p-22f; break;
      case 9: l[i] = std::log(g.u() + 1e-9f) * (a < 3 ? a : 0.2f); break;
      case 10: l[i] = sum += g.normal() * std::max(c, 0.01f); break;
      default: l[i] = g.normal() * 0.01f - (g.u() < 0.5f ? 0.f : deep);
    }
  }
  if (kind == 7) l[g.below(n)] += g.one({5.f, 10.f, 20.f, 40.f});
  const int mask = g.below(4);
  if (mask == 0) {  // a run, and a token above it
    const int from = g.below(n), to = std::min(n, from + g.one({1, 20, 129, 300, 1100, 5000}));
    float top = l[from];
    for (int i = 0; i < n; ++i) {
      if (i >= from && i < to) top = std::max(top, l[i]);
      else l[i] = -INFINITY;
    }
    if (g.below(2)) l[from] = top + g.one({3.f, 9.f, 15.f, 25.f});
  } else if (mask == 1) {
    const float gone = g.one({.1f, .5f, .95f});
    for (float &x : l)
      if (g.u() < gone) x = -INFINITY;
  }
  if (g.u() < 0.3f)
    for (float &x : l) x = float_of(bits_of(x) & 0xffff0000u);
  if (!std::isfinite(*std::max_element(l.begin(), l.end()))) l[0] = 0.f;
  return l;
}

}  // namespace

int main(int argc, char **argv) {
  const int rows = argc > 1 ? std::atoi(argv[1]) : 8000;
  std::map<int, int> took;
  for (int seed = 0; seed < rows; ++seed) {
    Random g((u64)seed);
    const int n = g.one({1 + g.below(40), 40 + g.below(700), 700 + g.below(2300), 3000 + g.below(6000)});
    const std::vector<float> l = logits(g, n);
    const float inv = 1.f / g.one({.05f, .3f, 1.f, 1.3f, 5.f, 50.f}), M = *std::max_element(l.begin(), l.end());
    Row r;
    for (float x : l) {
      const float y = (x - M) * inv;
      r.d.push_back(bits_of(size_of(y > -kDeepest ? std::min(y, 0.f) : -kDeepest)));
      r.W.push_back(whole_weight(r.d.back()));
    }
    const int pieces = g.one({8, 16, 32, 64});
    r.piece = ((n + pieces - 1) / pieces + kStep - 1) / kStep * kStep;
    r.order.resize((size_t)n);
    std::iota(r.order.begin(), r.order.end(), 0);
    std::sort(r.order.begin(), r.order.end(), [&](int a, int b) { return r.d[a] != r.d[b] ? r.d[a] < r.d[b] : a < b; });
    const u64 S = std::accumulate(r.W.begin(), r.W.end(), (u64)0);
    const int k = g.one({0, 1, 2, 5, 40, 130, 500, 1000, 1024, 1025, 2000, n - 1, n / 2});
    const float p = g.one({0.f, 1e-6f, .1f, .5f, .9f, .95f, .999f, .999999f, 0.99999994f, 1.f, g.u()});
    u64 total = S;
    int kept = n, most = 0;
    auto sum_inside = [&] {
      u64 s = 0;
      for (int i = 0; i < n; ++i) s += r.inside(i) ? r.W[i] : 0;
      return s;
    };
    if (k > 0 && k < n) {
      const int passes = find(r, false, (u64)k, S);
      if (passes < 0) return 1;
      most = passes;
      total = 0;
      for (int i = 0; i < k; ++i) total += r.W[r.order[i]];
      if (sum_inside() != total) return std::fprintf(stderr, "row %d: top-k %d\n", seed, k), 2;
      kept = k;
    }
    if (p < 1.f) {
      const u64 limit = std::max((u64)((double)p * (double)total), (u64)1);
      const int passes = find(r, true, limit, S);
      if (passes < 0) return 3;
      most = std::max(most, passes);
      u64 want = 0;
      for (int i = 0; i < kept && want < limit; ++i) want += r.W[r.order[i]];
      if (sum_inside() != want) return std::fprintf(stderr, "row %d: top-p %g\n", seed, p), 4;
    }
    ++took[most];
  }
  for (auto [passes, n] : took) std::printf("%d passes: %d rows\n", passes, n);
  std::puts("sample search driver ok");
  return 0;
}
