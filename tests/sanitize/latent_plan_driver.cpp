// Walks decode_attn_latent's plan (pskv_plan.cpp) over many batches and checks that no plan has more
// pieces of a row than the bound its workspace may be sized by.  Built and run by
// tests/test_latent_bound.py; returns non-zero on a failed check.
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include "pskv_plan.h"

int main() {
  using namespace pskv;
  // even rows that fill the pairs stay whole; one of them between short rows is cut
  std::vector<int32_t> even(40, 1500), odd(40, 100);
  odd[0] = 1500;
  if (plan_latent(76, 512, 40, even.data(), 1, 0).splits != 1) return 1;
  if (plan_latent(76, 512, 40, odd.data(), 1, 0).splits < 2) return 2;
  std::mt19937 rng(1);
  auto pick = [&](int lo, int hi) { return (int)(lo + rng() % (unsigned)(hi - lo + 1)); };
  for (int round = 0; round < 20000; ++round) {
    const int n = pick(1, 1 << pick(0, 9)), clusters = pick(0, 3) ? 76 : pick(1, 100);
    const int dc = pick(0, 1) ? 512 : 256, splits = pick(0, 2) ? 0 : 1 << pick(0, 10);
    const int64_t blocks = pick(0, 2) ? 1 : pick(1, 64);
    const int longest = 1 + (int)(rng() % (1u << pick(1, 20)));
    std::vector<int32_t> lens(n);
    for (auto &l : lens) l = pick(0, 3) ? pick(0, longest) : pick(0, 1) ? longest : pick(0, longest < 200 ? longest : 200);
    const LatentPlan p = plan_latent(clusters, dc, n, lens.data(), blocks, splits);
    const int bound = latent_most_splits(clusters, n, longest, blocks, splits);
    if (p.splits < 1 || p.splits > bound) {
      std::fprintf(stderr, "%d pieces, bound %d: %d rows up to %d keys, %lld blocks, %d splits\n", p.splits,
                   bound, n, longest, (long long)blocks, splits);
      return 3;
    }
    int64_t most = 1;
    for (int l : lens) most = (l + kLatentTile - 1) / kLatentTile > most ? (l + kLatentTile - 1) / kLatentTile : most;
    if ((int64_t)p.splits * p.tiles_per_piece < most) return 4;
  }
  std::puts("latent plan driver ok");
  return 0;
}
