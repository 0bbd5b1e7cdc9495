// kv_fork_rows' blocks: what all of them read to compare forks stays within one reading of the call's forks for every eight
// forks and a share that goes with the pieces copied.  Built and run by tests/test_fork_plan.py; non-zero on a failed check.
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "pskv_plan.h"

int main() {
  using namespace pskv;
  for (int64_t n : {1, 2, 63, 64, 1000, 1024, 1025, 4096, 16384, 40000, 65535})
    for (int64_t pieces : {1, 3, 8, 128, 512, 16384, 1 << 20}) {
      const ForkBlocks b = fork_blocks((int32_t)n, pieces);
      if (b.pieces < 1 || b.pieces > pieces || b.forks < 1 || b.forks > kForksTogether) return 1;
      if (n <= kForkScan && (b.pieces != 1 || b.forks != 1)) return 2;  // (few forks: as many blocks as there are pieces)
      if (b.forks > 1 && b.pieces != pieces) return 3;
      // reads of the call's forks by all blocks
      const int64_t blocks = ((pieces + b.pieces - 1) / b.pieces) * ((n + b.forks - 1) / b.forks);
      if (n > kForkScan && blocks * n > n * (n + kForksTogether) / kForksTogether + 2 * kForkScan * n * pieces) {
        std::fprintf(stderr, "%lld forks of %lld pieces: %lld blocks\n", (long long)n, (long long)pieces, (long long)blocks);
        return 4;
      }
    }
  std::puts("fork plan driver ok");
  return 0;
}
