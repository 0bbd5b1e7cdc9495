// verify_tree.cu -- the path of a drafted tree that stands.
//
// Token 0 stands; token t stands if its parent p (the highest ancestor bit below t) does and
// drafts[t] = sampled[p], the lowest of equal siblings.  So from a standing token the path goes on
// to the lowest token whose parent it is and whose draft it says, or ends.
// One warp a row holds two tokens a lane and takes a ballot a step (about 40 cycles), so that a window's 64 tokens cost
// one round of loads and as many steps as stand.  Bound by its launch: 1 row of 8 tokens 1.2 us, 64 rows of 64
// 1.9 us (132 KB), calls one after the other.
#include "pskv_internal.cuh"
#include "tree.h"

namespace pskv {

namespace {
constexpr int kWarps = 4;
}

__global__ void __launch_bounds__(kWarps * 32) pskv_verify_tree(const VerifyTreeArgs a) {
  const int b = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  if (b >= a.batch) return;
  const int T = a.num_tokens;
  const size_t row = (size_t)b * T;
  int parent[2], draft[2], says[2];
  bool bad = false;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int t = lane + 32 * h;
    parent[h] = draft[h] = says[h] = -1;
    if (t < T) {
      const unsigned long long mask = a.tree_mask[row + t], own = 1ull << t, below = mask & (own - 1);
      draft[h] = a.drafts[row + t];
      says[h] = a.sampled[row + t];
      bad |= !(mask & own) || (mask & ~(own | (own - 1)));
      parent[h] = below ? 63 - __clzll((long long)below) : -1;
    }
  }
  if (bad) raise_fault(a.status, PSKV_FAULT_BAD_MASK);
  int cur = 0, kept = 1, place[2] = {lane == 0 ? 0 : -1, -1}, token[2] = {-1, -1};
  for (;;) {
    // (cur goes up with every step, so there are fewer than T of them)
    const int s = __shfl_sync(0xffffffffu, cur < 32 ? says[0] : says[1], cur & 31);
    if (kept - 1 == lane) token[0] = s;
    if (kept - 33 == lane) token[1] = s;
    const uint32_t lo = __ballot_sync(0xffffffffu, s >= 0 && parent[0] == cur && draft[0] == s);
    const uint32_t hi = __ballot_sync(0xffffffffu, s >= 0 && parent[1] == cur && draft[1] == s);
    if (!(lo | hi)) break;
    cur = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
    if (kept == lane) place[0] = cur;
    if (kept - 32 == lane) place[1] = cur;
    ++kept;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (lane + 32 * h < T) {
      a.tokens[row + lane + 32 * h] = token[h];
      a.path[row + lane + 32 * h] = place[h];
    }
  if (lane == 0) a.kept[b] = kept;
}

cudaError_t launch_verify_tree(const VerifyTreeArgs &a, cudaStream_t s) {
  return launch_pdl(pskv_verify_tree, dim3((unsigned)((a.batch + kWarps - 1) / kWarps)), dim3(kWarps * 32), 0, s, a);
}

}  // namespace pskv
