// Host-side checks of the cache attention's work list (no GPU needed): the even shares of csa_attn.cuh
// cover the work, differ by one at most, and fit the fields that carry them, up to the largest
// calls that the entry point takes. Prints "ok <checks>" or the failures; run by
// tests/test_attn_plan.py.
#include <cstdio>

#include "csa_attn.cuh"

int main() {
  long checks = 0, failures = 0;
  auto expect = [&](bool cond, const char* what, int64_t work, int workers, int i) {
    ++checks;
    if (!cond && ++failures < 20)
      std::printf("FAIL %s (work=%lld workers=%d i=%d)\n", what, static_cast<long long>(work), workers, i);
  };
  // units (rows in 64ths, at most one a row: below 2^31) times their tiles (2^31 entries in 128ths) and cost
  const int64_t works[] = {0, 1, 5, 151, 152, 153, 4000, int64_t{1} << 31, (int64_t{1} << 31) * 152 - 1,
                           (int64_t{1} << 31) * 152 + 1, (int64_t{1} << 20) * ((int64_t{1} << 24) + 5),
                           ((int64_t{1} << 31) - 257) * ((int64_t{1} << 24) + 5)};
  const int counts[] = {1, 2, 76, 148, 152};
  for (int64_t work : works)
    for (int workers : counts) {
      const csa::AttnShares share(work, workers);
      expect(share(0) == 0 && share(workers) == work, "shares cover the work", work, workers, 0);
      for (int i = 0; i < workers; ++i) {
        const int64_t mine = share(i + 1) - share(i);
        expect(mine >= 0 && mine <= work / workers + 1, "shares are even", work, workers, i);
        csa::AttnStart start{};
        start.left = mine;
        expect(start.left == mine, "a share fits its field", work, workers, i);
      }
    }
  if (failures) return 1;
  std::printf("ok %ld\n", checks);
  return 0;
}
