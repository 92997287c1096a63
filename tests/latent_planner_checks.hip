// Shares of the latent attention, on the CPU: random batches of units, long and short ones beside one
// another.  Every tile of every unit is in one share, a part that the join reads is one that a share left,
// and positions stay within 32 bits at the largest calls.
#include "../pool_score_top_amd/csrc/latent.hip"

#include <cstdio>
#include <cstdlib>
#include <vector>

using namespace kpool;

#define CHECK(x)                                                       \
  do {                                                                 \
    if (!(x)) {                                                        \
      std::printf("batch %d: %s (line %d)\n", batch, #x, __LINE__);    \
      return 1;                                                        \
    }                                                                  \
  } while (0)

static uint64_t state = 1;
static int upto(int n) {  // 0 .. n - 1
  state = state * 6364136223846793005ull + 1442695040888963407ull;
  return (int)((state >> 33) % (uint64_t)n);
}

static int check(int batch) {
  const int units = 1 + upto(batch % 50 == 0 ? 3000 : 60);
  const int lengths[] = {1, 1, 2, 3, 4, 5, 7, 8, 9, 12, 40, 1 + upto(3000), 1 + upto(200)};
  std::vector<int> kt(units), start(units);
  int64_t tiles = 0;
  for (int &k : kt) k = lengths[upto(sizeof(lengths) / sizeof(int))], tiles += k;
  if (batch % 50 == 1) kt[upto(units)] += (1 << 28) - 1 - (int)tiles, tiles = (1 << 28) - 1;  // the most tiles
  const int most[] = {1, 2, 8, 100, kMostShares};
  const LatentCosts costs((int)tiles, units, most[upto(5)]);
  int64_t at = 0;
  for (int u = 0; u < units; ++u) start[u] = (int)at, at += kt[u] + costs.fixed;
  CHECK(at == costs.total && at < (int64_t(1) << 31) && costs.shares >= 1 && costs.shares <= tiles);
  CHECK(share_start(costs.total, costs.shares, 0) == 0);
  CHECK(share_start(costs.total, costs.shares, costs.shares) == costs.total);
  for (int u = 0; u < units; ++u) {
    int done = 0, first = -1, parts = 0;
    for (int s = 0; s < costs.shares; ++s) {
      const int pos = share_start(costs.total, costs.shares, s), hi = share_start(costs.total, costs.shares, s + 1);
      CHECK(pos < hi);
      // (the units that the kernel looks at: from the one that holds pos to the last that begins before hi)
      if (hi <= start[u] || pos >= start[u] + kt[u] + costs.fixed) continue;
      const int k0 = costs.cut(pos, start[u], kt[u]), k1 = costs.cut(hi, start[u], kt[u]);
      CHECK(k0 >= 0 && k1 <= kt[u]);
      if (k0 >= k1) continue;
      CHECK(k0 == done);
      if (first < 0) first = s;
      CHECK(s == first + parts);
      done = k1, ++parts;
    }
    CHECK(done == kt[u]);
    // the join of a unit in parts: the shares behind the first that begin before its last cut
    if (parts > 1) {
      const int end = start[u] + costs.fixed + kt[u] - costs.least + 1;
      int read = 1;
      for (int s = first + 1; s < costs.shares && share_start(costs.total, costs.shares, s) < end; ++s) ++read;
      CHECK(read == parts);
    }
  }
  return 0;
}

int main(int argc, char **argv) {
  const int n = argc > 1 ? std::atoi(argv[1]) : 1000;
  for (int batch = 0; batch < n; ++batch)
    if (check(batch)) return 1;
  std::printf("ok: %d batches\n", n);
  return 0;
}
