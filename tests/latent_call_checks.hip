// Calls of the latent attention on the CPU, as the kernel and the entry points see them: the keys that a
// share walks, block by block; the parts that shares leave, within the workspace that the call's plan asks
// for, whatever the lengths on the device.  Nothing here launches a kernel.
#include "../pool_score_top_amd/csrc/latent.hip"

#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

using namespace kpool;

static int g_case;
#define CHECK(x)                                                     \
  do {                                                               \
    if (!(x)) {                                                      \
      std::printf("case %d, line %d: %s\n", g_case, __LINE__, #x);   \
      std::exit(1);                                                  \
    }                                                                \
  } while (0)

struct Rng {
  std::mt19937_64 g;
  int64_t upto(int64_t n) { return (int64_t)(g() % (uint64_t)(n + 1)); }  // 0 .. n
};

constexpr int kLongest = 0x7FFFFF00;  // the most tokens of a sequence

// Keys [lo, hi) in blocks of `size`: each once, in order, and an end.
static void walk(int lo, int hi, int size) {
  const int64_t most = hi > lo ? ((int64_t)hi - lo + size - 1) / size : 0;
  int64_t next = lo, blocks = 0;
  for (KeyBlocks b(lo, hi); b.any(); b.next(size), ++blocks) {
    CHECK(blocks < most && b.at() == next);
    const int64_t here = std::min<int64_t>(size, hi - next);
    for (int64_t i : {int64_t(0), here - 1, here, (int64_t)size - 1})
      if (i < size) CHECK(b.key((int)i) == (i < here ? next + i : -1));
    next += here;
  }
  CHECK(blocks == most && (hi <= lo || next == hi));
}

// One query token of `heads` heads over each of the lengths, by the shares that the device finds.
static void walk_shares(const std::vector<int> &lens, int heads, int most) {
  std::vector<int32_t> cu;
  for (size_t s = 0; s <= lens.size(); ++s) cu.push_back((int32_t)s);
  const LatentPlan p = plan_latent(cu.data(), (int)lens.size(), heads, most);
  CHECK(p.tiles < 1 << 28);
  std::vector<int> kt;
  int64_t tiles = 0;
  const int per = (heads + 16 * p.rb - 1) / (16 * p.rb);  // units of a sequence
  for (int len : lens) kt.push_back(std::max(1, (len + 63) / 64)), tiles += (int64_t)per * kt.back();
  CHECK(tiles <= p.tiles);
  const LatentCosts costs((int)tiles, per * (int)lens.size(), p.shares);
  int start = 0;
  for (size_t u = 0; u < kt.size() * per; ++u) {
    const int len = lens[u / per], k = kt[u / per];
    for (int s = 0; s < costs.shares; ++s) {
      const int pos = share_start(costs.total, costs.shares, s), hi = share_start(costs.total, costs.shares, s + 1);
      if (hi <= start || pos >= start + k + costs.fixed) continue;
      const int k0 = costs.cut(pos, start, k), k1 = costs.cut(hi, start, k);
      if (k0 < k1) walk(k0 * kLatentKeys, std::min(k1 * kLatentKeys, len), 1024);
    }
    start += k + costs.fixed;
  }
}

// The parts of a call by the shares that the device finds: each in a slot of its own, within the workspace.
// `units` tiles of rows with kt[u] key tiles.
static void parts(const LatentPlan &p, int R, const std::vector<int> &kt) {
  int64_t tiles = 0;
  for (int k : kt) tiles += k;
  CHECK((int64_t)kt.size() == p.units && tiles <= p.tiles && p.shares >= 1 && p.shares <= kMostShares);
  if (kt.empty()) return;
  const LatentCosts costs((int)tiles, (int)kt.size(), p.shares);
  CHECK(costs.shares >= 1 && costs.shares <= p.shares);
  const int BQ = 16 * p.rb;
  const int64_t most = (int64_t)latent_workspace(p, R);
  std::vector<char> used(2 * p.shares);
  int64_t at = 0;
  size_t u = 0;
  for (int s = 0; s < costs.shares; ++s) {
    const int pos = share_start(costs.total, costs.shares, s), hi = share_start(costs.total, costs.shares, s + 1);
    while (at + kt[u] + costs.fixed <= pos) at += kt[u++] + costs.fixed;
    int64_t start = at;
    for (size_t v = u; v < kt.size() && start < hi; start += kt[v++] + costs.fixed) {
      const int k0 = costs.cut(pos, (int)start, kt[v]), k1 = costs.cut(hi, (int)start, kt[v]);
      if (k0 >= k1 || k1 - k0 == kt[v]) continue;
      CHECK(p.shares > 1);  // (one share leaves no parts)
      const int64_t slot = 2 * s + (k0 == 0);
      CHECK(slot < 2 * p.shares && !used[slot]);
      used[slot] = 1;
      const int64_t part_o = cut_bytes(p.shares), part_lse = part_o + (int64_t)2 * p.shares * BQ * R * 4;
      CHECK(part_o + (slot + 1) * BQ * R * 4 <= part_lse && part_lse + (slot + 1) * BQ * 4 <= most);
    }
  }
  CHECK(p.shares == 1 || (int64_t)p.shares * (int64_t)sizeof(LatentCut) <= cut_bytes(p.shares));
}

static void random_call(Rng &r) {
  const int H = 1 + (int)r.upto(r.upto(1) ? 20 : 150), R = 8 * (1 + (int)r.upto(63));
  const int nseq = 1 + (int)r.upto(r.upto(2) ? 8 : 400), most = (int)r.upto(r.upto(1) ? 300 : 60000);
  std::vector<int32_t> cu{0};
  for (int s = 0; s < nseq; ++s) cu.push_back(cu.back() + (int)(r.upto(9) ? r.upto(3) : r.upto(200)));
  const LatentPlan whole = plan_latent(cu.data(), nseq, H, most);
  std::vector<int> kt;
  for (int s = 0; s < nseq; ++s) {
    const int units = (int)(((int64_t)(cu[s + 1] - cu[s]) * H + 16 * whole.rb - 1) / (16 * whole.rb));
    kt.insert(kt.end(), units, std::max(1, (int)(((r.upto(1) ? r.upto(most) : most) + 63) / 64)));
  }
  parts(whole, R, kt);
  const int width = (int)(r.upto(2) ? r.upto(3000) : r.upto(2));  // (0 among them)
  const LatentPlan lists = plan_latent_list(cu.back(), H, width);
  const int64_t units = (int64_t)cu.back() * ((H + 16 * lists.rb - 1) / (16 * lists.rb));
  parts(lists, R, std::vector<int>(units, std::max(1, (width + 63) / 64)));
}

int main(int argc, char **argv) {
  const int n = argc > 1 ? std::atoi(argv[1]) : 1000;
  Rng r{std::mt19937_64(7)};
  for (int size : {1024, 2048})
    for (int left : {0, 1, 63, 64, 65, 1023, 1024, 1025, 2047, 2048, 2049, 5000}) {
      walk(kLongest - left, kLongest, size);
      walk(64, 64 + left, size);
      walk(left, 0, size);
      walk(left, -0x7FFFFF00 + left, size);
    }
  walk_shares({kLongest, 320}, 4, kLongest);
  walk_shares({320, kLongest, 1, 0}, 64, kLongest);
  for (g_case = 0; g_case < n; ++g_case) {
    const int64_t lo = r.upto(kLongest / 64) * 64;
    walk((int)lo, (int)std::min<int64_t>(kLongest, lo + r.upto(300000)), r.upto(1) ? 1024 : 2048);
    random_call(r);
    if (g_case % 100) continue;
    std::vector<int> lens;
    const int64_t most = r.upto(2) ? kLongest - r.upto(5000) : 1 + r.upto(1000000);
    for (int64_t s = r.upto(3); s >= 0; --s) lens.push_back((int)(r.upto(1) ? most : r.upto(most)));
    walk_shares(lens, 1 + (int)r.upto(80), (int)most);
  }
  std::printf("ok: %d batches\n", n);
  return 0;
}
