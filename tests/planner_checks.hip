// The host side of the attention and of the overlap checks, run by test_host_planners.py on the CPU
// with the sanitizers: tables of sequences, plans, parts and equal shares of random batches, against
// what the kernels assume of them.  Nothing here launches a kernel.
#include <cstdlib>
#include <map>
#include <random>
#include <set>

#include "../pool_score_top_amd/csrc/layer.hip"
#include "../pool_score_top_amd/csrc/attend.hip"
#include "../pool_score_top_amd/csrc/attend_bwd.hip"

using namespace kpool;

static int g_case;
#define CHECK(x)                                                     \
  do {                                                               \
    if (!(x)) {                                                      \
      printf("case %d, line %d: %s\n", g_case, __LINE__, #x);        \
      exit(1);                                                       \
    }                                                                \
  } while (0)

struct Rng {
  std::mt19937_64 g;
  int64_t upto(int64_t n) { return (int64_t)(g() % (uint64_t)(n + 1)); }  // 0 .. n
};

struct Batch {
  std::vector<int32_t> cu_q, cu_k;
  int nseq, Hq, Hkv, G;
};

// Lengths of every size, empty ones and more queries than keys among them; big: of up to 2^31 tokens.
static Batch batch(Rng &r, bool big) {
  Batch b;
  b.nseq = 1 + (int)r.upto(r.upto(3) ? 8 : 90);
  b.Hkv = 1 << r.upto(3), b.G = 1 + (int)r.upto(r.upto(2) ? 8 : 40), b.Hq = b.Hkv * b.G;
  b.cu_q.push_back(0), b.cu_k.push_back(0);
  const int64_t most = big ? (0x7FFFFF00ll / b.G) / b.nseq : int64_t(1) << r.upto(13);
  for (int s = 0; s < b.nseq; ++s) {
    const int64_t lk = r.upto(3) ? r.upto(most) : 0;
    const int64_t lq = big ? r.upto(std::min<int64_t>(lk, 3000)) : r.upto(2) ? (r.upto(1) ? lk : r.upto(most)) : r.upto(1);
    b.cu_q.push_back((int32_t)(b.cu_q.back() + lq)), b.cu_k.push_back((int32_t)(b.cu_k.back() + lk));
  }
  return b;
}

struct Tile {
  int64_t lq, lk, n0;
};
// The tiles by their numbers, each once and below ntiles, in rising order, and covering every row.
static std::map<int64_t, Tile> tiles_of(const TileTable &t, const int32_t *cu_q, const int32_t *cu_k, int nseq, int G,
                                        int BQ, int64_t ntiles) {
  std::map<int64_t, Tile> out;
  int64_t before = -1, rows = 0;
  for_tiles(t, cu_q, cu_k, nseq, G, BQ, ntiles, [&](int64_t tile, int64_t lq, int64_t lk, int64_t n0) {
    CHECK(tile > before && tile < ntiles);
    before = tile;
    CHECK(n0 >= 0 && n0 < lq * G && n0 % BQ == 0);
    rows += std::min<int64_t>(BQ, lq * G - n0);
    out[tile] = {lq, lk, n0};
  });
  CHECK(rows == (int64_t)cu_q[nseq] * G);
  return out;
}

static int64_t last_position(const Tile &t, int G, int BQ) {
  return (std::min<int64_t>(t.lq * G, t.n0 + BQ) - 1) / G + t.lk - t.lq;
}

static void forward(const Batch &b) {
  const AttendPlan p = plan_attend(b.cu_q.data(), b.cu_k.data(), b.nseq, b.Hq, b.Hkv);
  const int BQ = p.form == AttendPlan::kRows ? 32 : kTileWaves * 32;
  AttendCall c{};
  c.cu_q_host = b.cu_q.data(), c.cu_k_host = b.cu_k.data(), c.nseq = b.nseq, c.Hq = b.Hq, c.Hkv = b.Hkv, c.D = 64;
  c.Tq = b.cu_q.back(), c.Tk = b.cu_k.back();
  alignas(16) static char place[16];
  const AttendArgs a = make_args(c, p, p.nsplit > 1 ? place : nullptr);
  CHECK(a.ntiles <= p.ntiles);
  CHECK(p.nsplit >= 1 && p.chunk > 0 && (p.nsplit == 1 || p.chunk % 128 == 0));
  for (const auto &x : tiles_of(a.table, b.cu_q.data(), b.cu_k.data(), b.nseq, b.G, BQ, a.ntiles)) {
    const int64_t t1 = last_position(x.second, b.G, BQ);
    CHECK(t1 / p.chunk + 1 <= p.nsplit);  // every part has a place; the only one where there is no workspace
  }
}

static void lists(Rng &r) {
  const int64_t Tq = r.upto(int64_t(1) << r.upto(21));
  const int width = (int)r.upto(int64_t(1) << r.upto(30));
  const int Hkv = 1 << r.upto(5), G = 1 + (int)r.upto(70);
  const AttendPlan p = plan_list(Tq, 1, width, Hkv * G, Hkv);
  CHECK(p.nsplit >= 1 && p.chunk > 0 && (int64_t)p.nsplit * p.chunk >= width);
  CHECK(p.nsplit == 1 || ((int64_t)(p.nsplit - 1) * p.chunk < width && p.chunk % 32 == 0));
}

// Every step of every unit in one share, every part in a slot of its own that the sum kernel reads.
static int backward(const Batch &b) {
  const int32_t *cq = b.cu_q.data(), *ck = b.cu_k.data();
  const BwdPlan p = plan_attend_bwd(cq, ck, b.nseq, b.Hq, b.Hkv);
  TileTable t;
  const int64_t qtiles = make_table(t, cq, ck, b.nseq, b.G, kBwdWaves * 32, true);
  CHECK(qtiles <= p.qtiles && p.qsplit >= 1 && p.qchunk > 0);
  for (const auto &x : tiles_of(t, cq, ck, b.nseq, b.G, kBwdWaves * 32, qtiles))
    CHECK(last_position(x.second, b.G, kBwdWaves * 32) / p.qchunk + 1 <= p.qsplit);

  const int64_t ktiles = make_table(t, ck, cq, b.nseq, 1, 128, false);
  CHECK(ktiles <= p.ktiles);
  std::map<int64_t, int64_t> steps;
  for (const auto &x : tiles_of(t, ck, cq, b.nseq, 1, 128, ktiles))
    steps[x.first] = keys_cost(x.second.lq, x.second.lk, x.second.n0, b.G).steps;
  Shares sh;
  const bool cut = make_shares(sh, p.kshares, p.kcost, b.Hkv, t, ck, cq, b.nseq, 1, 128, ktiles,
                               [&](int64_t lk, int64_t lq, int64_t n0) { return keys_cost(lk, lq, n0, b.G); });
  CHECK(sh.n == p.kshares && sh.n <= kMostShares);
  if (sh.n == 0) {
    CHECK(!cut);
    return 0;
  }
  std::map<int64_t, int64_t> done;           // steps of a unit so far
  std::map<int64_t, std::vector<int>> slots;  // of a unit's parts, in order
  std::set<int64_t> whole;
  for (int w = 0; w < sh.n; ++w) {
    const int u0 = sh.unit[w], u1 = sh.unit[w + 1];
    CHECK(u0 <= u1 && sh.step[w] >= 0);
    for (int u = u0; u <= u1; ++u) {
      if (u == u1 && sh.step[w + 1] == 0) break;
      const auto it = steps.find(u / b.Hkv);
      if (it == steps.end()) continue;  // (no such tile)
      const int64_t s0 = u == u0 ? sh.step[w] : 0, s1 = u == u1 ? sh.step[w + 1] : it->second;
      CHECK(s0 == done[u] && s0 <= s1 && s1 <= it->second);
      done[u] = s1;
      if (s1 - s0 == it->second) CHECK(whole.insert(u).second);
      else slots[u].push_back(2 * w + (s0 == 0));
    }
  }
  CHECK(sh.unit[sh.n] >= (steps.empty() ? 0 : steps.rbegin()->first * b.Hkv + b.Hkv) && sh.step[sh.n] == 0);
  std::set<int> used;
  for (int w = 0; w < sh.n; ++w) {  // the sum kernel: the unit that share w begins and does not end
    const int u = sh.unit[w + 1];
    if (sh.step[w + 1] == 0 || (sh.unit[w] == u && sh.step[w] > 0)) continue;
    int end = w + 1;
    while (end < sh.n && sh.unit[end] == u && sh.step[end] > 0) ++end;
    std::vector<int> read{2 * w + 1};
    for (int s = w + 1; s < end; ++s) read.push_back(2 * s);
    CHECK(slots.count(u) && slots[u] == read);
    for (int s : read) CHECK(s < 2 * kMostShares && used.insert(s).second);
    CHECK(whole.insert(u).second);
    slots.erase(u);
  }
  CHECK(slots.empty() && cut == !used.empty());
  for (const auto &x : steps)
    for (int h = 0; h < b.Hkv; ++h) {
      const int64_t u = x.first * b.Hkv + h;
      CHECK(done[u] == x.second && (x.second == 0 || whole.count(u)));
    }
  // (a unit without steps is its share's too: its keys get their zeros)
  const size_t need = attend_bwd_workspace(p, b.cu_q.back(), b.cu_k.back(), b.Hq, b.Hkv, 64);
  CHECK(need >= (size_t)b.cu_q.back() * b.Hq * 8 + (size_t)sh.n * 4 * 128 * 64 * 4);
  return cut;
}

// meets() against the bytes themselves
static void overlaps(Rng &r) {
  const int64_t len = r.upto(9), rows = r.upto(5), pitch = std::max<int64_t>(len, 1) + r.upto(9), n = r.upto(12);
  const int64_t in = 1000, out = 940 + r.upto(160);
  bool any = false;
  for (int64_t i = 0; i < rows; ++i)
    for (int64_t j = 0; j < len; ++j) any |= in + i * pitch + j >= out && in + i * pitch + j < out + n;
  CHECK(meets({"", (const void *)out, n}, {"", (const void *)in, len, rows, pitch}) == any);
  bool flat = false;
  for (int64_t j = 0; j < len; ++j) flat |= in + j >= out && in + j < out + n;
  CHECK(meets({"", (const void *)out, n}, {"", (const void *)in, len}) == flat);
}

int main(int argc, char **argv) {
  const int cases = argc > 1 ? atoi(argv[1]) : 1000;
  int cut = 0;
  for (g_case = 0; g_case < cases; ++g_case) {
    Rng r{std::mt19937_64(g_case)};
    const Batch b = batch(r, g_case % 400 == 399);
    forward(b);
    cut += backward(b);
    lists(r);
    for (int i = 0; i < 20; ++i) overlaps(r);
  }
  printf("ok: %d batches, %d with units across shares\n", cases, cut);
}
