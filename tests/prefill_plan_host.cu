// The division of np_paged_prefill's work, on the host: the functions that the
// plan kernel, the attention's walk and the join run, as they stand, against
// brute force.  argv: seed, number of random batches.  Prints "ok" or the case.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <map>
#include <random>
#include <tuple>
#include <vector>

#include "prefill.cuh"

using namespace npk;
using Unit = std::tuple<int, int, int>;  // row, kv head, unit

#define CHECK(x)                                                     \
  do {                                                               \
    if (!(x)) {                                                      \
      printf("line %d: %s\n", __LINE__, #x);                         \
      return false;                                                  \
    }                                                                \
  } while (0)

static int64_t brute_floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t s = 0;
  for (int64_t i = 0; i < n; ++i) s += (a * i + b) / m;
  return s;
}

static bool floor_sums(std::mt19937& rng) {
  auto pick = [&](int64_t lo, int64_t hi) { return std::uniform_int_distribution<int64_t>(lo, hi)(rng); };
  for (int i = 0; i < 400; ++i) {
    const int64_t n = pick(0, 3000), m = pick(1, 1024), a = pick(0, 1024), b = pick(0, (1ll << 31) - 1);
    const int64_t want = brute_floor_sum(n, m, a, b);
    CHECK(floor_sum(n, m, a, b) == want);
    CHECK(floor_sum_in<int64_t>(n, m, a, b) == want);
    CHECK(floor_sum_in<uint32_t>(n, m, a, b) == want);
  }
  // both sides of the 32-bit form's borders, and its largest arguments
  for (int64_t n : {(1 << 20) - 1, 1 << 20})
    for (int64_t m : {1, 7, 64, 128, 1024, 1025})
      for (int64_t a : {0, 1, 255, 1023, 1024, 1025})
        for (int64_t b : {0ll, 127ll, (1ll << 31) - 1, 1ll << 31, (1ll << 32) + 5}) {
          CHECK(floor_sum(n, m, a, b) == brute_floor_sum(n, m, a, b));
        }
  return true;
}

static int64_t brute_row_prefix(const PrefillParams& p, const PrefillRow& g, int k) {
  int64_t cost = 0;
  const int64_t U = (int64_t)p.tile_tokens * p.tiles;
  for (int64_t u = 0; u < k; ++u) {
    // the positions that the unit's last token sees, in whole kv tiles
    const int64_t end = (int64_t)g.c - g.n + std::min<int64_t>(g.n, (u + 1) * U);
    const int64_t nk = std::max<int64_t>(1, end <= 0 ? 0 : (end + p.bn - 1) / p.bn);
    const bool full = p.tiles == 2 && u * U + p.tile_tokens < g.n;  // both tiles have tokens
    cost += p.unit_cost + nk * (full || p.tiles == 1 ? p.full_cost : p.single_cost);
  }
  return cost;
}

static bool batch(PrefillParams& p, const std::vector<std::pair<int, int>>& rows) {
  std::vector<int32_t> starts{0}, lens;
  for (auto& r : rows) {
    starts.push_back(starts.back() + r.first);
    lens.push_back(r.second);
  }
  int32_t err = 0;
  p.query_starts = starts.data();
  p.context_lens = lens.data();
  p.rows = (int)rows.size();
  p.tokens = starts.back();
  p.err = &err;
  p.max_blocks_per_row = 2147482;
  p.block_size = 1000;
  const int64_t U = (int64_t)p.tile_tokens * p.tiles;

  std::vector<int64_t> pre{0};
  std::map<Unit, int> want;  // kv tiles
  for (int r = 0; r < p.rows; ++r) {
    const PrefillRow g = prefill_row(p, r);
    CHECK(g.q0 == starts[r] && g.n == rows[r].first && g.c == rows[r].second);
    const int units = prefill_units(p, g.n);
    CHECK(units == (g.n + U - 1) / U);
    for (int k : {0, 1, units / 2, units - 1, units})
      if (k >= 0 && k <= units) CHECK(prefill_row_prefix(p, g, units, k) == brute_row_prefix(p, g, k));
    pre.push_back(pre.back() + brute_row_prefix(p, g, units) * p.kv_heads);
    CHECK(prefill_row_cost(p, r) == pre[r + 1] - pre[r]);
    for (int k = 0; k < p.kv_heads; ++k)
      for (int m = 0; m < units; ++m) want[Unit(r, k, m)] = prefill_kv_tiles(p, g, (m + 1) * U);
  }
  CHECK(err == 0);
  std::vector<int4> pos, cuts;
  for (int b = 0; b <= p.ctas; ++b) pos.push_back(prefill_share_start(p, pre.data(), b));
  for (int b = 0; b < p.ctas; ++b) cuts.push_back(prefill_share_cut(p, pos.data(), b));
  auto key = [](const int4& v) { return std::make_tuple(v.x, v.y, v.z, v.w); };
  for (int b = 0; b < p.ctas; ++b) CHECK(key(pos[b]) <= key(pos[b + 1]));

  struct Piece { int kv0, kv1, nk, block; };
  std::map<Unit, std::vector<Piece>> got;
  p.plan = pos.data();
  const int64_t W = pre[p.rows], share = W / std::max<int64_t>(1, std::min<int64_t>(p.ctas, (W + p.min_share - 1) / p.min_share));
  for (int b = 0; b < p.ctas; ++b) {
    PrefillWalk w;
    w.start(p, b);
    int partials[2] = {0, 0};
    int64_t work = 0;
    while (w.next(p)) {
      CHECK(0 <= w.kv0 && w.kv0 < w.kv1 && w.kv1 <= w.nk);
      CHECK(w.whole() == (w.kv0 == 0 && w.kv1 == w.nk));
      got[Unit(w.r, w.kvh, w.m)].push_back({w.kv0, w.kv1, w.nk, b});
      if (!w.whole()) ++partials[w.kv0 > 0 ? 0 : 1];
      work += (int64_t)(w.kv1 - w.kv0) * prefill_tile_cost(p, w.g, w.m) + (w.kv0 == 0 ? p.unit_cost : 0);
      w.advance();
    }
    CHECK(partials[0] <= 1 && partials[1] <= 1);  // a slot of the workspace each
    // a share is no larger than equal ones with both ends moved by 1/16, a tile and a unit's beginning
    CHECK(work <= share + share / 8 + 2 * (p.full_cost + p.unit_cost) + 1);
  }
  CHECK(got.size() == want.size());
  size_t cut = 0;
  for (auto& u : want) {
    const auto& ps = got[u.first];
    CHECK(!ps.empty() && ps[0].kv0 == 0 && ps.back().kv1 == u.second);
    for (size_t i = 0; i < ps.size(); ++i) {
      CHECK(ps[i].nk == u.second);
      if (i) CHECK(ps[i].kv0 == ps[i - 1].kv1 && ps[i].block > ps[i - 1].block);
    }
    if (ps.size() > 1) {
      ++cut;
      // named by the block of its first piece, with all blocks that hold one: the others between are empty
      const int4 c = cuts[ps[0].block];
      CHECK(Unit(c.x, c.y, c.z) == u.first);
      std::vector<int> blocks;
      for (int b = ps[0].block; b <= c.w; ++b)
        if (key(pos[b]) != key(pos[b + 1])) blocks.push_back(b);
      CHECK(blocks.size() == ps.size());
      for (size_t i = 0; i < ps.size(); ++i) CHECK(blocks[i] == ps[i].block);
    }
  }
  for (auto& c : cuts) cut -= c.x >= 0;
  CHECK(cut == 0);
  return true;
}

int main(int argc, char** argv) {
  std::mt19937 rng(argc > 1 ? atoi(argv[1]) : 0);
  const int count = argc > 2 ? atoi(argv[2]) : 100;
  auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  auto one_of = [&](std::vector<int> v) { return v[pick(0, (int)v.size() - 1)]; };
  if (!floor_sums(rng)) return 1;
  for (int i = 0; i < count; ++i) {
    PrefillParams p{};
    const np_dtype dtype = pick(0, 1) ? NP_BF16 : NP_F32;
    p.head_dim = one_of({16, 32, 64, 128, 256});
    p.group = pick(1, dtype == NP_BF16 ? 16 : 8);
    p.kv_heads = one_of({1, 2, 3, 8, 11});
    p.q_heads = p.kv_heads * p.group;
    p.ctas = one_of({1, 2, 7, 148, 152, 160});
    prefill_tiling(p, dtype);
    std::vector<std::pair<int, int>> rows;
    for (int r = one_of({1, 1, 2, 5, 30, 200}); r > 0; --r) {
      const int n = one_of({0, 1, 1, pick(1, 40), pick(1, 2000)});
      rows.push_back({n, one_of({n, n + pick(0, 9000), pick(0, 3 * n + 1), n + pick(0, 100)})});
    }
    if (i % 10 == 9) rows[0] = {pick(1, 700), 2147482000 - pick(0, 300)};  // far positions
    if (!batch(p, rows)) {
      printf("case %d: dtype %d head_dim %d group %d kv_heads %d ctas %d rows", i, dtype, p.head_dim, p.group,
             p.kv_heads, p.ctas);
      for (auto& r : rows) printf(" (%d, %d)", r.first, r.second);
      printf("\n");
      return 1;
    }
  }
  printf("ok\n");
  return 0;
}
