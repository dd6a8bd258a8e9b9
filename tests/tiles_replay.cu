// Replays the schedule of the products' tiles (csrc/tiles.cuh) on the host: every block of every tile is taken once, parts have slots of
// their own, and the join finds them in their order. Prints the first plan that is wrong. No kernel runs.
#include <stdio.h>

#include <map>
#include <random>
#include <vector>

#include "tiles.cuh"

using namespace gs;

struct Work {
  Order order;
  int blocks, pairs, waves, piece, group, span, stacked;
};

static const char* wrong_in(const Plan& p, bool stacked) {
  const Work a{p.order, p.blocks, p.pairs, p.waves, p.piece, p.group, p.span, stacked};
  std::map<std::pair<int, int>, std::vector<int>> taken;       // by tile, how often each block
  struct Slot { int m, n, from, to; };
  std::map<int64_t, Slot> slots;
  const int used = p.piece || p.waves ? p.pairs : p.tiles;
  for (int pair = 0; pair < used; ++pair) {
    Part q;
    for (int i = 0; part_of(a, pair, i, q); ++i) {
      std::vector<int>& t = taken[{q.m, q.n}];
      t.resize(p.blocks);
      if (q.from < 0 || q.to > p.blocks || q.from >= q.to) return "a part's range";
      for (int b = q.from; b < q.to; ++b) ++t[b];
      if (q.whole) continue;
      if (q.slot < 0 || q.slot >= 2 * p.pairs) return "a slot outside the workspace";
      if (!slots.insert({q.slot, {q.m, q.n, q.from, q.to}}).second) return "two parts in one slot";
    }
  }
  if ((int)taken.size() != p.tiles) return "a tile that nobody takes";
  for (const auto& t : taken)
    for (int n : t.second)
      if (n != 1) return "a block that is not taken once";
  if (!p.piece) return slots.empty() ? nullptr : "parts that nobody joins";
  const int split = p.tiles - p.waves * p.pairs;
  if (split <= 0) return "a join of no tiles";
  size_t joined = 0;
  for (int t = 0; t < split; ++t) {
    const Parts parts = parts_of(t, p.blocks, p.piece, p.group, p.span);
    if (parts.count == 1 && !stacked) continue;
    int m, n, at = 0;
    place_of(p.waves * p.pairs + t, p.order, m, n);
    for (int k = 0; k < parts.count; ++k) {
      const auto s = slots.find(parts.slot(k));
      if (s == slots.end()) return "a slot that nobody wrote";
      if (s->second.m != m || s->second.n != n || s->second.from != at) return "a part of another tile, or out of order";
      at = s->second.to;
      ++joined;
    }
    if (at != p.blocks) return "a tile that is not joined whole";
  }
  return joined == slots.size() ? nullptr : "parts that nobody joins";
}

int main() {
  long plans = 0;
  auto check = [&](int64_t rows, int64_t cols, int64_t blocks, int band, int pairs, bool stacked) {
    ++plans;
    const char* what = wrong_in(plan_of(rows, cols, blocks, band, pairs, stacked), stacked);
    if (what) printf("%s: %lld x %lld, %lld blocks, bands of %d, %d pairs%s\n", what, (long long)rows, (long long)cols, (long long)blocks, band, pairs,
                     stacked ? ", stacked" : "");
    return what == nullptr;
  };
  for (int pairs : {74, 66, 5, 1})
    for (int64_t n = 1; n <= pairs; ++n)
      for (int64_t blocks : {1, 2, 3, 4, 5, 7, 8, 11, 16, 37, 100, 1329})
        for (int64_t cols : {n * kTile, (n - 1) * kTile + 1})
          if (!check(kTile, cols, blocks, 8, pairs, true)) return 1;
  std::mt19937 rng(1);
  auto pick = [&](int a, int b) { return (int64_t)std::uniform_int_distribution<int>(a, b)(rng); };
  for (int i = 0; i < 6000; ++i)
    if (!check(pick(0, 20) * kTile + pick(1, kTile), pick(0, 40) * kTile + pick(1, kTile), pick(1, i % 4 ? 90 : 1200), i & 1 ? 8 : 16,
               i % 3 ? 74 : (int)pick(1, 80), false))
      return 1;
  printf("%ld plans\n", plans);
  return 0;
}
