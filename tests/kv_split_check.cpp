// Deals drawn lists of items out as the attention kernels do, CTA by CTA from the shared arithmetic, and checks that every
// tile is with exactly one CTA, that the pieces of a split item are numbered in the order of its tiles with the count each
// CTA expects, and that no two pieces share a place in the workspace or two split items an arrival word.
//   kv_split_check LISTS
#include <cstdio>
#include <cstdlib>
#include <set>
#include <utility>
#include <vector>

#include "../block_scaled_fp4_fp_gb300/csrc/kv_split.h"

using namespace fp4;

static uint64_t state = 88172645463325252ull;
static uint64_t next_random() {
  state ^= state << 13;
  state ^= state >> 7;
  state ^= state << 17;
  return state;
}
static int64_t draw(int64_t lo, int64_t hi) { return lo + (int64_t)(next_random() % (uint64_t)(hi - lo + 1)); }
// spread over the logarithm
static int64_t draw_log(int64_t hi) {
  int64_t v = hi;
  for (int64_t k = draw(0, 20); k > 0 && v > 1; --k) v = v * 2 / 3;
  return draw(v / 2, v);
}

struct Piece {
  int cta, from, to, slot, first, count;
};

static int failures = 0;
static void fail(const char* what, int list, int item) {
  if (++failures <= 20) std::printf("list %d, item %d: %s\n", list, item, what);
}

// pieces of every item, in CTA order
static void check(const std::vector<int>& tiles, const std::vector<std::vector<Piece>>& pieces, int list) {
  std::set<std::pair<int, int>> slots;
  std::set<int> words;
  for (size_t i = 0; i < tiles.size(); ++i) {
    int at = 0;
    for (const Piece& p : pieces[i]) {
      if (p.from != at || p.to <= p.from) fail("a tile is missing or done twice", list, (int)i);
      at = p.to;
    }
    if (at != tiles[i]) fail("its last tiles are missing", list, (int)i);
    if (pieces[i].size() < 2) continue;
    for (size_t k = 0; k < pieces[i].size(); ++k) {
      const Piece& p = pieces[i][k];
      if (p.cta != p.first + (int)k || p.count != (int)pieces[i].size() || p.first != pieces[i][0].first)
        fail("the CTAs do not agree on its pieces", list, (int)i);
      if (!slots.insert({p.cta, p.slot}).second) fail("two pieces in one place", list, (int)i);
    }
    if (!words.insert(pieces[i][0].first).second) fail("two items on one arrival word", list, (int)i);
  }
}

static void few(const std::vector<int>& tiles, int fixed, int grid, int list) {
  std::vector<int64_t> start;
  int64_t all = 0;
  for (int t : tiles) start.push_back(all), all += t > 0 ? t + fixed : 0;
  std::vector<std::vector<Piece>> pieces(tiles.size());
  if (all > 0) {
    const int n = (int)FewSplit::ctas(all, grid);
    auto boundary = [&](int k) {
      const int64_t f = FewSplit::share(all, k, n);
      if (f == all) return all;
      size_t i = 0;
      while (tiles[i] == 0 || f >= start[i] + tiles[i] + fixed) ++i;
      return f + FewSplit::move((int)(f - start[i]), tiles[i] + fixed);
    };
    for (int k = 0; k < n; ++k) {
      const int64_t f0 = boundary(k), f1 = boundary(k + 1);
      for (size_t i = 0; i < tiles.size(); ++i) {
        const int64_t from = split_max(f0, start[i]) - start[i], to = split_min(split_min(f1, start[i] + tiles[i]) - start[i], tiles[i]);
        if (tiles[i] == 0 || from >= to) continue;
        const int first = FewSplit::first(all, start[i], n), last = FewSplit::last(all, start[i], tiles[i], fixed, n);
        pieces[i].push_back({k, (int)from, (int)to, k == first, first, last - first + 1});
      }
    }
  }
  check(tiles, pieces, list);
}

static void prompts(const std::vector<int>& tiles, int grid, int list) {
  std::vector<int64_t> before{0};
  for (int t : tiles) before.push_back(before.back() + PromptSplit::kCost + t);
  const int64_t cost = before.back();
  std::vector<std::vector<Piece>> pieces(tiles.size());
  std::vector<int> described(tiles.size(), 0);
  const int64_t n = PromptSplit::shares(cost, (int64_t)tiles.size(), grid);
  auto item_at = [&](int64_t unit) {
    size_t i = 0;
    while (before[i + 1] <= unit) ++i;
    return i;
  };
  auto boundary = [&](int64_t k) {
    const int64_t cut = PromptSplit::cut(k, n, cost);
    if (cut >= cost) return cost;
    const size_t i = item_at(cut);
    return PromptSplit::moved(cut, before[i], before[i + 1]);
  };
  for (int k = 0; k < grid; ++k) {
    const int64_t end = boundary(k + 1);
    for (int64_t pos = boundary(k); pos < end;) {
      const size_t i = item_at(pos);
      const int64_t at = before[i], next = before[i + 1], stop = split_min(next, end);
      const int first = PromptSplit::first(at, next, n, cost), count = PromptSplit::last(at, next, n, cost) - first + 1;
      const int skip = PromptSplit::skip(pos, at), len = PromptSplit::length(stop, at, skip);
      ++described[i];
      if (tiles[i] > 0) pieces[i].push_back({k, skip, skip + len, k == first, first, count});
      else if (count != 1 || len != 0) fail("an item without tiles is in pieces", list, (int)i);
      if (count == 1 && stop != next) fail("a whole item is cut", list, (int)i);
      pos = stop;
    }
  }
  for (size_t i = 0; i < tiles.size(); ++i)
    if (described[i] == 0) fail("no CTA has it", list, (int)i);
  check(tiles, pieces, list);
}

int main(int argc, char** argv) {
  const int lists = argc > 1 ? std::atoi(argv[1]) : 1000;
  for (int list = 0; list < lists; ++list) {
    std::vector<int> tiles((size_t)draw_log(608));
    if (tiles.empty()) tiles.push_back(1);
    const int64_t top = draw_log(list % 50 == 0 ? 16000000 : 3000);
    const int alike = (int)draw(0, 2);
    for (int& t : tiles) t = (int)(alike == 0 ? top : alike == 1 ? draw(0, top) : draw_log(top));
    const int grid = (int)(list % 4 ? 152 : draw(1, 160));
    few(tiles, list % 2 ? 8 : 5, grid, list);
    prompts(tiles, grid, list);
  }
  std::printf("%d lists, %d failures\n", lists, failures);
  return failures != 0;
}
