// kv_split.h -- how the attention kernels deal the key tiles of all items out to the CTAs of a launch: the
// arithmetic that every CTA does for itself, and that must agree between them (a host program checks it
// over drawn lists of lengths).
//
// The items' costs (their tiles and a fixed cost) stand one after the other in a sequence, of which CTA k of n takes
// [start(k), start(k + 1)); a boundary near an item's end moves there.  An item whose tiles lie with several CTAs
// is in pieces, one for each CTA from the first to the last.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define KV_SPLIT_FN __host__ __device__ __forceinline__
#else
#define KV_SPLIT_FN inline
#endif

namespace fp4 {

KV_SPLIT_FN int64_t split_min(int64_t a, int64_t b) { return a < b ? a : b; }
KV_SPLIT_FN int64_t split_max(int64_t a, int64_t b) { return a > b ? a : b; }

// Few rows.  An item's tiles come first, then its fixed cost.
struct FewSplit {
  // Boundaries within this many units of an item's end move there: a piece costs two CTAs and its join more than the
  // tiles it moves.
  static constexpr int kSnap = 6;
  static constexpr int kMinShare = 8;  // units of a CTA at least (of all requests together, before boundaries move)
  static KV_SPLIT_FN int64_t ctas(int64_t all, int grid) { return split_max(1, split_min(grid, all / kMinShare)); }
  // where CTA k of n starts in a sequence of `all`, before boundaries move (n <= 160)
  static KV_SPLIT_FN int64_t share(int64_t all, int k, int n) {
    return all <= INT32_MAX / 160 ? (int64_t)((unsigned)all * (unsigned)k / (unsigned)n) : all * k / n;
  }
  // the CTA whose share, so far, holds position `at`
  static KV_SPLIT_FN int owner(int64_t all, int64_t at, int n) {
    return all <= INT32_MAX / 160 ? (int)(((unsigned)(at + 1) * (unsigned)n - 1) / (unsigned)all)
                                  : (int)(((at + 1) * n - 1) / all);
  }
  // by how much a boundary `at` units into an item of `cost` moves
  static KV_SPLIT_FN int move(int at, int cost) {
    if (at <= kSnap && at <= cost - at) return -at;
    return cost - at <= kSnap ? cost - at : 0;
  }
  // CTAs of the first and last piece of a split item that starts at `start`
  static KV_SPLIT_FN int first(int64_t all, int64_t start, int n) { return owner(all, start + kSnap, n); }
  static KV_SPLIT_FN int last(int64_t all, int64_t start, int tiles, int fixed, int n) {
    return owner(all, start + split_min(tiles - 1, tiles + fixed - kSnap - 1), n);
  }
};

// Prompts.  An item's fixed cost comes first, then its tiles.
struct PromptSplit {
  static constexpr int kCost = 3;          // what an item costs beside its key tiles, in tiles
  static constexpr int kSnap = 8;          // a share's end moves to an item's end that is nearer than this
  static constexpr int kShare = 2 * kSnap; // a CTA's share at least
  static KV_SPLIT_FN int64_t shares(int64_t cost, int64_t items, int grid) {
    return split_min(grid, split_max(split_max(cost / kShare, items), 1));
  }
  // where CTA k's share starts, before it moves
  static KV_SPLIT_FN int64_t cut(int64_t k, int64_t shares, int64_t cost) { return split_min(k, shares) * cost / shares; }
  // and after, in an item over [at, next)
  static KV_SPLIT_FN int64_t moved(int64_t cut, int64_t at, int64_t next) {
    return cut - at < kSnap ? at : next - cut < kSnap ? next : cut;
  }
  // the CTA whose share, before moves, holds a unit
  static KV_SPLIT_FN int owner(int64_t unit, int64_t shares, int64_t cost) { return (int)(((unit + 1) * shares - 1) / cost); }
  // CTAs of the first and last piece of an item over [at, next)
  static KV_SPLIT_FN int first(int64_t at, int64_t next, int64_t shares, int64_t cost) {
    return owner(split_min(at + kSnap, next) - 1, shares, cost);
  }
  static KV_SPLIT_FN int last(int64_t at, int64_t next, int64_t shares, int64_t cost) {
    return owner(split_min(next - 1, split_max(at + kSnap - 1, next - kSnap)), shares, cost);
  }
  // tiles of the item before, and in, the piece [pos, stop)
  static KV_SPLIT_FN int skip(int64_t pos, int64_t at) { return (int)split_max(pos - at - kCost, 0); }
  static KV_SPLIT_FN int length(int64_t stop, int64_t at, int skip) { return (int)(stop - at) - kCost - skip; }
};

}  // namespace fp4
