// Index arithmetic of the paged KV cache, shared by the kernels and the host
// (plain C++, so that it can be exercised without a GPU).
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define ATTN25_HD __host__ __device__ __forceinline__
#else
#define ATTN25_HD inline
#endif

namespace attn25 {

constexpr int kMaxCapacity = 1 << 20;  // slots of a batch row
constexpr int kMaxTreeTokens = 1024;   // new tokens of one attn_tree_fwd call

// page sizes that tile the kernels' 128-key tiles evenly, or are tiled by them
ATTN25_HD bool page_size_ok(int ps) {
  return ps == 16 || ps == 32 || ps == 64 || (ps >= 128 && ps % 128 == 0);
}

struct CacheIndex {
  const int32_t* table;  // [B][max_pages], or nullptr: pages b * max_pages + i
  const int32_t* lens;   // [B]
  int B, Hkv, num_pages, page_size, max_pages, capacity;
};

ATTN25_HD int clamp_count(int raw, int most, bool& bad) {
  if (raw < 0) {
    bad = true;
    return 0;
  }
  if (raw > most) {
    bad = true;
    return most;
  }
  return raw;
}

// Page i (0 <= i < max_pages) of row b; -1 if the table names no page of the pool.
ATTN25_HD int page_at(const CacheIndex& c, int b, int i) {
  const long long at = static_cast<long long>(b) * c.max_pages + i;
  const long long p = c.table != nullptr ? c.table[at] : at;
  return p >= 0 && p < c.num_pages ? static_cast<int>(p) : -1;
}

// Entry (b, hk, slot) of a [B][Hkv][capacity] array.
ATTN25_HD long long slot_entry(const CacheIndex& c, int b, int hk, int slot) {
  return (static_cast<long long>(b) * c.Hkv + hk) * c.capacity + slot;
}

// ------------------------------------------------------------------ query tiles
//
// A KV head's query rows (its G query heads x T new tokens) are cut into tiles
// of at most 128 rows = TMEM lanes: head_tile heads x tok_tile tokens, row
// r = token * head_tile + head, so that one TMA box of a [token][head] order
// fills a tile.  More than 128 heads to one KV head take several head chunks.
struct RowTiles {
  int head_tile, tok_tile, rows, head_chunks, tok_tiles, tiles;
};

ATTN25_HD RowTiles row_tiles(int G, int T) {
  RowTiles r;
  r.head_tile = G < 128 ? G : 128;
  r.tok_tile = 128 / r.head_tile < T ? 128 / r.head_tile : T;
  r.rows = r.head_tile * r.tok_tile;
  r.head_chunks = (G + r.head_tile - 1) / r.head_tile;
  r.tok_tiles = (T + r.tok_tile - 1) / r.tok_tile;
  r.tiles = r.head_chunks * r.tok_tiles;
  return r;
}

// ------------------------------------------------------------------ work split
//
// An item is one row's work for one KV head: its steps of 128 keys.  `groups`
// CTA groups share the items; the `tiles` CTAs of a group take one query tile
// each over the same steps, so that they share their K and V in L2.  What a
// group does of an item is a piece.  Starting and ending a piece costs a CTA
// about as much as four steps, so:
//   few items (at most one to a group): every group gets one piece; an item of s
//     steps is cut into ceil(s / L) even ones, L the least for which the groups suffice;
//   more items: their steps in order form one stream, cut into `groups` equal
//     ranges, where a cut within kSnap steps of an item's end moves there.
// The pieces of a cut item leave partial results, which are joined.  The cut
// depends on the lengths alone, so results are the same on every run.
constexpr int kTreeCtas = 148;  // one CTA on each SM of a B200
constexpr int kSnap = 4;

ATTN25_HD int tree_groups(int tiles) { return tiles >= kTreeCtas ? 1 : kTreeCtas / tiles; }

// Steps of one item: its filled slots, then its new tokens.  A row with
// queries but no key still takes one (empty) step, which writes its zeros.
ATTN25_HD int item_steps(int len, int n_new, bool has_new) {
  if (n_new == 0) return 0;
  const int s = (len + 127) / 128 + (has_new ? (n_new + 127) / 128 : 0);
  return s > 0 ? s : 1;
}

// floor(x y / z), x y below 2^63 (in 32 bits where it fits: y is at most 148)
ATTN25_HD long long mul_div(long long x, int y, long long z) {
  if (x < (1 << 24) && z < (1 << 24)) return static_cast<uint32_t>(x) * static_cast<uint32_t>(y) / static_cast<uint32_t>(z);
  return x * y / z;
}

// Steps [begin, end) of the k-th of n even pieces of an item of s steps.
ATTN25_HD int even_cut(int s, int k, int n) { return static_cast<int>(mul_div(s, k, n)); }

// The stream's raw cut before group g, and the same moved to the end of the
// item [i0, i1) that holds it if that is near.
ATTN25_HD long long raw_cut(long long total, int groups, int g) { return mul_div(total, g, groups); }
ATTN25_HD long long snapped(long long at, long long i0, long long i1) {
  if (at - i0 < kSnap) return i0;
  return i1 - at < kSnap ? i1 : at;
}

// The cuts that stay inside the item [i0, i1): those before the groups first,
// first + 1, ..., first + count - 1.
struct InnerCuts {
  int first, count;
};
ATTN25_HD InnerCuts inner_cuts(long long total, int groups, long long i0, long long i1) {
  InnerCuts c;
  // raw_cut(g) >= x  <=>  g >= x groups / total
  const long long a = i0 + kSnap, z = i1 - kSnap + 1;
  c.first = static_cast<int>(mul_div(a, groups, total));
  while (raw_cut(total, groups, c.first) < a) ++c.first;
  int end = z > 0 ? static_cast<int>(mul_div(z, groups, total)) : 0;
  while (raw_cut(total, groups, end) < z) ++end;
  if (c.first < 1) c.first = 1;
  if (end > groups) end = groups;
  c.count = end > c.first ? end - c.first : 0;
  return c;
}

// Partial results of a cut item of the stream: the piece from the cut before
// group g in slot 2 g, the piece from the item's begin in the slot before its
// first inner cut's.  (Few items: a group's piece in the slot of its number.)
ATTN25_HD int slot_from_cut(int g) { return 2 * g; }
ATTN25_HD int slot_from_begin(int first_cut) { return 2 * first_cut - 1; }

// The counters of the pieces written, one to a cut item (known by the group of
// its first inner cut, or of its first piece), lie at the head of the workspace.
constexpr int kTreeCounterBytes = 1024;

// --------------------------------------------------------------- eviction plan
//
// Shared memory of one CTA of a plan, of kPlanSmem bytes at most: `fixed` bytes
// of counters, then the ranks of `held` slots (4 bytes each), then a flag byte
// to four of its `share` of the slots.  The flags are always there; the ranks of
// a share that does not fit beside them are formed again from global memory.
constexpr int kPlanSmem = 227 * 1024;
constexpr int kPlanMaxCtas = 8;  // CTAs of a cluster, which share a head
constexpr int kPlanThreads = 1024;

struct PlanLayout {
  int ctas, share, held, kept, bytes;  // kept: offset of the flags
};

ATTN25_HD int plan_share(int slots, int ctas) { return ((slots + ctas - 1) / ctas + 31) / 32 * 32; }

// CTAs to a head: as many as it takes for a share's flags to fit (two above
// about 796 thousand slots); more while one to an SM is not exceeded and each
// keeps a quad for every thread.
ATTN25_HD PlanLayout plan_layout(int heads, int capacity, int sms, int fixed) {
  PlanLayout p;
  p.ctas = 1;
  while (p.ctas < kPlanMaxCtas &&
         (fixed + plan_share(capacity, p.ctas) / 4 > kPlanSmem ||
          (heads * p.ctas * 2 <= sms && capacity / (p.ctas * 2) >= 4 * kPlanThreads)))
    p.ctas *= 2;
  p.share = plan_share(capacity, p.ctas);
  const int room = (kPlanSmem - fixed - p.share / 4) / 16 * 4;
  p.held = p.share < room ? p.share : room;
  p.kept = fixed + p.held * 4;
  p.bytes = p.kept + p.share / 4;
  return p;
}

}  // namespace attn25
