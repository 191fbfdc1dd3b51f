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
// The steps (128 keys each) of all items (row b, KV head) in order form one
// stream, cut into `groups` equal ranges; the `tiles` CTAs of a group take one
// query tile each over the same range, so that they share its K and V in L2.
// A range's part of an item is a piece; an item cut over several groups leaves
// partial results that are joined afterwards.  The cut depends on the lengths
// alone, so results are the same on every run.
constexpr int kTreeCtas = 148;  // one CTA on each SM of a B200

ATTN25_HD int tree_groups(int tiles) { return tiles >= kTreeCtas ? 1 : kTreeCtas / tiles; }

// Steps of one item: its filled slots, then its new tokens.  A row with
// queries but no key still takes one (empty) step, which writes its zeros.
ATTN25_HD int item_steps(int len, int n_new, bool has_new) {
  if (n_new == 0) return 0;
  const int s = (len + 127) / 128 + (has_new ? (n_new + 127) / 128 : 0);
  return s > 0 ? s : 1;
}

ATTN25_HD long long range_start(long long total, int groups, int g) { return total * g / groups; }

// Partial results: group g keeps the piece that begins where its range begins
// in slot 2 g, and the one that begins inside its range in slot 2 g + 1.
ATTN25_HD int partial_slot(int g, bool at_range_start) { return 2 * g + (at_range_start ? 0 : 1); }

// Whether the boundary before group g (1 <= g < groups) is the first inside
// the item [i0, i1): the block of that boundary joins the item.
ATTN25_HD bool joins_item(long long total, int groups, int g, long long i0, long long i1) {
  const long long at = range_start(total, groups, g);
  return at > i0 && at < i1 && range_start(total, groups, g - 1) <= i0;
}

}  // namespace attn25
