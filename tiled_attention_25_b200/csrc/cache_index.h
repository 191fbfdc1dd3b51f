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

}  // namespace attn25
