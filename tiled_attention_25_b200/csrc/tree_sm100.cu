// Attention of new tokens over a paged KV cache and over their own ancestors
// (attn_tree_fwd), for sm_100a.
//
// A KV head's query rows (G heads x T tokens) are the rows of an M = 128 tile;
// its keys come in steps of 128: pages of the cache, then the new tokens.
// With few rows a step's two products cost 512 tensor clocks against the
// ~2800 clocks in which HBM delivers its 64 KB of K and V to one SM (its 148th
// share), so the kernel is a stream of K and V: what counts is that every SM
// has an equal share of the bytes of all rows, whatever their lengths, and
// always enough copies in flight (160 KB or more of rings).
//
// Work: the steps of all (row, KV head) items form one stream that is cut into
// equal ranges (cache_index.h), one CTA per SM.  The pieces of an item cut by a
// range boundary leave (m, l, O) partials in fp32, and the CTA that writes the
// last of them joins them (a second launch for the joins took 4 to 12 us more);
// the other items are written out directly.
//
// Warp roles (384 threads):
//   warps 0-3  softmax of the even steps of a piece
//   warps 4-7  softmax of the odd steps
//   warp  8    MMA issuer
//   warp  9    walks the ranges, publishes the pieces, loads K
//   warps 10, 11  load V, and Q
// (One producer for all held the stream up: a 128-key copy from pages of 64 rows
// takes a warp ~1400 clocks of page lookups and issue, and HBM delivers one
// every 1400.)
//
// Few rows would leave three of the four lane quarters, and their warps, idle
// while one warp works through 128 scores a row in ~3000 clocks.  So a tile of
// up to 32 (64) rows is loaded 4 (2) times over, S comes out R = 4 (2) times,
// and each copy's warps take 128 / R of the step's keys: P is zero elsewhere in
// their lanes, and every copy keeps its own (m, l, O) of its keys.  Together
// with the two warpgroups, 2 R states of a row are joined at the end of a
// piece, through shared memory.  Each running maximum moves only when exceeded
// by more than 2^8, as in the forward kernel.  P is rounded to bf16 for the PV
// product (half a step, 2^-8 relative, the forward kernel's choice: the product
// then runs at the full bf16 rate straight from tensor memory); sums, maxima
// and O stay in fp32.
//
// Keys a row does not see are masked by selection before the softmax, so K
// may hold anything there; V rows behind the last valid key of a step are
// overwritten with zeros in shared memory before the product (0 x NaN).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cache.h"
#include "kernel_common.cuh"
#include "launch.h"

namespace attn25 {

namespace {

constexpr int kTreeThreads = 384;
constexpr float kTreeRescale = 8.0f;
constexpr int kStageCols = 16;  // columns of O joined at a time

template <int D>
struct TreeCfg {
  static constexpr int kTileBytes = TILE * D * 2;
  // a ring each for K and V (96 + 64 KB, or 96 + 80), and 32 KB in which the
  // states of a row are joined: two buffers of 128 rows x 16 columns a warpgroup
  static constexpr int kKStages = D == 128 ? 3 : 6;
  static constexpr int kVStages = D == 128 ? 2 : 5;
  static constexpr int kKOff = kTileBytes;  // after Q
  static constexpr int kVOff = kKOff + kKStages * kTileBytes;
  static constexpr int kStageOff = kVOff + kVStages * kTileBytes;
  static constexpr int kBarOff = kStageOff + 4 * TILE * kStageCols * 4;
  static constexpr int kSmemBytes = kBarOff + 1024;
  static constexpr int kAllocBytes = kSmemBytes + 1024;  // + alignment slack
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, false, true);
};

// A piece: steps [j0, j0 + n) of item (b, hk).
struct Piece {
  int32_t b, hk, j0, n;     // b < 0: the end
  int32_t len, n_new;       // filled slots and new tokens of the row
  int32_t slot;             // partial-result slot, or -1: the whole item
  // of a cut item: its pieces, the slots of the first, the second, and from one
  // to the next, and its counter
  int32_t pieces, slot0, slot1, slot_step, counter;
};

struct TreeBarriers {
  uint64_t list_full[2], list_empty[2];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t o_final, ml_ready, staged[2], epi_done, written, counted;
  int32_t last;  // this CTA's piece is the last of its item to be written
  uint64_t drain;
  uint64_t k_full[6], k_empty[6], v_full[5], v_empty[5];
  uint32_t tmem_base, abort_flag, never_set;
  Piece piece[2];
};
static_assert(sizeof(TreeBarriers) <= 1024, "barrier block");

constexpr int kListReaders = 11;  // the MMA warp, the V and Q producers and the 8 softmax warps (lane 0 each)

// A place in a ring.
template <int STAGES>
struct RingPos {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == STAGES) {
      slot = 0;
      phase ^= 1;
    }
  }
};

__device__ __forceinline__ void flag_index(int* status) { atomicCAS(status, 0, kErrIndex); }

// The bounded wait, its polling loop out of line: with few rows one softmax
// warp of a quarter works alone, and what limits it is the fetch of its own
// instructions between those of five other roles.
__device__ __forceinline__ bool tree_wait(uint32_t bar, uint32_t parity, const WaitCtl& w) {
  return mbar_wait_warp_ool(bar, parity, w);
}

struct TreeParams {
  TreeArgs a;
  RowTiles rt;
  int groups;
  int* counters;   // [group][tile]: pieces written of a cut item
  float* part_o;   // [slot][tile][rows][D]
  float2* part_ml; // [slot][tile][rows]
  uint64_t wait_ns;
  // pages and steps: pages of up to 128 rows, 1 << page_lg to a step; larger
  // ones hold page_steps > 1 steps: step / page_steps = umulhi(step, page_magic)
  // (exact: step and page_steps are at most 8192)
  int page_lg, page_steps;
  uint32_t page_magic;
  uint32_t head_magic;  // row / head_tile = row * head_magic >> 16 (rows below 128)
};

// The stream of items as a warp walks it: 32 rows' lengths at a time, one to a lane.
struct RowScan {
  int base;              // first row of the window
  int len, n_new, steps; // this lane's row (steps of one head)
};

__device__ __forceinline__ void scan_load(RowScan& s, const TreeArgs& a, int base) {
  const int b = base + (threadIdx.x & 31);
  bool bad = false;
  s.base = base;
  s.len = s.n_new = s.steps = 0;
  if (b < a.c.ix.B) {
    s.len = clamp_count(a.c.ix.lens[b], a.c.ix.capacity, bad);
    s.n_new = a.counts != nullptr ? clamp_count(a.counts[b], a.T, bad) : a.T;
    s.steps = item_steps(s.len, s.n_new, a.k_new != nullptr);
  }
  if (bad) flag_index(a.c.status);
}

// Sum over all rows of f(steps of the row's items); `s` is left at the first window.
template <class F>
__device__ __forceinline__ int scan_sum(RowScan& s, const TreeArgs& a, F f) {
  if (s.base != 0) scan_load(s, a, 0);
  if (a.c.ix.B <= 32) return static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(f(s.steps))));
  int sum = f(s.steps);
  for (int base = 32; base < a.c.ix.B; base += 32) {
    RowScan w;
    scan_load(w, a, base);
    sum += f(w.steps);
  }
  return static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(sum)));
}

// Find the row that holds position `at` of a stream in which each of a row's
// items takes f(its steps) places: its index, the position of its first place,
// its lengths and its steps per head.
struct RowAt {
  int b, len, n_new, steps;
  int start;
};

template <class F>
__device__ __forceinline__ RowAt scan_find(RowScan& s, const TreeArgs& a, int at, F f) {
  const int lane = threadIdx.x & 31;
  if (s.base != 0) scan_load(s, a, 0);
  int before = 0;
  while (true) {
    const int places = f(s.steps) * a.c.ix.Hkv;
    int inc = places;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + inc > at);
    if (past != 0) {
      const int l = __ffs(past) - 1;
      RowAt r;
      r.b = s.base + l;
      r.len = __shfl_sync(0xffffffffu, s.len, l);
      r.n_new = __shfl_sync(0xffffffffu, s.n_new, l);
      r.steps = __shfl_sync(0xffffffffu, s.steps, l);
      r.start = before + __shfl_sync(0xffffffffu, inc - places, l);
      return r;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
    scan_load(s, a, s.base + 32);
  }
}

// The next row with steps after row `r.b` (one exists).
__device__ __forceinline__ void scan_next(RowScan& s, const TreeArgs& a, RowAt& r) {
  r.start += r.steps * a.c.ix.Hkv;
  int from = r.b + 1 - s.base;
  while (true) {
    const uint32_t later = from < 32 ? __ballot_sync(0xffffffffu, s.steps > 0) & (0xffffffffu << from) : 0u;
    if (later != 0) {
      const int l = __ffs(later) - 1;
      r.b = s.base + l;
      r.len = __shfl_sync(0xffffffffu, s.len, l);
      r.n_new = __shfl_sync(0xffffffffu, s.n_new, l);
      r.steps = __shfl_sync(0xffffffffu, s.steps, l);
      return;
    }
    scan_load(s, a, s.base + 32);
    from = 0;
  }
}

// A group's share of the work (cache_index.h).  Positions fit 32 bits: at most
// 65535 items of 8200 steps.
struct Walk {
  RowScan scan;
  RowAt row;             // the row of the next piece
  int total;             // steps of all items
  int at, end;           // more items than groups: what is left of the group's range
  int parts;             // few items: pieces of the group's item (0: more items than groups)
  int place;             // and which place of the row's items the group has
};

__device__ __forceinline__ int walk_cut(Walk& w, const TreeParams& p, int g) {
  const auto steps = [](int x) { return x; };
  if (g == 0) return 0;
  if (g == p.groups) return w.total;
  const int at = static_cast<int>(raw_cut(w.total, p.groups, g));
  const RowAt r = scan_find(w.scan, p.a, at, steps);
  const int i0 = r.start + (at - r.start) / r.steps * r.steps;
  return static_cast<int>(snapped(at, i0, i0 + r.steps));
}

__device__ __forceinline__ void walk_start(Walk& w, const TreeParams& p, int group) {
  const TreeArgs& a = p.a;
  const auto steps = [](int x) { return x; };
  scan_load(w.scan, a, 0);
  w.total = scan_sum(w.scan, a, steps) * a.c.ix.Hkv;
  const int items = scan_sum(w.scan, a, [](int x) { return x > 0 ? 1 : 0; }) * a.c.ix.Hkv;
  w.at = w.end = 0;
  w.parts = 0;
  if (w.total == 0) return;
  if (items <= p.groups) {
    // sum ceil(s / L) <= total / L + items bounds L from above
    int lo = (w.total + p.groups - 1) / p.groups, hi = item_steps(a.c.ix.capacity, a.T, a.k_new != nullptr);
    if (items < p.groups) hi = min(hi, (w.total + p.groups - items - 1) / (p.groups - items));
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (scan_sum(w.scan, a, [&](int x) { return static_cast<int>(static_cast<unsigned>(x + mid - 1) / static_cast<unsigned>(mid)); }) * a.c.ix.Hkv <= p.groups) hi = mid;
      else lo = mid + 1;
    }
    const auto pieces = [&](int x) { return static_cast<int>(static_cast<unsigned>(x + lo - 1) / static_cast<unsigned>(lo)); };
    if (group >= scan_sum(w.scan, a, pieces) * a.c.ix.Hkv) return;
    w.row = scan_find(w.scan, a, group, pieces);
    w.parts = pieces(w.row.steps);
    w.place = group - w.row.start;
    return;
  }
  w.at = walk_cut(w, p, group);
  w.end = walk_cut(w, p, group + 1);
  if (w.at < w.end) w.row = scan_find(w.scan, a, w.at, steps);
}

// The group's next piece; false at the end.
__device__ __forceinline__ bool walk_next(Walk& w, const TreeParams& p, int group, Piece& pc) {
  pc.slot = -1;
  if (w.parts > 0) {
    pc.hk = w.place / w.parts;
    const int k = w.place - pc.hk * w.parts;
    pc.j0 = even_cut(w.row.steps, k, w.parts);
    pc.n = even_cut(w.row.steps, k + 1, w.parts) - pc.j0;
    if (w.parts > 1) {
      pc.slot = group;
      pc.pieces = w.parts;
      pc.slot0 = pc.counter = group - k;
      pc.slot1 = pc.slot0 + 1;
      pc.slot_step = 1;
    }
    w.parts = 0;
  } else {
    if (w.at >= w.end) return false;
    if (w.at >= w.row.start + w.row.steps * p.a.c.ix.Hkv) scan_next(w.scan, p.a, w.row);
    const int in_row = w.at - w.row.start;
    pc.hk = in_row / w.row.steps;
    pc.j0 = in_row - pc.hk * w.row.steps;
    pc.n = min(w.row.steps - pc.j0, w.end - w.at);
    if (pc.n < w.row.steps) {
      const int i0 = w.at - pc.j0;
      const InnerCuts c = inner_cuts(w.total, p.groups, i0, i0 + w.row.steps);
      pc.pieces = c.count + 1;
      pc.slot0 = slot_from_begin(c.first);
      pc.slot1 = slot_from_cut(c.first);
      pc.slot_step = slot_from_cut(1);
      pc.counter = c.first;
      pc.slot = pc.j0 == 0 ? pc.slot0 : slot_from_cut(group);
    }
    w.at += pc.n;
  }
  pc.b = w.row.b;
  pc.len = w.row.len;
  pc.n_new = w.row.n_new;
  return true;
}

// ln of a row's sum l 2^m: -inf without a visible key, NaN where a score was NaN
// or +inf (l is NaN then; it adds to the slots' totals, and must not look like an
// empty row).
__device__ __forceinline__ float row_lse(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * LN2; }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 32 scores of one row: softcap (to base 2), mask.
template <bool SOFTCAP>
__device__ __forceinline__ void chunk_scores(float (&x)[32], bool partial, uint32_t keep, float cap_in, float cap_out) {
  if constexpr (SOFTCAP) {
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = cap_out * tanh_ex2(x[e] * cap_in);
  }
  if (partial) {
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = ((keep >> e) & 1u) ? x[e] : -INFINITY;
  }
}

__device__ __forceinline__ float chunk_max(const float (&x)[32], float mx) {
  float m0 = max3(x[0], x[1], x[2]), m1 = max3(x[3], x[4], x[5]);
  float m2 = max3(x[6], x[7], x[8]), m3 = max3(x[9], x[10], x[11]);
#pragma unroll
  for (int e = 12; e < 28; e += 8) {
    m0 = max3(m0, x[e], x[e + 1]);
    m1 = max3(m1, x[e + 2], x[e + 3]);
    m2 = max3(m2, x[e + 4], x[e + 5]);
    m3 = max3(m3, x[e + 6], x[e + 7]);
  }
  m0 = max3(m0, x[28], x[29]);
  m1 = max3(m1, x[30], x[31]);
  return max3(mx, max3(m0, m1, m2), m3);
}

// 2^(x - m) of 32 keys as bf16 pairs into 16 columns; adds to the fp32 sums.
template <bool SOFTCAP>
__device__ __forceinline__ void chunk_probs(const float (&x)[32], float sl2, float m_use, uint32_t p_addr, float2 (&acc)[2]) {
  const float2 neg_m = make_float2(-m_use, -m_use), sl2x2 = make_float2(sl2, sl2);
  uint32_t pk[16];
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float2 xs = make_float2(x[e], x[e + 1]);
    const float2 arg = SOFTCAP ? __fadd2_rn(xs, neg_m) : __ffma2_rn(xs, sl2x2, neg_m);
    const float2 pr = make_float2(ex2_approx(arg.x), ex2_approx(arg.y));
    acc[(e >> 1) & 1] = __fadd2_rn(acc[(e >> 1) & 1], pr);
    pk[e >> 1] = pack_bf16x2(pr.x, pr.y);
  }
  tmem_st16(p_addr, pk);
}

__device__ __forceinline__ uint32_t word_of(const uint4& k, int c) { return c == 0 ? k.x : (c == 1 ? k.y : (c == 2 ? k.z : k.w)); }

__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }
__device__ __forceinline__ uint4 first_bits(int n) {
  return make_uint4(low_bits(n), low_bits(n - 32), low_bits(n - 64), low_bits(n - 96));
}

// The keys x0 .. x0 + 127 of the new tokens that node t sees: itself and its
// ancestors.  A parent outside [-1, t) ends the walk.
__device__ __forceinline__ uint4 ancestor_bits(const TreeArgs& a, int b, int t, int x0) {
  if (a.parents == nullptr) return first_bits(t - x0 + 1);
  const int32_t* par = a.parents + static_cast<long long>(b) * a.T;
  uint4 w = make_uint4(0u, 0u, 0u, 0u);
  bool bad = false;
  for (int x = t; x >= x0;) {  // (ancestors only get smaller)
    const int i = x - x0;
    const uint32_t bit = 1u << (i & 31);
    if (i < 32) w.x |= bit;
    if (i >= 32 && i < 64) w.y |= bit;
    if (i >= 64 && i < 96) w.z |= bit;
    if (i >= 96 && i < 128) w.w |= bit;
    int up = __ldg(par + x);
    if (up >= x || up < -1) {
      bad = true;
      up = -1;
    }
    x = up;
  }
  if (bad) flag_index(a.c.status);
  return w;
}

// Copy one of a piece's tensors (K or V) into its ring, step by step.
template <int D, int STAGES>
__device__ __forceinline__ bool produce(const TreeParams& p, const Piece& pc, const CUtensorMap* pool, const CUtensorMap* fresh,
                                        uint32_t ring, uint64_t* full, uint64_t* empty, RingPos<STAGES>& pos,
                                        uint32_t& copies, const WaitCtl& wc) {
  const TreeArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const int ps = a.c.ix.page_size, box_rows = ps < TILE ? ps : TILE, box_lg = 7 - p.page_lg;
  const int n_prefix = (pc.len + TILE - 1) / TILE, pages = (pc.len + ps - 1) / ps;
  // page-table entries: two windows of 32, one entry to a lane, looked at when used
  const long long row0 = static_cast<long long>(pc.b) * a.c.ix.max_pages;
  auto entry = [&](int w) {
    const int i = w * 32 + lane;
    return i < pages ? (a.c.ix.table != nullptr ? __ldg(a.c.ix.table + row0 + i) : static_cast<int>(row0 + i)) : 0;
  };
  auto first_page = [&](int step) {
    return p.page_steps <= 1 ? step << p.page_lg : static_cast<int>(__umulhi(step, p.page_magic));
  };
  int window = first_page(pc.j0) >> 5;
  int tab0 = entry(window), tab1 = entry(window + 1);
#pragma unroll 1
  for (int step = pc.j0; step < pc.j0 + pc.n; ++step) {
    const int first = first_page(step);
    if ((first >> 5) != window) {
      ++window;
      tab0 = tab1;
      tab1 = entry(window + 1);
    }
    const uint32_t bar = smem_u32(full + pos.slot), dst = ring + pos.slot * TreeCfg<D>::kTileBytes;
    if (!tree_wait(smem_u32(empty + pos.slot), pos.phase ^ 1, wc)) return false;
    if (step < n_prefix) {
      // only the pages that hold filled slots
      const int boxes = min(TILE, pc.len - step * TILE + box_rows - 1) >> box_lg;
      const int y = p.page_steps > 1 ? (step - first * p.page_steps) * TILE : 0;
      // the step's pages (at most 8, within one window: their number divides 32), one to a lane
      int page = __shfl_sync(0xffffffffu, tab0, (first + lane) & 31);
      const bool outside = lane < boxes && (page < 0 || page >= a.c.ix.num_pages);
      if (outside) {
        flag_index(a.c.status);
        page = a.c.ix.num_pages;  // past the pool: the copy fills in zeros
      }
      int pg[TILE / 16];
#pragma unroll
      for (int i = 0; i < TILE / 16; ++i) pg[i] = __shfl_sync(0xffffffffu, page, i);
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, boxes * box_rows * D * 2);
#pragma unroll
        for (int i = 0; i < TILE / 16; ++i)
          if (i < boxes)
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tma_load_4d(dst + c * (TILE * 128) + i * box_rows * 128, pool, bar, c * 64, y, pc.hk, pg[i]);
      }
    } else if (lane == 0) {
      if (a.k_new != nullptr) {
        mbar_arrive_expect_tx(bar, TreeCfg<D>::kTileBytes);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_load_4d(dst + c * (TILE * 128), fresh, bar, c * 64, (step - n_prefix) * TILE, pc.hk, pc.b);
      } else {  // the empty step of a row without keys
        mbar_arrive(bar);
      }
    }
    __syncwarp();
    pos.next();
    ++copies;
  }
  return true;
}

// Let the last copy of each slot land before the CTA exits.
template <int STAGES>
__device__ __forceinline__ void drain_ring(uint64_t* full, uint32_t copies, const WaitCtl& wc) {
  for (uint32_t s = 0; s < STAGES; ++s) {
    const uint32_t uses = (copies + STAGES - 1 - s) / STAGES;
    if (uses > 0) mbar_wait_thread(smem_u32(full + s), (uses - 1) & 1, wc);
  }
}

// Keys of a step that exist (an empty row's step: none).
__device__ __forceinline__ int step_keys(const TreeArgs& a, const Piece& pc, int step) {
  const int n_prefix = (pc.len + TILE - 1) / TILE;
  if (step < n_prefix) return min(TILE, pc.len - step * TILE);
  return a.k_new != nullptr ? min(TILE, pc.n_new - (step - n_prefix) * TILE) : 0;
}

__device__ __forceinline__ int row_token(const TreeParams& p, int r) { return static_cast<int>(r * p.head_magic >> 16); }

// Quad (four columns) q of lane `lane` in a 128 x 16 staging buffer: the quads
// of a lane are rotated so that eight lanes' 16-byte accesses, whether one quad
// of eight lanes or all quads of two, fall into 32 banks.
__device__ __forceinline__ int stage_quad(int lane, int q) { return lane * 4 + ((q + (lane >> 1)) & 3); }

// Join the pieces of an item, by the CTA that wrote the last of them: a warp
// takes NR rows at a time, its lanes their columns, and reads NP pieces ahead
// (what it costs is the latency of the partials in L2).  The order is that of
// the pieces whichever of them came last, so the result does not depend on it.
template <int D, int NR, int NP>
__device__ __forceinline__ void join_rows(const TreeParams& p, const Piece& pc, int tile, int t0, int h0) {
  constexpr int kCols = D / 32;  // of a lane
  const TreeArgs& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = pc.pieces;
#pragma unroll 1
  for (int r0 = warp; r0 < p.rt.rows; r0 += 8 * NR) {
    float m[NR], l[NR], o[NR][kCols];
    int row[NR];
#pragma unroll
    for (int y = 0; y < NR; ++y) {
      row[y] = min(r0 + 8 * y, p.rt.rows - 1);  // (rows behind the tile's read its last row)
      m[y] = -INFINITY;
      l[y] = 0.f;
#pragma unroll
      for (int d = 0; d < kCols; ++d) o[y][d] = 0.f;
    }
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += NP) {
      float2 ml[NP][NR];
      float v[NP][NR][kCols];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int x = min(i0 + i, n - 1), slot = x == 0 ? pc.slot0 : pc.slot1 + (x - 1) * pc.slot_step;
        const int base = (slot * p.rt.tiles + tile) * p.rt.rows;
#pragma unroll
        for (int y = 0; y < NR; ++y) {
          const int part = base + row[y];  // below 2 x 148 x 128
          ml[i][y] = __ldcg(p.part_ml + part);
          if constexpr (kCols == 4) {
            const float4 u = __ldcg(reinterpret_cast<const float4*>(p.part_o + part * D) + lane);
            v[i][y][0] = u.x, v[i][y][1] = u.y, v[i][y][2] = u.z, v[i][y][3] = u.w;
          } else {
            const float2 u = __ldcg(reinterpret_cast<const float2*>(p.part_o + part * D) + lane);
            v[i][y][0] = u.x, v[i][y][1] = u.y;
          }
        }
      }
#pragma unroll
      for (int y = 0; y < NR; ++y) {
        float top = m[y];
#pragma unroll
        for (int i = 0; i < NP; ++i) top = fmaxf(top, ml[i][y].x);  // (the last piece may be read twice)
        const float f = m[y] == -INFINITY ? 0.f : ex2_approx(m[y] - top);
        m[y] = top;
        l[y] *= f;
#pragma unroll
        for (int d = 0; d < kCols; ++d) o[y][d] *= f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const float w = i0 + i < n && ml[i][y].x != -INFINITY ? ex2_approx(ml[i][y].x - top) : 0.f;
          l[y] = fmaf(w, ml[i][y].y, l[y]);
#pragma unroll
          for (int d = 0; d < kCols; ++d) o[y][d] = fmaf(w, v[i][y][d], o[y][d]);
        }
      }
    }
#pragma unroll
    for (int y = 0; y < NR; ++y) {
      const int r = r0 + 8 * y, r_tok = row_token(p, r), tok = t0 + r_tok, head = h0 + r - r_tok * p.rt.head_tile;
      if (r >= p.rt.rows || head >= a.G || tok >= pc.n_new) continue;
      const float inv = l[y] > 0.f ? 1.f / l[y] : 0.f;
      uint32_t* orow = reinterpret_cast<uint32_t*>(a.out + pc.b * a.o_st.b + (pc.hk * a.G + head) * a.o_st.h + tok * a.o_st.s);
#pragma unroll
      for (int d = 0; d < kCols; d += 2) orow[lane * (kCols / 2) + d / 2] = pack_bf16x2(o[y][d] * inv, o[y][d + 1] * inv);
      if (lane == 0 && a.lse != nullptr)
        a.lse[(static_cast<long long>(pc.b) * a.Hq + pc.hk * a.G + head) * a.T + tok] = row_lse(m[y], l[y]);
    }
  }
}

template <int D>
__device__ __noinline__ void join_pieces(const TreeParams& p, const Piece& pc, int tile, int t0, int h0) {
  if (p.rt.rows <= 8) join_rows<D, 1, 8>(p, pc, tile, t0, h0);
  else join_rows<D, 2, 4>(p, pc, tile, t0, h0);
}

template <int D, int R, bool SOFTCAP>
__global__ void __launch_bounds__(kTreeThreads, 1)
    attn_tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kn,
                     const __grid_constant__ CUtensorMap tm_vn, const __grid_constant__ TreeParams p) {
  using Cfg = TreeCfg<D>;
  const TreeArgs& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  TreeBarriers* bars = reinterpret_cast<TreeBarriers*>(smem + Cfg::kBarOff);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t q_smem = sbase, k_ring = sbase + Cfg::kKOff, v_ring = sbase + Cfg::kVOff;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.x % p.rt.tiles, group = blockIdx.x / p.rt.tiles;
  const int t0 = tile / p.rt.head_chunks * p.rt.tok_tile;   // first token of the tile
  const int h0 = tile % p.rt.head_chunks * p.rt.head_tile;  // first head of the tile, within the KV head

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->list_full[i]), 1);
      mbar_init(smem_u32(&bars->list_empty[i]), kListReaders);
      mbar_init(smem_u32(&bars->staged[i]), 4);
      mbar_init(smem_u32(&bars->s_full[i]), 1);
      mbar_init(smem_u32(&bars->p_full[i]), 128);
      mbar_init(smem_u32(&bars->o_full[i]), 1);
    }
    mbar_init(smem_u32(&bars->q_full), 1);
    mbar_init(smem_u32(&bars->q_empty), 1);
    mbar_init(smem_u32(&bars->o_final), 1);
    mbar_init(smem_u32(&bars->ml_ready), 8);
    mbar_init(smem_u32(&bars->written), 8);
    mbar_init(smem_u32(&bars->counted), 1);
    mbar_init(smem_u32(&bars->epi_done), 8);
    mbar_init(smem_u32(&bars->drain), 1);
    for (int s = 0; s < Cfg::kKStages; ++s) {
      mbar_init(smem_u32(&bars->k_full[s]), 1);
      mbar_init(smem_u32(&bars->k_empty[s]), 1);
    }
    for (int s = 0; s < Cfg::kVStages; ++s) {
      mbar_init(smem_u32(&bars->v_full[s]), 1);
      mbar_init(smem_u32(&bars->v_empty[s]), 1);
    }
    bars->abort_flag = 0;
    bars->never_set = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  if (warp == 9 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // the walk's lookups run under the set-up of the other warps
  Walk walk{};
  if (warp == 9) walk_start(walk, p, group);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const WaitCtl wc{p.wait_ns, smem_u32(&bars->abort_flag), a.c.status};

  if (warp >= 8) {
    if (warp == 9) {
      // ---------------------------------------------------------- walk and K
      RingPos<Cfg::kKStages> pos;
      uint32_t copies = 0;
      int n_pieces = 0;
      bool ok = true;
      while (ok) {
        Piece pc{};
        if (!walk_next(walk, p, group, pc)) pc.b = -1;
        else if (t0 >= pc.n_new) continue;  // none of the tile's tokens exist in this row
        const int buf = n_pieces & 1;
        if (!tree_wait(smem_u32(&bars->list_empty[buf]), ((n_pieces >> 1) & 1) ^ 1, wc)) { ok = false; break; }
        if (lane == 0) {
          bars->piece[buf] = pc;
          mbar_arrive(smem_u32(&bars->list_full[buf]));
        }
        __syncwarp();
        if (pc.b < 0) break;
        ++n_pieces;
        ok = produce<D>(p, pc, &tm_k, &tm_kn, k_ring, bars->k_full, bars->k_empty, pos, copies, wc);
      }
      if (lane == 0)  // let the copies in flight land before the CTA exits
        drain_ring<Cfg::kKStages>(bars->k_full, copies,
                                  WaitCtl{drain_limit(p.wait_ns), smem_u32(&bars->never_set), a.c.status});
    } else if (warp >= 10) {
      // ---------------------------------------------------------- V (warp 10), Q (warp 11)
      RingPos<Cfg::kVStages> pos;
      uint32_t copies = 0, q_loads = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const int buf = it & 1;
        if (!tree_wait(smem_u32(&bars->list_full[buf]), (it >> 1) & 1, wc)) break;
        const Piece pc = bars->piece[buf];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->list_empty[buf]));
        if (pc.b < 0) break;
        if (warp == 10) {
          ok = produce<D>(p, pc, &tm_v, &tm_vn, v_ring, bars->v_full, bars->v_empty, pos, copies, wc);
        } else {
          // free once the last piece's scores are formed; R copies
          if (!tree_wait(smem_u32(&bars->q_empty), (it & 1) ^ 1, wc)) break;
          if (lane == 0) {
            const uint32_t bar = smem_u32(&bars->q_full);
            mbar_arrive_expect_tx(bar, R * p.rt.rows * D * 2);
            for (int x = 0; x < R; ++x)
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_4d(q_smem + c * (TILE * 128) + x * (TILE / R * 128), &tm_q, bar, c * 64, pc.hk * a.G + h0, t0, pc.b);
          }
          __syncwarp();
          ++q_loads;
        }
      }
      if (lane == 0) {
        const WaitCtl drain_wc{drain_limit(p.wait_ns), smem_u32(&bars->never_set), a.c.status};
        drain_ring<Cfg::kVStages>(bars->v_full, copies, drain_wc);
        if (q_loads > 0) mbar_wait_thread(smem_u32(&bars->q_full), (q_loads - 1) & 1, drain_wc);
      }
    } else if (warp == 8) {
      // ---------------------------------------------------------- MMA issuer
      RingPos<Cfg::kKStages> kp;
      RingPos<Cfg::kVStages> vp;
      uint32_t p_cnt[2] = {0, 0};
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const int buf = it & 1;
        if (!tree_wait(smem_u32(&bars->list_full[buf]), (it >> 1) & 1, wc)) break;
        const Piece pc = bars->piece[buf];
        if (pc.b < 0) break;
        if (!tree_wait(smem_u32(&bars->q_full), it & 1, wc)) break;
        tc_fence_after();
        // S(0) S(1) | O(0) S(2) | O(1) S(3) | ... | O(n-1).  A step's products take
        // only as many of its keys (S columns, rows of V) as exist, in 16s.
#pragma unroll 1
        for (int i = 0; i < pc.n + 2; ++i) {
          const int t = i & 1;
          if (i >= 2) {
            // O of the last piece has been read before the first product overwrites it
            if ((i == 2 && !tree_wait(smem_u32(&bars->epi_done), (it & 1) ^ 1, wc)) ||
                !tree_wait(smem_u32(&bars->v_full[vp.slot]), vp.phase, wc) ||
                !tree_wait(smem_u32(&bars->p_full[t]), p_cnt[t] & 1, wc)) {
              ok = false;
              break;
            }
            ++p_cnt[t];
            tc_fence_after();
            const uint32_t v_lo = smem_desc_lo(v_ring + vp.slot * Cfg::kTileBytes, TILE * 128);
            const int kks = (max(step_keys(a, pc, pc.j0 + i - 2), 1) + 15) / 16;
            const uint32_t o_tm = tmem + 256 + t * D, p_tm = tmem + t * 128, first = i > 3 ? 1u : 0u;
            // (a full step's 8 products without a branch before each: 480 clocks to issue, not 850)
            if (kks == TILE / 16) {
#pragma unroll
              for (int kk = 0; kk < TILE / 16; ++kk)
                mma_ts_lo_w<smem_desc_hi_sw128(1024)>(o_tm, p_tm + kk * 8, v_lo + kk * (2048 >> 4), Cfg::kIdescPV,
                                                      kk > 0 ? 1u : first);
            } else {
#pragma unroll 1
              for (int kk = 0; kk < kks; ++kk)
                mma_ts_lo_w<smem_desc_hi_sw128(1024)>(o_tm, p_tm + kk * 8, v_lo + kk * (2048 >> 4), Cfg::kIdescPV,
                                                      kk > 0 ? 1u : first);
            }
            mma_commit_w(smem_u32(&bars->o_full[t]));
            mma_commit_w(smem_u32(&bars->v_empty[vp.slot]));
            vp.next();
          }
          if (i < pc.n) {
            const uint32_t k_lo = smem_desc_lo(k_ring + kp.slot * Cfg::kTileBytes, 16), q_lo = smem_desc_lo(q_smem, 16);
            if (!tree_wait(smem_u32(&bars->k_full[kp.slot]), kp.phase, wc)) { ok = false; break; }
            tc_fence_after();
            const uint32_t idesc = idesc_bf16_f32(128, (max(step_keys(a, pc, pc.j0 + i), 1) + 15) / 16 * 16, false, false);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * (TILE * 128) + (kk & 3) * 32) >> 4;
              mma_ss_lo_w<smem_desc_hi_sw128(1024)>(tmem + t * 128, q_lo + off, k_lo + off, idesc, kk > 0 ? 1u : 0u);
            }
            mma_commit_w(smem_u32(&bars->s_full[t]));
            mma_commit_w(smem_u32(&bars->k_empty[kp.slot]));
            if (i == pc.n - 1) mma_commit_w(smem_u32(&bars->q_empty));
            kp.next();
          }
        }
        if (!ok) break;
        mma_commit_w(smem_u32(&bars->o_final));
        if (lane == 0) mbar_arrive(smem_u32(&bars->list_empty[buf]));
        __syncwarp();
      }
      mma_commit_w(smem_u32(&bars->drain));
      tree_wait(smem_u32(&bars->drain), 0, WaitCtl{drain_limit(p.wait_ns), smem_u32(&bars->never_set), a.c.status});
    }
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    const int t = warp >> 2, tid = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + t * 128 + lane_off, o_addr = tmem + 256 + t * D + lane_off;
    // this lane's query row, and the 32-key chunks [c0, c0 + kChunks) of a step that its copy takes
    constexpr int kChunks = 4 / R;
    const int r = tid & (TILE / R - 1), copy = tid / (TILE / R), c0 = copy * kChunks;
    const int r_tok = row_token(p, r), tok = t0 + r_tok, head = h0 + r - r_tok * p.rt.head_tile;
    const bool in_tile = r < p.rt.rows && head < a.G;
    float4* stage = reinterpret_cast<float4*>(smem + Cfg::kStageOff) + t * 2 * TILE * 4;  // two buffers
    const float sl2 = a.scale * LOG2E;
    const float cap_in = SOFTCAP ? a.scale / a.softcap : 0.f, cap_out = SOFTCAP ? a.softcap * LOG2E : 0.f;
    uint32_t s_cnt = 0, p_cnt = 0, v_base = 0, rounds = 0, cuts = 0;  // v_base: V copies before the piece
    for (int it = 0;; ++it) {
      const int buf = it & 1;
      if (!tree_wait(smem_u32(&bars->list_full[buf]), (it >> 1) & 1, wc)) break;
      const Piece pc = bars->piece[buf];
      if (pc.b < 0) break;
      const bool valid = in_tile && tok < pc.n_new;
      const bool busy = __any_sync(0xffffffffu, valid);  // warps without a row only keep step
      const int n_prefix = (pc.len + TILE - 1) / TILE;
      float m_run = -INFINITY, l_run = 0.f;
      bool ok = true;
#pragma unroll 1
      for (int j = t; j < pc.n; j += 2) {
        const int step = pc.j0 + j;
        const int x0 = (step - n_prefix) * TILE;  // new tokens: first of the step
        // keys of the step that exist, and those this row sees
        const int n_keys = step_keys(a, pc, step), chunks = (max(n_keys, 1) + 31) / 32;  // chunks the product takes
        const bool partial = n_keys < TILE || step >= n_prefix;
        uint4 keep = first_bits(n_keys);
        if (step >= n_prefix) keep = valid && n_keys > 0 ? ancestor_bits(a, pc.b, tok, x0) : make_uint4(0u, 0u, 0u, 0u);
        if (!tree_wait(smem_u32(&bars->s_full[t]), s_cnt & 1, wc)) { ok = false; break; }
        ++s_cnt;
        tc_fence_after();
        if (busy) {
          // at most 64 scores in registers: with all 128 of R = 1 the kernel spills, and
          // local memory is slow beside 227 KB of shared memory
          constexpr int kHold = kChunks < 2 ? kChunks : 2;
          float x[kHold][32], mx = -INFINITY;
          const int mine = min(kChunks, chunks - c0);  // chunks of this copy that hold keys
          auto load = [&](int from) {
#pragma unroll
            for (int c = 0; c < kHold; ++c)
              if (from + c < mine) tmem_ld32(s_addr + (c0 + from + c) * 32, reinterpret_cast<uint32_t(&)[32]>(x[c]));
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < kHold; ++c)
              if (from + c < mine) chunk_scores<SOFTCAP>(x[c], partial, word_of(keep, c0 + from + c), cap_in, cap_out);
          };
#pragma unroll 1
          for (int from = kChunks - kHold; from >= 0; from -= kHold) {  // the first chunks last: they stay
            load(from);
#pragma unroll
            for (int c = 0; c < kHold; ++c)
              if (from + c < mine) mx = chunk_max(x[c], mx);
          }
          if (!SOFTCAP) mx *= sl2;  // -inf stays -inf (sl2 > 0)
          const float m_new = fmaxf(m_run, mx);
          const bool need = valid && m_new > m_run + kTreeRescale;  // (the other rows are not looked at: they hold anything)
          if (__any_sync(0xffffffffu, need)) {
            const float alpha = m_run == -INFINITY ? 0.f : ex2_approx(m_run - m_new);
            if (j > 1) {  // O must be complete before it is rescaled
              if (!tree_wait(smem_u32(&bars->o_full[t]), (p_cnt - 1) & 1, wc)) { ok = false; break; }
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(o_addr + c * 16, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st16(o_addr + c * 16, o);
              }
            }
            l_run *= alpha;
            m_run = m_new;
          }
          const float m_use = m_run == -INFINITY ? 0.f : m_run;
          float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          // P of chunk c lands in columns 16 c .. 16 c + 15, whose scores are read by
          // then; the other copies' keys are zero in these lanes
#pragma unroll 1
          for (int from = 0; from < kChunks; from += kHold) {
            if (from > 0) load(from);
#pragma unroll
            for (int c = 0; c < kHold; ++c)
              if (from + c < mine) chunk_probs<SOFTCAP>(x[c], sl2, m_use, s_addr + (c0 + from + c) * 16, acc);
          }
          if constexpr (R > 1) {
            const uint32_t zero[16] = {};
            for (int c = 0; c < chunks; ++c)
              if (c < c0 || c >= c0 + kChunks) tmem_st16(s_addr + c * 16, zero);
          }
          l_run += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
          tmem_wait_st();
        }
        if (n_keys < TILE) {
          // V rows of no key, up to the last the product takes: zeros, whatever lies there
          const uint32_t pos = v_base + j, slot = pos % Cfg::kVStages;
          if (!tree_wait(smem_u32(&bars->v_full[slot]), (pos / Cfg::kVStages) & 1, wc)) { ok = false; break; }
          uint8_t* v = smem + Cfg::kVOff + slot * Cfg::kTileBytes;
          const int rows = (max(n_keys, 1) + 15) / 16 * 16 - n_keys;
          for (int i = tid; i < rows * (D / 8); i += 128) {  // 16-byte chunks; whole rows, so the swizzle does not matter
            const int row = n_keys + i / (D / 8), ch = i % (D / 8);
            *reinterpret_cast<uint4*>(v + (ch >> 3) * (TILE * 128) + row * 128 + (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(smem_u32(&bars->p_full[t]));
        ++p_cnt;
      }
      if (!ok) break;
      v_base += pc.n;
      // ---- end of the piece: join the states of each row, 2 warpgroups x R copies.
      // Both warpgroups' (m, l) go into both warpgroups' first buffer, so that each
      // reads its own only.
      if (!tree_wait(smem_u32(&bars->o_final), it & 1, wc)) break;
      tc_fence_after();
      float2* ml = reinterpret_cast<float2*>(smem + Cfg::kStageOff);
      constexpr int kRegion = 2 * TILE * kStageCols / 2;  // a warpgroup's two buffers, in float2
      ml[t * TILE + tid] = make_float2(m_run, l_run);
      ml[kRegion + t * TILE + tid] = make_float2(m_run, l_run);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->ml_ready));
      if (!tree_wait(smem_u32(&bars->ml_ready), it & 1, wc)) break;
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int x = 0; x < 2 * R; ++x) m = fmaxf(m, ml[t * kRegion + (x & 1) * TILE + r + (x >> 1) * (TILE / R)].x);
      float g[2];
#pragma unroll
      for (int x = 0; x < 2 * R; ++x) {
        const float2 v = ml[t * kRegion + (x & 1) * TILE + r + (x >> 1) * (TILE / R)];
        const float f = v.x == -INFINITY ? 0.f : ex2_approx(v.x - m);
        l = fmaf(f, v.y, l);
        if ((x >> 1) == copy) g[x & 1] = f;
      }
      if (pc.slot < 0) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        g[0] *= inv;
        g[1] *= inv;
      }
      const long long part = (static_cast<long long>(pc.slot) * p.rt.tiles + tile) * p.rt.rows;
      if (valid && t == 0 && copy == 0) {
        if (pc.slot >= 0) p.part_ml[part + r] = make_float2(m, l);
        else if (a.lse != nullptr)
          a.lse[(static_cast<long long>(pc.b) * a.Hq + pc.hk * a.G + head) * a.T + tok] = row_lse(m, l);
      }
      // where this thread writes: rows w_row + 32 x, four columns
      const int w_row = (warp & 3) * 8 + (lane >> 2), quad = lane & 3;
      constexpr int kRows = 4 / R;
      long long to[kRows];  // elements; -1: no such row
#pragma unroll
      for (int x = 0; x < kRows; ++x) {
        const int row = w_row + 32 * x, rt = row_token(p, row), w_head = h0 + row - rt * p.rt.head_tile;
        to[x] = -1;
        if (row < p.rt.rows && w_head < a.G && t0 + rt < pc.n_new)
          to[x] = pc.slot >= 0 ? (part + row) * D
                               : pc.b * a.o_st.b + (pc.hk * a.G + w_head) * a.o_st.h + (t0 + rt) * a.o_st.s;
      }
      // O, 16 columns at a time (even rounds in the second buffer): scaled into the
      // buffer, then summed over the copies and written, coalesced, by the warpgroup
#pragma unroll 1
      for (int k = 0; k < D / 2 / kStageCols; ++k) {
        float4* sb = stage + ((k & 1) ^ 1) * TILE * 4;
        if (busy) {
          uint32_t o0[16], o1[16];
          tmem_ld16(tmem + 256 + lane_off + t * (D / 2) + k * kStageCols, o0);
          tmem_ld16(tmem + 256 + D + lane_off + t * (D / 2) + k * kStageCols, o1);
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[e] = __uint_as_float(o0[4 * q + e]) * g[0];
              if (pc.n > 1) o[e] = fmaf(__uint_as_float(o1[4 * q + e]), g[1], o[e]);  // (one step: the odd O is stale)
            }
            sb[stage_quad(tid, q)] = make_float4(o[0], o[1], o[2], o[3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->staged[t]));
        if (!tree_wait(smem_u32(&bars->staged[t]), rounds & 1, wc)) { ok = false; break; }
        ++rounds;
        const int col = t * (D / 2) + k * kStageCols + quad * 4;
#pragma unroll
        for (int x = 0; x < kRows; ++x) {
          float4 v = sb[stage_quad(w_row + 32 * x, quad)];
#pragma unroll
          for (int y = 1; y < R; ++y) {
            const float4 u = sb[stage_quad(w_row + 32 * x + y * (TILE / R), quad)];
            v.x += u.x;
            v.y += u.y;
            v.z += u.z;
            v.w += u.w;
          }
          if (to[x] >= 0) {
            if (pc.slot >= 0) *reinterpret_cast<float4*>(p.part_o + to[x] + col) = v;
            else *reinterpret_cast<uint2*>(a.out + to[x] + col) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
          }
        }
      }
      if (!ok) break;
      if (pc.slot >= 0) {
        // count this piece in once all warps' parts of it are visible to the device;
        // whoever counts in last joins the item and leaves the counter at zero
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->written));
        if (!tree_wait(smem_u32(&bars->written), cuts & 1, wc)) break;
        if (threadIdx.x == 0) {
          int* counter = p.counters + pc.counter * p.rt.tiles + tile;
          const bool last = atomicAdd(counter, 1) == pc.pieces - 1;
          __threadfence();
          if (last) *counter = 0;
          bars->last = last ? 1 : 0;
          mbar_arrive(smem_u32(&bars->counted));
        }
        __syncwarp();
        if (!tree_wait(smem_u32(&bars->counted), cuts & 1, wc)) break;
        ++cuts;
        if (bars->last != 0) join_pieces<D>(p, bars->piece[buf], tile, t0, h0);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&bars->epi_done));
        mbar_arrive(smem_u32(&bars->list_empty[buf]));
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

template <int D, int R, bool SOFTCAP>
cudaError_t launch_tree_t(const TreeMaps& m, const TreeParams& p, cudaStream_t stream) {
  auto kernel = attn_tree_kernel<D, R, SOFTCAP>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = prepare_kernel(done, kernel, TreeCfg<D>::kAllocBytes, 0);
  if (e != cudaSuccess) return e;
  kernel<<<p.groups * p.rt.tiles, kTreeThreads, TreeCfg<D>::kAllocBytes, stream>>>(m.q, m.k, m.v, m.kn, m.vn, p);
  return cudaGetLastError();
}

// Copies of the query tile: as many as fit its 128 rows, up to 4.
template <int D, bool SOFTCAP>
cudaError_t launch_tree_r(const TreeMaps& m, const TreeParams& p, cudaStream_t stream) {
  if (p.rt.rows <= 32) return launch_tree_t<D, 4, SOFTCAP>(m, p, stream);
  if (p.rt.rows <= 64) return launch_tree_t<D, 2, SOFTCAP>(m, p, stream);
  return launch_tree_t<D, 1, SOFTCAP>(m, p, stream);
}

}  // namespace

static_assert(kTreeCtas * sizeof(int) <= kTreeCounterBytes, "counters");

size_t tree_workspace_bytes(int G, int T, int D) {
  const RowTiles rt = row_tiles(G, T);
  // groups * tiles <= 148 where there is more than one group
  const size_t rows = static_cast<size_t>(2) * kTreeCtas * rt.rows;
  return kTreeCounterBytes + (rows * D * 4 + 255) / 256 * 256 + (rows * 8 + 255) / 256 * 256;
}

cudaError_t launch_tree(const TreeMaps& m, const TreeArgs& a, void* workspace, uint64_t wait_ns, cudaStream_t stream) {
  TreeParams p{};
  p.a = a;
  p.rt = row_tiles(a.G, a.T);
  p.groups = tree_groups(p.rt.tiles);
  p.head_magic = 65535u / p.rt.head_tile + 1;
  const int ps = a.c.ix.page_size;
  while (ps << p.page_lg < TILE) ++p.page_lg;
  p.page_steps = ps / TILE;
  if (p.page_steps > 1) p.page_magic = static_cast<uint32_t>(((1ull << 32) + p.page_steps - 1) / p.page_steps);
  const size_t rows = static_cast<size_t>(2) * kTreeCtas * p.rt.rows;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.counters = reinterpret_cast<int*>(ws);
  p.part_o = reinterpret_cast<float*>(ws + kTreeCounterBytes);
  p.part_ml = reinterpret_cast<float2*>(ws + kTreeCounterBytes + (rows * a.c.D * 4 + 255) / 256 * 256);
  p.wait_ns = wait_ns;
  if (a.c.D == 128) return a.softcap > 0.f ? launch_tree_r<128, true>(m, p, stream) : launch_tree_r<128, false>(m, p, stream);
  return a.softcap > 0.f ? launch_tree_r<64, true>(m, p, stream) : launch_tree_r<64, false>(m, p, stream);
}

}  // namespace attn25
