// Attention of new tokens over a paged KV cache and over their own ancestors
// (attn_tree_fwd), for sm_100a.
//
// A KV head's query rows (G heads x T tokens) are the rows of an M = 128 tile;
// its keys come in steps of 128: pages of the cache, then the new tokens.
// With few rows a step's two products cost 512 tensor clocks against the
// ~2800 clocks in which HBM delivers its 64 KB of K and V to one SM (its 148th
// share), so the kernel is a stream of K and V: what counts is that every SM
// has an equal share of the bytes of all rows, whatever their lengths, and
// always enough copies in flight (192 KB of rings).
//
// Work: the steps of all (row, KV head) items form one stream that is cut into
// equal ranges (cache_index.h), one CTA per SM.  Items cut by a range boundary
// leave (m, l, O) partials in fp32, which tree_join_kernel joins; the others
// are written out directly.
//
// Warp roles (384 threads, as in the forward kernel):
//   warps 0-3  softmax of the even steps of a piece (thread = query row)
//   warps 4-7  softmax of the odd steps
//   warp  8    MMA issuer
//   warp  9    TMA producer of Q and K: walks the ranges, publishes the pieces
//   warp 10    TMA producer of V
// (One producer for both rings held the stream up: a 128-key copy from pages of
// 64 rows takes a warp ~1400 clocks of page lookups and issue, and HBM delivers
// one every 1400.)
// The two softmax warpgroups keep separate (m, l, O) of the same rows, so that
// one's softmax runs under the other's products; both are joined at the end of
// a piece.  Each running maximum moves only when exceeded by more than 2^8, as
// in the forward kernel.  P is rounded to bf16 for the PV product (half a step,
// 2^-8 relative, the forward kernel's choice: the product then runs at the full
// bf16 rate straight from tensor memory); sums, maxima and O stay in fp32.
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
// Where a tile has at most 64 rows, two Q tiles share one tile's room (rows 0
// and 64 of it), so that the next piece's Q need not wait for this piece's last
// product; that product's rows from 64 on then read whatever follows.
constexpr int kQBufBytes = 64 * 128;

template <int D>
struct TreeCfg {
  static constexpr int kTileBytes = TILE * D * 2;
  // a ring each for K and V: 96 + 96 KB
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kKOff = kTileBytes;  // after Q
  static constexpr int kVOff = kKOff + kStages * kTileBytes;
  static constexpr int kBarOff = kVOff + kStages * kTileBytes;
  static constexpr int kSmemBytes = kBarOff + 1024;
  static constexpr int kAllocBytes = kSmemBytes + 1024;  // + alignment slack
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, false, true);
};

// A piece: steps [j0, j0 + n) of item (b, hk).
struct Piece {
  int32_t b, hk, j0, n;     // b < 0: the end
  int32_t len, n_new;       // filled slots and new tokens of the row
  int32_t slot;             // partial-result slot, or -1: the whole item
};

struct TreeBarriers {
  uint64_t list_full[2], list_empty[2];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t o_final, s_free, epi_done;
  uint64_t ml_ready[4];  // the two warps of a lane quarter have exchanged (m, l)
  uint64_t drain;
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6];
  uint32_t tmem_base, abort_flag, never_set;
  Piece piece[2];
};
static_assert(sizeof(TreeBarriers) <= 1024, "barrier block");

constexpr int kListReaders = 10;  // the MMA warp, the V producer and the 8 softmax warps (lane 0 each)

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
  float* part_o;   // [slot][tile][rows][D]
  float2* part_ml; // [slot][tile][rows]
  uint64_t wait_ns;
  // pages and steps: pages of up to 128 rows, 1 << page_lg to a step; larger
  // ones hold page_steps > 1 steps: step / page_steps = umulhi(step, page_magic)
  // (exact: step and page_steps are at most 8192)
  int page_lg, page_steps;
  uint32_t page_magic;
  int q_bufs;  // 2 where two Q tiles fit one tile's room (up to 64 rows)
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

// Steps of the stream (all rows and heads).  `s` is left at the first window.
__device__ __forceinline__ long long scan_total(RowScan& s, const TreeArgs& a) {
  long long total = 0;
  scan_load(s, a, 0);
  total = s.steps;
  for (int base = 32; base < a.c.ix.B; base += 32) {
    RowScan w;
    scan_load(w, a, base);
    total += w.steps;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  return total * a.c.ix.Hkv;
}

// Find the row that holds stream position `at` (< total): its index, the
// position of its first step, its lengths and its steps per head.
struct RowAt {
  int b, len, n_new, steps;
  long long start;
};

__device__ __forceinline__ RowAt scan_find(RowScan& s, const TreeArgs& a, long long at) {
  const int lane = threadIdx.x & 31;
  if (s.base != 0) scan_load(s, a, 0);
  long long before = 0;
  while (true) {
    long long inc = static_cast<long long>(s.steps) * a.c.ix.Hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, inc, o);
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
      r.start = before + __shfl_sync(0xffffffffu, inc, l) - static_cast<long long>(r.steps) * a.c.ix.Hkv;
      return r;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
    scan_load(s, a, s.base + 32);
  }
}

// The next row with steps after row `r.b` (one exists).
__device__ __forceinline__ void scan_next(RowScan& s, const TreeArgs& a, RowAt& r) {
  r.start += static_cast<long long>(r.steps) * a.c.ix.Hkv;
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
  for (int x = t; x >= 0;) {
    const int i = x - x0;
    const uint32_t bit = 1u << (i & 31);
    if (i >= 0 && i < 32) w.x |= bit;
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

__device__ __forceinline__ void tmem_st2(uint32_t taddr, float x, float y) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};" ::"r"(taddr), "r"(__float_as_uint(x)),
               "r"(__float_as_uint(y))
               : "memory");
}
__device__ __forceinline__ float2 tmem_ld2(uint32_t taddr) {
  uint32_t x, y;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(x), "=r"(y) : "r"(taddr));
  tmem_wait_ld();
  return make_float2(__uint_as_float(x), __uint_as_float(y));
}

// Copy one of a piece's tensors (K or V) into its ring, step by step.
template <int D>
__device__ __forceinline__ bool produce(const TreeParams& p, const Piece& pc, const CUtensorMap* pool, const CUtensorMap* fresh,
                                        uint32_t ring, uint64_t* full, uint64_t* empty, RingPos<TreeCfg<D>::kStages>& pos,
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
      if (lane == 0) mbar_arrive_expect_tx(bar, boxes * box_rows * D * 2);
      const int y = p.page_steps > 1 ? (step - first * p.page_steps) * TILE : 0;
      for (int i = 0; i < boxes; ++i) {
        int page = __shfl_sync(0xffffffffu, tab0, (first + i) & 31);
        const bool outside = page < 0 || page >= a.c.ix.num_pages;
        if (outside) page = a.c.ix.num_pages;  // past the pool: the copy fills in zeros
        if (lane == 0) {
          if (outside) flag_index(a.c.status);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(dst + c * (TILE * 128) + i * box_rows * 128, pool, bar, c * 64, y, pc.hk, page);
        }
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

template <int D, bool SOFTCAP>
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
      mbar_init(smem_u32(&bars->q_full[i]), 1);
      mbar_init(smem_u32(&bars->q_empty[i]), 1);
      mbar_init(smem_u32(&bars->s_full[i]), 1);
      mbar_init(smem_u32(&bars->p_full[i]), 128);
      mbar_init(smem_u32(&bars->o_full[i]), 1);
    }
    mbar_init(smem_u32(&bars->o_final), 1);
    mbar_init(smem_u32(&bars->s_free), 8);
    mbar_init(smem_u32(&bars->epi_done), 8);
    mbar_init(smem_u32(&bars->drain), 1);
    for (int w = 0; w < 4; ++w) mbar_init(smem_u32(&bars->ml_ready[w]), 2);
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(smem_u32(&bars->k_full[s]), 1);
      mbar_init(smem_u32(&bars->k_empty[s]), 1);
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
  RowScan scan{};
  RowAt row{};
  long long total = 0, at = 0, end = 0;
  if (warp == 9) {
    total = scan_total(scan, a);
    at = range_start(total, p.groups, group);
    end = range_start(total, p.groups, group + 1);
    if (at < end) row = scan_find(scan, a, at);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join's blocks may start and wait
  const uint32_t tmem = bars->tmem_base;
  const WaitCtl wc{p.wait_ns, smem_u32(&bars->abort_flag), a.c.status};

  if (warp >= 8) {
    if (warp == 9) {
      // ---------------------------------------------------------- walk, Q and K
      RingPos<Cfg::kStages> pos;
      uint32_t copies = 0;
      int n_pieces = 0;
      bool ok = true;
      while (ok) {
        Piece pc{};
        pc.b = -1;
        if (at < end) {
          if (at >= row.start + static_cast<long long>(row.steps) * a.c.ix.Hkv) scan_next(scan, a, row);
          const long long in_row = at - row.start;
          pc.hk = static_cast<int>(in_row / row.steps);
          pc.j0 = static_cast<int>(in_row - static_cast<long long>(pc.hk) * row.steps);
          const long long left = end - at;
          pc.n = row.steps - pc.j0 < left ? row.steps - pc.j0 : static_cast<int>(left);
          pc.slot = pc.n == row.steps ? -1 : partial_slot(group, at == range_start(total, p.groups, group));
          at += pc.n;
          if (t0 >= row.n_new) continue;  // none of the tile's tokens exist in this row
          pc.b = row.b;
          pc.len = row.len;
          pc.n_new = row.n_new;
        }
        const int buf = n_pieces & 1;
        if (!tree_wait(smem_u32(&bars->list_empty[buf]), ((n_pieces >> 1) & 1) ^ 1, wc)) { ok = false; break; }
        if (lane == 0) {
          bars->piece[buf] = pc;
          mbar_arrive(smem_u32(&bars->list_full[buf]));
        }
        __syncwarp();
        if (pc.b < 0) break;
        // Q: free once the products of the last piece that used the buffer have read it
        const int qb = p.q_bufs == 2 ? n_pieces & 1 : 0, q_use = p.q_bufs == 2 ? n_pieces >> 1 : n_pieces;
        if (!tree_wait(smem_u32(&bars->q_empty[qb]), (q_use & 1) ^ 1, wc)) { ok = false; break; }
        if (lane == 0) {
          const uint32_t bar = smem_u32(&bars->q_full[qb]);
          mbar_arrive_expect_tx(bar, p.rt.rows * D * 2);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(q_smem + qb * kQBufBytes + c * (TILE * 128), &tm_q, bar, c * 64, pc.hk * a.G + h0, t0, pc.b);
        }
        __syncwarp();
        ++n_pieces;
        ok = produce<D>(p, pc, &tm_k, &tm_kn, k_ring, bars->k_full, bars->k_empty, pos, copies, wc);
      }
      if (lane == 0) {
        const WaitCtl drain_wc{drain_limit(p.wait_ns), smem_u32(&bars->never_set), a.c.status};
        drain_ring<Cfg::kStages>(bars->k_full, copies, drain_wc);
        for (int s = 0; s < p.q_bufs; ++s) {
          const int uses = p.q_bufs == 2 ? (n_pieces + 1 - s) / 2 : n_pieces;
          if (uses > 0) mbar_wait_thread(smem_u32(&bars->q_full[s]), (uses - 1) & 1, drain_wc);
        }
      }
    } else if (warp == 10) {
      // ---------------------------------------------------------- V
      RingPos<Cfg::kStages> pos;
      uint32_t copies = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const int buf = it & 1;
        if (!tree_wait(smem_u32(&bars->list_full[buf]), (it >> 1) & 1, wc)) break;
        const Piece pc = bars->piece[buf];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->list_empty[buf]));
        if (pc.b < 0) break;
        ok = produce<D>(p, pc, &tm_v, &tm_vn, v_ring, bars->v_full, bars->v_empty, pos, copies, wc);
      }
      if (lane == 0)
        drain_ring<Cfg::kStages>(bars->v_full, copies,
                                 WaitCtl{drain_limit(p.wait_ns), smem_u32(&bars->never_set), a.c.status});
    } else if (warp == 8) {
      // ---------------------------------------------------------- MMA issuer
      RingPos<Cfg::kStages> kp, vp;
      uint32_t p_cnt[2] = {0, 0};
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const int buf = it & 1;
        if (!tree_wait(smem_u32(&bars->list_full[buf]), (it >> 1) & 1, wc)) break;
        const Piece pc = bars->piece[buf];
        if (pc.b < 0) break;
        const int qb = p.q_bufs == 2 ? it & 1 : 0, q_use = p.q_bufs == 2 ? it >> 1 : it;
        const uint32_t q = q_smem + qb * kQBufBytes;
        // the columns of the scores, in which the last piece's (m, l) were exchanged, are free
        if (!tree_wait(smem_u32(&bars->s_free), (it & 1) ^ 1, wc)) break;
        if (!tree_wait(smem_u32(&bars->q_full[qb]), q_use & 1, wc)) break;
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
            const uint32_t v_smem = v_ring + vp.slot * Cfg::kTileBytes;
            const int kks = (max(step_keys(a, pc, pc.j0 + i - 2), 1) + 15) / 16;
#pragma unroll
            for (int kk = 0; kk < TILE / 16; ++kk)
              if (kk < kks)
                mma_ts_w(tmem + 256 + t * D, tmem + t * 128 + kk * 8, smem_desc_sw128(v_smem + kk * 2048, TILE * 128, 1024),
                         Cfg::kIdescPV, (i > 3 || kk > 0) ? 1u : 0u);
            mma_commit_w(smem_u32(&bars->o_full[t]));
            mma_commit_w(smem_u32(&bars->v_empty[vp.slot]));
            vp.next();
          }
          if (i < pc.n) {
            const uint32_t k_smem = k_ring + kp.slot * Cfg::kTileBytes;
            if (!tree_wait(smem_u32(&bars->k_full[kp.slot]), kp.phase, wc)) { ok = false; break; }
            tc_fence_after();
            const uint32_t idesc = idesc_bf16_f32(128, (max(step_keys(a, pc, pc.j0 + i), 1) + 15) / 16 * 16, false, false);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * (TILE * 128) + (kk & 3) * 32;
              mma_ss_w(tmem + t * 128, smem_desc_sw128(q + off, 16, 1024), smem_desc_sw128(k_smem + off, 16, 1024), idesc,
                       kk > 0 ? 1u : 0u);
            }
            mma_commit_w(smem_u32(&bars->s_full[t]));
            mma_commit_w(smem_u32(&bars->k_empty[kp.slot]));
            kp.next();
          }
        }
        if (!ok) break;
        mma_commit_w(smem_u32(&bars->q_empty[qb]));
        mma_commit_w(smem_u32(&bars->o_final));
        if (lane == 0) mbar_arrive(smem_u32(&bars->list_empty[buf]));
        __syncwarp();
      }
      mma_commit_w(smem_u32(&bars->drain));
      tree_wait(smem_u32(&bars->drain), 0, WaitCtl{drain_limit(p.wait_ns), smem_u32(&bars->never_set), a.c.status});
    }
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    const int t = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + t * 128 + lane_off, o_addr = tmem + 256 + t * D + lane_off;
    const int tok = t0 + r / p.rt.head_tile, head = h0 + r % p.rt.head_tile;
    const bool in_tile = r < p.rt.rows && head < a.G;
    const float sl2 = a.scale * LOG2E;
    const float cap_in = SOFTCAP ? a.scale / a.softcap : 0.f, cap_out = SOFTCAP ? a.softcap * LOG2E : 0.f;
    uint32_t s_cnt = 0, p_cnt = 0, v_base = 0;  // v_base: V copies before the piece
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
        const int n_keys = step_keys(a, pc, step), chunks = (max(n_keys, 1) + 31) / 32;
        const bool partial = n_keys < TILE || step >= n_prefix;
        uint4 keep = first_bits(n_keys);
        if (step >= n_prefix) keep = valid && n_keys > 0 ? ancestor_bits(a, pc.b, tok, x0) : make_uint4(0u, 0u, 0u, 0u);
        if (!tree_wait(smem_u32(&bars->s_full[t]), s_cnt & 1, wc)) { ok = false; break; }
        ++s_cnt;
        tc_fence_after();
        if (busy) {
          // Two passes over the scores in tensor memory, 32 at a time with the next
          // 32 on their way: a loop body small enough for the instruction cache
          // (128 scores in registers, fully unrolled, took twice as long).
          float xa[32], xb[32], mx = -INFINITY;
          tmem_ld32(s_addr, reinterpret_cast<uint32_t(&)[32]>(xa));
#pragma unroll 1
          for (int c = 0; c < chunks; c += 2) {
            tmem_wait_ld();
            if (c + 1 < chunks) tmem_ld32(s_addr + (c + 1) * 32, reinterpret_cast<uint32_t(&)[32]>(xb));
            chunk_scores<SOFTCAP>(xa, partial, word_of(keep, c), cap_in, cap_out);
            mx = chunk_max(xa, mx);
            if (c + 1 < chunks) {
              tmem_wait_ld();
              if (c + 2 < chunks) tmem_ld32(s_addr + (c + 2) * 32, reinterpret_cast<uint32_t(&)[32]>(xa));
              chunk_scores<SOFTCAP>(xb, partial, word_of(keep, c + 1), cap_in, cap_out);
              mx = chunk_max(xb, mx);
            }
          }
          tmem_ld32(s_addr, reinterpret_cast<uint32_t(&)[32]>(xa));  // for the second pass
          if (!SOFTCAP) mx *= sl2;  // -inf stays -inf (sl2 > 0)
          const float m_new = fmaxf(m_run, mx);
          const bool need = m_new > m_run + kTreeRescale;
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
          // P of chunk c lands in columns 16 c .. 16 c + 15, scores already read
#pragma unroll 1
          for (int c = 0; c < chunks; c += 2) {
            tmem_wait_ld();
            if (c + 1 < chunks) tmem_ld32(s_addr + (c + 1) * 32, reinterpret_cast<uint32_t(&)[32]>(xb));
            chunk_scores<SOFTCAP>(xa, partial, word_of(keep, c), cap_in, cap_out);
            if (c + 1 < chunks) {
              chunk_probs<SOFTCAP>(xa, sl2, m_use, s_addr + c * 16, acc);
              tmem_wait_ld();
              if (c + 2 < chunks) tmem_ld32(s_addr + (c + 2) * 32, reinterpret_cast<uint32_t(&)[32]>(xa));
              chunk_scores<SOFTCAP>(xb, partial, word_of(keep, c + 1), cap_in, cap_out);
              chunk_probs<SOFTCAP>(xb, sl2, m_use, s_addr + (c + 1) * 16, acc);
            } else {
              chunk_probs<SOFTCAP>(xa, sl2, m_use, s_addr + c * 16, acc);
            }
          }
          l_run += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
          tmem_wait_st();
        }
        if (n_keys < TILE) {
          // V rows of no key, up to the last the product takes: zeros, whatever lies there
          const uint32_t pos = v_base + j, slot = pos % Cfg::kStages;
          if (!tree_wait(smem_u32(&bars->v_full[slot]), (pos / Cfg::kStages) & 1, wc)) { ok = false; break; }
          uint8_t* v = smem + Cfg::kVOff + slot * Cfg::kTileBytes;
          const int rows = (max(n_keys, 1) + 15) / 16 * 16 - n_keys;
          for (int i = r; i < rows * (D / 8); i += 128) {  // 16-byte chunks; whole rows, so the swizzle does not matter
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
      // ---- end of the piece: join the even and the odd steps
      if (!tree_wait(smem_u32(&bars->o_final), it & 1, wc)) break;
      tc_fence_after();
      const uint32_t other_s = tmem + (1 - t) * 128 + lane_off;
      tmem_st2(s_addr, m_run, l_run);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->ml_ready[warp & 3]));
      if (!tree_wait(smem_u32(&bars->ml_ready[warp & 3]), it & 1, wc)) break;
      tc_fence_after();
      const float2 other = tmem_ld2(other_s);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->s_free));
      if (busy) {
        const float m0 = t == 0 ? m_run : other.x, m1 = t == 0 ? other.x : m_run;
        const float l0 = t == 0 ? l_run : other.y, l1 = t == 0 ? other.y : l_run;
        const float m = fmaxf(m0, m1);
        const float f0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - m), f1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - m);
        const float l = f0 * l0 + f1 * l1;
        const float inv = pc.slot >= 0 ? 1.f : (l > 0.f ? 1.f / l : 0.f);
        const float g0 = f0 * inv, g1 = f1 * inv;
        const long long part = static_cast<long long>(pc.slot) * p.rt.tiles + tile;
        float* po = p.part_o + (part * p.rt.rows + r) * D + t * (D / 2);
        __nv_bfloat16* orow = a.out + pc.b * a.o_st.b + (pc.hk * a.G + head) * a.o_st.h + tok * a.o_st.s + t * (D / 2);
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t o0[32], o1[32];
          const uint32_t col = t * (D / 2) + c * 32;
          tmem_ld32(tmem + 256 + lane_off + col, o0);
          if (pc.n > 1) tmem_ld32(tmem + 256 + D + lane_off + col, o1);
          tmem_wait_ld();
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            // a row whose even (odd) steps kept nothing holds zeros there
            o[e] = __uint_as_float(o0[e]) * g0;
            if (pc.n > 1) o[e] = fmaf(__uint_as_float(o1[e]), g1, o[e]);
          }
          if (valid) {
            if (pc.slot >= 0) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                reinterpret_cast<float4*>(po + c * 32)[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            } else {
              uint32_t pk[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) pk[e] = pack_bf16x2(o[2 * e], o[2 * e + 1]);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                reinterpret_cast<uint4*>(orow + c * 32)[e] = make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
            }
          }
        }
        if (valid && t == 0) {
          if (pc.slot >= 0) p.part_ml[part * p.rt.rows + r] = make_float2(m, l);
          else if (a.lse != nullptr)
            a.lse[(static_cast<long long>(pc.b) * a.Hq + pc.hk * a.G + head) * a.T + tok] =
                l > 0.f ? (m + log2f(l)) * LN2 : -INFINITY;
        }
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

// Join the pieces of the items that a range boundary cut: block (boundary,
// tile, 8 rows), one warp to a row, in the order of the pieces.
constexpr int kJoinThreads = 256, kJoinRows = 8;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const __grid_constant__ TreeParams p) {
  const TreeArgs& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tile = blockIdx.x % p.rt.tiles, g = blockIdx.x / p.rt.tiles + 1;
  RowScan scan;
  const long long total = scan_total(scan, a);
  const long long at = range_start(total, p.groups, g);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces are written
  if (at >= total) return;
  const RowAt row = scan_find(scan, a, at);
  const long long hk = (at - row.start) / row.steps, i0 = row.start + hk * row.steps, i1 = i0 + row.steps;
  if (!joins_item(total, p.groups, g, i0, i1)) return;
  const int t0 = tile / p.rt.head_chunks * p.rt.tok_tile, h0 = tile % p.rt.head_chunks * p.rt.head_tile;
  for (int r = blockIdx.y * kJoinRows + warp; r < min(p.rt.rows, (static_cast<int>(blockIdx.y) + 1) * kJoinRows);
       r += kJoinThreads / 32) {
    const int tok = t0 + r / p.rt.head_tile, head = h0 + r % p.rt.head_tile;
    if (head >= a.G || tok >= row.n_new) continue;
    // 32 pieces at a time: a lane to each for its (m, l), then their O rows in order
    float m = -INFINITY, l = 0.f, o[D / 32] = {};
    for (int x0 = g - 1; x0 < p.groups && range_start(total, p.groups, x0) < i1; x0 += 32) {
      const int x = x0 + lane;
      long long part = -1;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (x < p.groups) {
        const long long s = range_start(total, p.groups, x), e = range_start(total, p.groups, x + 1);
        if (s < i1 && e > s) {
          part = (static_cast<long long>(partial_slot(x, s >= i0)) * p.rt.tiles + tile) * p.rt.rows + r;
          ml = p.part_ml[part];
        }
      }
      float top = ml.x;
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      const float m2 = fmaxf(m, top);
      const float f = m == -INFINITY ? 0.f : exp2f(m - m2), mine = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m2);
      float sum = ml.y * mine;
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      m = m2;
      l = l * f + sum;
#pragma unroll
      for (int d = 0; d < D / 32; ++d) o[d] *= f;
      uint32_t left = __ballot_sync(0xffffffffu, part >= 0);
      while (left != 0) {  // four rows' loads at a time
        float v[4][D / 32], wt[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int src = left != 0 ? __ffs(left) - 1 : 0;
          const bool any = left != 0;
          left &= left - 1;
          const long long from = __shfl_sync(0xffffffffu, part, src);
          wt[i] = __shfl_sync(0xffffffffu, mine, src);
          if (!any) wt[i] = 0.f;
#pragma unroll
          for (int d = 0; d < D / 32; ++d) v[i][d] = any ? p.part_o[from * D + lane + 32 * d] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int d = 0; d < D / 32; ++d) o[d] = fmaf(v[i][d], wt[i], o[d]);
      }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    __nv_bfloat16* orow = a.out + row.b * a.o_st.b + (hk * a.G + head) * a.o_st.h + tok * a.o_st.s;
#pragma unroll
    for (int d = 0; d < D / 32; ++d) orow[lane + 32 * d] = __float2bfloat16(o[d] * inv);
    if (lane == 0 && a.lse != nullptr)
      a.lse[(static_cast<long long>(row.b) * a.Hq + hk * a.G + head) * a.T + tok] = l > 0.f ? (m + log2f(l)) * LN2 : -INFINITY;
  }
}

template <int D, bool SOFTCAP>
cudaError_t launch_tree_t(const TreeMaps& m, const TreeParams& p, cudaStream_t stream) {
  auto kernel = attn_tree_kernel<D, SOFTCAP>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = prepare_kernel(done, kernel, TreeCfg<D>::kAllocBytes, 0);
  if (e != cudaSuccess) return e;
  kernel<<<p.groups * p.rt.tiles, kTreeThreads, TreeCfg<D>::kAllocBytes, stream>>>(m.q, m.k, m.v, m.kn, m.vn, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.groups == 1) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((p.groups - 1) * p.rt.tiles, (p.rt.rows + kJoinRows - 1) / kJoinRows);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_join_kernel<D>, p);
}

}  // namespace

size_t tree_workspace_bytes(int G, int T, int D) {
  const RowTiles rt = row_tiles(G, T);
  // groups * tiles <= 148 where there is more than one group
  const size_t rows = static_cast<size_t>(2) * kTreeCtas * rt.rows;
  return (rows * D * 4 + 255) / 256 * 256 + (rows * 8 + 255) / 256 * 256;
}

cudaError_t launch_tree(const TreeMaps& m, const TreeArgs& a, void* workspace, uint64_t wait_ns, cudaStream_t stream) {
  TreeParams p{};
  p.a = a;
  p.rt = row_tiles(a.G, a.T);
  p.groups = tree_groups(p.rt.tiles);
  p.q_bufs = p.rt.rows <= 64 ? 2 : 1;
  const int ps = a.c.ix.page_size;
  while (ps << p.page_lg < TILE) ++p.page_lg;
  p.page_steps = ps / TILE;
  if (p.page_steps > 1) p.page_magic = static_cast<uint32_t>(((1ull << 32) + p.page_steps - 1) / p.page_steps);
  const size_t rows = static_cast<size_t>(2) * kTreeCtas * p.rt.rows;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + (rows * a.c.D * 4 + 255) / 256 * 256);
  p.wait_ns = wait_ns;
  if (a.c.D == 128) return a.softcap > 0.f ? launch_tree_t<128, true>(m, p, stream) : launch_tree_t<128, false>(m, p, stream);
  return a.softcap > 0.f ? launch_tree_t<64, true>(m, p, stream) : launch_tree_t<64, false>(m, p, stream);
}

}  // namespace attn25
