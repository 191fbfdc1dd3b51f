// The attention weight each slot of a paged KV cache received
// (attn_cache_weights), for sm_100a.
//
// For a key tile the scores are formed transposed, S^T = K Q^T: the 128 keys
// are the rows (TMEM lanes) and the query rows (heads of the group x tokens)
// the columns, so that a key's sum over all queries is a sum over one thread's
// columns, with no exchange between lanes and no atomics:
//   w_j += sum_r 2^(s_jr scale log2 e - LSE_r log2 e).
// A unit is a pair of key tiles (256 slots) of one (row, KV head); each of two
// warpgroups owns one of the tiles, and both use the same Q tiles.  A tile's
// 128 columns are summed from zero and added to a compensated (Kahan) total:
// a prompt adds up to a million exponentials into one fp32 number.
//
// Bounds.  A draft's few rows: the bytes of K, streamed once.  A prompt: the
// exponentials, one per visible (query, key) pair, on the special-function unit
// (1024 clocks to a 128x128 tile; the products take half of that).  Evaluating
// some of them on the FMA pipe instead, as the forward kernel does, was slower
// (a 4096-token prompt 198 us with none, 209 with a quarter, 219 with 3 of 8).
//
// Which unit a CTA takes: with one Q tile to a row, an equal contiguous range
// of the units in (row, head, pair) order, Q staying in shared memory while
// the head stays; with more, units in the order of their pair index over all
// rows and heads, i.e. longest first under the causal limit, in a snake.
// Prompts (no path) whose new tokens make fewer units than half the SMs are shared by clusters of
// 2 to 8 CTAs, each of which takes every C-th Q tile of a unit; the sums meet in
// the first CTA's shared memory and are added in the order of the CTAs.
//
// Warp roles (640 threads): four warpgroups of exponentials and sums, two to
// each key tile of the pair, which take its score buffers in turn (with one to a
// tile, two warps to an SM quarter, the quarter issued 0.47 instructions a
// clock: their latencies showed); warp 16 MMA issuer; warp 17 publishes the
// units and loads Q and the first tile of K, warp 19 the second (a copy from
// pages of 64 rows takes a warp ~1400 clocks, as long as HBM takes for it);
// warp 18 the columns' LSE and limits, and, when a path chooses the queries,
// the gather of their Q rows.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "cache.h"
#include "kernel_common.cuh"
#include "launch.h"

namespace attn25 {

namespace {

constexpr int kSumWarps = 16, kMmaWarp = 16, kTmaWarp = 17, kColumnWarp = 18, kTma2Warp = 19;
constexpr int kWThreads = 20 * 32;  // five warps to an SM quarter: a sixth would leave 80 registers a thread
constexpr int kLaneCols = TILE / 32;  // columns of a lane of the column warp
constexpr int kColSlots = 4;
constexpr int kUnits = 4;  // published ahead, so that the next head's Q is gathered in time

constexpr int kMaxSplit = 8;  // CTAs of a cluster
constexpr int kXStride = (kMaxSplit + 1) * TILE;  // sums of a key tile: the other warpgroup's, the other CTAs'

// Shared memory: Q slots, K slots of one tile each, sums on their way.  With
// one Q tile to a row (which stays while the head stays) one Q slot and all the
// rest for K; with more, Q tiles stream as well.
template <int D>
struct WCfg {
  static constexpr int kTileBytes = TILE * D * 2;
  static constexpr int kTiles = D == 128 ? 6 : 12;  // 192 KB
  static constexpr int kQSlots = D == 128 ? 2 : 4;  // where Q tiles stream
  static constexpr int kXOff = kTiles * kTileBytes;
  static constexpr int kBarOff = kXOff + 2 * (kMaxSplit + 1) * TILE * 4;
  static constexpr int kSmemBytes = kBarOff + 6144;
  static constexpr int kAllocBytes = kSmemBytes + 1024;
};

struct Unit {
  int32_t b, hk, kp;     // row, KV head, pair of key tiles; b < 0: the end
  int32_t len, n;        // filled slots and queries of the row
  int32_t rt0, n_rt;     // Q tiles rt0, rt0 + split, ... (n_rt of them) are this CTA's that see some of its keys
  int32_t new_q, keep_q; // the first Q tile has to be loaded / the last one serves the next unit too
};

struct WBarriers {
  uint64_t unit_full[kUnits], unit_empty[kUnits];
  uint64_t k_full[12], k_empty[12];
  uint64_t q_full[4], q_empty[4];  // a Q slot's copies; its products are done
  // a Q tile's columns (and, with a path, its gathered rows); read.  A ring of its
  // own, since the sums keep them for longer than the products keep Q.
  uint64_t c_full[kColSlots], c_empty[kColSlots];
  uint64_t s_full[2][2], s_empty[2][2];
  uint64_t j_full[2], j_empty[2];  // the other warpgroup's sum of a key tile: written (all 8 warps); read (4)
  uint64_t x_full[2], x_empty[2];  // a cluster's sums: written by the others (first CTA, all their threads of the
                                   // key tile); read (the others, 8 warps)
  uint64_t drain;
  uint32_t tmem_base, abort_flag, never_set;
  Unit unit[kUnits];
  int32_t min_lim[kColSlots];   // smallest limit of a Q tile's columns
  alignas(16) float neg[kColSlots][TILE];  // -LSE log2 e of the columns
  alignas(16) int32_t lim[kColSlots][TILE];  // the slots below the column's limit are the ones it sees
};
static_assert(sizeof(WBarriers) <= 6144, "barrier block");

constexpr int kUnitReaders = kSumWarps + 3;  // and the MMA, column and second TMA warps

struct WParams {
  WeightsArgs a;
  RowTiles rt;
  bool one_tile;  // every row's queries fit one Q tile
  int split;      // CTAs of a cluster that share a unit
  int q_slots, k_slots[2], q_stride;  // slots of each key tile's ring; bytes between Q slots
  uint32_t head_magic;  // row / head_tile = row * head_magic >> 16 (rows below 128)
  uint64_t wait_ns;
};

__device__ __forceinline__ void flag_index(int* status) { atomicCAS(status, 0, kErrIndex); }

// A place in a ring of `n` slots.
struct SlotPos {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) {
      slot = 0;
      phase ^= 1;
    }
  }
};

__device__ __forceinline__ bool w_wait(uint32_t bar, uint32_t parity, const WaitCtl& w) {
  return mbar_wait_warp_ool(bar, parity, w);
}

// ------------------------------------------------------------------ cluster
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The bounded warp wait for arrivals of other CTAs (acquire at cluster scope).
static __device__ __noinline__ bool wait_cluster(uint32_t bar, uint32_t parity, WaitCtl w) {
  const uint64_t t0 = globaltimer();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (__all_sync(0xffffffffu, ok != 0)) return true;
    bool give_up = aborted(w);
    if (!give_up && globaltimer() - t0 > w.limit_ns) {
      give_up = true;
      record_error(kErrTimeout, w);
    }
    if (__any_sync(0xffffffffu, give_up)) return false;
  }
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ------------------------------------------------------------------ units
//
// 32 rows' lengths at a time, one to a lane; pairs of key tiles of a row.
struct WScan {
  int base, len, n, pairs;
};

__device__ __forceinline__ void w_load(WScan& s, const WeightsArgs& a, int base) {
  const int b = base + (threadIdx.x & 31);
  bool bad = false;
  s.base = base;
  s.len = s.n = s.pairs = 0;
  if (b < a.c.ix.B) {
    s.len = clamp_count(a.c.ix.lens[b], a.c.ix.capacity, bad);
    s.n = clamp_count(a.counts != nullptr ? a.counts[b] : a.T, min(a.T, s.len), bad);
    s.pairs = (s.len + 2 * TILE - 1) / (2 * TILE);
  }
  if (bad) flag_index(a.c.status);
}

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Units whose pair index is below k (all of them: k = INT_MAX), over all rows and heads.
__device__ __forceinline__ long long units_below(WScan& s, const WeightsArgs& a, int k) {
  long long sum = 0;
  if (a.c.ix.B <= 32) {
    sum = min(s.pairs, k);
  } else {
    for (int base = 0; base < a.c.ix.B; base += 32) {
      w_load(s, a, base);
      sum += min(s.pairs, k);
    }
  }
  return warp_sum(sum) * a.c.ix.Hkv;
}

__device__ __forceinline__ int inclusive(int x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Find the row in which a running count over rows passes `at`: per-row counts
// by `count(lane's window)`; leaves the offset inside the row in `at`.
template <class F>
__device__ __forceinline__ Unit find_row(WScan& s, const WeightsArgs& a, long long& at, F count) {
  if (s.base != 0) w_load(s, a, 0);
  while (true) {
    const int c = count(s), inc = inclusive(c);
    const uint32_t past = __ballot_sync(0xffffffffu, inc > at);
    if (past != 0) {
      const int l = __ffs(past) - 1;
      Unit u{};
      u.b = s.base + l;
      u.len = __shfl_sync(0xffffffffu, s.len, l);
      u.n = __shfl_sync(0xffffffffu, s.n, l);
      at -= __shfl_sync(0xffffffffu, inc - c, l);
      return u;
    }
    at -= __shfl_sync(0xffffffffu, inc, 31);
    w_load(s, a, s.base + 32);
  }
}

// The Q tiles that see some key of the unit: those from the first query at or
// behind the pair's first slot.
__device__ __forceinline__ void set_tiles(Unit& u, const RowTiles& rt, int rank, int split) {
  const int first = u.kp * 2 * TILE - (u.len - u.n);
  u.rt0 = (first > 0 ? first / rt.tok_tile * rt.head_chunks : 0) + rank;
  const int all = (u.n + rt.tok_tile - 1) / rt.tok_tile * rt.head_chunks;
  u.n_rt = all > u.rt0 ? (all - u.rt0 + split - 1) / split : 0;
  u.new_q = u.n_rt > 0;
  u.keep_q = 0;
}

// First token, first head and valid rows of a Q tile of a row with n queries.
struct QTile {
  int i0, h0, rows, cols;
};
__device__ __forceinline__ QTile q_tile(const RowTiles& rt, int G, int n, int tile) {
  QTile q;
  q.i0 = tile / rt.head_chunks * rt.tok_tile;
  q.h0 = tile % rt.head_chunks * rt.head_tile;
  q.rows = min(rt.tok_tile, n - q.i0) * rt.head_tile;
  q.cols = (q.rows + 31) / 32 * 32;  // columns that are formed and summed
  return q;
}

// ------------------------------------------------------------------ sums
//
// One thread's 32 columns: 2^(x sl2 + neg), added into acc (pairs).
template <bool SOFTCAP>
__device__ __forceinline__ void sum_full(const uint32_t (&x)[32], const float* neg, float sl2, float cap_in, float cap_out,
                                         float2 (&acc)[2]) {
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const float4 ng = *reinterpret_cast<const float4*>(neg + e);
    float2 a0, a1;
    if constexpr (SOFTCAP) {
      a0 = make_float2(fmaf(tanh_ex2(__uint_as_float(x[e]) * cap_in), cap_out, ng.x),
                       fmaf(tanh_ex2(__uint_as_float(x[e + 1]) * cap_in), cap_out, ng.y));
      a1 = make_float2(fmaf(tanh_ex2(__uint_as_float(x[e + 2]) * cap_in), cap_out, ng.z),
                       fmaf(tanh_ex2(__uint_as_float(x[e + 3]) * cap_in), cap_out, ng.w));
    } else {
      const float2 s2 = make_float2(sl2, sl2);
      a0 = __ffma2_rn(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), s2, make_float2(ng.x, ng.y));
      a1 = __ffma2_rn(make_float2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), s2, make_float2(ng.z, ng.w));
    }
    acc[0] = __fadd2_rn(acc[0], make_float2(ex2_approx(a0.x), ex2_approx(a0.y)));
    acc[1] = __fadd2_rn(acc[1], make_float2(ex2_approx(a1.x), ex2_approx(a1.y)));
  }
}

// The same where some columns do not see some keys (or do not exist): those are left out by selection.
template <bool SOFTCAP>
__device__ __forceinline__ void sum_limited(const uint32_t (&x)[32], const float* neg, const int32_t* lim, int key, float sl2,
                                            float cap_in, float cap_out, float2 (&acc)[2]) {
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    float s = __uint_as_float(x[e]);
    s = SOFTCAP ? fmaf(tanh_ex2(s * cap_in), cap_out, neg[e]) : fmaf(s, sl2, neg[e]);
    const float v = key < lim[e] ? ex2_approx(s) : 0.f;
    if (e & 1) acc[(e >> 1) & 1].y += v;
    else acc[(e >> 1) & 1].x += v;
  }
}

// Load key tile t of a unit into its ring (the second follows the first's
// slots).  false: a wait ran out.
template <int D>
__device__ __forceinline__ bool load_k(const WParams& p, const Unit& u, int t, const CUtensorMap* map, uint32_t k_ring,
                                       WBarriers* bars, SlotPos& kp, int& copies, const WaitCtl& wc) {
  const WeightsArgs& a = p.a;
  const int s0 = u.kp * 2 * TILE + t * TILE;
  if (u.n_rt == 0 || s0 >= u.len) return true;
  const int lane = threadIdx.x & 31, ps = a.c.ix.page_size, box_rows = ps < TILE ? ps : TILE;
  const int boxes = (min(TILE, u.len - s0) + box_rows - 1) / box_rows;
  int entry = 0;  // of the tile's page `lane` (at most 8)
  if (lane < boxes) {
    const long long e = static_cast<long long>(u.b) * a.c.ix.max_pages + (s0 + lane * box_rows) / ps;
    entry = a.c.ix.table != nullptr ? __ldg(a.c.ix.table + e) : static_cast<int>(e);
  }
  const int y = ps > TILE ? s0 % ps : 0, slot = (t == 0 ? 0 : p.k_slots[0]) + kp.slot;
  const uint32_t bar = smem_u32(&bars->k_full[slot]), dst = k_ring + slot * WCfg<D>::kTileBytes;
  if (!w_wait(smem_u32(&bars->k_empty[slot]), kp.phase ^ 1, wc)) return false;
  if (lane == 0) mbar_arrive_expect_tx(bar, boxes * box_rows * D * 2);
  for (int i = 0; i < boxes; ++i) {
    int page = __shfl_sync(0xffffffffu, entry, i);
    const bool outside = page < 0 || page >= a.c.ix.num_pages;
    if (outside) page = a.c.ix.num_pages;  // past the pool: the copy fills in zeros
    if (lane == 0) {
      if (outside) flag_index(a.c.status);
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        tma_load_4d(dst + c * (TILE * 128) + i * box_rows * 128, map, bar, c * 64, y, u.hk, page);
    }
  }
  __syncwarp();
  kp.next(p.k_slots[t]);
  ++copies;
  return true;
}

// Let a ring's last copies land before the CTA exits (one thread).
__device__ __forceinline__ void drain_slots(uint64_t* full, int slots, int copies, const WaitCtl& wc) {
  for (int s = 0; s < slots; ++s) {
    const int uses = (copies + slots - 1 - s) / slots;
    if (uses > 0) mbar_wait_thread(smem_u32(full + s), (uses - 1) & 1, wc);
  }
}

template <int D, bool SOFTCAP>
__global__ void __launch_bounds__(kWThreads, 1)
    cache_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ WParams p) {
  using Cfg = WCfg<D>;
  const WeightsArgs& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  WBarriers* bars = reinterpret_cast<WBarriers*>(smem + Cfg::kBarOff);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t k_ring = sbase + (p.one_tile ? 1 : p.q_slots) * Cfg::kTileBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? static_cast<int>(cta_rank()) : 0;
  const int walkers = gridDim.x / p.split, walker = blockIdx.x / p.split;  // clusters walk together

  if (threadIdx.x == 0) {
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(smem_u32(&bars->unit_full[i]), 1);
      mbar_init(smem_u32(&bars->unit_empty[i]), kUnitReaders);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->j_full[i]), 8);
      mbar_init(smem_u32(&bars->j_empty[i]), 4);
      mbar_init(smem_u32(&bars->x_full[i]), max(1, (p.split - 1) * 2 * TILE));  // (unused where split is 1)
      mbar_init(smem_u32(&bars->x_empty[i]), 8);
      for (int t = 0; t < 2; ++t) {
        mbar_init(smem_u32(&bars->s_full[t][i]), 1);
        mbar_init(smem_u32(&bars->s_empty[t][i]), 4);
      }
    }
    for (int i = 0; i < 12; ++i) {
      mbar_init(smem_u32(&bars->k_full[i]), 1);
      mbar_init(smem_u32(&bars->k_empty[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&bars->q_full[i]), 1);
      mbar_init(smem_u32(&bars->q_empty[i]), 1);
    }
    for (int i = 0; i < kColSlots; ++i) {
      mbar_init(smem_u32(&bars->c_full[i]), 32);
      mbar_init(smem_u32(&bars->c_empty[i]), kSumWarps);
    }
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort_flag = 0;
    bars->never_set = 0;
    fence_mbar_init();
  }
  // rows that no Q tile fills stay zero (their columns' sums then add 2^-inf)
  const int room = p.one_tile && p.q_slots == 2 ? 64 : TILE;  // rows of a slot
  for (int s = 0; s < p.q_slots; ++s)
    for (int i = threadIdx.x; i < (room - p.rt.rows) * (D / 8); i += kWThreads) {
      const int row = p.rt.rows + i / (D / 8), ch = i % (D / 8);
      *reinterpret_cast<uint4*>(smem + s * p.q_stride + (ch >> 3) * (TILE * 128) + row * 128 + (ch & 7) * 16) =
          make_uint4(0u, 0u, 0u, 0u);
    }
  fence_proxy_async_smem();
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
  }
  tc_fence_before();
  __syncthreads();
  if (p.split > 1) cluster_sync_all();  // the others' barriers are there
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const WaitCtl wc{p.wait_ns, smem_u32(&bars->abort_flag), a.c.status};

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------ TMA producer
    WScan scan;
    w_load(scan, a, 0);
    const long long total = units_below(scan, a, INT_MAX);
    long long at = raw_cut(total, walkers, walker);
    const long long end = raw_cut(total, walkers, walker + 1);
    auto nth = [&](long long u) {  // unit u in the order of the grid's walk
      Unit x;
      if (p.one_tile) {
        x = find_row(scan, a, u, [&](const WScan& s) { return s.pairs * a.c.ix.Hkv; });
        const int pairs = (x.len + 2 * TILE - 1) / (2 * TILE);
        x.hk = static_cast<int>(u) / pairs;
        x.kp = static_cast<int>(u) % pairs;
      } else {
        int lo = 0, hi = a.c.ix.capacity / (2 * TILE) + 1;  // the last pair index with units_below <= u
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (units_below(scan, a, mid) <= u) lo = mid;
          else hi = mid;
        }
        u -= units_below(scan, a, lo);
        if (a.c.ix.B > 32) w_load(scan, a, 0);
        x = find_row(scan, a, u, [&](const WScan& s) { return s.pairs > lo ? a.c.ix.Hkv : 0; });
        x.hk = static_cast<int>(u);
        x.kp = lo;
      }
      set_tiles(x, p.rt, rank, p.split);
      return x;
    };
    Unit next{};
    next.b = -1;
    int wave = 0;
    if (p.one_tile) {
      if (at < end) next = nth(at);
    } else if (walker < total) {
      next = nth(walker);
    }
    SlotPos kp, qp;
    int k_copies = 0, q_copies = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      Unit u = next;
      // the next unit, so that this one's record can say whether Q stays
      next.b = -1;
      if (u.b >= 0) {
        if (p.one_tile) {
          if (++at < end) {
            const int pairs = (u.len + 2 * TILE - 1) / (2 * TILE);
            if (u.kp + 1 < pairs) {
              next = u;
              ++next.kp;
              next.new_q = 0;
              u.keep_q = u.n_rt > 0;
            } else {
              next = nth(at);
            }
          }
        } else {
          ++wave;
          const long long base = static_cast<long long>(wave) * walkers;
          const long long v = (wave & 1) ? base + walkers - 1 - walker : base + walker;
          if (v < total) next = nth(v);
        }
      }
      const int buf = it % kUnits;
      if (!w_wait(smem_u32(&bars->unit_empty[buf]), ((it / kUnits) & 1) ^ 1, wc)) { ok = false; break; }
      if (lane == 0) {
        bars->unit[buf] = u;
        mbar_arrive(smem_u32(&bars->unit_full[buf]));
      }
      __syncwarp();
      if (u.b < 0) break;
      if (!load_k<D>(p, u, 0, &tm_k, k_ring, bars, kp, k_copies, wc)) { ok = false; break; }
      // Q tiles (with a path the column warps gather them instead)
      for (int j = u.new_q ? 0 : 1; a.path == nullptr && j < u.n_rt; ++j) {
        if (!w_wait(smem_u32(&bars->q_empty[qp.slot]), qp.phase ^ 1, wc)) { ok = false; break; }
        if (lane == 0) {
          const uint32_t bar = smem_u32(&bars->q_full[qp.slot]);
          const QTile q = q_tile(p.rt, a.G, u.n, u.rt0 + j * p.split);
          mbar_arrive_expect_tx(bar, p.rt.rows * D * 2);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(sbase + qp.slot * p.q_stride + c * (TILE * 128), &tm_q, bar, c * 64, u.hk * a.G + q.h0, q.i0, u.b);
        }
        __syncwarp();
        qp.next(p.q_slots);
        ++q_copies;
      }
    }
    if (lane == 0) {  // let the copies in flight land before the CTA exits
      const WaitCtl drain_wc{drain_limit(p.wait_ns), smem_u32(&bars->never_set), a.c.status};
      drain_slots(bars->k_full, p.k_slots[0], k_copies, drain_wc);
      drain_slots(bars->q_full, p.q_slots, q_copies, drain_wc);
    }
  } else if (warp == kTma2Warp) {
    // ------------------------------------------------------------ second K tiles
    SlotPos kp;
    int copies = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int buf = it % kUnits;
      if (!w_wait(smem_u32(&bars->unit_full[buf]), (it / kUnits) & 1, wc)) break;
      const Unit u = bars->unit[buf];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->unit_empty[buf]));
      if (u.b < 0) break;
      ok = load_k<D>(p, u, 1, &tm_k, k_ring, bars, kp, copies, wc);
    }
    if (lane == 0)
      drain_slots(bars->k_full + p.k_slots[0], p.k_slots[1], copies,
                  WaitCtl{drain_limit(p.wait_ns), smem_u32(&bars->never_set), a.c.status});
  } else if (warp == kColumnWarp) {
    // ------------------------------------------------------------ columns of the Q tiles
    SlotPos qp, cp;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int buf = it % kUnits;
      if (!w_wait(smem_u32(&bars->unit_full[buf]), (it / kUnits) & 1, wc)) break;
      const Unit u = bars->unit[buf];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->unit_empty[buf]));
      if (u.b < 0) break;
      // this lane's columns (lane + 32 x) of tile j: read one tile ahead, looked at when it is published
      float lse[kLaneCols] = {};
      int lim[kLaneCols] = {}, node[kLaneCols] = {};  // node -1: no query
      auto fetch = [&](int j) {
        const QTile q = q_tile(p.rt, a.G, u.n, u.rt0 + j * p.split);
#pragma unroll
        for (int x = 0; x < kLaneCols; ++x) {
          const int r = lane + 32 * x, r_tok = static_cast<int>(r * p.head_magic >> 16), i = q.i0 + r_tok;
          const int head = q.h0 + r - r_tok * p.rt.head_tile;
          node[x] = r < p.rt.rows && i < u.n && head < a.G ? i : -1;
          if (node[x] >= 0 && a.path != nullptr) {
            node[x] = a.path[static_cast<long long>(u.b) * a.T + i];
            if (node[x] < 0 || node[x] >= a.T) {
              node[x] = -1;
              flag_index(a.c.status);
            }
          }
          // what no query fills holds zeros behind the tile's rows and where rows are
          // gathered: its column adds 2^-inf; elsewhere it may hold anything and is left out
          const bool zeros = r >= p.rt.rows || a.path != nullptr;
          lim[x] = node[x] >= 0 ? u.len - u.n + i + 1 : (zeros ? INT_MAX : 0);
          if (node[x] >= 0) lse[x] = __ldg(a.lse + (static_cast<long long>(u.b) * a.Hq + u.hk * a.G + head) * a.T + node[x]);
        }
      };
      const int j0 = u.new_q ? 0 : 1;
      if (j0 < u.n_rt) fetch(j0);
#pragma unroll 1
      for (int j = j0; j < u.n_rt; ++j) {
        const int slot = cp.slot;
        const QTile q = q_tile(p.rt, a.G, u.n, u.rt0 + j * p.split);
        float lse_now[kLaneCols];
        int lim_now[kLaneCols], node_now[kLaneCols], low = INT_MAX;
#pragma unroll
        for (int x = 0; x < kLaneCols; ++x) {
          lse_now[x] = lse[x];
          lim_now[x] = lim[x];
          node_now[x] = node[x];
          if (lane + 32 * x < q.cols) low = min(low, lim[x]);
        }
        if (j + 1 < u.n_rt) fetch(j + 1);
        low = __reduce_min_sync(0xffffffffu, low);
        if (!w_wait(smem_u32(&bars->c_empty[slot]), cp.phase ^ 1, wc)) { ok = false; break; }
        if (lane == 0) bars->min_lim[slot] = low;
#pragma unroll
        for (int x = 0; x < kLaneCols; ++x) {
          bars->neg[slot][lane + 32 * x] = node_now[x] >= 0 ? -lse_now[x] * LOG2E : -INFINITY;
          bars->lim[slot][lane + 32 * x] = lim_now[x];
        }
        if (a.path != nullptr) {
          // the chosen queries' rows, in the 128-byte swizzle (chunk c of row r at
          // c ^ (r & 7))
          if (!w_wait(smem_u32(&bars->q_empty[qp.slot]), qp.phase ^ 1, wc)) { ok = false; break; }
          uint8_t* dst = smem + qp.slot * p.q_stride;
          constexpr int kChunks = D / 8, kRows = 32 / kChunks;  // chunks of a row, rows of a pass
          const int ch = lane % kChunks, sub = lane / kChunks;
#pragma unroll
          for (int x = 0; x < kLaneCols; ++x) {
            const int base = 32 * x;
            if (base >= q.cols) continue;
            // all loads of a batch before its stores
            constexpr int kBatch = 8;
#pragma unroll 1
            for (int y0 = 0; y0 < 32; y0 += kBatch * kRows) {
              uint4 v[kBatch];
#pragma unroll
              for (int e = 0; e < kBatch; ++e) {
                const int y = y0 + e * kRows + sub, r = base + y, r_tok = static_cast<int>(r * p.head_magic >> 16);
                const int n = __shfl_sync(0xffffffffu, node_now[x], y & 31);
                const long long at = u.b * a.q_st.b + (u.hk * a.G + q.h0 + r - r_tok * p.rt.head_tile) * a.q_st.h + n * a.q_st.s;
                v[e] = __ldg(reinterpret_cast<const uint4*>(a.q + (n >= 0 ? at : 0) + ch * 8));
                if (n < 0) v[e] = make_uint4(0u, 0u, 0u, 0u);
              }
#pragma unroll
              for (int e = 0; e < kBatch; ++e) {
                const int r = base + y0 + e * kRows + sub;
                *reinterpret_cast<uint4*>(dst + (ch >> 3) * (TILE * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v[e];
              }
            }
          }
          fence_proxy_async_smem();
          qp.next(p.q_slots);
        }
        mbar_arrive(smem_u32(&bars->c_full[slot]));
        cp.next(kColSlots);
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    SlotPos kp[2], qp, cp, cur, cols;  // cur, cols: the Q and column slots in use
    uint32_t sc[2] = {0, 0};
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int buf = it % kUnits;
      if (!w_wait(smem_u32(&bars->unit_full[buf]), (it / kUnits) & 1, wc)) break;
      const Unit u = bars->unit[buf];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->unit_empty[buf]));
      if (u.b < 0) break;
      if (u.n_rt == 0) continue;
      const int tiles = u.len - u.kp * 2 * TILE > TILE ? 2 : 1;
#pragma unroll 1
      for (int j = 0; j < u.n_rt && ok; ++j) {
        if (j > 0 || u.new_q) {
          cur = qp;
          qp.next(p.q_slots);
          cols = cp;
          cp.next(kColSlots);
        }
        // (gathered rows come with their columns)
        if (!(a.path == nullptr ? w_wait(smem_u32(&bars->q_full[cur.slot]), cur.phase, wc)
                                : w_wait(smem_u32(&bars->c_full[cols.slot]), cols.phase, wc))) {
          ok = false;
          break;
        }
        const QTile q = q_tile(p.rt, a.G, u.n, u.rt0 + j * p.split);
        const uint32_t idesc = idesc_bf16_f32(128, q.cols, false, false);
        const uint32_t q_smem = sbase + cur.slot * p.q_stride;
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
          const int sb = sc[t] & 1;
          const int k_slot = t == 0 ? kp[0].slot : p.k_slots[0] + kp[1].slot;
          if ((j == 0 && !w_wait(smem_u32(&bars->k_full[k_slot]), t == 0 ? kp[0].phase : kp[1].phase, wc)) ||
              !w_wait(smem_u32(&bars->s_empty[t][sb]), ((sc[t] >> 1) & 1) ^ 1, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          ++sc[t];
          const uint32_t k_smem = k_ring + k_slot * Cfg::kTileBytes;
          const uint32_t a_lo = smem_desc_lo(k_smem, 16), b_lo = smem_desc_lo(q_smem, 16), d = tmem + (t * 2 + sb) * 128;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * (TILE * 128) + (kk & 3) * 32) >> 4;
            mma_ss_lo_w<smem_desc_hi_sw128(1024)>(d, a_lo + off, b_lo + off, idesc, kk > 0 ? 1u : 0u);
          }
          mma_commit_w(smem_u32(&bars->s_full[t][sb]));
          if (j == u.n_rt - 1) mma_commit_w(smem_u32(&bars->k_empty[k_slot]));
        }
        if (ok && (j < u.n_rt - 1 || !u.keep_q)) mma_commit_w(smem_u32(&bars->q_empty[cur.slot]));
      }
      kp[0].next(p.k_slots[0]);
      if (tiles > 1) kp[1].next(p.k_slots[1]);
    }
    mma_commit_w(smem_u32(&bars->drain));
    w_wait(smem_u32(&bars->drain), 0, WaitCtl{drain_limit(p.wait_ns), smem_u32(&bars->never_set), a.c.status});
  } else {
    // ------------------------------------------------------------ exponentials and sums
    const int t = (warp >> 2) & 1, sb = warp >> 3, r = threadIdx.x & 127;  // key tile, score buffer, key
    const uint32_t s_addr = tmem + (t * 2 + sb) * 128 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const float sl2 = a.scale * LOG2E;
    const float cap_in = SOFTCAP ? a.scale / a.softcap : 0.f, cap_out = SOFTCAP ? a.softcap * LOG2E : 0.f;
    SlotPos cp, cur;
    uint32_t sc = 0;      // steps of the tile so far: buffer sc & 1 holds the next
    uint32_t joins = 0, shared = 0;  // units that both warpgroups, or several CTAs, had a part of
    float* x_buf = reinterpret_cast<float*>(smem + Cfg::kXOff) + t * kXStride;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int buf = it % kUnits;
      if (!w_wait(smem_u32(&bars->unit_full[buf]), (it / kUnits) & 1, wc)) break;
      const Unit u = bars->unit[buf];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->unit_empty[buf]));
      if (u.b < 0) break;
      const int key0 = u.kp * 2 * TILE + t * TILE, key = key0 + r;
      const bool here = key0 < u.len;  // the second tile of a row's last pair may hold nothing
      // the warpgroup that takes the last step writes the unit (without steps: the one whose turn it is)
      const bool owner = ((sc + (u.n_rt > 0 ? u.n_rt - 1 : 0)) & 1) == static_cast<uint32_t>(sb);
      const long long entry = slot_entry(a.c.ix, u.b, u.hk, key);
      float base = 0.f;
      if (owner && rank == 0 && a.w_in != nullptr && key < u.len - u.n) base = a.w_in[entry];
      float total = 0.f, lost = 0.f;
#pragma unroll 1
      for (int j = 0; j < u.n_rt; ++j) {
        if (j > 0 || u.new_q) {
          cur = cp;
          cp.next(kColSlots);
        }
        const int slot = cur.slot;
        // (waited for also where there is nothing to do, so that no slot is handed back twice in one use)
        if (!w_wait(smem_u32(&bars->c_full[slot]), cur.phase, wc)) { ok = false; break; }
        if (here) {
          if ((sc & 1) == static_cast<uint32_t>(sb)) {
            const QTile q = q_tile(p.rt, a.G, u.n, u.rt0 + j * p.split);
            if (!w_wait(smem_u32(&bars->s_full[t][sb]), (sc >> 1) & 1, wc)) { ok = false; break; }
            tc_fence_after();
            const bool full = bars->min_lim[slot] >= key0 + TILE;
            float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
            for (int c = 0; c < q.cols; c += 32) {
              uint32_t x[32];
              tmem_ld32(s_addr + c, x);
              tmem_wait_ld();
              if (c + 32 >= q.cols) {  // the scores are read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->s_empty[t][sb]));
              }
              if (full) sum_full<SOFTCAP>(x, bars->neg[slot] + c, sl2, cap_in, cap_out, acc);
              else sum_limited<SOFTCAP>(x, bars->neg[slot] + c, bars->lim[slot] + c, key, sl2, cap_in, cap_out, acc);
            }
            const float tile_sum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
            const float y = tile_sum - lost, z = total + y;  // Kahan
            lost = (z - total) - y;
            total = z;
          }
          ++sc;
        }
        __syncwarp();
        if (lane == 0 && (j < u.n_rt - 1 || !u.keep_q)) mbar_arrive(smem_u32(&bars->c_empty[slot]));
      }
      if (!ok) break;
      // A barrier's parity tells a phase only from its neighbours.  So that no warp
      // can run ahead of a phase, or fall behind one, every warp of the key tile has a
      // part in each: it waits for the phase before, and the next needs its arrival.
      if (here && u.n_rt > 1) {  // both warpgroups had steps
        if (joins > 0 && !w_wait(smem_u32(&bars->j_empty[t]), (joins - 1) & 1, wc)) break;
        if (!owner) x_buf[r] = total;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->j_full[t]));
        if (owner) {
          if (!w_wait(smem_u32(&bars->j_full[t]), joins & 1, wc)) break;
          total += x_buf[r];
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars->j_empty[t]));
        }
        ++joins;
      }
      if (p.split > 1) {
        if (rank > 0) {  // hand the sum to the first CTA once it has read the last unit's
          if (shared > 0 && !wait_cluster(smem_u32(&bars->x_empty[t]), (shared - 1) & 1, wc)) break;
          if (owner) st_cluster(in_cta(smem_u32(x_buf + rank * TILE + r), 0), total);
          arrive_cluster(in_cta(smem_u32(&bars->x_full[t]), 0));
        } else {
          if (!wait_cluster(smem_u32(&bars->x_full[t]), shared & 1, wc)) break;
          if (owner)
            for (int x = 1; x < p.split; ++x) total += x_buf[x * TILE + r];
          __syncwarp();
          if (lane > 0 && lane < p.split) arrive_cluster(in_cta(smem_u32(&bars->x_empty[t]), lane));
        }
        ++shared;
      }
      if (owner && rank == 0 && key < u.len) a.w_out[entry] = base + total;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (p.split > 1) cluster_sync_all();  // no CTA leaves while another may reach into its shared memory
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int D, bool SOFTCAP>
cudaError_t launch_weights_t(const CUtensorMap& tq, const CUtensorMap& tk, const WParams& p, int sms, cudaStream_t stream) {
  auto kernel = cache_weights_kernel<D, SOFTCAP>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = prepare_kernel(done, kernel, WCfg<D>::kAllocBytes, 0);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(sms / p.split * p.split);
  cfg.blockDim = dim3(kWThreads);
  cfg.dynamicSmemBytes = WCfg<D>::kAllocBytes;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = p.split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, tq, tk, p);
}

}  // namespace

cudaError_t launch_cache_weights(const CUtensorMap& tq, const CUtensorMap& tk, const WeightsArgs& a, uint64_t wait_ns, int sms,
                                 cudaStream_t stream) {
  WParams p{};
  p.a = a;
  p.rt = row_tiles(a.G, a.T);
  p.one_tile = p.rt.tiles == 1;
  const int q_slots = a.c.D == 128 ? WCfg<128>::kQSlots : WCfg<64>::kQSlots, tiles = a.c.D == 128 ? WCfg<128>::kTiles : WCfg<64>::kTiles;
  // one Q tile to a row: one slot's room for it, which holds two tiles of up to 64 rows
  const bool two = p.one_tile && p.rt.rows <= 64;
  p.q_slots = p.one_tile ? (two ? 2 : 1) : q_slots;
  p.q_stride = two ? 64 * 128 : TILE * a.c.D * 2;
  const int k_slots = tiles - (p.one_tile ? 1 : q_slots);
  p.k_slots[0] = (k_slots + 1) / 2;
  p.k_slots[1] = k_slots / 2;
  // a prompt's units, counted from its new tokens alone (the filled lengths are on the device):
  // shared while they fill less than half the SMs.  Not with a path: accepted drafts are few
  // queries over many more units than those, and each CTA of a cluster would read all their
  // keys (28 of 15 rows 51 against 38 us).  A chunk of a prompt, or a chain of drafts, over a
  // filled cache has more units too, and is shared all the same
  p.split = 1;
  if (!p.one_tile && a.path == nullptr) {
    const long long units = static_cast<long long>(a.c.ix.B) * a.c.ix.Hkv * ((a.T + 2 * TILE - 1) / (2 * TILE));
    while (p.split < kMaxSplit && units * p.split * 2 <= sms && p.rt.tiles >= p.split * 2) p.split *= 2;
  }
  p.head_magic = 65535u / p.rt.head_tile + 1;
  p.wait_ns = wait_ns;
  if (a.c.D == 128) return a.softcap > 0.f ? launch_weights_t<128, true>(tq, tk, p, sms, stream) : launch_weights_t<128, false>(tq, tk, p, sms, stream);
  return a.softcap > 0.f ? launch_weights_t<64, true>(tq, tk, p, sms, stream) : launch_weights_t<64, false>(tq, tk, p, sms, stream);
}

}  // namespace attn25
