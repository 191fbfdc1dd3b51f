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
// Bounds.  A draft's few rows: the bytes of K, streamed once (two units' 128
// KB of K in flight per SM).  A prompt: the exponentials, one per visible
// (query, key) pair; the products take a quarter of their time.
//
// Which unit a CTA takes: with one Q tile to a row, an equal contiguous range
// of the units in (row, head, pair) order, Q staying in shared memory while
// the head stays; with more, units in the order of their pair index over all
// rows and heads, i.e. longest first under the causal limit, in a snake.
//
// Warp roles (384 threads): warps 0-3 and 4-7 exponentials and sums of key
// tile 0 and 1 of the pair; warp 8 MMA issuer; warp 9 TMA producer, which
// publishes the units; warps 10-11 the columns' LSE and limits, and, when a
// path chooses the queries, the gather of their Q rows.
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

constexpr int kWThreads = 384;
constexpr int kMetaThreads = 64;

template <int D>
struct WCfg {
  static constexpr int kTileBytes = TILE * D * 2;
  static constexpr int kKBufs = D == 128 ? 2 : 4;  // K pairs in flight: 128 KB
  static constexpr int kQSlots = D == 128 ? 2 : 4;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQSlots * kTileBytes;
  static constexpr int kBarOff = kKOff + kKBufs * 2 * kTileBytes;
  static constexpr int kSmemBytes = kBarOff + 8192;
  static constexpr int kAllocBytes = kSmemBytes + 1024;
};

struct Unit {
  int32_t b, hk, kp;     // row, KV head, pair of key tiles; b < 0: the end
  int32_t len, n;        // filled slots and queries of the row
  int32_t rt0, n_rt;     // Q tiles [rt0, rt0 + n_rt) see some of its keys
  int32_t new_q, keep_q; // the first Q tile has to be loaded / the last one serves the next unit too
};

struct WBarriers {
  uint64_t unit_full[2], unit_empty[2];
  uint64_t k_full[4], k_empty[4];
  uint64_t q_full[4], c_full[4], q_empty[4];  // a Q slot's copies; its columns' values (and gathered rows); both used up
  uint64_t s_full[2][2], s_empty[2][2];
  uint64_t drain;
  uint32_t tmem_base, abort_flag, never_set;
  Unit unit[2];
  int32_t min_lim[4][2];           // smallest limit of each half of a Q tile's columns
  alignas(16) float neg[4][TILE];  // -LSE log2 e of the columns of a Q slot
  alignas(16) int32_t lim[4][TILE];  // the slots below the column's limit are the ones it sees
};
static_assert(sizeof(WBarriers) <= 8192, "barrier block");

constexpr int kUnitReaders = 11;  // MMA warp, 8 sum warps, 2 column warps

struct WParams {
  WeightsArgs a;
  RowTiles rt;
  bool one_tile;  // every row's queries fit one Q tile
  uint64_t wait_ns;
};

__device__ __forceinline__ void flag_index(int* status) { atomicCAS(status, 0, kErrIndex); }

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
__device__ __forceinline__ void set_tiles(Unit& u, const RowTiles& rt) {
  const int first = u.kp * 2 * TILE - (u.len - u.n);
  u.rt0 = first > 0 ? first / rt.tok_tile * rt.head_chunks : 0;
  const int all = (u.n + rt.tok_tile - 1) / rt.tok_tile * rt.head_chunks;
  u.n_rt = all > u.rt0 ? all - u.rt0 : 0;
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
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->unit_full[i]), 1);
      mbar_init(smem_u32(&bars->unit_empty[i]), kUnitReaders);
      for (int t = 0; t < 2; ++t) {
        mbar_init(smem_u32(&bars->s_full[t][i]), 1);
        mbar_init(smem_u32(&bars->s_empty[t][i]), 4);
      }
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&bars->k_full[i]), 1);
      mbar_init(smem_u32(&bars->k_empty[i]), 1);
      mbar_init(smem_u32(&bars->q_full[i]), 1);
      mbar_init(smem_u32(&bars->c_full[i]), kMetaThreads);
      mbar_init(smem_u32(&bars->q_empty[i]), 1 + 8);
    }
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort_flag = 0;
    bars->never_set = 0;
    fence_mbar_init();
  }
  // rows that no Q tile fills stay zero (their columns' sums then add 2^-inf)
  for (int s = 0; s < Cfg::kQSlots; ++s)
    for (int i = threadIdx.x; i < (TILE - p.rt.rows) * (D / 8); i += kWThreads) {
      const int row = p.rt.rows + i / (D / 8), ch = i % (D / 8);
      *reinterpret_cast<uint4*>(smem + Cfg::kQOff + s * Cfg::kTileBytes + (ch >> 3) * (TILE * 128) + row * 128 + (ch & 7) * 16) =
          make_uint4(0u, 0u, 0u, 0u);
    }
  fence_proxy_async_smem();
  if (warp == 8) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  if (warp == 9 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const WaitCtl wc{p.wait_ns, smem_u32(&bars->abort_flag), a.c.status};

  if (warp == 9) {
    // ------------------------------------------------------------ TMA producer
    const int ps = a.c.ix.page_size;
    const int box_rows = ps < TILE ? ps : TILE;
    WScan scan;
    w_load(scan, a, 0);
    const long long total = units_below(scan, a, INT_MAX);
    long long at = raw_cut(total, gridDim.x, blockIdx.x);
    const long long end = raw_cut(total, gridDim.x, blockIdx.x + 1);
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
      set_tiles(x, p.rt);
      return x;
    };
    Unit next{};
    next.b = -1;
    int wave = 0;
    if (p.one_tile) {
      if (at < end) next = nth(at);
    } else if (blockIdx.x < total) {
      next = nth(blockIdx.x);
    }
    uint32_t kn = 0, ql = 0;
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
          const long long base = static_cast<long long>(wave) * gridDim.x;
          const long long v = (wave & 1) ? base + gridDim.x - 1 - blockIdx.x : base + blockIdx.x;
          if (v < total) next = nth(v);
        }
      }
      const int buf = it & 1;
      if (!mbar_wait_warp(smem_u32(&bars->unit_empty[buf]), ((it >> 1) & 1) ^ 1, wc)) { ok = false; break; }
      if (lane == 0) {
        bars->unit[buf] = u;
        mbar_arrive(smem_u32(&bars->unit_full[buf]));
      }
      __syncwarp();
      if (u.b < 0) break;
      if (u.n_rt > 0) {
        // K of both tiles: the pages that hold filled slots, one box of a page
        // and 64 columns to a lane (at most 16 pages x 2)
        const int s0 = u.kp * 2 * TILE, used = min(2 * TILE, u.len - s0), boxes = (used + box_rows - 1) / box_rows;
        const int bx = lane / (D / 64), c = lane % (D / 64), kb = kn % Cfg::kKBufs;
        int page = a.c.ix.num_pages;  // past the pool: the copy fills in zeros
        const bool mine = bx < boxes;
        if (mine) {
          const int e = page_at(a.c.ix, u.b, (s0 + bx * box_rows) / ps);
          if (e >= 0) page = e;
          else flag_index(a.c.status);
        }
        if (!mbar_wait_warp(smem_u32(&bars->k_empty[kb]), ((kn / Cfg::kKBufs) & 1) ^ 1, wc)) { ok = false; break; }
        const uint32_t bar = smem_u32(&bars->k_full[kb]);
        if (lane == 0) mbar_arrive_expect_tx(bar, boxes * box_rows * D * 2);
        __syncwarp();
        const int row = bx * box_rows;  // within the pair
        if (mine)
          tma_load_4d(sbase + Cfg::kKOff + (kb * 2 + row / TILE) * Cfg::kTileBytes + c * (TILE * 128) + row % TILE * 128, &tm_k,
                      bar, c * 64, ps > TILE ? (s0 + row) % ps : 0, u.hk, page);
        __syncwarp();
        ++kn;
      }
      // Q tiles (with a path the column warps gather them instead)
      for (int j = u.new_q ? 0 : 1; a.path == nullptr && j < u.n_rt; ++j) {
        const int slot = ql % Cfg::kQSlots;
        if (!mbar_wait_warp(smem_u32(&bars->q_empty[slot]), ((ql / Cfg::kQSlots) & 1) ^ 1, wc)) { ok = false; break; }
        if (lane == 0) {
          const uint32_t bar = smem_u32(&bars->q_full[slot]);
          const QTile q = q_tile(p.rt, a.G, u.n, u.rt0 + j);
          mbar_arrive_expect_tx(bar, p.rt.rows * D * 2);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(sbase + Cfg::kQOff + slot * Cfg::kTileBytes + c * (TILE * 128), &tm_q, bar, c * 64,
                        u.hk * a.G + q.h0, q.i0, u.b);
        }
        __syncwarp();
        ++ql;
      }
    }
    if (lane == 0) {  // let the copies in flight land before the CTA exits
      const WaitCtl drain_wc{drain_limit(p.wait_ns), smem_u32(&bars->never_set), a.c.status};
      for (uint32_t s = 0; s < Cfg::kKBufs; ++s) {
        const uint32_t uses = (kn + Cfg::kKBufs - 1 - s) / Cfg::kKBufs;
        if (uses > 0) mbar_wait_thread(smem_u32(&bars->k_full[s]), (uses - 1) & 1, drain_wc);
      }
      for (uint32_t s = 0; s < Cfg::kQSlots; ++s) {
        const uint32_t uses = (ql + Cfg::kQSlots - 1 - s) / Cfg::kQSlots;
        if (uses > 0) mbar_wait_thread(smem_u32(&bars->q_full[s]), (uses - 1) & 1, drain_wc);
      }
    }
  } else if (warp >= 10) {
    // ------------------------------------------------------------ columns of the Q tiles
    const int m = threadIdx.x - 10 * 32;
    uint32_t ql = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int buf = it & 1;
      if (!mbar_wait_warp(smem_u32(&bars->unit_full[buf]), (it >> 1) & 1, wc)) break;
      const Unit u = bars->unit[buf];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->unit_empty[buf]));
      if (u.b < 0) break;
      for (int j = u.new_q ? 0 : 1; j < u.n_rt; ++j) {
        const int slot = ql % Cfg::kQSlots;
        const QTile q = q_tile(p.rt, a.G, u.n, u.rt0 + j);
        // read ahead of the slot: its columns' LSE and nodes
        float neg[2];
        int lim[2], low = INT_MAX;
        bool bad = false;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = m + 64 * x, i = q.i0 + r / p.rt.head_tile, head = q.h0 + r % p.rt.head_tile;
          neg[x] = -INFINITY;
          lim[x] = INT_MAX;
          if (r < p.rt.rows) {
            int node = i;
            if (i < u.n && a.path != nullptr) {
              node = a.path[static_cast<long long>(u.b) * a.T + i];
              if (node < 0 || node >= a.T) bad = true;
            }
            const bool real = i < u.n && head < a.G && node >= 0 && node < a.T;
            // a gathered tile holds zeros where there is no query: its column adds 2^-inf
            const bool zeros = a.path != nullptr && !real;
            lim[x] = real ? u.len - u.n + i + 1 : (zeros ? INT_MAX : 0);
            neg[x] = real ? -a.lse[(static_cast<long long>(u.b) * a.Hq + u.hk * a.G + head) * a.T + node] * LOG2E : -INFINITY;
            if (r < q.cols) low = min(low, lim[x]);
          }
        }
        if (bad) flag_index(a.c.status);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) low = min(low, __shfl_xor_sync(0xffffffffu, low, o));
        if (!mbar_wait_warp(smem_u32(&bars->q_empty[slot]), ((ql / Cfg::kQSlots) & 1) ^ 1, wc)) { ok = false; break; }
        if (lane == 0) bars->min_lim[slot][warp - 10] = low;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          bars->neg[slot][m + 64 * x] = neg[x];
          bars->lim[slot][m + 64 * x] = lim[x];
        }
        if (a.path != nullptr) {
          // the chosen queries' rows, in the 128-byte swizzle: chunk c of row r at c ^ (r & 7)
          uint8_t* dst = smem + Cfg::kQOff + slot * Cfg::kTileBytes;
#pragma unroll 4
          for (int x = m; x < q.cols * (D / 8); x += kMetaThreads) {
            const int r = x / (D / 8), ch = x % (D / 8), i = q.i0 + r / p.rt.head_tile, head = q.h0 + r % p.rt.head_tile;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (r < q.rows && head < a.G) {
              const int node = a.path[static_cast<long long>(u.b) * a.T + i];
              if (node >= 0 && node < a.T)
                v = __ldg(reinterpret_cast<const uint4*>(a.q + u.b * a.q_st.b + (u.hk * a.G + head) * a.q_st.h +
                                                         node * a.q_st.s + ch * 8));
            }
            *reinterpret_cast<uint4*>(dst + (ch >> 3) * (TILE * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v;
          }
          fence_proxy_async_smem();
        }
        mbar_arrive(smem_u32(&bars->c_full[slot]));
        ++ql;
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ MMA issuer
    uint32_t kn = 0, ql = 0, sc[2] = {0, 0};
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int buf = it & 1;
      if (!mbar_wait_warp(smem_u32(&bars->unit_full[buf]), (it >> 1) & 1, wc)) break;
      const Unit u = bars->unit[buf];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->unit_empty[buf]));
      if (u.b < 0) break;
      if (u.n_rt == 0) continue;
      const int kb = kn % Cfg::kKBufs;
      if (!mbar_wait_warp(smem_u32(&bars->k_full[kb]), (kn / Cfg::kKBufs) & 1, wc)) break;
      ++kn;
      const int tiles = u.len - u.kp * 2 * TILE > TILE ? 2 : 1;
      for (int j = 0; j < u.n_rt && ok; ++j) {
        if (j > 0 || u.new_q) ++ql;  // load ql - 1 is the one in use
        const int slot = (ql - 1) % Cfg::kQSlots;
        const uint32_t phase = ((ql - 1) / Cfg::kQSlots) & 1;
        if (!mbar_wait_warp(smem_u32(&bars->c_full[slot]), phase, wc) ||
            (a.path == nullptr && !mbar_wait_warp(smem_u32(&bars->q_full[slot]), phase, wc))) {
          ok = false;
          break;
        }
        const QTile q = q_tile(p.rt, a.G, u.n, u.rt0 + j);
        const uint32_t idesc = idesc_bf16_f32(128, q.cols, false, false);
        const uint32_t q_smem = sbase + Cfg::kQOff + slot * Cfg::kTileBytes;
        for (int t = 0; t < tiles; ++t) {
          const int sb = sc[t] & 1;
          if (!mbar_wait_warp(smem_u32(&bars->s_empty[t][sb]), ((sc[t] >> 1) & 1) ^ 1, wc)) { ok = false; break; }
          tc_fence_after();
          ++sc[t];
          const uint32_t k_smem = sbase + Cfg::kKOff + (kb * 2 + t) * Cfg::kTileBytes;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * (TILE * 128) + (kk & 3) * 32;
            mma_ss_w(tmem + (t * 2 + sb) * 128, smem_desc_sw128(k_smem + off, 16, 1024),
                     smem_desc_sw128(q_smem + off, 16, 1024), idesc, kk > 0 ? 1u : 0u);
          }
          mma_commit_w(smem_u32(&bars->s_full[t][sb]));
        }
        if (ok && (j < u.n_rt - 1 || !u.keep_q)) mma_commit_w(smem_u32(&bars->q_empty[slot]));
      }
      if (ok) mma_commit_w(smem_u32(&bars->k_empty[kb]));
    }
    mma_commit_w(smem_u32(&bars->drain));
    mbar_wait_warp(smem_u32(&bars->drain), 0, WaitCtl{drain_limit(p.wait_ns), smem_u32(&bars->never_set), a.c.status});
  } else {
    // ------------------------------------------------------------ exponentials and sums
    const int t = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float sl2 = a.scale * LOG2E;
    const float cap_in = SOFTCAP ? a.scale / a.softcap : 0.f, cap_out = SOFTCAP ? a.softcap * LOG2E : 0.f;
    uint32_t ql = 0, sc = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int buf = it & 1;
      if (!mbar_wait_warp(smem_u32(&bars->unit_full[buf]), (it >> 1) & 1, wc)) break;
      const Unit u = bars->unit[buf];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->unit_empty[buf]));
      if (u.b < 0) break;
      const int key0 = u.kp * 2 * TILE + t * TILE, key = key0 + r;
      const bool here = key0 < u.len;  // the second tile of a row's last pair may hold nothing
      const long long entry = slot_entry(a.c.ix, u.b, u.hk, key);
      float base = 0.f;
      if (a.w_in != nullptr && key < u.len - u.n) base = a.w_in[entry];
      float total = 0.f, lost = 0.f;
      for (int j = 0; j < u.n_rt; ++j) {
        if (j > 0 || u.new_q) ++ql;
        const int slot = (ql - 1) % Cfg::kQSlots;
        // (waited for also where the tile holds nothing, so that no slot is handed back twice in one use)
        if (!mbar_wait_warp(smem_u32(&bars->c_full[slot]), ((ql - 1) / Cfg::kQSlots) & 1, wc)) { ok = false; break; }
        if (here) {
          const QTile q = q_tile(p.rt, a.G, u.n, u.rt0 + j);
          const int sb = sc & 1;
          if (!mbar_wait_warp(smem_u32(&bars->s_full[t][sb]), (sc >> 1) & 1, wc)) { ok = false; break; }
          ++sc;
          tc_fence_after();
          const uint32_t s_addr = tmem + (t * 2 + sb) * 128 + lane_off;
          const float* neg = bars->neg[slot];
          const int32_t* lim = bars->lim[slot];
          const bool full = min(bars->min_lim[slot][0], bars->min_lim[slot][1]) >= key0 + TILE;
          float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          const int chunks = q.cols / 32;
          uint32_t x[2][32];
          tmem_ld32(s_addr, x[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c < chunks) {
              tmem_wait_ld();
              if (c + 1 < chunks) {
                if (c < 3) tmem_ld32(s_addr + (c + 1) * 32, x[(c + 1) & 1]);
              } else {  // the scores are read: the buffer is free
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->s_empty[t][sb]));
              }
              if (full) sum_full<SOFTCAP>(x[c & 1], neg + c * 32, sl2, cap_in, cap_out, acc);
              else sum_limited<SOFTCAP>(x[c & 1], neg + c * 32, lim + c * 32, key, sl2, cap_in, cap_out, acc);
            }
          }
          const float tile_sum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
          const float y = tile_sum - lost, z = total + y;  // Kahan
          lost = (z - total) - y;
          total = z;
        }
        __syncwarp();
        if (lane == 0 && (j < u.n_rt - 1 || !u.keep_q)) mbar_arrive(smem_u32(&bars->q_empty[slot]));
      }
      if (!ok) break;
      if (key < u.len) a.w_out[entry] = base + total;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

template <int D, bool SOFTCAP>
cudaError_t launch_weights_t(const CUtensorMap& tq, const CUtensorMap& tk, const WParams& p, int sms, cudaStream_t stream) {
  auto kernel = cache_weights_kernel<D, SOFTCAP>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = prepare_kernel(done, kernel, WCfg<D>::kAllocBytes, 0);
  if (e != cudaSuccess) return e;
  kernel<<<sms, kWThreads, WCfg<D>::kAllocBytes, stream>>>(tq, tk, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_weights(const CUtensorMap& tq, const CUtensorMap& tk, const WeightsArgs& a, uint64_t wait_ns, int sms,
                                 cudaStream_t stream) {
  WParams p{};
  p.a = a;
  p.rt = row_tiles(a.G, a.T);
  p.one_tile = p.rt.tiles == 1;
  p.wait_ns = wait_ns;
  if (a.c.D == 128) return a.softcap > 0.f ? launch_weights_t<128, true>(tq, tk, p, sms, stream) : launch_weights_t<128, false>(tq, tk, p, sms, stream);
  return a.softcap > 0.f ? launch_weights_t<64, true>(tq, tk, p, sms, stream) : launch_weights_t<64, false>(tq, tk, p, sms, stream);
}

}  // namespace attn25
