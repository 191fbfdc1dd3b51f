// KV-cache maintenance: append new rows, plan an eviction, carry its moves out.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "cache.h"

namespace attn25 {

namespace {

__device__ __forceinline__ void flag_index(int* status) { atomicCAS(status, 0, kErrIndex); }

// ------------------------------------------------------------------ row copies
//
// Append and compaction are copies of K and V rows, read once and written
// once, bound by HBM.  A row's place is two dependent lookups away (its token
// or move, then the page table), so a block first resolves the element offsets
// of a batch of rows, one thread to a row, into shared memory, and then
// streams the batch with eight 16-byte loads of a thread in flight.  (With the
// lookups in every copying thread the halving of 16 x 8 heads of 8192 slots
// took 94 to 109 us.)
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;

template <int D>
struct CopyBatch {
  static constexpr int kChunks = D / 8;                                    // 16-byte chunks of a row
  static constexpr int kRows = kCopyThreads * kCopyUnroll / (2 * kChunks);  // rows of a batch
  long long src[2][kRows], dst[2][kRows];  // elements, K and V; src < 0: no copy
};

// Executed by the block after a __syncthreads.  Thread order: chunk, K or V, row.
template <int D>
__device__ __forceinline__ void copy_rows(const CopyBatch<D>& t, const __nv_bfloat16* src_k, const __nv_bfloat16* src_v,
                                          __nv_bfloat16* dst_k, __nv_bfloat16* dst_v) {
  using T = CopyBatch<D>;
  constexpr int kStep = kCopyThreads / (2 * T::kChunks);
  const int chunk = threadIdx.x % T::kChunks, is_v = threadIdx.x / T::kChunks % 2, r = threadIdx.x / (2 * T::kChunks);
  const __nv_bfloat16* src = (is_v ? src_v : src_k) + chunk * 8;
  __nv_bfloat16* dst = (is_v ? dst_v : dst_k) + chunk * 8;
  uint4 v[kCopyUnroll];
#pragma unroll
  for (int x = 0; x < kCopyUnroll; ++x) {
    const long long at = t.src[is_v][r + x * kStep];
    if (at >= 0) v[x] = *reinterpret_cast<const uint4*>(src + at);
  }
#pragma unroll
  for (int x = 0; x < kCopyUnroll; ++x)
    if (t.src[is_v][r + x * kStep] >= 0) *reinterpret_cast<uint4*>(dst + t.dst[is_v][r + x * kStep]) = v[x];
}

template <int D>
__global__ void __launch_bounds__(kCopyThreads) append_kernel(const AppendArgs a) {
  using T = CopyBatch<D>;
  __shared__ T t;
  const int b = blockIdx.z, hk = blockIdx.y;
  bool bad = false;
  const int n = a.counts != nullptr ? clamp_count(a.counts[b], a.T, bad) : a.T;
  const int len = clamp_count(a.c.ix.lens[b], a.c.ix.capacity, bad);
  const int ps = a.c.ix.page_size;
  for (int i0 = blockIdx.x * T::kRows; i0 < n; i0 += gridDim.x * T::kRows) {
    if (threadIdx.x < T::kRows) {
      const int i = i0 + threadIdx.x, slot = len + i;
      long long from = -1;
      if (i < n) {
        const int node = a.path != nullptr ? a.path[static_cast<long long>(b) * a.T + i] : i;
        if (slot < a.c.ix.capacity && node >= 0 && node < a.T) {
          if (a.positions != nullptr)
            a.positions[slot_entry(a.c.ix, b, hk, slot)] = (a.seen != nullptr ? a.seen[b] : len) + i;
          const int page = page_at(a.c.ix, b, slot / ps), row = slot % ps;
          if (page >= 0) {
            from = node;
            t.dst[0][threadIdx.x] = page * a.c.k_st.b + row * a.c.k_st.s;
            t.dst[1][threadIdx.x] = page * a.c.v_st.b + row * a.c.v_st.s;
          }
        }
        bad = bad || from < 0;
      }
      t.src[0][threadIdx.x] = from < 0 ? -1 : from * a.kn_st.s;
      t.src[1][threadIdx.x] = from < 0 ? -1 : from * a.vn_st.s;
    }
    __syncthreads();
    copy_rows<D>(t, a.k_new + b * a.kn_st.b + hk * a.kn_st.h, a.v_new + b * a.vn_st.b + hk * a.vn_st.h, a.c.k + hk * a.c.k_st.h,
                 a.c.v + hk * a.c.v_st.h);
    __syncthreads();
  }
  if (!a.late && blockIdx.x == 0 && hk == 0 && threadIdx.x == 0)
    a.lens_out[b] = min(len + n, a.c.ix.capacity);
  if (bad) flag_index(a.c.status);
}

// The new lengths where they replace an array that the blocks of append_kernel
// read, after all of them.
__global__ void advance_kernel(const AppendArgs a) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= a.c.ix.B) return;
  bool bad = false;
  const int n = a.counts != nullptr ? clamp_count(a.counts[b], a.T, bad) : a.T;
  const int len = clamp_count(a.c.ix.lens[b], a.c.ix.capacity, bad);
  a.lens_out[b] = min(len + n, a.c.ix.capacity);
}

template <int D>
__global__ void __launch_bounds__(kCopyThreads) compact_kernel(const CompactArgs a) {
  using T = CopyBatch<D>;
  __shared__ T t;
  const int b = blockIdx.y / a.c.ix.Hkv, hk = blockIdx.y % a.c.ix.Hkv;
  bool bad = false;
  const int n = clamp_count(a.n_moves[blockIdx.y], a.budget, bad);
  const int ps = a.c.ix.page_size;
  const int2* moves = reinterpret_cast<const int2*>(a.moves) + static_cast<long long>(blockIdx.y) * a.budget;
  for (int i0 = blockIdx.x * T::kRows; i0 < n; i0 += gridDim.x * T::kRows) {
    if (threadIdx.x < T::kRows) {
      const int i = i0 + threadIdx.x;
      bool moved = false;
      if (i < n) {
        const int2 mv = moves[i];
        if (mv.x >= 0 && mv.x < a.c.ix.capacity && mv.y >= 0 && mv.y < a.c.ix.capacity) {
          const long long to = slot_entry(a.c.ix, b, hk, mv.x), from = slot_entry(a.c.ix, b, hk, mv.y);
          const float weight = a.weights != nullptr ? a.weights[from] : 0.f;
          const int32_t position = a.positions != nullptr ? a.positions[from] : 0;
          const int pt = page_at(a.c.ix, b, mv.x / ps), pf = page_at(a.c.ix, b, mv.y / ps);
          if (pt >= 0 && pf >= 0) {  // weight and position go with the row, or stay with it
            if (a.weights != nullptr) a.weights[to] = weight;
            if (a.positions != nullptr) a.positions[to] = position;
            moved = true;
            t.dst[0][threadIdx.x] = pt * a.c.k_st.b + mv.x % ps * a.c.k_st.s;
            t.dst[1][threadIdx.x] = pt * a.c.v_st.b + mv.x % ps * a.c.v_st.s;
            t.src[0][threadIdx.x] = pf * a.c.k_st.b + mv.y % ps * a.c.k_st.s;
            t.src[1][threadIdx.x] = pf * a.c.v_st.b + mv.y % ps * a.c.v_st.s;
          }
        }
        bad = bad || !moved;
      }
      if (!moved) t.src[0][threadIdx.x] = t.src[1][threadIdx.x] = -1;
    }
    __syncthreads();
    copy_rows<D>(t, a.c.k + hk * a.c.k_st.h, a.c.v + hk * a.c.v_st.h, a.c.k + hk * a.c.k_st.h, a.c.v + hk * a.c.v_st.h);
    __syncthreads();
  }
  if (blockIdx.x == 0 && hk == 0 && threadIdx.x == 0) a.lens[b] = min(clamp_count(a.lens[b], a.c.ix.capacity, bad), a.budget);
  if (bad) flag_index(a.c.status);
}

// ------------------------------------------------------------------ eviction plan
//
// The order of a slot's value: protected slots first, then larger weights
// (as the unsigned order of the float bits), NaN last.
__device__ __forceinline__ uint32_t slot_rank(float w, int pos, int first, int recent_from) {
  if (pos < first || pos >= recent_from) return 0xffffffffu;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One cluster of 1 to 8 CTAs per (row, head), each with an equal share of the
// slots, whose ranks it keeps in shared memory (read again from global where
// they do not fit).  A radix select finds the budget-th largest rank in at
// most three passes of 11, 11 and 10 bits; every CTA adds its filled bins to the
// histograms of the whole cluster (reductions into distributed shared memory,
// which nothing waits for until the cluster's barrier; reading the others' bins
// instead took 10 us a pass) and takes the same decision.  Then
// each warp walks its part in slot order: ranks of equal ones, kept slots, and
// the places of the holes and of the rows that fill them, from prefix counts
// over the lanes, the warps and the CTAs.  A walk's cost is its latency, so a
// lane takes four neighbouring slots at a time (one 16-byte access): halving 32
// heads of up to 65000 slots took 34 us with one slot to a lane.
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kBins = 2048;

struct alignas(16) PlanShared {
  int hist[kBins];      // this CTA's, of the current pass
  int total[3][kBins];  // the cluster's, of each pass
  int warp_sum[kPlanWarps];
  int tie_warp[kPlanWarps], hole_warp[kPlanWarps], extra_warp[kPlanWarps];
  int ties, holes, extras;  // of this CTA, read by the cluster
  uint32_t digit;
  int need, in_bin;
};
// the longest row's flags fit beside the counters
static_assert(sizeof(PlanShared) + kMaxCapacity / kPlanMaxCtas / 4 <= kPlanSmem, "flags of a share");

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// The word at `p` of the same shared layout in CTA `rank` of the cluster.
__device__ __forceinline__ int ld_cluster(const int* p, uint32_t rank) {
  int v;
  asm volatile(
      "{\n\t.reg .u32 r;\n\t"
      "mapa.shared::cluster.u32 r, %1, %2;\n\t"
      "ld.shared::cluster.s32 %0, [r];\n\t}"
      : "=r"(v)
      : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank)
      : "memory");
  return v;
}

__device__ __forceinline__ void add_cluster(int* p, int v, uint32_t rank) {
  asm volatile(
      "{\n\t.reg .u32 r;\n\t"
      "mapa.shared::cluster.u32 r, %0, %1;\n\t"
      "red.relaxed.cluster.shared::cluster.add.s32 [r], %2;\n\t}" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))),
      "r"(rank), "r"(v)
      : "memory");
}

// Sum of the counts of the warps before this one.
__device__ __forceinline__ int warps_before(const int* counts) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = lane < warp && lane < kPlanWarps ? counts[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ int warp_total(int x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Sum of the counts of the CTAs before this one, and of all: a lane to a CTA.
__device__ __forceinline__ int ctas_before(const int* count, int& all) {
  const uint32_t lane = threadIdx.x & 31;
  const int v = lane < cluster_size() ? ld_cluster(count, lane) : 0;
  all = warp_total(v);
  return warp_total(lane < cluster_rank() ? v : 0);
}

// Sum of a count of 0 to 4 over the lanes before this one, and over the warp.
__device__ __forceinline__ int lanes_before(int x, int& all) {
  const uint32_t lt = (1u << (threadIdx.x & 31)) - 1u;
  int before = 0;
  all = 0;
#pragma unroll
  for (int bit = 0; bit < 3; ++bit) {
    const uint32_t v = __ballot_sync(0xffffffffu, (x >> bit) & 1);
    before += __popc(v & lt) << bit;
    all += __popc(v) << bit;
  }
  return before;
}

// Which of quad q's slots, counted from j0, lie below `end`.
__device__ __forceinline__ uint32_t quad_below(int end, int j0, int q) {
  const int left = end - j0 - 4 * q;
  return left <= 0 ? 0u : (left >= 4 ? 15u : (1u << left) - 1u);
}

__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(const PlanArgs a) {
  extern __shared__ __align__(16) uint8_t plan_smem[];
  PlanShared& sh = *reinterpret_cast<PlanShared*>(plan_smem);
  uint4* keys = reinterpret_cast<uint4*>(plan_smem + sizeof(PlanShared));  // ranks of the share
  uint8_t* kept = plan_smem + sizeof(PlanShared) + a.held_keys * 4;        // its kept slots, four to a byte
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ctas = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int bh = blockIdx.x / ctas, b = bh / a.ix.Hkv;
  bool bad = false;
  const int n = clamp_count(a.ix.lens[b], a.ix.capacity, bad);
  if (bad && threadIdx.x == 0) flag_index(a.status);
  int2* moves = reinterpret_cast<int2*>(a.moves) + static_cast<long long>(bh) * a.budget;
  int n_moves = 0;
  if (n > a.budget) {  // the same for the whole cluster
    const float* w = a.weights + static_cast<long long>(bh) * a.ix.capacity;
    const int32_t* pos = a.positions + static_cast<long long>(bh) * a.ix.capacity;
    const int recent_from = static_cast<int>(max(static_cast<long long>(a.seen[b]) - a.recent, static_cast<long long>(INT_MIN)));
    // this CTA's slots [j0, j0 + m) in quads of four
    const int share = plan_share(n, ctas);
    const int j0 = min(n, rank * share), m = min(n - j0, share), quads = (m + 3) / 4;
    const bool held = share <= a.held_keys;
    auto fresh = [&](int q) {
      uint32_t k[4] = {0u, 0u, 0u, 0u};
      const int j = j0 + 4 * q;
      if (a.aligned && 4 * q + 4 <= m) {
        const float4 x = *reinterpret_cast<const float4*>(w + j);
        const int4 y = *reinterpret_cast<const int4*>(pos + j);
        k[0] = slot_rank(x.x, y.x, a.first, recent_from);
        k[1] = slot_rank(x.y, y.y, a.first, recent_from);
        k[2] = slot_rank(x.z, y.z, a.first, recent_from);
        k[3] = slot_rank(x.w, y.w, a.first, recent_from);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * q + e < m) k[e] = slot_rank(w[j + e], pos[j + e], a.first, recent_from);
      }
      return make_uint4(k[0], k[1], k[2], k[3]);
    };
    auto quad = [&](int q) { return held ? keys[q] : fresh(q); };
    // f(rank, bit of the quad) for the slots of quad q that exist
    auto each = [&](int q, const uint4& k, auto f) {
      const int left = m - 4 * q;
      if (left > 0) f(k.x, 1u);
      if (left > 1) f(k.y, 2u);
      if (left > 2) f(k.z, 4u);
      if (left > 3) f(k.w, 8u);
    };
    for (int i = threadIdx.x; i < 3 * kBins; i += kPlanThreads) (&sh.total[0][0])[i] = 0;
    for (int i = threadIdx.x; i < kBins; i += kPlanThreads) sh.hist[i] = 0;
    if (ctas > 1) cluster_sync();  // the others add to the totals
    else __syncthreads();
    uint32_t prefix = 0;     // the bits decided so far
    int need = a.budget;     // slots still to take among those that share them
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bins = pass == 2 ? 1024 : kBins;
      const int above = pass == 0 ? 32 : (pass == 1 ? 21 : 10);  // bits below the decided ones
      if (pass == 0) {
        for (int q = threadIdx.x; q < quads; q += kPlanThreads) {
          const uint4 k = fresh(q);
          if (held) keys[q] = k;
          each(q, k, [&](uint32_t x, uint32_t) { atomicAdd(&sh.hist[x >> shift], 1); });
        }
      } else {
        for (int q = threadIdx.x; q < quads; q += kPlanThreads)
          each(q, quad(q), [&](uint32_t x, uint32_t) {
            if ((x >> above) == (prefix >> above)) atomicAdd(&sh.hist[(x >> shift) & (bins - 1)], 1);
          });
      }
      __syncthreads();
      int* total = sh.hist;
      if (ctas > 1) {
        total = sh.total[pass];
        for (int i = threadIdx.x; i < bins; i += kPlanThreads) {
          const int v = sh.hist[i];
          if (v != 0) {
            sh.hist[i] = 0;
            for (int q = 0; q < ctas; ++q) add_cluster(&total[i], v, q);
          }
        }
        cluster_sync();
      }
      // the bin in which the count from the top reaches `need`: two bins to a thread, from the top
      int c[2], sum = 0;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int bin = bins - 1 - (2 * static_cast<int>(threadIdx.x) + x);
        c[x] = bin >= 0 ? total[bin] : 0;
        if (ctas == 1 && bin >= 0) total[bin] = 0;  // for the next pass
        sum += c[x];
      }
      int inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) sh.warp_sum[warp] = inc;
      __syncthreads();
      int before = warps_before(sh.warp_sum) + inc - sum;
      if (before < need && before + sum >= need) {
        const int x = before + c[0] < need ? 1 : 0;
        if (x == 1) before += c[0];
        sh.digit = bins - 1 - (2 * threadIdx.x + x);
        sh.need = need - before;
        sh.in_bin = x == 1 ? c[1] : c[0];
      }
      __syncthreads();
      prefix |= sh.digit << shift;
      need = sh.need;
      if (need == sh.in_bin) {  // the whole bin stays: what is at or above its lowest rank
        prefix -= 1;            // (something lies below, or n <= budget)
        need = 0;
        break;
      }
    }
    // slots of rank above `prefix` stay, and the first `need` (in slot order) of equal rank
    const int per = (quads + kPlanWarps * 32 - 1) / (kPlanWarps * 32) * 32;  // quads of a warp
    const int q0 = min(quads, warp * per), q1 = min(quads, q0 + per);
    int t = 0;
    if (need > 0)
      for (int q = q0 + lane; q < q1; q += 32) each(q, quad(q), [&](uint32_t k, uint32_t) { t += k == prefix; });
    t = warp_total(t);
    if (lane == 0) sh.tie_warp[warp] = t;
    __syncthreads();
    if (warp == 0) {
      const int v = warp_total(sh.tie_warp[lane]);
      if (lane == 0) sh.ties = v;
    }
    if (ctas > 1) cluster_sync();
    else __syncthreads();
    int all;
    int tie = ctas_before(&sh.ties, all) + warps_before(sh.tie_warp);
    int holes = 0, extras = 0;  // of this lane
    for (int qb = q0; qb < q1; qb += 32) {
      const int q = qb + lane;
      uint32_t keep = 0, eq = 0;
      if (q < q1)
        each(q, quad(q), [&](uint32_t k, uint32_t bit) {
          if (k > prefix) keep |= bit;
          if (need > 0 && k == prefix) eq |= bit;
        });
      if (need > 0) {  // the first of equal rank, in slot order
        int here = 0, rank_of = tie + lanes_before(__popc(eq), here);
        tie += here;
#pragma unroll
        for (uint32_t bit = 1; bit < 16; bit <<= 1)
          if (eq & bit) {
            if (rank_of < need) keep |= bit;
            ++rank_of;
          }
      }
      if (q < q1) {
        kept[q] = static_cast<uint8_t>(keep);
        const uint32_t low = quad_below(a.budget, j0, q), there = quad_below(m, 0, q);
        holes += __popc(low & there & ~keep);
        extras += __popc(keep & ~low);
      }
    }
    const int warp_holes = warp_total(holes), warp_extras = warp_total(extras);
    if (lane == 0) {
      sh.hole_warp[warp] = warp_holes;
      sh.extra_warp[warp] = warp_extras;
    }
    __syncthreads();
    if (warp == 0) {
      const int h = warp_total(sh.hole_warp[lane]), e = warp_total(sh.extra_warp[lane]);
      if (lane == 0) {
        sh.holes = h;
        sh.extras = e;
      }
    }
    if (ctas > 1) cluster_sync();
    else __syncthreads();
    int at_h = ctas_before(&sh.holes, n_moves) + warps_before(sh.hole_warp);
    int at_e = ctas_before(&sh.extras, all) + warps_before(sh.extra_warp);
    for (int qb = q0; qb < q1; qb += 32) {
      const int q = qb + lane, j = j0 + 4 * q;
      uint32_t hole = 0, extra = 0;
      if (q < q1) {
        const uint32_t keep = kept[q], low = quad_below(a.budget, j0, q);
        hole = low & quad_below(m, 0, q) & ~keep;
        extra = keep & ~low;
      }
      int here_h = 0, here_e = 0;
      int to = at_h + lanes_before(__popc(hole), here_h), from = at_e + lanes_before(__popc(extra), here_e);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if ((hole >> e) & 1u) moves[to++].x = j + e;
        if ((extra >> e) & 1u) moves[from++].y = j + e;
      }
      at_h += here_h;
      at_e += here_e;
    }
    if (ctas > 1) cluster_sync();  // the others may still read this CTA's counts
  }
  for (int i = n_moves + rank * kPlanThreads + threadIdx.x; i < a.budget; i += ctas * kPlanThreads) moves[i] = make_int2(-1, -1);
  if (rank == 0 && threadIdx.x == 0) a.n_moves[bh] = n_moves;
}

}  // namespace

// Blocks to a head: enough for eight to an SM over all heads, each with a batch at least.
static int copy_blocks(int rows, int batch, long long heads, int sms) {
  const long long most = (static_cast<long long>(rows) + batch - 1) / batch, want = (8LL * sms + heads - 1) / heads;
  return static_cast<int>(most < want ? most : want);
}

cudaError_t launch_cache_append(const AppendArgs& a, int sms, cudaStream_t stream) {
  const int batch = a.c.D == 128 ? CopyBatch<128>::kRows : CopyBatch<64>::kRows;
  const dim3 grid(copy_blocks(a.T, batch, static_cast<long long>(a.c.ix.B) * a.c.ix.Hkv, sms), a.c.ix.Hkv, a.c.ix.B);
  if (a.c.D == 128) append_kernel<128><<<grid, kCopyThreads, 0, stream>>>(a);
  else append_kernel<64><<<grid, kCopyThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.late) return e;
  advance_kernel<<<(a.c.ix.B + 255) / 256, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CompactArgs& a, int sms, cudaStream_t stream) {
  const int batch = a.c.D == 128 ? CopyBatch<128>::kRows : CopyBatch<64>::kRows, heads = a.c.ix.B * a.c.ix.Hkv;
  const dim3 grid(copy_blocks(a.budget, batch, heads, sms), heads);
  if (a.c.D == 128) compact_kernel<128><<<grid, kCopyThreads, 0, stream>>>(a);
  else compact_kernel<64><<<grid, kCopyThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_evict_plan(const PlanArgs& args, int sms, cudaStream_t stream) {
  PlanArgs a = args;
  const int heads = a.ix.B * a.ix.Hkv;
  // a row shorter than the capacity has a smaller share
  const PlanLayout lay = plan_layout(heads, a.ix.capacity, sms, static_cast<int>(sizeof(PlanShared)));
  a.held_keys = lay.held;
  a.aligned = ((reinterpret_cast<uintptr_t>(a.weights) | reinterpret_cast<uintptr_t>(a.positions)) & 15u) == 0;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = prepare_kernel(done, plan_kernel, kPlanSmem, 0);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(heads * lay.ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = lay.bytes;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = lay.ctas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_kernel, a);
}

}  // namespace attn25
