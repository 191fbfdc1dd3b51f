// KV-cache maintenance: append new rows, plan an eviction, carry its moves out.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cache.h"

namespace attn25 {

namespace {

__device__ __forceinline__ void flag_index(int* status) { atomicCAS(status, 0, kErrIndex); }

// ------------------------------------------------------------------ append
//
// A copy: every new row is read once and written once, 16 bytes a thread.
// Thread order within a block: 16-byte chunk of the row, K or V, row.
constexpr int kCopyThreads = 256;

template <int D>
__global__ void __launch_bounds__(kCopyThreads) append_kernel(const AppendArgs a) {
  constexpr int kChunks = D / 8;                              // 16-byte chunks of a row
  constexpr int kRows = kCopyThreads / (2 * kChunks);         // rows of a block's pass
  const int b = blockIdx.z, hk = blockIdx.y;
  bool bad = false;
  const int n = a.counts != nullptr ? clamp_count(a.counts[b], a.T, bad) : a.T;
  const int len = clamp_count(a.c.ix.lens[b], a.c.ix.capacity, bad);
  const int chunk = threadIdx.x % kChunks, is_v = threadIdx.x / kChunks % 2, r = threadIdx.x / (2 * kChunks);
  for (int i = blockIdx.x * kRows + r; i < n; i += gridDim.x * kRows) {
    const int slot = len + i, node = a.path != nullptr ? a.path[static_cast<long long>(b) * a.T + i] : i;
    if (slot >= a.c.ix.capacity || node < 0 || node >= a.T) {
      bad = true;
      continue;
    }
    if (a.positions != nullptr && chunk == 0 && is_v == 0)
      a.positions[slot_entry(a.c.ix, b, hk, slot)] = (a.seen != nullptr ? a.seen[b] : len) + i;
    const int page = page_at(a.c.ix, b, slot / a.c.ix.page_size), row = slot % a.c.ix.page_size;
    if (page < 0) {
      bad = true;
      continue;
    }
    const Strides& from = is_v ? a.vn_st : a.kn_st;
    const Strides& to = is_v ? a.c.v_st : a.c.k_st;
    const __nv_bfloat16* src = (is_v ? a.v_new : a.k_new) + b * from.b + hk * from.h + node * from.s + chunk * 8;
    __nv_bfloat16* dst = (is_v ? a.c.v : a.c.k) + page * to.b + hk * to.h + row * to.s + chunk * 8;
    *reinterpret_cast<uint4*>(dst) = __ldg(reinterpret_cast<const uint4*>(src));
  }
  if (a.lens_out != nullptr && blockIdx.x == 0 && hk == 0 && threadIdx.x == 0)
    a.lens_out[b] = min(len + n, a.c.ix.capacity);
  if (bad) flag_index(a.c.status);
}

// The in-place advance of lens, after every block of append_kernel has read them.
__global__ void advance_kernel(const AppendArgs a) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= a.c.ix.B) return;
  bool bad = false;
  const int n = a.counts != nullptr ? clamp_count(a.counts[b], a.T, bad) : a.T;
  const int len = clamp_count(a.lens[b], a.c.ix.capacity, bad);
  a.lens[b] = min(len + n, a.c.ix.capacity);
}

// ------------------------------------------------------------------ compact

template <int D>
__global__ void __launch_bounds__(kCopyThreads) compact_kernel(const CompactArgs a) {
  constexpr int kChunks = D / 8;
  constexpr int kRows = kCopyThreads / (2 * kChunks);
  const int b = blockIdx.y / a.c.ix.Hkv, hk = blockIdx.y % a.c.ix.Hkv;
  bool bad = false;
  const int n = clamp_count(a.n_moves[blockIdx.y], a.budget, bad);
  const int chunk = threadIdx.x % kChunks, is_v = threadIdx.x / kChunks % 2, r = threadIdx.x / (2 * kChunks);
  const int ps = a.c.ix.page_size;
  for (int i = blockIdx.x * kRows + r; i < n; i += gridDim.x * kRows) {
    const int2 mv = reinterpret_cast<const int2*>(a.moves)[static_cast<long long>(blockIdx.y) * a.budget + i];
    if (mv.x < 0 || mv.x >= a.c.ix.capacity || mv.y < 0 || mv.y >= a.c.ix.capacity) {
      bad = true;
      continue;
    }
    if (chunk == 0 && is_v == 0 && a.weights != nullptr)
      a.weights[slot_entry(a.c.ix, b, hk, mv.x)] = a.weights[slot_entry(a.c.ix, b, hk, mv.y)];
    if (chunk == 0 && is_v == 1 && a.positions != nullptr)
      a.positions[slot_entry(a.c.ix, b, hk, mv.x)] = a.positions[slot_entry(a.c.ix, b, hk, mv.y)];
    const int pt = page_at(a.c.ix, b, mv.x / ps), pf = page_at(a.c.ix, b, mv.y / ps);
    if (pt < 0 || pf < 0) {
      bad = true;
      continue;
    }
    const Strides& st = is_v ? a.c.v_st : a.c.k_st;
    __nv_bfloat16* base = (is_v ? a.c.v : a.c.k) + hk * st.h + chunk * 8;
    *reinterpret_cast<uint4*>(base + pt * st.b + mv.x % ps * st.s) =
        *reinterpret_cast<const uint4*>(base + pf * st.b + mv.y % ps * st.s);
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

constexpr int kPlanThreads = 1024;

// Exclusive prefix sum over the block of one count a thread; total in `sum`.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int& sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int before = 0;
  sum = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    sum += warp_sums[w];
  }
  __syncthreads();
  return before + inc - x;
}

// One block per (row, head): a radix select of the budget-th largest rank (8
// bits a pass), then one pass in slot order that hands the holes below the
// budget and the kept slots above it their places in the move list.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
  const int bh = blockIdx.x, b = bh / a.ix.Hkv;
  bool bad = false;
  const int n = clamp_count(a.ix.lens[b], a.ix.capacity, bad);
  if (bad && threadIdx.x == 0) flag_index(a.status);
  int2* moves = reinterpret_cast<int2*>(a.moves) + static_cast<long long>(bh) * a.budget;
  __shared__ int hist[256];
  __shared__ int sums[kPlanThreads / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  int n_moves = 0;
  if (n > a.budget) {
    const float* w = a.weights + static_cast<long long>(bh) * a.ix.capacity;
    const int32_t* pos = a.positions + static_cast<long long>(bh) * a.ix.capacity;
    const int recent_from = a.seen[b] - a.recent;
    uint32_t prefix = 0;
    int need = a.budget;  // slots still to take among those that share the prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += kPlanThreads) hist[i] = 0;
      __syncthreads();
      for (int j = threadIdx.x; j < n; j += kPlanThreads) {
        const uint32_t k = slot_rank(w[j], pos[j], a.first, recent_from);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        int left = need, d = 255;
        while (d > 0 && hist[d] < left) left -= hist[d--];
        s_prefix = prefix | (static_cast<uint32_t>(d) << shift);
        s_need = left;
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
      __syncthreads();
    }
    // slots of rank above `prefix` stay, and the first `need` of equal rank
    int ties = 0, holes = 0, extras = 0;
    for (int j0 = 0; j0 < n; j0 += kPlanThreads) {
      const int j = j0 + threadIdx.x;
      const uint32_t k = j < n ? slot_rank(w[j], pos[j], a.first, recent_from) : 0;
      const int tie = j < n && k == prefix;
      int sum;
      const int t = ties + block_scan(tie, sums, sum);
      ties += sum;
      const bool keep = j < n && (k > prefix || (tie && t < need));
      const int hole = j < min(n, a.budget) && !keep, extra = keep && j >= a.budget;
      // a chunk may hold both sides of the budget: two scans
      const int at_h = holes + block_scan(hole, sums, sum);
      holes += sum;
      const int at_e = extras + block_scan(extra, sums, sum);
      extras += sum;
      if (hole) moves[at_h].x = j;
      if (extra) moves[at_e].y = j;
    }
    n_moves = holes;
  }
  for (int i = n_moves + threadIdx.x; i < a.budget; i += kPlanThreads) moves[i] = make_int2(-1, -1);
  if (threadIdx.x == 0) a.n_moves[bh] = n_moves;
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, int sms, cudaStream_t stream) {
  const int rows = kCopyThreads / (2 * a.c.D / 8);
  const long long heads = static_cast<long long>(a.c.ix.B) * a.c.ix.Hkv;
  const long long most = (a.T + rows - 1) / rows, want = (8LL * sms + heads - 1) / heads;
  const dim3 grid(static_cast<unsigned>(most < want ? most : want), a.c.ix.Hkv, a.c.ix.B);
  if (a.c.D == 128) append_kernel<128><<<grid, kCopyThreads, 0, stream>>>(a);
  else append_kernel<64><<<grid, kCopyThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.lens_out != nullptr) return e;
  advance_kernel<<<(a.c.ix.B + 255) / 256, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CompactArgs& a, int sms, cudaStream_t stream) {
  const int rows = kCopyThreads / (2 * a.c.D / 8);
  const int heads = a.c.ix.B * a.c.ix.Hkv;
  const int most = (a.budget + rows - 1) / rows, want = (8 * sms + heads - 1) / heads;
  const dim3 grid(most < want ? most : want, heads);
  if (a.c.D == 128) compact_kernel<128><<<grid, kCopyThreads, 0, stream>>>(a);
  else compact_kernel<64><<<grid, kCopyThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_evict_plan(const PlanArgs& a, cudaStream_t stream) {
  plan_kernel<<<a.ix.B * a.ix.Hkv, kPlanThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace attn25
