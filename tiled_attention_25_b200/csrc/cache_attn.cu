// Attention over a paged KV cache, and the weights its slots receive: direct
// forms, one block per query row (attention) or per 128 slots (weights).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cache.h"
#include "sm100.cuh"

namespace attn25 {

namespace {

__device__ __forceinline__ void flag_index(int* status) { atomicCAS(status, 0, kErrIndex); }

constexpr int kRowThreads = 128;

// lane l's D / 32 elements of a row
template <int D>
__device__ __forceinline__ void load_lane(const __nv_bfloat16* row, float (&x)[D / 32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) x[j] = __bfloat162float(row[lane * (D / 32) + j]);
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) tree_row_kernel(const TreeArgs a) {
  constexpr int V = D / 32;
  const int t = blockIdx.x % a.T, h = blockIdx.x / a.T % a.Hq, b = blockIdx.x / a.T / a.Hq, hk = h / a.G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool bad = false;
  const int n_new = a.counts != nullptr ? clamp_count(a.counts[b], a.T, bad) : a.T;
  const int len = clamp_count(a.c.ix.lens[b], a.c.ix.capacity, bad);
  __shared__ uint32_t above[kMaxTreeTokens / 32];
  __shared__ float sm[4], sl[4], so[4][D];
  for (int i = threadIdx.x; i < kMaxTreeTokens / 32; i += kRowThreads) above[i] = 0;
  __syncthreads();
  if (threadIdx.x == 0 && t < n_new && a.k_new != nullptr) {
    for (int x = t; x >= 0;) {
      above[x >> 5] |= 1u << (x & 31);
      int up = a.parents != nullptr ? a.parents[static_cast<long long>(b) * a.T + x] : x - 1;
      if (up >= x || up < -1) {
        bad = true;
        up = -1;
      }
      x = up;
    }
  }
  __syncthreads();
  if (t >= n_new) {
    if (bad) flag_index(a.c.status);
    return;
  }
  float q[V], o[V] = {}, m = -INFINITY, l = 0.f;
  load_lane<D>(a.q + b * a.q_st.b + h * a.q_st.h + t * a.q_st.s, q);
  const int total = len + (a.k_new != nullptr ? n_new : 0);
  for (int j = warp; j < total; j += 4) {
    float k[V] = {}, v[V] = {};
    if (j < len) {
      const int page = page_at(a.c.ix, b, j / a.c.ix.page_size), row = j % a.c.ix.page_size;
      if (page >= 0) {
        load_lane<D>(a.c.k + page * a.c.k_st.b + hk * a.c.k_st.h + row * a.c.k_st.s, k);
        load_lane<D>(a.c.v + page * a.c.v_st.b + hk * a.c.v_st.h + row * a.c.v_st.s, v);
      } else {
        bad = true;
      }
    } else {
      const int x = j - len;
      if (!((above[x >> 5] >> (x & 31)) & 1)) continue;
      load_lane<D>(a.k_new + b * a.kn_st.b + hk * a.kn_st.h + x * a.kn_st.s, k);
      load_lane<D>(a.v_new + b * a.vn_st.b + hk * a.vn_st.h + x * a.vn_st.s, v);
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= a.scale;
    if (a.softcap > 0.f) s = a.softcap * tanh_ex2(s / a.softcap);
    const float m2 = fmaxf(m, s * LOG2E), f = m == -INFINITY ? 0.f : exp2f(m - m2), p = exp2f(s * LOG2E - m2);
    m = m2;
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = o[e] * f + p * v[e];
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < V; ++e) so[warp][lane * V + e] = o[e];
  __syncthreads();
  const float mx = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float f[4], lt = 0.f;
  for (int w = 0; w < 4; ++w) {
    f[w] = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - mx);
    lt += f[w] * sl[w];
  }
  for (int d = threadIdx.x; d < D; d += kRowThreads) {
    float x = 0.f;
    for (int w = 0; w < 4; ++w) x += f[w] * so[w][d];
    a.out[b * a.o_st.b + h * a.o_st.h + t * a.o_st.s + d] = __float2bfloat16(lt > 0.f ? x / lt : 0.f);
  }
  if (threadIdx.x == 0 && a.lse != nullptr)
    a.lse[(static_cast<long long>(b) * a.Hq + h) * a.T + t] = lt > 0.f ? (mx + log2f(lt)) * LN2 : -INFINITY;
  if (bad) flag_index(a.c.status);
}

template <int D>
__global__ void __launch_bounds__(128) weights_slot_kernel(const WeightsArgs a) {
  const int b = blockIdx.z, hk = blockIdx.y, j = blockIdx.x * 128 + threadIdx.x;
  bool bad = false;
  const int len = clamp_count(a.c.ix.lens[b], a.c.ix.capacity, bad);
  const int n = clamp_count(a.counts != nullptr ? a.counts[b] : a.T, min(a.T, len), bad);
  if (blockIdx.x * 128 >= len) return;
  float k[D];
#pragma unroll
  for (int d = 0; d < D; ++d) k[d] = 0.f;
  if (j < len) {
    const int page = page_at(a.c.ix, b, j / a.c.ix.page_size);
    if (page >= 0) {
      const __nv_bfloat16* row = a.c.k + page * a.c.k_st.b + hk * a.c.k_st.h + j % a.c.ix.page_size * a.c.k_st.s;
#pragma unroll
      for (int d = 0; d < D; ++d) k[d] = __bfloat162float(row[d]);
    } else {
      bad = true;
    }
  }
  __shared__ float q[D];
  float sum = 0.f;
  const int i0 = max(0, static_cast<int>(blockIdx.x) * 128 - (len - n));
  for (int i = i0; i < n; ++i) {
    const int node = a.path != nullptr ? a.path[static_cast<long long>(b) * a.T + i] : i;
    if (node < 0 || node >= a.T) {
      bad = true;
      continue;
    }
    for (int h = hk * a.G; h < (hk + 1) * a.G; ++h) {
      __syncthreads();
      for (int d = threadIdx.x; d < D; d += 128)
        q[d] = __bfloat162float(a.q[b * a.q_st.b + h * a.q_st.h + node * a.q_st.s + d]);
      __syncthreads();
      const float lse = a.lse[(static_cast<long long>(b) * a.Hq + h) * a.T + node];
      float s = 0.f;
#pragma unroll
      for (int d = 0; d < D; ++d) s = fmaf(q[d], k[d], s);
      s *= a.scale;
      if (a.softcap > 0.f) s = a.softcap * tanh_ex2(s / a.softcap);
      if (j <= len - n + i) sum += exp2f((s - lse) * LOG2E);
    }
  }
  if (j < len) {
    const long long at = slot_entry(a.c.ix, b, hk, j);
    a.w_out[at] = (a.w_in != nullptr && j < len - n ? a.w_in[at] : 0.f) + sum;
  }
  if (bad) flag_index(a.c.status);
}

}  // namespace

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream) {
  const unsigned blocks = static_cast<unsigned>(a.c.ix.B) * a.Hq * a.T;
  if (a.c.D == 128) tree_row_kernel<128><<<blocks, kRowThreads, 0, stream>>>(a);
  else tree_row_kernel<64><<<blocks, kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_weights(const WeightsArgs& a, cudaStream_t stream) {
  const dim3 grid((a.c.ix.capacity + 127) / 128, a.c.ix.Hkv, a.c.ix.B);
  if (a.c.D == 128) weights_slot_kernel<128><<<grid, 128, 0, stream>>>(a);
  else weights_slot_kernel<64><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace attn25
