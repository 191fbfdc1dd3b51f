// The attention weights the slots of a paged KV cache receive: a direct form,
// one block per 128 slots.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cache.h"
#include "sm100.cuh"

namespace attn25 {

namespace {

__device__ __forceinline__ void flag_index(int* status) { atomicCAS(status, 0, kErrIndex); }

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

cudaError_t launch_cache_weights(const WeightsArgs& a, cudaStream_t stream) {
  const dim3 grid((a.c.ix.capacity + 127) / 128, a.c.ix.Hkv, a.c.ix.B);
  if (a.c.D == 128) weights_slot_kernel<128><<<grid, 128, 0, stream>>>(a);
  else weights_slot_kernel<64><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace attn25
