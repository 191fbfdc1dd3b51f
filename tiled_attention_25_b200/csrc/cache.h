// Argument blocks and launchers of the KV-cache kernels.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cache_index.h"
#include "launch.h"

namespace attn25 {

constexpr int kErrIndex = -8;

// Raise a kernel's dynamic shared memory limit, and check the registers it
// launches with, once per device (`done`: one bit a device, one word a kernel).
template <class K>
cudaError_t prepare_kernel(std::atomic<uint64_t>& done, K kernel, int smem, int min_regs) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  cudaFuncAttributes attr;
  e = cudaFuncGetAttributes(&attr, kernel);
  if (e != cudaSuccess) return e;
  if (attr.numRegs < min_regs) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

struct CacheDev {
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  Strides k_st, v_st;  // page, head, row
  CacheIndex ix;
  int D;
  int* status;
};

struct AppendArgs {
  CacheDev c;
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  Strides kn_st, vn_st;
  const int32_t* path;
  const int32_t* counts;
  const int32_t* seen;
  int32_t* positions;
  int32_t* lens_out;
  bool late;  // lens_out is one of the arrays read here: written by a launch of its own
  int T;
};

struct TreeArgs {
  CacheDev c;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k_new;  // nullptr: the cache alone
  const __nv_bfloat16* v_new;
  Strides q_st, kn_st, vn_st, o_st;
  __nv_bfloat16* out;
  float* lse;  // or nullptr
  const int32_t* parents;
  const int32_t* counts;
  int Hq, G, T;
  float scale, softcap;  // softcap 0: none
};

struct WeightsArgs {
  CacheDev c;
  const __nv_bfloat16* q;
  Strides q_st;
  const float* lse;
  const float* w_in;
  float* w_out;
  const int32_t* path;
  const int32_t* counts;
  int Hq, G, T;
  float scale, softcap;
};

struct PlanArgs {
  CacheIndex ix;
  const float* weights;
  const int32_t* positions;
  const int32_t* seen;
  int32_t* moves;
  int32_t* n_moves;
  int budget, first, recent;
  int* status;
  // set by the launcher: ranks of a CTA's share that fit shared memory; weights and positions on 16 bytes
  int held_keys;
  bool aligned;
};

struct CompactArgs {
  CacheDev c;
  const int32_t* moves;
  const int32_t* n_moves;
  float* weights;
  int32_t* positions;
  int32_t* lens;
  int budget;
};

cudaError_t launch_cache_append(const AppendArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_cache_compact(const CompactArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_evict_plan(const PlanArgs& a, int sms, cudaStream_t stream);
// TMA maps of a tree call: q as (D, head, token, row) with boxes of one query
// tile; the pools as (D, row of the page, head, page) with boxes of
// min(page_size, 128) rows; k_new and v_new as (D, token, head, row) with
// boxes of 128 tokens.
struct TreeMaps {
  CUtensorMap q, k, v, kn, vn;
};
size_t tree_workspace_bytes(int G, int T, int D);
cudaError_t launch_tree(const TreeMaps& m, const TreeArgs& a, void* workspace, uint64_t wait_ns, cudaStream_t stream);
// tq, tk: maps as in TreeMaps
cudaError_t launch_cache_weights(const CUtensorMap& tq, const CUtensorMap& tk, const WeightsArgs& a, uint64_t wait_ns, int sms,
                                 cudaStream_t stream);

}  // namespace attn25
