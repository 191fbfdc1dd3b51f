// Host-side helpers shared by the C entry points: the per-device record,
// argument checks and TMA descriptor encoding (defined in api.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "attn25.h"
#include "launch.h"

namespace attn25 {

struct DeviceInfo {
  bool ready = false;
  bool usable = false;
  int sms = 0;
  int* status = nullptr;
  unsigned long long* trace = nullptr;
  void* scratch = nullptr;  // device address of attn_bwd_noalloc's block (nullptr if unavailable)
};

// The current device's record; ATTN_ERR_DEVICE if it cannot run the kernels.
int current_device(DeviceInfo** out);

// A [B][H][S][D] bf16 tensor whose D elements are contiguous, as the 4-D map
// (D, S, H, B) with the tensor's own strides; boxes of 64 x box_rows x 1 x 1.
bool encode_bf16_4d(CUtensorMap* m, const void* base, int D, int S, int H, int B, const Strides& st, int box_rows);

// Any 4-D bf16 view, dims and boxes innermost first, dim 0 contiguous, element
// strides of dims 1 to 3; 64-column boxes with the 128-byte swizzle.
bool encode_bf16_dims(CUtensorMap* m, const void* base, const long long (&dims)[4], const long long (&strides)[3],
                      int box1, int box2);

// The strides of a tensor: the caller's, or those of contiguous [B][H][S][D];
// false if a stride is not a positive multiple of 8 elements.
bool layout_of(const attn_strides* given, int H, int S, int D, Strides& st);

// A mod code split into its score transform and mask bits (composition:
// one of the seven kinds, optionally ORed with ATTN_MASK_* flags).
struct ModSpec {
  int score;      // MOD_NONE, MOD_ALIBI, MOD_SOFTCAP or MOD_BOOST
  int mask;       // kMask* bits; window and document imply causal
  int key;        // kernel specialisation key
  int canonical;  // score | ATTN_MASK_* flags: equal for codes that mean the same mod
};
bool split_mod(int code, ModSpec& m);

uint64_t wait_ns();  // the per-wait limit of the kernels

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline int cdiv(int a, int b) { return (a + b - 1) / b; }
inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace attn25
