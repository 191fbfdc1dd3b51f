// Hand-written inline-PTX primitives for sm_100a: mbarriers with bounded
// waits, TMA tensor copies, and the tcgen05 tensor-memory / MMA instructions.
// Written from the PTX ISA description of these instructions.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "exp2_poly.h"

namespace attn25 {

// ------------------------------------------------------------------ status

constexpr int kErrTimeout = -6;

// Profiling builds (-DATTN25_TRACE) time selected waits and phases per warp
// role with clock64 and add the totals into a device trace buffer; in normal
// builds the macro is the bare expression and the counters compile away.
#if defined(ATTN25_TRACE)
#define ATTN25_TIMED(acc, expr)            \
  ({                                       \
    const long long _t0 = clock64();       \
    auto _r = (expr);                      \
    (acc) += clock64() - _t0;              \
    _r;                                    \
  })
#define ATTN25_TRACE_ONLY(x) x
#else
#define ATTN25_TIMED(acc, expr) (expr)
#define ATTN25_TRACE_ONLY(x)
#endif

// Trace buffer of profiling builds: 256 per-role counters (word 255 holds the
// first step of the event window), then the event clocks of a window of
// backward steps on CTA 0 (kEvSteps x kEvPerStep).
constexpr int kTraceCounters = 256;
constexpr int kEvSteps = 32, kEvPerStep = 16;
constexpr int kTraceWords = kTraceCounters + kEvSteps * kEvPerStep;

// Add one warp's counters into the trace buffer (lane 0 only).
template <int N>
__device__ __forceinline__ void trace_flush(unsigned long long* trace, int base, const long long (&tr)[N]) {
#if defined(ATTN25_TRACE)
  if (trace != nullptr && (threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) atomicAdd(trace + base + i, static_cast<unsigned long long>(tr[i]));
  }
#else
  (void)trace;
  (void)base;
  (void)tr;
#endif
}

struct WaitCtl {
  uint64_t limit_ns;     // per-wait time limit
  uint32_t abort_addr;   // shared-memory word: non-zero once any role gave up
  int* status;           // device status word (0, or the first error recorded)
};

// Limit of the waits by which a role lets its own copies and MMAs land before
// the CTA exits: those complete on their own within microseconds, so they get
// at least a second whatever limit the caller set for the other waits.
constexpr uint64_t kDrainFloorNs = 1000000000ull;
__device__ __forceinline__ uint64_t drain_limit(uint64_t limit_ns) {
  return limit_ns > kDrainFloorNs ? limit_ns : kDrainFloorNs;
}

__device__ __forceinline__ uint64_t globaltimer() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ uint32_t ld_shared_volatile(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void st_shared_volatile(uint32_t addr, uint32_t v) {
  asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void record_error(int code, WaitCtl w) {
  if (w.status != nullptr) atomicCAS(w.status, 0, code);
  st_shared_volatile(w.abort_addr, 1u);
}

__device__ __forceinline__ bool aborted(WaitCtl w) { return ld_shared_volatile(w.abort_addr) != 0u; }

// ------------------------------------------------------------------ smem / mbarrier

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Wait for the phase with the given parity, executed by ONE thread.  Returns
// false (after recording a timeout) if the limit passes or another role
// already gave up.
static __device__ __forceinline__ bool mbar_wait_thread(uint32_t bar, uint32_t parity, WaitCtl w) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (aborted(w)) return false;
    if (globaltimer() - t0 > w.limit_ns) {
      record_error(kErrTimeout, w);
      return false;
    }
  }
}

// Warp-collective wait: every lane of the (converged) warp calls it and all
// lanes get the same answer, so warp-collective instructions that follow stay
// aligned even when the wait gives up.
static __device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, WaitCtl w) {
  const uint64_t t0 = globaltimer();
  while (true) {
    const bool ok = mbar_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    bool give_up = aborted(w);
    if (!give_up && globaltimer() - t0 > w.limit_ns) {
      give_up = true;
      record_error(kErrTimeout, w);
    }
    if (__any_sync(0xffffffffu, give_up)) return false;
  }
}

// Forms with the polling loop out of line (one check inline): kernels with
// many wait sites and several distinct warp roles otherwise spend a large
// part of their instruction-cache space on polling loops that rarely run.
// ptxas cannot place these calls inside setmaxnreg register regions, so
// only kernels without a register split use them.
static __device__ __noinline__ bool mbar_wait_thread_loop(uint32_t bar, uint32_t parity, WaitCtl w) {
  return mbar_wait_thread(bar, parity, w);
}
static __device__ __noinline__ bool mbar_wait_warp_loop(uint32_t bar, uint32_t parity, WaitCtl w) {
  return mbar_wait_warp(bar, parity, w);
}
static __device__ __forceinline__ bool mbar_wait_thread_ool(uint32_t bar, uint32_t parity, WaitCtl w) {
  return mbar_try_wait(bar, parity) || mbar_wait_thread_loop(bar, parity, w);
}
static __device__ __forceinline__ bool mbar_wait_warp_ool(uint32_t bar, uint32_t parity, WaitCtl w) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || mbar_wait_warp_loop(bar, parity, w);
}

// ------------------------------------------------------------------ TMA

__device__ __forceinline__ void tma_prefetch_desc(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// 3-D tiled load global -> shared, completion counted in bytes on `bar`.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// 4-D tiled load global -> shared (coordinates innermost first).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// Make generic-proxy writes to shared memory visible to the async (TMA) proxy.
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ------------------------------------------------------------------ tcgen05

__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T-ish per descriptors; kind::f16 (bf16 in, fp32 acc).
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive once on `bar` when every tcgen05 operation this thread issued so far has completed.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

// Warp-wide forms: every lane of a converged warp calls them with the same
// operands and one lane, chosen by elect.sync, issues.  The descriptors then
// stay warp-uniform; issuing from a single-lane branch instead was measured
// at about 3x fewer MMAs per clock next to ALU-bound warps on the same SM
// sub-partition (157 vs 62 clk per 128x64x16 MMA).
__device__ __forceinline__ void mma_ss_w(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same for 8-bit floating-point operands (kind::f8f6f4: K = 32 per MMA).
__device__ __forceinline__ void mma_ss_f8_w(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void mma_ts_w(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void mma_commit_w(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

#define ATTN25_R32(a)                                                                          \
  "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]),         \
      "=r"(a[7]), "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]),  \
      "=r"(a[14]), "=r"(a[15]), "=r"(a[16]), "=r"(a[17]), "=r"(a[18]), "=r"(a[19]),            \
      "=r"(a[20]), "=r"(a[21]), "=r"(a[22]), "=r"(a[23]), "=r"(a[24]), "=r"(a[25]),            \
      "=r"(a[26]), "=r"(a[27]), "=r"(a[28]), "=r"(a[29]), "=r"(a[30]), "=r"(a[31])

#define ATTN25_W32(a)                                                                          \
  "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(a[4]), "r"(a[5]), "r"(a[6]), "r"(a[7]),     \
      "r"(a[8]), "r"(a[9]), "r"(a[10]), "r"(a[11]), "r"(a[12]), "r"(a[13]), "r"(a[14]),        \
      "r"(a[15]), "r"(a[16]), "r"(a[17]), "r"(a[18]), "r"(a[19]), "r"(a[20]), "r"(a[21]),      \
      "r"(a[22]), "r"(a[23]), "r"(a[24]), "r"(a[25]), "r"(a[26]), "r"(a[27]), "r"(a[28]),      \
      "r"(a[29]), "r"(a[30]), "r"(a[31])

// Lane l of the warp reads TMEM lane (base lane + l), 32 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : ATTN25_R32(r)
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      ATTN25_W32(r)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

// ------------------------------------------------------------------ descriptors

// Shared-memory matrix descriptor, 128-byte swizzle, Blackwell version field.
// lbo / sbo in bytes.  K-major: sbo = distance between 8-row groups, lbo unused.
// MN-major: lbo = distance between 64-element MN blocks, sbo = distance between
// 8-row K groups.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32;
  d |= 1ull << 46;  // descriptor version for tcgen05
  d |= 2ull << 61;  // SWIZZLE_128B
  return d;
}

// The same descriptor in two words.  The low one holds the address, so that
// tiles a fixed distance apart differ by a constant added to it (16-byte units;
// addresses stay below 256 KB, so the field does not overflow); the high one
// depends on sbo alone.
__device__ __forceinline__ uint32_t smem_desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr >> 4) & 0x3FFFu) | (((lbo >> 4) & 0x3FFFu) << 16);
}
__host__ __device__ constexpr uint32_t smem_desc_hi_sw128(uint32_t sbo) {
  return ((sbo >> 4) & 0x3FFFu) | (1u << 14) | (2u << 29);
}

// mma_ss_w and mma_ts_w with descriptors in two words: two additions to an MMA
// instead of two descriptors put together, which beside busy warps took as long
// as the MMA itself (130 against 64 clocks for 128x128x16).
template <uint32_t HI>
__device__ __forceinline__ void mma_ss_lo_w(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(HI)
      : "memory");
}
template <uint32_t HI>
__device__ __forceinline__ void mma_ts_lo_w(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(HI)
      : "memory");
}

// Instruction descriptor of kind::f16 with bf16 A/B and fp32 accumulation.
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N, bool a_mn_major,
                                                      bool b_mn_major) {
  return (1u << 4)                                  // D format: f32
         | (1u << 7)                                // A format: bf16
         | (1u << 10)                               // B format: bf16
         | (static_cast<uint32_t>(a_mn_major) << 15)  // A major
         | (static_cast<uint32_t>(b_mn_major) << 16)  // B major
         | (static_cast<uint32_t>(N >> 3) << 17)    // N / 8
         | (static_cast<uint32_t>(M >> 4) << 24);   // M / 16
}

// Instruction descriptor of kind::f8f6f4 with e4m3 A and B (format code 0)
// and fp32 accumulation; the other fields as in the bf16 descriptor.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4)                                  // D format: f32
         | (0u << 7)                                // A format: e4m3
         | (0u << 10)                               // B format: e4m3
         | (static_cast<uint32_t>(a_mn_major) << 15)
         | (static_cast<uint32_t>(b_mn_major) << 16)
         | (static_cast<uint32_t>(N >> 3) << 17)
         | (static_cast<uint32_t>(M >> 4) << 24);
}

// ------------------------------------------------------------------ math

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh from its exponential form, tanh(t) = (1 - e^-2t) / (1 + e^-2t) for
// t = |y| >= 0 (so that e^-2t <= 1 never overflows), with the sign restored:
// one ex2 and one reciprocal on the MUFU pipe.  With the hardware bounds of
// both approximations (relative 2^-22 and 2^-23) the absolute error is below
// 3e-7 over all y; a softcap of c = 50 turns that into 1.5e-5 in the score.
__device__ __forceinline__ float tanh_ex2(float y) {
  const float e = ex2_approx(-2.8853900817779268f * fabsf(y));  // 2^(-2 log2(e) |y|)
  return copysignf((1.f - e) * rcp_approx(1.f + e), y);
}

// tanh(u) for |u| <= 0.4 on the FMA pipe, from the Taylor series of tanh
// through the u^9 term: u (1 - u^2/3 + 2u^4/15 - 17u^6/315 + 62u^8/2835).
// The first omitted term, 1382 u^11 / 155925, is below 4e-7 at |u| = 0.4.
constexpr float kTanhSeriesLimit = 0.4f;
constexpr float kTanhS4 = 0.021869488f, kTanhS3 = -0.053968254f, kTanhS2 = 0.13333334f, kTanhS1 = -0.33333334f;

// k tanh(aux x) for a pair of scores x with |aux x| <= 0.4, on the FMA pipe in
// packed fp32 pairs: u = aux x, w = u^2, and the series' factor with every
// coefficient multiplied by k, so that k tanh(u) = u (k + k c1 w + ... + k c4 w^4).
__device__ __forceinline__ float2 tanh_series2(float2 x, float aux, float k) {
  const float2 u = __fmul2_rn(x, make_float2(aux, aux));
  const float2 w = __fmul2_rn(u, u);
  float2 p = __ffma2_rn(w, make_float2(k * kTanhS4, k * kTanhS4), make_float2(k * kTanhS3, k * kTanhS3));
  p = __ffma2_rn(p, w, make_float2(k * kTanhS2, k * kTanhS2));
  p = __ffma2_rn(p, w, make_float2(k * kTanhS1, k * kTanhS1));
  p = __ffma2_rn(p, w, make_float2(k, k));
  return __fmul2_rn(u, p);
}

// 2^x on the FMA pipe (finite x only): x = n + f with n = round(x) taken from
// the low mantissa bits of x + 1.5 * 2^23 (round-to-nearest, Cody-Waite
// style), 2^f from the minimax polynomial of exp2_poly.h, and 2^n added into
// the exponent field.  x is clamped to -126 first, so tiny results become the
// smallest normal number instead of garbage.
__device__ __forceinline__ float exp2_poly(float x) {
  x = fmaxf(x, -126.0f);
  const float t = x + 12582912.0f;
  const float n = t - 12582912.0f;
  const float f = x - n;
  float p = fmaf(kExp2C3, f, kExp2C2);
  p = fmaf(p, f, kExp2C1);
  p = fmaf(p, f, kExp2C0);
  return __int_as_float(__float_as_int(p) + (__float_as_int(t) << 23));
}

// 32-byte global store of eight words (the address must be 32-byte aligned)
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  // cvt packs its first source operand into the upper half
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ------------------------------------------------------------------ cluster launch control
//
// Ask the hardware to cancel a CTA of this grid that has not started yet, so
// that the asking CTA takes over its work.  The 16-byte response lands in
// shared memory and completes `bar` (armed by the caller with expect_tx of
// 16 bytes).  Once a response reports that nothing was cancelled, no further
// request may be made.
__device__ __forceinline__ void clc_try_cancel(uint32_t resp, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(resp),
      "r"(bar)
      : "memory");
}

// The x index of the CTA a completed response cancelled, or -1 if it cancelled none.
__device__ __forceinline__ int clc_cancelled_x(uint32_t resp) {
  uint32_t ok, x = 0;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(ok), "+r"(x)
      : "r"(resp)
      : "memory");
  return ok ? static_cast<int>(x) : -1;
}

}  // namespace attn25
