// tcgen05.cuh -- inline-PTX helpers of the prompt kernels (prefill_tc.cu,
// prompt_masked.cuh): matrix instructions of the fifth generation, their operand
// descriptors, loads and stores of tensor memory, and the swizzled layout.
#pragma once

#include <cuda.h>

#include "device_common.cuh"

namespace pkv {
namespace prefill_tc {

constexpr unsigned FULL = 0xffffffffu;

// ---- tcgen05 ---------------------------------------------------------------

// Shared-memory operand descriptor of the 128-byte swizzled layout: rows of
// 128 bytes, 8-row groups 1024 bytes apart (the stride field), 16-byte chunk
// c of row t stored at chunk c ^ (t mod 8).  The start address advances by
// 32 bytes per 16-element K step inside a 64-element half; every block
// starts on a 1024-byte boundary, so the base-offset field stays 0.  `lead`
// (the leading field) is the distance of neighbouring 64-element halves of an
// MN-major operand wider than 64.  Addresses are below 2^18, so a descriptor
// of the same layout `bytes` further is the sum with bytes / 16.
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lead = 16) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// True on one lane of the (converged) warp.  What that thread does alone,
// descriptors included, then runs on the warp's uniform registers: with
// `lane == 0` instead, an MMA took 80 to 100 cycles to issue.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// Instruction descriptor of kind::f16: fp32 accumulator, fp16 A and B, A
// K-major, B K-major or (mn_major) MN-major, M x N.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
    return (1u << 4) | (b_mn_major ? (1u << 16) : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void umma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
        : "memory");
}

// The same with A in tensor memory: row m of A in lane m, 16-bit elements
// two per column from a_tmem on.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
        : "memory");
}

// The mbarrier gets one arrival when every MMA this thread issued so far has
// completed.
__device__ __forceinline__ void umma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tc_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define PKV_R8(i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), \
                  "=r"(v[i + 6]), "=r"(v[i + 7])
#define PKV_W8(i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), \
                  "r"(v[i + 6]), "r"(v[i + 7])

// Lane l of the warp reads lane (32 (warp mod 4) + l) of tensor memory,
// columns col .. col + 31 (resp. 15); complete with tmem_ld_wait().
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : PKV_R8(0), PKV_R8(8), PKV_R8(16), PKV_R8(24)
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : PKV_R8(0), PKV_R8(8)
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        PKV_W8(0), PKV_W8(8), PKV_W8(16), PKV_W8(24)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        PKV_W8(0), PKV_W8(8)
        : "memory");
}
#undef PKV_R8
#undef PKV_W8
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Bounded wait on an mbarrier phase by every lane of the warp (each lane
// observes the completion itself; cheaper than one lane polling and a
// broadcast when the phase has already completed); true on every lane only
// if it completed for all of them, so the warp leaves its loops together.
__device__ __forceinline__ bool wait_lanes(uint32_t bar, uint32_t parity, int *status,
                                           unsigned long long limit_ns = kWaitLimitNs) {
    return __all_sync(FULL, mbar_wait(bar, parity, status, 0, limit_ns));
}

// Packed pairs of fp32 for Blackwell's two-wide add.
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 4-D tiled TMA load (no cache hint): K/V tiles are read again by the other
// query tiles of the same head, so they keep the default L2 policy.
__device__ __forceinline__ void tma_load_4d_plain(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                                  int c3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// Byte offset of 16-byte chunk c (elements 8c .. 8c + 7) of row t in a block
// of `rows` rows stored as 64-element halves, each half [rows][128 bytes]
// swizzled.
__device__ __forceinline__ uint32_t swz(int t, int c, int rows) {
    return (uint32_t)((((c >> 3) * rows + t) << 7) + (((c & 7) ^ (t & 7)) << 4));
}

// 16-byte cp.async that reads `bytes` (16 or 0) and zero-fills the rest.
__device__ __forceinline__ void cp_async16_zfill(uint32_t smem, const void *gmem, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4_zfill(uint32_t smem, const void *gmem, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem), "l"(gmem), "r"(bytes) : "memory");
}

}  // namespace prefill_tc
}  // namespace pkv
