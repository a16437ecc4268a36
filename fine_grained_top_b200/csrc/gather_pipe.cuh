// gather_pipe.cuh -- what the warp-specialised gather attention kernels share:
// bounded mbarrier waits, votes over named barriers, TMEM stores and the
// descriptors of their MN-major operands.
#pragma once

#include "ptx.cuh"

namespace sa {

// Arrive on `bar` once every cp.async this thread issued so far has landed
// (the arrival counts against the barrier's expected count).
__device__ __forceinline__ void cp_async_arrive_noinc(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Bounded wait for a phase that parks the thread in mbarrier.try_wait (with a
// suspend-time hint of 20 us) instead of polling: eleven warps wait on
// barriers most of the time here, and polling waits flood the issue slots
// and the pipe that executes the barrier tests.  Gives up like mbar_wait.
__device__ __forceinline__ bool try_wait_parked(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool gwait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    if (try_wait_parked(bar, parity)) return true;
    const unsigned long long t0 = globaltimer();
    while (true) {
        if (try_wait_parked(bar, parity)) return true;
        if (*abort) return false;
        if (globaltimer() - t0 > kWaitLimitNs) {
            *abort = 1;
            return false;
        }
    }
}
// The two MMA-issuing threads poll with plain mbarrier.try_wait (no suspend
// hint): each is one thread, and a parked issuer wakes late and delays the
// hand-off it waits for.
__device__ __forceinline__ bool try_wait_issuer(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool iwait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    if (try_wait_issuer(bar, parity)) return true;
    const unsigned long long t0 = globaltimer();
    while (true) {
        for (int i = 0; i < 16; ++i) if (try_wait_issuer(bar, parity)) return true;
        if (*abort) return false;
        if (globaltimer() - t0 > kWaitLimitNs) { *abort = 1; return false; }
    }
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// Arrive at barrier `id` without waiting for it.
__device__ __forceinline__ void bar_arrive_n(int id, int n) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }
// Barrier `id` over `n` threads that also returns the OR / AND of a predicate.
__device__ __forceinline__ bool bar_or(int id, int n, bool p) {
    uint32_t r;
    asm volatile(
        "{ .reg .pred a, b; setp.ne.u32 a, %1, 0; bar.red.or.pred b, %2, %3, a; selp.u32 %0, 1, 0, b; }"
        : "=r"(r)
        : "r"((uint32_t)p), "r"(id), "r"(n)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ bool bar_and(int id, int n, bool p) {
    uint32_t r;
    asm volatile(
        "{ .reg .pred a, b; setp.ne.u32 a, %1, 0; bar.red.and.pred b, %2, %3, a; selp.u32 %0, 1, 0, b; }"
        : "=r"(r)
        : "r"((uint32_t)p), "r"(id), "r"(n)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void bar_sync_n(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait_all() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void mma_acc(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t acc) {
    tc_mma_f16(d_tmem, a_desc, b_desc, idesc, acc);
}
// MN-major SW128 operand: 64-element MN chunks `lbo` bytes apart, 8-row K
// groups 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_mn128(uint32_t addr, uint32_t lbo) {
    uint64_t d = 0;
    d |= (uint64_t)((addr >> 4) & 0x3FFF);
    d |= (uint64_t)((lbo >> 4) & 0x3FFF) << 16;
    d |= (uint64_t)((1024 >> 4) & 0x3FFF) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// MN-major operand without swizzle: 8 x 16-byte core matrices (8 K rows of 8
// MN elements, 128 contiguous bytes); K groups of 8 rows `kgroup` bytes apart,
// MN chunks of 8 elements `mnchunk` bytes apart.  (For this layout the
// descriptor's leading offset is the K-group stride and its stride offset the
// MN-chunk stride.)
__device__ __forceinline__ uint64_t desc_mn_plain(uint32_t addr, uint32_t kgroup, uint32_t mnchunk) {
    uint64_t d = 0;
    d |= (uint64_t)((addr >> 4) & 0x3FFF);
    d |= (uint64_t)((kgroup >> 4) & 0x3FFF) << 16;
    d |= (uint64_t)((mnchunk >> 4) & 0x3FFF) << 32;
    d |= (uint64_t)1 << 46;   // layout type 0 (no swizzle) in bits 61-63
    return d;
}

}  // namespace sa
