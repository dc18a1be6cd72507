// tcgen05.cuh -- the fifth-generation tensor cores' instructions that the kernels use, and the
// barriers around them.  One CTA's products: D[128 x N] (fp32, tensor memory) += A[128 x 16] B[N x 16]^T,
// both operands 16-bit in shared memory, K-major, in the 128-byte swizzle: rows of 128 bytes, eight of
// them 1024 bytes, whose 16-byte chunk c lies at chunk c ^ (row mod 8).
#pragma once

#include "device.cuh"

namespace vc {

__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// ---- mbarriers -----------------------------------------------------------------------------------

__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(smem_at(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(smem_at(bar)) : "memory");
}
// At the barrier that CTA `rank` of the cluster has at this address.
__device__ __forceinline__ void bar_arrive_at(uint64_t* bar, unsigned rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_at(bar)), "r"(rank));
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(r) : "memory");
}
__device__ __forceinline__ bool bar_test(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(smem_at(bar)), "r"(parity) : "memory");
    return done != 0;
}
// Wait for the phase of this parity, at most `limit` nanoseconds; a wait that gives up sets *failed, which
// ends the CTA's other waits too.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int* failed, unsigned long long limit) {
    if (bar_test(bar, parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    while (!bar_test(bar, parity)) {
        if (*failed) return false;
        if (global_timer_ns() - t0 > limit) {
            *failed = 1;
            return false;
        }
    }
    return true;
}

// The same for what has to be over before the CTA gives its memory back, whatever failed.
__device__ __forceinline__ void bar_drain(uint64_t* bar, uint32_t parity, volatile int* failed, unsigned long long limit) {
    const unsigned long long t0 = global_timer_ns();
    while (!bar_test(bar, parity)) {
        if (global_timer_ns() - t0 > limit) {
            *failed = 1;
            return;
        }
    }
}

// ---- tensor memory ---------------------------------------------------------------------------------

// By one whole warp; the address is written to shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t* at, int columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_at(at)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t at, int columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(at), "r"(columns) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Sixteen columns of the warp's 32 rows, one row a lane.  The warp's number mod 4 is its quarter.
__device__ __forceinline__ void tmem_load(uint32_t at, float (&v)[16]) {
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
}

// ---- products --------------------------------------------------------------------------------------

// Operand at shared address `at` (its first row 1024-byte aligned; 32 bytes on for every 16 columns).
__device__ __forceinline__ uint64_t operand(uint32_t at) {
    return (uint64_t)((at & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// M = 128 rows by N columns (a multiple of 16), both operands of the type, fp32 sums.
template <int DT>
__device__ __forceinline__ uint32_t product_shape(int n) {
    constexpr uint32_t type = DT == kBF16 ? 1u : 0u;
    return 1u << 4 | type << 7 | type << 10 | (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}
// By one thread.  add false: D starts from zero.
__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(shape), "r"((uint32_t)add) : "memory");
}
// Arrive at the barrier when all products issued by this thread are done.
__device__ __forceinline__ void products_done(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(smem_at(bar)) : "memory");
}

}  // namespace vc
