// tcgen05 wrappers and row output shared by the tensor-core attention kernels.
#pragma once

#include "hikv_packed.cuh"

namespace hikv {

// instruction descriptor: fp32 accumulator, bf16 A and B, A k-major; B
// k-major or (trans) n-major
constexpr uint32_t idesc_of(int M, int N, bool b_trans) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_trans ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}
// shared-memory matrix descriptor, 128-byte swizzle: lbo between 64-element
// blocks along the contiguous dimension, sbo between groups of eight rows
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
// arrive on `bar` when every product this thread has issued is complete
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), \
                 "=r"(r[i + 6]), "=r"(r[i + 7])
#define RW8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), \
                  "+r"(r[i + 6]), "+r"(r[i + 7])
#define I8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), \
                 "r"(r[i + 6]), "r"(r[i + 7])
// 32 columns of this thread's lane; the registers are valid after
// tmem_wait_ld() and held() in front of their first use
__device__ __forceinline__ void tmem_ld32(uint32_t* r, uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : R8(r, 0), R8(r, 8), R8(r, 16), R8(r, 24)
        : "r"(addr));
}
__device__ __forceinline__ void held(uint32_t* r) {
    asm volatile("" : RW8(r, 0), RW8(r, 8), RW8(r, 16), RW8(r, 24));
}
__device__ __forceinline__ void tmem_ld8(uint32_t* r, uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];" : R8(r, 0) : "r"(addr));
}
__device__ __forceinline__ void held8(uint32_t* r) { asm volatile("" : RW8(r, 0)); }
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::I8(r, 0), "r"(addr)
                 : "memory");
}
// one column, complete
__device__ __forceinline__ void tmem_ld1(uint32_t& r, uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r)
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tmem_st1(uint32_t addr, uint32_t r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%1], {%0};" ::"r"(r), "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t* r, uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : R8(r, 0), R8(r, 8)
        : "r"(addr));
}
__device__ __forceinline__ void held16(uint32_t* r) { asm volatile("" : RW8(r, 0), RW8(r, 8)); }
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15};" ::I8(r, 0),
        I8(r, 8), "r"(addr)
        : "memory");
}
#undef R8
#undef RW8
#undef I8
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
// a bounded wait of a whole warp: all lanes agree on the outcome
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* where, uint32_t index) {
    return __all_sync(0xffffffffu, attend_wait(bar, parity, where, index));
}

__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

// a turn between the two issuing threads (it orders no memory)
__device__ __forceinline__ bool turn_begin(uint32_t* turn, volatile uint32_t* where) {
    if (atomicExch(turn, 1u) == 0u) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 0; i < (1u << 28); ++i) {
        if (atomicExch(turn, 1u) == 0u) return true;
        if ((i & 255u) == 255u && global_ns() - t0 > kWaitLimitNs) break;
    }
    *where = 0x508;
    return false;
}
__device__ __forceinline__ void turn_end(uint32_t* turn) { atomicExch(turn, 0u); }

// Among each four lanes: x[j] of lane i becomes x[i] of lane j (items of eight words)
__device__ __forceinline__ void quad_transpose(uint32_t (&x)[4][8], int lane) {
    const bool hi = lane & 2, lo = lane & 1;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t y = __shfl_xor_sync(0xffffffffu, hi ? x[j][k] : x[j + 2][k], 2);
            if (hi) x[j][k] = y;
            else x[j + 2][k] = y;
        }
#pragma unroll
    for (int j = 0; j < 4; j += 2)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t y = __shfl_xor_sync(0xffffffffu, lo ? x[j][k] : x[j + 1][k], 1);
            if (lo) x[j][k] = y;
            else x[j + 1][k] = y;
        }
}
// 32 bytes; `wide`: p is 32-byte aligned
__device__ __forceinline__ void store32(void* p, const uint32_t* x, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                     "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(x[4], x[5], x[6], x[7]);
    }
}

}  // namespace hikv
