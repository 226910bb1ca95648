// tcgen05 (5th-generation tensor core) wrappers of the gated delta rule's kernels: bfloat16 products
// with float32 accumulators in tensor memory, the A operand in tensor memory, the B operand in shared
// memory with the 128-byte swizzle.
#pragma once

#include "delta_internal.cuh"

namespace sdm {

// Operands in shared memory lie as tc_at puts them.
// K-major operand (a row is one N index, its elements run along K): 8-row groups 1024 bytes apart;
// a K step of 16 is 32 bytes along the row
__device__ __forceinline__ uint64_t tc_k_major(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// MN-major operand (a row is one K index, its elements run along N): 64 columns of N a tile, the next
// tile `next` bytes on; 8 rows of K every 1024 bytes, so a K step of 16 is 2048 bytes
__device__ __forceinline__ uint64_t tc_n_major(uint32_t addr, uint32_t next) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(next >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// instruction descriptor: bfloat16 x bfloat16 -> float32, M = 128, N columns
template <bool N_MAJOR>
__device__ __forceinline__ constexpr uint32_t tc_idesc(int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (N_MAJOR ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(128 >> 4) << 24);
}

// d [128 lanes x N] (+)= a [128 lanes x 16, two bfloat16 a column] b
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

__device__ __forceinline__ void tc_commit_to(unsigned long long *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of the warp's 32 lanes
__device__ __forceinline__ void tc_load32(uint32_t addr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
          "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
          "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
          "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(addr)
        : "memory");
}
// 16 columns of the warp's 32 lanes
__device__ __forceinline__ void tc_store16(uint32_t addr, const unsigned (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// 32 floats as N bfloat16 planes of 16 packed columns, plane p at addr + p * step
template <int N>
__device__ __forceinline__ void tc_store_planes(uint32_t addr, uint32_t step, const float (&x)[32]) {
    unsigned p[N][16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        unsigned s[N];
        split_bf16<N>(x[2 * i], x[2 * i + 1], s);
#pragma unroll
        for (int m = 0; m < N; ++m) p[m][i] = s[m];
    }
#pragma unroll
    for (int m = 0; m < N; ++m) tc_store16(addr + m * step, p[m]);
}

// Waits for a phase of `bar`, at most `limit` polls; gives up at once when another thread of the
// block has. Returns whether the phase completed.
__device__ __forceinline__ bool tc_wait(unsigned long long *bar, unsigned parity, volatile int *dead,
                                        long long limit) {
    for (long long i = 0; i < limit; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*dead) return false;
    }
    *dead = 1;
    return false;
}
// the same for a whole warp, with one answer
__device__ __forceinline__ bool tc_warp_wait(unsigned long long *bar, unsigned parity, volatile int *dead,
                                             long long limit) {
    return __all_sync(0xffffffffu, tc_wait(bar, parity, dead, limit));
}

}  // namespace sdm
