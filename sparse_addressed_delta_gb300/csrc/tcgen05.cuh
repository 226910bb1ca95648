// tcgen05 (5th-generation tensor core) wrappers of the gated delta rule's kernels: bfloat16 products
// with float32 accumulators in tensor memory, the A operand in tensor memory, the B operand in shared
// memory with the 128-byte swizzle.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "delta_internal.cuh"

namespace sdm {

// Operands in shared memory lie as tc_at puts them.
// An operand's descriptor: the lower word holds its address and the offset between tiles (both in units
// of 16 bytes, so that steps are added to it), the upper one is the same for all: 8-row groups 1024 bytes
// apart, 128-byte swizzle.
__device__ __forceinline__ uint64_t tc_descriptor(uint32_t lower) {
    return (uint64_t)((1024u >> 4) | (1u << 14) | (2u << 29)) << 32 | lower;
}
// K-major operand (a row is one M or N index, its elements run along K): a K step of 16 is 32 bytes along
// the row
__device__ __forceinline__ uint32_t tc_k_major(uint32_t addr) { return ((addr >> 4) & 0x3FFFu) | (1u << 16); }
// MN-major operand (a row is one K index, its elements run along M or N): 64 of them a tile, the next tile
// `next` bytes on; a K step of 16 is 16 rows, 2048 bytes
__device__ __forceinline__ uint32_t tc_n_major(uint32_t addr, uint32_t next) {
    return ((addr >> 4) & 0x3FFFu) | ((next >> 4) << 16);
}

// instruction descriptor: bfloat16 x bfloat16 -> float32, M = 128, N columns
template <bool B_N_MAJOR, bool A_M_MAJOR = false>
__device__ __forceinline__ constexpr uint32_t tc_idesc(int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (A_M_MAJOR ? 1u << 15 : 0u) | (B_N_MAJOR ? 1u << 16 : 0u) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// The products are issued by one lane (`one`: elected once) of a converged warp whose operands are
// uniform: they then stay in uniform registers, and a product issues in 14 cycles; issued from a branch
// that only one lane takes, each one costs 48 whatever its size (measured with M = 128; N = 64 runs in 33).
__device__ __forceinline__ uint32_t tc_elect() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one;
}
// d [128 lanes x N] (+)= a [128 lanes x 16, two bfloat16 a column of tensor memory] b
__device__ __forceinline__ void tc_mma_ts(uint32_t one, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(tc_descriptor(b)), "r"(idesc), "r"((uint32_t)add), "r"(one)
        : "memory");
}
// the same with both operands in shared memory
__device__ __forceinline__ void tc_mma_ss(uint32_t one, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(tc_descriptor(a)), "l"(tc_descriptor(b)), "r"(idesc), "r"((uint32_t)add), "r"(one)
        : "memory");
}

__device__ __forceinline__ void tc_commit_to(uint32_t one, unsigned long long *bar) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar)),
        "r"(one)
        : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 columns of the warp's 32 lanes
__device__ __forceinline__ void tc_load16(uint32_t addr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
          "=f"(v[14]), "=f"(v[15])
        : "r"(addr)
        : "memory");
}
// 16 columns of 16 lanes at each of two addresses, in the fragments of 8 x 8 blocks: for 8 columns c,
// v[4 c ..] is (lane / 4, 2 (lane % 4)), its right neighbour, and both of row + 8
__device__ __forceinline__ void tc_load_frag16(uint32_t a, uint32_t b, float (&v)[8], float (&u)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n"
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(u[0]), "=f"(u[1]), "=f"(u[2]), "=f"(u[3]), "=f"(u[4]), "=f"(u[5]), "=f"(u[6]), "=f"(u[7])
        : "r"(a), "r"(b)
        : "memory");
}
__device__ __forceinline__ void tc_load_frag16(uint32_t a, float (&v)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
        : "r"(a)
        : "memory");
}
__device__ __forceinline__ void tc_store8(uint32_t addr, const unsigned (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// 16 floats as three bfloat16 planes of 8 packed columns
__device__ __forceinline__ void tc_store_planes(uint32_t hi, uint32_t mid, uint32_t lo, const float (&x)[16]) {
    constexpr int N = 3;
    unsigned p[N][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        unsigned s[N];
        split_bf16<N>(x[2 * i], x[2 * i + 1], s);
#pragma unroll
        for (int m = 0; m < N; ++m) p[m][i] = s[m];
    }
    tc_store8(hi, p[0]);
    tc_store8(mid, p[1]);
    tc_store8(lo, p[2]);
}

// Tensor copies of 64 tokens x 64 columns of one head of a [B, T, heads, D] bfloat16 tensor, between
// global memory and a tile as tc_at lays it out. Loads are 0, stores are left out, past T and D.
cudaError_t tc_tensor_map(CUtensorMap *m, const void *p, const long long *strides, int B, int T, int heads, int D);
// boxes of 32 columns x `box` rows of float32 [slots, rows, columns] (0 past the rows and columns)
cudaError_t tc_state_map(CUtensorMap *m, const void *p, long long slots, int rows, int columns, int box);
// whether such a map can describe the tensor (a broadcast dimension has no stride to give)
inline bool tc_tensor_fits(const long long *s, int B, int T, int heads) {
    const int n[3] = {B, T, heads};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && s[i] * 2 >= (1LL << 40)) return false;
    return true;
}
// coordinate of a sequence or head: an input broadcast along it has one of them in its map
__device__ __forceinline__ int tc_coord(long long stride, int i) { return stride ? i : 0; }
__device__ __forceinline__ void tc_tensor_load(void *dst, const CUtensorMap *m, int col, int head, int token, int seq,
                                               unsigned long long *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(m), "r"(col), "r"(head), "r"(token), "r"(seq), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tc_tensor_store(const CUtensorMap *m, int col, int head, int token, int seq, const void *src) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(m),
                 "r"(col), "r"(head), "r"(token), "r"(seq), "r"(smem_u32(src))
                 : "memory");
}

// four 8 x 8 blocks of bfloat16 fragments stored transposed: lane 8 b + r gives the address of row r (a
// column of block b)
__device__ __forceinline__ void stsm4t(unsigned addr, const unsigned (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

__device__ __forceinline__ bool mbar_test_wait(unsigned long long *bar, unsigned parity) {
    unsigned ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// What a block's `*dead` begins with: with a limit of one it has given up, whatever its waits' looks find. (Asked in each wait
// it takes the 16384 tokens below 195 us.)
__device__ __forceinline__ bool tc_gives_up(long long limit) { return limit < 2; }
// Waits for a phase of `bar`, at most `limit` polls; gives up at once when another thread of the
// block has. Returns whether the phase completed.
__device__ __forceinline__ bool tc_wait(unsigned long long *bar, unsigned parity, volatile int *dead,
                                        long long limit) {
    // one look by test_wait first: with try_wait alone linear attention of 16384 tokens takes 198 us for 192
    if (mbar_test_wait(bar, parity)) return true;
    for (long long i = 1; i < limit; ++i) {
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

// A value down a column of a matrix in global memory. In order, so that a column's addresses take one register
// pair: computed at once they are spilled, and the reloads then stand behind the stores.
__device__ __forceinline__ void tc_put(float *&at, float x, int row) {
    asm volatile("st.global.f32 [%0], %1;" ::"l"(at), "f"(x) : "memory");
    at += row;
}

}  // namespace sdm
