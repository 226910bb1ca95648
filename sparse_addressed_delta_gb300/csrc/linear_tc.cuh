// Arithmetic of the linear attention's tensor-core kernels: floats split into bfloat16 planes and pairs of floats in
// packed operations. The scans issue instructions at 85 % of what an SM can, so these count: a pair's three planes take
// seven (three conversions, four mixed-precision subtractions), where widening the planes to floats takes eleven.
#pragma once

#include "linear_internal.cuh"
#include "pairs.cuh"
#include "tcgen05.cuh"

namespace sdm {

// the sequences from the longest down, so that the last blocks to start are short
__device__ __forceinline__ int linear_longest_first(const LinearDims &d, const int32_t *valid, int b) {
    if (!valid || d.B > 32) return b;
    const int lane = threadIdx.x & 31, mine = lane < d.B ? linear_valid(valid, lane, d.T) : -1;
    int rank = 0;
    for (int i = 0; i < d.B; ++i) {
        const int other = __shfl_sync(~0u, mine, i);
        rank += other > mine || (other == mine && i < lane);
    }
    return __ffs(__ballot_sync(~0u, rank == b)) - 1;
}

// The loading warp: chunk after chunk of `nch` into ST stages of shared memory as they are emptied, by tensor copies that
// complete full[stage] (of one arrival); issue(stage, first token, barrier) starts a stage's, `bytes` of them in tiles of
// 64 rows. Copies of all stages are in flight at once (with each awaited before the next, a carry's chunk took 1.2 us).
// A chunk of fewer than 64 tokens, of which a sequence has one at most, goes by a barrier of its own: what lies past the
// tokens is not used, so its rows are cleared before the stage counts as full.
template <int ST, typename At, typename Issue>
__device__ __forceinline__ void linear_loads(unsigned char *smem, int bytes, unsigned long long *full, unsigned long long *empty,
                                             unsigned long long *partial, int nch, int ntok, At chunk_at, Issue issue, volatile int *dead, long long spin) {
    constexpr int C = 64, TILE = C * 128;
    const int lane = threadIdx.x & 31;
    int it = 0;
    for (; it < nch; ++it) {
        const int s = it % ST, t0 = chunk_at(it) * C, nt = ntok - t0 < C ? ntok - t0 : C;
        unsigned char *st = smem + s * bytes;
        if (it >= ST && !tc_warp_wait(empty + s, (it / ST - 1) & 1, dead, spin)) break;
        unsigned long long *to = nt < C ? partial : full + s;
        if (lane == 0) {
            mbar_arrive_expect_tx(to, bytes);
            issue(st, t0, to);
        }
        __syncwarp();
        if (nt == C) continue;
        if (!tc_warp_wait(to, 0, dead, spin)) {
            mbar_wait_bounded(to, 0);                              // nothing in flight behind a give-up
            break;
        }
        for (int i = lane; i < (C - nt) * 8; i += 32) {
            const int off = tc_at(nt + (i >> 3), i & 7);
            for (int c = 0; c < bytes / TILE; ++c) *reinterpret_cast<uint4 *>(st + c * TILE + off) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full + s);
    }
    // nothing is in flight when the block ends, also where its other warps gave up
    for (int i = it > ST ? it - ST : 0; i < it; ++i) {
        const int t0 = chunk_at(i) * C;
        if (ntok - t0 >= C) mbar_wait_bounded(full + i % ST, i / ST & 1);
    }
}

// x minus the lower or upper bfloat16 of a pair, exact where that is x rounded
__device__ __forceinline__ float minus_lo(float x, unsigned p) {
    float r;
    asm("{\n .reg .b16 l, h, m;\n mov.b32 {l, h}, %1;\n mov.b16 m, 0xBF80;\n fma.rn.f32.bf16 %0, l, m, %2;\n}" : "=f"(r) : "r"(p), "f"(x));
    return r;
}
__device__ __forceinline__ float minus_hi(float x, unsigned p) {
    float r;
    asm("{\n .reg .b16 l, h, m;\n mov.b32 {l, h}, %1;\n mov.b16 m, 0xBF80;\n fma.rn.f32.bf16 %0, h, m, %2;\n}" : "=f"(r) : "r"(p), "f"(x));
    return r;
}

// x0, x1 as sums of three bfloat16 terms each
__device__ __forceinline__ void split3(float x0, float x1, unsigned (&p)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        p[i] = pack_bf16(x0, x1);
        if (i < 2) {
            x0 = minus_lo(x0, p[i]);
            x1 = minus_hi(x1, p[i]);
        }
    }
}

// 16 floats as three planes of 8 packed columns of tensor memory
__device__ __forceinline__ void store_planes3(uint32_t hi, uint32_t mid, uint32_t lo, const float2 *x) {
    unsigned p[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        unsigned s[3];
        split3(x[i].x, x[i].y, s);
        p[0][i] = s[0]; p[1][i] = s[1]; p[2][i] = s[2];
    }
    tc_store8(hi, p[0]);
    tc_store8(mid, p[1]);
    tc_store8(lo, p[2]);
}

// 8 columns of a row of a [64 tokens] tile whose NP planes lie SRC bytes apart
template <int NP, int SRC>
__device__ __forceinline__ void load_piece(const unsigned char *src, float2 (&x)[4]) {
#pragma unroll
    for (int m = NP - 1; m >= 0; --m) {
        const uint4 r = *reinterpret_cast<const uint4 *>(src + m * SRC);
        const unsigned u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 y = make_float2(lo_f32(u[e]), hi_f32(u[e]));
            x[e] = m == NP - 1 ? y : make_float2(x[e].x + y.x, x[e].y + y.y);
        }
    }
}
// such a piece times w, as three planes `plane` bytes apart
__device__ __forceinline__ void scale_piece(const float2 (&x)[4], float w, unsigned char *dst, int plane) {
    unsigned pl[3][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        unsigned s[3];
        const float2 y = mul2(x[e], make_float2(w, w));
        split3(y.x, y.y, s);
        pl[0][e] = s[0]; pl[1][e] = s[1]; pl[2][e] = s[2];
    }
#pragma unroll
    for (int m = 0; m < 3; ++m) *reinterpret_cast<uint4 *>(dst + m * plane) = make_uint4(pl[m][0], pl[m][1], pl[m][2], pl[m][3]);
}

}  // namespace sdm
