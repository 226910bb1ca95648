// Shared by the norms over rows (norm.cu, group_norm.cu): rows in registers, the ring of rows ahead, sums over a
// row's threads, column sums of blocks' partials.
#pragma once

#include "chain.cuh"
#include "sdm_internal.cuh"

namespace sdm {
namespace {

constexpr int kNormBlock = 128;        // threads of a block whose rows belong to parts of warps
constexpr int kNormMaxCols = 16384;
constexpr int kNormRegCols = 8192;     // backward: column sums in registers up to this width
// columns and runs of partials of a block that adds them, 32 lanes of which take two runs each. Whole training call,
// us, with 16 x 64 and (runs in shared memory throughout) 32 x 32: 5003 x 1007 float32 41, 42; 20000 x 1007 94, 96;
// 262144 x 128 bfloat16 68, 68; 2000 x 4096 49, 46; 32768 x 4096 259, 257
constexpr int kNormColThreads = 16, kNormColSlices = 64;
template <typename T>
constexpr int kNormStages = sizeof(T) == 2 ? 4 : 3;   // rows in the ring, the one in use among them
// backward: at least this many rows a block, for fewer partials. Whole training call, us, with 4, 6, 8 and 12: 5003 x
// 1007 float32 39, 41, 45, 49; 2000 x 4096 bfloat16 49, 49, 48, 54; the same with each: 500 x 2048, 32768 x 4096,
// 262144 x 128, 20000 x 1007 and 3000 x 8192 (a block has more rows, or there are too few for it)
constexpr int kNormRowsBlock = 6;

template <int BYTES> struct VecOf;
template <> struct VecOf<16> { using type = uint4; };
template <> struct VecOf<4> { using type = unsigned; };
template <> struct VecOf<2> { using type = unsigned short; };

template <typename T, int VEC>
using Vec = typename VecOf<VEC * (int)sizeof(T)>::type;

template <typename T, int VEC>
__device__ __forceinline__ void unpack(const Vec<T, VEC> &r, float *o) {
    const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] = to_f32(e[j]);
}

// A thread's own pieces of the rows ahead: `stage` holds NV vectors of each of ROWS tensors (and 8 bytes
// of statistics) at [vector][thread].
// HULL: rows one behind the other whose length is no multiple of 16 bytes. A row is then copied from the 16-byte
// boundary at or before its start (bytes of the row before; the first row starts on one), and its threads read
// their elements from what they all copied, so they wait for one another. Forward and backward, us, by each
// thread's own pieces and by hulls: 65536 x 1007 float32 121 + 193, 111 + 160; bfloat16 147 + 234, 114 + 142;
// 16384 x 4099 bfloat16 220 + 433, 146 + 226. (Results put back and stored in whole pieces: no better, 121 + 136
// and 142 + 218, and 126 + 153 for float32.)
template <typename T, int VEC, int NV, int ROWS, bool STATS, bool HULL>
struct RowRing {
    static constexpr int VB = VEC * (int)sizeof(T), ROW = NV * VB, THREAD = ROWS * ROW + (STATS ? 8 : 0);
    static __host__ __device__ size_t hull(int n) { return ((size_t)n * sizeof(T) + 30) / 16 * 16; }
    // bytes of the block: of rows (HULL), of the threads' pieces and statistics
    static __host__ __device__ size_t stage_bytes(int n, int threads, int rows) {
        return HULL ? (size_t)ROWS * rows * hull(n) + (STATS ? 8 : 0) * threads : (size_t)THREAD * threads;
    }
    unsigned char *base;               // of the block
    int t, tpr, n;                     // thread of the row, threads of the row, columns
    int sub, rpb;                      // row of the block, rows of a block

    __device__ __forceinline__ unsigned char *row_at(int stage, int which) const {
        return base + stage * stage_bytes(n, blockDim.x, rpb) + (which * rpb + sub) * hull(n);
    }

    __device__ __forceinline__ unsigned char *at(int stage, int vector) const {
        return base + ((size_t)stage * THREAD) * blockDim.x + ((size_t)vector * blockDim.x + threadIdx.x) * VB;
    }
    __device__ __forceinline__ unsigned char *stats_at(int stage) const {
        if (HULL) return base + stage * stage_bytes(n, blockDim.x, rpb) + ROWS * rpb * hull(n) + 8 * threadIdx.x;
        return base + ((size_t)stage * THREAD + ROWS * ROW) * blockDim.x + 8 * threadIdx.x;
    }
    // row `which` of `stage`; 0 past the row's end, or when the row is not live
    __device__ __forceinline__ void fetch(int stage, int which, const T *row, bool live) const {
        if constexpr (HULL) {
            const int shift = (int)((uintptr_t)row & 15), bytes = live ? shift + n * (int)sizeof(T) : (int)hull(n);
            const unsigned char *src = reinterpret_cast<const unsigned char *>(row) - shift;
            const unsigned dst = smem_u32(row_at(stage, which));
            for (int at = 16 * t; at < bytes; at += 16 * tpr) {
                const int take = !live ? 0 : bytes - at < 16 ? bytes - at : 16;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + at), "l"(src + at), "r"(take) : "memory");
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + t) * VEC;
            const bool in = live && c < n;
            unsigned char *dst = at(stage, which * NV + i);
            if constexpr (VB == 16) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(row + (in ? c : 0)), "r"(in ? 16 : 0) : "memory");
            } else if constexpr (VB == 4) {
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(row + (in ? c : 0)), "r"(in ? 4 : 0) : "memory");
            } else {
                *reinterpret_cast<T *>(dst) = in ? row[c] : from_f32<T>(0.f);
            }
        }
    }
    __device__ __forceinline__ void fetch_stats(int stage, const float2 *p, bool live) const {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(stats_at(stage))), "l"(p), "r"(live ? 8 : 0) : "memory");
    }
    __device__ __forceinline__ void read(int stage, int which, const T *row, float *o) const {
        if constexpr (HULL) {
            const unsigned char *at = row_at(stage, which) + ((uintptr_t)row & 15);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * tpr + t) * VEC;
                const Vec<T, VEC> r = c < n ? *reinterpret_cast<const Vec<T, VEC> *>(at + c * sizeof(T)) : Vec<T, VEC>{};
                unpack<T, VEC>(r, o + i * VEC);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Vec<T, VEC> r = *reinterpret_cast<const Vec<T, VEC> *>(at(stage, which * NV + i));
            unpack<T, VEC>(r, o + i * VEC);
        }
    }
};

// the thread's pieces of a row (0 past its end), straight to registers (the row may be the result's: no read-only loads)
template <typename T, int VEC, int NV>
__device__ __forceinline__ void load_row(const T *row, int t, int tpr, int n, float *o) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + t) * VEC;
        const Vec<T, VEC> r = c < n ? *reinterpret_cast<const Vec<T, VEC> *>(row + c) : Vec<T, VEC>{};
        unpack<T, VEC>(r, o + i * VEC);
    }
}

template <typename T, int VEC, int NV>
__device__ __forceinline__ void store_row(T *row, int t, int tpr, int n, const float *v) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + t) * VEC;
        if (c < n) {
            float o[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) o[j] = v[i * VEC + j];
            store_vec<T, VEC>(row + c, o);
        }
    }
}

// per-column parameters (float32, or the row's type), `fill` where there are none
template <typename T, int VEC, int NV>
__device__ __forceinline__ void load_cols(const void *p, bool f32, float fill, int t, int tpr,
                                          int n, float *o) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int c = (i * tpr + t) * VEC + j;
            o[i * VEC + j] = !p || c >= n ? fill
                             : f32 ? static_cast<const float *>(p)[c]
                                   : to_f32(static_cast<const T *>(p)[c]);
        }
}

template <int M>
__device__ __forceinline__ void warp_sum(float (&v)[M], int width) {
    for (int o = width >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
}

// Sums of M values over the threads of one row, returned to all of them. BLOCK: over the block,
// warps added in warp order (`red` holds 2 * M * 32 floats, its halves used in turn so that one
// barrier a call is enough).
template <bool BLOCK, int M>
__device__ __forceinline__ void row_sum(float (&v)[M], int tpr, float *red, int &turn) {
    warp_sum<M>(v, BLOCK ? 32 : tpr);
    if constexpr (BLOCK) {
        float *r = red + turn * M * 32;
        turn ^= 1;
        const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int m = 0; m < M; ++m) r[m * 32 + warp] = v[m];
        __syncthreads();
#pragma unroll
        for (int m = 0; m < M; ++m) {
            float s = 0.f;
            for (int w = 0; w < nw; ++w) s += r[m * 32 + w];
            v[m] = s;
        }
    }
}

// the next row's pieces are there; with HULL, all its threads' (who are then also done with the row before)
template <bool HULL, bool BLOCK, int PENDING>
__device__ __forceinline__ void row_ready() {
    cp_async_wait<PENDING>();
    if constexpr (HULL) {
        if constexpr (BLOCK) __syncthreads();
        else __syncwarp();
    }
}

// s + x as the rounded sum and what the rounding lost, added to `low`
__device__ __forceinline__ float add_exact(float s, float x, float &low) {
    const float sum = s + x, of_x = sum - s;
    low += (s - (sum - of_x)) + (x - of_x);
    return sum;
}

// column sums of the blocks' partials, in a fixed order: kNormColSlices runs of blocks, then them in pairs, with what
// the roundings lose kept beside (5003 x 1007 float32, in one float each: 1.7e-7 off float64 with the runs one after
// the other, 1.4e-7 in pairs)
__device__ __forceinline__ void norm_cols(int block, const float *part, int parts, int n, float *dw, float *db) {
    static_assert(kNormColSlices == 64 && kNormColThreads <= 32, "a warp a column, two runs a lane");
    __shared__ float sh[kNormColSlices][kNormColThreads + 1], lost[kNormColSlices][kNormColThreads + 1];
    const int tx = threadIdx.x % kNormColThreads, ty = threadIdx.x / kNormColThreads;
    const int c = block * kNormColThreads + tx;          // over [2][n]
    float s = 0.f, low = 0.f;
    if (c < 2 * n)
#pragma unroll 8
        for (int p = ty; p < parts; p += kNormColSlices) s = add_exact(s, __ldcg(part + (size_t)p * 2 * n + c), low);
    sh[ty][tx] = s;
    lost[ty][tx] = low;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = block * kNormColThreads + warp;
    if (warp >= kNormColThreads) return;
    low = lost[lane][warp] + lost[lane + 32][warp];
    s = add_exact(sh[lane][warp], sh[lane + 32][warp], low);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        const float x = __shfl_down_sync(~0u, s, m);
        low += __shfl_down_sync(~0u, low, m);
        s = add_exact(s, x, low);
    }
    if (lane == 0 && col < 2 * n) {
        if (fabsf(s) <= 3.402823466e38f) s += low;           // an infinite sum is one; what it lost is a NaN
        if (col < n) {
            if (dw) dw[col] = s;
        } else if (db) {
            db[col - n] = s;
        }
    }
}
__global__ void __launch_bounds__(kNormColThreads *kNormColSlices)
    k_norm_cols(const float *part, int parts, int n, float *dw, float *db) {
    chain_wait();                                        // (where it is chained to what makes the partials)
    norm_cols(blockIdx.x, part, parts, n, dw, db);
}
inline unsigned norm_col_blocks(int n) { return (2 * n + kNormColThreads - 1) / kNormColThreads; }

struct NormGeom {
    int vec;        // elements per vector
    bool hull;      // copied from 16-byte boundaries all the same (RowRing)
    int e;          // elements per thread
    int tpr;        // threads per row
    bool block;     // a row belongs to a whole block
    int threads, rpb;
};

// 16 elements a thread leave room for the weights and sums in registers; the forward (no sums) takes 32
// once 128 threads do not cover the row with 16: fewer threads to a barrier.
NormGeom norm_geom(int n, int vec, bool backward) {
    NormGeom g;
    g.vec = vec;
    g.hull = false;
    g.e = !backward && n > 16 * kNormBlock ? 32 : 16;
    const int need = (n + g.e - 1) / g.e;
    if (need <= 32) {
        g.tpr = 1;
        while (g.tpr < need) g.tpr *= 2;
        g.block = false;
        g.threads = kNormBlock;
        g.rpb = kNormBlock / g.tpr;
    } else {
        g.tpr = (need + 31) / 32 * 32;
        g.block = true;
        g.threads = g.tpr;
        g.rpb = 1;
    }
    return g;
}

// blocks of a backward: at most one per row group, and per kNormRowsBlock rows as long as every SM has
// one; 512 threads an SM (by their registers)
int norm_back_blocks(const NormGeom &g, long long rows) {
    const int per_sm = g.threads >= 512 ? 1 : 512 / g.threads;
    const long long few = rows / kNormRowsBlock > kRefSms ? rows / kNormRowsBlock : kRefSms;
    const long long need = (rows + g.rpb - 1) / g.rpb, fill = (long long)kRefSms * per_sm;
    const long long most = fill < few ? fill : few;
    return (int)(need < most ? need : most);
}

// the widest vector that divides the rows, their strides (in elements) and the addresses
int norm_vec(int es, int n, long long s0, long long s1, const void *a, const void *b,
             const void *c) {
    const uintptr_t any = (uintptr_t)a | (uintptr_t)b | (uintptr_t)c | (uintptr_t)((long long)n * es) |
                          (uintptr_t)(s0 * es) | (uintptr_t)(s1 * es);
    if (any % 16 == 0) return 16 / es;
    return any % 4 == 0 ? 4 / es : 1;
}

// rows that no 16-byte vector divides, one behind the other from a 16-byte boundary
bool norm_hull(int es, int vec, int n, long long stride, const void *p) {
    return vec * es < 16 && stride == n && (uintptr_t)p % 16 == 0;
}

}  // namespace
}  // namespace sdm
