// Layer norm over the last dimension, forward and backward: the norm before a memory layer (rows
// of the model's width) and on its readings (rows of one head's width).
//   mean = sum(x) / n;  rstd = 1 / sqrt(sum((x - mean)^2) / n + eps);  xhat = (x - mean) rstd
//   y  = xhat w + b
//   dx = rstd (w dy - mean(w dy) - xhat mean(w dy xhat));  dw = sum_rows dy xhat;  db = sum_rows dy
// All arithmetic is float32; y and dx are rounded once. The variance is the sum of squares around
// the mean, from the row kept in registers: no cancellation, and x is read once.
//
// Bound by memory: a row is read once, held in registers and written once (bfloat16, 1048576 x 128: 92 us,
// 87 % of the copy rate; 32768 x 4096 107 us and its backward 144 us; 262144 x 128 forward and backward 70 us,
// the second behind the first's warm cache). A row belongs to TPR
// threads (a part of a warp up to 32, else the whole block), each with E elements as whole vectors
// (16 bytes when the row length, its stride and the pointers allow it, else 4 or one element).
// Blocks stay resident and walk over the rows with the weights in registers. Every thread copies its
// own pieces of the next kNormStages - 1 rows into shared memory (cp.async; nobody else reads them, so
// there is no barrier), which keeps about 100 KB an SM in flight. The backward's column sums stay in
// the same threads over all the rows of a block (in shared memory above 8192 columns), go to one
// partial per block, and a second kernel adds the partials in block order: no atomics, so results are
// reproducible.
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

// the thread's pieces of a row (0 past its end), straight to registers
template <typename T, int VEC, int NV>
__device__ __forceinline__ void load_row(const T *row, int t, int tpr, int n, float *o) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + t) * VEC;
        const Vec<T, VEC> r = c < n ? __ldg(reinterpret_cast<const Vec<T, VEC> *>(row + c)) : Vec<T, VEC>{};
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

template <typename T, int VEC, int NV, bool BLOCK, bool HULL>
__global__ void __launch_bounds__(BLOCK ? 512 : kNormBlock)
    k_norm(const T *x, long long xs, long long rows, int n, int tpr, const void *w, const void *b,
           bool wf32, float eps, T *y, float2 *stats) {
    constexpr int E = VEC * NV, ST = kNormStages<T>;
    extern __shared__ __align__(16) unsigned char ring_smem[];
    __shared__ float2 red[2 * 32];
    __shared__ float counts[32];           // BLOCK: columns of each warp
    float warp_cols = 0.f;
    int turn = 0;
    const int sub = BLOCK ? 0 : threadIdx.x / tpr, t = BLOCK ? threadIdx.x : threadIdx.x % tpr;
    const int rpb = BLOCK ? 1 : kNormBlock / tpr;
    const long long step = (long long)gridDim.x * rpb;
    float wv[E], bv[E];
    load_cols<T, VEC, NV>(w, wf32, 1.f, t, tpr, n, wv);
    load_cols<T, VEC, NV>(b, wf32, 0.f, t, tpr, n, bv);
    if constexpr (BLOCK) {
        float c[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((i * tpr + t) * VEC < n) c[0] += VEC;
        warp_sum<1>(c, 32);
        warp_cols = c[0];                  // at least one: the block has no warp past the row's end
        if ((threadIdx.x & 31) == 0) counts[threadIdx.x >> 5] = warp_cols;
        __syncthreads();
    }
    const RowRing<T, VEC, NV, 1, false, HULL> ring{ring_smem, t, tpr, n, sub, rpb};
    long long base = (long long)blockIdx.x * rpb;
    auto fetch = [&](int stage, long long row) {
        ring.fetch(stage, 0, x + (row < rows ? row : 0) * xs, row < rows);
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) fetch(i, base + sub + i * step);
    for (int stage = 0; base < rows; base += step, stage = (stage + 1) % ST) {
        const long long row = base + sub;
        if constexpr (HULL) row_ready<HULL, BLOCK, ST - 2>();
        fetch((stage + ST - 1) % ST, row + (ST - 1) * step);
        if constexpr (!HULL) row_ready<HULL, BLOCK, ST - 1>();
        float v[E];
        ring.read(stage, 0, x + row * xs, v);
        float s[1] = {0.f}, mean, m2;
#pragma unroll
        for (int j = 0; j < E; ++j) s[0] += v[j];
        auto around = [&](float c) {                       // this thread's squares around c
            float q = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if ((i * tpr + t) * VEC < n)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const float d = v[i * VEC + j] - c;
                        q = fmaf(d, d, q);
                    }
            return q;
        };
        warp_sum<1>(s, BLOCK ? 32 : tpr);
        if constexpr (BLOCK) {
            // each warp's sum and squares around its own mean; together, the squares around the row's
            // mean are those and count (mean_w - mean)^2: one barrier a row
            const float sw = s[0];
            float q[1] = {around(sw / warp_cols)};
            warp_sum<1>(q, 32);
            float2 *r = red + 32 * turn;
            turn ^= 1;
            if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = make_float2(sw, q[0]);
            __syncthreads();
            float sum = 0.f;
            for (int w = 0; w < (int)(blockDim.x >> 5); ++w) sum += r[w].x;
            mean = sum / (float)n;
            m2 = 0.f;
            for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
                const float c = counts[w], d = r[w].x / c - mean;
                m2 += fmaf(c * d, d, r[w].y);
            }
        } else {
            mean = s[0] / (float)n;
            float q[1] = {around(mean)};
            warp_sum<1>(q, tpr);
            m2 = q[0];
        }
        const float rstd = 1.f / sqrtf(m2 / (float)n + eps);
#pragma unroll
        for (int j = 0; j < E; ++j) v[j] -= mean;
        if (row < rows) {
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] = fmaf(v[j] * rstd, wv[j], bv[j]);
            store_row<T, VEC, NV>(y + row * n, t, tpr, n, v);
            if (stats && t == 0) stats[row] = make_float2(mean, rstd);
        }
    }
}

// part [blocks][2][n]: the block's column sums of dy xhat and of dy
template <typename T, int VEC, int NV, bool BLOCK, bool WIDE, bool HULL>
__global__ void __launch_bounds__(BLOCK ? (WIDE ? 1024 : 512) : kNormBlock)
    k_norm_bwd(const T *dy, long long ds, const T *x, long long xs, long long rows, int n, int tpr,
               const void *w, bool wf32, const float2 *stats, T *dx, float *part) {
    constexpr int E = VEC * NV, ST = kNormStages<T>;
    extern __shared__ __align__(16) unsigned char ring_smem[];
    using Ring = RowRing<T, VEC, NV, 2, true, HULL>;
    // WIDE: no ring, the column sums [2][n]; else they take the ring's place at the end
    float *cols = reinterpret_cast<float *>(ring_smem);
    __shared__ float red[2 * 2 * 32];
    int turn = 0;
    const int sub = BLOCK ? 0 : threadIdx.x / tpr, t = BLOCK ? threadIdx.x : threadIdx.x % tpr;
    const int rpb = BLOCK ? 1 : kNormBlock / tpr;
    const long long step = (long long)gridDim.x * rpb;
    float wv[WIDE ? 1 : E], aw[WIDE ? 1 : E], ab[WIDE ? 1 : E];
    if constexpr (WIDE) {
        for (int c = threadIdx.x; c < 2 * n; c += blockDim.x) cols[c] = 0.f;
        __syncthreads();
    } else {
        load_cols<T, VEC, NV>(w, wf32, 1.f, t, tpr, n, wv);
#pragma unroll
        for (int j = 0; j < E; ++j) aw[j] = ab[j] = 0.f;
    }
    const Ring ring{ring_smem, t, tpr, n, sub, rpb};
    long long base = (long long)blockIdx.x * rpb;
    auto fetch = [&](int stage, long long row) {
        const bool live = row < rows;
        const long long at = live ? row : 0;
        ring.fetch(stage, 0, x + at * xs, live);
        ring.fetch(stage, 1, dy + at * ds, live);
        ring.fetch_stats(stage, stats + at, live);
        cp_async_commit();
    };
    if constexpr (!WIDE)
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) fetch(i, base + sub + i * step);
    for (int stage = 0; base < rows; base += step, stage = (stage + 1) % ST) {
        const long long row = base + sub;
        float2 ns;
        float h[E], g[E], s[2] = {0.f, 0.f};
        if constexpr (WIDE) {                              // a row a block: it is live
            ns = __ldg(stats + row);
            load_row<T, VEC, NV>(x + row * xs, t, tpr, n, h);
            load_row<T, VEC, NV>(dy + row * ds, t, tpr, n, g);
        } else {
            if constexpr (HULL) row_ready<HULL, BLOCK, ST - 2>();
            fetch((stage + ST - 1) % ST, row + (ST - 1) * step);
            if constexpr (!HULL) row_ready<HULL, BLOCK, ST - 1>();
            ns = *reinterpret_cast<const float2 *>(ring.stats_at(stage));
            ring.read(stage, 0, x + row * xs, h);
            ring.read(stage, 1, dy + row * ds, g);
        }
        const float mean = ns.x, rstd = ns.y;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c0 = (i * tpr + t) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int e = i * VEC + j;
                // past the row's end x and dy are 0, and dy = 0 keeps the sums clean
                h[e] = (h[e] - mean) * rstd;
                if constexpr (WIDE) {
                    if (c0 + j < n) {
                        cols[c0 + j] = fmaf(g[e], h[e], cols[c0 + j]);
                        cols[n + c0 + j] += g[e];
                        g[e] *= !w ? 1.f : wf32 ? static_cast<const float *>(w)[c0 + j]
                                                : to_f32(static_cast<const T *>(w)[c0 + j]);
                    }
                } else {
                    aw[e] = fmaf(g[e], h[e], aw[e]);
                    ab[e] += g[e];
                    g[e] *= wv[e];
                }
                s[0] += g[e];
                s[1] = fmaf(g[e], h[e], s[1]);
            }
        }
        row_sum<BLOCK, 2>(s, tpr, red, turn);
        const float c1 = s[0] / (float)n, c2 = s[1] / (float)n;
        if (row < rows) {
#pragma unroll
            for (int j = 0; j < E; ++j) g[j] = rstd * (g[j] - c1 - h[j] * c2);
            store_row<T, VEC, NV>(dx + row * n, t, tpr, n, g);
        }
    }
    if (!part) return;
    cp_async_wait<0>();
    __syncthreads();
    float *out = part + (size_t)blockIdx.x * 2 * n;
    if constexpr (WIDE) {
        for (int c = threadIdx.x; c < 2 * n; c += blockDim.x) out[c] = cols[c];
    } else {
        // the block's row groups, added in their order: cols [2][groups][tpr * E]
        const int wide = tpr * E;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int c = (i * tpr + t) * VEC + j, e = i * VEC + j;
                if constexpr (BLOCK) {
                    if (c < n) {
                        out[c] = aw[e];
                        out[n + c] = ab[e];
                    }
                } else {
                    cols[sub * wide + c] = aw[e];
                    cols[(rpb + sub) * wide + c] = ab[e];
                }
            }
        if constexpr (!BLOCK) {
            __syncthreads();
            for (int c = threadIdx.x; c < n; c += kNormBlock) {
                float a = 0.f, d = 0.f;
                for (int r = 0; r < rpb; ++r) {
                    a += cols[r * wide + c];
                    d += cols[(rpb + r) * wide + c];
                }
                out[c] = a;
                out[n + c] = d;
            }
        }
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
__global__ void __launch_bounds__(kNormColThreads *kNormColSlices)
    k_norm_cols(const float *part, int parts, int n, float *dw, float *db) {
    static_assert(kNormColSlices == 64 && kNormColThreads <= 32, "a warp a column, two runs a lane");
    __shared__ float sh[kNormColSlices][kNormColThreads + 1], lost[kNormColSlices][kNormColThreads + 1];
    const int tx = threadIdx.x % kNormColThreads, ty = threadIdx.x / kNormColThreads;
    const int c = blockIdx.x * kNormColThreads + tx;     // over [2][n]
    float s = 0.f, low = 0.f;
    if (c < 2 * n)
#pragma unroll 8
        for (int p = ty; p < parts; p += kNormColSlices) s = add_exact(s, __ldg(part + (size_t)p * 2 * n + c), low);
    sh[ty][tx] = s;
    lost[ty][tx] = low;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = blockIdx.x * kNormColThreads + warp;
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

int norm_check(const char *what, const void *x, long long rows, int n, long long xs, int wdtype,
               int dtype) {
    if (dtype != SDM_F32 && dtype != SDM_BF16)
        return set_error(SDM_ERR_INVALID, "%s: dtype must be SDM_F32 or SDM_BF16", what);
    if (wdtype != SDM_F32 && wdtype != dtype)
        return set_error(SDM_ERR_INVALID, "%s: the weight's dtype must be SDM_F32 or the rows'", what);
    if (rows < 0 || n < 1 || xs < 0)
        return set_error(SDM_ERR_INVALID, "%s: rows must be >= 0, columns >= 1 and the row stride "
                         ">= 0, got %lld, %d, %lld", what, rows, n, xs);
    if (n > kNormMaxCols)
        return set_error(SDM_ERR_UNSUPPORTED, "%s: at most %d columns, got %d", what, kNormMaxCols, n);
    if (rows > 0 && !x) return set_error(SDM_ERR_INVALID, "%s: NULL pointer", what);
    return SDM_OK;
}

int norm_status(cudaError_t e) {
    if (e == cudaSuccess) return SDM_OK;
    return set_error(SDM_ERR_CUDA, "layer norm: %s", cudaGetErrorString(e));
}

// rows that no 16-byte vector divides, one behind the other from a 16-byte boundary
bool norm_hull(int es, int vec, int n, long long stride, const void *p) {
    return vec * es < 16 && stride == n && (uintptr_t)p % 16 == 0;
}

template <typename T, int VEC, int E, bool HULL>
void norm_launch(const NormGeom &g, const T *x, long long xs, long long rows, int n, const void *w,
                 const void *b, bool wf32, float eps, T *y, float2 *stats, cudaStream_t st) {
    const size_t smem = kNormStages<T> * RowRing<T, VEC, E / VEC, 1, false, HULL>::stage_bytes(n, g.threads, g.rpb);
    const long long need = (rows + g.rpb - 1) / g.rpb;
    auto go = [&](auto kern) {
        set_kernel_smem(kern, smem);
        // as many blocks as fit the card at once: they walk over the rows, and a second wave of blocks
        // would leave part of it idle (32768 x 4096 bfloat16: 122 us with one and a half waves)
        int per_sm = 1;
        if (need > kRefSms) cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, g.threads, smem);
        const long long most = (long long)kRefSms * (per_sm > 1 ? per_sm : 1);
        const unsigned grid = (unsigned)(need < most ? need : most);
        kern<<<grid, g.threads, smem, st>>>(x, xs, rows, n, g.tpr, w, b, wf32, eps, y, stats);
    };
    if (g.block) go(k_norm<T, VEC, E / VEC, true, HULL>);
    else go(k_norm<T, VEC, E / VEC, false, HULL>);
}

template <typename T>
void norm_forward(const NormGeom &g, const T *x, long long xs, long long rows, int n, const void *w,
                  const void *b, bool wf32, float eps, T *y, float2 *stats, cudaStream_t st) {
    constexpr int V16 = 16 / (int)sizeof(T), V4 = 4 / (int)sizeof(T);
    auto go = [&](auto vec) {
        constexpr int VEC = decltype(vec)::value;
        auto with = [&](auto hull) {
            constexpr bool HULL = decltype(hull)::value;
            if (g.e == 32) norm_launch<T, VEC, 32, HULL>(g, x, xs, rows, n, w, b, wf32, eps, y, stats, st);
            else norm_launch<T, VEC, 16, HULL>(g, x, xs, rows, n, w, b, wf32, eps, y, stats, st);
        };
        // wide rows of bfloat16 pairs fare better by their own pieces (8192 x 8190: 97 us, 117 by hulls)
        if constexpr (VEC < V16)
            if (g.hull && !(VEC == 2 && g.e == 32)) return with(std::true_type{});
        with(std::false_type{});
    };
    if (g.vec == V16) return go(std::integral_constant<int, V16>{});
    if constexpr (V4 > 1)
        if (g.vec == V4) return go(std::integral_constant<int, V4>{});
    go(std::integral_constant<int, 1>{});
}

template <typename T, int VEC>
void norm_bwd_launch(const NormGeom &g, int grid, const T *dy, long long ds, const T *x,
                     long long xs, long long rows, int n, const void *w, bool wf32,
                     const float2 *stats, T *dx, float *part, cudaStream_t st) {
    constexpr int NV = 16 / VEC;
    const size_t sums = (size_t)2 * (n > kNormRegCols ? n : kNormBlock * 16) * 4;
    auto go = [&](auto kern, size_t smem) {
        set_kernel_smem(kern, smem);
        kern<<<grid, g.threads, smem, st>>>(dy, ds, x, xs, rows, n, g.tpr, w, wf32, stats, dx, part);
    };
    if (n > kNormRegCols) return go(k_norm_bwd<T, VEC, NV, true, true, false>, sums);
    auto with = [&](auto hull) {
        constexpr bool HULL = decltype(hull)::value;
        const size_t ring = kNormStages<T> * RowRing<T, VEC, NV, 2, true, HULL>::stage_bytes(n, g.threads, g.rpb);
        if (g.block) go(k_norm_bwd<T, VEC, NV, true, false, HULL>, ring);
        else go(k_norm_bwd<T, VEC, NV, false, false, HULL>, ring > sums ? ring : sums);
    };
    if constexpr (VEC * sizeof(T) < 16)
        if (g.hull) return with(std::true_type{});
    with(std::false_type{});
}

template <typename T>
void norm_backward(const NormGeom &g, int grid, const T *dy, long long ds, const T *x, long long xs,
                   long long rows, int n, const void *w, bool wf32, const float2 *stats, T *dx,
                   float *part, cudaStream_t st) {
    constexpr int V16 = 16 / (int)sizeof(T), V4 = 4 / (int)sizeof(T);
    if (g.vec == V16)
        return norm_bwd_launch<T, V16>(g, grid, dy, ds, x, xs, rows, n, w, wf32, stats, dx, part, st);
    if constexpr (V4 > 1)
        if (g.vec == V4)
            return norm_bwd_launch<T, V4>(g, grid, dy, ds, x, xs, rows, n, w, wf32, stats, dx, part, st);
    norm_bwd_launch<T, 1>(g, grid, dy, ds, x, xs, rows, n, w, wf32, stats, dx, part, st);
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" {

int sdm_layer_norm(const void *x, long long rows, int n, long long x_stride, const void *weight,
                   const void *bias, int weight_dtype, float eps, int dtype, void *y, float *stats,
                   void *stream) {
    const int rc = norm_check("layer norm", x, rows, n, x_stride, weight_dtype, dtype);
    if (rc != SDM_OK) return rc;
    if (!(eps >= 0.f)) return set_error(SDM_ERR_INVALID, "layer norm: eps must be >= 0");
    if (rows == 0) return SDM_OK;
    if (!y) return set_error(SDM_ERR_INVALID, "layer norm: NULL pointer");
    if ((uintptr_t)stats % 8) return set_error(SDM_ERR_INVALID, "layer norm: stats must be 8-byte aligned");
    const int es = dtype == SDM_BF16 ? 2 : 4;
    NormGeom g = norm_geom(n, norm_vec(es, n, x_stride, x_stride, x, y, y), false);
    g.hull = norm_hull(es, g.vec, n, x_stride, x);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto s2 = reinterpret_cast<float2 *>(stats);
    const bool wf32 = weight_dtype == SDM_F32;
    if (dtype == SDM_BF16)
        norm_forward(g, static_cast<const __nv_bfloat16 *>(x), x_stride, rows, n, weight, bias, wf32,
                     eps, static_cast<__nv_bfloat16 *>(y), s2, st);
    else
        norm_forward(g, static_cast<const float *>(x), x_stride, rows, n, weight, bias, wf32, eps,
                     static_cast<float *>(y), s2, st);
    return norm_status(cudaGetLastError());
}

size_t sdm_layer_norm_workspace_bytes(long long rows, int n) {
    if (rows < 0 || n < 1 || n > kNormMaxCols) {
        set_error(SDM_ERR_INVALID, "layer norm: bad sizes %lld, %d", rows, n);
        return 0;
    }
    const NormGeom g = norm_geom(n, 1, true);
    const size_t blocks = rows ? (size_t)norm_back_blocks(g, rows) : 1;
    return (blocks * 2 * n * 4 + kAlign - 1) / kAlign * kAlign;
}

int sdm_layer_norm_backward(const void *grad, long long grad_stride, const void *x,
                            long long x_stride, long long rows, int n, const void *weight,
                            int weight_dtype, const float *stats, int dtype, void *grad_x,
                            float *grad_weight, float *grad_bias, void *workspace,
                            size_t workspace_bytes, void *stream) {
    int rc = norm_check("layer norm backward", x, rows, n, x_stride, weight_dtype, dtype);
    if (rc != SDM_OK) return rc;
    if (grad_stride < 0)
        return set_error(SDM_ERR_INVALID, "layer norm backward: the gradient's row stride must be "
                         ">= 0, got %lld", grad_stride);
    if (rows > 0 && (!grad || !stats || !grad_x))
        return set_error(SDM_ERR_INVALID, "layer norm backward: NULL pointer");
    if (rows > 0 && (uintptr_t)stats % 8)
        return set_error(SDM_ERR_INVALID, "layer norm backward: stats must be 8-byte aligned");
    const bool sums = grad_weight || grad_bias;
    if (sums && (!workspace || workspace_bytes < sdm_layer_norm_workspace_bytes(rows, n) ||
                 (uintptr_t)workspace % kAlign))
        return set_error(SDM_ERR_WORKSPACE, "layer norm backward: workspace NULL, too small or not "
                         "%zu-byte aligned", (size_t)kAlign);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int es = dtype == SDM_BF16 ? 2 : 4;
    NormGeom g = norm_geom(n, norm_vec(es, n, x_stride, grad_stride, x, grad, grad_x), true);
    g.hull = norm_hull(es, g.vec, n, x_stride, x) && norm_hull(es, g.vec, n, grad_stride, grad);
    const int grid = rows ? norm_back_blocks(g, rows) : 0;
    float *part = sums ? static_cast<float *>(workspace) : nullptr;
    auto s2 = reinterpret_cast<const float2 *>(stats);
    const bool wf32 = weight_dtype == SDM_F32;
    if (rows > 0) {
        if (dtype == SDM_BF16)
            norm_backward(g, grid, static_cast<const __nv_bfloat16 *>(grad), grad_stride,
                          static_cast<const __nv_bfloat16 *>(x), x_stride, rows, n, weight, wf32, s2,
                          static_cast<__nv_bfloat16 *>(grad_x), part, st);
        else
            norm_backward(g, grid, static_cast<const float *>(grad), grad_stride,
                          static_cast<const float *>(x), x_stride, rows, n, weight, wf32, s2,
                          static_cast<float *>(grad_x), part, st);
    }
    if (sums)
        k_norm_cols<<<(2 * n + kNormColThreads - 1) / kNormColThreads, kNormColThreads * kNormColSlices,
                      0, st>>>(part, grid, n, grad_weight, grad_bias);
    return norm_status(cudaGetLastError());
}

}  // extern "C"
