// Group norm with an activation over [N, L, C], channels last: the statistics of a sample's group are over its L
// positions and C / G channels.
//   mean, rstd of the group;  xhat = (x - mean) rstd;  z = xhat w + b;  y = z, or z / (1 + e^-z)
//   dz = dy act'(z);  dx = rstd (w dz - mean(w dz) - xhat mean(w dz xhat));  dw = sum dz xhat;  db = sum dz
// All arithmetic is float32; y and dx are rounded once.
//
// Three forms. One position a sample (a token's heads): a group is a row of C / G elements, kept in registers, read
// once (k_group_row*): a row belongs to a part of a warp or to a block, blocks walk over the samples with a stride
// that keeps every thread at its group, so weights and column sums stay in registers. Small samples: several of them
// whole in a block's registers (k_group_small*). Else a sample's positions are split over blocks, each thread at its
// channels: a first launch makes every split's statistics (or column sums and terms), the second joins them, the third
// reads the rows again, from L2 where they fit.
#include <type_traits>

#include "norm_rows.cuh"
#include "pairs.cuh"

namespace sdm {
namespace {

constexpr int kGroupThreads = 256, kGroupSm = 3, kGroupBatch = 8, kGroupMaxCols = 16384, kGroupRowCols = 8192;
constexpr int kSmallMany = 4, kSmallBack = 2, kSmallBlocks = 2 * kRefSms;   // vectors a thread of small samples; the backward's blocks
// An SM's threads over rows, in blocks of several rows (rows as wide as a block and wider: 512, 16384 x 4096 bfloat16 in one
// group 61 us, one block of 256 113). With the activation the issue of instructions bounds them and more threads help as long
// as they fit the registers, without it memory does and fewer rows at once are read in better order. 32768 x 4096 in 32
// groups, forward: bfloat16 with silu 640 / 512 / 384 threads 95 / 89 / 101 us, without 98 / 98 / 85; half as many of float32 89 /
// 99 / 122 and 88 / 88 / 90. Backward: bfloat16 with silu 512 / 384 / 256 threads (up to 168 registers each, so 512 end in
// a second wave) 150 / 138 / 161 us, without 146 / 142 / 132; float32 176 / 133 / 178 and 131 / 129 / 131.
template <typename T>
constexpr int group_row_threads(bool block, bool act) {
    return block ? 512 : !act ? 384 : sizeof(T) == 4 ? 640 : 512;
}
int group_back_threads(bool block, bool act) { return block ? 512 : act ? 384 : 256; }

// The sigmoid. bfloat16: by the approximate exponential and reciprocal instructions, within 2^-20 of it where it is not
// negligible, far inside the results' rounding of 2^-8; the exact ones would bound the kernel (25 instructions an
// element). An infinite e^-z makes 0 of both.
template <typename T>
__device__ __forceinline__ float2 sigmoid(float2 z) {
    if constexpr (sizeof(T) == 2) {
        float2 e = mul2(z, both(-1.44269504089f)), p;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(e.x));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(e.y));
        e = add2(e, both(1.f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p.x) : "f"(e.x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p.y) : "f"(e.y));
        return p;
    } else {
        return make_float2(1.f / (1.f + expf(-z.x)), 1.f / (1.f + expf(-z.y)));
    }
}
template <typename T, bool ACT>
__device__ __forceinline__ float2 activate(float2 z) {
    return ACT ? mul2(z, sigmoid<T>(z)) : z;
}
// dy times the activation's slope at z
template <typename T, bool ACT>
__device__ __forceinline__ float2 back(float2 dy, float2 z) {
    if constexpr (!ACT) return dy;
    const float2 p = sigmoid<T>(z);
    return mul2(dy, mul2(p, fma2(z, fma2(p, both(-1.f), both(1.f)), both(1.f))));
}

// a running count, mean and sum of squares around it
struct Moments {
    float n, mean, m2;
    // those of nb values joined
    __device__ __forceinline__ void join(float nb, float mb, float qb) {
        if (n == 0.f) {                                  // (0 times a difference's square, which may be infinite)
            *this = Moments{nb, mb, qb};
            return;
        }
        const float d = mb - mean, f = __fdividef(nb, n + nb);   // (a weight's error moves the mean by 2^-22 of the difference)
        mean = fmaf(d, f, mean);
        m2 += fmaf(d * d, n * f, qb);
        n += nb;
    }
};
// The mean and the squares around it of `many` parts by LANES lanes: entry(i) is a part's count, mean and squares. In two
// passes, sums alone: joined one by one, each with a division, the parts of 76 blocks took 20 us.
template <int LANES, typename F>
__device__ __forceinline__ float2 join_parts(int many, float all, F entry) {
    const int lane = threadIdx.x % LANES;
    float sum = 0.f, q = 0.f;
#pragma unroll 4
    for (int i = lane; i < many; i += LANES) {
        const Moments p = entry(i);
        sum = fmaf(p.n, p.mean, sum);
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    const float mean = sum / all;
#pragma unroll 4
    for (int i = lane; i < many; i += LANES) {
        const Moments p = entry(i);
        const float d = p.mean - mean;
        q += p.n > 0.f ? fmaf(p.n * d, d, p.m2) : 0.f;
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) q += __shfl_xor_sync(~0u, q, o);
    return make_float2(mean, q);
}

struct GroupShape {
    long long N, L, xs, gs;              // samples, positions, elements between positions of x and of the gradient
    int C, G;
    bool wf32;
    float eps;
    const void *w, *b;
    int splits, more;                    // blocks of a sample: `per` positions each, the first `more` of them one more
    long long per;
    // into how many, and how
    void split(int n) {
        splits = n;
        per = L / n;
        more = (int)(L % n);
    }
};

// ---- one position a sample ----------------------------------------------------------------------

// What bounds these is the issue of instructions (the first form, one float at a time, took 25 an element, 125 us for
// 32768 x 4096 bfloat16 with the activation, where memory takes 80), so the arithmetic is in pairs and the addresses
// step along.

// The threads' own pieces of the rows ahead, as in the layer norm (RowRing): a thread copies NV vectors of each of ROWS
// tensors (and 8 bytes of statistics) into shared memory and reads them back itself.
template <typename T, int VEC, int NV, int ROWS, bool STATS>
struct GroupRing {
    static constexpr int ST = kNormStages<T>, VB = VEC * (int)sizeof(T), THREAD = ROWS * NV * VB + (STATS ? 8 : 0);
    static __host__ __device__ size_t bytes(int threads) { return (size_t)ST * THREAD * threads; }
    unsigned at, stage_bytes, read_at, write_at, end;
    int c, tpr, t;
    __device__ GroupRing(unsigned char *smem, int t_, int tpr_, int c_) : c(c_), tpr(tpr_), t(t_) {
        at = smem_u32(smem) + threadIdx.x * VB;
        stage_bytes = THREAD * blockDim.x;
        read_at = write_at = 0;
        end = ST * stage_bytes;
        // vectors past the row's end are never fetched
        for (int s = 0; s < ST; ++s)
            for (int i = 0; i < ROWS * NV; ++i)
                if ((i % NV * tpr + t) * VEC >= c)
                    *reinterpret_cast<Vec<T, VEC> *>(smem + threadIdx.x * VB + s * stage_bytes + i * VB * blockDim.x) = Vec<T, VEC>{};
    }
    // row `which` into the stage that is written next
    __device__ __forceinline__ void fetch(int which, const T *row) const {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((i * tpr + t) * VEC < c) {
                const unsigned to = at + write_at + (which * NV + i) * VB * blockDim.x;
                const T *src = row + (i * tpr + t) * VEC;
                if constexpr (VB == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
                else if constexpr (VB == 4) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(src) : "memory");
                else asm volatile("st.shared.b16 [%0], %1;" ::"r"(to), "h"(*reinterpret_cast<const unsigned short *>(src)) : "memory");
            }
    }
    __device__ __forceinline__ unsigned stats_at(unsigned stage) const { return at - threadIdx.x * VB + stage + (THREAD - 8) * blockDim.x + 8 * threadIdx.x; }
    __device__ __forceinline__ void fetch_stats(const float2 *p) const {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(stats_at(write_at)), "l"(p) : "memory");
    }
    __device__ __forceinline__ void fetched() {
        cp_async_commit();
        write_at = write_at + stage_bytes == end ? 0 : write_at + stage_bytes;
    }
    __device__ __forceinline__ void next() { read_at = read_at + stage_bytes == end ? 0 : read_at + stage_bytes; }
    __device__ __forceinline__ void read(int which, float2 (&o)[VEC * NV / 2]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const unsigned from = at + read_at + (which * NV + i) * VB * blockDim.x;
            Vec<T, VEC> r;
            if constexpr (VB == 16) asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(from) : "memory");
            else if constexpr (VB == 4) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(from) : "memory");
            else asm volatile("ld.shared.b16 %0, [%1];" : "=h"(r) : "r"(from) : "memory");
            unpack<T, VEC>(r, reinterpret_cast<float *>(o) + i * VEC);
        }
    }
    __device__ __forceinline__ float2 read_stats() const {
        float2 r;
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(r.x), "=f"(r.y) : "r"(stats_at(read_at)) : "memory");
        return r;
    }
};

// sums over a row's threads, a part of a warp or the block
template <bool BLOCK, int M>
__device__ __forceinline__ void group_sum(float (&v)[M], int tpr, float *red, int &turn) {
    if constexpr (BLOCK) {
        row_sum<true, M>(v, tpr, red, turn);
    } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (o < tpr)
#pragma unroll
                for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(~0u, v[m], o);
    }
}

template <typename T>
__device__ __forceinline__ float reciprocal_root(float x) {
    if constexpr (sizeof(T) == 2) return rsqrtf(x);                // (2 units in the last place of float32)
    return 1.f / sqrtf(x);
}

// NV vectors of a row at `row`
template <typename T, int VEC, int NV>
__device__ __forceinline__ void store_pairs(T *row, int t, int tpr, int c, const float2 (&v)[VEC * NV / 2]) {
    store_row<T, VEC, NV>(row, t, tpr, c, reinterpret_cast<const float *>(v));
}

template <typename T, int VEC, int NV, bool BLOCK, bool ACT>
__global__ void __launch_bounds__(BLOCK ? 512 : kNormBlock, group_row_threads<T>(BLOCK, ACT) / (BLOCK ? 512 : kNormBlock))
    k_group_row(const __grid_constant__ GroupShape s, const T *x, int tpr, T *y, float2 *stats) {
    constexpr int E = VEC * NV, ST = kNormStages<T>;
    extern __shared__ __align__(16) unsigned char ring_smem[];
    __shared__ float red[2 * 2 * 32];
    int turn = 0;
    const int sub = BLOCK ? 0 : threadIdx.x / tpr, t = BLOCK ? threadIdx.x : threadIdx.x % tpr, rpb = BLOCK ? 1 : kNormBlock / tpr;
    const int c = s.C / s.G;
    // (the rows at once are a multiple of G)
    const long long row0 = (long long)blockIdx.x * rpb + sub;
    const int step = (int)((long long)gridDim.x * rpb / s.G), g = (int)(row0 % s.G);
    int n = (int)(row0 / s.G), turns = (int)s.N - (int)((long long)blockIdx.x * rpb / s.G);   // (of the block: its first row's)
    float2 wv[E / 2], bv[E / 2];
    const size_t at = (size_t)g * c, ws = s.wf32 ? 4 : sizeof(T);
    load_cols<T, VEC, NV>(s.w ? static_cast<const char *>(s.w) + at * ws : nullptr, s.wf32, 1.f, t, tpr, c, reinterpret_cast<float *>(wv));
    load_cols<T, VEC, NV>(s.b ? static_cast<const char *>(s.b) + at * ws : nullptr, s.wf32, 0.f, t, tpr, c, reinterpret_cast<float *>(bv));
    GroupRing<T, VEC, NV, 1, false> ring(ring_smem, t, tpr, c);
    const T *src = x + n * s.xs + at;
    T *dst = y + (long long)n * s.C + at;
    const long long src_step = step * s.xs, dst_step = (long long)step * s.C;
    const int N = (int)s.N;
    int ahead = n;
    auto fetch = [&] {
        if (ahead < N) ring.fetch(0, src);
        ring.fetched();
        ahead += step;
        src += src_step;
    };
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) fetch();
    const float inv = 1.f / (float)c;
    for (; turns > 0; turns -= step, n += step, dst += dst_step) {
        fetch();
        cp_async_wait<ST - 1>();
        float2 v[E / 2], two = both(0.f);
        ring.read(0, v);
        ring.next();
#pragma unroll
        for (int j = 0; j < E / 2; ++j) two = add2(two, v[j]);
        float sum[1] = {two.x + two.y};
        group_sum<BLOCK, 1>(sum, tpr, red, turn);
        const float mean = sum[0] * inv;
        two = both(0.f);
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
            v[j] = add2(v[j], both(-mean));
            if constexpr (VEC > 1) {
                if ((j * 2 / VEC * tpr + t) * VEC < c) two = fma2(v[j], v[j], two);
            } else {
                if (2 * j * tpr + t < c) two.x = fmaf(v[j].x, v[j].x, two.x);
                if ((2 * j + 1) * tpr + t < c) two.y = fmaf(v[j].y, v[j].y, two.y);
            }
        }
        sum[0] = two.x + two.y;
        group_sum<BLOCK, 1>(sum, tpr, red, turn);
        const float rstd = reciprocal_root<T>(fmaf(sum[0], inv, s.eps));
        if (n < N) {
#pragma unroll
            for (int j = 0; j < E / 2; ++j) v[j] = activate<T, ACT>(fma2(mul2(v[j], both(rstd)), wv[j], bv[j]));
            store_pairs<T, VEC, NV>(dst, t, tpr, c, v);
            if (stats && t == 0) stats[(long long)n * s.G + g] = make_float2(mean, rstd);
        }
    }
}

// part [..][2][C]: column sums of dz xhat and of dz, of a block (same) or of each of its rows
template <typename T, int VEC, int NV, bool BLOCK, bool ACT>
__global__ void __launch_bounds__(BLOCK ? 512 : kNormBlock)
    k_group_row_bwd(const __grid_constant__ GroupShape s, const T *dy, const T *x, int tpr, bool same, const float2 *stats, T *dx, float *part) {
    constexpr int E = VEC * NV, ST = kNormStages<T>;
    extern __shared__ __align__(16) unsigned char ring_smem[];
    __shared__ float red[2 * 2 * 32];
    chain_next();
    int turn = 0;
    const int sub = BLOCK ? 0 : threadIdx.x / tpr, t = BLOCK ? threadIdx.x : threadIdx.x % tpr, rpb = BLOCK ? 1 : kNormBlock / tpr;
    const int c = s.C / s.G;
    // a block's rows are one group's of several samples, so that it adds their column sums itself; fewer samples than
    // that: as in the forward
    const long long row0 = (long long)blockIdx.x * rpb + sub;
    const int step = (int)((long long)gridDim.x * rpb / s.G), N = (int)s.N;
    const int first0 = (int)(same ? (long long)(blockIdx.x / s.G) * rpb : (long long)blockIdx.x * rpb / s.G);
    const int g = (int)(same ? blockIdx.x % s.G : row0 % s.G);
    int n = same ? first0 + sub : (int)(row0 / s.G);
    float2 wv[E / 2], bv[ACT ? E / 2 : 1], aw[E / 2], ab[E / 2];
    const size_t at = (size_t)g * c, ws = s.wf32 ? 4 : sizeof(T);
    load_cols<T, VEC, NV>(s.w ? static_cast<const char *>(s.w) + at * ws : nullptr, s.wf32, 1.f, t, tpr, c, reinterpret_cast<float *>(wv));
    if constexpr (ACT)
        load_cols<T, VEC, NV>(s.b ? static_cast<const char *>(s.b) + at * ws : nullptr, s.wf32, 0.f, t, tpr, c, reinterpret_cast<float *>(bv));
#pragma unroll
    for (int j = 0; j < E / 2; ++j) aw[j] = ab[j] = both(0.f);
    GroupRing<T, VEC, NV, 2, true> ring(ring_smem, t, tpr, c);
    const T *xp = x + n * s.xs + at, *gp = dy + n * s.gs + at;
    const float2 *sp = stats + (long long)n * s.G + g;
    T *dst = dx + (long long)n * s.C + at;
    const long long x_step = step * s.xs, g_step = step * s.gs, s_step = (long long)step * s.G, d_step = (long long)step * s.C;
    int ahead = n;
    auto fetch = [&] {
        if (ahead < N) {
            ring.fetch(0, xp);
            ring.fetch(1, gp);
            ring.fetch_stats(sp);
        }
        ring.fetched();
        ahead += step;
        xp += x_step;
        gp += g_step;
        sp += s_step;
    };
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) fetch();
    const float inv = 1.f / (float)c;
    for (int turns = N - first0; turns > 0; turns -= step, n += step, dst += d_step) {
        fetch();
        cp_async_wait<ST - 1>();
        const float2 ns = ring.read_stats();
        float2 h[E / 2], d[E / 2], s0 = both(0.f), s1 = both(0.f);
        ring.read(0, h);
        ring.read(1, d);
        ring.next();
        if (n < N) {                                               // (what a stage without a row holds is an earlier one)
#pragma unroll
            for (int j = 0; j < E / 2; ++j) {
                // past the row's end x and dy are 0, and dy = 0 keeps the sums clean
                h[j] = mul2(add2(h[j], both(-ns.x)), both(ns.y));
                if constexpr (ACT) d[j] = back<T, ACT>(d[j], fma2(h[j], wv[j], bv[j]));
                aw[j] = fma2(d[j], h[j], aw[j]);
                ab[j] = add2(ab[j], d[j]);
                d[j] = mul2(d[j], wv[j]);
                s0 = add2(s0, d[j]);
                s1 = fma2(d[j], h[j], s1);
            }
        }
        float sum[2] = {s0.x + s0.y, s1.x + s1.y};
        group_sum<BLOCK, 2>(sum, tpr, red, turn);
        const float2 c1 = both(-sum[0] * inv), c2 = both(-sum[1] * inv);
        if (n < N) {
#pragma unroll
            for (int j = 0; j < E / 2; ++j) d[j] = mul2(both(ns.y), fma2(h[j], c2, add2(d[j], c1)));
            store_pairs<T, VEC, NV>(dst, t, tpr, c, d);
        }
    }
    if (!part) return;
    cp_async_wait<0>();
    const float *sw = reinterpret_cast<const float *>(aw), *sb = reinterpret_cast<const float *>(ab);
    if (!BLOCK && same) {
        // the block's rows, added in their order: cols [2][rows][tpr E]
        __syncthreads();
        float *cols = reinterpret_cast<float *>(ring_smem);
        const int wide = tpr * E;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int col = (i * tpr + t) * VEC + j;
                cols[sub * wide + col] = sw[i * VEC + j];
                cols[(rpb + sub) * wide + col] = sb[i * VEC + j];
            }
        __syncthreads();
        float *out = part + (size_t)(blockIdx.x / s.G) * 2 * s.C + at;
        for (int col = threadIdx.x; col < c; col += kNormBlock) {
            float a = 0.f, b = 0.f;
            for (int r = 0; r < rpb; ++r) {
                a += cols[r * wide + col];
                b += cols[(rpb + r) * wide + col];
            }
            out[col] = a;
            out[s.C + col] = b;
        }
        return;
    }
    float *out = part + (size_t)(same ? blockIdx.x / s.G : row0 / s.G) * 2 * s.C + at;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int col = (i * tpr + t) * VEC + j;
            if (col < c) {
                out[col] = sw[i * VEC + j];
                out[s.C + col] = sb[i * VEC + j];
            }
        }
}

// ---- positions split over blocks ----------------------------------------------------------------

// A block's threads over a [positions][C] tile: CV = C / VEC vectors a position; up to kGroupThreads of them are taken
// side by side, with several positions (slots) where there are fewer.
struct Spread {
    int cv, slots;
    __device__ Spread(int C, int vec) : cv(C / vec), slots(cv < kGroupThreads ? kGroupThreads / cv : 1) {}
};
// this block's sample and positions
struct Piece {
    long long n, from, to;
    int split;
    __device__ explicit Piece(const GroupShape &s) {
        split = (int)(blockIdx.x % s.splits);
        n = blockIdx.x / s.splits;
        from = split * s.per + (split < s.more ? split : s.more);
        to = from + s.per + (split < s.more);
    }
};

template <typename T, int VEC>
__device__ __forceinline__ void load_params(const void *p, bool f32, float fill, int c0, float (&o)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
        o[j] = !p ? fill : f32 ? static_cast<const float *>(p)[c0 + j] : to_f32(static_cast<const T *>(p)[c0 + j]);
}

// The result may be x, or x's gradient y's: what a kernel overwrites itself it reads by plain loads (a read-only
// one may be moved behind the store), each vector before it stores there and no other thread's.

// The vectors of the kernels below are parts of a group, or (OWN) groups end inside them: then every channel has a group, a
// partial and statistics of its own.

// part [N][splits][G]: mean and sum of squares around it
template <typename T, int VEC, bool OWN>
__global__ void __launch_bounds__(kGroupThreads, kGroupSm) k_group_stats(const __grid_constant__ GroupShape s, const T *x, float2 *part) {
    extern __shared__ float2 acc[];                      // [slots][cv], of channels (OWN) [slots][C]
    chain_next();
    const Piece p(s);
    const Spread sp(s.C, VEC);
    const int at_slot = (int)threadIdx.x / sp.cv, slot = at_slot < sp.slots ? at_slot : -1;
    const T *base = x + p.n * s.L * s.xs;
    for (int cv = sp.slots > 1 ? threadIdx.x % sp.cv : threadIdx.x; cv < sp.cv; cv += kGroupThreads) {
        Moments m{0.f, 0.f, 0.f};
        float mean[OWN ? VEC : 1] = {}, m2[OWN ? VEC : 1] = {};
        if (slot >= 0 || sp.slots == 1) {
            const T *col = base + cv * VEC;
            for (long long r = p.from + (sp.slots > 1 ? slot : 0); r < p.to; r += (long long)sp.slots * kGroupBatch) {
                // (kept as they came: widened they would take the registers of another block)
                Vec<T, VEC> raw[kGroupBatch];
                float2 sum = both(0.f), q = both(0.f);
                float count = 0.f;
#pragma unroll
                for (int i = 0; i < kGroupBatch; ++i) {
                    const long long at = r + (long long)i * sp.slots;
                    raw[i] = Vec<T, VEC>{};
                    if (at < p.to) {
                        raw[i] = __ldg(reinterpret_cast<const Vec<T, VEC> *>(col + at * s.xs));
                        count += OWN ? 1 : VEC;
                    }
                }
                if constexpr (OWN) {                               // as below, a channel at a time
                    const float f = __fdividef(count, m.n + count), by = 1.f / count;
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        float v[kGroupBatch], t = 0.f, q = 0.f;
#pragma unroll
                        for (int i = 0; i < kGroupBatch; ++i) {
                            v[i] = to_f32(reinterpret_cast<const T *>(raw + i)[j]);
                            t += v[i];
                        }
                        t *= by;
#pragma unroll
                        for (int i = 0; i < kGroupBatch; ++i)
                            if (r + (long long)i * sp.slots < p.to) q = fmaf(v[i] - t, v[i] - t, q);
                        const float d = m.n > 0.f ? t - mean[j] : 0.f;
                        mean[j] = m.n > 0.f ? fmaf(d, f, mean[j]) : t;
                        m2[j] += fmaf(d * d, m.n * f, q);
                    }
                    m.n += count;
                    continue;
                }
                auto each_pair = [&](auto f) {
#pragma unroll
                    for (int i = 0; i < kGroupBatch; ++i) {
                        float v[VEC];
                        unpack<T, VEC>(raw[i], v);
#pragma unroll
                        for (int j = 0; j < VEC; j += 2) f(r + (long long)i * sp.slots < p.to, make_float2(v[j], VEC > 1 ? v[VEC > 1 ? j + 1 : 0] : 0.f));
                    }
                };
                each_pair([&](bool, float2 v) { sum = add2(sum, v); });
                const float mean = (sum.x + sum.y) / count;
                each_pair([&](bool live, float2 v) {
                    const float2 d = add2(v, both(-mean));
                    if (live) q = fma2(d, d, q);
                });
                if (VEC == 1) q.y = 0.f;                           // (no second one of the pair)
                m.join(count, mean, q.x + q.y);
            }
        }
        if (slot >= 0 || sp.slots == 1) {
            const int at = (sp.slots > 1 ? slot : 0) * sp.cv + cv;
            if constexpr (OWN)
#pragma unroll
                for (int j = 0; j < VEC; ++j) acc[at * VEC + j] = make_float2(mean[j], m2[j]);
            else acc[at] = make_float2(m.mean, m.m2);
        }
        if (sp.slots > 1) break;
    }
    __syncthreads();
    constexpr int PART = OWN ? 1 : VEC;                            // channels of a partial
    const int each = s.C / PART / s.G, line = s.C / PART;
    const long long rows = p.to - p.from;
    const float all = (float)rows * (float)(s.C / s.G);
    for (int g0 = 0; g0 < s.G; g0 += kGroupThreads / 8) {
        const int g = g0 + (threadIdx.x >> 3);
        const float2 a = join_parts<8>(g < s.G ? each * sp.slots : 0, all, [&](int i) {
            const int sl = i / each;
            const float2 e = acc[sl * line + g * each + i % each];
            return Moments{(float)((rows > sl ? (rows - sl + sp.slots - 1) / sp.slots : 0) * PART), e.x, e.y};
        });
        if (g < s.G && (threadIdx.x & 7) == 0) part[((size_t)p.n * s.splits + p.split) * s.G + g] = a;
    }
}

// joined [N][G] mean and rstd from the splits', a warp a group
__global__ void __launch_bounds__(kGroupThreads) k_group_join(const __grid_constant__ GroupShape s, const float2 *part, float2 *joined) {
    const long long i = (long long)blockIdx.x * (kGroupThreads / 32) + (threadIdx.x >> 5);
    chain_wait();
    chain_next();
    if (i >= s.N * s.G) return;
    const float c = (float)(s.C / s.G), all = (float)s.L * c;
    const float2 *at = part + i / s.G * s.splits * s.G + i % s.G;
    const float2 a = join_parts<32>(s.splits, all, [&](int k) {
        const float2 e = __ldcg(at + (size_t)k * s.G);
        return Moments{(float)(s.per + (k < s.more)) * c, e.x, e.y};
    });
    if ((threadIdx.x & 31) == 0) joined[i] = make_float2(a.x, 1.f / sqrtf(a.y / all + s.eps));
}

template <typename T, int VEC, bool OWN, bool ACT>
__global__ void __launch_bounds__(kGroupThreads, OWN ? 2 : kGroupSm) k_group_apply(const __grid_constant__ GroupShape s, const T *x, const float2 *stats, T *y) {
    const Piece p(s);
    const Spread sp(s.C, VEC);
    const int slot = sp.slots > 1 ? threadIdx.x / sp.cv : 0, each = s.C / s.G;
    const int cv0 = sp.slots > 1 ? threadIdx.x % sp.cv : threadIdx.x, wide = sp.slots > 1 ? sp.cv : kGroupThreads;
    if (slot >= sp.slots) return;
    const T *base = x + p.n * s.L * s.xs;
    T *out = y + p.n * s.L * s.C;
    Vec<T, VEC> raw[kGroupBatch];
    auto fetch = [&](long long r, int c0) {
#pragma unroll
        for (int i = 0; i < kGroupBatch; ++i) {
            const long long at = r + (long long)i * sp.slots;
            if (at < p.to) raw[i] = *reinterpret_cast<const Vec<T, VEC> *>(base + at * s.xs + c0);
        }
    };
    for (int cv = cv0; cv < sp.cv; cv += wide) {
        const int c0 = cv * VEC;
        fetch(p.from + slot, c0);
        float w[VEC], b[VEC];
        load_params<T, VEC>(s.w, s.wf32, 1.f, c0, w);
        load_params<T, VEC>(s.b, s.wf32, 0.f, c0, b);
        chain_wait();
        float2 a[OWN ? VEC : 1];
#pragma unroll
        for (int j = 0; j < (OWN ? VEC : 1); ++j) a[j] = stats[p.n * s.G + (c0 + j) / each];
        for (long long r = p.from + slot; r < p.to; r += (long long)sp.slots * kGroupBatch) {
#pragma unroll
            for (int i = 0; i < kGroupBatch; ++i) {
                const long long at = r + (long long)i * sp.slots;
                if (at >= p.to) continue;
                float v[VEC];
                unpack<T, VEC>(raw[i], v);
                const long long next = at + (long long)sp.slots * kGroupBatch;
                if (next < p.to) raw[i] = *reinterpret_cast<const Vec<T, VEC> *>(base + next * s.xs + c0);
#pragma unroll
                for (int j = 0; j < VEC; j += 2) {
                    float2 z = make_float2(v[j], j + 1 < VEC ? v[j + 1] : 0.f);
                    if constexpr (OWN) z = mul2(add2(z, make_float2(-a[j].x, -a[j + 1].x)), make_float2(a[j].y, a[j + 1].y));
                    else z = mul2(add2(z, both(-a[0].x)), both(a[0].y));
                    z = activate<T, ACT>(fma2(z, make_float2(w[j], j + 1 < VEC ? w[j + 1] : 0.f), make_float2(b[j], j + 1 < VEC ? b[j + 1] : 0.f)));
                    v[j] = z.x;
                    if (j + 1 < VEC) v[j + 1] = z.y;
                }
                store_vec<T, VEC>(out + at * s.C + c0, v);
            }
        }
    }
}

// part [N][splits][2][C], where it is wanted: column sums of dz xhat and of dz; terms [N][splits][G]: sums over a group of
// w dz and of w dz xhat
template <typename T, int VEC, bool OWN, bool ACT>
__global__ void __launch_bounds__(kGroupThreads, OWN ? 2 : kGroupSm)
    k_group_sums(const __grid_constant__ GroupShape s, const T *dy, const T *x, const float2 *stats, float *part, float2 *terms) {
    extern __shared__ __align__(16) float sums[];        // [slots][2][C] where there are several slots; then [slots][cv] a thread's terms
    chain_next();
    const Piece p(s);
    const Spread sp(s.C, VEC);
    const int slot = sp.slots > 1 ? threadIdx.x / sp.cv : 0, each = s.C / s.G;
    const T *base = x + p.n * s.L * s.xs, *gbase = dy + p.n * s.L * s.gs;
    float2 *pairs = reinterpret_cast<float2 *>(sums + (sp.slots > 1 ? sp.slots * 2 * s.C : 0));
    float *out = part ? part + ((size_t)p.n * s.splits + p.split) * 2 * s.C : nullptr;
    if (slot < sp.slots)
        for (int cv = sp.slots > 1 ? threadIdx.x % sp.cv : threadIdx.x; cv < sp.cv; cv += sp.slots > 1 ? sp.cv : kGroupThreads) {
            const int c0 = cv * VEC;
            float2 a[OWN ? VEC : 1];
#pragma unroll
            for (int j = 0; j < (OWN ? VEC : 1); ++j) a[j] = stats[p.n * s.G + (c0 + j) / each];
            float w[VEC], b[VEC], sw[VEC], sb[VEC];
            load_params<T, VEC>(s.w, s.wf32, 1.f, c0, w);
            load_params<T, VEC>(s.b, s.wf32, 0.f, c0, b);
#pragma unroll
            for (int j = 0; j < VEC; ++j) sw[j] = sb[j] = 0.f;
            constexpr int BATCH = VEC == 8 && ACT ? 2 : 4;   // (8 x 4096 x 512 bfloat16: 25 us, with 4, which spill, 33; without silu 23, 20)
            for (long long r = p.from + slot; r < p.to; r += (long long)sp.slots * BATCH) {
                Vec<T, VEC> rx[BATCH], rg[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const long long at = r + (long long)i * sp.slots;
                    rx[i] = rg[i] = Vec<T, VEC>{};
                    if (at < p.to) {
                        rx[i] = __ldg(reinterpret_cast<const Vec<T, VEC> *>(base + at * s.xs + c0));
                        rg[i] = __ldg(reinterpret_cast<const Vec<T, VEC> *>(gbase + at * s.gs + c0));
                    }
                }
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    float h[VEC], d[VEC];
                    unpack<T, VEC>(rx[i], h);
                    unpack<T, VEC>(rg[i], d);
#pragma unroll
                    for (int j = 0; j < VEC; j += 2) {   // where no position is, dy is 0
                        constexpr bool TWO = VEC > 1;
                        float2 z = make_float2(h[j], TWO ? h[j + 1] : 0.f);
                        if constexpr (OWN) z = mul2(add2(z, make_float2(-a[j].x, -a[j + 1].x)), make_float2(a[j].y, a[j + 1].y));
                        else z = mul2(add2(z, both(-a[0].x)), both(a[0].y));
                        const float2 t = back<T, ACT>(make_float2(d[j], TWO ? d[j + 1] : 0.f),
                                                      fma2(z, make_float2(w[j], TWO ? w[j + 1] : 0.f), make_float2(b[j], TWO ? b[j + 1] : 0.f)));
                        sw[j] = fmaf(t.x, z.x, sw[j]);
                        sb[j] += t.x;
                        if constexpr (TWO) {
                            sw[j + 1] = fmaf(t.y, z.y, sw[j + 1]);
                            sb[j + 1] += t.y;
                        }
                    }
                }
            }
            float2 mine = both(0.f);
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if constexpr (OWN) pairs[slot * s.C + c0 + j] = make_float2(sb[j] * w[j], sw[j] * w[j]);
                else mine = fma2(make_float2(sb[j], sw[j]), both(w[j]), mine);
            if (out) {
                float *to = (sp.slots > 1 ? sums + (size_t)slot * 2 * s.C : out) + c0;
                store_vec<float, VEC>(to, sw);
                store_vec<float, VEC>(to + s.C, sb);
            }
            if constexpr (!OWN) pairs[slot * sp.cv + cv] = mine;
        }
    __syncthreads();
    const int line = OWN ? s.C : sp.cv, wide = line / s.G;
    for (int g0 = 0; g0 < s.G; g0 += kGroupThreads / 8) {
        const int g = g0 + (threadIdx.x >> 3);
        float2 a = both(0.f);
        if (g < s.G)
            for (int i = threadIdx.x & 7; i < wide * sp.slots; i += 8) a = add2(a, pairs[i / wide * line + g * wide + i % wide]);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) a = add2(a, make_float2(__shfl_xor_sync(~0u, a.x, o), __shfl_xor_sync(~0u, a.y, o)));
        if (g < s.G && (threadIdx.x & 7) == 0) terms[((size_t)p.n * s.splits + p.split) * s.G + g] = a;
    }
    if (sp.slots == 1 || !out) return;
    for (int c = threadIdx.x; c < 2 * s.C; c += kGroupThreads) {
        float t = 0.f;
        for (int i = 0; i < sp.slots; ++i) t += sums[(size_t)i * 2 * s.C + c];
        out[c] = t;
    }
}

// terms [N][G]: means over the group from the splits' sums, a warp a group; and in blocks behind those the column sums of
// all samples' splits (norm_cols), where they are wanted: a launch of their own was 5 us of the backward of 8 x 4096 x 512.
// (8 groups a block: as many as it has warps, 32, make one block of 32 groups of 456 splits, 9.4 us.)
constexpr int kGroupTermThreads = kNormColThreads * kNormColSlices, kGroupTermWarps = 8;
__global__ void __launch_bounds__(kGroupTermThreads) k_group_terms(const __grid_constant__ GroupShape s, const float2 *part, float2 *terms, int blocks,
                                                                   const float *cols, float *dw, float *db) {
    chain_wait();
    chain_next();
    if ((int)blockIdx.x >= blocks) return norm_cols(blockIdx.x - blocks, cols, (int)(s.N * s.splits), s.C, dw, db);
    const long long i = (long long)blockIdx.x * kGroupTermWarps + (threadIdx.x >> 5);
    if (threadIdx.x >= 32 * kGroupTermWarps || i >= s.N * s.G) return;
    const float2 *at = part + i / s.G * s.splits * s.G + i % s.G;
    float2 a = both(0.f);
#pragma unroll 4
    for (int k = threadIdx.x & 31; k < s.splits; k += 32) a = add2(a, __ldcg(at + (size_t)k * s.G));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = add2(a, make_float2(__shfl_xor_sync(~0u, a.x, o), __shfl_xor_sync(~0u, a.y, o)));
    const float count = (float)s.L * (float)(s.C / s.G);
    if ((threadIdx.x & 31) == 0) terms[i] = make_float2(a.x / count, a.y / count);
}

template <typename T, int VEC, bool OWN, bool ACT>
__global__ void __launch_bounds__(kGroupThreads, OWN ? 2 : kGroupSm)
    k_group_apply_bwd(const __grid_constant__ GroupShape s, const T *dy, const T *x, const float2 *stats, const float2 *terms, T *dx) {
    const Piece p(s);
    const Spread sp(s.C, VEC);
    const int slot = sp.slots > 1 ? threadIdx.x / sp.cv : 0, each = s.C / s.G;
    if (slot >= sp.slots) return;
    const T *base = x + p.n * s.L * s.xs, *gbase = dy + p.n * s.L * s.gs;
    T *out = dx + p.n * s.L * s.C;
    for (int cv = sp.slots > 1 ? threadIdx.x % sp.cv : threadIdx.x; cv < sp.cv; cv += sp.slots > 1 ? sp.cv : kGroupThreads) {
        const int c0 = cv * VEC;
        float w[VEC], b[VEC];
        load_params<T, VEC>(s.w, s.wf32, 1.f, c0, w);
        load_params<T, VEC>(s.b, s.wf32, 0.f, c0, b);
        chain_wait();
        float2 a[OWN ? VEC : 1], m[OWN ? VEC : 1];
#pragma unroll
        for (int j = 0; j < (OWN ? VEC : 1); ++j) {
            a[j] = stats[p.n * s.G + (c0 + j) / each];
            m[j] = __ldcg(terms + p.n * s.G + (c0 + j) / each);
        }
        constexpr int BATCH = 4;
        for (long long r = p.from + slot; r < p.to; r += (long long)sp.slots * BATCH) {
            Vec<T, VEC> rx[BATCH], rg[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const long long at = r + (long long)i * sp.slots;
                if (at < p.to) {
                    rx[i] = *reinterpret_cast<const Vec<T, VEC> *>(base + at * s.xs + c0);
                    rg[i] = *reinterpret_cast<const Vec<T, VEC> *>(gbase + at * s.gs + c0);
                }
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const long long at = r + (long long)i * sp.slots;
                if (at >= p.to) continue;
                float h[VEC], d[VEC];
                unpack<T, VEC>(rx[i], h);
                unpack<T, VEC>(rg[i], d);
#pragma unroll
                for (int j = 0; j < VEC; j += 2) {
                    constexpr bool TWO = VEC > 1;
                    const float2 wj = make_float2(w[j], TWO ? w[j + 1] : 0.f);
                    constexpr int J = OWN ? 1 : 0;                 // (the pair's statistics: their own or the vector's)
                    const float2 a0 = a[J * j], a1 = a[J * (j + 1)], m0 = m[J * j], m1 = m[J * (j + 1)];
                    const float2 rstd = make_float2(a0.y, a1.y);
                    const float2 z = mul2(add2(make_float2(h[j], TWO ? h[j + 1] : 0.f), make_float2(-a0.x, -a1.x)), rstd);
                    float2 t = mul2(back<T, ACT>(make_float2(d[j], TWO ? d[j + 1] : 0.f), fma2(z, wj, make_float2(b[j], TWO ? b[j + 1] : 0.f))), wj);
                    t = mul2(rstd, fma2(z, make_float2(-m0.y, -m1.y), add2(t, make_float2(-m0.x, -m1.x))));
                    d[j] = t.x;
                    if constexpr (TWO) d[j + 1] = t.y;
                }
                store_vec<T, VEC>(out + at * s.C + c0, d);
            }
        }
    }
}

// ---- small samples ------------------------------------------------------------------------------

// Samples of a few vectors: a block takes several whole ones into registers, MANY vectors a thread, so that they are read
// once and one launch does all. A thread's vectors lie at the same channels in every turn.
template <typename T, int VEC, int MANY>
struct Small {
    int cv, vectors, ev, all;            // vectors of a position, of a sample, of a group's channels; of the block's samples
    long long from[MANY];                // this thread's, from the block's first sample on, in x
    int at[MANY];                        // sample of the block and group, (.. G + g); -1: none
    __device__ Small(const GroupShape &s, int samples)
        : cv(s.C / VEC), vectors((int)s.L * cv), ev(cv / s.G), all(samples * vectors) {
#pragma unroll
        for (int k = 0; k < MANY; ++k) {
            const int i = (int)threadIdx.x + k * kGroupThreads, n = i / vectors, v = i % vectors;
            from[k] = (n * s.L + v / cv) * s.xs + v % cv * VEC;
            at[k] = i < all ? n * s.G + v % cv / ev : -1;
        }
    }
    // a sample's group, e-th vector
    __device__ __forceinline__ int entry(int n, int g, int e) const { return n * vectors + e / ev * cv + g * ev + e % ev; }
};

template <typename T, int VEC, bool ACT>
__global__ void __launch_bounds__(kGroupThreads, 2) k_group_small(const __grid_constant__ GroupShape s, const T *x, int samples, T *y, float2 *stats) {
    extern __shared__ float2 acc[];                      // [vectors] mean and squares around it; [samples][G] mean and rstd
    const Small<T, VEC, kSmallMany> m(s, samples);
    float2 *joined = acc + m.all;
    const float all = (float)s.L * (float)(s.C / s.G);
    for (long long n0 = (long long)blockIdx.x * samples; n0 < s.N; n0 += (long long)gridDim.x * samples) {
        const T *base = x + n0 * s.L * s.xs;
        const int live = (int)(s.N - n0 < samples ? s.N - n0 : samples) * s.G;
        Vec<T, VEC> raw[kSmallMany];
#pragma unroll
        for (int k = 0; k < kSmallMany; ++k)
            raw[k] = m.at[k] >= 0 && m.at[k] < live ? *reinterpret_cast<const Vec<T, VEC> *>(base + m.from[k]) : Vec<T, VEC>{};
#pragma unroll
        for (int k = 0; k < kSmallMany; ++k) {
            float v[VEC], mean = 0.f, q = 0.f;
            unpack<T, VEC>(raw[k], v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) mean += v[j];
            mean *= 1.f / VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) q = fmaf(v[j] - mean, v[j] - mean, q);
            if (m.at[k] >= 0) acc[threadIdx.x + k * kGroupThreads] = make_float2(mean, VEC > 1 ? q : 0.f);
        }
        __syncthreads();
        for (int p0 = 0; p0 < live; p0 += kGroupThreads / 8) {
            const int p = p0 + (int)(threadIdx.x >> 3), n = p / s.G, g = p % s.G;
            const float2 a = join_parts<8>(p < live ? (int)s.L * m.ev : 0, all, [&](int e) {
                const float2 part = acc[m.entry(n, g, e)];
                return Moments{(float)VEC, part.x, part.y};
            });
            if (p < live && (threadIdx.x & 7) == 0) {
                joined[p] = make_float2(a.x, 1.f / sqrtf(a.y / all + s.eps));
                if (stats) stats[n0 * s.G + p] = joined[p];
            }
        }
        __syncthreads();
        T *out = y + n0 * s.L * s.C;
#pragma unroll
        for (int k = 0; k < kSmallMany; ++k) {
            if (m.at[k] < 0 || m.at[k] >= live) continue;
            const int i = threadIdx.x + k * kGroupThreads;
            const float2 a = joined[m.at[k]];
            float v[VEC], w[VEC], b[VEC];
            unpack<T, VEC>(raw[k], v);
            load_params<T, VEC>(s.w, s.wf32, 1.f, i % m.cv * VEC, w);
            load_params<T, VEC>(s.b, s.wf32, 0.f, i % m.cv * VEC, b);
#pragma unroll
            for (int j = 0; j < VEC; j += 2) {
                constexpr bool TWO = VEC > 1;
                float2 z = mul2(add2(make_float2(v[j], TWO ? v[j + 1] : 0.f), both(-a.x)), both(a.y));
                z = activate<T, ACT>(fma2(z, make_float2(w[j], TWO ? w[j + 1] : 0.f), make_float2(b[j], TWO ? b[j + 1] : 0.f)));
                v[j] = z.x;
                if constexpr (TWO) v[j + 1] = z.y;
            }
            store_vec<T, VEC>(out + (long long)i * VEC, v);
        }
    }
}

// part [blocks][2][C], where it is wanted: column sums of dz xhat and of dz
template <typename T, int VEC, bool ACT>
__global__ void __launch_bounds__(kGroupThreads, 2)
    k_group_small_bwd(const __grid_constant__ GroupShape s, const T *dy, const T *x, int samples, const float2 *stats, T *dx, float *part) {
    // [vectors] terms, [samples][G] their means; in the end [2][vectors][VEC], sums
    extern __shared__ __align__(16) float2 terms[];
    chain_next();
    const Small<T, VEC, kSmallBack> m(s, samples);
    float2 *means = terms + m.all;
    const float count = (float)s.L * (float)(s.C / s.G);
    float sw[kSmallBack][VEC], sb[kSmallBack][VEC];
#pragma unroll
    for (int k = 0; k < kSmallBack; ++k)
#pragma unroll
        for (int j = 0; j < VEC; ++j) sw[k][j] = sb[k][j] = 0.f;
    for (long long n0 = (long long)blockIdx.x * samples; n0 < s.N; n0 += (long long)gridDim.x * samples) {
        const T *base = x + n0 * s.L * s.xs, *gbase = dy + n0 * s.L * s.gs;
        const int live = (int)(s.N - n0 < samples ? s.N - n0 : samples) * s.G;
        float h[kSmallBack][VEC], d[kSmallBack][VEC];      // xhat and w dz
        float2 a[kSmallBack];
#pragma unroll
        for (int k = 0; k < kSmallBack; ++k) {
            const int i = threadIdx.x + k * kGroupThreads, v = i % m.vectors;
            Vec<T, VEC> rx{}, rg{};
            a[k] = both(0.f);
            if (m.at[k] >= 0 && m.at[k] < live) {
                rx = *reinterpret_cast<const Vec<T, VEC> *>(base + m.from[k]);
                rg = *reinterpret_cast<const Vec<T, VEC> *>(gbase + (i / m.vectors * s.L + v / m.cv) * s.gs + v % m.cv * VEC);
                a[k] = stats[n0 * s.G + m.at[k]];
            }
            unpack<T, VEC>(rx, h[k]);
            unpack<T, VEC>(rg, d[k]);
        }
#pragma unroll
        for (int k = 0; k < kSmallBack; ++k) {
            const int i = threadIdx.x + k * kGroupThreads;
            if (m.at[k] < 0) continue;
            float w[VEC], b[VEC];
            load_params<T, VEC>(s.w, s.wf32, 1.f, i % m.cv * VEC, w);
            load_params<T, VEC>(s.b, s.wf32, 0.f, i % m.cv * VEC, b);
            float2 mine = both(0.f);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                h[k][j] = (h[k][j] - a[k].x) * a[k].y;
                const float t = back<T, ACT>(make_float2(d[k][j], 0.f), make_float2(fmaf(h[k][j], w[j], b[j]), 0.f)).x;
                sw[k][j] = fmaf(t, h[k][j], sw[k][j]);
                sb[k][j] += t;
                d[k][j] = t * w[j];
                mine = fma2(make_float2(1.f, h[k][j]), both(d[k][j]), mine);
            }
            terms[i] = mine;
        }
        __syncthreads();
        for (int p0 = 0; p0 < live; p0 += kGroupThreads / 8) {
            const int p = p0 + (int)(threadIdx.x >> 3), n = p / s.G, g = p % s.G;
            float2 t = both(0.f);
            if (p < live)
                for (int e = threadIdx.x & 7; e < (int)s.L * m.ev; e += 8) t = add2(t, terms[m.entry(n, g, e)]);
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) t = add2(t, make_float2(__shfl_xor_sync(~0u, t.x, o), __shfl_xor_sync(~0u, t.y, o)));
            if (p < live && (threadIdx.x & 7) == 0) means[p] = make_float2(t.x / count, t.y / count);
        }
        __syncthreads();
        T *out = dx + n0 * s.L * s.C;
#pragma unroll
        for (int k = 0; k < kSmallBack; ++k) {
            if (m.at[k] < 0 || m.at[k] >= live) continue;
            const float2 t = means[m.at[k]];
#pragma unroll
            for (int j = 0; j < VEC; ++j) d[k][j] = a[k].y * fmaf(-h[k][j], t.y, d[k][j] - t.x);
            store_vec<T, VEC>(out + (long long)(threadIdx.x + k * kGroupThreads) * VEC, d[k]);
        }
    }
    if (!part) return;
    float *cols = reinterpret_cast<float *>(terms);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSmallBack; ++k) {
        const int i = threadIdx.x + k * kGroupThreads;
        if (m.at[k] < 0) continue;
        store_vec<float, VEC>(cols + (long long)i * VEC, sw[k]);
        store_vec<float, VEC>(cols + (long long)(m.all + i) * VEC, sb[k]);
    }
    __syncthreads();
    float *out = part + (size_t)blockIdx.x * 2 * s.C;
    for (int c = threadIdx.x; c < 2 * s.C; c += kGroupThreads) {
        const float *from = cols + (c < s.C ? c : m.all * VEC + c - s.C);
        float t = 0.f;
        for (int i = 0; i < m.all * VEC; i += s.C) t += from[i];
        out[c] = t;
    }
}

// ---- which form, and its launches ---------------------------------------------------------------

// Blocks of a sample: kGroupSm an SM in all, 8 positions at least each. kGroupSm 3, of 80 registers: 8 x 4096 x 512 bfloat16
// with silu 25 us and backward 47; 4, with spills, 29; 2, of 128 registers, 28 and 72. At least 8 / 16 / 32 positions, forward
// and backward: 2 x 64 x 1280 10.2, 15.5 / 12.8, 21.0 / 18.0, 31.8 us; 8 x 256 x 512 11.1, 14.2 / 10.3, 13.6 / 11.0, 16.1.
int group_splits(long long N, long long L) {
    const long long want = (long long)kGroupSm * kRefSms / (N ? N : 1), most = L / 8;
    const long long s = want < most ? want : most;
    return s < 1 ? 1 : (int)s;
}

// The rows' blocks: a multiple of as many as make their rows at once a multiple of G, at most `most` where that allows it
long long group_grid(long long rows, int rpb, int G, long long most) {
    int a = rpb, b = G;
    while (b) {
        const int r = a % b;
        a = b;
        b = r;
    }
    const long long unit = G / a, need = ((rows + rpb - 1) / rpb + unit - 1) / unit, fit = most / unit;
    return unit * (need < fit ? need : fit > 1 ? fit : 1);
}

// Rows in registers wherever they fit: 32768 x 4096 bfloat16 of 32 groups with silu 87 us forward and 136 backward (the split
// form, one position a block: 365 and 464), half as many 46 and 72 (188 and 242), 1024 x 8192 of 8 10 and 32 (31 and 80). The
// registers end at 8192 columns (512 threads of 16 elements).
bool group_rows(long long L, int each) { return L == 1 && each <= kGroupRowCols; }
// Samples that a block of `many` vectors a thread takes whole, in one launch; 0: they are too large. Wherever they fit,
// forward and backward: 31337 x 10 x 8 bfloat16 15 and 17 us (split, a block a sample: 754 and 482), 1000 x 8 x 512 15 and 18
// (27 and 36), 300 x 9 x 40 4.6 and 7.0 (9.5 and 9.1).
int group_small(long long N, long long L, int C, int vec, int many) {
    const long long vectors = L * (C / vec), fit = many * kGroupThreads / (vectors ? vectors : 1), spread = (N + kSmallBlocks - 1) / kSmallBlocks;
    return (int)(fit < spread ? fit : spread);
}

// The backward's blocks over rows, and how many partials of the column sums they leave. `same`: all rows of a block are
// of one group and joined before they leave, as soon as there are samples enough for a block (32768 x 256 of 16 groups 29 us,
// by rows side by side, each with its own partial, 37; 200000 x 64 of one group 23 and 57; 1024 x 4096 of 32 13.6 and 19.7).
struct GroupBack {
    bool same;
    long long blocks, parts;
};
GroupBack group_back(const NormGeom &g, long long N, int G, bool act) {
    const int per_sm = group_back_threads(g.block, act) / g.threads;
    const long long few = N * G / g.rpb / kNormRowsBlock;
    const long long fill = (long long)kRefSms * per_sm, most = few > kRefSms ? few : kRefSms, cap = fill < most ? fill : most;
    if (N < g.rpb) {
        const long long blocks = group_grid(N * G, g.rpb, G, cap);
        return {false, blocks, blocks * g.rpb / G};
    }
    const long long need = (N + g.rpb - 1) / g.rpb, fit = cap / G, parts = need < fit ? need : fit > 1 ? fit : 1;
    return {true, parts * G, parts};
}

// (what any kernel may take, 48 KB with its own arrays, needs no call)
template <typename K>
void group_smem(K kern, size_t bytes) {
    if (bytes > 40 * 1024) set_kernel_smem(kern, bytes);
}

// The launches below return the first error, and none follows a launch that failed: it would read what that one has not
// written.
template <typename T, typename F>
cudaError_t group_by_vec(int vec, F f) {
    constexpr int V16 = 16 / (int)sizeof(T), V4 = 4 / (int)sizeof(T);
    if (vec == V16) return f(std::integral_constant<int, V16>{});
    if constexpr (V4 > 1)
        if (vec == V4) return f(std::integral_constant<int, V4>{});
    return f(std::integral_constant<int, 1>{});
}

// Whether channels have statistics of their own, so that the loads are wide: a block's end costs more then, so it pays from 16
// rows a thread on. Forward and backward, so and by narrow vectors: 24 rows, 2 x 16384 x 640 bfloat16 in 32 groups 47 and 88 us
// (63 and 96), 8 x 4096 x 320 float32 37 and 72 (73 and 106); 12 rows, the latter in bfloat16 28 and 46 (25 and 40); 4 rows,
// 8 x 4096 x 128 20 and 28 (14 and 18).
bool group_own(const GroupShape &s, int vec) {
    const int cv = s.C / vec;
    return s.per >= 16LL * (cv < kGroupThreads ? kGroupThreads / cv : 1);
}

template <typename T, int VEC, bool OWN, bool ACT>
cudaError_t group_forward_split(const GroupShape &s, const T *x, T *y, float2 *stats, float2 *part, cudaStream_t st) {
    const int cv = s.C / VEC, slots = cv < kGroupThreads ? kGroupThreads / cv : 1;
    const unsigned grid = (unsigned)(s.N * s.splits);
    const size_t smem = (size_t)slots * cv * (OWN ? VEC : 1) * 8;
    group_smem(k_group_stats<T, VEC, OWN>, smem);
    k_group_stats<T, VEC, OWN><<<grid, kGroupThreads, smem, st>>>(s, x, part);
    cudaError_t e = cudaGetLastError();
    float2 *joined = stats ? stats : part + (size_t)s.N * s.splits * s.G;
    const long long warps = s.N * s.G;
    if (e == cudaSuccess)
        e = chain_launch(k_group_join, (unsigned)((warps + kGroupThreads / 32 - 1) / (kGroupThreads / 32)), kGroupThreads, 0, st, s, part, joined);
    if (e == cudaSuccess) e = chain_launch(k_group_apply<T, VEC, OWN, ACT>, grid, kGroupThreads, 0, st, s, x, joined, y);
    return e;
}

template <typename T, int VEC, bool OWN, bool ACT>
cudaError_t group_backward_split(const GroupShape &s, const T *dy, const T *x, const float2 *stats, T *dx, float *dw, float *db, float *part, float2 *terms,
                          cudaStream_t st) {
    const bool sums = dw || db;
    const int cv = s.C / VEC, slots = cv < kGroupThreads ? kGroupThreads / cv : 1;
    const unsigned grid = (unsigned)(s.N * s.splits);
    const size_t smem = (size_t)slots * cv * (OWN ? VEC : 1) * 8 + (slots > 1 ? (size_t)slots * 2 * s.C * 4 : 0);
    group_smem(k_group_sums<T, VEC, OWN, ACT>, smem);
    float2 *split_terms = terms + s.N * s.G;
    k_group_sums<T, VEC, OWN, ACT><<<grid, kGroupThreads, smem, st>>>(s, dy, x, stats, sums ? part : nullptr, split_terms);
    cudaError_t e = cudaGetLastError();
    const int blocks = (int)((s.N * s.G + kGroupTermWarps - 1) / kGroupTermWarps);
    if (e == cudaSuccess)
        e = chain_launch(k_group_terms, blocks + (sums ? norm_col_blocks(s.C) : 0), kGroupTermThreads, 0, st, s, split_terms, terms, blocks, part, dw, db);
    if (e == cudaSuccess) e = chain_launch(k_group_apply_bwd<T, VEC, OWN, ACT>, grid, kGroupThreads, 0, st, s, dy, x, stats, terms, dx);
    return e;
}

// vec: of vectors that are parts of groups; wide: 16-byte vectors that are not would do
template <typename T, bool ACT>
cudaError_t group_forward(const GroupShape &s, const T *x, T *y, float2 *stats, float2 *part, int vec, bool wide, cudaStream_t st) {
    const int each = s.C / s.G;
    return group_by_vec<T>(vec, [&](auto v) {
        constexpr int VEC = decltype(v)::value;
        if (group_rows(s.L, each)) {
            const NormGeom g = norm_geom(each, VEC, true);
            auto go = [&](auto kern, size_t smem) {
                group_smem(kern, smem);
                const long long grid = group_grid(s.N * s.G, g.rpb, s.G, (long long)kRefSms * (group_row_threads<T>(g.block, ACT) / g.threads));
                kern<<<(unsigned)grid, g.threads, smem, st>>>(s, x, g.tpr, y, stats);
                return cudaGetLastError();
            };
            // rows of up to 8 elements, a thread each: 8 registers of them, not 16 (116871 x 128 bfloat16 in 16 groups 14 us
            // forward and 41 backward, 20 and 43 with 16; 120216 x 256 float32 in 32 57 and 132, 75 and 137)
            constexpr int NV = 16 / VEC, HALF = 8 / VEC;
            if (g.block) return go(k_group_row<T, VEC, NV, true, ACT>, GroupRing<T, VEC, NV, 1, false>::bytes(g.threads));
            if (each <= 8) return go(k_group_row<T, VEC, HALF, false, ACT>, GroupRing<T, VEC, HALF, 1, false>::bytes(g.threads));
            return go(k_group_row<T, VEC, NV, false, ACT>, GroupRing<T, VEC, NV, 1, false>::bytes(g.threads));
        }
        const int cv = s.C / VEC;
        if (const int samples = group_small(s.N, s.L, s.C, VEC, kSmallMany)) {
            const size_t smem = (size_t)samples * ((size_t)s.L * cv + s.G) * 8;
            const long long need = (s.N + samples - 1) / samples, most = 2 * kSmallBlocks;
            k_group_small<T, VEC, ACT><<<(unsigned)(need < most ? need : most), kGroupThreads, smem, st>>>(s, x, samples, y, stats);
            return cudaGetLastError();
        }
        constexpr int V16 = 16 / (int)sizeof(T);
        if (VEC < V16 && wide && group_own(s, V16)) return group_forward_split<T, V16, true, ACT>(s, x, y, stats, part, st);
        return group_forward_split<T, VEC, false, ACT>(s, x, y, stats, part, st);
    });
}

template <typename T, bool ACT>
cudaError_t group_backward(const GroupShape &s, const T *dy, const T *x, const float2 *stats, T *dx, float *dw, float *db, float *part, float2 *terms, int vec,
                    bool wide, cudaStream_t st) {
    const int each = s.C / s.G;
    const bool sums = dw || db;
    auto columns = [&](cudaError_t e, long long parts) {
        if (e != cudaSuccess || !sums) return e;
        return chain_launch(k_norm_cols, norm_col_blocks(s.C), kNormColThreads * kNormColSlices, 0, st, part, (int)parts, s.C, dw, db);
    };
    return group_by_vec<T>(vec, [&](auto v) {
        constexpr int VEC = decltype(v)::value;
        if (group_rows(s.L, each)) {
            const NormGeom g = norm_geom(each, VEC, true);
            const GroupBack to = group_back(g, s.N, s.G, ACT);
            const size_t cols = g.block ? 0 : (size_t)2 * kNormBlock * 16 * 4;
            auto go = [&](auto kern, size_t smem) {
                const size_t bytes = smem > cols ? smem : cols;
                group_smem(kern, bytes);
                kern<<<(unsigned)to.blocks, g.threads, bytes, st>>>(s, dy, x, g.tpr, to.same, stats, dx, sums ? part : nullptr);
                return columns(cudaGetLastError(), to.parts);
            };
            constexpr int NV = 16 / VEC, HALF = 8 / VEC;
            if (g.block) return go(k_group_row_bwd<T, VEC, NV, true, ACT>, GroupRing<T, VEC, NV, 2, true>::bytes(g.threads));
            if (each <= 8) return go(k_group_row_bwd<T, VEC, HALF, false, ACT>, GroupRing<T, VEC, HALF, 2, true>::bytes(g.threads));
            return go(k_group_row_bwd<T, VEC, NV, false, ACT>, GroupRing<T, VEC, NV, 2, true>::bytes(g.threads));
        }
        const int cv = s.C / VEC;
        if (const int samples = group_small(s.N, s.L, s.C, VEC, kSmallBack)) {
            const size_t vectors = (size_t)samples * s.L * cv, one = (vectors + (size_t)samples * s.G) * 8, two = vectors * VEC * 8;
            const long long need = (s.N + samples - 1) / samples, blocks = need < kSmallBlocks ? need : kSmallBlocks;
            k_group_small_bwd<T, VEC, ACT><<<(unsigned)blocks, kGroupThreads, one > two ? one : two, st>>>(s, dy, x, samples, stats, dx, sums ? part : nullptr);
            return columns(cudaGetLastError(), blocks);
        }
        constexpr int V16 = 16 / (int)sizeof(T);
        if (VEC < V16 && wide && group_own(s, V16)) return group_backward_split<T, V16, true, ACT>(s, dy, x, stats, dx, dw, db, part, terms, st);
        return group_backward_split<T, VEC, false, ACT>(s, dy, x, stats, dx, dw, db, part, terms, st);
    });
}

int group_check(const char *what, long long N, long long L, int C, int G, long long xs, int wdtype, int act, int dtype) {
    if (dtype != SDM_F32 && dtype != SDM_BF16) return set_error(SDM_ERR_INVALID, "%s: dtype must be SDM_F32 or SDM_BF16", what);
    if (wdtype != SDM_F32 && wdtype != dtype)
        return set_error(SDM_ERR_INVALID, "%s: the weight's dtype must be SDM_F32 or the channels'", what);
    if (act != SDM_ACT_NONE && act != SDM_ACT_SILU) return set_error(SDM_ERR_INVALID, "%s: unknown activation %d", what, act);
    if (N < 0 || L < 0 || C < 1 || G < 1 || C % G || xs < 0)
        return set_error(SDM_ERR_INVALID, "%s: N and L must be >= 0, C a multiple of G >= 1 and the stride >= 0, got %lld, %lld, %d, %d, %lld",
                         what, N, L, C, G, xs);
    if (C > kGroupMaxCols) return set_error(SDM_ERR_UNSUPPORTED, "%s: at most %d channels, got %d", what, kGroupMaxCols, C);
    // Rows in registers count samples in an int and run up to five steps past the last (a step: the rows at once, 5 blocks of
    // 128 an SM at most); the other forms keep partials of every sample in the workspace.
    const bool rows = group_rows(L, C / G);
    if (N && L && (N > (rows ? (1LL << 31) - (1 << 20) : 1LL << 23) || L >= (1LL << 31) || N * G >= (1LL << 31)))
        return set_error(SDM_ERR_UNSUPPORTED, "%s: N G and L must be below 2^31, N at most 2^31 - 2^20 for one position a sample and groups of up to "
                         "%d channels, else 2^23, got %lld, %lld, %d", what, kGroupRowCols, N, L, G);
    return SDM_OK;
}

// the parts of a workspace: partials, then (a backward of split positions) the groups' terms and those of the splits
size_t group_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
size_t group_part_bytes(long long N, long long L, int C, int G, bool back) {
    if (group_rows(L, C / G)) {
        if (!back) return 0;
        // every vector width has the same blocks, without an activation there are no more of them
        const NormGeom g = norm_geom(C / G, 1, true);
        return group_up((size_t)group_back(g, N, G, true).parts * 2 * C * 4);
    }
    const size_t pieces = (size_t)N * group_splits(N, L);
    // (a forward that keeps no statistics: those of the whole samples behind the splits')
    return group_up(pieces * (back ? (size_t)2 * C * 4 : (size_t)G * 8) + (back ? 0 : (size_t)N * G * 8));
}
size_t group_bytes(long long N, long long L, int C, int G, bool back) {
    if (N == 0 || L == 0) return kAlign;
    const bool terms = back && !group_rows(L, C / G);
    return group_part_bytes(N, L, C, G, back) + (terms ? group_up((size_t)N * (1 + group_splits(N, L)) * G * 8) : 0) + kAlign;
}

int group_check_ws(const char *what, const void *ws, size_t have, size_t need) {
    if (!ws || have < need || (uintptr_t)ws % kAlign)
        return set_error(SDM_ERR_WORKSPACE, "%s: workspace NULL, too small (%zu of %zu bytes) or not %zu-byte aligned", what, have, need, (size_t)kAlign);
    return SDM_OK;
}

int group_status(const char *what, cudaError_t e) {
    return e == cudaSuccess ? SDM_OK : set_error(SDM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" {

size_t sdm_group_norm_workspace_bytes(long long N, long long L, int C, int G) {
    if (group_check("group norm", N, L, C, G, 0, SDM_F32, SDM_ACT_NONE, SDM_F32) != SDM_OK) return 0;
    return group_bytes(N, L, C, G, false);
}

int sdm_group_norm(const void *x, long long x_stride, long long N, long long L, int C, int G, const void *weight, const void *bias,
                   int weight_dtype, float eps, int activation, int dtype, void *y, float *stats, void *workspace, size_t workspace_bytes,
                   void *stream) {
    const char *what = "group norm";
    int rc = group_check(what, N, L, C, G, x_stride, weight_dtype, activation, dtype);
    if (rc != SDM_OK) return rc;
    if (!(eps >= 0.f)) return set_error(SDM_ERR_INVALID, "group norm: eps must be >= 0");
    if (N == 0 || L == 0) return SDM_OK;
    if (!x || !y) return set_error(SDM_ERR_INVALID, "group norm: NULL pointer");
    if ((uintptr_t)stats % 8) return set_error(SDM_ERR_INVALID, "group norm: stats must be 8-byte aligned");
    if (!group_rows(L, C / G)) {
        rc = group_check_ws(what, workspace, workspace_bytes, group_bytes(N, L, C, G, false) - kAlign);
        if (rc != SDM_OK) return rc;
    }
    GroupShape s{N, L, x_stride, 0, C, G, weight_dtype == SDM_F32, eps, weight, bias};
    s.split(group_splits(N, L));
    const int vec = norm_vec(dtype == SDM_BF16 ? 2 : 4, C / G, x_stride, C, x, y, y);
    const bool wide = norm_vec(dtype == SDM_BF16 ? 2 : 4, C, x_stride, C, x, y, y) == (dtype == SDM_BF16 ? 8 : 4);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto go = [&](auto type, auto act) {
        using T = decltype(type);
        return group_forward<T, decltype(act)::value>(s, static_cast<const T *>(x), static_cast<T *>(y), reinterpret_cast<float2 *>(stats),
                                               static_cast<float2 *>(workspace), vec, wide, st);
    };
    const bool silu = activation == SDM_ACT_SILU;
    if (dtype == SDM_BF16) return group_status(what, silu ? go(__nv_bfloat16{}, std::true_type{}) : go(__nv_bfloat16{}, std::false_type{}));
    return group_status(what, silu ? go(float{}, std::true_type{}) : go(float{}, std::false_type{}));
}

size_t sdm_group_norm_backward_workspace_bytes(long long N, long long L, int C, int G) {
    if (group_check("group norm backward", N, L, C, G, 0, SDM_F32, SDM_ACT_NONE, SDM_F32) != SDM_OK) return 0;
    return group_bytes(N, L, C, G, true);
}

int sdm_group_norm_backward(const void *grad, long long grad_stride, const void *x, long long x_stride, long long N, long long L, int C, int G,
                            const void *weight, const void *bias, int weight_dtype, int activation, const float *stats, int dtype, void *grad_x,
                            float *grad_weight, float *grad_bias, void *workspace, size_t workspace_bytes, void *stream) {
    const char *what = "group norm backward";
    int rc = group_check(what, N, L, C, G, x_stride, weight_dtype, activation, dtype);
    if (rc != SDM_OK) return rc;
    if (grad_stride < 0) return set_error(SDM_ERR_INVALID, "group norm backward: the gradient's stride must be >= 0, got %lld", grad_stride);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool sums = grad_weight || grad_bias, rows = group_rows(L, C / G);
    if (N == 0 || L == 0) {
        cudaError_t e = cudaSuccess;
        if (grad_weight) e = cudaMemsetAsync(grad_weight, 0, (size_t)C * 4, st);
        if (e == cudaSuccess && grad_bias) e = cudaMemsetAsync(grad_bias, 0, (size_t)C * 4, st);
        return group_status(what, e);
    }
    if (!grad || !x || !stats || !grad_x) return set_error(SDM_ERR_INVALID, "group norm backward: NULL pointer");
    if ((uintptr_t)stats % 8) return set_error(SDM_ERR_INVALID, "group norm backward: stats must be 8-byte aligned");
    if (sums || !rows) {
        rc = group_check_ws(what, workspace, workspace_bytes, group_bytes(N, L, C, G, true) - kAlign);
        if (rc != SDM_OK) return rc;
    }
    GroupShape s{N, L, x_stride, grad_stride, C, G, weight_dtype == SDM_F32, 0.f, weight, bias};
    s.split(group_splits(N, L));
    const int vec = norm_vec(dtype == SDM_BF16 ? 2 : 4, C / G, x_stride, grad_stride, x, grad, grad_x);
    const bool wide = norm_vec(dtype == SDM_BF16 ? 2 : 4, C, x_stride, grad_stride, x, grad, grad_x) == (dtype == SDM_BF16 ? 8 : 4);
    auto part = static_cast<float *>(workspace);
    auto terms = rows ? nullptr : reinterpret_cast<float2 *>(static_cast<unsigned char *>(workspace) + group_part_bytes(N, L, C, G, true));
    auto go = [&](auto type, auto act) {
        using T = decltype(type);
        return group_backward<T, decltype(act)::value>(s, static_cast<const T *>(grad), static_cast<const T *>(x), reinterpret_cast<const float2 *>(stats),
                                                static_cast<T *>(grad_x), grad_weight, grad_bias, part, terms, vec, wide, st);
    };
    const bool silu = activation == SDM_ACT_SILU;
    if (dtype == SDM_BF16) return group_status(what, silu ? go(__nv_bfloat16{}, std::true_type{}) : go(__nv_bfloat16{}, std::false_type{}));
    return group_status(what, silu ? go(float{}, std::true_type{}) : go(float{}, std::false_type{}));
}

}  // extern "C"
