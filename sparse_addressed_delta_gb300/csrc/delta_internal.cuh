// Shared by the gated delta rule's kernels (delta*.cu): sizes, the chunk workspace, bf16 tensor-core
// fragments and the split of a float into bfloat16 terms.
#pragma once

#include "sdm_internal.cuh"

namespace sdm {

constexpr int kDeltaMaxDk = 128, kDeltaMaxDv = 512;
constexpr int kDeltaAux = 5;
// Up to this many tokens take the token-by-token kernel. Token by token and in a chunk, us: 16 heads x 8 tokens
// 16 and 27, x 12 21 and 27, x 16 25 and 27; 64 sequences of 32 heads x 8 125 and 182, x 12 168 and 182, x 16 211 and
// 184 (bfloat16, 128 x 128); 16 heads of 64 x 64 x 8 55 and 80, x 12 78 and 80; float32, 8 of 6 heads of 64 x 96 x 8
// 16 and 25, x 16 27 and 25. The two cross between 12 and 14 tokens; callers without a workspace have the promise of 8.
constexpr int kDeltaStepTokens = 8;
// A log-decay below this is taken as this: exp(-110) is 0 in float32, so the state is forgotten
// whole, and -inf (a hard reset) stays out of the running sums' differences.
constexpr float kDeltaMinDecay = -110.f;

struct DeltaDims {
    int B, T, H, Hk, Dk, Dv;
    int C, Nt;                           // chunk length, chunks a sequence
    int back;                            // 1: the chunk-local work of a backward
    int dtype;
    int tc;                              // 1: the scans run on tcgen05 (planes of X and P in its layout)
    int segs, first;                     // the sequence's segments, scanned at once (DeltaBlock)
    float scale;
    long long spin;                      // polls before a kernel's wait gives up (sdm_set_wait_limit)
    long long qs[3], ks[3], vs[3], gs[3], bs[3], os[3];   // element strides of (b, t, h)
};

struct DeltaIn {
    const void *q, *k, *v;
    const float *g, *beta;
    const int32_t *valid;                // may be null
};

// bfloat16 operands of the products: planes whose sum is the input (one for bfloat16 inputs, three
// for float32 inputs, split by launch_delta_split into contiguous [B, T, heads, D])
struct DeltaPlanes {
    const __nv_bfloat16 *p;
    long long plane;                     // elements from one plane to the next
    long long s[3];                      // element strides of (b, t, h)
};

// Per chunk and head, written by the chunk-local kernel (k_delta_local) for the scans:
//   x   [3][C][C] bfloat16 planes of X
//   p   [3][C][C] planes of P diag(beta) (for the tcgen05 scan: of P diag(beta) X)
//   aux [kDeltaAux][C] float: exp(L_t), exp(L_C - L_t) beta_t, beta_t, L_t as the sum of two
// and for a backward: planes of (I + diag(beta) A)^-1 =: X and of P (for tcgen05: of P X), and exp(L_C -
// L_t) without beta.
// The planes' rows have shared memory's layout (delta_pitch, or tcgen05's 128-byte rows with permuted
// pieces, tc_at), so the scans copy them as they are. Blocks above the diagonal are never written and
// never used. k_delta_local also clears the workspace's status block.
struct DeltaLocal {
    unsigned char *x, *p;
    float *aux;
    DevStatus *status;
    // with segments: their first states (a backward: end states' gradients) [segs][B, H, Dk, Dv], and what
    // the inner ones make of a unit matrix [segs - 2][B, H, Dk, Dk]
    float *starts, *units;
};

__host__ __device__ constexpr int delta_chunk(int dtype) { return dtype == SDM_BF16 ? 64 : 32; }

// A sequence in segments (d.segs > 1), for the scans. A segment's end state is linear in its first state,
// M S + E. A first launch takes every segment but the last from a state of zeros (the first one from the
// caller's, so it needs no M) to E, and the inner ones' M from a unit matrix with no values; a join
// (launch_delta_join) makes the first states from these; a second launch runs all segments at once. Segment
// 0's blocks come last, several after one another where SMs are free; it is first / 256 as long as the others.
// A backward goes the same way from the end (gradients of a segment's first state are M^T times those of its
// end, and E), with the M that its forward saved.
__host__ __device__ inline long long delta_states(const DeltaDims &d) { return (long long)d.B * d.H * d.Dk * d.Dv; }
// first chunk of segment i of a sequence of `chunks`
__host__ __device__ inline int delta_bound(const DeltaDims &d, int chunks, int i) {
    return i == 0 ? 0 : (int)((long long)chunks * (d.first + (i - 1) * 256) / ((d.segs - 1) * 256 + d.first));
}

__device__ __forceinline__ int delta_valid(const int32_t *valid, int b, int T) {
    const int v = valid ? valid[b] : T;
    return v < 0 ? 0 : (v > T ? T : v);
}

struct DeltaBlock {
    int seg, tile;
    bool unit;
    long long bh;
};
// The scans' blocks take the sequences from the longest down, so that the last ones to start are short
// (8 sequences of 2048 to 4096 tokens, 32 heads, whole call by five draws of lengths: 600 to 660 us, in their order
// 623 to 682). More than 32 sequences stay in their
// order: their many blocks level out by themselves.
__device__ __forceinline__ long long delta_longest_first(const DeltaDims &d, const int32_t *valid, long long bh) {
    if (!valid || d.B > 32) return bh;
    const int lane = threadIdx.x & 31, mine = lane < d.B ? delta_valid(valid, lane, d.T) : -1;
    int rank = 0;
    for (int i = 0; i < d.B; ++i) {
        const int other = __shfl_sync(~0u, mine, i);
        rank += other > mine || (other == mine && i < lane);
    }
    const int b = __ffs(__ballot_sync(~0u, rank == (int)(bh / d.H))) - 1;
    return (long long)b * d.H + bh % d.H;
}

enum { DELTA_RUN, DELTA_CARRY, DELTA_CARRY_BACK };                // the second launch, the first ones

__host__ __device__ inline int delta_tiles(int columns, int of) { return (columns + of - 1) / of; }
inline long long delta_blocks(const DeltaDims &d, int mode, int of) {
    const long long heads = (long long)d.B * d.H, run = heads * delta_tiles(d.Dv, of);
    return mode == DELTA_CARRY ? (d.segs - 2) * (run + heads * delta_tiles(d.Dk, of)) + run : mode == DELTA_RUN ? d.segs * run : (d.segs - 1) * run;
}
// this block's head, segment and tile of `of` columns, of the state or of a unit matrix
__device__ __forceinline__ DeltaBlock delta_block(const DeltaDims &d, const int32_t *valid, bool segs, int mode, int of) {
    DeltaBlock k;
    const int tiles = delta_tiles(d.Dv, of), heads = d.B * d.H;
    const int per = mode == DELTA_CARRY ? tiles + delta_tiles(d.Dk, of) : tiles;
    const int inner = !segs ? 0 : mode == DELTA_CARRY ? d.segs - 2 : d.segs - 1;
    unsigned i = blockIdx.x;
    const bool first = !segs || i >= (unsigned)(inner * heads * per);
    if (first) i -= inner * heads * per;
    const int each = first ? tiles : per;
    k.tile = (int)(i % each);
    i /= each;
    k.bh = delta_longest_first(d, valid, segs ? i % heads : i);
    k.seg = first ? 0 : 1 + (int)(i / heads);
    k.unit = mode == DELTA_CARRY && k.tile >= tiles;
    if (k.unit) k.tile -= tiles;
    return k;
}

inline size_t delta_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline size_t delta_chunks(const DeltaDims &d) { return (size_t)d.B * d.H * d.Nt; }
inline size_t delta_plane_bytes(const DeltaDims &d) { return (size_t)d.C * (d.C * 2 + 16); }

cudaError_t launch_delta_step(const DeltaDims &d, const DeltaIn &in, float *state, void *o,
                              cudaStream_t st);
cudaError_t launch_delta_split(const DeltaDims &d, const void *q, const void *k, __nv_bfloat16 *q_planes,
                               __nv_bfloat16 *k_planes, cudaStream_t st);
// a bfloat16 [B, T, heads, width] of strides s, contiguous
cudaError_t launch_delta_unroll(const DeltaDims &d, const void *x, const long long *s, int heads, int width, void *to, cudaStream_t st);
cudaError_t launch_delta_local(const DeltaDims &d, const DeltaIn &in, const DeltaPlanes &q,
                               const DeltaPlanes &k, const DeltaLocal &w, cudaStream_t st);
// snap [B, H, Nt + 1, Dk, Dv] the state at each chunk's start and, behind the last chunk with tokens, the
// final one; r [B, H, Nt, C, Dv] what each value lacks; null unless saving
cudaError_t launch_delta_scan(const DeltaDims &d, const DeltaIn &in, const DeltaPlanes &q,
                              const DeltaPlanes &k, const DeltaLocal &w, float *state, void *o,
                              float *snap, float *r, cudaStream_t st);

// the segments' first states (back: end states' gradients) into w.starts; state: the first (back: the last,
// null: 0) of them
cudaError_t launch_delta_join(const DeltaDims &d, const DeltaLocal &w, const float *state, bool back, cudaStream_t st);

cudaError_t launch_delta_scan_tc(const DeltaDims &d, const DeltaIn &in, const DeltaLocal &w, float *state,
                                 void *o, float *snap, float *r, cudaStream_t st);

// Outputs of the backward and what its kernels hand on.
struct DeltaBack {
    const void *grad;                    // [B, T, H, Dv] (strides os) gradient of the readings
    const float *state_in;               // [B, H, Dk, Dv] gradient of the final state, or null: 0
    float *state_out;                    // [B, H, Dk, Dv]
    void *grad_q, *grad_k, *grad_v;      // contiguous, the inputs' type
    float *grad_decay, *grad_beta;       // [B, T, H]
    const float *snap, *r;               // saved by the forward
    float *ends;                         // [B, H, Nt, Dk, Dv] gradient of each chunk's end state
    float *w;                            // [B, H, Nt, C, Dv] X^T (gradient of u)
    float *dq, *dk;                      // [B, T, H, Dk] before shared heads are summed (H > Hk)
};

cudaError_t launch_delta_back_scan(const DeltaDims &d, const DeltaIn &in, const DeltaPlanes &q,
                                   const DeltaPlanes &k, const DeltaLocal &w, const DeltaBack &o,
                                   cudaStream_t st);
cudaError_t launch_delta_back_scan_tc(const DeltaDims &d, const DeltaIn &in, const DeltaLocal &w, const DeltaBack &o,
                                      cudaStream_t st);
cudaError_t launch_delta_back_local(const DeltaDims &d, const DeltaIn &in, const DeltaPlanes &q,
                                    const DeltaPlanes &k, const DeltaLocal &w, const DeltaBack &o,
                                    cudaStream_t st);
cudaError_t launch_delta_back_local_tc(const DeltaDims &d, const DeltaIn &in, const DeltaLocal &w, const DeltaBack &o,
                                       cudaStream_t st);

// ---------------------------------------------------------------------------------------
// device helpers
// ---------------------------------------------------------------------------------------

__device__ __forceinline__ float delta_decay(float g) { return g < kDeltaMinDecay ? kDeltaMinDecay : g; }

__device__ __forceinline__ bool delta_finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// One column of a chunk token by token, by one warp: S its state [Dk] at the chunk's start (Dv apart), o its readings
// and r (may be null) what its values lack. For columns whose update in a chunk is not finite: in the chunk's products
// a NaN or infinity of one token meets the zeros of the tokens before it (0 x inf is NaN), here it reaches the
// later ones alone.
template <typename T>
__device__ __forceinline__ void delta_column(const DeltaDims &d, const DeltaIn &in, int b, int h, int dv, int t0, int nt, const float *S,
                                             T *o, float *r) {
    constexpr int NR = kDeltaMaxDk / 32;
    const int lane = threadIdx.x & 31, hk = h / (d.H / d.Hk);
    const T *q = static_cast<const T *>(in.q) + b * d.qs[0] + hk * d.qs[2] + t0 * d.qs[1];
    const T *k = static_cast<const T *>(in.k) + b * d.ks[0] + hk * d.ks[2] + t0 * d.ks[1];
    const T *v = static_cast<const T *>(in.v) + b * d.vs[0] + h * d.vs[2] + t0 * d.vs[1] + dv;
    const float *g = in.g + b * d.gs[0] + h * d.gs[2] + t0 * d.gs[1], *be = in.beta + b * d.bs[0] + h * d.bs[2] + t0 * d.bs[1];
    float s[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) s[i] = lane + 32 * i < d.Dk ? S[(size_t)(lane + 32 * i) * d.Dv] : 0.f;
#pragma unroll 1
    for (int t = 0; t < nt; ++t) {
        const float fade = expf(delta_decay(g[t * d.gs[1]]));
        float a = 0.f, c = 0.f;
#pragma unroll
        for (int i = 0; i < NR; ++i)
            if (lane + 32 * i < d.Dk) {
                s[i] *= fade;
                a = fmaf(to_f32(k[t * d.ks[1] + lane + 32 * i]), s[i], a);
            }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) a += __shfl_xor_sync(~0u, a, m);
        const float lack = to_f32(v[t * d.vs[1]]) - a, u = be[t * d.bs[1]] * lack;
#pragma unroll
        for (int i = 0; i < NR; ++i)
            if (lane + 32 * i < d.Dk) {
                s[i] = fmaf(to_f32(k[t * d.ks[1] + lane + 32 * i]), u, s[i]);
                c = fmaf(to_f32(q[t * d.qs[1] + lane + 32 * i]), s[i], c);
            }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) c += __shfl_xor_sync(~0u, c, m);
        if (lane == 0) {
            o[(long long)t * d.H * d.Dv] = from_f32<T>(d.scale * c);
            if (r) r[(long long)t * d.Dv] = lack;
        }
    }
}

// The log-decays' gradients of a chunk, TL tokens a lane: x summed from each token on, y up to the one before,
// and what crosses the whole chunk
template <int TL>
__device__ __forceinline__ void delta_decay_sums(const float (&x)[TL], const float (&y)[TL], double whole, double (&dg)[TL]) {
    const int lane = threadIdx.x & 31;
    double xs = 0.0, ys = 0.0;
#pragma unroll
    for (int i = 0; i < TL; ++i) {
        xs += (double)x[i];
        ys += (double)y[i];
    }
    double from = xs, upto = ys;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
        const double a = __shfl_down_sync(~0u, from, m), b = __shfl_up_sync(~0u, upto, m);
        if (lane + m < 32) from += a;
        if (lane >= m) upto += b;
    }
    upto -= ys;
    double rest = from - xs;                       // of the lanes behind
#pragma unroll
    for (int i = TL - 1; i >= 0; --i) {
        rest += (double)x[i];
        dg[i] = rest;
    }
#pragma unroll
    for (int i = 0; i < TL; ++i) {
        dg[i] += upto + whole;
        upto += (double)y[i];
    }
}

// Tiles in shared memory have rows of PITCH bytes, an odd multiple of 16: ldmatrix's eight rows at
// one column then fall into different banks, and every fragment's address is the lane's own offset
// plus a constant.
__host__ __device__ constexpr int delta_pitch(int bytes) { return bytes + 16; }
template <int PITCH>
__device__ __forceinline__ int delta_at(int r, int c) { return r * PITCH + c * 16; }

// The tensor core's tiles (tcgen05): rows of 128 bytes (64 bfloat16), 16-byte piece c of row r at piece
// c ^ (r % 8); tiles start at multiples of 1024 bytes; wider rows are several such tiles.
__device__ __forceinline__ int tc_at(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

__device__ __forceinline__ void cp_async16_zfill(unsigned dst, const void *src, bool live) {
    const int n = live ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}

__device__ __forceinline__ void ldsm4(unsigned (&r)[4], unsigned addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(unsigned (&r)[4], unsigned addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Fragments of a tile in shared memory (rows of PITCH bytes):
// rows r0.., bfloat16 columns c0.. (multiples of 8). ldmatrix lane i addresses row i % 8 of 8 x 8
// block i / 8.
//   frag_rc: blocks (r, c), (r + 8, c), (r, c + 8), (r + 8, c + 8)
//     plain: an A operand of 16 rows x 16 of K;  transposed: two 8-column B operands with K = rows
//   frag_cr: blocks (r, c), (r, c + 8), (r + 8, c), (r + 8, c + 8)
//     plain: two 8-column B operands with N = rows, K = columns; transposed: an A operand, M = columns
template <int PITCH>
__device__ __forceinline__ unsigned frag_rc(unsigned base, int r0, int c0, int lane) {
    return base + delta_at<PITCH>(lane & 15, lane >> 4) + delta_at<PITCH>(r0, c0 >> 3);
}
template <int PITCH>
__device__ __forceinline__ unsigned frag_cr(unsigned base, int r0, int c0, int lane) {
    return base + delta_at<PITCH>((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1) + delta_at<PITCH>(r0, c0 >> 3);
}

// c += a b, one 16 x 8 x 16 bfloat16 product with float32 sums
__device__ __forceinline__ void mma_bf16(float (&c)[4], const unsigned (&a)[4], unsigned b0,
                                         unsigned b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ unsigned pack_bf16(float x0, float x1) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
    return *reinterpret_cast<const unsigned *>(&h);
}
__device__ __forceinline__ float lo_f32(unsigned h) { return __uint_as_float(h << 16); }
__device__ __forceinline__ float hi_f32(unsigned h) { return __uint_as_float(h & 0xffff0000u); }

// x0, x1 as sums of N bfloat16 terms each (8 bits a term: three keep float32's 24 bits)
template <int N>
__device__ __forceinline__ void split_bf16(float x0, float x1, unsigned (&p)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        p[i] = pack_bf16(x0, x1);
        if (i + 1 < N) {
            x0 -= lo_f32(p[i]);
            x1 -= hi_f32(p[i]);
        }
    }
}

// A operand (K step ks) of the transposed product from accumulators acc[tile][4] whose columns are
// its K: N planes
template <int N, int TILES>
__device__ __forceinline__ void split_frag(const float (&acc)[TILES][4], int ks,
                                           unsigned (&a)[N][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        unsigned p[N];
        split_bf16<N>(acc[2 * ks + (i >> 1)][2 * (i & 1)], acc[2 * ks + (i >> 1)][2 * (i & 1) + 1], p);
#pragma unroll
        for (int s = 0; s < N; ++s) a[s][i] = p[s];
    }
}

// whether the product of terms a and b (counted from the largest) is above 2^-8 `most` of the whole
__device__ __forceinline__ constexpr bool plane_pair(int a, int b, int most) { return a + b < most; }
// The same in two passes over a sum's steps, 1: the smaller terms' products, then 0: the largest terms'. The
// tensor core cuts an accumulator's low bits at every step, so the sum is kept small for as long as it can be.
__device__ __forceinline__ constexpr bool plane_pair(int a, int b, int most, int pass) { return a + b < most && (a + b > 0) == (pass > 0); }

// K or Q planes of a chunk's `nt` live tokens into tiles [KP][C] of DKP columns, zero elsewhere
template <int KP, int DKP, int C, int THREADS>
__device__ __forceinline__ void load_tokens(unsigned dst, const DeltaPlanes &x, long long base,
                                            int Dk, int nt, int tid) {
    constexpr int PC = DKP / 8, PITCH = delta_pitch(DKP * 2);
    for (int i = tid; i < KP * C * PC; i += THREADS) {
        const int c = i % PC, r = (i / PC) % C, pl = i / (PC * C);
        const bool live = r < nt && c * 8 < Dk;
        const __nv_bfloat16 *src = x.p + pl * x.plane + base + (live ? r * x.s[1] + c * 8 : 0);
        cp_async16_zfill(dst + pl * (C * PITCH) + delta_at<PITCH>(r, c), src, live);
    }
}

// PL planes [C][C] of X or P as k_delta_local stored them (blocks on and below the diagonal)
template <int PL, int C, int THREADS>
__device__ __forceinline__ void load_planes(unsigned dst, const unsigned char *src, int tid) {
    constexpr int XP = delta_pitch(C * 2);
    for (int i = tid; i < PL * C * (C / 8); i += THREADS) {
        const int c = i % (C / 8), r = (i / (C / 8)) % C, pl = i / (C * (C / 8));
        if (c > 2 * (r >> 4) + 1) continue;
        const int off = pl * C * XP + delta_at<XP>(r, c);
        cp_async16_zfill(dst + off, src + off, true);
    }
}

// COLS columns of a [tokens, Dv] tile (values, gradients), zero past the live tokens and columns
template <typename T, int COLS, int C, int THREADS>
__device__ __forceinline__ void load_values(unsigned dst, const T *src, long long row, int nt,
                                            int cols, int tid) {
    constexpr int VE = 16 / (int)sizeof(T), PC = COLS / VE, PITCH = delta_pitch(COLS * (int)sizeof(T));
    for (int i = tid; i < C * PC; i += THREADS) {
        const int c = i % PC, r = i / PC;
        const bool live = r < nt && c * VE < cols;
        cp_async16_zfill(dst + delta_at<PITCH>(r, c), live ? src + r * row + c * VE : src, live);
    }
}

}  // namespace sdm
