// Backward of the gated delta rule in chunks (notation of delta_chunk.cu; dO the readings' gradient,
// D1 the gradient of a chunk's end state, D0 of its start state):
//   du = P^T dO + (e^{L_C - L} K) D1;   dw = X^T du;   dv = beta dw
//   D0 = G_C D1 + (scale G Q)^T dO - K^T (beta G dw)
// is a recurrence over the chunks from the last to the first (k_delta_back_scan), the forward scan's
// mirror image: a warp owns 16 columns, and accumulators pass from product to product as A operands.
// Everything else needs only a chunk's own S0, u (saved by the forward), D1 and dw (left by the scan),
// and runs for all chunks at once (k_delta_back_local):
//   E = dw u^T, dA = -beta E (s < t);   dP = dO u^T (s <= t);   a = dA e^{L_t - L_s}, p = scale dP e^{L_t - L_s}
//   dq = p K + scale G (dO S0^T)
//   dk = p^T Q + (a + a^T) K - beta G (dw S0^T) + e^{L_C - L} (u D1^T)
//   dbeta_t = <dw_t, v_t> - G_t <k_t, dw_t S0^T> - sum_s E[t,s] A[t,s]
//   dL from a, p (rows minus columns), from the three products with the states (row products with q and
//   k) and from G_C <S0, D1>;  dg = the suffix sums of dL.
// The gates' gradients are float32: every product that reaches them keeps float32's accuracy.
#include "delta_internal.cuh"

namespace sdm {
namespace {

template <typename T, int DKP, int NW>
struct BackSmem {
    static constexpr bool BF = sizeof(T) == 2;
    static constexpr int C = BF ? 64 : 32, KP = BF ? 1 : 3, PP = 3;
    static constexpr int XP = delta_pitch(C * 2), VP = delta_pitch(NW * 16 * (int)sizeof(T));
    static constexpr int KPI = delta_pitch(DKP * 2), TILE = C * KPI;
    static constexpr int Q = KP * TILE, X = 2 * KP * TILE, P = X + 3 * C * XP, V = P + PP * C * XP;
    static constexpr int AUX = V + C * VP, STAGE = AUX + 3 * C * 4;
    static constexpr int STAGES = 2 * STAGE <= 227 * 1024 ? 2 : 1;
    static constexpr int BYTES = STAGES * STAGE;
};

// One block per head and NW * 16 of its columns, from the last chunk to the first.
template <typename T, int DKP, int NW>
__global__ void __launch_bounds__(NW * 32, 1)
    k_delta_back_scan(DeltaDims d, DeltaIn in, DeltaPlanes q, DeltaPlanes k, DeltaLocal w, DeltaBack o) {
    using L = BackSmem<T, DKP, NW>;
    constexpr bool BF = L::BF;
    constexpr int C = L::C, KP = L::KP, PP = L::PP, XP = L::XP, VP = L::VP, KPI = L::KPI, THREADS = NW * 32;
    constexpr int NT = C / 8, ND = DKP / 8, VE = 16 / (int)sizeof(T);
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g4 = lane >> 2, i4 = lane & 3;
    const int slices = (d.Dv + NW * 16 - 1) / (NW * 16);
    const int dv_blk = (blockIdx.x % slices) * NW * 16;
    const long long bh = blockIdx.x / slices;
    const int b = (int)(bh / d.H), h = (int)(bh % d.H), hk = h / (d.H / d.Hk);
    const int dv0 = dv_blk + 16 * warp;
    const bool mine = dv0 < d.Dv;
    const int ntok = delta_valid(in.valid, b, d.T), nch = (ntok + C - 1) / C;
    const T *grad = static_cast<const T *>(o.grad) + b * d.os[0] + h * d.os[2] + dv_blk;
    const long long kbase = b * k.s[0] + hk * k.s[2], qbase = b * q.s[0] + hk * q.s[2];
    T *gv = static_cast<T *>(o.grad_v) + ((long long)b * d.T * d.H + h) * d.Dv;
    const long long orow = (long long)d.H * d.Dv;
    const unsigned s0 = smem_u32(smem);

    auto load = [&](int n, int stage) {
        const unsigned st = s0 + stage * L::STAGE;
        const long long t0 = (long long)n * C, bhn = bh * d.Nt + n;
        const int nt = ntok - (int)t0 < C ? ntok - (int)t0 : C;
        load_tokens<KP, DKP, C, THREADS>(st, k, kbase + t0 * k.s[1], d.Dk, nt, tid);
        load_tokens<KP, DKP, C, THREADS>(st + L::Q, q, qbase + t0 * q.s[1], d.Dk, nt, tid);
        load_planes<3, C, THREADS>(st + L::X, w.x + bhn * (3 * C * XP), tid);
        load_planes<PP, C, THREADS>(st + L::P, w.p + bhn * (PP * C * XP), tid);
        load_values<T, NW * 16, C, THREADS>(st + L::V, grad + t0 * d.os[1], d.os[1], nt, d.Dv - dv_blk, tid);
        for (int i = tid; i < 3 * C / 4; i += THREADS)
            cp_async16_zfill(st + L::AUX + 16 * i, w.aux + bhn * 3 * C + 4 * i, true);
        cp_async_commit();
    };
    // element e of the state's fragment j: row 8 j + 2 i4 + (e & 1), column dv0 + g4 + 8 (e >> 1)
    float S[ND][4];
    const float *sp = o.state_in + (bh * d.Dk) * d.Dv + dv0;
#pragma unroll
    for (int j = 0; j < ND; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int dk = 8 * j + 2 * i4 + (e & 1);
            S[j][e] = mine && o.state_in && dk < d.Dk ? sp[(size_t)dk * d.Dv + g4 + 8 * (e >> 1)] : 0.f;
        }
    auto store_state = [&](float *dst) {
#pragma unroll
        for (int j = 0; j < ND; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int dk = 8 * j + 2 * i4 + (e & 1);
                if (dk < d.Dk) dst[(size_t)dk * d.Dv + g4 + 8 * (e >> 1)] = S[j][e];
            }
    };
    if (L::STAGES == 2 && nch > 0) load(nch - 1, 0);
    for (int it = 0; it < nch; ++it) {
        const int n = nch - 1 - it;
        if constexpr (L::STAGES == 2) {
            if (n > 0) {
                load(n - 1, (it + 1) & 1);
                cp_async_wait<1>();
            } else {
                cp_async_wait<0>();
            }
        } else {
            load(n, 0);
            cp_async_wait<0>();
        }
        __syncthreads();
        const int stage = L::STAGES == 2 ? (it & 1) * L::STAGE : 0;
        const unsigned sk = s0 + stage, sq = sk + L::Q, sx = sk + L::X, spp = sk + L::P, sv = sk + L::V;
        const float *from = reinterpret_cast<const float *>(smem + stage + L::AUX), *to = from + C, *be = to + C;
        const int nt = ntok - n * C < C ? ntok - n * C : C;
        if (mine) {
            store_state(o.ends + ((bh * d.Nt + n) * (long long)d.Dk) * d.Dv + dv0);
            // dO^T as an A operand, K step ks: KP planes of the stored values times `f` of the token
            auto grads = [&](int ks, float (&x)[4][2]) {
                if constexpr (BF) {
                    unsigned r[4];
                    ldsm4t(r, frag_cr<VP>(sv, 16 * ks, 16 * warp, lane));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[i][0] = lo_f32(r[i]);
                        x[i][1] = hi_f32(r[i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int t = 16 * ks + 8 * (i >> 1) + 2 * i4 + e, c = 16 * warp + g4 + 8 * (i & 1);
                            x[i][e] = *reinterpret_cast<const float *>(smem + stage + L::V + delta_at<VP>(t, c >> 2) + 4 * (c & 3));
                        }
                }
            };
            float D[NT][4] = {};
#pragma unroll
            for (int ks = 0; ks < DKP / 16; ++ks) {          // D = (K D1)^T
                unsigned a[3][4], bb[KP][C / 16][4];
                split_frag<3>(S, ks, a);
#pragma unroll
                for (int p = 0; p < KP; ++p)
#pragma unroll
                    for (int jj = 0; jj < C / 16; ++jj)
                        ldsm4(bb[p][jj], frag_cr<KPI>(sk + p * L::TILE, 16 * jj, 16 * ks, lane));
#pragma unroll
                for (int x = 2; x >= 0; --x)
#pragma unroll
                    for (int p = KP - 1; p >= 0; --p)
                        if (plane_pair(x, p, 3))
#pragma unroll
                            for (int j = 0; j < NT; ++j)
                                mma_bf16(D[j], a[x], bb[p][j >> 1][2 * (j & 1)], bb[p][j >> 1][2 * (j & 1) + 1]);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) D[j][e] *= to[8 * j + 2 * i4 + (e & 1)];
#pragma unroll
            for (int ks = 0; ks < C / 16; ++ks) {            // D += (P^T dO)^T
                float x[4][2];
                unsigned a[KP][4];
                grads(ks, x);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    unsigned pl[KP];
                    split_bf16<KP>(x[i][0], x[i][1], pl);
#pragma unroll
                    for (int p = 0; p < KP; ++p) a[p][i] = pl[p];
                }
#pragma unroll
                for (int jj = 0; jj <= ks; ++jj) {
                    unsigned bb[PP][4];
#pragma unroll
                    for (int p = 0; p < PP; ++p) ldsm4t(bb[p], frag_rc<XP>(spp + p * C * XP, 16 * ks, 16 * jj, lane));
#pragma unroll
                    for (int y = KP - 1; y >= 0; --y)
#pragma unroll
                        for (int p = PP - 1; p >= 0; --p)
                            if (plane_pair(y, p, 3)) {
                                mma_bf16(D[2 * jj], a[y], bb[p][0], bb[p][1]);
                                mma_bf16(D[2 * jj + 1], a[y], bb[p][2], bb[p][3]);
                            }
                }
            }
            float W[NT][4] = {};
#pragma unroll
            for (int ks = 0; ks < C / 16; ++ks) {            // W = (X^T du)^T
                unsigned a[3][4];
                split_frag<3>(D, ks, a);
#pragma unroll
                for (int jj = 0; jj <= ks; ++jj) {
                    unsigned bb[3][4];
#pragma unroll
                    for (int p = 0; p < 3; ++p) ldsm4t(bb[p], frag_rc<XP>(sx + p * C * XP, 16 * ks, 16 * jj, lane));
#pragma unroll
                    for (int x = 2; x >= 0; --x)
#pragma unroll
                        for (int p = 2; p >= 0; --p)
                            if (plane_pair(x, p, 3)) {
                                mma_bf16(W[2 * jj], a[x], bb[p][0], bb[p][1]);
                                mma_bf16(W[2 * jj + 1], a[x], bb[p][2], bb[p][3]);
                            }
                }
            }
            // D1 <- G_C D1 + (scale G dO)^T Q - (beta G dw)^T K
            unsigned ua[C / 16][3][4];
#pragma unroll
            for (int ks = 0; ks < C / 16; ++ks) {
                float x[4][2];
                grads(ks, x);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 16 * ks + 8 * (i >> 1) + 2 * i4;
                    unsigned pl[3];
                    split_bf16<3>(x[i][0] * (d.scale * from[t]), x[i][1] * (d.scale * from[t + 1]), pl);
#pragma unroll
                    for (int p = 0; p < 3; ++p) ua[ks][p][i] = pl[p];
                }
            }
            const float whole = from[C - 1];
            auto update = [&](unsigned tile, float keep) {
#pragma unroll
                for (int nn = 0; nn < ND / 2; nn += 2) {
                    float acc[4][4] = {};
#pragma unroll
                    for (int ks = 0; ks < C / 16; ++ks) {
                        unsigned bb[KP][2][4];
#pragma unroll
                        for (int p = 0; p < KP; ++p)
#pragma unroll
                            for (int m = 0; m < 2; ++m)
                                ldsm4t(bb[p][m], frag_rc<KPI>(tile + p * L::TILE, 16 * ks, 16 * (nn + m), lane));
#pragma unroll
                        for (int x = 2; x >= 0; --x)
#pragma unroll
                            for (int p = KP - 1; p >= 0; --p)
                                if (plane_pair(x, p, 3))
#pragma unroll
                                    for (int m = 0; m < 4; ++m)
                                        mma_bf16(acc[m], ua[ks][x], bb[p][m >> 1][2 * (m & 1)], bb[p][m >> 1][2 * (m & 1) + 1]);
                    }
#pragma unroll
                    for (int m = 0; m < 4; ++m)
#pragma unroll
                        for (int e = 0; e < 4; ++e) S[2 * nn + m][e] = fmaf(keep, S[2 * nn + m][e], acc[m][e]);
                }
            };
            update(sq, whole);
            // dw leaves for the chunk-local kernel; beta dw is the values' gradient
            float *dst = o.w + ((bh * d.Nt + n) * (long long)C) * d.Dv + dv0;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 8 * j + 2 * i4 + (e & 1), c = 16 * warp + g4 + 8 * (e >> 1);
                    dst[(size_t)t * d.Dv + g4 + 8 * (e >> 1)] = W[j][e];
                    const float x = be[t] * W[j][e];
                    *reinterpret_cast<T *>(smem + stage + L::V + delta_at<VP>(t, c / VE) + (c % VE) * sizeof(T)) = from_f32<T>(x);
                    W[j][e] = -from[t] * x;
                }
#pragma unroll
            for (int ks = 0; ks < C / 16; ++ks) split_frag<3>(W, ks, ua[ks]);
            update(sk, 1.f);
            __syncwarp();
            constexpr int PR = 16 / VE, RP = 32 / PR;
#pragma unroll
            for (int r0 = 0; r0 < C; r0 += RP) {
                const int r = r0 + lane / PR, c = lane % PR;
                const long long t = (long long)n * C + r;
                uint4 x = *reinterpret_cast<const uint4 *>(smem + stage + L::V + delta_at<VP>(r, 16 * warp / VE + c));
                if (r >= nt) x = make_uint4(0u, 0u, 0u, 0u);
                if (t < d.T) *reinterpret_cast<uint4 *>(gv + t * orow + dv0 + c * VE) = x;
            }
        }
        __syncthreads();
    }
    if (!mine) return;
    store_state(o.state_out + (bh * d.Dk) * d.Dv + dv0);
    constexpr int PR = 16 / VE;
    for (long long t = (long long)nch * C + lane / PR; t < d.T; t += 32 / PR)
        *reinterpret_cast<uint4 *>(gv + t * orow + dv0 + (lane % PR) * VE) = make_uint4(0u, 0u, 0u, 0u);
}

constexpr int kBackThreads = 256, kBackCols = 64;     // columns of the state at a time

template <typename T, int DKP>
struct BackLocalSmem {
    static constexpr bool BF = sizeof(T) == 2;
    static constexpr int C = BF ? 64 : 32, KP = BF ? 1 : 3, GP = BF ? 2 : 3;
    static constexpr int KPI = delta_pitch(DKP * 2), TILE = C * KPI;
    static constexpr int VPI = delta_pitch(kBackCols * 2), VT = C * VPI;   // planes of dO, dw and u
    static constexpr int GPI = delta_pitch(C * 2), GT = C * GPI;           // planes of p and a
    static constexpr int NB = C / 16;
    static constexpr int Q = KP * TILE, O = 2 * KP * TILE, W = O + KP * VT, U = W + 3 * VT;
    static constexpr int P = U + 3 * VT, A = P + GP * GT, F = A + GP * GT;
    // floats: hi, lo, from, to, beta [C]; <dw, v> [C]; row and column sums of z and row sums of E A
    // [NB][C]; row products [8 warps][3][C]; <S0, D1> [8]
    static constexpr int FLOATS = 6 * C + 3 * NB * C + 8 * 3 * C + 8;
    static constexpr int BYTES = F + FLOATS * 4;
};

// One block of eight warps per chunk and head. For the products with the states a warp owns 16 of
// the Dk columns (with Dk up to 64, half of the tokens too) and reads its rows of S0 and D1 straight
// into fragments; the C x C products are split into 16 x 16 blocks.
template <typename T, int DKP>
__global__ void __launch_bounds__(kBackThreads, 1)
    k_delta_back_local(DeltaDims d, DeltaIn in, DeltaPlanes q, DeltaPlanes k, DeltaLocal lw, DeltaBack o) {
    using L = BackLocalSmem<T, DKP>;
    constexpr bool BF = L::BF;
    constexpr int C = L::C, KP = L::KP, GP = L::GP, NB = L::NB, KPI = L::KPI, VPI = L::VPI, GPI = L::GPI;
    constexpr int NWK = DKP / 16, MS = 8 / NWK, MT = NB / MS;     // warps over Dk, over tokens; token tiles
    constexpr int BLOCKS = NB * (NB + 1) / 2, BPW = (BLOCKS + 7) / 8;
    static_assert(MT >= 1, "token tiles");
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g4 = lane >> 2, i4 = lane & 3;
    const long long bhn = blockIdx.x;
    const int n = (int)(bhn % d.Nt);
    const long long bh = bhn / d.Nt;
    const int b = (int)(bh / d.H), h = (int)(bh % d.H), hk = h / (d.H / d.Hk);
    const int t0 = n * C;
    const int rows = d.T - t0 < C ? d.T - t0 : C;                 // of the output
    int nt = delta_valid(in.valid, b, d.T) - t0;
    nt = nt < 0 ? 0 : nt < C ? nt : C;
    const bool shared = d.H != d.Hk;
    // rows of the gradients of q and k: the result, or this head's part of it
    const long long orow = (long long)d.H * d.Dk, obase = ((long long)b * d.T + t0) * orow + (long long)h * d.Dk;
    auto store2 = [&](bool key, int r, int c, float x, float y) {
        const long long at = obase + r * orow + c;
        if (shared) {
            *reinterpret_cast<float2 *>((key ? o.dk : o.dq) + at) = make_float2(x, y);
        } else if constexpr (BF) {
            *reinterpret_cast<unsigned *>(static_cast<T *>(key ? o.grad_k : o.grad_q) + at) = pack_bf16(x, y);
        } else {
            *reinterpret_cast<float2 *>(static_cast<T *>(key ? o.grad_k : o.grad_q) + at) = make_float2(x, y);
        }
    };
    float *gdec = o.grad_decay + ((long long)b * d.T + t0) * d.H + h, *gbeta = o.grad_beta + ((long long)b * d.T + t0) * d.H + h;
    if (nt == 0) {
        for (int i = tid; i < rows * (d.Dk / 2); i += kBackThreads) {
            store2(false, i / (d.Dk / 2), 2 * (i % (d.Dk / 2)), 0.f, 0.f);
            store2(true, i / (d.Dk / 2), 2 * (i % (d.Dk / 2)), 0.f, 0.f);
        }
        for (int r = tid; r < rows; r += kBackThreads) gdec[(long long)r * d.H] = gbeta[(long long)r * d.H] = 0.f;
        return;
    }
    const unsigned sk = smem_u32(smem), sq = sk + L::Q, so = sk + L::O, sw = sk + L::W, su = sk + L::U;
    float *hi = reinterpret_cast<float *>(smem + L::F), *lo = hi + C, *from = lo + C, *to = from + C, *be = to + C;
    float *dwv = be + C, *zrow = dwv + C, *zcol = zrow + NB * C, *erow = zcol + NB * C, *dots = erow + NB * C;
    float *ends = dots + 8 * 3 * C;

    load_tokens<KP, DKP, C, kBackThreads>(sk, k, b * k.s[0] + t0 * k.s[1] + hk * k.s[2], d.Dk, nt, tid);
    load_tokens<KP, DKP, C, kBackThreads>(sq, q, b * q.s[0] + t0 * q.s[1] + hk * q.s[2], d.Dk, nt, tid);
    cp_async_commit();
    if (warp == 0) {
        const float *aux = lw.aux + bhn * 3 * C;
        double s = 0.0;
        constexpr int PL = C / 32;
        double run[PL];
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const int r = lane * PL + i;
            if (r < nt) s += (double)delta_decay(in.g[b * d.gs[0] + (long long)(t0 + r) * d.gs[1] + h * d.gs[2]]);
            run[i] = s;
            from[r] = aux[r];
            to[r] = aux[C + r];
            be[r] = aux[2 * C + r];
        }
        double before = s;
#pragma unroll
        for (int m = 1; m < 32; m *= 2) {
            const double x = __shfl_up_sync(~0u, before, m);
            if (lane >= m) before += x;
        }
        before -= s;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const double x = before + run[i];
            hi[lane * PL + i] = (float)x;
            lo[lane * PL + i] = (float)(x - (double)(float)x);
        }
    }
    for (int i = tid; i < C; i += kBackThreads) dwv[i] = 0.f;

    const T *grad = static_cast<const T *>(o.grad) + b * d.os[0] + t0 * d.os[1] + h * d.os[2];
    const T *val = static_cast<const T *>(in.v) + b * d.vs[0] + t0 * d.vs[1] + h * d.vs[2];
    const float *wp = o.w + bhn * C * (long long)d.Dv, *up = o.u + bhn * C * (long long)d.Dv;
    const int dk0 = 16 * (warp % NWK), m0 = (warp / NWK) * MT;    // this warp's Dk columns and token tiles
    const float *s0p = o.snap + (bhn * d.Dk) * (long long)d.Dv, *d1p = o.ends + (bhn * d.Dk) * (long long)d.Dv;
    float G1[MT][2][4] = {}, G2[MT][2][4] = {}, G3[MT][2][4] = {}, E[BPW][2][4] = {}, DP[BPW][2][4] = {};
    float inner = 0.f;
    for (int c0 = 0; c0 < d.Dv; c0 += kBackCols) {
        __syncthreads();
        // dO, dw and u of this column tile as planes; <dw, v>
        for (int i = tid; i < C * (kBackCols / 8); i += kBackThreads) {
            const int r = i / (kBackCols / 8), c = i % (kBackCols / 8), col = c0 + 8 * c;
            const bool live = r < nt && col < d.Dv;
            float g[8] = {}, x[8] = {}, u[8] = {}, v[8] = {};
            if (live) {
                load_vec<T, 8, true>(grad + r * d.os[1] + col, g);
                load_vec<float, 8, true>(wp + (long long)r * d.Dv + col, x);
                load_vec<float, 8, true>(up + (long long)r * d.Dv + col, u);
                load_vec<T, 8, true>(val + r * d.vs[1] + col, v);
            }
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(x[e], v[e], s);
#pragma unroll
            for (int m = 1; m < kBackCols / 8; m *= 2) s += __shfl_xor_sync(~0u, s, m);
            if (c == 0) dwv[r] += s;
            auto put = [&](unsigned char *dst, const float (&y)[8], auto planes) {
                constexpr int PL = decltype(planes)::value;
                unsigned p[4][PL];
#pragma unroll
                for (int e = 0; e < 4; ++e) split_bf16<PL>(y[2 * e], y[2 * e + 1], p[e]);
#pragma unroll
                for (int m = 0; m < PL; ++m)
                    *reinterpret_cast<uint4 *>(dst + m * L::VT + delta_at<VPI>(r, c)) = make_uint4(p[0][m], p[1][m], p[2][m], p[3][m]);
            };
            put(smem + L::O, g, std::integral_constant<int, KP>{});
            put(smem + L::W, x, std::integral_constant<int, 3>{});
            put(smem + L::U, u, std::integral_constant<int, 3>{});
        }
        cp_async_wait<0>();
        __syncthreads();
        // E += dw u^T, dP += dO u^T, 16 x 16 blocks on and below the diagonal
#pragma unroll
        for (int x = 0; x < BPW; ++x) {
            const int idx = warp + 8 * x;
            if (idx >= BLOCKS) break;
            const int bi = idx < 1 ? 0 : idx < 3 ? 1 : idx < 6 ? 2 : 3, bj = idx - bi * (bi + 1) / 2;
#pragma unroll
            for (int ks = 0; ks < kBackCols / 16; ++ks) {
                unsigned aw[3][4], ao[KP][4], bu[3][4];
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    ldsm4(aw[p], frag_rc<VPI>(sw + p * L::VT, 16 * bi, 16 * ks, lane));
                    ldsm4(bu[p], frag_cr<VPI>(su + p * L::VT, 16 * bj, 16 * ks, lane));
                }
#pragma unroll
                for (int p = 0; p < KP; ++p) ldsm4(ao[p], frag_rc<VPI>(so + p * L::VT, 16 * bi, 16 * ks, lane));
#pragma unroll
                for (int s = 2; s >= 0; --s)
#pragma unroll
                    for (int p = 2; p >= 0; --p)
                        if (plane_pair(s, p, 3))
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                mma_bf16(E[x][e], aw[s], bu[p][2 * e], bu[p][2 * e + 1]);
                                if (s < KP) mma_bf16(DP[x][e], ao[s < KP ? s : 0], bu[p][2 * e], bu[p][2 * e + 1]);
                            }
            }
        }
        // products with the states over this column tile
        const int rest = d.Dv - c0 < kBackCols ? d.Dv - c0 : kBackCols;
        for (int ks = 0; ks < rest / 16; ++ks) {
            unsigned bs[2][2][3], be1[2][2][3];                   // [8-column tile][k half][plane]
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int row = dk0 + 8 * e + g4;
                    const long long at = (long long)row * d.Dv + c0 + 16 * ks + 8 * m + 2 * i4;
                    float2 x = make_float2(0.f, 0.f), y = x;
                    if (row < d.Dk) {
                        x = __ldg(reinterpret_cast<const float2 *>(s0p + at));
                        y = __ldg(reinterpret_cast<const float2 *>(d1p + at));
                    }
                    inner = fmaf(x.x, y.x, fmaf(x.y, y.y, inner));
                    split_bf16<3>(x.x, x.y, bs[e][m]);
                    split_bf16<3>(y.x, y.y, be1[e][m]);
                }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                unsigned ao[KP][4], aw[3][4], au[3][4];
#pragma unroll
                for (int p = 0; p < KP; ++p) ldsm4(ao[p], frag_rc<VPI>(so + p * L::VT, 16 * (m0 + mt), 16 * ks, lane));
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    ldsm4(aw[p], frag_rc<VPI>(sw + p * L::VT, 16 * (m0 + mt), 16 * ks, lane));
                    ldsm4(au[p], frag_rc<VPI>(su + p * L::VT, 16 * (m0 + mt), 16 * ks, lane));
                }
#pragma unroll
                for (int s = 2; s >= 0; --s)
#pragma unroll
                    for (int p = 2; p >= 0; --p)
                        if (plane_pair(s, p, 3))
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                if (s < KP) mma_bf16(G1[mt][e], ao[s < KP ? s : 0], bs[e][0][p], bs[e][1][p]);
                                mma_bf16(G2[mt][e], aw[s], bs[e][0][p], bs[e][1][p]);
                                mma_bf16(G3[mt][e], au[s], be1[e][0][p], be1[e][1][p]);
                            }
            }
        }
    }
    // row products with q and k over this warp's columns, then the three terms in place
    auto tile2 = [&](int base, int r, int c) {                    // two neighbouring elements
        float2 x = make_float2(0.f, 0.f);
#pragma unroll
        for (int p = KP - 1; p >= 0; --p) {
            const unsigned y = *reinterpret_cast<const unsigned *>(smem + base + p * L::TILE + r * KPI + 2 * c);
            x.x += lo_f32(y);
            x.y += hi_f32(y);
        }
        return x;
    };
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = 16 * (m0 + mt) + g4 + 8 * half;
            float s1 = 0.f, s2 = 0.f, s3 = 0.f;
            const float f = from[r], f1 = f * d.scale, f2 = -be[r] * f, f3 = to[r];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int c = dk0 + 8 * e + 2 * i4;
                const float2 qq = tile2(L::Q, r, c), kk = tile2(0, r, c);
                float *a = &G1[mt][e][2 * half], *x = &G2[mt][e][2 * half], *y = &G3[mt][e][2 * half];
                a[0] *= f1; a[1] *= f1;
                y[0] *= f3; y[1] *= f3;
                s1 = fmaf(qq.x, a[0], fmaf(qq.y, a[1], s1));
                s2 = fmaf(kk.x, x[0], fmaf(kk.y, x[1], s2));
                s3 = fmaf(kk.x, y[0], fmaf(kk.y, y[1], s3));
                x[0] = fmaf(f2, x[0], y[0]);                      // both terms of dk
                x[1] = fmaf(f2, x[1], y[1]);
            }
#pragma unroll
            for (int m = 1; m < 4; m *= 2) {
                s1 += __shfl_xor_sync(~0u, s1, m);
                s2 += __shfl_xor_sync(~0u, s2, m);
                s3 += __shfl_xor_sync(~0u, s3, m);
            }
            if (i4 == 0) {
                float *p = dots + (warp % NWK) * 3 * C + r;
                p[0] = s1;
                p[C] = s2;
                p[2 * C] = s3;
            }
        }
    if (warp / NWK == 0) {                                        // warps that share columns agree
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) inner += __shfl_xor_sync(~0u, inner, m);
        if (lane == 0) ends[warp] = inner;
    }
    // the C x C blocks: A and P again, then a, p, and what goes into the gates
#pragma unroll
    for (int x = 0; x < BPW; ++x) {
        const int idx = warp + 8 * x;
        if (idx >= BLOCKS) break;
        const int bi = idx < 1 ? 0 : idx < 3 ? 1 : idx < 6 ? 2 : 3, bj = idx - bi * (bi + 1) / 2;
        float kk[2][4] = {}, qk[2][4] = {};
#pragma unroll
        for (int ks = 0; ks < DKP / 16; ++ks) {
            unsigned ak[KP][4], aq[KP][4], bk[KP][4];
#pragma unroll
            for (int p = 0; p < KP; ++p) {
                ldsm4(ak[p], frag_rc<KPI>(sk + p * L::TILE, 16 * bi, 16 * ks, lane));
                ldsm4(aq[p], frag_rc<KPI>(sq + p * L::TILE, 16 * bi, 16 * ks, lane));
                ldsm4(bk[p], frag_cr<KPI>(sk + p * L::TILE, 16 * bj, 16 * ks, lane));
            }
#pragma unroll
            for (int s = KP - 1; s >= 0; --s)
#pragma unroll
                for (int p = KP - 1; p >= 0; --p)
                    if (plane_pair(s, p, KP))
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            mma_bf16(kk[e], ak[s], bk[p][2 * e], bk[p][2 * e + 1]);
                            mma_bf16(qk[e], aq[s], bk[p][2 * e], bk[p][2 * e + 1]);
                        }
        }
        float col[2][2] = {};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int t = 16 * bi + g4 + 8 * half;
            float zr = 0.f, er = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float pa[2], aa[2];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int s = 16 * bj + 8 * e + 2 * i4 + m, i = 2 * half + m;
                    const float f = s <= t ? expf((hi[t] - hi[s]) + (lo[t] - lo[s])) : 0.f;
                    const float A = s < t ? kk[e][i] * f : 0.f, Pq = s <= t ? d.scale * (qk[e][i] * f) : 0.f;
                    const float da = s < t ? -be[t] * E[x][e][i] : 0.f, dp = s <= t ? DP[x][e][i] : 0.f;
                    const float z = fmaf(da, A, dp * Pq);
                    er = s < t ? fmaf(E[x][e][i], A, er) : er;
                    zr += z;
                    col[e][m] += z;
                    aa[m] = da * f;
                    pa[m] = d.scale * (dp * f);
                }
                unsigned pl[GP];
                const int at = t * GPI + 2 * (16 * bj + 8 * e + 2 * i4);
                split_bf16<GP>(pa[0], pa[1], pl);
#pragma unroll
                for (int p = 0; p < GP; ++p) *reinterpret_cast<unsigned *>(smem + L::P + p * L::GT + at) = pl[p];
                split_bf16<GP>(aa[0], aa[1], pl);
#pragma unroll
                for (int p = 0; p < GP; ++p) *reinterpret_cast<unsigned *>(smem + L::A + p * L::GT + at) = pl[p];
            }
#pragma unroll
            for (int m = 1; m < 4; m *= 2) {
                zr += __shfl_xor_sync(~0u, zr, m);
                er += __shfl_xor_sync(~0u, er, m);
            }
            if (i4 == 0) {
                zrow[bj * C + t] = zr;
                erow[bj * C + t] = er;
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float c = col[e][m];
                c += __shfl_xor_sync(~0u, c, 4);
                c += __shfl_xor_sync(~0u, c, 8);
                c += __shfl_xor_sync(~0u, c, 16);
                if (g4 == 0) zcol[bi * C + 16 * bj + 8 * e + 2 * i4 + m] = c;
            }
    }
    __syncthreads();
    // dq += p K;  dk += p^T Q + (a + a^T) K
    const unsigned gp = sk + L::P, ga = sk + L::A;
#pragma unroll
    for (int ks = 0; ks < NB; ++ks) {
        unsigned bk[KP][4], bq[KP][4];
#pragma unroll
        for (int p = 0; p < KP; ++p) {
            ldsm4t(bk[p], frag_rc<KPI>(sk + p * L::TILE, 16 * ks, dk0, lane));
            ldsm4t(bq[p], frag_rc<KPI>(sq + p * L::TILE, 16 * ks, dk0, lane));
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int m = m0 + mt;
            auto add = [&](float (&acc)[2][4], const unsigned (&a)[GP][4], const unsigned (&bb)[KP][4]) {
#pragma unroll
                for (int s = GP - 1; s >= 0; --s)
#pragma unroll
                    for (int p = KP - 1; p >= 0; --p)
                        if (plane_pair(s, p, GP))
#pragma unroll
                            for (int e = 0; e < 2; ++e) mma_bf16(acc[e], a[s], bb[p][2 * e], bb[p][2 * e + 1]);
            };
            unsigned a[GP][4];
            if (ks <= m) {
#pragma unroll
                for (int p = 0; p < GP; ++p) ldsm4(a[p], frag_rc<GPI>(gp + p * L::GT, 16 * m, 16 * ks, lane));
                add(G1[mt], a, bk);
#pragma unroll
                for (int p = 0; p < GP; ++p) ldsm4(a[p], frag_rc<GPI>(ga + p * L::GT, 16 * m, 16 * ks, lane));
                add(G2[mt], a, bk);
            }
            if (ks >= m) {
#pragma unroll
                for (int p = 0; p < GP; ++p) ldsm4t(a[p], frag_cr<GPI>(gp + p * L::GT, 16 * ks, 16 * m, lane));
                add(G2[mt], a, bq);
#pragma unroll
                for (int p = 0; p < GP; ++p) ldsm4t(a[p], frag_cr<GPI>(ga + p * L::GT, 16 * ks, 16 * m, lane));
                add(G2[mt], a, bk);
            }
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = 16 * (m0 + mt) + g4 + 8 * half;
            if (r >= rows) continue;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int c = dk0 + 8 * e + 2 * i4;
                if (c >= d.Dk) continue;
                const bool live = r < nt;
                store2(false, r, c, live ? G1[mt][e][2 * half] : 0.f, live ? G1[mt][e][2 * half + 1] : 0.f);
                store2(true, r, c, live ? G2[mt][e][2 * half] : 0.f, live ? G2[mt][e][2 * half + 1] : 0.f);
            }
        }
    if (warp == 0) {
        // dg_t = sum_{t' >= t} (rows - columns + products) + sum_{t' < t} (products with D1) + G_C <S0, D1>
        constexpr int PL = C / 32;
        double suf[PL], pre[PL], run = 0.0, rev = 0.0;
        float dbeta[PL];
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const int r = lane * PL + i;
            float zr = 0.f, zc = 0.f, er = 0.f, x1 = 0.f, x2 = 0.f, x3 = 0.f;
#pragma unroll
            for (int p = 0; p < NB; ++p) {
                if (16 * p <= r) {
                    zr += zrow[p * C + r];
                    er += erow[p * C + r];
                }
                if (16 * p + 15 >= r) zc += zcol[p * C + r];
            }
#pragma unroll
            for (int p = 0; p < NWK; ++p) {
                x1 += dots[(p * 3) * C + r];
                x2 += dots[(p * 3 + 1) * C + r];
                x3 += dots[(p * 3 + 2) * C + r];
            }
            dbeta[i] = dwv[r] - from[r] * x2 - er;
            pre[i] = run;                                         // of this lane's earlier tokens
            run += (double)x3;
            suf[i] = (double)((zr - zc) + (x1 - be[r] * from[r] * x2));
        }
#pragma unroll
        for (int i = PL - 1; i >= 0; --i) {
            rev += suf[i];
            suf[i] = rev;
        }
        double before = run, after = rev;
#pragma unroll
        for (int m = 1; m < 32; m *= 2) {
            const double x = __shfl_up_sync(~0u, before, m), y = __shfl_down_sync(~0u, after, m);
            if (lane >= m) before += x;
            if (lane + m < 32) after += y;
        }
        before -= run;
        after -= rev;
        double whole = 0.0;
#pragma unroll
        for (int p = 0; p < NWK; ++p) whole += (double)ends[p];
        whole *= (double)from[C - 1];
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const int r = lane * PL + i;
            if (r < rows) {
                gdec[(long long)r * d.H] = r < nt ? (float)(after + suf[i] + before + pre[i] + whole) : 0.f;
                gbeta[(long long)r * d.H] = r < nt ? dbeta[i] : 0.f;
            }
        }
    }
}

// value heads that share a key head: their parts added in head order
template <typename T>
__global__ void __launch_bounds__(256) k_delta_heads(const float *part, T *out, long long rows, int Hk, int group, int Dk) {
    const long long all = rows * Hk * (Dk / 4);
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
        const int c = (int)(i % (Dk / 4)) * 4;
        const long long rh = i / (Dk / 4);                        // row * Hk + key head
        float s[4] = {};
        for (int g = 0; g < group; ++g) {
            const float4 x = *reinterpret_cast<const float4 *>(part + (rh * group + g) * Dk + c);
            s[0] += x.x; s[1] += x.y; s[2] += x.z; s[3] += x.w;
        }
        store_vec<T, 4>(out + rh * Dk + c, s);
    }
}

template <typename T, int DKP, int NW>
cudaError_t back_scan_one(const DeltaDims &d, const DeltaIn &in, const DeltaPlanes &q, const DeltaPlanes &k,
                          const DeltaLocal &w, const DeltaBack &o, cudaStream_t st) {
    using L = BackSmem<T, DKP, NW>;
    auto kern = k_delta_back_scan<T, DKP, NW>;
    set_kernel_smem(kern, L::BYTES);
    const long long slices = (d.Dv + NW * 16 - 1) / (NW * 16);
    kern<<<(unsigned)((long long)d.B * d.H * slices), NW * 32, L::BYTES, st>>>(d, in, q, k, w, o);
    return cudaGetLastError();
}

template <typename T, int DKP>
cudaError_t back_local_one(const DeltaDims &d, const DeltaIn &in, const DeltaPlanes &q, const DeltaPlanes &k,
                           const DeltaLocal &w, const DeltaBack &o, cudaStream_t st) {
    auto kern = k_delta_back_local<T, DKP>;
    constexpr int bytes = BackLocalSmem<T, DKP>::BYTES;
    set_kernel_smem(kern, bytes);
    kern<<<(unsigned)delta_chunks(d), kBackThreads, bytes, st>>>(d, in, q, k, w, o);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || d.H == d.Hk) return e;
    const long long rows = (long long)d.B * d.T, units = rows * d.Hk * (d.Dk / 4), blocks = (units + 255) / 256;
    const unsigned grid = (unsigned)(blocks < 8 * kRefSms ? blocks : 8 * kRefSms);
    k_delta_heads<T><<<grid, 256, 0, st>>>(o.dq, static_cast<T *>(o.grad_q), rows, d.Hk, d.H / d.Hk, d.Dk);
    k_delta_heads<T><<<grid, 256, 0, st>>>(o.dk, static_cast<T *>(o.grad_k), rows, d.Hk, d.H / d.Hk, d.Dk);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_back_scan(const DeltaDims &d, const DeltaIn &in, const DeltaPlanes &q, const DeltaPlanes &k,
                                   const DeltaLocal &w, const DeltaBack &o, cudaStream_t st) {
    // as the forward's scan
    const bool wide = d.Dv > 64 && (long long)d.B * d.H * ((d.Dv + 127) / 128) >= kRefSms;
    auto go = [&](auto t, auto dkp) {
        using T = decltype(t);
        constexpr int DKP = decltype(dkp)::value;
        return wide ? back_scan_one<T, DKP, 8>(d, in, q, k, w, o, st) : back_scan_one<T, DKP, 4>(d, in, q, k, w, o, st);
    };
    auto size = [&](auto t) {
        return d.Dk <= 64 ? go(t, std::integral_constant<int, 64>{}) : go(t, std::integral_constant<int, 128>{});
    };
    return d.dtype == SDM_BF16 ? size(__nv_bfloat16{}) : size(float{});
}

cudaError_t launch_delta_back_local(const DeltaDims &d, const DeltaIn &in, const DeltaPlanes &q, const DeltaPlanes &k,
                                    const DeltaLocal &w, const DeltaBack &o, cudaStream_t st) {
    if (d.dtype == SDM_BF16)
        return d.Dk <= 64 ? back_local_one<__nv_bfloat16, 64>(d, in, q, k, w, o, st)
                          : back_local_one<__nv_bfloat16, 128>(d, in, q, k, w, o, st);
    return d.Dk <= 64 ? back_local_one<float, 64>(d, in, q, k, w, o, st)
                      : back_local_one<float, 128>(d, in, q, k, w, o, st);
}

}  // namespace sdm
