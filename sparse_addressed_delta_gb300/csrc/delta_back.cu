// Backward of the gated delta rule in chunks (notation of delta_chunk.cu; dO the readings' gradient,
// D1 the gradient of a chunk's end state, D0 of its start state):
//   du = P^T dO + (e^{L_C - L} K) D1;   dw = X^T du;   dv = beta dw
//   D0 = G_C D1 + (scale G Q)^T dO - K^T (beta G dw)
// is a recurrence over the chunks from the last to the first (k_delta_back_scan; 32 chunks of 8 float32 heads
// of 64 x 64 in segments 44 us and the join 16, in one run 95), the forward scan's
// mirror image: a warp owns 16 columns, and accumulators pass from product to product as A operands.
// (X = (I + diag(beta) A)^-1 here.) Everything else needs only a chunk's own S0 and r (saved by the forward), D1 and dw (left by the scan), and runs for all chunks at once (k_delta_back_local):
//   a[t,s] = -beta_t beta_s <dw_t, r_s> e^{L_t - L_s}  (s < t)
//   p[t,s] = scale beta_s <dO_t, r_s> e^{L_t - L_s}    (s <= t)
//   dq = p K + scale G (dO S0^T)
//   dk = p^T Q + (a + a^T) K - beta G (dw S0^T) + e^{L_C - L} beta (r D1^T)
//   dbeta_t = <dw_t, r_t>
// A log-decay's gradient is the sum of everything that crosses its token, all of it scaled by the decay itself:
//   z[t,s] = p[t,s] (q_t . k_s) + a[t,s] (k_t . k_s)  (s < t);   x_t = <q_t, scale G dO_t S0^T> - <k_t, beta G dw_t S0^T>
//   y_s = <k_s, e^{L_C - L} beta r_s D1^T>
//   dg_t = sum_{t' >= t, s < t} z[t',s] + sum_{t' >= t} x_t' + sum_{s < t} y_s + G_C <S0, D1>
// the first by suffix sums of row sums less column sums. (Sums without that scale, as of <o, dO> - <v, dv>, cancel
// to it: at g = -10 they leave an error of 1 %.) Where e^g is 0 it is 0. All products keep float32's accuracy.
#include "delta_internal.cuh"

namespace sdm {
namespace {

template <int DKP, int NW>
struct BackSmem {
    static constexpr int C = 32, KP = 3, PP = 3;
    static constexpr int XP = delta_pitch(C * 2), VP = delta_pitch(NW * 16 * 4);
    static constexpr int KPI = delta_pitch(DKP * 2), TILE = C * KPI;
    static constexpr int Q = KP * TILE, X = 2 * KP * TILE, P = X + 3 * C * XP, V = P + PP * C * XP;
    static constexpr int AUX = V + C * VP, STAGE = AUX + 3 * C * 4;
    static constexpr int BYTES = 2 * STAGE;
    static_assert(BYTES <= 227 * 1024, "shared memory");
};

// One block per head and NW * 16 of its columns, from the last chunk to the first.
template <int DKP, int NW>
__global__ void __launch_bounds__(NW * 32, 1)
    k_delta_back_scan(DeltaDims d, DeltaIn in, DeltaPlanes q, DeltaPlanes k, DeltaLocal w, DeltaBack o, int mode) {
    using L = BackSmem<DKP, NW>;
    constexpr int C = L::C, KP = L::KP, PP = L::PP, XP = L::XP, VP = L::VP, KPI = L::KPI, THREADS = NW * 32;
    constexpr int NT = C / 8, ND = DKP / 8, VE = 16 / 4;
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g4 = lane >> 2, i4 = lane & 3;
    const bool carry = mode == DELTA_CARRY_BACK;
    const DeltaBlock blk = delta_block(d, in.valid, d.segs > 1, mode, NW * 16);
    const int dv_blk = blk.tile * NW * 16;
    const long long bh = blk.bh;
    const int b = (int)(bh / d.H), h = (int)(bh % d.H), hk = h / (d.H / d.Hk);
    const int dv0 = dv_blk + 16 * warp;
    const bool mine = dv0 < d.Dv;
    const int ntok = delta_valid(in.valid, b, d.T), chunks = (ntok + C - 1) / C;
    const int n0 = delta_bound(d, chunks, blk.seg), n1 = delta_bound(d, chunks, blk.seg + 1), nch = n1 - n0;
    const bool last = blk.seg + 1 == d.segs;
    const float *grad = static_cast<const float *>(o.grad) + b * d.os[0] + h * d.os[2] + dv_blk;
    const long long kbase = b * k.s[0] + hk * k.s[2], qbase = b * q.s[0] + hk * q.s[2];
    float *gv = static_cast<float *>(o.grad_v) + ((long long)b * d.T * d.H + h) * d.Dv;
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
        load_values<float, NW * 16, C, THREADS>(st + L::V, grad + t0 * d.os[1], d.os[1], nt, d.Dv - dv_blk, tid);
        for (int i = tid; i < 3 * C / 4; i += THREADS)
            cp_async16_zfill(st + L::AUX + 16 * i, w.aux + bhn * kDeltaAux * C + 4 * i, true);
        cp_async_commit();
    };
    // element e of the state's fragment j: row 8 j + 2 i4 + (e & 1), column dv0 + g4 + 8 (e >> 1)
    float S[ND][4];
    const float *from_end = d.segs > 1 && !carry ? w.starts + blk.seg * delta_states(d) : carry && !last ? nullptr : o.state_in;
    const float *sp = from_end + (bh * d.Dk) * d.Dv + dv0;
#pragma unroll
    for (int j = 0; j < ND; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int dk = 8 * j + 2 * i4 + (e & 1);
            S[j][e] = mine && from_end && dk < d.Dk ? sp[(size_t)dk * d.Dv + g4 + 8 * (e >> 1)] : 0.f;
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
    if (nch > 0) load(n1 - 1, 0);
    for (int it = 0; it < nch; ++it) {
        const int n = n1 - 1 - it;
        if (n > n0) {
            load(n - 1, (it + 1) & 1);
            cp_async_wait<1>();
        } else {
            cp_async_wait<0>();
        }
        __syncthreads();
        const int stage = (it & 1) * L::STAGE;
        const unsigned sk = s0 + stage, sq = sk + L::Q, sx = sk + L::X, spp = sk + L::P, sv = sk + L::V;
        const float *from = reinterpret_cast<const float *>(smem + stage + L::AUX), *to = from + C, *be = to + C;
        const int nt = ntok - n * C < C ? ntok - n * C : C;
        if (mine) {
            if (!carry) store_state(o.ends + ((bh * d.Nt + n) * (long long)d.Dk) * d.Dv + dv0);
            // dO^T as an A operand, K step ks: KP planes of the stored values times `f` of the token
            auto grads = [&](int ks, float (&x)[4][2]) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int t = 16 * ks + 8 * (i >> 1) + 2 * i4 + e, c = 16 * warp + g4 + 8 * (i & 1);
                        x[i][e] = *reinterpret_cast<const float *>(smem + stage + L::V + delta_at<VP>(t, c >> 2) + 4 * (c & 3));
                    }
            };
            float D[NT][4] = {};
#pragma unroll
            for (int pk = 2 * DKP / 16 - 1; pk >= 0; --pk) { // D = (K D1)^T
                const int pass = pk / (DKP / 16), ks = pk % (DKP / 16);
                unsigned a[3][4], bb[KP][C / 16][4];
                split_frag<3>(S, ks, a);
#pragma unroll
                for (int p = 0; p < KP; ++p)
#pragma unroll
                    for (int jj = 0; jj < C / 16; ++jj)
                        if (pass > 0 || p == 0) ldsm4(bb[p][jj], frag_cr<KPI>(sk + p * L::TILE, 16 * jj, 16 * ks, lane));
#pragma unroll
                for (int x = 2; x >= 0; --x)
#pragma unroll
                    for (int p = KP - 1; p >= 0; --p)
                        if (plane_pair(x, p, 3, pass))
#pragma unroll
                            for (int j = 0; j < NT; ++j)
                                mma_bf16(D[j], a[x], bb[p][j >> 1][2 * (j & 1)], bb[p][j >> 1][2 * (j & 1) + 1]);
            }
            float W[NT][4] = {};
#pragma unroll
            for (int pk = 2 * C / 16 - 1; pk >= 0; --pk) {   // D += (P^T dO)^T
                const int pass = pk / (C / 16), ks = pk % (C / 16);
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
                    for (int p = 0; p < PP; ++p)
                        if (pass > 0 || p == 0) ldsm4t(bb[p], frag_rc<XP>(spp + p * C * XP, 16 * ks, 16 * jj, lane));
#pragma unroll
                    for (int y = KP - 1; y >= 0; --y)
#pragma unroll
                        for (int p = PP - 1; p >= 0; --p)
                            if (plane_pair(y, p, 3, pass)) {
                                mma_bf16(W[2 * jj], a[y], bb[p][0], bb[p][1]);
                                mma_bf16(W[2 * jj + 1], a[y], bb[p][2], bb[p][3]);
                            }
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    D[j][e] = fmaf(D[j][e], to[8 * j + 2 * i4 + (e & 1)], W[j][e]);
                    W[j][e] = 0.f;
                }
#pragma unroll
            for (int pk = 2 * C / 16 - 1; pk >= 0; --pk) {   // W = (X^T du)^T
                const int pass = pk / (C / 16), ks = pk % (C / 16);
                unsigned a[3][4];
                split_frag<3>(D, ks, a);
#pragma unroll
                for (int jj = 0; jj <= ks; ++jj) {
                    unsigned bb[3][4];
#pragma unroll
                    for (int p = 0; p < 3; ++p)
                        if (pass > 0 || p == 0) ldsm4t(bb[p], frag_rc<XP>(sx + p * C * XP, 16 * ks, 16 * jj, lane));
#pragma unroll
                    for (int x = 2; x >= 0; --x)
#pragma unroll
                        for (int p = 2; p >= 0; --p)
                            if (plane_pair(x, p, 3, pass)) {
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
                    for (int pk = 2 * C / 16 - 1; pk >= 0; --pk) {
                        const int pass = pk / (C / 16), ks = pk % (C / 16);
                        unsigned bb[KP][2][4];
#pragma unroll
                        for (int p = 0; p < KP; ++p)
#pragma unroll
                            for (int m = 0; m < 2; ++m)
                                if (pass > 0 || p == 0) ldsm4t(bb[p][m], frag_rc<KPI>(tile + p * L::TILE, 16 * ks, 16 * (nn + m), lane));
#pragma unroll
                        for (int x = 2; x >= 0; --x)
#pragma unroll
                            for (int p = KP - 1; p >= 0; --p)
                                if (plane_pair(x, p, 3, pass))
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
                    if (!carry) dst[(size_t)t * d.Dv + g4 + 8 * (e >> 1)] = W[j][e];
                    const float x = be[t] * W[j][e];
                    *reinterpret_cast<float *>(smem + stage + L::V + delta_at<VP>(t, c / VE) + (c % VE) * 4) = x;
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
                if (t < d.T && !carry) *reinterpret_cast<uint4 *>(gv + t * orow + dv0 + c * VE) = x;
            }
        }
        __syncthreads();
    }
    if (!mine) return;
    if (carry)
        store_state(w.starts + (blk.seg - 1) * delta_states(d) + (bh * d.Dk) * d.Dv + dv0);
    else if (blk.seg == 0)
        store_state(o.state_out + (bh * d.Dk) * d.Dv + dv0);
    if (carry || !last) return;
    constexpr int PR = 16 / VE;
    for (long long t = (long long)chunks * C + lane / PR; t < d.T; t += 32 / PR)
        *reinterpret_cast<uint4 *>(gv + t * orow + dv0 + (lane % PR) * VE) = make_uint4(0u, 0u, 0u, 0u);
}

constexpr int kBackCols = 128;                        // columns of the state at a time

template <typename T, int DKP>
struct BackLocalSmem {
    static constexpr bool BF = sizeof(T) == 2;
    static constexpr int C = BF ? 64 : 32, NB = C / 16;
    static constexpr int KP = BF ? 1 : 3;             // planes of q, k and dO
    static constexpr int PL = 3;                      // terms of float32 operands
    static constexpr int NWK = DKP / 16, WARPS = NWK * NB < 16 ? NWK * NB : 16;
    static constexpr int KPI = delta_pitch(DKP * 2), TILE = C * KPI;
    static constexpr int VPI = delta_pitch(kBackCols * 2), VT = C * VPI;   // planes of dO, dw and r
    static constexpr int GPI = delta_pitch(C * 2), GT = C * GPI;           // planes of p and a
    static constexpr int Q = KP * TILE, O = 2 * KP * TILE, W = O + KP * VT, R = W + PL * VT;
    static constexpr int P = R + 3 * VT, A = P + PL * GT, F = A + PL * GT;
    // floats: hi, lo, from, to, beta, <dw, r> [C]; row and column sums of z [NB][C]; x and y [NWK][C]; <S0, D1>
    // [WARPS]
    static constexpr int FLOATS = 6 * C + 2 * NB * C + 2 * NWK * C + WARPS;
    static constexpr int BYTES = F + FLOATS * 4;
    static_assert(BYTES <= 227 * 1024, "shared memory");
};

// One block per chunk and head. For the products with the states a warp owns 16 of the Dk columns and a
// part of the tokens, and reads its rows of S0 and D1 straight into fragments, one step ahead; the C x C
// products are split into 16 x 16 blocks, a warp each.
// What bounds it: the m16n8k16 products, about 11400 a chunk of 64 and head at Dk = Dv = 128 (8 cycles each on
// one of four tensor cores), and its phases in turn with one block an SM (tensor pipe 30 %); 8 float32 heads of 64 x
// 64 x 32 chunks take 25 us, 64 bfloat16 heads of 128 x 192 x 64 chunks 1340.
template <typename T, int DKP>
__global__ void __launch_bounds__(BackLocalSmem<T, DKP>::WARPS * 32, 1)
    k_delta_back_local(DeltaDims d, DeltaIn in, DeltaPlanes q, DeltaPlanes k, DeltaLocal lw, DeltaBack o) {
    using L = BackLocalSmem<T, DKP>;
    constexpr bool BF = L::BF;
    constexpr int C = L::C, KP = L::KP, PL = L::PL, NB = L::NB, KPI = L::KPI, VPI = L::VPI, GPI = L::GPI;
    constexpr int THREADS = L::WARPS * 32, NWK = L::NWK, MS = L::WARPS / NWK, MT = NB / MS;
    constexpr int BLOCKS = NB * (NB + 1) / 2;
    static_assert(MT >= 1 && BLOCKS <= L::WARPS, "tokens and blocks");
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
        for (int i = tid; i < rows * (d.Dk / 2); i += THREADS) {
            store2(false, i / (d.Dk / 2), 2 * (i % (d.Dk / 2)), 0.f, 0.f);
            store2(true, i / (d.Dk / 2), 2 * (i % (d.Dk / 2)), 0.f, 0.f);
        }
        for (int r = tid; r < rows; r += THREADS) gdec[(long long)r * d.H] = gbeta[(long long)r * d.H] = 0.f;
        return;
    }
    const unsigned sk = smem_u32(smem), sq = sk + L::Q, so = sk + L::O, sw = sk + L::W, sr = sk + L::R;
    float *hi = reinterpret_cast<float *>(smem + L::F), *lo = hi + C, *from = lo + C, *to = from + C, *be = to + C;
    float *dwr = be + C, *zrow = dwr + C, *zcol = zrow + NB * C, *xs_t = zcol + NB * C, *ys_t = xs_t + NWK * C, *ends = ys_t + NWK * C;

    load_tokens<KP, DKP, C, THREADS>(sk, k, b * k.s[0] + t0 * k.s[1] + hk * k.s[2], d.Dk, nt, tid);
    load_tokens<KP, DKP, C, THREADS>(sq, q, b * q.s[0] + t0 * q.s[1] + hk * q.s[2], d.Dk, nt, tid);
    cp_async_commit();
    for (int i = tid; i < C; i += THREADS) {
        const float *aux = lw.aux + bhn * kDeltaAux * C;
        from[i] = aux[i];
        to[i] = aux[C + i];
        be[i] = aux[2 * C + i];
        hi[i] = aux[3 * C + i];
        lo[i] = aux[4 * C + i];
    }
    for (int i = tid; i < C; i += THREADS) dwr[i] = 0.f;

    const T *grad = static_cast<const T *>(o.grad) + b * d.os[0] + t0 * d.os[1] + h * d.os[2];
    const float *wp = o.w + bhn * C * (long long)d.Dv, *rp = o.r + bhn * C * (long long)d.Dv;
    const int dk0 = 16 * (warp % NWK), m0 = (warp / NWK) * MT;    // this warp's Dk columns and token tiles
    const long long cells = (long long)d.Dk * d.Dv;
    const float *s0p = o.snap + (bh * (d.Nt + 1) + n) * cells, *d1p = o.ends + bhn * cells;
    {
        const float4 *x = reinterpret_cast<const float4 *>(s0p), *y = reinterpret_cast<const float4 *>(d1p);
        float s = 0.f;
#pragma unroll 2
        for (int i = tid; i < (int)(cells / 4); i += THREADS) {
            const float4 u = __ldg(x + i), v = __ldg(y + i);
            s = fmaf(u.x, v.x, fmaf(u.y, v.y, fmaf(u.z, v.z, fmaf(u.w, v.w, s))));
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(~0u, s, m);
        if (lane == 0) ends[warp] = s;
    }
    // 16 x 16 block (bi, bj) of the C x C products, on or below the diagonal
    const bool block = warp < BLOCKS;
    const int bi = warp < 1 ? 0 : warp < 3 ? 1 : warp < 6 ? 2 : 3, bj = warp - bi * (bi + 1) / 2;
    // of the products that reach the gates or float32 gradients, the lesser terms have sums of their own: the
    // tensor core cuts an accumulator's low bits at every step
    float G1[MT][2][4] = {}, L1[MT][2][4] = {}, G2[MT][2][4] = {}, G3[MT][2][4] = {}, E[2][4] = {}, DP[2][4] = {}, LP[2][4] = {};
    float low2[BF ? 1 : MT][2][4] = {}, low3[BF ? 1 : MT][2][4] = {}, lowe[2][4] = {};
    auto &L2 = *(BF ? (float (*)[MT][2][4])&G2 : (float (*)[MT][2][4])&low2);
    auto &L3 = *(BF ? (float (*)[MT][2][4])&G3 : (float (*)[MT][2][4])&low3);
    auto &LE = *(BF ? &E : &lowe);
    for (int c0 = 0; c0 < d.Dv; c0 += kBackCols) {
        __syncthreads();
        // dO, dw and r of this column tile as planes; <dw, r>
        for (int i = tid; i < C * (kBackCols / 8); i += THREADS) {
            const int r = i / (kBackCols / 8), c = i % (kBackCols / 8), col = c0 + 8 * c;
            const bool live = r < nt && col < d.Dv;
            float g[8] = {}, x[8] = {}, u[8] = {};
            if (live) {
                load_vec<T, 8, true>(grad + r * d.os[1] + col, g);
                load_vec<float, 8, true>(wp + (long long)r * d.Dv + col, x);
                load_vec<float, 8, true>(rp + (long long)r * d.Dv + col, u);
            }
            float z = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) z = fmaf(x[e], u[e], z);
#pragma unroll
            for (int m = 1; m < kBackCols / 8; m *= 2) z += __shfl_xor_sync(~0u, z, m);
            if (c == 0) dwr[r] += z;
            auto put = [&](unsigned char *dst, const float (&y)[8], auto planes) {
                constexpr int N = decltype(planes)::value;
                unsigned p[4][N];
#pragma unroll
                for (int e = 0; e < 4; ++e) split_bf16<N>(y[2 * e], y[2 * e + 1], p[e]);
#pragma unroll
                for (int m = 0; m < N; ++m)
                    *reinterpret_cast<uint4 *>(dst + m * L::VT + delta_at<VPI>(r, c)) = make_uint4(p[0][m], p[1][m], p[2][m], p[3][m]);
            };
            put(smem + L::O, g, std::integral_constant<int, KP>{});
            put(smem + L::W, x, std::integral_constant<int, PL>{});
            put(smem + L::R, u, std::integral_constant<int, 3>{});
        }
        const int rest = d.Dv - c0 < kBackCols ? d.Dv - c0 : kBackCols;
        // this lane's two rows of the states: columns 2 i4 and 8 + 2 i4 of each 16
        float2 xs[2][2], ys[2][2];
        auto fetch_into = [&](float2 (&x)[2][2], const float *from, int ks) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int row = dk0 + 8 * e + g4;
                    const bool live = row < d.Dk && 16 * ks < rest;
                    x[e][m] = live ? __ldg(reinterpret_cast<const float2 *>(from + (long long)row * d.Dv + c0 + 16 * ks + 8 * m + 2 * i4)) : make_float2(0.f, 0.f);
                }
        };
        fetch_into(xs, s0p, 0);
        fetch_into(ys, d1p, 0);
        cp_async_wait<0>();
        __syncthreads();
        // E += dw r^T, dP += dO r^T
        if (block) {
#pragma unroll 1
            for (int ks = 0; ks < rest / 16; ++ks) {
                unsigned aw[PL][4], ao[KP][4], br[3][4];
#pragma unroll
                for (int p = 0; p < PL; ++p) ldsm4(aw[p], frag_rc<VPI>(sw + p * L::VT, 16 * bi, 16 * ks, lane));
#pragma unroll
                for (int p = 0; p < 3; ++p) ldsm4(br[p], frag_cr<VPI>(sr + p * L::VT, 16 * bj, 16 * ks, lane));
#pragma unroll
                for (int p = 0; p < KP; ++p) ldsm4(ao[p], frag_rc<VPI>(so + p * L::VT, 16 * bi, 16 * ks, lane));
#pragma unroll
                for (int s = 2; s >= 0; --s)
#pragma unroll
                    for (int p = 2; p >= 0; --p)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (s < PL && plane_pair(s, p, PL)) mma_bf16(s + p ? LE[e] : E[e], aw[s < PL ? s : 0], br[p][2 * e], br[p][2 * e + 1]);
                            if (s < KP && plane_pair(s, p, 3)) mma_bf16(s + p ? LP[e] : DP[e], ao[s < KP ? s : 0], br[p][2 * e], br[p][2 * e + 1]);
                        }
            }
        }
        // products with the states over this column tile
        for (int ks = 0; ks < rest / 16; ++ks) {
            unsigned bs[2][2][3];                                 // [8-column tile][k half][plane]
            auto split = [&](const float2 (&x)[2][2]) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int m = 0; m < 2; ++m) split_bf16<3>(x[e][m].x, x[e][m].y, bs[e][m]);
            };
            split(ys);
            fetch_into(ys, d1p, ks + 1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                unsigned a[PL][4];
#pragma unroll
                for (int p = 0; p < PL; ++p) ldsm4(a[p], frag_rc<VPI>(sr + p * L::VT, 16 * (m0 + mt), 16 * ks, lane));
#pragma unroll
                for (int s = PL - 1; s >= 0; --s)
#pragma unroll
                    for (int p = PL - 1; p >= 0; --p)
                        if (plane_pair(s, p, PL))
#pragma unroll
                            for (int e = 0; e < 2; ++e) mma_bf16(s + p ? L3[mt][e] : G3[mt][e], a[s], bs[e][0][p], bs[e][1][p]);
            }
            split(xs);
            fetch_into(xs, s0p, ks + 1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                unsigned a[3][4];
                const int r0 = 16 * (m0 + mt);
#pragma unroll
                for (int p = 0; p < KP; ++p) ldsm4(a[p], frag_rc<VPI>(so + p * L::VT, r0, 16 * ks, lane));
#pragma unroll
                for (int s = KP - 1; s >= 0; --s)
#pragma unroll
                    for (int p = 2; p >= 0; --p)
                        if (plane_pair(s, p, 3))
#pragma unroll
                            for (int e = 0; e < 2; ++e) mma_bf16(s + p ? L1[mt][e] : G1[mt][e], a[s], bs[e][0][p], bs[e][1][p]);
#pragma unroll
                for (int p = 0; p < PL; ++p) ldsm4(a[p], frag_rc<VPI>(sw + p * L::VT, r0, 16 * ks, lane));
#pragma unroll
                for (int s = PL - 1; s >= 0; --s)
#pragma unroll
                    for (int p = PL - 1; p >= 0; --p)
                        if (plane_pair(s, p, PL))
#pragma unroll
                            for (int e = 0; e < 2; ++e) mma_bf16(s + p ? L2[mt][e] : G2[mt][e], a[s], bs[e][0][p], bs[e][1][p]);
            }
        }
    }
    // the terms of dq and dk in place, and x and y over this warp's columns
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = 16 * (m0 + mt) + g4 + 8 * half;
            float s1 = 0.f, s2 = 0.f;
            const float f = from[r], f1 = f * d.scale, f2 = -be[r] * f, f3 = to[r] * be[r];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int c = dk0 + 8 * e + 2 * i4;
                float *a = &G1[mt][e][2 * half], *x = &G2[mt][e][2 * half], *y = &G3[mt][e][2 * half];
                a[0] = (a[0] + L1[mt][e][2 * half]) * f1;
                a[1] = (a[1] + L1[mt][e][2 * half + 1]) * f1;
                if constexpr (!BF) {
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        x[m] += L2[mt][e][2 * half + m];
                        y[m] += L3[mt][e][2 * half + m];
                    }
                }
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    x[m] *= f2;
                    y[m] *= f3;
                }
#pragma unroll
                for (int p = KP - 1; p >= 0; --p) {
                    const int at = p * L::TILE + r * KPI + 2 * c;
                    const unsigned qq = *reinterpret_cast<const unsigned *>(smem + L::Q + at), kk = *reinterpret_cast<const unsigned *>(smem + at);
                    s1 = fmaf(lo_f32(qq), a[0], fmaf(hi_f32(qq), a[1], fmaf(lo_f32(kk), x[0], fmaf(hi_f32(kk), x[1], s1))));
                    s2 = fmaf(lo_f32(kk), y[0], fmaf(hi_f32(kk), y[1], s2));
                }
                x[0] += y[0];
                x[1] += y[1];
            }
#pragma unroll
            for (int m = 1; m < 4; m *= 2) {
                s1 += __shfl_xor_sync(~0u, s1, m);
                s2 += __shfl_xor_sync(~0u, s2, m);
            }
            if (i4 == 0) {
                xs_t[(warp % NWK) * C + r] = s1;
                ys_t[(warp % NWK) * C + r] = s2;
            }
        }
    // the C x C blocks: q k^T and k k^T again, then a, p and the row and column sums of z
    if (block) {
        float qk[2][4] = {}, lq[2][4] = {}, kk[2][4] = {}, lk[2][4] = {};
#pragma unroll
        for (int ks = 0; ks < DKP / 16; ++ks) {
            unsigned aq[KP][4], ak[KP][4], bk[KP][4];
#pragma unroll
            for (int p = 0; p < KP; ++p) {
                ldsm4(aq[p], frag_rc<KPI>(sq + p * L::TILE, 16 * bi, 16 * ks, lane));
                ldsm4(ak[p], frag_rc<KPI>(sk + p * L::TILE, 16 * bi, 16 * ks, lane));
                ldsm4(bk[p], frag_cr<KPI>(sk + p * L::TILE, 16 * bj, 16 * ks, lane));
            }
#pragma unroll
            for (int s = KP - 1; s >= 0; --s)
#pragma unroll
                for (int p = KP - 1; p >= 0; --p)
                    if (plane_pair(s, p, KP))
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            mma_bf16(s + p ? lq[e] : qk[e], aq[s], bk[p][2 * e], bk[p][2 * e + 1]);
                            mma_bf16(s + p ? lk[e] : kk[e], ak[s], bk[p][2 * e], bk[p][2 * e + 1]);
                        }
        }
        float zc[2][2] = {};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int t = 16 * bi + g4 + 8 * half;
            float zr = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float pa[2], aa[2];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int s = 16 * bj + 8 * e + 2 * i4 + m, i = 2 * half + m;
                    const float f = s <= t ? expf((hi[t] - hi[s]) + (lo[t] - lo[s])) * be[s] : 0.f;
                    pa[m] = s <= t ? d.scale * ((DP[e][i] + LP[e][i]) * f) : 0.f;
                    aa[m] = s < t ? -be[t] * ((BF ? E[e][i] : E[e][i] + LE[e][i]) * f) : 0.f;
                    const float z = s < t ? fmaf(pa[m], qk[e][i] + lq[e][i], aa[m] * (kk[e][i] + lk[e][i])) : 0.f;
                    zr += z;
                    zc[e][m] += z;
                }
                unsigned pl[PL];
                const int at = t * GPI + 2 * (16 * bj + 8 * e + 2 * i4);
                split_bf16<PL>(pa[0], pa[1], pl);
#pragma unroll
                for (int p = 0; p < PL; ++p) *reinterpret_cast<unsigned *>(smem + L::P + p * L::GT + at) = pl[p];
                split_bf16<PL>(aa[0], aa[1], pl);
#pragma unroll
                for (int p = 0; p < PL; ++p) *reinterpret_cast<unsigned *>(smem + L::A + p * L::GT + at) = pl[p];
            }
            zr += __shfl_xor_sync(~0u, zr, 1);
            zr += __shfl_xor_sync(~0u, zr, 2);
            if (i4 == 0) zrow[bj * C + t] = zr;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
#pragma unroll
                for (int w = 4; w < 32; w *= 2) zc[e][m] += __shfl_xor_sync(~0u, zc[e][m], w);
                if (g4 == 0) zcol[bi * C + 16 * bj + 8 * e + 2 * i4 + m] = zc[e][m];
            }
    }
    __syncthreads();
    if (warp == L::WARPS - 1) {
        constexpr int TL = C / 32;
        float x[TL], y[TL];
        double whole = 0.0;
#pragma unroll
        for (int i = 0; i < TL; ++i) {
            const int r = lane * TL + i;
            x[i] = y[i] = 0.f;
#pragma unroll
            for (int p = 0; p < NB; ++p) {
                if (16 * p <= r) x[i] += zrow[p * C + r];
                if (16 * p + 15 >= r) x[i] -= zcol[p * C + r];
            }
#pragma unroll
            for (int p = 0; p < NWK; ++p) {
                x[i] += xs_t[p * C + r];
                y[i] += ys_t[p * C + r];
            }
        }
#pragma unroll
        for (int p = 0; p < L::WARPS; ++p) whole += (double)ends[p];
        double dg[TL];
        delta_decay_sums(x, y, (double)from[C - 1] * whole, dg);
#pragma unroll
        for (int i = 0; i < TL; ++i) {
            const int r = lane * TL + i;
            if (r < rows) {
                const bool some = r < nt && expf(delta_decay(in.g[b * d.gs[0] + (t0 + r) * d.gs[1] + h * d.gs[2]])) != 0.f;
                gdec[(long long)r * d.H] = some ? (float)dg[i] : 0.f;
                gbeta[(long long)r * d.H] = r < nt ? dwr[r] : 0.f;
            }
        }
    }
    // dq += p K;  dk += p^T Q + (a + a^T) K: float32 gradients in sums of their own, joined at the end
    float H1[MT][2][4] = {};
    if constexpr (!BF) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) G3[mt][e][i] = L1[mt][e][i] = L2[mt][e][i] = 0.f;
    }
    auto &Q1 = *(BF ? &G1 : &H1), &QL = *(BF ? &G1 : &L1), &K1 = *(BF ? &G2 : &G3), &KL = L2;
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
            auto add = [&](float (&acc)[2][4], float (&low)[2][4], const unsigned (&a)[PL][4], const unsigned (&bb)[KP][4]) {
#pragma unroll
                for (int s = PL - 1; s >= 0; --s)
#pragma unroll
                    for (int p = KP - 1; p >= 0; --p)
                        if (plane_pair(s, p, PL))
#pragma unroll
                            for (int e = 0; e < 2; ++e) mma_bf16(s + p ? low[e] : acc[e], a[s], bb[p][2 * e], bb[p][2 * e + 1]);
            };
            unsigned a[PL][4];
            if (ks <= m) {
#pragma unroll
                for (int p = 0; p < PL; ++p) ldsm4(a[p], frag_rc<GPI>(gp + p * L::GT, 16 * m, 16 * ks, lane));
                add(Q1[mt], QL[mt], a, bk);
#pragma unroll
                for (int p = 0; p < PL; ++p) ldsm4(a[p], frag_rc<GPI>(ga + p * L::GT, 16 * m, 16 * ks, lane));
                add(K1[mt], KL[mt], a, bk);
            }
            if (ks >= m) {
#pragma unroll
                for (int p = 0; p < PL; ++p) ldsm4t(a[p], frag_cr<GPI>(gp + p * L::GT, 16 * ks, 16 * m, lane));
                add(K1[mt], KL[mt], a, bq);
#pragma unroll
                for (int p = 0; p < PL; ++p) ldsm4t(a[p], frag_cr<GPI>(ga + p * L::GT, 16 * ks, 16 * m, lane));
                add(K1[mt], KL[mt], a, bk);
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
                if constexpr (!BF) {
#pragma unroll
                    for (int j = 2 * half; j < 2 * half + 2; ++j) {
                        G1[mt][e][j] += H1[mt][e][j] + L1[mt][e][j];
                        G2[mt][e][j] += G3[mt][e][j] + L2[mt][e][j];
                    }
                }
                store2(false, r, c, live ? G1[mt][e][2 * half] : 0.f, live ? G1[mt][e][2 * half + 1] : 0.f);
                store2(true, r, c, live ? G2[mt][e][2 * half] : 0.f, live ? G2[mt][e][2 * half + 1] : 0.f);
            }
        }
}

// value heads that share a key head: their parts of the gradients of q and k (blockIdx.y) added in head order
template <typename T>
__global__ void __launch_bounds__(256) k_delta_heads(DeltaBack o, long long rows, int Hk, int group, int Dk) {
    const float *part = blockIdx.y ? o.dk : o.dq;
    T *out = static_cast<T *>(blockIdx.y ? o.grad_k : o.grad_q);
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

template <int DKP, int NW>
cudaError_t back_scan_one(const DeltaDims &d, const DeltaIn &in, const DeltaPlanes &q, const DeltaPlanes &k,
                          const DeltaLocal &w, const DeltaBack &o, cudaStream_t st) {
    using L = BackSmem<DKP, NW>;
    auto kern = k_delta_back_scan<DKP, NW>;
    set_kernel_smem(kern, L::BYTES);
    auto run = [&](int mode) {
        kern<<<(unsigned)delta_blocks(d, mode, NW * 16), NW * 32, L::BYTES, st>>>(d, in, q, k, w, o, mode);
        return cudaGetLastError();
    };
    if (d.segs > 1) {
        cudaError_t e = run(DELTA_CARRY_BACK);
        if (e == cudaSuccess) e = launch_delta_join(d, w, o.state_in, true, st);
        if (e != cudaSuccess) return e;
    }
    return run(DELTA_RUN);
}

template <typename T, int DKP>
cudaError_t back_local_one(const DeltaDims &d, const DeltaIn &in, const DeltaPlanes &q, const DeltaPlanes &k,
                           const DeltaLocal &w, const DeltaBack &o, cudaStream_t st) {
    auto kern = k_delta_back_local<T, DKP>;
    constexpr int bytes = BackLocalSmem<T, DKP>::BYTES;
    set_kernel_smem(kern, bytes);
    kern<<<(unsigned)delta_chunks(d), BackLocalSmem<T, DKP>::WARPS * 32, bytes, st>>>(d, in, q, k, w, o);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || d.H == d.Hk) return e;
    const long long rows = (long long)d.B * d.T, units = rows * d.Hk * (d.Dk / 4), blocks = (units + 255) / 256;
    const unsigned grid = (unsigned)(blocks < 4 * kRefSms ? blocks : 4 * kRefSms);
    k_delta_heads<T><<<dim3(grid, 2), 256, 0, st>>>(o, rows, d.Hk, d.H / d.Hk, d.Dk);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_back_scan(const DeltaDims &d, const DeltaIn &in, const DeltaPlanes &q, const DeltaPlanes &k,
                                   const DeltaLocal &w, const DeltaBack &o, cudaStream_t st) {
    // as the forward's scan
    const bool wide = d.Dv > 64 && (long long)d.B * d.H * ((d.Dv + 127) / 128) >= kRefSms;
    auto go = [&](auto dkp) {
        constexpr int DKP = decltype(dkp)::value;
        return wide ? back_scan_one<DKP, 8>(d, in, q, k, w, o, st) : back_scan_one<DKP, 4>(d, in, q, k, w, o, st);
    };
    return d.Dk <= 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, 128>{});
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
