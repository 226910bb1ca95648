// The gated delta rule in chunks of C tokens. With S0 the state at a chunk's start, L the running
// sum of the log-decays inside the chunk (inclusive) and G = e^L:
//   A[t,s] = k_t . k_s e^{L_t - L_s}  (s < t);   P[t,s] = scale q_t . k_s e^{L_t - L_s}  (s <= t)
//   X = (I + A diag(beta))^-1;   r = X (v - G (K S0)), what each value lacks;   u = beta r
//   o = scale G (Q S0) + P u;    S1 = G_C S0 + K^T (e^{L_C - L} u)
// X, P diag(beta) and the gates need no state: k_delta_local computes them for all chunks at once. k_delta_scan
// then walks over each head's chunks.
//
// The scan (32 chunks of 8 float32 heads of 64 x 64 in segments: 40 us and the join 16, in one run 92) keeps
// everything transposed, [Dv] x [tokens or Dk]: a warp owns 16 of the state's columns
// as the accumulators of m16n8k16 products, and the accumulators of one product are, in place, the A
// operand of the next (S^T -> (K S)^T -> u^T -> S^T). Columns never mix, so warps share only the
// loads of K, Q, X and P, and no value crosses a warp in the whole recurrence.
//
// Accuracy: K and Q are bfloat16, for the scan here three bfloat16 planes of a float32 input (bfloat16 inputs
// take the tcgen05 scan, delta_scan_tc.cu); S, the corrections w and u, X and P are float32 and enter products as
// three bfloat16 terms, the products of terms below 2^-24 of the result left out. The chunk's update of the state is summed by itself and added to the
// decayed state in float32, outside the tensor cores' accumulation.
#include "delta_internal.cuh"

namespace sdm {
namespace {

constexpr int kLocalHeads = 4;          // value heads of one key head a block takes at most

template <int KP, int DKP, int C, bool TC>
struct LocalSmem {
    static constexpr int KPITCH = delta_pitch(DKP * 2), TILE = C * KPITCH, NP = C + 4, XP = delta_pitch(C * 2);
    // K and Q make room for the inverse and for N, and N for the inverse's planes (TC), as each has been used
    static constexpr int Q = KP * TILE, X = 0, N = C * NP * 4, XPL = N, FIRST = 2 * KP * TILE;
    static constexpr int SECOND = N + (TC && 3 * XP > NP * 4 ? 3 * C * XP : C * NP * 4);
    static constexpr int G = FIRST > SECOND ? FIRST : SECOND;
    static constexpr int BYTES = G + kLocalHeads * 3 * C * 4;
};

// acc[i][e] += sum over m of A[row0 + i][m0 + m] B[m0 + m][col + e], m < M (a multiple of 4); both in
// shared memory with rows of NP floats
template <int ROWS, int NP>
__device__ __forceinline__ void tile_product(float (&acc)[ROWS][2], const float *A, const float *B, int M) {
    for (int m = 0; m < M; m += 4) {
        float2 x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = *reinterpret_cast<const float2 *>(B + (m + e) * NP);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const float4 a = *reinterpret_cast<const float4 *>(A + i * NP + m);
            acc[i][0] = fmaf(a.x, x[0].x, fmaf(a.y, x[1].x, fmaf(a.z, x[2].x, fmaf(a.w, x[3].x, acc[i][0]))));
            acc[i][1] = fmaf(a.x, x[0].y, fmaf(a.y, x[1].y, fmaf(a.z, x[2].y, fmaf(a.w, x[3].y, acc[i][1]))));
        }
    }
}

// X[lo.., c0..] = -X[lo.., lo..] N[lo.., c0..] X[c0.., c0..] for blocks of HALF rows and columns whose
// diagonal blocks are inverted: a warp takes 8 of the columns, which are its own in both products, so
// it needs no other warp. `part`: which 8.
template <int HALF, int NP>
__device__ __forceinline__ void merge_columns(const float *N, float *X, int c0, int part, int lane) {
    constexpr int ROWS = HALF / 8;                     // a lane: ROWS rows x 2 columns
    const int lo = c0 + HALF, col = c0 + 8 * part + 2 * (lane & 3), row = lo + ROWS * (lane >> 2);
    const int first = 8 * part / 16 * 16;              // the right factor is 0 above its diagonal blocks
    float acc[ROWS][2] = {};
    tile_product<ROWS, NP>(acc, N + row * NP + c0 + first, X + (c0 + first) * NP + col, HALF - first);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) *reinterpret_cast<float2 *>(X + (row + i) * NP + col) = make_float2(acc[i][0], acc[i][1]);
    __syncwarp();
    float out[ROWS][2] = {};
    const int upto = (row - lo) / 16 * 16 + 16;        // and the left one
    tile_product<ROWS, NP>(out, X + row * NP + lo, X + lo * NP + col, upto);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < ROWS; ++i) *reinterpret_cast<float2 *>(X + (row + i) * NP + col) = make_float2(-out[i][0], -out[i][1]);
}

// One block per chunk and up to kLocalHeads value heads that share a key head, one warp per 16 tokens.
// The products K K^T and Q K^T (blocks on and below the diagonal) are taken once for all of them and
// stay in registers. For each head: the decays, then the inverse of I + N, N = A diag(beta) (BACK:
// diag(beta) A): 16 x 16 diagonal blocks by substitution, a warp each, a lane a column, then merged
// in pairs, -X_2 N X_1, with the columns spread over the warps.
// TC: for the tcgen05 scans, Z = P X in the place of P.
// What bounds it: the latency of its steps, each behind a barrier, at 15 warps an SM (128 registers, 48 KB a
// block): issue 47 %. At C = 64 the merges are about 40 % of its instructions, the planes a quarter. Measured at Dk =
// 128 with two value heads a key head: 12300 chunks of heads 268 us, 8192 187 us. (Three blocks an SM, without the 64
// bytes spilled: 16384 tokens 643 us a call, 632 with four. With Z from two terms, 242 us then: the merges' operands
// fetched a step ahead 252; decays as products of factors by blocks of 16 and running sums as pairs of floats, for
// fewer exponentials and no doubles, 239, within what two runs differ.)
template <int KP, int DKP, int C, bool TC, bool BACK>
__global__ void __launch_bounds__(2 * C, C != 64 ? 1 : 4)
    k_delta_local(DeltaDims d, DeltaIn in, DeltaPlanes q, DeltaPlanes k, DeltaLocal w, int heads) {
    using L = LocalSmem<KP, DKP, C, TC>;
    constexpr int THREADS = 2 * C, NB = C / 16, NP = L::NP, XP = delta_pitch(C * 2), KPI = L::KPITCH, PP = 3;
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (blockIdx.x == 0 && tid == 0) *w.status = DevStatus{};
    auto plane_at = [](int r, int c) { return TC ? tc_at(r, c) : delta_at<XP>(r, c); };
    constexpr int PLANE = C * (TC ? 128 : XP);
    const int n = (int)(blockIdx.x % d.Nt);
    const long long bg = blockIdx.x / d.Nt;                        // sequence and group of heads
    const int groups = d.H / heads, b = (int)(bg / groups), h0 = (int)(bg % groups) * heads, hk = h0 / (d.H / d.Hk);
    const int t0 = n * C;
    int nt = delta_valid(in.valid, b, d.T) - t0;
    if (nt <= 0) return;
    nt = nt < C ? nt : C;
    const unsigned sk = smem_u32(smem), sq = sk + L::Q;
    float *N = reinterpret_cast<float *>(smem + L::N), *X = reinterpret_cast<float *>(smem + L::X);
    float *gates = reinterpret_cast<float *>(smem + L::G);         // [head][hi, lo, beta][C]

    load_tokens<KP, DKP, C, THREADS>(sk, k, b * k.s[0] + t0 * k.s[1] + hk * k.s[2], d.Dk, nt, tid);
    load_tokens<KP, DKP, C, THREADS>(sq, q, b * q.s[0] + t0 * q.s[1] + hk * q.s[2], d.Dk, nt, tid);
    cp_async_commit();
    for (int hh = warp; hh < heads; hh += NB) {
        // running sums in double: differences of large sums (resets inside the chunk) stay exact
        constexpr int PL = C / 32;
        const int h = h0 + hh;
        float *hi = gates + hh * 3 * C, *lo = hi + C, *be = lo + C;
        double run[PL];
        float bt[PL];
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const int r = lane * PL + i;
            const long long t = t0 + r;
            const bool live = r < nt;
            s += live ? (double)delta_decay(in.g[b * d.gs[0] + t * d.gs[1] + h * d.gs[2]]) : 0.0;
            bt[i] = live ? in.beta[b * d.bs[0] + t * d.bs[1] + h * d.bs[2]] : 0.f;
            run[i] = s;
        }
        double before = s;
#pragma unroll
        for (int m = 1; m < 32; m *= 2) {
            const double x = __shfl_up_sync(~0u, before, m);
            if (lane >= m) before += x;
        }
        const double all = __shfl_sync(~0u, before, 31);
        before -= s;
        float *aux = w.aux + (((long long)b * d.H + h) * d.Nt + n) * kDeltaAux * C;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const int r = lane * PL + i;
            const double x = before + run[i];
            hi[r] = (float)x;
            lo[r] = (float)(x - (double)(float)x);
            be[r] = bt[i];
            aux[r] = expf((float)x);
            aux[C + r] = expf((float)(all - x)) * (BACK ? 1.f : bt[i]);
            aux[2 * C + r] = bt[i];
            aux[3 * C + r] = hi[r];
            aux[4 * C + r] = lo[r];
        }
    }
    cp_async_wait<0>();
    __syncthreads();

    float kk[C / 8][4] = {}, qk[C / 8][4] = {};
#pragma unroll
    for (int pk = KP > 1 ? 2 * DKP / 16 - 1 : DKP / 16 - 1; pk >= 0; --pk) {   // passes of K steps
        const int pass = pk / (DKP / 16), ks = pk % (DKP / 16);
        unsigned ak[KP][4], aq[KP][4];
#pragma unroll
        for (int p = 0; p < KP; ++p) {
            if (pass == 0 && p > 0) break;
            ldsm4(ak[p], frag_rc<KPI>(sk + p * L::TILE, 16 * warp, 16 * ks, lane));
            ldsm4(aq[p], frag_rc<KPI>(sq + p * L::TILE, 16 * warp, 16 * ks, lane));
        }
#pragma unroll
        for (int jj = 0; jj < NB; ++jj) {
            if (jj > warp) break;
            unsigned bk[KP][4];
#pragma unroll
            for (int p = 0; p < KP; ++p)
                if (pass > 0 || p == 0) ldsm4(bk[p], frag_cr<KPI>(sk + p * L::TILE, 16 * jj, 16 * ks, lane));
#pragma unroll
            for (int x = KP - 1; x >= 0; --x)
#pragma unroll
                for (int y = KP - 1; y >= 0; --y)
                    if (plane_pair(x, y, KP, pass))
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            mma_bf16(kk[2 * jj + e], ak[x], bk[y][2 * e], bk[y][2 * e + 1]);
                            mma_bf16(qk[2 * jj + e], aq[x], bk[y][2 * e], bk[y][2 * e + 1]);
                        }
        }
    }
    __syncthreads();                                               // K and Q are used
    for (int hh = 0; hh < heads; ++hh) {
        const long long bhn = ((long long)b * d.H + h0 + hh) * d.Nt + n;
        const float *hi = gates + hh * 3 * C, *lo = hi + C, *be = lo + C;
        unsigned char *pimg = w.p + bhn * (size_t)(PP * PLANE);
        // P of a forward carries the corrections' beta: u = beta r
        auto p_pair = [&](int j, int half, float (&pp)[2], float (&nn)[2]) {
            const int t = 16 * warp + (lane >> 2) + 8 * half;
            const float ht = hi[t], lt = lo[t], bt = be[t];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int s = 8 * j + 2 * (lane & 3) + e;
                const float f = s <= t ? expf((ht - hi[s]) + (lt - lo[s])) : 0.f, bs = be[s];
                nn[e] = s < t ? kk[j][2 * half + e] * f * (BACK ? bt : bs) : 0.f;
                pp[e] = s <= t ? d.scale * qk[j][2 * half + e] * f * (BACK ? 1.f : bs) : 0.f;
            }
        };
        float pv[TC ? C / 8 : 1][4];
#pragma unroll
        for (int j = 0; j < C / 8; ++j) {
            if (j > 2 * warp + 1) break;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int t = 16 * warp + (lane >> 2) + 8 * half;
                float nn[2], pp[2];
                p_pair(j, half, pp, nn);
                *reinterpret_cast<float2 *>(N + t * NP + 8 * j + 2 * (lane & 3)) = make_float2(nn[0], nn[1]);
                if constexpr (TC) {
                    pv[j][2 * half] = pp[0];
                    pv[j][2 * half + 1] = pp[1];
                } else {
                    unsigned pl[PP];
                    split_bf16<PP>(pp[0], pp[1], pl);
#pragma unroll
                    for (int p = 0; p < PP; ++p)
                        *reinterpret_cast<unsigned *>(pimg + p * PLANE + plane_at(t, j) + 4 * (lane & 3)) = pl[p];
                }
            }
        }
        __syncwarp();
        if (lane < 16) {
            float x[16];
            const float *D = N + (16 * warp) * NP + 16 * warp;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s0 = i == lane ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
                for (int l = 0; l < i; l += 4) {
                    const float4 a = *reinterpret_cast<const float4 *>(D + i * NP + l);
                    s0 = fmaf(-a.x, x[l], s0);
                    if (l + 1 < i) s1 = fmaf(-a.y, x[l + 1], s1);
                    if (l + 2 < i) s0 = fmaf(-a.z, x[l + 2], s0);
                    if (l + 3 < i) s1 = fmaf(-a.w, x[l + 3], s1);
                }
                x[i] = s0 + s1;
                X[(16 * warp + i) * NP + 16 * warp + lane] = x[i];
            }
        }
        __syncthreads();
        // 16 -> 32: each pair's 16 columns over two warps; 32 -> 64: the 32 columns over four
        merge_columns<16, NP>(N, X, 32 * (warp >> 1), warp & 1, lane);
        __syncthreads();
        if constexpr (C == 64) {
            merge_columns<32, NP>(N, X, 0, warp, lane);
            __syncthreads();
        }
        unsigned char *ximg = w.x + bhn * (size_t)(3 * PLANE);
        for (int i = tid; i < C * (C / 8); i += THREADS) {
            const int r = i / (C / 8), c = i % (C / 8);
            if (c > 2 * (r >> 4) + 1) continue;
            unsigned pl[4][3];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x = *reinterpret_cast<const float2 *>(X + r * NP + 8 * c + 2 * e);
                split_bf16<3>(x.x, x.y, pl[e]);
            }
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                const uint4 y = make_uint4(pl[0][p], pl[1][p], pl[2][p], pl[3][p]);
                *reinterpret_cast<uint4 *>(ximg + p * PLANE + plane_at(r, c)) = y;
                if constexpr (TC) *reinterpret_cast<uint4 *>(smem + L::XPL + p * C * XP + delta_at<XP>(r, c)) = y;
            }
        }
        if constexpr (TC) {
            __syncthreads();
            float z[C / 8][4] = {};
            const unsigned sx = smem_u32(smem) + L::XPL;
#pragma unroll
            for (int ks = 0; ks < NB; ++ks) {                      // the accumulators of P are its A operand
                if (ks > warp) break;
                unsigned a[PP][4];
                split_frag<PP>(pv, ks, a);
#pragma unroll
                for (int jj = 0; jj <= ks; ++jj) {
                    unsigned bb[PP][4];
#pragma unroll
                    for (int p = 0; p < PP; ++p) ldsm4t(bb[p], frag_rc<XP>(sx + p * C * XP, 16 * ks, 16 * jj, lane));
#pragma unroll
                    for (int x = PP - 1; x >= 0; --x)
#pragma unroll
                        for (int y = PP - 1; y >= 0; --y)
                            if (plane_pair(x, y, PP))
#pragma unroll
                                for (int e = 0; e < 2; ++e) mma_bf16(z[2 * jj + e], a[x], bb[y][2 * e], bb[y][2 * e + 1]);
                }
            }
#pragma unroll
            for (int j = 0; j < C / 8; ++j) {
                if (j > 2 * warp + 1) break;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    unsigned pl[PP];
                    split_bf16<PP>(z[j][2 * half], z[j][2 * half + 1], pl);
#pragma unroll
                    for (int p = 0; p < PP; ++p)
                        *reinterpret_cast<unsigned *>(pimg + p * PLANE + plane_at(16 * warp + (lane >> 2) + 8 * half, j) + 4 * (lane & 3)) = pl[p];
                }
            }
        }
        if (hh + 1 < heads) __syncthreads();                       // X and N for the next head
    }
}

template <int DKP, int NW>
struct ScanSmem {
    static constexpr int C = 32, KP = 3, PP = 3;
    static constexpr int XP = delta_pitch(C * 2);            // row pitch of the X and P planes
    static constexpr int VP = delta_pitch(NW * 16 * 4);   // of the value tile
    static constexpr int KPI = delta_pitch(DKP * 2), TILE = C * KPI;
    static constexpr int Q = KP * TILE, X = 2 * KP * TILE, P = X + 3 * C * XP, V = P + PP * C * XP;
    static constexpr int AUX = V + C * VP, STAGE = AUX + 3 * C * 4;
    static constexpr int BAD = 2 * STAGE, BYTES = BAD + NW * 16 * 4;   // per column: the first chunk delta_column takes
};

// One block per head and NW * 16 of its columns; two stages of chunk inputs, the next chunk's copies
// in flight while this one is computed. SAVE: also stores S0 and r for the backward.
template <int DKP, int NW, bool SAVE>
__global__ void __launch_bounds__(NW * 32, 1)
    k_delta_scan(DeltaDims d, DeltaIn in, DeltaPlanes q, DeltaPlanes k, DeltaLocal w, float *state,
                 float *o, float *snap, float *rsave, int mode) {
    using L = ScanSmem<DKP, NW>;
    constexpr int C = L::C, KP = L::KP, PP = L::PP, XP = L::XP, VP = L::VP, KPI = L::KPI, THREADS = NW * 32;
    constexpr int NT = C / 8, ND = DKP / 8, VE = 16 / 4;
    // X's diagonal blocks, its largest, and the latest tokens' updates come last in either pass over the terms
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g4 = lane >> 2, i4 = lane & 3;
    const bool carry = !SAVE && mode == DELTA_CARRY;
    const DeltaBlock blk = delta_block(d, in.valid, d.segs > 1, mode, NW * 16);
    const int dv_blk = blk.tile * NW * 16, width = blk.unit ? d.Dk : d.Dv;
    const long long bh = blk.bh;
    const int b = (int)(bh / d.H), h = (int)(bh % d.H), hk = h / (d.H / d.Hk);
    const int dv0 = dv_blk + 16 * warp;
    const bool mine = dv0 < width;                           // else the warp only helps to load
    const int ntok = delta_valid(in.valid, b, d.T), chunks = (ntok + C - 1) / C;
    const int n0 = delta_bound(d, chunks, blk.seg), nch = delta_bound(d, chunks, blk.seg + 1);   // its chunks' ends
    const bool last = blk.seg + 1 == d.segs;
    const float *v = static_cast<const float *>(in.v) + b * d.vs[0] + h * d.vs[2] + dv_blk;
    const long long kbase = b * k.s[0] + hk * k.s[2], qbase = b * q.s[0] + hk * q.s[2];
    float *out = o + ((long long)b * d.T * d.H + h) * d.Dv;
    const long long orow = (long long)d.H * d.Dv;
    const unsigned s0 = smem_u32(smem);
    int *bad = reinterpret_cast<int *>(smem + L::BAD) + 16 * warp;
    if (lane < 16) bad[lane] = -1;
    __syncwarp();

    auto load = [&](int n, int stage) {
        const unsigned st = s0 + stage * L::STAGE;
        const long long t0 = (long long)n * C, bhn = bh * d.Nt + n;
        const int nt = ntok - (int)t0 < C ? ntok - (int)t0 : C;
        load_tokens<KP, DKP, C, THREADS>(st, k, kbase + t0 * k.s[1], d.Dk, nt, tid);
        load_planes<3, C, THREADS>(st + L::X, w.x + bhn * (3 * C * XP), tid);
        if (!carry) {
            load_tokens<KP, DKP, C, THREADS>(st + L::Q, q, qbase + t0 * q.s[1], d.Dk, nt, tid);
            load_planes<PP, C, THREADS>(st + L::P, w.p + bhn * (PP * C * XP), tid);
        }
        load_values<float, NW * 16, C, THREADS>(st + L::V, v + t0 * d.vs[1], d.vs[1], nt, blk.unit ? 0 : d.Dv - dv_blk, tid);
        for (int i = tid; i < 3 * C / 4; i += THREADS)
            cp_async16_zfill(st + L::AUX + 16 * i, w.aux + bhn * kDeltaAux * C + 4 * i, true);
        cp_async_commit();
    };

    float S[ND][4];
    const bool real = !carry || blk.seg == 0;
    float *sp = (d.segs > 1 && !carry ? w.starts + blk.seg * delta_states(d) : state) + (bh * d.Dk) * d.Dv + dv0;
#pragma unroll
    for (int j = 0; j < ND; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int dk = 8 * j + 2 * i4 + (e & 1);
            const bool one = blk.unit && dk == dv0 + g4 + 8 * (e >> 1);
            S[j][e] = real && mine && dk < d.Dk ? sp[(size_t)dk * d.Dv + g4 + 8 * (e >> 1)] : one ? 1.f : 0.f;
        }
    auto store_state = [&](float *dst) {
#pragma unroll
        for (int j = 0; j < ND; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int dk = 8 * j + 2 * i4 + (e & 1);
                if (dk < d.Dk) dst[(size_t)dk * width + g4 + 8 * (e >> 1)] = S[j][e];
            }
    };
    if (n0 < nch) load(n0, 0);
    for (int n = n0; n < nch; ++n) {
        if (n + 1 < nch) {
            load(n + 1, (n + 1 - n0) & 1);
            cp_async_wait<1>();
        } else {
            cp_async_wait<0>();
        }
        __syncthreads();
        const int stage = ((n - n0) & 1) * L::STAGE;
        const unsigned sk = s0 + stage, sq = sk + L::Q, sx = sk + L::X, spp = sk + L::P, sv = sk + L::V;
        const float *from = reinterpret_cast<const float *>(smem + stage + L::AUX), *to = from + C;
        const int nt = ntok - n * C < C ? ntok - n * C : C;
        if (mine) {
            if constexpr (SAVE) store_state(snap + ((bh * (d.Nt + 1) + n) * (long long)d.Dk) * d.Dv + dv0);
            float R[NT][4] = {}, O[NT][4] = {};
#pragma unroll
            for (int pk = 0; pk < 2 * DKP / 16; ++pk) { // R = (K S)^T, O = (Q S)^T
                const int pass = 1 - pk / (DKP / 16), ks = pk % (DKP / 16);
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
                                mma_bf16(R[j], a[x], bb[p][j >> 1][2 * (j & 1)], bb[p][j >> 1][2 * (j & 1) + 1]);
                if (carry) continue;
#pragma unroll
                for (int p = 0; p < KP; ++p)
#pragma unroll
                    for (int jj = 0; jj < C / 16; ++jj)
                        if (pass > 0 || p == 0) ldsm4(bb[p][jj], frag_cr<KPI>(sq + p * L::TILE, 16 * jj, 16 * ks, lane));
#pragma unroll
                for (int x = PP - 1; x >= 0; --x)
#pragma unroll
                    for (int p = KP - 1; p >= 0; --p)
                        if (plane_pair(x, p, PP, pass))
#pragma unroll
                            for (int j = 0; j < NT; ++j)
                                mma_bf16(O[j], a[x], bb[p][j >> 1][2 * (j & 1)], bb[p][j >> 1][2 * (j & 1) + 1]);
            }
            // R <- v - G R, O <- scale G O
#pragma unroll
            for (int jj = 0; jj < C / 16; ++jj) {
                float vv[2][4];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int t = 16 * jj + 8 * (e >> 2) + 2 * i4 + (e & 1);
                    const int c = 16 * warp + g4 + 8 * ((e >> 1) & 1);
                    vv[e >> 2][e & 3] = *reinterpret_cast<const float *>(
                        smem + stage + L::V + delta_at<VP>(t, c >> 2) + 4 * (c & 3));
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int j = 2 * jj + (e >> 2), t = 8 * j + 2 * i4 + (e & 1);
                    const float f = from[t];
                    // spelled out: a contraction the compiler takes in one form and not in the other would give a
                    // saving forward other bits
                    R[j][e & 3] = fmaf(-f, R[j][e & 3], vv[e >> 2][e & 3]);
                    O[j][e & 3] = __fmul_rn(O[j][e & 3], __fmul_rn(d.scale, f));
                }
            }
            float U[NT][4] = {};
#pragma unroll
            for (int pk = 0; pk < 2 * C / 16; ++pk) {   // U = r^T = (X (v - G K S))^T
                const int pass = 1 - pk / (C / 16), ks = pk % (C / 16);
                unsigned a[3][4];
                split_frag<3>(R, ks, a);
#pragma unroll
                for (int jj = ks; jj < C / 16; ++jj) {
                    unsigned bb[3][4];
#pragma unroll
                    for (int p = 0; p < 3; ++p)
                        if (pass > 0 || p == 0) ldsm4(bb[p], frag_cr<XP>(sx + p * C * XP, 16 * jj, 16 * ks, lane));
#pragma unroll
                    for (int x = 2; x >= 0; --x)
#pragma unroll
                        for (int p = 2; p >= 0; --p)
                            if (plane_pair(x, p, 3, pass)) {
                                mma_bf16(U[2 * jj], a[x], bb[p][0], bb[p][1]);
                                mma_bf16(U[2 * jj + 1], a[x], bb[p][2], bb[p][3]);
                            }
                }
            }
            if constexpr (SAVE) {
                float *dst = rsave + ((bh * d.Nt + n) * (long long)C) * d.Dv + dv0;
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        dst[(size_t)(8 * j + 2 * i4 + (e & 1)) * d.Dv + g4 + 8 * (e >> 1)] = U[j][e];
            }
            // O += (P diag(beta) r)^T, in sums of its own (R's place)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) R[j][e] = 0.f;
#pragma unroll
            for (int pk = 0; pk < 2 * C / 16; ++pk) {
                if (carry) break;
                const int pass = 1 - pk / (C / 16), ks = pk % (C / 16);
                unsigned a[PP][4];
                split_frag<PP>(U, ks, a);
#pragma unroll
                for (int jj = ks; jj < C / 16; ++jj) {
                    unsigned bb[PP][4];
#pragma unroll
                    for (int p = 0; p < PP; ++p)
                        if (pass > 0 || p == 0) ldsm4(bb[p], frag_cr<XP>(spp + p * C * XP, 16 * jj, 16 * ks, lane));
#pragma unroll
                    for (int x = PP - 1; x >= 0; --x)
#pragma unroll
                        for (int p = PP - 1; p >= 0; --p)
                            if (plane_pair(x, p, PP, pass)) {
                                mma_bf16(R[2 * jj], a[x], bb[p][0], bb[p][1]);
                                mma_bf16(R[2 * jj + 1], a[x], bb[p][2], bb[p][3]);
                            }
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) O[j][e] += R[j][e];
            // the readings take the place of the warp's columns of the value tile, then leave as rows
            if (!carry) {
                __syncwarp();
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = 8 * j + 2 * i4 + (e & 1), c = 16 * warp + g4 + 8 * (e >> 1);
                        *reinterpret_cast<float *>(smem + stage + L::V + delta_at<VP>(t, c / VE) +
                                               (c % VE) * 4) = O[j][e];
                    }
                __syncwarp();
                constexpr int PR = 16 / VE, RP = 32 / PR;    // pieces a row, rows at once
#pragma unroll
                for (int r0 = 0; r0 < C; r0 += RP) {
                    const int r = r0 + lane / PR, c = lane % PR;
                    const long long t = (long long)n * C + r;
                    uint4 x = *reinterpret_cast<const uint4 *>(smem + stage + L::V + delta_at<VP>(r, 16 * warp / VE + c));
                    if (r >= nt) x = make_uint4(0u, 0u, 0u, 0u);
                    if (t < d.T) *reinterpret_cast<uint4 *>(out + t * orow + dv0 + c * VE) = x;
                }
            }
            // S <- G_C S + (e^{L_C - L} beta r)^T K
            unsigned ua[C / 16][3][4];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) U[j][e] *= to[8 * j + 2 * i4 + (e & 1)];
#pragma unroll
            for (int ks = 0; ks < C / 16; ++ks) split_frag<3>(U, ks, ua[ks]);
            const float whole = from[C - 1];
#pragma unroll
            for (int nn = 0; nn < ND / 2; nn += 2) {
                float acc[4][4] = {};
#pragma unroll
                for (int pk = 0; pk < 2 * C / 16; ++pk) {
                    const int pass = 1 - pk / (C / 16), ks = pk % (C / 16);
                    unsigned bb[KP][2][4];
#pragma unroll
                    for (int p = 0; p < KP; ++p)
#pragma unroll
                        for (int m = 0; m < 2; ++m)
                            if (pass > 0 || p == 0) ldsm4t(bb[p][m], frag_rc<KPI>(sk + p * L::TILE, 16 * ks, 16 * (nn + m), lane));
#pragma unroll
                    for (int x = 2; x >= 0; --x)
#pragma unroll
                        for (int p = KP - 1; p >= 0; --p)
                            if (plane_pair(x, p, 3, pass))
#pragma unroll
                                for (int m = 0; m < 4; ++m)
                                    mma_bf16(acc[m], ua[ks][x], bb[p][m >> 1][2 * (m & 1)], bb[p][m >> 1][2 * (m & 1) + 1]);
                }
                // a column's first update that is finite in no row (as a NaN or infinity of a token leaves it): its
                // state before goes back to where it came from, for delta_column
                if (nn == 0 && !carry) {
                    const unsigned off[2] = {__ballot_sync(~0u, !delta_finite(acc[0][0])), __ballot_sync(~0u, !delta_finite(acc[0][2]))};
                    if (off[0] | off[1]) {
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            const bool now = (off[f] >> (4 * g4) & 15) == 15 && bad[g4 + 8 * f] < 0;
                            __syncwarp();
                            if (now && i4 == 0) bad[g4 + 8 * f] = n;
                            if (now)
#pragma unroll
                                for (int j = 0; j < ND; ++j)
#pragma unroll
                                    for (int e = 0; e < 2; ++e)
                                        if (8 * j + 2 * i4 + e < d.Dk) sp[(size_t)(8 * j + 2 * i4 + e) * d.Dv + g4 + 8 * f] = S[j][2 * f + e];
                        }
                    }
                }
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[2 * nn + m][e] = fmaf(whole, S[2 * nn + m][e], acc[m][e]);
            }
        }
        __syncthreads();
    }
    if (!mine) return;
    if (!carry) {
        __syncwarp();
        for (int c = 0; c < 16; ++c) {
            const int n = bad[c], t0 = n * C;
            if (n < 0) continue;
            delta_column<float>(d, in, b, h, dv0 + c, t0, ntok - t0 < C ? ntok - t0 : C, sp + c, out + t0 * orow + dv0 + c,
                                SAVE ? rsave + (bh * d.Nt + n) * (long long)C * d.Dv + dv0 + c : nullptr);
        }
        __syncwarp();                                              // before the last state is stored over it
    }
    if (carry) {
        store_state((blk.unit ? w.units + ((blk.seg - 1) * (long long)d.B * d.H + bh) * d.Dk * d.Dk
                              : w.starts + (blk.seg + 1) * delta_states(d) + bh * d.Dk * (long long)d.Dv) + dv0);
        return;
    }
    if (!last) return;
    if (nch > 0) store_state(state + (bh * d.Dk) * d.Dv + dv0);
    if (SAVE) store_state(snap + ((bh * (d.Nt + 1) + chunks) * (long long)d.Dk) * d.Dv + dv0);
    constexpr int PR = 16 / VE;
    for (long long t = (long long)chunks * C + lane / PR; t < d.T; t += 32 / PR)
        *reinterpret_cast<uint4 *>(out + t * orow + dv0 + (lane % PR) * VE) = make_uint4(0u, 0u, 0u, 0u);
}

constexpr int kJoinPitch = kDeltaMaxDk + 4;                        // floats: eight rows in a row lie in different banks
constexpr int kJoinUnit = kDeltaMaxDk * kJoinPitch, kJoinBytes = (kJoinUnit + kDeltaMaxDk * 16) * 4;

// starts[i + 1] += units[i] starts[i], segment after segment (DeltaBlock): one block per head and 16 columns,
// a thread 8 of them of a row; what the next step reads is in flight before this one's results are put down.
// Bound by the chain over the segments, about 3 us a step of 128 x 128 states (the unit's 64 KB from the level 2
// cache, then its product). starts[0] is the caller's state. BACK: starts[i - 1] += units[i]^T starts[i], from
// the last down. A tile of zeros is not multiplied, so a state of zeros stays one whatever the unit's columns
// hold.
template <bool BACK>
__global__ void __launch_bounds__(2 * kDeltaMaxDk) k_delta_join(DeltaDims d, DeltaLocal w, const float *state) {
    extern __shared__ __align__(16) float M[];
    float *S = M + kJoinUnit;                                      // [rows][16]
    const int tid = threadIdx.x, row = tid & (kDeltaMaxDk - 1), c0 = tid / kDeltaMaxDk * 8, slices = d.Dv / 16;
    const long long bh = blockIdx.x / slices, base = (bh * d.Dk + row) * d.Dv + blockIdx.x % slices * 16 + c0;
    const bool live = row < d.Dk;
    auto slot = [&](int s) { return BACK ? d.segs - 1 - s : s; };  // the s-th in the chain
    auto fetch = [&](int s) {                                      // what leads to it from the one before
        if (s >= 2 && s < d.segs) {
            const float *m = w.units + ((BACK ? d.segs - 1 - s : s - 2) * (long long)d.B * d.H + bh) * d.Dk * d.Dk;
            const int pieces = d.Dk / 4;
            for (int i = tid; i < d.Dk * pieces; i += 2 * kDeltaMaxDk)
                cp_async16_zfill(smem_u32(M) + (i / pieces * kJoinPitch + i % pieces * 4) * 4, m + 4 * i, true);
        }
        cp_async_commit();
    };
    __align__(16) float x[8] = {}, next[8] = {};
    auto first = [&](int s) {
        if (live && s < d.segs && (s > 0 || state)) {
            const float *from = (s == 0 ? state : w.starts + slot(s) * delta_states(d)) + base;
            if (BACK && s == 0) {                                  // the caller's gradient: any alignment
#pragma unroll
                for (int i = 0; i < 8; ++i) next[i] = from[i];
                return;
            }
#pragma unroll
            for (int i = 0; i < 8; i += 4) *reinterpret_cast<float4 *>(next + i) = *reinterpret_cast<const float4 *>(from + i);
        }
    };
    fetch(2);
    first(0);
    for (int s = 0; s < d.segs; ++s) {
        bool some = false;                                         // of the state before
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            some |= x[i] != 0.f;
            x[i] = next[i];
        }
        first(s + 1);
        cp_async_wait<0>();
        if (__syncthreads_or(some) && s >= 2) {
            const float *m = BACK ? M + row : M + row * kJoinPitch;
#pragma unroll 2
            for (int k = 0; k < d.Dk; k += 4) {
                __align__(16) float av[4];
                if constexpr (BACK) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) av[e] = m[(k + e) * kJoinPitch];
                } else {
                    *reinterpret_cast<float4 *>(av) = *reinterpret_cast<const float4 *>(m + k);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    __align__(16) float y[8];
#pragma unroll
                    for (int i = 0; i < 8; i += 4) *reinterpret_cast<float4 *>(y + i) = *reinterpret_cast<const float4 *>(S + (k + e) * 16 + c0 + i);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = fmaf(av[e], y[i], x[i]);
                }
            }
        }
        __syncthreads();                                           // M and S are used
        if (s >= 2) fetch(s + 1);
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 y = *reinterpret_cast<const float4 *>(x + i);
            *reinterpret_cast<float4 *>(S + row * 16 + c0 + i) = y;
            if (live && s != 1) *reinterpret_cast<float4 *>(w.starts + slot(s) * delta_states(d) + base + i) = y;
        }
    }
}

// float32 queries and keys (blockIdx.y), rows [b, t, h] of Dk columns -> three contiguous bfloat16 planes [B, T,
// Hk, Dk] each
__global__ void __launch_bounds__(256) k_delta_split(DeltaDims d, const float *q, const float *k,
                                                     __nv_bfloat16 *q_planes, __nv_bfloat16 *k_planes) {
    const float *x = blockIdx.y ? k : q;
    const long long sb = blockIdx.y ? d.ks[0] : d.qs[0], st = blockIdx.y ? d.ks[1] : d.qs[1], sh = blockIdx.y ? d.ks[2] : d.qs[2];
    __nv_bfloat16 *planes = blockIdx.y ? k_planes : q_planes;
    const int heads = d.Hk, D = d.Dk;
    const long long all = (long long)d.B * d.T * heads * (D / 4), plane = all * 4;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
        const long long row = i / (D / 4), h = row % heads, bt = row / heads, t = bt % d.T, b = bt / d.T;
        const int c = (int)(i % (D / 4)) * 4;
        unsigned p0[3] = {0u, 0u, 0u}, p1[3] = {0u, 0u, 0u};
        const float4 a = *reinterpret_cast<const float4 *>(x + b * sb + t * st + h * sh + c);
        split_bf16<3>(a.x, a.y, p0);
        split_bf16<3>(a.z, a.w, p1);
#pragma unroll
        for (int p = 0; p < 3; ++p)
            *reinterpret_cast<uint2 *>(planes + p * plane + 4 * i) = make_uint2(p0[p], p1[p]);
    }
}

__global__ void __launch_bounds__(256) k_delta_unroll(DeltaDims d, const __nv_bfloat16 *x, long long sb, long long st, long long sh, int heads,
                                                      int width, __nv_bfloat16 *to) {
    const long long all = (long long)d.B * d.T * heads * (width / 8);
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
        const long long row = i / (width / 8), h = row % heads, bt = row / heads, t = bt % d.T, b = bt / d.T;
        reinterpret_cast<uint4 *>(to)[i] = *reinterpret_cast<const uint4 *>(x + b * sb + t * st + h * sh + i % (width / 8) * 8);
    }
}

template <int DKP, int NW, bool SAVE>
cudaError_t scan_one(const DeltaDims &d, const DeltaIn &in, const DeltaPlanes &q, const DeltaPlanes &k,
                     const DeltaLocal &w, float *state, float *o, float *snap, float *r, int mode, cudaStream_t st) {
    using L = ScanSmem<DKP, NW>;
    auto kern = k_delta_scan<DKP, NW, SAVE>;
    set_kernel_smem(kern, L::BYTES);
    kern<<<(unsigned)delta_blocks(d, mode, NW * 16), NW * 32, L::BYTES, st>>>(d, in, q, k, w, state, o, snap, r, mode);
    return cudaGetLastError();
}

template <int KP, int DKP, int C, bool TC, bool BACK>
cudaError_t local_one(const DeltaDims &d, const DeltaIn &in, const DeltaPlanes &q, const DeltaPlanes &k,
                      const DeltaLocal &w, cudaStream_t st) {
    auto kern = k_delta_local<KP, DKP, C, TC, BACK>;
    constexpr int bytes = LocalSmem<KP, DKP, C, TC>::BYTES;
    set_kernel_smem(kern, bytes);
    // as many heads of a key head to a block as still leave four blocks for every SM (8 x 4096 tokens, 32 heads by
    // fours: whole call 639 us with one head a block, 594 with two, 571 with four)
    const int group = d.H / d.Hk;
    int heads = kLocalHeads;
    while (heads > 1 && (group % heads || delta_chunks(d) / heads < 4 * kRefSms)) --heads;
    kern<<<(unsigned)(delta_chunks(d) / heads), 2 * C, bytes, st>>>(d, in, q, k, w, heads);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_local(const DeltaDims &d, const DeltaIn &in, const DeltaPlanes &q, const DeltaPlanes &k,
                               const DeltaLocal &w, cudaStream_t st) {
    auto go = [&](auto kp, auto dkp, auto c, auto tc, auto back) {
        return local_one<decltype(kp)::value, decltype(dkp)::value, decltype(c)::value, decltype(tc)::value,
                         decltype(back)::value>(d, in, q, k, w, st);
    };
    using std::integral_constant;
    auto size = [&](auto dkp) {
        const std::true_type yes;
        const std::false_type no;
        if (d.dtype == SDM_F32)
            return d.back ? go(integral_constant<int, 3>{}, dkp, integral_constant<int, 32>{}, no, yes)
                          : go(integral_constant<int, 3>{}, dkp, integral_constant<int, 32>{}, no, no);
        return d.back ? go(integral_constant<int, 1>{}, dkp, integral_constant<int, 64>{}, yes, yes)
                      : go(integral_constant<int, 1>{}, dkp, integral_constant<int, 64>{}, yes, no);
    };
    return d.Dk <= 64 ? size(integral_constant<int, 64>{}) : size(integral_constant<int, 128>{});
}

cudaError_t launch_delta_join(const DeltaDims &d, const DeltaLocal &w, const float *state, bool back, cudaStream_t st) {
    auto kern = back ? k_delta_join<true> : k_delta_join<false>;
    set_kernel_smem(kern, kJoinBytes);
    kern<<<(unsigned)((long long)d.B * d.H * (d.Dv / 16)), 2 * kDeltaMaxDk, kJoinBytes, st>>>(d, w, state);
    return cudaGetLastError();
}

cudaError_t launch_delta_scan(const DeltaDims &d, const DeltaIn &in, const DeltaPlanes &q, const DeltaPlanes &k,
                              const DeltaLocal &w, float *state, void *o, float *snap, float *r, cudaStream_t st) {
    auto out = static_cast<float *>(o);
    // eight warps (two an SM sub-core) share a chunk's loads once there is a block for every SM (float32, 8 x 1000
    // tokens of 32 heads of 128 x 128: 688 us, 832 with four; of 128 x 256 1219 and 1358; 4 x 1000 of 64 heads of 64 x
    // 128 422 and 449); with fewer heads four, so that every warp has a
    // tensor core of its own
    const bool wide = d.Dv > 64 && (long long)d.B * d.H * ((d.Dv + 127) / 128) >= kRefSms;
    auto go = [&](auto dkp, auto nw, auto save, int mode) {
        return scan_one<decltype(dkp)::value, decltype(nw)::value, decltype(save)::value>(
            d, in, q, k, w, state, out, snap, r, mode, st);
    };
    auto pick = [&](auto dkp, auto nw) {
        if (d.segs > 1) {
            cudaError_t e = go(dkp, nw, std::false_type{}, DELTA_CARRY);
            if (e == cudaSuccess) e = launch_delta_join(d, w, state, false, st);
            if (e != cudaSuccess) return e;
        }
        return snap ? go(dkp, nw, std::true_type{}, DELTA_RUN) : go(dkp, nw, std::false_type{}, DELTA_RUN);
    };
    auto size = [&](auto dkp) {
        return wide ? pick(dkp, std::integral_constant<int, 8>{}) : pick(dkp, std::integral_constant<int, 4>{});
    };
    return d.Dk <= 64 ? size(std::integral_constant<int, 64>{}) : size(std::integral_constant<int, 128>{});
}

cudaError_t launch_delta_unroll(const DeltaDims &d, const void *x, const long long *s, int heads, int width, void *to, cudaStream_t st) {
    const long long units = (long long)d.B * d.T * heads * (width / 8), blocks = (units + 255) / 256;
    k_delta_unroll<<<(unsigned)(blocks < 8 * kRefSms ? blocks : 8 * kRefSms), 256, 0, st>>>(
        d, static_cast<const __nv_bfloat16 *>(x), s[0], s[1], s[2], heads, width, static_cast<__nv_bfloat16 *>(to));
    return cudaGetLastError();
}

cudaError_t launch_delta_split(const DeltaDims &d, const void *q, const void *k, __nv_bfloat16 *q_planes, __nv_bfloat16 *k_planes, cudaStream_t st) {
    const long long units = (long long)d.B * d.T * d.Hk * (d.Dk / 4), blocks = (units + 255) / 256;
    k_delta_split<<<dim3((unsigned)(blocks < 4 * kRefSms ? blocks : 4 * kRefSms), 2), 256, 0, st>>>(
        d, static_cast<const float *>(q), static_cast<const float *>(k), q_planes, k_planes);
    return cudaGetLastError();
}

}  // namespace sdm
