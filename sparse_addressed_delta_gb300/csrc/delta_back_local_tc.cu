// The chunk-local gradients of the gated delta rule (k_delta_back_local in delta_back.cu has the formulas)
// on the 5th-generation tensor cores, for bfloat16 inputs with up to 128 value columns. All sums lie in
// tensor memory, with a product's M = 128 in its lanes:
//   [dw; dO] r^T, q k^T  (rows: the tokens, 64 + 64)
//   G1 = S0 dO^T;  G2 = S0 dw^T;  G3 = D1 r^T  (rows: Dk)
//   dq^T = scale G G1 + K^T p^T;    dk^T = -beta G G2 + e^{L_C - L} beta G3 + Q^T p + K^T (a + a^T)
// S0 and D1 are A operands in tensor memory, as planes that their own lanes' threads store; dO, dw, r, K
// and Q are operands in shared memory, and so are the planes of p and a, which serve in both majors. Float32
// operands are three planes (24 bits), so that dq and dk differ from float32 arithmetic's only where that rounds
// the other way.
//
// A block stays on its SM and takes chunk after chunk, for all the value heads of one key head in turn:
// dq and dk are summed over them in registers, in head order. Warps 0..15 compute, warp 16 issues the
// products, warp 17 loads: K and Q of a chunk, dO of a head, and in boxes of 32 columns (four slots, in
// turn) dw and r, D1, S0 for <S0, D1>, and S0 again for its planes, whose place the first products have until
// then; always as far ahead as their places are free.
// What bounds it: a head's chunk reads 230 KB and writes its gradients (10000 cycles at the card's copy
// rate); its phases (planes, p and a, states, results) follow one another with one block an SM. Measured at
// 128 x 128, 32 heads by twos x 2 x 64 chunks: 460 us (2.2 TB/s), the whole backward 855; by m16n8k16 products
// (delta_back.cu) 1408. At 64 x 128 763 and 941.
//
// Every wait is bounded: one that gives up sets SDM_ERR_TIMEOUT in the status block; the computing warps
// then run through without waiting (they meet at barriers), the others stop and wait for what they have
// in flight.
#include "tcgen05.cuh"

namespace sdm {
namespace {

constexpr int kC = 64, kWarps = 16, kThreads = 32 * (kWarps + 2);

struct BackLocalTc {
    static constexpr int TILE = kC * 128, BOX = 128 * 128;         // 64 tokens; 32 float columns of a state
    // K and Q, dw's first plane and dO: two tiles (columns) each, alternating, so that one operand of 128
    // rows takes both
    static constexpr int K = 0, Q = K + TILE, W = 4 * TILE, G = W + TILE, PAIR = 2 * TILE;
    static constexpr int W1 = 8 * TILE, W2 = 10 * TILE, R = 12 * TILE;   // dw's other planes, r's three
    static constexpr int P = R, A = R + 3 * TILE;                  // three planes each, in the place of r's
    static constexpr int S = 18 * TILE;                            // four boxes
    static constexpr int F = S + 4 * BOX;
    // floats: from, to, beta, L (two) [5][C]; <dw, r>, row sums of a's part of z and of p's, column sums (of 32 rows
    // of either), x, y [4][C] each; <S0, D1> [warps]
    static constexpr int FLOATS = 5 * kC + 6 * 4 * kC + kWarps;
    static constexpr int BARS = F + FLOATS * 4, BYTES = BARS + 256 + 1024;
    static_assert(BYTES <= 227 * 1024 && BARS % 8 == 0, "shared memory");
    // tensor memory columns: [dw; dO] r^T, dw's other planes, [k; q] k^T, then in their place the planes of
    // S0; planes of D1, then in their place G1, G2 and dq's second terms; G3; dk's second terms
    static constexpr int E = 0, E2 = 64, QK = 128, SP = 0, DP = 192, G1 = 192, G2 = 256, DQ = 320, G3 = 384, DK = 448;
};

enum {
    B_T = 0, B_TFREE, B_DO, B_DOFREE, B_BOX, B_BFREE = B_BOX + 4, B_PL = B_BFREE + 4, B_E, B_D1, B_G3, B_PA, B_DQ, B_S0, B_G, B_DRAIN, B_COUNT
};

// blocks (r, c), (r + 8, c), (r, c + 8), (r + 8, c + 8) of a [tokens][128] operand in two tiles, PAIR apart
__device__ __forceinline__ unsigned at_rc(unsigned base, int r0, int c0, int lane) {
    const int r = r0 + (lane & 15), c = (c0 >> 3) + (lane >> 4);
    return base + (c >> 3) * BackLocalTc::PAIR + tc_at(r, c & 7);
}

__device__ __forceinline__ void state_load(void *dst, const CUtensorMap *m, int col, int slot, unsigned long long *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(m), "r"(col), "r"(0), "r"(slot), "r"(smem_u32(bar))
        : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
    k_delta_back_local_tc(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                          const __grid_constant__ CUtensorMap mg, const __grid_constant__ CUtensorMap ms,
                          const __grid_constant__ CUtensorMap md, const __grid_constant__ CUtensorMap mw,
                          const __grid_constant__ CUtensorMap mr, const __grid_constant__ CUtensorMap mdq,
                          const __grid_constant__ CUtensorMap mdk, DeltaDims d, DeltaIn in, DeltaLocal lw, DeltaBack o) {
    using L = BackLocalTc;
    using T = __nv_bfloat16;
    constexpr int C = kC;
    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    auto bar = reinterpret_cast<unsigned long long *>(smem + L::BARS);
    volatile int *dead = reinterpret_cast<int *>(bar + B_COUNT);
    auto slot = reinterpret_cast<uint32_t *>(bar + B_COUNT + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g4 = lane >> 2, i4 = lane & 3;
    const int group = d.H / d.Hk;
    const unsigned items = (unsigned)((long long)d.B * d.Hk * d.Nt);    // below 2^31

    if (tid == 0) {
        for (int i = 0; i < B_COUNT; ++i) {
            const bool all = i == B_PL || i == B_D1 || i == B_PA || i == B_S0;
            mbar_init(bar + i, all ? kWarps : i == B_TFREE ? kWarps + 1 : i >= B_BFREE && i < B_PL ? 4 : 1);
        }
        *dead = tc_gives_up(d.spin);
        fence_mbar_init();
    }
    if (warp == kWarps) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *slot;
    struct Item {
        int b, hk, n, nt;
    };
    auto item = [&](unsigned i) {
        Item x;
        x.n = (int)(i % (unsigned)d.Nt);
        const unsigned bh = i / (unsigned)d.Nt;
        x.b = (int)(bh / (unsigned)d.Hk);
        x.hk = (int)(bh % (unsigned)d.Hk);
        const int nt = delta_valid(in.valid, x.b, d.T) - x.n * C;
        x.nt = nt < 0 ? 0 : nt < C ? nt : C;
        return x;
    };

    if (warp < kWarps) {
        const int part = warp >> 2, lane0 = 32 * (warp & 3);
        const uint32_t at = tm + ((uint32_t)lane0 << 16);
        const unsigned sb = smem_u32(smem);
        float *from = reinterpret_cast<float *>(smem + L::F), *to = from + C, *be = to + C, *hi = be + C, *lo = hi + C;
        float *dwr = lo + C, *zrow = dwr + 4 * C, *zcol = zrow + 8 * C, *xs_t = zcol + 4 * C, *ys_t = xs_t + 4 * C, *ends = ys_t + 4 * C;
        auto meet = [] { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); };
        auto arrive = [&](int which) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + which);
        };
        // rows past the valid tokens of a [tokens][128] tile pair
        auto clear_rows = [&](unsigned char *tile, int nt) {
            for (int i = tid; i < (C - nt) * 16; i += 32 * kWarps) {
                const int r = nt + (i >> 4), c = i & 15;
                *reinterpret_cast<uint4 *>(tile + (c >> 3) * L::PAIR + tc_at(r, c & 7)) = make_uint4(0u, 0u, 0u, 0u);
            }
        };
        unsigned it = 0, unit = 0;                                 // items and heads so far
        for (unsigned i = blockIdx.x; i < items; i += gridDim.x) {
            const Item x = item(i);
            const int t0 = x.n * C, rows = d.T - t0 < C ? d.T - t0 : C;
            const long long tok = (long long)x.b * d.T + t0;
            if (x.nt == 0) {
                T *gq = static_cast<T *>(o.grad_q) + (tok * d.Hk + x.hk) * d.Dk, *gk = static_cast<T *>(o.grad_k) + (tok * d.Hk + x.hk) * d.Dk;
                for (int e = tid; e < rows * (d.Dk / 8); e += 32 * kWarps) {
                    const long long off = (long long)(e / (d.Dk / 8)) * d.Hk * d.Dk + 8 * (e % (d.Dk / 8));
                    *reinterpret_cast<uint4 *>(gq + off) = make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4 *>(gk + off) = make_uint4(0u, 0u, 0u, 0u);
                }
                for (int e = tid; e < rows * group; e += 32 * kWarps) {
                    const long long off = (tok + e / group) * d.H + x.hk * group + e % group;
                    o.grad_decay[off] = o.grad_beta[off] = 0.f;
                }
                continue;
            }
            tc_warp_wait(bar + B_T, it & 1, dead, d.spin);
            if (x.nt < C) {
                clear_rows(smem + L::K, x.nt);
                clear_rows(smem + L::Q, x.nt);
                fence_proxy_async_smem();
                meet();
            }
            // this warp's 32 of Dk x 16 tokens of dq^T and dk^T, in fragments: [16 lanes][..]
            float dq[2][8] = {}, dk[2][8] = {};
            for (int hh = 0; hh < group; ++hh, ++unit) {
                const int h = x.hk * group + hh;
                const long long bh = (long long)x.b * d.H + h, bhn = bh * d.Nt + x.n;
                meet();                                            // the last head's floats are used
                if (tid < 5 * C) from[tid] = lw.aux[bhn * kDeltaAux * C + tid];
                const unsigned par = unit & 1;
                const unsigned char *box = smem + L::S + part * L::BOX;    // this quarter's slot
                // dw and r as planes, <dw, r>: a thread takes 16 of the quarter's columns of a row
                {
                    const int r = (tid & 127) >> 1, hc = tid & 1;
                    meet();                                        // the gates; the last head's floats and planes
                    tc_warp_wait(bar + B_BOX + part, 0, dead, d.spin);
                    float z = 0.f;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {                  // 8 columns: one piece of each plane
                        float y[8], u[8];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int off = tc_at(r, 4 * hc + 2 * c + e);
                            *reinterpret_cast<float4 *>(y + 4 * e) = *reinterpret_cast<const float4 *>(box + off);
                            *reinterpret_cast<float4 *>(u + 4 * e) = *reinterpret_cast<const float4 *>(box + L::BOX / 2 + off);
                        }
                        unsigned p2[4][3], p3[4][3];
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            split_bf16<3>(y[2 * m], y[2 * m + 1], p2[m]);
                            split_bf16<3>(u[2 * m], u[2 * m + 1], p3[m]);
                        }
#pragma unroll
                        for (int m = 0; m < 8; ++m) z = fmaf(y[m], u[m], z);
                        const int pc = 4 * part + 2 * hc + c, off = tc_at(r, pc & 7), hf = pc >> 3;
                        *reinterpret_cast<uint4 *>(smem + L::W + hf * L::PAIR + off) = make_uint4(p2[0][0], p2[1][0], p2[2][0], p2[3][0]);
                        *reinterpret_cast<uint4 *>(smem + L::W1 + hf * L::TILE + off) = make_uint4(p2[0][1], p2[1][1], p2[2][1], p2[3][1]);
                        *reinterpret_cast<uint4 *>(smem + L::W2 + hf * L::TILE + off) = make_uint4(p2[0][2], p2[1][2], p2[2][2], p2[3][2]);
#pragma unroll
                        for (int p = 0; p < 3; ++p)
                            *reinterpret_cast<uint4 *>(smem + L::R + (2 * p + hf) * L::TILE + off) = make_uint4(p3[0][p], p3[1][p], p3[2][p], p3[3][p]);
                    }
                    arrive(B_BFREE + part);
                    z += __shfl_xor_sync(~0u, z, 1);
                    if (hc == 0) dwr[part * C + r] = z;
                }
                tc_warp_wait(bar + B_DO, par, dead, d.spin);
                if (x.nt < C) clear_rows(smem + L::G, x.nt);
                fence_proxy_async_smem();
                arrive(B_PL);
                // boxes of the states: 32 columns of the lane's row
                auto piece = [&](int c) { return *reinterpret_cast<const float4 *>(box + tc_at(lane0 + lane, c)); };
                auto planes = [&](uint32_t dst, const float4 (&y)[8]) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float x[16];
#pragma unroll
                        for (int e = 0; e < 4; ++e) *reinterpret_cast<float4 *>(x + 4 * e) = y[4 * half + e];
#pragma unroll
                        for (int m = 0; m < 3; ++m) {              // a term of each, then what is left of it
                            unsigned w[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                w[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
                                x[2 * e] -= lo_f32(w[e]);
                                x[2 * e + 1] -= hi_f32(w[e]);
                            }
                            tc_store8(dst + 64 * m + 16 * part + 8 * half, w);
                        }
                    }
                    tc_wait_st();
                    tc_fence_before();
                };
                {
                    float4 y[8];
                    tc_warp_wait(bar + B_BOX + part, 1, dead, d.spin);
#pragma unroll
                    for (int c = 0; c < 8; ++c) y[c] = piece(c);
                    arrive(B_BFREE + part);
                    planes(at + L::DP, y);
                    arrive(B_D1);
                    float s = 0.f;
                    tc_warp_wait(bar + B_BOX + part, 0, dead, d.spin);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const float4 z = piece(c);
                        s = fmaf(y[c].x, z.x, fmaf(y[c].y, z.y, fmaf(y[c].z, z.z, fmaf(y[c].w, z.w, s))));
                    }
                    arrive(B_BFREE + part);
#pragma unroll
                    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(~0u, s, m);
                    if (lane == 0) ends[warp] = s;
                }
                // a (lanes 0..63) and p (lanes 64..127) with the sums of their parts of z: a row t, 16 columns s
                tc_warp_wait(bar + B_E, par, dead, d.spin);
                tc_fence_after();
                {
                    const int t = (lane0 & 32) + lane;
                    const bool is_p = lane0 >= 64;
                    float y[16], z[16];
                    tc_load16(at + L::E + 16 * part, y);
                    if (!is_p) {
                        tc_load16(at + L::E2 + 16 * part, z);
#pragma unroll
                        for (int e = 0; e < 16; ++e) y[e] += z[e];
                    }
                    tc_load16(at + L::QK + 16 * part, z);
                    tc_fence_before();
                    if (16 * part <= (lane0 & 32) + 31) {          // else above the diagonal: never used
                        const float ht = hi[t], lt = lo[t], ft = is_p ? d.scale : -be[t];
                        float zr = 0.f;
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            float hs[4], ls[4], bs[4];
                            *reinterpret_cast<float4 *>(hs) = *reinterpret_cast<const float4 *>(hi + 16 * part + e);
                            *reinterpret_cast<float4 *>(ls) = *reinterpret_cast<const float4 *>(lo + 16 * part + e);
                            *reinterpret_cast<float4 *>(bs) = *reinterpret_cast<const float4 *>(be + 16 * part + e);
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                const int s = 16 * part + e + m;
                                const float f = s <= t ? expf((ht - hs[m]) + (lt - ls[m])) * bs[m] : 0.f;
                                const float w = ft * f * y[e + m];
                                y[e + m] = s < t || (is_p && s == t) ? w : 0.f;
                                z[e + m] = s < t ? w * z[e + m] : 0.f;
                                zr += z[e + m];
                            }
                        }
                        zrow[(is_p ? 4 : 0) * C + part * C + t] = zr;
                        // columns over the warp's rows: at each step a lane keeps the half of its columns that its bit names
#pragma unroll
                        for (int n = 8; n > 0; n /= 2)
#pragma unroll
                            for (int e = 0; e < n; ++e) {
                                const bool up = lane & (2 * n);
                                const float give = up ? z[e] : z[e + n];
                                z[e] = (up ? z[e + n] : z[e]) + __shfl_xor_sync(~0u, give, 2 * n);
                            }
                        z[0] += __shfl_xor_sync(~0u, z[0], 1);
                        if (!(lane & 1)) zcol[(warp & 3) * C + 16 * part + (lane >> 1)] = z[0];
                        unsigned char *dst = smem + (is_p ? L::P : L::A);
                        tc_warp_wait(bar + B_G3, par, dead, d.spin);   // r's planes are used
#pragma unroll
                        for (int p = 0; p < 3; ++p) {
                            unsigned w[8];                         // a term of each, then what is left of it
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                w[e] = pack_bf16(y[2 * e], y[2 * e + 1]);
                                y[2 * e] -= lo_f32(w[e]);
                                y[2 * e + 1] -= hi_f32(w[e]);
                            }
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                *reinterpret_cast<uint4 *>(dst + p * L::TILE + tc_at(t, 2 * part + e)) =
                                    make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                        }
                    }
                    fence_proxy_async_smem();
                    arrive(B_PA);
                }
                {
                    float4 y[8];
                    tc_warp_wait(bar + B_BOX + part, 1, dead, d.spin);
#pragma unroll
                    for (int c = 0; c < 8; ++c) y[c] = piece(c);
                    arrive(B_BFREE + part);
                    planes(at + L::SP, y);
                    arrive(B_S0);
                }
                // results: this warp's lanes (32 of Dk) and 16 tokens
                tc_warp_wait(bar + B_G, par, dead, d.spin);
                tc_fence_after();
                float f1[4], f2[4], f3[4], s1[4] = {}, s2[4] = {};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 16 * part + 8 * (e >> 1) + 2 * i4 + (e & 1);
                    f1[e] = d.scale * from[t];
                    f2[e] = -be[t] * from[t];
                    f3[e] = to[t] * be[t];
                }
#pragma unroll
                for (int l = 0; l < 2; ++l) {
                    const uint32_t a = at + ((uint32_t)(16 * l) << 16);
                    float y[8], z[8];
                    unsigned qf[4];
                    ldsm4t(qf, at_rc(sb + L::Q, 16 * part, lane0 + 16 * l, lane));
                    // blocks (tokens, Dk): (0, 0), (8, 0), (0, 8), (8, 8), transposed
                    tc_load_frag16(a + L::G1 + 16 * part, y);
#pragma unroll
                    for (int m = 0; m < 8; ++m) {
                        const int e = 2 * (m >> 2) + (m & 1);      // of the token
                        const unsigned qq = qf[2 * ((m >> 1) & 1) + (m >> 2)];
                        y[m] *= f1[e];
                        s1[e] = fmaf(m & 1 ? hi_f32(qq) : lo_f32(qq), y[m], s1[e]);
                        dq[l][m] += y[m];
                    }
                    tc_load_frag16(a + L::G2 + 16 * part, a + L::G3 + 16 * part, y, z);
                    ldsm4t(qf, at_rc(sb + L::K, 16 * part, lane0 + 16 * l, lane));
#pragma unroll
                    for (int m = 0; m < 8; ++m) {
                        const int e = 2 * (m >> 2) + (m & 1);
                        const unsigned kk = qf[2 * ((m >> 1) & 1) + (m >> 2)];
                        const float kv = m & 1 ? hi_f32(kk) : lo_f32(kk);
                        y[m] *= f2[e];
                        z[m] *= f3[e];
                        s1[e] = fmaf(kv, y[m], s1[e]);
                        s2[e] = fmaf(kv, z[m], s2[e]);
                        dk[l][m] += y[m] + z[m];
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
#pragma unroll
                    for (int m = 4; m < 32; m *= 2) {
                        s1[e] += __shfl_xor_sync(~0u, s1[e], m);
                        s2[e] += __shfl_xor_sync(~0u, s2[e], m);
                    }
                    if (g4 == 0) {
                        const int r = (warp & 3) * C + 16 * part + 8 * (e >> 1) + 2 * i4 + (e & 1);
                        xs_t[r] = s1[e];
                        ys_t[r] = s2[e];
                    }
                }
#pragma unroll
                for (int l = 0; l < 2; ++l) {
                    const uint32_t a = at + ((uint32_t)(16 * l) << 16);
                    float y[8], z[8];
                    tc_load_frag16(a + L::DQ + 16 * part, a + L::DK + 16 * part, y, z);
#pragma unroll
                    for (int m = 0; m < 8; ++m) {
                        dq[l][m] += y[m];
                        dk[l][m] += z[m];
                    }
                }
                tc_fence_before();
                meet();
                if (warp == kWarps - 1) {
                    float xt[2], yt[2];
                    double whole = 0.0, dg[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = 2 * lane + e;
                        xt[e] = yt[e] = 0.f;
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            if (16 * p <= r) xt[e] += zrow[p * C + r] + zrow[(4 + p) * C + r];
                            if ((p & 1) || r < 32) xt[e] -= zcol[p * C + r];   // rows 32 (p % 2)..
                            xt[e] += xs_t[p * C + r];
                            yt[e] += ys_t[p * C + r];
                        }
                    }
#pragma unroll
                    for (int p = 0; p < kWarps; ++p) whole += (double)ends[p];
                    delta_decay_sums(xt, yt, (double)from[C - 1] * whole, dg);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = 2 * lane + e;
                        if (r < rows) {
                            const bool some = r < x.nt && expf(delta_decay(in.g[x.b * d.gs[0] + (t0 + r) * d.gs[1] + h * d.gs[2]])) != 0.f;
                            o.grad_decay[(tok + r) * d.H + h] = some ? (float)dg[e] : 0.f;
                            o.grad_beta[(tok + r) * d.H + h] = r < x.nt ? (dwr[r] + dwr[C + r]) + (dwr[2 * C + r] + dwr[3 * C + r]) : 0.f;
                        }
                    }
                }
            }
            // dq and dk as rows in the places of dw's second plane and r's first, stored as tensors
            {
                const int orow = 16 * part + 8 * (lane >> 4) + (lane & 7), ocol = (lane0 >> 3) + ((lane >> 3) & 1);
#pragma unroll
                for (int l = 0; l < 2; ++l) {
                    unsigned r[4];
                    const int c = ocol + 2 * l;
                    const unsigned dst = sb + (c >> 3) * L::TILE + tc_at(orow, c & 7);
                    auto live = [&](int m) { return 16 * part + 8 * (m >> 2) + 2 * i4 + (m & 1) < x.nt; };
#pragma unroll
                    for (int e = 0; e < 4; ++e) r[e] = pack_bf16(live(2 * e) ? dq[l][2 * e] : 0.f, live(2 * e + 1) ? dq[l][2 * e + 1] : 0.f);
                    stsm4t(dst + L::W1, r);
#pragma unroll
                    for (int e = 0; e < 4; ++e) r[e] = pack_bf16(live(2 * e) ? dk[l][2 * e] : 0.f, live(2 * e + 1) ? dk[l][2 * e + 1] : 0.f);
                    stsm4t(dst + L::R, r);
                }
                fence_proxy_async_smem();
                arrive(B_TFREE);
                meet();
                if (warp == 0 && lane == 0) {
                    for (int c = 0; c < 2; ++c)
                        if (64 * c < d.Dk) {
                            tc_tensor_store(&mdq, 64 * c, x.hk, t0, x.b, smem + L::W1 + c * L::TILE);
                            tc_tensor_store(&mdk, 64 * c, x.hk, t0, x.b, smem + L::R + c * L::TILE);
                        }
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                }
                // the next head's first barrier keeps the others off those planes until this is read
            }
            ++it;
        }
        if (warp == 0 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    } else if (warp == kWarps) {
        // ---- the products
        const uint32_t one = tc_elect(), tu = __shfl_sync(~0u, tm, 0);
        // one tile's K steps of 16 columns, then the other's: `pair` bytes apart
        auto at_ks = [](int ks, int pair) { return ((ks >> 2) * pair + 32 * (ks & 3)) / 16; };
        unsigned it = 0, unit = 0;
        bool ok = true;
        for (unsigned i = blockIdx.x; i < items && ok; i += gridDim.x) {
            const Item x = item(i);
            if (x.nt == 0) continue;
            for (int hh = 0; hh < group && ok; ++hh, ++unit) {
                const unsigned par = unit & 1;
                // anew for every head: kept over the loop, the 230 descriptors are spilled
                const uint32_t base = __shfl_sync(~0u, smem_u32(smem), 0);
                const uint32_t kq = tc_k_major(base + L::K), wg = tc_k_major(base + L::W), w1 = tc_k_major(base + L::W1), w2 = tc_k_major(base + L::W2);
                const uint32_t gk = tc_k_major(base + L::G), rk = tc_k_major(base + L::R);
                const uint32_t km = tc_n_major(base + L::K, L::PAIR), qm = tc_n_major(base + L::Q, L::PAIR);
                const uint32_t pk = tc_k_major(base + L::P), pn = tc_n_major(base + L::P, L::TILE);
                const uint32_t ak = tc_k_major(base + L::A), an = tc_n_major(base + L::A, L::TILE);
                auto states = [&](uint32_t dst, uint32_t a, uint32_t tile, int pair, bool first) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        tc_mma_ts(one, tu + dst, tu + a + 8 * ks, tile + at_ks(ks, pair), tc_idesc<false>(C), !first || ks > 0);
                };
                auto rows = [&](uint32_t dst, uint32_t a, uint32_t tile, int apair, int pair, bool first) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        tc_mma_ss(one, tu + dst, a + at_ks(ks, apair), tile + at_ks(ks, pair), tc_idesc<false>(C), !first || ks > 0);
                };
                ok = tc_warp_wait(bar + B_PL, par, dead, d.spin);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int p = 2; p >= 0; --p) rows(L::E, wg, rk + 2 * p * L::TILE / 16, L::PAIR, L::TILE, p == 2);
                rows(L::E2, w2, rk, L::TILE, L::TILE, true);
                rows(L::E2, w1, rk + 2 * L::TILE / 16, L::TILE, L::TILE, false);
                rows(L::E2, w1, rk, L::TILE, L::TILE, false);
                rows(L::QK, kq, kq, L::PAIR, L::PAIR, true);
                tc_commit_to(one, bar + B_E);
                ok = tc_warp_wait(bar + B_D1, par, dead, d.spin);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int sum = 2; sum >= 0; --sum)                 // pairs of terms from the smallest up
#pragma unroll
                    for (int a = sum; a >= 0; --a) states(L::G3, L::DP + 64 * a, rk + 2 * (sum - a) * L::TILE / 16, L::TILE, a == 2);
                tc_commit_to(one, bar + B_G3);
                ok = tc_warp_wait(bar + B_S0, par, dead, d.spin) && tc_warp_wait(bar + B_G3, par, dead, d.spin);
                if (!ok) break;
                tc_fence_after();
                states(L::G1, L::SP + 128, gk, L::PAIR, true);
                states(L::G1, L::SP + 64, gk, L::PAIR, false);
                states(L::G1, L::SP, gk, L::PAIR, false);
                states(L::G2, L::SP + 128, wg, L::PAIR, true);
                states(L::G2, L::SP + 64, w1, L::TILE, false);
                states(L::G2, L::SP, w2, L::TILE, false);
                states(L::G2, L::SP + 64, wg, L::PAIR, false);
                states(L::G2, L::SP, w1, L::TILE, false);
                states(L::G2, L::SP, wg, L::PAIR, false);
                ok = tc_warp_wait(bar + B_PA, par, dead, d.spin);
                if (!ok) break;
                tc_fence_after();
                // B = lower triangular [t][s]: with t its N, K step s reaches the columns from 16 ks on; with
                // s its N, K step t those up to 16 ks + 15
#pragma unroll
                for (int p = 2; p >= 0; --p) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        tc_mma_ss(one, tu + L::DQ + 16 * ks, km + 2048 * ks / 16, pk + (p * L::TILE + 16 * ks * 128 + 32 * ks) / 16,
                                  tc_idesc<false, true>(C - 16 * ks), p < 2 || ks > 0);
#pragma unroll
                    for (int ks = 3; ks >= 0; --ks)
                        tc_mma_ss(one, tu + L::DK, qm + 2048 * ks / 16, pn + (p * L::TILE + 2048 * ks) / 16, tc_idesc<true, true>(16 * ks + 16),
                                  p < 2 || ks < 3);
#pragma unroll
                    for (int ks = 3; ks >= 0; --ks)
                        tc_mma_ss(one, tu + L::DK, km + 2048 * ks / 16, an + (p * L::TILE + 2048 * ks) / 16, tc_idesc<true, true>(16 * ks + 16), true);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        tc_mma_ss(one, tu + L::DK + 16 * ks, km + 2048 * ks / 16, ak + (p * L::TILE + 16 * ks * 128 + 32 * ks) / 16,
                                  tc_idesc<false, true>(C - 16 * ks), true);
                }
                tc_commit_to(one, bar + B_G);
                tc_commit_to(one, bar + B_DOFREE);
                if (hh + 1 == group) tc_commit_to(one, bar + B_TFREE);
            }
            ++it;
        }
        __syncwarp();
    } else {
        // ---- the loads
        unsigned it = 0, unit = 0, boxes = 0, grads = 0;           // the last two: started
        bool ok = true;
        for (unsigned i = blockIdx.x; i < items && ok; i += gridDim.x) {
            const Item x = item(i);
            if (x.nt == 0) continue;
            const int t0 = x.n * C;
            for (int hh = 0; hh < group && ok; ++hh, ++unit) {
                const int h = x.hk * group + hh;
                const long long bh = (long long)x.b * d.H + h, chunk = bh * d.Nt + x.n;
                // the slots free up in the middle of the head before: the next one's dw and r first
                for (int e = 0; e < 16 && ok; ++e) {
                    const int s = e & 3, j = e >> 2;
                    if (unit > 0 || j > 0) ok = tc_warp_wait(bar + B_BFREE + s, (j + 1) & 1, dead, d.spin);
                    if (!ok) break;
                    if (lane == 0) {
                        unsigned char *dst = smem + L::S + s * L::BOX;
                        mbar_arrive_expect_tx(bar + B_BOX + s, L::BOX);
                        if (j == 0) {
                            state_load(dst, &mw, 32 * s, (int)chunk, bar + B_BOX + s);
                            state_load(dst + L::BOX / 2, &mr, 32 * s, (int)chunk, bar + B_BOX + s);
                        } else {
                            state_load(dst, j == 1 ? &md : &ms, 32 * s, (int)(j == 1 ? chunk : bh * (d.Nt + 1) + x.n), bar + B_BOX + s);
                        }
                    }
                    __syncwarp();
                    ++boxes;
                    if (e == 3) {
                        if (unit > 0) ok = tc_warp_wait(bar + B_DOFREE, (unit - 1) & 1, dead, d.spin);
                        if (!ok) break;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(bar + B_DO, 2 * L::TILE);
                            for (int c = 0; c < 2; ++c) tc_tensor_load(smem + L::G + c * L::PAIR, &mg, 64 * c, tc_coord(d.os[2], h), t0, tc_coord(d.os[0], x.b), bar + B_DO);
                        }
                        ++grads;
                        if (hh == 0) {
                            if (it > 0) ok = tc_warp_wait(bar + B_TFREE, (it - 1) & 1, dead, d.spin);
                            if (!ok) break;
                            if (lane == 0) {
                                mbar_arrive_expect_tx(bar + B_T, 4 * L::TILE);
                                for (int c = 0; c < 2; ++c) {
                                    tc_tensor_load(smem + L::K + c * L::PAIR, &mk, 64 * c, tc_coord(d.ks[2], x.hk), t0, tc_coord(d.ks[0], x.b), bar + B_T);
                                    tc_tensor_load(smem + L::Q + c * L::PAIR, &mq, 64 * c, tc_coord(d.qs[2], x.hk), t0, tc_coord(d.qs[0], x.b), bar + B_T);
                                }
                            }
                            ++it;
                        }
                        __syncwarp();
                    }
                }
            }
        }
        // nothing in flight behind a give-up: the last copies started on each barrier
        if (it > 0) mbar_wait_bounded(bar + B_T, (it - 1) & 1);
        if (grads > 0) mbar_wait_bounded(bar + B_DO, (grads - 1) & 1);
        for (unsigned s = 0; s < 4; ++s)
            if (boxes > s) mbar_wait_bounded(bar + B_BOX + s, ((boxes - 1 - s) / 4) & 1);
        __syncwarp();
    }
    __syncthreads();
    if (*dead) {
        if (tid == 32 * kWarps) {                                  // the products issued so far
            tc_commit_to(1, bar + B_DRAIN);
            mbar_wait_bounded(bar + B_DRAIN, 0);
            atomicCAS(&lw.status->code, 0, (int)SDM_ERR_TIMEOUT);
        }
        __syncthreads();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarps) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512));
}

}  // namespace

cudaError_t launch_delta_back_local_tc(const DeltaDims &d, const DeltaIn &in, const DeltaLocal &w, const DeltaBack &o,
                                       cudaStream_t st) {
    const long long ks[3] = {(long long)d.T * d.Hk * d.Dk, (long long)d.Hk * d.Dk, d.Dk};
    CUtensorMap mq, mk, mg, ms, md, mw, mr, mdq, mdk;
    cudaError_t e = tc_tensor_map(&mq, in.q, d.qs, d.B, d.T, d.Hk, d.Dk);
    if (e == cudaSuccess) e = tc_tensor_map(&mk, in.k, d.ks, d.B, d.T, d.Hk, d.Dk);
    if (e == cudaSuccess) e = tc_tensor_map(&mg, o.grad, d.os, d.B, d.T, d.H, d.Dv);
    if (e == cudaSuccess) e = tc_tensor_map(&mdq, o.grad_q, ks, d.B, d.T, d.Hk, d.Dk);
    if (e == cudaSuccess) e = tc_tensor_map(&mdk, o.grad_k, ks, d.B, d.T, d.Hk, d.Dk);
    if (e == cudaSuccess) e = tc_state_map(&ms, o.snap, (long long)d.B * d.H * (d.Nt + 1), d.Dk, d.Dv, 128);
    if (e == cudaSuccess) e = tc_state_map(&md, o.ends, (long long)d.B * d.H * d.Nt, d.Dk, d.Dv, 128);
    if (e == cudaSuccess) e = tc_state_map(&mw, o.w, (long long)d.B * d.H * d.Nt, kC, d.Dv, kC);
    if (e == cudaSuccess) e = tc_state_map(&mr, o.r, (long long)d.B * d.H * d.Nt, kC, d.Dv, kC);
    if (e != cudaSuccess) return e;
    set_kernel_smem(k_delta_back_local_tc, BackLocalTc::BYTES);
    const long long items = (long long)d.B * d.Hk * d.Nt;
    k_delta_back_local_tc<<<(unsigned)(items < kRefSms ? items : kRefSms), kThreads, BackLocalTc::BYTES, st>>>(
        mq, mk, mg, ms, md, mw, mr, mdq, mdk, d, in, w, o);
    return cudaGetLastError();
}

}  // namespace sdm
