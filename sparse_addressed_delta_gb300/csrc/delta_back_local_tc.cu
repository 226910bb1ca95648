// The chunk-local gradients of the gated delta rule (k_delta_back_local in delta_back.cu has the formulas)
// on the 5th-generation tensor cores, for bfloat16 inputs. Transposed: 128 of Dk are the lanes of tensor
// memory, the chunk's 64 tokens its columns.
//   G1 = S0 dO^T (3 planes of S0);  G2 = S0 dw^T;  G3 = D1 r^T (two planes of each operand)
//   dq^T = scale G G1 + K^T p^T;    dk^T = -beta G G2 + e^{L_C - L} beta G3 + Q^T p + K^T (a + a^T)
// S0 and D1 are A operands in tensor memory, as planes that their own lanes' threads store; dO, dw and r
// are B operands in shared memory; K and Q are A operands there for the second line, whose B operands p
// and a serve in both majors. The C x C products dw r^T, dO r^T and q k^T, ten 16 x 16 blocks on and below
// the diagonal, are a warp's m16n8k16 products each, beside the others.
//
// A block stays on its SM and takes chunk after chunk, for all the value heads of one key head in turn:
// dq and dk are summed over them in registers, in head order. Warps 0..15 compute, warp 16 issues the
// products, warp 17 loads: K and Q of a chunk, dO of a head, the states in boxes of 32 columns (four
// slots), always as far ahead as their places are free.
// What bounds it: a head's chunk reads 225 KB and writes its gradients; the phases (planes, states,
// products, results) follow one another with one block an SM.
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
    static constexpr int K = 0, Q = 2 * TILE, G = 4 * TILE;        // G: the readings' gradient
    static constexpr int W = 6 * TILE, R = 10 * TILE;              // two planes of dw, three of r
    static constexpr int P = W, A = W + 2 * TILE;                  // two planes each, once dw's are used
    static constexpr int S = 16 * TILE;                            // four boxes
    static constexpr int F = S + 4 * BOX;
    // floats: from, to, beta, L (two) [5][C]; <dw, v>, <dw, r> [C]; row sums of p * qk [4][C]; row products
    // with q [4][C]; <S1, D1> [warps]
    static constexpr int FLOATS = 7 * kC + 4 * kC + 4 * kC + kWarps;
    static constexpr int BARS = F + FLOATS * 4, BYTES = BARS + 256 + 1024;
    static_assert(BYTES <= 227 * 1024 && BARS % 8 == 0, "shared memory");
    // tensor memory columns: planes of S0 (then dq's and dk's second terms), of D1, G1, G2, G3
    static constexpr int SP = 0, DQ = 0, DK = 64, DP = 192, G1 = 320, G2 = 384, G3 = 448;
};

enum {
    B_T = 0, B_TFREE, B_DO, B_DOFREE, B_BOX, B_BFREE = B_BOX + 4, B_PL = B_BFREE + 4, B_S0, B_D1, B_G, B_PA, B_DQ, B_DRAIN, B_COUNT
};

// fragments of a [tokens][128] operand in two tiles as tc_at lays them out (frag_rc, frag_cr)
__device__ __forceinline__ unsigned at_rc(unsigned base, int r0, int c0, int lane) {
    const int r = r0 + (lane & 15), c = (c0 >> 3) + (lane >> 4);
    return base + (c >> 3) * BackLocalTc::TILE + tc_at(r, c & 7);
}
__device__ __forceinline__ unsigned at_cr(unsigned base, int r0, int c0, int lane) {
    const int r = r0 + (lane & 7) + ((lane >> 4) << 3), c = (c0 >> 3) + ((lane >> 3) & 1);
    return base + (c >> 3) * BackLocalTc::TILE + tc_at(r, c & 7);
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
                          const __grid_constant__ CUtensorMap md, const __grid_constant__ CUtensorMap mdq,
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
    const int group = d.H / d.Hk, tiles = (d.Dv + 127) / 128;
    const long long items = (long long)d.B * d.Hk * d.Nt;

    if (tid == 0) {
        for (int i = 0; i < B_COUNT; ++i) {
            const bool all = i == B_PL || i == B_S0 || i == B_D1;
            mbar_init(bar + i, all ? kWarps : i == B_TFREE || i == B_DOFREE ? kWarps + 1 : i >= B_BFREE && i < B_PL ? 4 : i == B_PA ? 10 : 1);
        }
        *dead = 0;
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
    auto item = [&](long long i) {
        Item x;
        x.n = (int)(i % d.Nt);
        const long long bh = i / d.Nt;
        x.b = (int)(bh / d.Hk);
        x.hk = (int)(bh % d.Hk);
        const int nt = delta_valid(in.valid, x.b, d.T) - x.n * C;
        x.nt = nt < 0 ? 0 : nt < C ? nt : C;
        return x;
    };

    if (warp < kWarps) {
        const int part = warp >> 2, lane0 = 32 * (warp & 3);
        const uint32_t at = tm + ((uint32_t)lane0 << 16);
        const unsigned sb = smem_u32(smem);
        float *from = reinterpret_cast<float *>(smem + L::F), *to = from + C, *be = to + C, *hi = be + C, *lo = hi + C;
        float *dwv = lo + C, *dwr = dwv + C, *zrow = dwr + C, *dots = zrow + 4 * C, *ends = dots + 4 * C;
        const bool block = warp < 10;
        const int bi = warp < 1 ? 0 : warp < 3 ? 1 : warp < 6 ? 2 : 3, bj = warp - bi * (bi + 1) / 2;
        auto meet = [] { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); };
        auto arrive = [&](int which) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + which);
        };
        // rows past the valid tokens of a [tokens][128] tile pair
        auto clear_rows = [&](unsigned char *tile, int nt) {
            for (int i = tid; i < (C - nt) * 16; i += 32 * kWarps) {
                const int r = nt + (i >> 4), c = i & 15;
                *reinterpret_cast<uint4 *>(tile + (c >> 3) * L::TILE + tc_at(r, c & 7)) = make_uint4(0u, 0u, 0u, 0u);
            }
        };
        unsigned it = 0, unit = 0, step = 0;                       // items, heads and column tiles so far
        for (long long i = blockIdx.x; i < items; i += gridDim.x) {
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
            float qk[2][4] = {};
            if (block) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    unsigned a[4], bb[4];
                    ldsm4(a, at_rc(sb + L::Q, 16 * bi, 16 * ks, lane));
                    ldsm4(bb, at_cr(sb + L::K, 16 * bj, 16 * ks, lane));
#pragma unroll
                    for (int e = 0; e < 2; ++e) mma_bf16(qk[e], a, bb[2 * e], bb[2 * e + 1]);
                }
            }
            // this warp's 32 of Dk x 16 tokens of dq^T and dk^T, in fragments: [16 lanes][..]
            float dq[2][8] = {}, dk[2][8] = {};
            for (int hh = 0; hh < group; ++hh, ++unit) {
                const int h = x.hk * group + hh;
                const long long bh = (long long)x.b * d.H + h, bhn = bh * d.Nt + x.n, cells = (long long)d.Dk * d.Dv;
                meet();                                            // the last head's floats are used
                if (tid < 5 * C) from[tid] = lw.aux[bhn * kDeltaAux * C + tid];
                else if (tid - 5 * C < 2 * C) dwv[tid - 5 * C] = 0.f;
                const T *val = static_cast<const T *>(in.v) + x.b * d.vs[0] + t0 * d.vs[1] + h * d.vs[2];
                const float *wp = o.w + bhn * C * (long long)d.Dv, *rp = o.r + bhn * C * (long long)d.Dv;
                {
                    const float4 *u = reinterpret_cast<const float4 *>(o.snap + (bh * (d.Nt + 1) + x.n + 1) * cells);
                    const float4 *v = reinterpret_cast<const float4 *>(o.ends + bhn * cells);
                    float s = 0.f;
#pragma unroll 4
                    for (int e = tid; e < (int)(cells / 4); e += 32 * kWarps) {
                        const float4 a = __ldg(u + e), c = __ldg(v + e);
                        s = fmaf(a.x, c.x, fmaf(a.y, c.y, fmaf(a.z, c.z, fmaf(a.w, c.w, s))));
                    }
#pragma unroll
                    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(~0u, s, m);
                    if (lane == 0) ends[warp] = s;
                }
                meet();
                // dP's lesser terms have a sum of their own: the tensor core cuts an accumulator's low bits
                float E[2][4] = {}, DP[2][4] = {}, LP[2][4] = {};
                for (int tl = 0; tl < tiles; ++tl, ++step) {
                    const unsigned par = step & 1;
                    const int c0 = 128 * tl;
                    if (tl > 0) tc_warp_wait(bar + B_G, par ^ 1, dead, d.spin);   // the planes are used
                    if (tl > 0) meet();
                    // dw and r as planes; <dw, v> and <dw, r>
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int idx = tid + 32 * kWarps * e, r = idx >> 4, c = idx & 15, col = c0 + 8 * c;
                        float y[8] = {}, u[8] = {}, v[8] = {};
                        if (r < x.nt && col < d.Dv) {
                            load_vec<float, 8, true>(wp + (long long)r * d.Dv + col, y);
                            load_vec<float, 8, true>(rp + (long long)r * d.Dv + col, u);
                            load_vec<T, 8, true>(val + r * d.vs[1] + col, v);
                        }
                        float s = 0.f, z = 0.f;
#pragma unroll
                        for (int m = 0; m < 8; ++m) {
                            s = fmaf(y[m], v[m], s);
                            z = fmaf(y[m], u[m], z);
                        }
#pragma unroll
                        for (int m = 1; m < 16; m *= 2) {
                            s += __shfl_xor_sync(~0u, s, m);
                            z += __shfl_xor_sync(~0u, z, m);
                        }
                        if (c == 0) {
                            dwv[r] += s;
                            dwr[r] += z;
                        }
                        unsigned char *dst = smem + L::W + (c >> 3) * L::TILE + tc_at(r, c & 7);
                        unsigned p2[4][2], p3[4][3];
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            split_bf16<2>(y[2 * m], y[2 * m + 1], p2[m]);
                            split_bf16<3>(u[2 * m], u[2 * m + 1], p3[m]);
                        }
#pragma unroll
                        for (int p = 0; p < 2; ++p)
                            *reinterpret_cast<uint4 *>(dst + 2 * p * L::TILE) = make_uint4(p2[0][p], p2[1][p], p2[2][p], p2[3][p]);
#pragma unroll
                        for (int p = 0; p < 3; ++p)
                            *reinterpret_cast<uint4 *>(dst + (L::R - L::W) + 2 * p * L::TILE) = make_uint4(p3[0][p], p3[1][p], p3[2][p], p3[3][p]);
                    }
                    tc_warp_wait(bar + B_DO, par, dead, d.spin);
                    if (x.nt < C) clear_rows(smem + L::G, x.nt);
                    fence_proxy_async_smem();
                    arrive(B_PL);
                    // this quarter's box of a state, 32 columns of the lane's row, as N planes
                    auto box = [&](auto planes, uint32_t dst, unsigned phase) {
                        constexpr int N = decltype(planes)::value;
                        tc_warp_wait(bar + B_BOX + part, phase, dead, d.spin);
                        const unsigned char *src = smem + L::S + part * L::BOX;
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            unsigned p[N][8];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float4 y = *reinterpret_cast<const float4 *>(src + tc_at(lane0 + lane, 4 * half + e));
                                unsigned s0[N], s1[N];
                                split_bf16<N>(y.x, y.y, s0);
                                split_bf16<N>(y.z, y.w, s1);
#pragma unroll
                                for (int m = 0; m < N; ++m) {
                                    p[m][2 * e] = s0[m];
                                    p[m][2 * e + 1] = s1[m];
                                }
                            }
#pragma unroll
                            for (int m = 0; m < N; ++m) tc_store8(at + dst + 64 * m + 16 * part + 8 * half, p[m]);
                        }
                        arrive(B_BFREE + part);
                        tc_wait_st();
                        tc_fence_before();
                    };
                    box(std::integral_constant<int, 3>{}, L::SP, 0);
                    arrive(B_S0);
                    box(std::integral_constant<int, 2>{}, L::DP, 1);
                    arrive(B_D1);
                    tc_warp_wait(bar + B_PL, par, dead, d.spin);
                    if (block) {
#pragma unroll 2
                        for (int ks = 0; ks < 8; ++ks) {
                            unsigned aw[2][4], ao[4], br[3][4];
#pragma unroll
                            for (int p = 0; p < 2; ++p) ldsm4(aw[p], at_rc(sb + L::W + 2 * p * L::TILE, 16 * bi, 16 * ks, lane));
#pragma unroll
                            for (int p = 0; p < 3; ++p) ldsm4(br[p], at_cr(sb + L::R + 2 * p * L::TILE, 16 * bj, 16 * ks, lane));
                            ldsm4(ao, at_rc(sb + L::G, 16 * bi, 16 * ks, lane));
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                mma_bf16(LP[e], ao, br[2][2 * e], br[2][2 * e + 1]);
                                mma_bf16(E[e], aw[1], br[0][2 * e], br[0][2 * e + 1]);
                                mma_bf16(DP[e], ao, br[0][2 * e], br[0][2 * e + 1]);
                                mma_bf16(E[e], aw[0], br[1][2 * e], br[1][2 * e + 1]);
                                mma_bf16(LP[e], ao, br[1][2 * e], br[1][2 * e + 1]);
                                mma_bf16(E[e], aw[0], br[0][2 * e], br[0][2 * e + 1]);
                            }
                        }
                    }
                    arrive(B_DOFREE);
                }
                tc_warp_wait(bar + B_G, (step - 1) & 1, dead, d.spin);
                tc_fence_after();
                meet();                                            // dw's planes are used by all
                if (block) {                                       // p, a and the row sums of p * (q k^T)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int t = 16 * bi + g4 + 8 * half;
                        const float ht = hi[t], lt = lo[t], bt = be[t];
                        float zr = 0.f;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float pa[2], aa[2];
#pragma unroll
                            for (int m = 0; m < 2; ++m) {
                                const int s = 16 * bj + 8 * e + 2 * i4 + m, j = 2 * half + m;
                                const float f = s <= t ? expf((ht - hi[s]) + (lt - lo[s])) * be[s] : 0.f;
                                pa[m] = s <= t ? d.scale * ((DP[e][j] + LP[e][j]) * f) : 0.f;
                                aa[m] = s < t ? -bt * (E[e][j] * f) : 0.f;
                                zr = s <= t ? fmaf(pa[m], qk[e][j], zr) : zr;
                            }
                            const int off = tc_at(t, 2 * bj + e) + 4 * i4;
                            unsigned pl[2];
                            split_bf16<2>(pa[0], pa[1], pl);
                            *reinterpret_cast<unsigned *>(smem + L::P + off) = pl[0];
                            *reinterpret_cast<unsigned *>(smem + L::P + L::TILE + off) = pl[1];
                            split_bf16<2>(aa[0], aa[1], pl);
                            *reinterpret_cast<unsigned *>(smem + L::A + off) = pl[0];
                            *reinterpret_cast<unsigned *>(smem + L::A + L::TILE + off) = pl[1];
                        }
                        zr += __shfl_xor_sync(~0u, zr, 1);
                        zr += __shfl_xor_sync(~0u, zr, 2);
                        if (i4 == 0) zrow[bj * C + t] = zr;
                    }
                    fence_proxy_async_smem();
                    arrive(B_PA);
                }
                // results: this warp's lanes (32 of Dk) and 16 tokens
                float f1[4], f2[4], f3[4], s1[4] = {};
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
#pragma unroll
                    for (int m = 0; m < 8; ++m) {
                        const int e = 2 * (m >> 2) + (m & 1);
                        dk[l][m] += fmaf(f2[e], y[m], f3[e] * z[m]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
#pragma unroll
                    for (int m = 4; m < 32; m *= 2) s1[e] += __shfl_xor_sync(~0u, s1[e], m);
                    if (g4 == 0) dots[(warp & 3) * C + 16 * part + 8 * (e >> 1) + 2 * i4 + (e & 1)] = s1[e];
                }
                tc_warp_wait(bar + B_DQ, unit & 1, dead, d.spin);
                tc_fence_after();
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
                    double suf[2], rev = 0.0;
#pragma unroll
                    for (int e = 1; e >= 0; --e) {
                        const int r = 2 * lane + e;
                        float z = 0.f;
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            if (16 * p <= r) z += zrow[p * C + r];
                            z += dots[p * C + r];
                        }
                        rev += (double)z - (double)be[r] * (double)dwv[r];
                        suf[e] = rev;
                    }
                    double after = rev;
#pragma unroll
                    for (int m = 1; m < 32; m *= 2) {
                        const double y = __shfl_down_sync(~0u, after, m);
                        if (lane + m < 32) after += y;
                    }
                    after -= rev;
#pragma unroll
                    for (int p = 0; p < kWarps; ++p) after += (double)ends[p];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = 2 * lane + e;
                        if (r < rows) {
                            o.grad_decay[(tok + r) * d.H + h] = r < x.nt ? (float)(after + suf[e]) : 0.f;
                            o.grad_beta[(tok + r) * d.H + h] = r < x.nt ? dwr[r] : 0.f;
                        }
                    }
                }
            }
            // dq and dk as rows in the places of dw's planes and r's first, stored as tensors
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
                    stsm4t(dst + L::W, r);
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
                            tc_tensor_store(&mdq, 64 * c, x.hk, t0, x.b, smem + L::W + c * L::TILE);
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
        const uint32_t one = tc_elect(), tu = __shfl_sync(~0u, tm, 0), base = __shfl_sync(~0u, smem_u32(smem), 0);
        const uint64_t gk = tc_k_major(base + L::G), wk = tc_k_major(base + L::W), rk = tc_k_major(base + L::R);
        const uint64_t km = tc_n_major(base + L::K, L::TILE), qm = tc_n_major(base + L::Q, L::TILE);
        const uint64_t pk = tc_k_major(base + L::P), pn = tc_n_major(base + L::P, L::TILE);
        const uint64_t ak = tc_k_major(base + L::A), an = tc_n_major(base + L::A, L::TILE);
        unsigned unit = 0, step = 0;
        bool ok = true;
        for (long long i = blockIdx.x; i < items && ok; i += gridDim.x) {
            const Item x = item(i);
            if (x.nt == 0) continue;
            for (int hh = 0; hh < group && ok; ++hh, ++unit) {
                for (int tl = 0; tl < tiles && ok; ++tl, ++step) {
                    const unsigned par = step & 1;
                    // 8 K steps of 16 columns; plane `a` of a state, plane tile of dO, dw or r
                    auto states = [&](uint32_t dst, uint32_t a, uint64_t tile, bool first) {
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            tc_mma_ts(one, tu + dst, tu + a + 8 * ks, tile + ((ks >> 2) * L::TILE + 32 * (ks & 3)) / 16, tc_idesc<false>(C), !first || ks > 0 || tl > 0);
                    };
                    ok = tc_warp_wait(bar + B_PL, par, dead, d.spin) && tc_warp_wait(bar + B_S0, par, dead, d.spin);
                    if (!ok) break;
                    tc_fence_after();
                    states(L::G1, L::SP + 128, gk, true);
                    states(L::G1, L::SP + 64, gk, false);
                    states(L::G1, L::SP, gk, false);
                    states(L::G2, L::SP + 64, wk, true);
                    states(L::G2, L::SP, wk + 2 * L::TILE / 16, false);
                    states(L::G2, L::SP, wk, false);
                    ok = tc_warp_wait(bar + B_D1, par, dead, d.spin);
                    if (!ok) break;
                    tc_fence_after();
                    states(L::G3, L::DP + 64, rk, true);
                    states(L::G3, L::DP, rk + 2 * L::TILE / 16, false);
                    states(L::G3, L::DP, rk, false);
                    tc_commit_to(one, bar + B_G);
                    tc_commit_to(one, bar + B_DOFREE);
                }
                if (!ok) break;
                ok = tc_warp_wait(bar + B_PA, unit & 1, dead, d.spin) && tc_warp_wait(bar + B_G, (step - 1) & 1, dead, d.spin);
                if (!ok) break;
                tc_fence_after();
                // B = lower triangular [t][s]: with t its N, K step s reaches the columns from 16 ks on; with
                // s its N, K step t those up to 16 ks + 15
#pragma unroll
                for (int p = 1; p >= 0; --p) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        tc_mma_ss(one, tu + L::DQ + 16 * ks, km + 2048 * ks / 16, pk + (p * L::TILE + 16 * ks * 128 + 32 * ks) / 16,
                                  tc_idesc<false, true>(C - 16 * ks), p < 1 || ks > 0);
#pragma unroll
                    for (int ks = 3; ks >= 0; --ks)
                        tc_mma_ss(one, tu + L::DK, qm + 2048 * ks / 16, pn + (p * L::TILE + 2048 * ks) / 16, tc_idesc<true, true>(16 * ks + 16),
                                  p < 1 || ks < 3);
#pragma unroll
                    for (int ks = 3; ks >= 0; --ks)
                        tc_mma_ss(one, tu + L::DK, km + 2048 * ks / 16, an + (p * L::TILE + 2048 * ks) / 16, tc_idesc<true, true>(16 * ks + 16), true);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        tc_mma_ss(one, tu + L::DK + 16 * ks, km + 2048 * ks / 16, ak + (p * L::TILE + 16 * ks * 128 + 32 * ks) / 16,
                                  tc_idesc<false, true>(C - 16 * ks), true);
                }
                tc_commit_to(one, bar + B_DQ);
                if (hh + 1 == group) tc_commit_to(one, bar + B_TFREE);
            }
        }
        __syncwarp();
    } else {
        // ---- the loads
        unsigned it = 0, step = 0;
        unsigned boxes = 0, grads = 0;                             // started
        bool ok = true;
        for (long long i = blockIdx.x; i < items && ok; i += gridDim.x) {
            const Item x = item(i);
            if (x.nt == 0) continue;
            const int t0 = x.n * C;
            if (it > 0) ok = tc_warp_wait(bar + B_TFREE, (it - 1) & 1, dead, d.spin);
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar + B_T, 4 * L::TILE);
                for (int c = 0; c < 2; ++c) {
                    tc_tensor_load(smem + L::K + c * L::TILE, &mk, 64 * c, x.hk, t0, x.b, bar + B_T);
                    tc_tensor_load(smem + L::Q + c * L::TILE, &mq, 64 * c, x.hk, t0, x.b, bar + B_T);
                }
            }
            ++it;
            for (int hh = 0; hh < group && ok; ++hh) {
                const int h = x.hk * group + hh;
                const long long bh = (long long)x.b * d.H + h;
                for (int tl = 0; tl < tiles && ok; ++tl, ++step) {
                    if (step > 0) ok = tc_warp_wait(bar + B_DOFREE, (step - 1) & 1, dead, d.spin);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar + B_DO, 2 * L::TILE);
                        for (int c = 0; c < 2; ++c) tc_tensor_load(smem + L::G + c * L::TILE, &mg, 128 * tl + 64 * c, h, t0, x.b, bar + B_DO);
                    }
                    __syncwarp();
                    ++grads;
                    for (int e = 0; e < 8 && ok; ++e) {            // S0's four boxes, then D1's
                        const int s = e & 3;
                        if (step > 0 || e >= 4) ok = tc_warp_wait(bar + B_BFREE + s, e >= 4 ? 0 : 1, dead, d.spin);
                        if (!ok) break;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(bar + B_BOX + s, L::BOX);
                            state_load(smem + L::S + s * L::BOX, e < 4 ? &ms : &md, 128 * tl + 32 * s,
                                       (int)(e < 4 ? bh * (d.Nt + 1) + x.n : bh * d.Nt + x.n), bar + B_BOX + s);
                        }
                        __syncwarp();
                        ++boxes;
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
    CUtensorMap mq, mk, mg, ms, md, mdq, mdk;
    cudaError_t e = tc_tensor_map(&mq, in.q, d.qs, d.B, d.T, d.Hk, d.Dk);
    if (e == cudaSuccess) e = tc_tensor_map(&mk, in.k, d.ks, d.B, d.T, d.Hk, d.Dk);
    if (e == cudaSuccess) e = tc_tensor_map(&mg, o.grad, d.os, d.B, d.T, d.H, d.Dv);
    if (e == cudaSuccess) e = tc_tensor_map(&mdq, o.grad_q, ks, d.B, d.T, d.Hk, d.Dk);
    if (e == cudaSuccess) e = tc_tensor_map(&mdk, o.grad_k, ks, d.B, d.T, d.Hk, d.Dk);
    if (e == cudaSuccess) e = tc_state_map(&ms, o.snap, (long long)d.B * d.H * (d.Nt + 1), d.Dk, d.Dv);
    if (e == cudaSuccess) e = tc_state_map(&md, o.ends, (long long)d.B * d.H * d.Nt, d.Dk, d.Dv);
    if (e != cudaSuccess) return e;
    set_kernel_smem(k_delta_back_local_tc, BackLocalTc::BYTES);
    const long long items = (long long)d.B * d.Hk * d.Nt;
    k_delta_back_local_tc<<<(unsigned)(items < kRefSms ? items : kRefSms), kThreads, BackLocalTc::BYTES, st>>>(
        mq, mk, mg, ms, md, mdq, mdk, d, in, w, o);
    return cudaGetLastError();
}

}  // namespace sdm
