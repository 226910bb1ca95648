// The reverse scan of the gated delta rule's backward (notation of delta_back.cu) on the 5th-generation
// tensor cores, for bfloat16 inputs: the forward scan's mirror image (delta_scan_tc.cu). 128 of the
// state's columns are the 128 lanes of tensor memory. With X and Z = P X from k_delta_local, a chunk is
//   E = D1^T K^T;  W = (e^{L_C - L} E) X + dO^T Z;  dv = beta W
//   D0 = G_C D1 + (scale G dO)^T Q - (beta G W) K        (W is dw, all transposed; D1 after the chunk)
// D1, the decayed E, scale G dO and -beta G W are A operands in tensor memory as three bfloat16 planes
// (24 bits), dO is one in shared memory; K, Q, X and Z are B operands there, K in both its majors. A
// thread keeps its part of its lane of D in registers in float32 for the whole sequence.
//
// What bounds it: every chunk's chain E -> decayed E -> W -> its planes -> D, in two halves as in the
// forward, here with the chunk's last 32 tokens ahead. The products with dO run in the gaps. Measured at 128
// x 128: 64 heads x 64 chunks 280 us (4.4 a chunk); in registers (as delta_back.cu's for float32) 543.
//
// Warps 0..15 compute (lanes 32 (warp % 4).., quarter warp / 4 of Dk and quarter 3 - warp / 4 of the
// tokens), warp 16 issues the products, warp 17 loads, warp 18 stores the values' gradient. Two stages
// of chunk inputs. Every wait is bounded: one that gives up sets SDM_ERR_TIMEOUT in the status block, and
// the block leaves after its copies and products in flight.
#include "tcgen05.cuh"

namespace sdm {
namespace {

constexpr int kTcC = 64;
constexpr int kTcWarps = 16, kTcThreads = 32 * (kTcWarps + 3);

template <int DKP>
struct TcBack {
    static constexpr int TILE = kTcC * 128;                        // 64 columns of a token tile
    static constexpr int K = 0, Q = K + DKP / 64 * TILE, X = Q + DKP / 64 * TILE, Z = X + 3 * TILE;
    static constexpr int G = Z + 3 * TILE, STAGE = G + 2 * TILE;   // G: the readings' gradient
    static constexpr int O = 2 * STAGE, AUX = O + 2 * 2 * TILE;    // the values' gradient: two buffers
    static constexpr int AB = 3 * kTcC * 4, BARS = AUX + 2 * AB, BYTES = BARS + 256 + 1024;
    static_assert(BYTES <= 227 * 1024, "shared memory");
    // Tensor memory columns: planes of D1; planes of the decayed E, then the update; E, then in each
    // quarter's own 16 columns two planes of scale G dO, the third in GL; W, then in each quarter's own
    // columns two planes of -beta G W. Their third takes the second half of D1's third, which only E reads.
    static constexpr int SP = 0, UP = 3 * (DKP / 2), E = UP + 128, W = E + 64, GL = W + 64;
    static constexpr int LO = DKP == 128 ? SP + 160 : GL + 32;
    static_assert(GL + 64 <= 512, "tensor memory");
};

enum {
    B_FULL = 0, B_EMPTY = 2, B_OUT = 4, B_OFREE = 6,               // [stage]
    B_S = 8, B_DE = 10, B_W = 12, B_E = 14, B_WACC = 16, B_UPD = 18, // [half]
    B_GRAD = 20, B_DRAIN, B_BULK, B_COUNT = B_BULK + 2
};

// CARRY: the segments' first gradients only. SEG: the sequences are in segments (DeltaBlock).
template <int DKP, bool SEG, bool CARRY>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_delta_back_scan_tc(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                         const __grid_constant__ CUtensorMap mg, const __grid_constant__ CUtensorMap mo, DeltaDims d,
                         DeltaIn in, DeltaLocal w, DeltaBack o) {
    using L = TcBack<DKP>;
    constexpr int C = kTcC, HD = DKP / 4;                          // columns of D a thread
    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    auto bar = reinterpret_cast<unsigned long long *>(smem + L::BARS);
    volatile int *dead = reinterpret_cast<int *>(bar + B_COUNT);
    auto slot = reinterpret_cast<uint32_t *>(bar + B_COUNT + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const DeltaBlock blk = delta_block(d, in.valid, SEG, CARRY ? DELTA_CARRY_BACK : DELTA_RUN, 128);
    const int dv_blk = blk.tile * 128, seg = blk.seg;
    const long long bh = blk.bh;
    const int b = (int)(bh / d.H), h = (int)(bh % d.H), hk = h / (d.H / d.Hk);
    const int ntok = delta_valid(in.valid, b, d.T), chunks = (ntok + C - 1) / C;
    const int n0 = SEG ? delta_bound(d, chunks, seg) : 0, n1 = SEG ? delta_bound(d, chunks, seg + 1) : chunks, nch = n1 - n0;
    const bool last = !SEG || seg + 1 == d.segs;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar + B_FULL + i, 32);
            mbar_init(bar + B_EMPTY + i, kTcWarps + 1);
            mbar_init(bar + B_OUT + i, kTcWarps);
            mbar_init(bar + B_OFREE + i, 1);
        }
        for (int i = B_S; i < B_E; ++i) mbar_init(bar + i, kTcWarps / 2);
        for (int i = B_E; i < B_COUNT; ++i) mbar_init(bar + i, i == B_GRAD ? kTcWarps : 1);
        *dead = SEG && !CARRY && w.status->code != 0;              // an earlier kernel of this call gave up
        fence_mbar_init();
    }
    if (warp == kTcWarps) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *slot;

    if (warp < kTcWarps) {
        // ---- the lanes' threads
        const int part = warp >> 2, half = part >> 1, lane0 = 32 * (warp & 3), dv = dv_blk + lane0 + lane;
        const int quarter = 3 - part;                              // of the tokens
        const bool mine = dv < d.Dv;
        const uint32_t at = tm + ((uint32_t)lane0 << 16);
        const int dk0 = part * HD;
        float S[HD];
        {
            const float *end = SEG && !CARRY ? w.starts + seg * delta_states(d) : CARRY && !last ? nullptr : o.state_in;
            const float *sp = end + (bh * d.Dk + dk0) * d.Dv + dv;
#pragma unroll
            for (int i = 0; i < HD; ++i) S[i] = end && mine && dk0 + i < d.Dk ? sp[(size_t)i * d.Dv] : 0.f;
        }
        // columns [i0, i1) of D as rows of a [Dk, Dv] state
        auto keep_state = [&](float *dst, int i0, int i1) {
            dst += (dk0 + i0) * d.Dv + dv;
#pragma unroll
            for (int c = 0; c < HD; c += 16) {                     // Dk is a multiple of 16
                if (c < i0 || c >= i1 || !mine || dk0 + c >= d.Dk) continue;
#pragma unroll
                for (int i = 0; i < 16; ++i) tc_put(dst, S[c + i], d.Dv);
            }
        };
        auto planes_of_s = [&] {
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = S[c + i];
                const uint32_t dst = at + L::SP + (dk0 + c) / 2;
                tc_store_planes(dst, dst + DKP / 2, dst + DKP, x);
            }
            tc_wait_st();
        };
        auto arrive = [&](int which) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + which);
        };
        if (nch > 0) {
            planes_of_s();
            arrive(B_S + half);
        }
        // the 8 x 8 blocks of the values' gradient in its buffer: block b of a store is 8 columns of dv
        // (b % 2) and 8 tokens (b / 2), a lane's row one token
        const int orow = 16 * quarter + 8 * (lane >> 4) + (lane & 7), ocol = (lane0 >> 3) + ((lane >> 3) & 1);
        const int gcol = lane0 + lane;                             // this lane's column in dO's tiles
        for (int it = 0; it < nch; ++it) {
            const int n = n1 - 1 - it;
            const unsigned par = it & 1;
            float *keep = o.ends + (bh * d.Nt + n) * (long long)d.Dk * d.Dv;
            if (!tc_warp_wait(bar + B_FULL + par, (it >> 1) & 1, dead, d.spin)) break;
            const float *aux = reinterpret_cast<const float *>(smem + L::AUX + L::AB * par);
            const float *from = aux + 16 * quarter, *to = aux + C + 16 * quarter, *be = aux + 2 * C + 16 * quarter;
            const float whole = aux[C - 1];
            float x[16];
            if (!tc_warp_wait(bar + B_E + half, par, dead, d.spin)) break;
            tc_fence_after();
            tc_load16(at + L::E + 16 * quarter, x);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] *= to[i];
            {
                const uint32_t dst = at + L::UP + 8 * quarter;
                tc_store_planes(dst, dst + C / 2, dst + C, x);
            }
            tc_wait_st();
            arrive(B_DE + half);
            // in the products' time: scale G dO in E's place, and D1 for the chunk-local kernel
            {
                const unsigned char *gt = smem + par * L::STAGE + L::G + (gcol >> 6) * L::TILE + 2 * (gcol & 7);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    x[i] = d.scale * from[i] *
                           __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(gt + tc_at(16 * quarter + i, (gcol & 63) >> 3)));
                const uint32_t dst = at + L::E + 16 * quarter;
                tc_store_planes(dst, dst + 8, at + L::GL + 8 * quarter, x);
                tc_wait_st();
                arrive(B_GRAD);
            }
            if (!CARRY) keep_state(keep, 0, HD);
            if (!tc_warp_wait(bar + B_WACC + half, par, dead, d.spin)) break;
            if (!CARRY && it >= 2 && !tc_warp_wait(bar + B_OFREE + par, ((it >> 1) - 1) & 1, dead, d.spin)) break;
            tc_fence_after();
            // the values' gradient, in a buffer that warp 18 stores; 0 past the valid tokens
#pragma unroll
            for (int l = 0; l < (CARRY ? 0 : 2); ++l) {            // 16 lanes of dv
                float y[8];
                tc_load_frag16(at + ((uint32_t)(16 * l) << 16) + L::W + 16 * quarter, y);
                unsigned r[4];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int t = 8 * (i >> 2) + 2 * (lane & 3) + (i & 1);
                    y[i] = n * C + 16 * quarter + t < ntok ? be[t] * y[i] : 0.f;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) r[i] = pack_bf16(y[2 * i], y[2 * i + 1]);
                const int c = ocol + 2 * l;
                stsm4t(smem_u32(smem) + L::O + (2 * par + (c >> 3)) * L::TILE + tc_at(orow, c & 7), r);
            }
            if constexpr (!CARRY) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + B_OUT + par);
            }
            tc_load16(at + L::W + 16 * quarter, x);
            if (!CARRY && mine) {
                float *dst = o.w + ((bh * d.Nt + n) * (long long)C + 16 * quarter) * d.Dv + dv;
#pragma unroll
                for (int i = 0; i < 16; ++i) tc_put(dst, x[i], d.Dv);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] *= -be[i] * from[i];
            {
                const uint32_t dst = at + L::W + 16 * quarter;
                tc_store_planes(dst, dst + 8, at + L::LO + 8 * quarter, x);
            }
            tc_wait_st();
            arrive(B_W + half);
            if (!tc_warp_wait(bar + B_UPD + half, par, dead, d.spin)) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
                tc_load16(at + L::UP + dk0 + c, x);
#pragma unroll
                for (int i = 0; i < 16; ++i) S[c + i] = fmaf(whole, S[c + i], x[i]);
            }
            if (it + 1 < nch) planes_of_s();
            arrive(B_S + half);
            if (lane == 0) mbar_arrive(bar + B_EMPTY + par);
        }
        if (CARRY)
            keep_state(w.starts + (seg - 1) * delta_states(d) + bh * d.Dk * (long long)d.Dv, 0, HD);
        else if (seg == 0 && !*dead)
            keep_state(o.state_out + bh * d.Dk * (long long)d.Dv, 0, HD);
    } else if (warp == kTcWarps) {
        // ---- the products
        const uint32_t one = tc_elect(), tu = __shfl_sync(~0u, tm, 0), base = __shfl_sync(~0u, smem_u32(smem), 0);
        for (int it = 0; it < nch; ++it) {
            const unsigned par = it & 1;
            const uint32_t st = base + par * L::STAGE;
            // a descriptor's address counts 16 bytes
            const uint32_t kd = tc_k_major(st + L::K), xn = tc_n_major(st + L::X, L::TILE), zn = tc_n_major(st + L::Z, L::TILE);
            const uint32_t kn = tc_n_major(st + L::K, L::TILE), qn = tc_n_major(st + L::Q, L::TILE), gm = tc_n_major(st + L::G, L::TILE);
            constexpr int KS = DKP / 16;
            auto rows = [&](int t0, int tokens, int p, int ks, bool add) {
                tc_mma_ts(one, tu + L::E + t0, tu + L::SP + p * (DKP / 2) + 8 * ks, kd + (t0 * 128 + (ks >> 2) * L::TILE + 32 * (ks & 3)) / 16,
                          tc_idesc<false>(tokens), add);
            };
            // K step ks (tokens 16 ks ..) of a lower triangular B reaches the columns up to 16 ks + 15
            auto tri = [&](uint32_t a, uint32_t tile, int ks) {
                tc_mma_ts(one, tu + L::W, tu + a + 8 * ks, tile + 2048 * ks / 16, tc_idesc<true>(16 * ks + 16), true);
            };
            constexpr int N = DKP == 128 ? 64 : DKP;
            auto update = [&](int ks, int hd, int p, uint32_t tile, uint32_t two, uint32_t third, bool add) {
                tc_mma_ts(one, tu + L::UP + 64 * hd, tu + (p < 2 ? two + 16 * ks + 8 * p : third + 8 * ks),
                          tile + (2048 * ks + hd * L::TILE) / 16, tc_idesc<true>(N), add);
            };
            if (!tc_warp_wait(bar + B_FULL + par, (it >> 1) & 1, dead, d.spin)) break;
            if (!tc_warp_wait(bar + B_S, par, dead, d.spin)) break;
            tc_fence_after();
            // D1's largest terms wait for the second half of Dk: the lesser ones of both come first (268 us without,
            // and the log-decays' gradients up to 1.1e-6 off instead of 7e-7)
#pragma unroll
            for (int p = 2; p >= 1; --p)
#pragma unroll
                for (int ks = 0; ks < KS / 2; ++ks) rows(0, C, p, ks, p < 2 || ks > 0);
            if (!tc_warp_wait(bar + B_S + 1, par, dead, d.spin)) break;
            tc_fence_after();
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                for (int p = 2; p >= 0; --p)
#pragma unroll
                    for (int ks = p > 0 ? KS / 2 : 0; ks < KS; ++ks) rows(32 - 32 * hf, 32, p, ks, true);
                tc_commit_to(one, bar + B_E + hf);
            }
            // sums from their smallest terms up: the tensor core cuts an accumulator's low bits at every step
            auto grads = [&](int p, int ks, bool add) {
                tc_mma_ss(one, tu + L::W, gm + 2048 * ks / 16, zn + (p * L::TILE + 2048 * ks) / 16, tc_idesc<true, true>(16 * ks + 16), add);
            };
#pragma unroll
            for (int p = 2; p >= 1; --p)
#pragma unroll
                for (int ks = C / 16 - 1; ks >= 0; --ks) grads(p, ks, p < 2 || ks < C / 16 - 1);
            bool ok = true;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                ok = ok && tc_warp_wait(bar + B_DE + hf, par, dead, d.spin);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int sum = 2; sum >= 0; --sum)
#pragma unroll
                    for (int a = sum; a >= 0; --a)
#pragma unroll
                        for (int ks = 3 - 2 * hf; ks >= 2 - 2 * hf; --ks) tri(L::UP + a * (C / 2), xn + (sum - a) * L::TILE / 16, ks);
#pragma unroll
                for (int ks = 3 - 2 * hf; ks >= 2 - 2 * hf; --ks) grads(0, ks, true);
                tc_commit_to(one, bar + B_WACC + hf);
            }
            if (!ok) break;
            if (!tc_warp_wait(bar + B_GRAD, par, dead, d.spin)) break;
            if (!tc_warp_wait(bar + B_WACC + 1, par, dead, d.spin)) break;   // the decayed E makes room for the update
            tc_fence_after();
#pragma unroll
            for (int p = 2; p >= 1; --p)
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks)
#pragma unroll
                    for (int hd = 0; hd < DKP / 64; ++hd) update(ks, hd, p, qn, L::E, L::GL, p < 2 || ks > 0);
            if (!tc_warp_wait(bar + B_W, par, dead, d.spin)) break;
            tc_fence_after();
#pragma unroll
            for (int p = 2; p >= 1; --p)
#pragma unroll
                for (int hd = 0; hd < DKP / 64; ++hd) {
                    update(3, hd, p, kn, L::W, L::LO, true);
                    update(2, hd, p, kn, L::W, L::LO, true);
                }
            if (!tc_warp_wait(bar + B_W + 1, par, dead, d.spin)) break;
            tc_fence_after();
#pragma unroll
            for (int hd = 0; hd < DKP / 64; ++hd) {
#pragma unroll
                for (int p = 2; p >= 1; --p) {
                    update(1, hd, p, kn, L::W, L::LO, true);
                    update(0, hd, p, kn, L::W, L::LO, true);
                }
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks) {
                    update(ks, hd, 0, kn, L::W, L::LO, true);
                    update(ks, hd, 0, qn, L::E, L::GL, true);
                }
                tc_commit_to(one, bar + B_UPD + hd);
            }
            if (DKP == 64) tc_commit_to(one, bar + B_UPD + 1);
            tc_commit_to(one, bar + B_EMPTY + par);
        }
        __syncwarp();
    } else if (warp == kTcWarps + 1) {
        // ---- the chunks' inputs
        for (int it = 0; it < nch; ++it) {
            const int n = n1 - 1 - it, s = it & 1, t0 = n * C, nt = ntok - t0 < C ? ntok - t0 : C;
            unsigned char *st = smem + s * L::STAGE;
            const long long bhn = bh * d.Nt + n;
            unsigned long long *full = bar + B_BULK + s;
            if (it >= 2 && !tc_warp_wait(bar + B_EMPTY + s, ((it >> 1) - 1) & 1, dead, d.spin)) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(full, L::STAGE + L::AB);
                for (int c = 0; c < DKP / 64; ++c) {
                    tc_tensor_load(st + L::K + c * L::TILE, &mk, 64 * c, tc_coord(d.ks[2], hk), t0, tc_coord(d.ks[0], b), full);
                    tc_tensor_load(st + L::Q + c * L::TILE, &mq, 64 * c, tc_coord(d.qs[2], hk), t0, tc_coord(d.qs[0], b), full);
                }
                for (int c = 0; c < 2; ++c) tc_tensor_load(st + L::G + c * L::TILE, &mg, dv_blk + 64 * c, tc_coord(d.os[2], h), t0, tc_coord(d.os[0], b), full);
                bulk_g2s(st + L::X, w.x + bhn * (3 * L::TILE), 3 * L::TILE, full);
                bulk_g2s(st + L::Z, w.p + bhn * (3 * L::TILE), 3 * L::TILE, full);
                bulk_g2s(smem + L::AUX + L::AB * s, w.aux + bhn * kDeltaAux * C, L::AB, full);
            }
            __syncwarp();
            if (!tc_warp_wait(full, (it >> 1) & 1, dead, d.spin)) {
                mbar_wait_bounded(full, (it >> 1) & 1);            // nothing in flight behind a give-up
                break;
            }
            if (nt < C) {                                          // what lies past the valid tokens is not used
                const int rows = C - nt;
                for (int i = lane; i < rows * 8; i += 32) {
                    const int off = tc_at(nt + (i >> 3), i & 7);
                    for (int c = 0; c < DKP / 64; ++c) {
                        *reinterpret_cast<uint4 *>(st + L::K + c * L::TILE + off) = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4 *>(st + L::Q + c * L::TILE + off) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    for (int c = 0; c < 2; ++c) *reinterpret_cast<uint4 *>(st + L::G + c * L::TILE + off) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
            }
            mbar_arrive(bar + B_FULL + s);
        }
    } else if (!CARRY) {
        // ---- the values' gradient
        for (int it = 0; it < nch; ++it) {
            if (!tc_warp_wait(bar + B_OUT + (it & 1), (it >> 1) & 1, dead, d.spin)) break;
            if (lane == 0) {
                for (int c = 0; c < 2; ++c)
                    if (dv_blk + 64 * c < d.Dv)
                        tc_tensor_store(&mo, dv_blk + 64 * c, h, (n1 - 1 - it) * C, b, smem + L::O + (2 * (it & 1) + c) * L::TILE);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                mbar_arrive(bar + B_OFREE + (it & 1));
            }
            __syncwarp();
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        const int cols = d.Dv - dv_blk < 128 ? d.Dv - dv_blk : 128;
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(o.grad_v) + ((long long)b * d.T * d.H + h) * d.Dv + dv_blk;
        for (long long t = (long long)chunks * C + (lane >> 4); last && t < d.T; t += 2)
            if ((lane & 15) * 8 < cols) *reinterpret_cast<uint4 *>(out + t * d.H * d.Dv + (lane & 15) * 8) = make_uint4(0u, 0u, 0u, 0u);
    }
    __syncthreads();
    if (*dead) {
        // the products issued so far are waited for (the copies were, by their own warps)
        if (tid == 32 * kTcWarps) {
            tc_commit_to(1, bar + B_DRAIN);
            mbar_wait_bounded(bar + B_DRAIN, 0);
            atomicCAS(&w.status->code, 0, (int)SDM_ERR_TIMEOUT);
        }
        __syncthreads();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kTcWarps) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512));
}

template <int DKP>
cudaError_t back_scan_tc(const DeltaDims &d, const DeltaIn &in, const DeltaLocal &w, const DeltaBack &o, cudaStream_t st) {
    const long long os[3] = {(long long)d.T * d.H * d.Dv, (long long)d.H * d.Dv, d.Dv};
    CUtensorMap mq, mk, mg, mo;
    cudaError_t e = tc_tensor_map(&mq, in.q, d.qs, d.B, d.T, d.Hk, d.Dk);
    if (e == cudaSuccess) e = tc_tensor_map(&mk, in.k, d.ks, d.B, d.T, d.Hk, d.Dk);
    if (e == cudaSuccess) e = tc_tensor_map(&mg, o.grad, d.os, d.B, d.T, d.H, d.Dv);
    if (e == cudaSuccess) e = tc_tensor_map(&mo, o.grad_v, os, d.B, d.T, d.H, d.Dv);
    if (e != cudaSuccess) return e;
    auto run = [&](auto kern, int mode) {
        set_kernel_smem(kern, TcBack<DKP>::BYTES);
        kern<<<(unsigned)delta_blocks(d, mode, 128), kTcThreads, TcBack<DKP>::BYTES, st>>>(mq, mk, mg, mo, d, in, w, o);
        return cudaGetLastError();
    };
    if (d.segs == 1) return run(k_delta_back_scan_tc<DKP, false, false>, DELTA_RUN);
    e = run(k_delta_back_scan_tc<DKP, true, true>, DELTA_CARRY_BACK);
    if (e == cudaSuccess) e = launch_delta_join(d, w, o.state_in, true, st);
    return e == cudaSuccess ? run(k_delta_back_scan_tc<DKP, true, false>, DELTA_RUN) : e;
}

}  // namespace

cudaError_t launch_delta_back_scan_tc(const DeltaDims &d, const DeltaIn &in, const DeltaLocal &w, const DeltaBack &o,
                                      cudaStream_t st) {
    return d.Dk <= 64 ? back_scan_tc<64>(d, in, w, o, st) : back_scan_tc<128>(d, in, w, o, st);
}

}  // namespace sdm
