// The gated delta rule's scan over a head's chunks (notation of delta_chunk.cu) on the 5th-generation
// tensor cores, for bfloat16 inputs. As in the register form everything is transposed: 128 of the
// state's columns are the 128 lanes of tensor memory, and S^T, w^T and u^T are A operands there, as
// bfloat16 planes that their own lanes' threads store; K, Q, X and P are the B operands in shared
// memory, K with both its majors (K S has Dk along K, the state's update has the tokens along K).
//   R = S^T K^T  (3 planes)          O1 = S^T Q^T (2)
//   w = beta (v - G R);  U = w^T X^T (3 x 3, terms below 2^-24 left out)
//   S += (e^{L_C - L} u)^T K (3)     O2 = u^T P^T (2 x 2)
// A thread keeps its lane's half of S in registers in float32 for the whole sequence; the tensor core
// only ever sums one chunk's update.
//
// What bounds it: the chain R -> w -> U -> u -> update -> S of every chunk, products (768, 480 and 768
// cycles at Dk = 128) and the threads' work between them in turn; O1, O2 and the readings run beside it.
//
// Warps 0..7 compute (lanes 32 (warp % 4).., column half warp / 4), warp 8 issues the products, warps 9
// and 10 copy. Two stages of chunk inputs. Every wait is bounded: one that gives up sets
// SDM_ERR_TIMEOUT in the status block, and the block leaves after its copies and products in flight.
#include "tcgen05.cuh"

namespace sdm {
namespace {

constexpr int kTcC = 64;
constexpr int kTcCompute = 256, kTcCopy = 64, kTcThreads = kTcCompute + 32 + kTcCopy;

template <int DKP>
struct TcScan {
    static constexpr int TILE = kTcC * 128;                        // 64 columns of a token tile
    static constexpr int K = 0, Q = K + DKP / 64 * TILE, X = Q + DKP / 64 * TILE, P = X + 3 * TILE;
    static constexpr int VP = 128 * 2 + 16;                        // row pitch of the value tile
    static constexpr int V = P + 2 * TILE, AUX = V + kTcC * VP, STAGE = AUX + 1024;
    static constexpr int BARS = 2 * STAGE, BYTES = BARS + 256 + 1024;
    static_assert(AUX % 1024 == 0 && BYTES <= 227 * 1024, "shared memory");
    // tensor memory columns: planes of S (after R and O1: of u), the update (before it: O1), R (then U,
    // then O2), planes of w (then of the decayed u)
    static constexpr int SP = 0, UP = 3 * (DKP / 2), R = UP + (DKP < 128 ? 64 : DKP), WP = R + 64;
    static_assert(WP + 96 <= 512, "tensor memory");
};

enum { B_FULL = 0, B_EMPTY = 2, B_S = 4, B_W, B_U, B_R, B_O1, B_UACC, B_UPD, B_O2, B_DRAIN, B_BULK, B_COUNT = B_BULK + 2 };

template <int DKP, bool SAVE>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_delta_scan_tc(DeltaDims d, DeltaIn in, DeltaLocal w, float *state, __nv_bfloat16 *o, float *snap,
                    float *usave) {
    using L = TcScan<DKP>;
    constexpr int C = kTcC, HD = DKP / 2;                          // columns of S a thread
    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    auto bar = reinterpret_cast<unsigned long long *>(smem + L::BARS);
    volatile int *dead = reinterpret_cast<int *>(bar + B_COUNT);
    auto slot = reinterpret_cast<uint32_t *>(bar + B_COUNT + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tiles = (d.Dv + 127) / 128, dv_blk = (blockIdx.x % tiles) * 128;
    const long long bh = blockIdx.x / tiles;
    const int b = (int)(bh / d.H), h = (int)(bh % d.H), hk = h / (d.H / d.Hk);
    const int ntok = delta_valid(in.valid, b, d.T), nch = (ntok + C - 1) / C;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar + B_FULL + i, kTcCopy);
            mbar_init(bar + B_EMPTY + i, 8 + 1);
        }
        for (int i = B_S; i <= B_U; ++i) mbar_init(bar + i, 8);
        for (int i = B_R; i < B_COUNT; ++i) mbar_init(bar + i, 1);
        *dead = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *slot;

    if (warp < 8) {
        // ---- the lanes' threads
        const int half = warp >> 2, dv = dv_blk + 32 * (warp & 3) + lane;
        const bool mine = dv < d.Dv;
        const uint32_t at = tm + ((uint32_t)(32 * (warp & 3)) << 16);
        const int dk0 = half * HD;
        float S[HD];
        float *sp = state + (bh * d.Dk + dk0) * d.Dv + dv;
#pragma unroll
        for (int i = 0; i < HD; ++i) S[i] = mine && dk0 + i < d.Dk ? sp[(size_t)i * d.Dv] : 0.f;
        auto keep_state = [&](float *dst) {
#pragma unroll
            for (int i = 0; i < HD; ++i)
                if (mine && dk0 + i < d.Dk) dst[(size_t)(dk0 + i) * d.Dv + dv] = S[i];
        };
        auto planes_of_s = [&] {
#pragma unroll
            for (int c = 0; c < HD; c += 32) {
                float x[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = S[c + i];
                tc_store_planes<3>(at + L::SP + half * (HD / 2) + c / 2, DKP / 2, x);
            }
        };
        auto hand_over = [&](int which) {                          // tensor memory stores -> the products
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + which);
        };
        if (nch > 0) {
            planes_of_s();
            hand_over(B_S);
        }
        __nv_bfloat16 *out = o + ((long long)b * d.T * d.H + h) * d.Dv + dv;
        const long long orow = (long long)d.H * d.Dv;
        for (int n = 0; n < nch; ++n) {
            const unsigned par = n & 1;
            const unsigned char *st = smem + par * L::STAGE;
            if (SAVE) keep_state(snap + ((bh * d.Nt + n) * (long long)d.Dk) * d.Dv);
            if (!tc_warp_wait(bar + B_FULL + par, (n >> 1) & 1, dead, d.spin)) break;
            const float *from = reinterpret_cast<const float *>(st + L::AUX) + 32 * half, *to = from + C, *be = to + C;
            const float whole = reinterpret_cast<const float *>(st + L::AUX)[C - 1];
            const unsigned char *vp = st + L::V + 32 * half * L::VP + 2 * (32 * (warp & 3) + lane);
            float x[32];
            if (!tc_warp_wait(bar + B_R, par, dead, d.spin)) break;
            tc_fence_after();
            tc_load32(at + L::R + 32 * half, x);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float v = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(vp + i * L::VP));
                x[i] = be[i] * (v - from[i] * x[i]);
            }
            tc_store_planes<3>(at + L::WP + 16 * half, C / 2, x);
            hand_over(B_W);
            float y[32];
            if (!tc_warp_wait(bar + B_O1, par, dead, d.spin)) break;
            tc_fence_after();
            tc_load32(at + L::UP + 32 * half, y);
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] *= d.scale * from[i];
            if (!tc_warp_wait(bar + B_UACC, par, dead, d.spin)) break;
            tc_fence_after();
            tc_load32(at + L::R + 32 * half, x);
            if (SAVE && mine) {
                float *dst = usave + ((bh * d.Nt + n) * (long long)C + 32 * half) * d.Dv + dv;
#pragma unroll
                for (int i = 0; i < 32; ++i) dst[(size_t)i * d.Dv] = x[i];
            }
            tc_store_planes<2>(at + L::SP + 16 * half, C / 2, x);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] *= to[i];
            tc_store_planes<3>(at + L::WP + 16 * half, C / 2, x);
            hand_over(B_U);
            if (!tc_warp_wait(bar + B_UPD, par, dead, d.spin)) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < HD; c += 32) {
                tc_load32(at + L::UP + dk0 + c, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) S[c + i] = fmaf(whole, S[c + i], x[i]);
            }
            if (!tc_warp_wait(bar + B_O2, par, dead, d.spin)) break;
            tc_fence_after();
            tc_load32(at + L::R + 32 * half, x);
            if (n + 1 < nch) planes_of_s();
            hand_over(B_S);
            if (lane == 0) mbar_arrive(bar + B_EMPTY + par);
            const long long t0 = (long long)n * C + 32 * half;
            if (mine) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (t0 + i < d.T) out[(t0 + i) * orow] = __float2bfloat16_rn(t0 + i < ntok ? x[i] + y[i] : 0.f);
            }
        }
        if (nch > 0 && !*dead) keep_state(state + bh * d.Dk * (long long)d.Dv);
        if (mine)
            for (long long t = (long long)nch * C + half; t < d.T; t += 2) out[t * orow] = __float2bfloat16_rn(0.f);
    } else if (warp == 8) {
        // ---- the products, one thread
        if (lane == 0) {
            for (int n = 0; n < nch; ++n) {
                const unsigned par = n & 1;
                const uint32_t st = smem_u32(smem) + par * L::STAGE;
                if (!tc_wait(bar + B_FULL + par, (n >> 1) & 1, dead, d.spin)) break;
                if (!tc_wait(bar + B_S, par, dead, d.spin)) break;
                tc_fence_after();
                for (int p = 2; p >= 0; --p)
                    for (int ks = 0; ks < DKP / 16; ++ks)
                        tc_mma_ts(tm + L::R, tm + L::SP + p * (DKP / 2) + 8 * ks,
                                  tc_k_major(st + L::K + (ks >> 2) * L::TILE + 32 * (ks & 3)), tc_idesc<false>(C), p < 2 || ks > 0);
                tc_commit_to(bar + B_R);
                for (int p = 1; p >= 0; --p)
                    for (int ks = 0; ks < DKP / 16; ++ks)
                        tc_mma_ts(tm + L::UP, tm + L::SP + p * (DKP / 2) + 8 * ks,
                                  tc_k_major(st + L::Q + (ks >> 2) * L::TILE + 32 * (ks & 3)), tc_idesc<false>(C), p < 1 || ks > 0);
                tc_commit_to(bar + B_O1);
                // lower triangular: K step ks reaches the columns from 16 ks on
                auto triangle = [&](uint32_t dst, uint32_t a, uint32_t tile, bool first) {
                    for (int ks = 0; ks < C / 16; ++ks)
                        tc_mma_ts(dst + 16 * ks, a + 8 * ks, tc_k_major(tile + 16 * ks * 128 + 32 * ks), tc_idesc<false>(C - 16 * ks),
                                  !first || ks > 0);
                };
                if (!tc_wait(bar + B_W, par, dead, d.spin)) break;
                tc_fence_after();
                for (int a = 2; a >= 0; --a)
                    for (int p = 2 - a; p >= 0; --p)
                        triangle(tm + L::R, tm + L::WP + a * (C / 2), st + L::X + p * L::TILE, a == 2 && p == 0);
                tc_commit_to(bar + B_UACC);
                if (!tc_wait(bar + B_U, par, dead, d.spin)) break;
                tc_fence_after();
                for (int p = 2; p >= 0; --p)
                    for (int ks = 0; ks < C / 16; ++ks)
                        tc_mma_ts(tm + L::UP, tm + L::WP + p * (C / 2) + 8 * ks, tc_n_major(st + L::K + 2048 * ks, L::TILE),
                                  tc_idesc<true>(DKP), p < 2 || ks > 0);
                tc_commit_to(bar + B_UPD);
                for (int a = 1; a >= 0; --a)
                    for (int p = 1 - a; p >= 0; --p)
                        triangle(tm + L::R, tm + L::SP + a * (C / 2), st + L::P + p * L::TILE, a == 1 && p == 0);
                tc_commit_to(bar + B_O2);
                tc_commit_to(bar + B_EMPTY + par);
            }
        }
        __syncwarp();
    } else {
        // ---- the copies
        const int ct = tid - kTcCompute - 32;
        const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(in.k) + b * d.ks[0] + hk * d.ks[2];
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(in.q) + b * d.qs[0] + hk * d.qs[2];
        const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(in.v) + b * d.vs[0] + h * d.vs[2] + dv_blk;
        for (int n = 0; n < nch; ++n) {
            const int s = n & 1;
            unsigned char *st = smem + s * L::STAGE;
            const uint32_t sa = smem_u32(st);
            if (n >= 2 && !tc_wait(bar + B_EMPTY + s, ((n >> 1) - 1) & 1, dead, d.spin)) break;
            const long long t0 = (long long)n * C, bhn = bh * d.Nt + n;
            const int nt = ntok - (int)t0 < C ? ntok - (int)t0 : C;
            if (ct == 0) {
                mbar_arrive_expect_tx(bar + B_BULK + s, 5 * L::TILE + 3 * C * 4);
                bulk_g2s(st + L::X, w.x + bhn * (3 * L::TILE), 3 * L::TILE, bar + B_BULK + s);
                bulk_g2s(st + L::P, w.p + bhn * (2 * L::TILE), 2 * L::TILE, bar + B_BULK + s);
                bulk_g2s(st + L::AUX, w.aux + bhn * 3 * C, 3 * C * 4, bar + B_BULK + s);
            }
            constexpr int PC = DKP / 8;
#pragma unroll 4
            for (int i = ct; i < C * PC; i += kTcCopy) {
                const int c = i % PC, r = i / PC, dst = (c >> 3) * L::TILE + tc_at(r, c & 7);
                const bool live = r < nt && c * 8 < d.Dk;
                cp_async16_zfill(sa + L::K + dst, live ? k + (t0 + r) * d.ks[1] + c * 8 : k, live);
                cp_async16_zfill(sa + L::Q + dst, live ? q + (t0 + r) * d.qs[1] + c * 8 : q, live);
            }
#pragma unroll 4
            for (int i = ct; i < C * 16; i += kTcCopy) {
                const int c = i % 16, r = i / 16;
                const bool live = r < nt && dv_blk + c * 8 < d.Dv;
                cp_async16_zfill(sa + L::V + r * L::VP + c * 16, live ? v + (t0 + r) * d.vs[1] + c * 8 : v, live);
            }
            cp_async_commit();
            cp_async_wait<0>();
            if (ct == 0 && !tc_wait(bar + B_BULK + s, (n >> 1) & 1, dead, d.spin)) {
                mbar_wait_bounded(bar + B_BULK + s, (n >> 1) & 1);    // nothing in flight behind a give-up
                break;
            }
            fence_proxy_async_smem();                              // the tiles, before the tensor core reads them
            mbar_arrive(bar + B_FULL + s);
        }
    }
    __syncthreads();
    if (*dead) {
        // the products issued so far are waited for (the copies were, by their own thread)
        if (tid == kTcCompute) {
            tc_commit_to(bar + B_DRAIN);
            mbar_wait_bounded(bar + B_DRAIN, 0);
            atomicCAS(&w.status->code, 0, (int)SDM_ERR_TIMEOUT);
        }
        __syncthreads();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512));
}

template <int DKP, bool SAVE>
cudaError_t scan_tc(const DeltaDims &d, const DeltaIn &in, const DeltaLocal &w, float *state, void *o, float *snap,
                    float *u, cudaStream_t st) {
    auto kern = k_delta_scan_tc<DKP, SAVE>;
    set_kernel_smem(kern, TcScan<DKP>::BYTES);
    kern<<<(unsigned)((long long)d.B * d.H * ((d.Dv + 127) / 128)), kTcThreads, TcScan<DKP>::BYTES, st>>>(
        d, in, w, state, static_cast<__nv_bfloat16 *>(o), snap, u);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_scan_tc(const DeltaDims &d, const DeltaIn &in, const DeltaLocal &w, float *state, void *o,
                                 float *snap, float *u, cudaStream_t st) {
    if (d.Dk <= 64)
        return snap ? scan_tc<64, true>(d, in, w, state, o, snap, u, st)
                    : scan_tc<64, false>(d, in, w, state, o, snap, u, st);
    return snap ? scan_tc<128, true>(d, in, w, state, o, snap, u, st)
                : scan_tc<128, false>(d, in, w, state, o, snap, u, st);
}

}  // namespace sdm
