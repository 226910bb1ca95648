// The gated delta rule's scan over a head's chunks (notation of delta_chunk.cu) on the 5th-generation
// tensor cores, for bfloat16 inputs. As in the register form everything is transposed: 128 of the
// state's columns are the 128 lanes of tensor memory. With Y = X diag(beta) and Z = P Y from
// k_delta_local, a chunk is
//   R = S^T K^T;  w = -G R;  U = V^T Y^T + w Y^T;  S = G_C S + (e^{L_C - L} U) K
//   o = scale G (S^T Q^T) + V^T Z^T + w Z^T                 (all transposed; S before the chunk)
// S, w and the decayed U are A operands in tensor memory, as bfloat16 planes that their own lanes'
// threads store; V is an A operand in shared memory; K, Q, Y and Z are B operands there, K in both its
// majors (K S runs over Dk, the state's update over the tokens). Three planes (24 bits) go into R, U
// and the update, two into the bfloat16 readings. A thread keeps its part of its lane of S in registers
// in float32 for the whole sequence; the tensor core only ever sums one chunk's update.
//
// What bounds it: every chunk's chain R -> w -> U -> update -> S, products and the threads' work in
// turn; the values' products and the readings run in its gaps.
//
// Warps 0..15 compute (lanes 32 (warp % 4).., column quarter warp / 4), warp 16 issues the products,
// warps 17..20 copy (a thread a 16-byte column, so that its addresses only step). Two stages of chunk inputs. Every wait is bounded: one that gives up sets
// SDM_ERR_TIMEOUT in the status block, and the block leaves after its copies and products in flight.
#include "tcgen05.cuh"

namespace sdm {
namespace {

constexpr int kTcC = 64;
constexpr int kTcWarps = 16, kTcCopy = 128, kTcThreads = 32 * kTcWarps + 32 + kTcCopy;

template <int DKP>
struct TcScan {
    static constexpr int TILE = kTcC * 128;                        // 64 columns of a token tile
    static constexpr int K = 0, Q = K + DKP / 64 * TILE, Y = Q + DKP / 64 * TILE, Z = Y + 3 * TILE;
    static constexpr int V = Z + 2 * TILE, STAGE = V + 2 * TILE;
    static constexpr int AUX = 2 * STAGE, BARS = AUX + 2 * 512, BYTES = BARS + 256 + 1024;
    static_assert(BYTES <= 227 * 1024, "shared memory");
    // Tensor memory columns: planes of S (once they are used: of the decayed U), planes of w (then the
    // update), R (then S^T Q^T), U, the readings' rest
    static constexpr int SP = 0, UP = 3 * (DKP / 2), R = UP + 128, U = R + 64, O = U + 64;
    static_assert(O + 64 <= 512, "tensor memory");
};

enum { B_FULL = 0, B_EMPTY = 2, B_S = 4, B_W, B_U, B_READ, B_R, B_O1, B_UACC, B_O2, B_UPD, B_DRAIN, B_BULK, B_COUNT = B_BULK + 2 };

template <int DKP, bool SAVE>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_delta_scan_tc(DeltaDims d, DeltaIn in, DeltaLocal w, float *state, __nv_bfloat16 *o, float *snap,
                    float *usave) {
    using L = TcScan<DKP>;
    constexpr int C = kTcC, HD = DKP / 4;                          // columns of S a thread
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
            mbar_init(bar + B_EMPTY + i, kTcWarps + 1);
        }
        for (int i = B_S; i <= B_READ; ++i) mbar_init(bar + i, kTcWarps);
        for (int i = B_R; i < B_COUNT; ++i) mbar_init(bar + i, 1);
        *dead = 0;
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
        const int part = warp >> 2, lane0 = 32 * (warp & 3), dv = dv_blk + lane0 + lane;
        const bool mine = dv < d.Dv;
        const uint32_t at = tm + ((uint32_t)lane0 << 16);
        const int dk0 = part * HD;
        float S[HD];
        {
            const float *sp = state + (bh * d.Dk + dk0) * d.Dv + dv;
#pragma unroll
            for (int i = 0; i < HD; ++i) S[i] = mine && dk0 + i < d.Dk ? sp[(size_t)i * d.Dv] : 0.f;
        }
        auto keep_state = [&](float *dst) {
            dst += (size_t)dk0 * d.Dv + dv;
#pragma unroll
            for (int i = 0; i < HD; ++i)
                if (mine && dk0 + i < d.Dk) dst[(size_t)i * d.Dv] = S[i];
        };
        auto planes_of_s = [&] {
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = S[c + i];
                tc_store_planes<3>(at + L::SP + (dk0 + c) / 2, DKP / 2, x);
            }
        };
        auto arrive = [&](int which) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + which);
        };
        if (nch > 0) {
            planes_of_s();
            tc_wait_st();
            arrive(B_S);
        }
        // the readings' 8 x 8 blocks in the value tile: block b of a store is 8 columns of dv (b % 2) and
        // 8 tokens (b / 2), a lane's row one token
        const int orow = 16 * part + 8 * (lane >> 4) + (lane & 7), ocol = (lane0 >> 3) + ((lane >> 3) & 1);
        for (int n = 0; n < nch; ++n) {
            const unsigned par = n & 1;
            if (SAVE) keep_state(snap + ((bh * d.Nt + n) * (long long)d.Dk) * d.Dv);
            if (!tc_warp_wait(bar + B_FULL + par, (n >> 1) & 1, dead, d.spin)) break;
            const float *aux = reinterpret_cast<const float *>(smem + L::AUX + 512 * par);
            const float *from = aux + 16 * part, *to = aux + C + 16 * part;
            const float whole = aux[C - 1];
            float x[16], y[2][8];
            if (!tc_warp_wait(bar + B_R, par, dead, d.spin)) break;
            tc_fence_after();
            tc_load16(at + L::R + 16 * part, x);
            arrive(B_READ);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] *= -from[i];
            tc_store_planes<3>(at + L::UP + 8 * part, C / 2, x);
            tc_wait_st();
            arrive(B_W);
            if (!tc_warp_wait(bar + B_O1, par, dead, d.spin)) break;
            tc_fence_after();
            tc_load_frag16(at + L::R + 16 * part, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = d.scale * from[8 * (i >> 2) + 2 * (lane & 3) + (i & 1)];
                y[0][i] *= f;
                y[1][i] *= f;
            }
            if (!tc_warp_wait(bar + B_UACC, par, dead, d.spin)) break;
            tc_fence_after();
            tc_load16(at + L::U + 16 * part, x);
            if (SAVE && mine) {
                float *dst = usave + ((bh * d.Nt + n) * (long long)C + 16 * part) * d.Dv + dv;
#pragma unroll
                for (int i = 0; i < 16; ++i) dst[(size_t)i * d.Dv] = x[i];
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] *= to[i];
            tc_store_planes<3>(at + L::SP + 8 * part, C / 2, x);
            tc_wait_st();
            arrive(B_U);
            // the readings, in the values' place; the copying warps store them as rows
            if (!tc_warp_wait(bar + B_O2, par, dead, d.spin)) break;
            tc_fence_after();
            {
                float z[2][8];
                tc_load_frag16(at + L::O + 16 * part, z);
                unsigned char *vt = smem + par * L::STAGE + L::V;
#pragma unroll
                for (int l = 0; l < 2; ++l) {
                    unsigned r[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[i] = pack_bf16(y[l][2 * i] + z[l][2 * i], y[l][2 * i + 1] + z[l][2 * i + 1]);
                    const int c = ocol + 2 * l;
                    stsm4t(smem_u32(vt) + (c >> 3) * L::TILE + tc_at(orow, c & 7), r);
                }
            }
            if (!tc_warp_wait(bar + B_UPD, par, dead, d.spin)) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
                tc_load16(at + L::UP + dk0 + c, x);
#pragma unroll
                for (int i = 0; i < 16; ++i) S[c + i] = fmaf(whole, S[c + i], x[i]);
            }
            if (n + 1 < nch) planes_of_s();
            tc_wait_st();
            arrive(B_S);
            if (lane == 0) mbar_arrive(bar + B_EMPTY + par);
        }
        if (nch > 0 && !*dead) keep_state(state + bh * d.Dk * (long long)d.Dv);
    } else if (warp == kTcWarps) {
        // ---- the products
        {
            const uint32_t one = tc_elect(), tu = __shfl_sync(~0u, tm, 0), base = __shfl_sync(~0u, smem_u32(smem), 0);
            for (int n = 0; n < nch; ++n) {
                const unsigned par = n & 1;
                const uint32_t st = base + par * L::STAGE;
                const uint64_t kd = tc_k_major(st + L::K), qd = tc_k_major(st + L::Q), yd = tc_k_major(st + L::Y),
                               zd = tc_k_major(st + L::Z), kn = tc_n_major(st + L::K, L::TILE), vm = tc_n_major(st + L::V, L::TILE);
                // lower triangular B: K step ks reaches the columns from 16 ks on. A descriptor's address
                // counts 16 bytes.
                auto tri_ts = [&](uint32_t dst, uint32_t a, uint64_t tile) {
#pragma unroll
                    for (int ks = 0; ks < C / 16; ++ks)
                        tc_mma_ts(one, tu + dst + 16 * ks, tu + a + 8 * ks, tile + (16 * ks * 128 + 32 * ks) / 16, tc_idesc<false>(C - 16 * ks), true);
                };
                auto tri_ss = [&](uint32_t dst, uint64_t tile, bool first) {
#pragma unroll
                    for (int ks = 0; ks < C / 16; ++ks)
                        tc_mma_ss(one, tu + dst + 16 * ks, vm + 2048 * ks / 16, tile + (16 * ks * 128 + 32 * ks) / 16,
                                  tc_idesc<false, true>(C - 16 * ks), !first || ks > 0);
                };
                if (!tc_warp_wait(bar + B_FULL + par, (n >> 1) & 1, dead, d.spin)) break;
                if (!tc_warp_wait(bar + B_S, par, dead, d.spin)) break;
                tc_fence_after();
#pragma unroll
                for (int p = 2; p >= 0; --p)
#pragma unroll
                    for (int ks = 0; ks < DKP / 16; ++ks)
                        tc_mma_ts(one, tu + L::R, tu + L::SP + p * (DKP / 2) + 8 * ks, kd + ((ks >> 2) * L::TILE + 32 * (ks & 3)) / 16,
                                  tc_idesc<false>(C), p < 2 || ks > 0);
                tc_commit_to(one, bar + B_R);
#pragma unroll
                for (int p = 2; p >= 0; --p) tri_ss(L::U, yd + p * L::TILE / 16, p == 2);
#pragma unroll
                for (int p = 1; p >= 0; --p) tri_ss(L::O, zd + p * L::TILE / 16, p == 1);
                if (!tc_warp_wait(bar + B_READ, par, dead, d.spin)) break;
                tc_fence_after();
#pragma unroll
                for (int p = 1; p >= 0; --p)
#pragma unroll
                    for (int ks = 0; ks < DKP / 16; ++ks)
                        tc_mma_ts(one, tu + L::R, tu + L::SP + p * (DKP / 2) + 8 * ks, qd + ((ks >> 2) * L::TILE + 32 * (ks & 3)) / 16,
                                  tc_idesc<false>(C), p < 1 || ks > 0);
                tc_commit_to(one, bar + B_O1);
                if (!tc_warp_wait(bar + B_W, par, dead, d.spin)) break;
                tc_fence_after();
#pragma unroll
                for (int a = 2; a >= 0; --a)
#pragma unroll
                    for (int p = 2 - a; p >= 0; --p) tri_ts(L::U, L::UP + a * (C / 2), yd + p * L::TILE / 16);
                tc_commit_to(one, bar + B_UACC);
#pragma unroll
                for (int a = 1; a >= 0; --a)
#pragma unroll
                    for (int p = 1 - a; p >= 0; --p) tri_ts(L::O, L::UP + a * (C / 2), zd + p * L::TILE / 16);
                tc_commit_to(one, bar + B_O2);
                if (!tc_warp_wait(bar + B_U, par, dead, d.spin)) break;
                if (!tc_warp_wait(bar + B_O2, par, dead, d.spin)) break;      // w's planes make room for the update
                tc_fence_after();
#pragma unroll
                for (int p = 2; p >= 0; --p)
#pragma unroll
                    for (int ks = 0; ks < C / 16; ++ks)
                        tc_mma_ts(one, tu + L::UP, tu + L::SP + p * (C / 2) + 8 * ks, kn + 2048 * ks / 16, tc_idesc<true>(DKP), p < 2 || ks > 0);
                tc_commit_to(one, bar + B_UPD);
                tc_commit_to(one, bar + B_EMPTY + par);
            }
        }
        __syncwarp();
    } else {
        // ---- the copies
        const int ct = tid - 32 * (kTcWarps + 1);
        // a thread copies 16-byte piece ck of K's and Q's rows rk + RK i, and piece c of V's rows r + 8 i
        constexpr int PC = DKP / 8, RK = kTcCopy / PC;
        const int ck = ct % PC, rk = ct / PC, c = ct & 15, r = ct >> 4;
        const int koff = (ck >> 3) * L::TILE + tc_at(rk, ck & 7), voff = L::V + (c >> 3) * L::TILE + tc_at(r, c & 7);
        const int pieces = d.Dv - dv_blk < 128 ? (d.Dv - dv_blk) / 8 : 16;
        const bool kin = ck * 8 < d.Dk, vin = c < pieces;
        const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(in.k) + b * d.ks[0] + hk * d.ks[2];
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(in.q) + b * d.qs[0] + hk * d.qs[2];
        const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(in.v) + b * d.vs[0] + h * d.vs[2] + dv_blk;
        const long long orow = (long long)d.H * d.Dv;
        __nv_bfloat16 *out = o + (((long long)b * d.T + r) * d.H + h) * d.Dv + dv_blk + c * 8;
        bool good = true;                                          // this thread's waits so far
        // The readings of chunk n, once its stage is done with (rows past the valid tokens are 0). Returns
        // whether all copying threads' waits have succeeded: they leave together.
        auto store = [&](int n) {
            good = good && tc_wait(bar + B_EMPTY + (n & 1), (n >> 1) & 1, dead, d.spin);
            const unsigned char *src = smem + (n & 1) * L::STAGE + voff;
            const int t0 = n * C + r;
            if (good && vin) {
                __nv_bfloat16 *dst = out + (long long)n * C * orow;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint4 x = *reinterpret_cast<const uint4 *>(src + 1024 * i);
                    if (t0 + 8 * i >= ntok) x = make_uint4(0u, 0u, 0u, 0u);
                    if (t0 + 8 * i < d.T) *reinterpret_cast<uint4 *>(dst + 8 * i * orow) = x;
                }
            }
            // also: every thread's reads, before any copy into the stage
            int all;
            asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.and.pred q, 1, %2, p;\n"
                         " selp.b32 %0, 1, 0, q;\n}" : "=r"(all) : "r"((int)good), "n"(kTcCopy) : "memory");
            return all != 0;
        };
        bool ok = true;
        for (int n = 0; n < nch; ++n) {
            const int s = n & 1;
            unsigned char *st = smem + s * L::STAGE;
            const uint32_t sa = smem_u32(st);
            if (n >= 2 && !(ok = store(n - 2))) break;
            const long long t0 = (long long)n * C, bhn = bh * d.Nt + n;
            const int nt = ntok - (int)t0 < C ? ntok - (int)t0 : C;
            if (ct == 0) {
                mbar_arrive_expect_tx(bar + B_BULK + s, 5 * L::TILE + 2 * C * 4);
                bulk_g2s(st + L::Y, w.x + bhn * (3 * L::TILE), 3 * L::TILE, bar + B_BULK + s);
                bulk_g2s(st + L::Z, w.p + bhn * (2 * L::TILE), 2 * L::TILE, bar + B_BULK + s);
                bulk_g2s(smem + L::AUX + 512 * s, w.aux + bhn * 3 * C, 2 * C * 4, bar + B_BULK + s);
            }
            const __nv_bfloat16 *kp = k + (t0 + rk) * d.ks[1] + ck * 8, *qp = q + (t0 + rk) * d.qs[1] + ck * 8;
#pragma unroll
            for (int i = 0; i < C / RK; ++i) {
                const bool live = kin && rk + RK * i < nt;
                cp_async16_zfill(sa + L::K + koff + RK * 128 * i, live ? kp + RK * i * d.ks[1] : k, live);
                cp_async16_zfill(sa + L::Q + koff + RK * 128 * i, live ? qp + RK * i * d.qs[1] : q, live);
            }
            const __nv_bfloat16 *vp = v + (t0 + r) * d.vs[1] + c * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool live = vin && r + 8 * i < nt;
                cp_async16_zfill(sa + voff + 1024 * i, live ? vp + 8 * i * d.vs[1] : v, live);
            }
            cp_async_commit();
            cp_async_wait<0>();
            if (ct == 0 && !tc_wait(bar + B_BULK + s, (n >> 1) & 1, dead, d.spin)) {
                mbar_wait_bounded(bar + B_BULK + s, (n >> 1) & 1);    // nothing in flight behind a give-up
                good = false;
            }
            fence_proxy_async_smem();                              // the tiles, before the tensor core reads them
            mbar_arrive(bar + B_FULL + s);
        }
        for (int n = nch > 2 ? nch - 2 : 0; ok && n < nch; ++n) ok = store(n);
        if (vin)
            for (long long t = (long long)nch * C; t + r < d.T; t += 8) *reinterpret_cast<uint4 *>(out + t * orow) = make_uint4(0u, 0u, 0u, 0u);
    }
    __syncthreads();
    if (*dead) {
        // the products issued so far are waited for (the copies were, by their own thread)
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
