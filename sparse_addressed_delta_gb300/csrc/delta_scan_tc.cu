// The gated delta rule's scan over a head's chunks (notation of delta_chunk.cu) on the 5th-generation
// tensor cores, for bfloat16 inputs. As in the register form everything is transposed: 128 of the
// state's columns are the 128 lanes of tensor memory. With X and Z = P diag(beta) X from k_delta_local,
// a chunk is
//   R = S^T K^T;  w = -G R;  U = V^T X^T + w X^T;  S = G_C S + (e^{L_C - L} beta U) K
//   o = scale G (S^T Q^T) + V^T Z^T + w Z^T      (all transposed; S before the chunk; U is r)
// S, w and the decayed U are A operands in tensor memory, as bfloat16 planes that their own lanes'
// threads store; V is an A operand in shared memory; K, Q, X and Z are B operands there, K in both its
// majors (K S runs over Dk, the state's update over the tokens). Three planes (24 bits) go into every
// product, so that readings differ from float32 arithmetic's only where that rounds the other way. A thread keeps its part of its lane of S in registers
// in float32 for the whole sequence; the tensor core only ever sums one chunk's update.
//
// What bounds it: every chunk's chain R -> w -> U -> update -> S, products and the threads' work in
// turn. The chain runs in two halves, one behind the other: half the warps own the chunk's first 32
// tokens and the first half of Dk, the others the rest. The triangular products let the first tokens'
// U finish before the second tokens' w is there, the update's products start with the first tokens,
// and the first half of the new S enters the next chunk's R while the second is being made. The values'
// products and the readings run in the gaps. Measured at 128 x 128: 64 heads x 64 chunks, saving, 253 us (4.0 a
// chunk; 3 to 3.4 without saving); 256 ragged heads x up to 64 chunks, 335 us. In registers (as delta_chunk.cu's
// for float32) the first took 425: an m16n8k16 product is 8 cycles on one of four tensor cores.
//
// Warps 0..15 compute (lanes 32 (warp % 4).., quarter warp / 4 of the tokens and of Dk), warp 16 issues
// the products, warp 17 loads, warp 18 stores the readings; K, Q, V and the readings move as tensor
// copies. Two stages of chunk inputs, two buffers of readings. Every wait is bounded: one that gives up
// sets SDM_ERR_TIMEOUT in the status block, and the block leaves after its copies and products in flight.
#include "tcgen05.cuh"

namespace sdm {
namespace {

constexpr int kTcC = 64;
constexpr int kTcWarps = 16, kTcThreads = 32 * (kTcWarps + 3);

template <int DKP>
struct TcScan {
    static constexpr int TILE = kTcC * 128;                        // 64 columns of a token tile
    static constexpr int K = 0, Q = K + DKP / 64 * TILE, X = Q + DKP / 64 * TILE, Z = X + 3 * TILE;
    static constexpr int V = Z + 3 * TILE, STAGE = V + 2 * TILE;
    static constexpr int O = 2 * STAGE, AUX = O + 2 * 2 * TILE,   // readings: two buffers like V's
                          BARS = AUX + 2 * 512, BAD = BARS + 256,   // per column: the first chunk delta_column takes
                          BYTES = BAD + 512 + 1024;
    static_assert(BYTES <= 227 * 1024, "shared memory");
    // Tensor memory columns: planes of S, planes of w (then the update), R (then the readings' corrections), U
    // (then, in each quarter's own 16 columns, two planes of the decayed U), S^T Q^T. The decayed U's third plane
    // takes the second half of S's third, whose products with K and Q come before U's.
    static constexpr int SP = 0, UP = 3 * (DKP / 2), R = UP + 128, U = R + 64, OA = U + 64;
    static constexpr int LO = DKP == 128 ? SP + 160 : OA + 64;
    static_assert((DKP == 128 ? OA + 64 : LO + 32) <= 512, "tensor memory");
};

enum {
    B_FULL = 0, B_EMPTY = 2, B_OUT = 4, B_OFREE = 6,               // [stage]
    B_S = 8, B_W = 10, B_U = 12, B_R = 14, B_UACC = 16, B_UPD = 18, // [half]
    B_READ = 20, B_O1, B_O2, B_DRAIN, B_BULK, B_COUNT = B_BULK + 2
};

enum { SCAN_READ, SCAN_SAVE, SCAN_CARRY };

// SCAN_SAVE: also what a backward needs. SCAN_CARRY: the segments' end states only (DeltaBlock). SEG: the
// sequences are in segments; a form of its own, for its registers (one form for both spilled: a call with 8
// sequences of up to 4096 tokens, 32 heads, took 4 % longer).
template <int DKP, int MODE, bool SEG>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_delta_scan_tc(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo, DeltaDims d,
                    DeltaIn in, DeltaLocal w, float *state, __nv_bfloat16 *o, float *snap, float *rsave) {
    using L = TcScan<DKP>;
    constexpr int C = kTcC, HD = DKP / 4;                          // columns of S a thread
    constexpr bool SAVE = MODE == SCAN_SAVE, CARRY = MODE == SCAN_CARRY;
    constexpr int UPD = CARRY ? (DKP == 128 ? L::R : L::OA) : L::UP, UPD1 = CARRY ? L::OA : L::UP + 64;   // the update's halves
    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    auto bar = reinterpret_cast<unsigned long long *>(smem + L::BARS);
    volatile int *dead = reinterpret_cast<int *>(bar + B_COUNT);
    auto slot = reinterpret_cast<uint32_t *>(bar + B_COUNT + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const DeltaBlock blk = delta_block(d, in.valid, SEG, CARRY ? DELTA_CARRY : DELTA_RUN, 128);
    const int dv_blk = blk.tile * 128, seg = blk.seg, width = CARRY && blk.unit ? d.Dk : d.Dv;
    const long long bh = blk.bh;
    const int b = (int)(bh / d.H), h = (int)(bh % d.H), hk = h / (d.H / d.Hk);
    const int ntok = delta_valid(in.valid, b, d.T), chunks = (ntok + C - 1) / C;
    const int n0 = SEG ? delta_bound(d, chunks, seg) : 0, nch = SEG ? delta_bound(d, chunks, seg + 1) - n0 : chunks;
    const bool last = !SEG || seg + 1 == d.segs;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar + B_FULL + i, 32);
            mbar_init(bar + B_EMPTY + i, kTcWarps + 1);
            mbar_init(bar + B_OUT + i, kTcWarps);
            mbar_init(bar + B_OFREE + i, 1);
        }
        for (int i = B_S; i < B_R; ++i) mbar_init(bar + i, kTcWarps / 2);
        for (int i = B_R; i < B_COUNT; ++i) mbar_init(bar + i, i == B_READ ? kTcWarps : 1);
        *dead = tc_gives_up(d.spin) || (SEG && !CARRY && w.status->code != 0);   // an earlier kernel of this call gave up
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
    int first = -1;                                                // chunk of the column's first update that is not finite

    if (warp < kTcWarps) {
        // ---- the lanes' threads
        const int part = warp >> 2, half = part >> 1, lane0 = 32 * (warp & 3), dv = dv_blk + lane0 + lane;
        const bool mine = dv < width;
        const uint32_t at = tm + ((uint32_t)lane0 << 16);
        const int dk0 = part * HD;
        float S[HD];
        {
            const bool real = !CARRY || seg == 0;
            const float *sp = (SEG && !CARRY ? w.starts + seg * delta_states(d) : state) + (bh * d.Dk + dk0) * d.Dv + dv;
#pragma unroll
            for (int i = 0; i < HD; ++i) S[i] = real && mine && dk0 + i < d.Dk ? sp[(size_t)i * d.Dv] : blk.unit && dk0 + i == dv ? 1.f : 0.f;
        }
        // columns [i0, i1) of S as rows of a [Dk, Dv] state
        auto keep_state = [&](float *dst, int i0, int i1) {
            dst += (dk0 + i0) * width + dv;
#pragma unroll
            for (int c = 0; c < HD; c += 16) {                     // Dk is a multiple of 16
                if (c < i0 || c >= i1 || !mine || dk0 + c >= d.Dk) continue;
#pragma unroll
                for (int i = 0; i < 16; ++i) tc_put(dst, S[c + i], width);
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
        // the readings' 8 x 8 blocks in the row buffer: block b of a store is 8 columns of dv (b % 2) and
        // 8 tokens (b / 2), a lane's row one token
        const int orow = 16 * part + 8 * (lane >> 4) + (lane & 7), ocol = (lane0 >> 3) + ((lane >> 3) & 1);
        for (int it = 0; it < nch; ++it) {
            const unsigned par = it & 1;
            const int n = n0 + it;
            float *keep = snap + ((bh * (d.Nt + 1) + n) * (long long)d.Dk) * d.Dv;
            if (!tc_warp_wait(bar + B_FULL + par, (it >> 1) & 1, dead, d.spin)) break;
            const float *aux = reinterpret_cast<const float *>(smem + L::AUX + 512 * par);
            const float *from = aux + 16 * part, *to = aux + C + 16 * part;
            const float whole = aux[C - 1];
            float x[16];
            if (!tc_warp_wait(bar + B_R + half, par, dead, d.spin)) break;
            tc_fence_after();
            tc_load16(at + L::R + 16 * part, x);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] *= -from[i];
            {
                const uint32_t dst = at + L::UP + 8 * part;
                tc_store_planes(dst, dst + C / 2, dst + C, x);
            }
            tc_wait_st();
            arrive(B_W + half);
            if (SAVE) keep_state(keep, 0, HD / 2);                 // in the products' time
            if (!tc_warp_wait(bar + B_UACC + half, par, dead, d.spin)) break;
            tc_fence_after();
            tc_load16(at + L::U + 16 * part, x);
            if (SAVE && mine) {
                float *dst = rsave + ((bh * d.Nt + n) * (long long)C + 16 * part) * d.Dv + dv;
#pragma unroll
                for (int i = 0; i < 16; ++i) tc_put(dst, x[i], d.Dv);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] *= to[i];
            {
                const uint32_t dst = at + L::U + 16 * part;
                tc_store_planes(dst, dst + 8, at + L::LO + 8 * part, x);
            }
            tc_wait_st();
            arrive(B_U + half);
            if (SAVE) keep_state(keep, HD / 2, HD);
            // the readings, in a buffer that warp 18 stores; 0 past the valid tokens
            if constexpr (!CARRY) {
                if (!tc_warp_wait(bar + B_O2, par, dead, d.spin)) break;
                if (!tc_warp_wait(bar + B_O1, par, dead, d.spin)) break;
                if (it >= 2 && !tc_warp_wait(bar + B_OFREE + par, ((it >> 1) - 1) & 1, dead, d.spin)) break;
                tc_fence_after();
#pragma unroll
                for (int l = 0; l < 2; ++l) {                          // 16 lanes of dv
                    float y[8], z[8];
                    tc_load_frag16(at + ((uint32_t)(16 * l) << 16) + L::OA + 16 * part, at + ((uint32_t)(16 * l) << 16) + L::R + 16 * part, y, z);
                    unsigned r[4];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int t = 8 * (i >> 2) + 2 * (lane & 3) + (i & 1);
                        z[i] = n * C + 16 * part + t < ntok ? fmaf(d.scale * from[t], y[i], z[i]) : 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[i] = pack_bf16(z[2 * i], z[2 * i + 1]);
                    const int c = ocol + 2 * l;
                    stsm4t(smem_u32(smem) + L::O + (2 * par + (c >> 3)) * L::TILE + tc_at(orow, c & 7), r);
                }
                fence_proxy_async_smem();
                arrive(B_READ);
                if (lane == 0) mbar_arrive(bar + B_OUT + par);
            }
            if (!tc_warp_wait(bar + B_UPD + half, par, dead, d.spin)) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
                tc_load16(at + (half == 0 || DKP == 64 ? UPD + dk0 : UPD1 + dk0 - 64) + c, x);
                // a NaN or infinity of a token leaves no row of the update finite; the column's state before is kept
                if (!CARRY && c == 0 && mine && !delta_finite(x[0]) && first < 0) {
                    first = n;
                    keep_state(w.starts + seg * delta_states(d) + bh * d.Dk * (long long)d.Dv, 0, HD);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) S[c + i] = fmaf(whole, S[c + i], x[i]);
            }
            if (it + 1 < nch) planes_of_s();
            arrive(B_S + half);
            if (lane == 0) mbar_arrive(bar + B_EMPTY + par);
        }
        if (CARRY)
            keep_state(blk.unit ? w.units + ((seg - 1) * (long long)d.B * d.H + bh) * d.Dk * d.Dk
                                : w.starts + (seg + 1) * delta_states(d) + bh * d.Dk * (long long)d.Dv, 0, HD);
        else if (last && nch > 0 && !*dead)
            keep_state(state + bh * d.Dk * (long long)d.Dv, 0, HD);
        if (SAVE && last) keep_state(snap + ((bh * (d.Nt + 1) + chunks) * (long long)d.Dk) * d.Dv, 0, HD);
        if (part == 0) reinterpret_cast<int *>(smem + L::BAD)[lane0 + lane] = first;   // if the other parts agree
    } else if (warp == kTcWarps) {
        // ---- the products
        const uint32_t one = tc_elect(), tu = __shfl_sync(~0u, tm, 0), base = __shfl_sync(~0u, smem_u32(smem), 0);
        for (int it = 0; it < nch; ++it) {
            const unsigned par = it & 1;
            const uint32_t st = base + par * L::STAGE;
            // a descriptor's address counts 16 bytes
            const uint32_t kd = tc_k_major(st + L::K), qd = tc_k_major(st + L::Q), xd = tc_k_major(st + L::X),
                           zd = tc_k_major(st + L::Z), kn = tc_n_major(st + L::K, L::TILE), vm = tc_n_major(st + L::V, L::TILE);
            // lower triangular B: K step ks reaches the columns from 16 ks on
            auto tri = [&](uint32_t dst, uint32_t a, uint32_t tile, int ks) {
                tc_mma_ts(one, tu + dst + 16 * ks, tu + a + 8 * ks, tile + (16 * ks * 128 + 32 * ks) / 16, tc_idesc<false>(C - 16 * ks), true);
            };
            auto tri_v = [&](uint32_t dst, uint32_t tile, int ks, bool add) {
                tc_mma_ss(one, tu + dst + 16 * ks, vm + 2048 * ks / 16, tile + (16 * ks * 128 + 32 * ks) / 16,
                          tc_idesc<false, true>(C - 16 * ks), add);
            };
            // 16 tokens' or more rows of a [tokens][DKP] tile against the planes of S
            auto rows = [&](uint32_t dst, uint32_t tile, int t0, int tokens, int p, int ks, bool add) {
                tc_mma_ts(one, tu + dst + t0, tu + L::SP + p * (DKP / 2) + 8 * ks, tile + (t0 * 128 + (ks >> 2) * L::TILE + 32 * (ks & 3)) / 16,
                          tc_idesc<false>(tokens), add);
            };
            auto update = [&](int ks, int hd, int p, bool add) {   // half hd of Dk, or (Dk 64) all of it at once
                tc_mma_ts(one, tu + (hd ? UPD1 : UPD), tu + (p < 2 ? L::U + 16 * ks + 8 * p : L::LO + 8 * ks),
                          kn + (2048 * ks + hd * L::TILE) / 16, tc_idesc<true>(DKP == 128 ? 64 : DKP), add);
            };
            if (!tc_warp_wait(bar + B_FULL + par, (it >> 1) & 1, dead, d.spin)) break;
            if (!CARRY && it > 0 && !tc_warp_wait(bar + B_READ, par ^ 1, dead, d.spin)) break;
            if (!tc_warp_wait(bar + B_S, par, dead, d.spin)) break;
            tc_fence_after();
            constexpr int KS = DKP / 16;
#pragma unroll
            for (int p = 2; p >= 0; --p)
#pragma unroll
                for (int ks = 0; ks < KS / 2; ++ks) rows(L::R, kd, 0, C, p, ks, p < 2 || ks > 0);
            if (!tc_warp_wait(bar + B_S + 1, par, dead, d.spin)) break;
            tc_fence_after();
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                for (int p = 2; p >= 0; --p)
#pragma unroll
                    for (int ks = KS / 2; ks < KS; ++ks) rows(L::R, kd, 32 * hf, 32, p, ks, true);
                tc_commit_to(one, bar + B_R + hf);
            }
            // sums from their smallest terms up: the tensor core cuts an accumulator's low bits at every step
#pragma unroll
            for (int p = 2; p >= 1; --p)
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks) tri_v(L::U, xd + p * L::TILE / 16, ks, p < 2 || ks > 0);
            if constexpr (!CARRY) {
#pragma unroll
                for (int p = 2; p >= 1; --p)
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) rows(L::OA, qd, 0, C, p, ks, p < 2 || ks > 0);
            }
            bool ok = true;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                ok = ok && tc_warp_wait(bar + B_W + hf, par, dead, d.spin);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int sum = 2; sum >= 0; --sum)
#pragma unroll
                    for (int a = sum; a >= 0; --a)
#pragma unroll
                        for (int ks = 2 * hf; ks < 2 * hf + 2; ++ks)
                            tri(L::U, L::UP + a * (C / 2), xd + (sum - a) * L::TILE / 16, ks);
#pragma unroll
                for (int ks = 2 * hf; ks < 2 * hf + 2; ++ks) tri_v(L::U, xd, ks, true);
                tc_commit_to(one, bar + B_UACC + hf);
            }
            if (!ok) break;
            if constexpr (!CARRY) {
#pragma unroll
                for (int sum = 2; sum >= 0; --sum) {                   // R is used: V^T Z^T + w Z^T in its place
#pragma unroll
                    for (int ks = 0; ks < C / 16; ++ks)
                        if (sum > 0) tri_v(L::R, zd + sum * L::TILE / 16, ks, sum < 2 || ks > 0);
#pragma unroll
                    for (int a = sum; a >= 0; --a)
#pragma unroll
                        for (int ks = 0; ks < C / 16; ++ks) tri(L::R, L::UP + a * (C / 2), zd + (sum - a) * L::TILE / 16, ks);
                }
                tc_commit_to(one, bar + B_O2);
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks) tri_v(L::R, zd, ks, true);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) rows(L::OA, qd, 0, C, 0, ks, true);
                tc_commit_to(one, bar + B_O1);
                if (!tc_warp_wait(bar + B_O2, par, dead, d.spin)) break;      // w's planes make room for the update
            }
            if (!tc_warp_wait(bar + B_U, par, dead, d.spin)) break;
            tc_fence_after();
#pragma unroll
            for (int p = 2; p >= 1; --p)
#pragma unroll
                for (int hd = 0; hd < DKP / 64; ++hd) {
                    update(0, hd, p, p < 2);
                    update(1, hd, p, true);
                }
            if (!tc_warp_wait(bar + B_U + 1, par, dead, d.spin)) break;
            tc_fence_after();
#pragma unroll
            for (int hd = 0; hd < DKP / 64; ++hd) {
#pragma unroll
                for (int p = 2; p >= 1; --p) {
                    update(2, hd, p, true);
                    update(3, hd, p, true);
                }
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks) update(ks, hd, 0, true);
                tc_commit_to(one, bar + B_UPD + hd);
            }
            if (DKP == 64) tc_commit_to(one, bar + B_UPD + 1);
            tc_commit_to(one, bar + B_EMPTY + par);
        }
        __syncwarp();
    } else if (warp == kTcWarps + 1) {
        // ---- the chunks' inputs
        if (blk.unit) {                                            // no values
            for (int i = lane; i < 2 * 2 * L::TILE / 16; i += 32)
                *reinterpret_cast<uint4 *>(smem + (i / (2 * L::TILE / 16)) * L::STAGE + L::V + i % (2 * L::TILE / 16) * 16) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
        }
        const uint32_t bytes = 2 * C * 4 + (!CARRY ? L::STAGE : DKP / 64 * L::TILE + 3 * L::TILE + (blk.unit ? 0 : 2 * L::TILE));
        for (int it = 0; it < nch; ++it) {
            const int n = n0 + it, s = it & 1, t0 = n * C, nt = ntok - t0 < C ? ntok - t0 : C;
            unsigned char *st = smem + s * L::STAGE;
            const long long bhn = bh * d.Nt + n;
            unsigned long long *full = bar + B_BULK + s;
            if (it >= 2 && !tc_warp_wait(bar + B_EMPTY + s, ((it >> 1) - 1) & 1, dead, d.spin)) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(full, bytes);
                for (int c = 0; c < DKP / 64; ++c) {
                    tc_tensor_load(st + L::K + c * L::TILE, &mk, 64 * c, tc_coord(d.ks[2], hk), t0, tc_coord(d.ks[0], b), full);
                    if (!CARRY) tc_tensor_load(st + L::Q + c * L::TILE, &mq, 64 * c, tc_coord(d.qs[2], hk), t0, tc_coord(d.qs[0], b), full);
                }
                for (int c = 0; c < (blk.unit ? 0 : 2); ++c) tc_tensor_load(st + L::V + c * L::TILE, &mv, dv_blk + 64 * c, tc_coord(d.vs[2], h), t0, tc_coord(d.vs[0], b), full);
                bulk_g2s(st + L::X, w.x + bhn * (3 * L::TILE), 3 * L::TILE, full);
                if (!CARRY) bulk_g2s(st + L::Z, w.p + bhn * (3 * L::TILE), 3 * L::TILE, full);
                bulk_g2s(smem + L::AUX + 512 * s, w.aux + bhn * kDeltaAux * C, 2 * C * 4, full);
            }
            __syncwarp();
            if (!tc_warp_wait(full, (it >> 1) & 1, dead, d.spin)) {
                mbar_wait_bounded(full, (it >> 1) & 1);             // nothing in flight behind a give-up
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
                    for (int c = 0; c < 2; ++c) *reinterpret_cast<uint4 *>(st + L::V + c * L::TILE + off) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
            }
            mbar_arrive(bar + B_FULL + s);
        }
    } else if (!CARRY) {
        // ---- the readings
        for (int it = 0; it < nch; ++it) {
            if (!tc_warp_wait(bar + B_OUT + (it & 1), (it >> 1) & 1, dead, d.spin)) break;
            if (lane == 0) {
                for (int c = 0; c < 2; ++c)
                    if (dv_blk + 64 * c < d.Dv)
                        tc_tensor_store(&mo, dv_blk + 64 * c, h, (n0 + it) * C, b, smem + L::O + (2 * (it & 1) + c) * L::TILE);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                mbar_arrive(bar + B_OFREE + (it & 1));
            }
            __syncwarp();
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        const int cols = d.Dv - dv_blk < 128 ? d.Dv - dv_blk : 128;
        __nv_bfloat16 *out = o + ((long long)b * d.T * d.H + h) * d.Dv + dv_blk;
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
    const bool bad = __syncthreads_or(first >= 0);
    if (warp == kTcWarps) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512));
    if (CARRY || !bad || *dead) return;
    if (warp >= 4 && warp < kTcWarps) {
        int *own = reinterpret_cast<int *>(smem + L::BAD) + 32 * (warp & 3) + lane;
        if (first != *own) *own = -1;
    }
    __syncthreads();
    for (int c = warp; c < 128; c += kTcThreads / 32) {
        const int n = reinterpret_cast<int *>(smem + L::BAD)[c], t0 = n * C, dv = dv_blk + c;
        if (n < 0) continue;
        delta_column(d, in, b, h, dv, t0, ntok - t0 < C ? ntok - t0 : C, w.starts + seg * delta_states(d) + bh * d.Dk * (long long)d.Dv + dv, o + (((long long)b * d.T + t0) * d.H + h) * d.Dv + dv,
                     SAVE ? rsave + (bh * d.Nt + n) * (long long)C * d.Dv + dv : nullptr);
    }
}

template <int DKP>
cudaError_t scan_tc(const DeltaDims &d, const DeltaIn &in, const DeltaLocal &w, float *state, void *o, float *snap,
                    float *r, cudaStream_t st) {
    const long long os[3] = {(long long)d.T * d.H * d.Dv, (long long)d.H * d.Dv, d.Dv};
    CUtensorMap mq, mk, mv, mo;
    cudaError_t e = tc_tensor_map(&mq, in.q, d.qs, d.B, d.T, d.Hk, d.Dk);
    if (e == cudaSuccess) e = tc_tensor_map(&mk, in.k, d.ks, d.B, d.T, d.Hk, d.Dk);
    if (e == cudaSuccess) e = tc_tensor_map(&mv, in.v, d.vs, d.B, d.T, d.H, d.Dv);
    if (e == cudaSuccess) e = tc_tensor_map(&mo, o, os, d.B, d.T, d.H, d.Dv);
    if (e != cudaSuccess) return e;
    auto run = [&](auto kern, int mode) {
        set_kernel_smem(kern, TcScan<DKP>::BYTES);
        kern<<<(unsigned)delta_blocks(d, mode, 128), kTcThreads, TcScan<DKP>::BYTES, st>>>(mq, mk, mv, mo, d, in, w, state, static_cast<__nv_bfloat16 *>(o), snap, r);
        return cudaGetLastError();
    };
    if (d.segs > 1) {
        e = run(k_delta_scan_tc<DKP, SCAN_CARRY, true>, DELTA_CARRY);
        if (e == cudaSuccess) e = launch_delta_join(d, w, state, false, st);
        if (e != cudaSuccess) return e;
        return snap ? run(k_delta_scan_tc<DKP, SCAN_SAVE, true>, DELTA_RUN) : run(k_delta_scan_tc<DKP, SCAN_READ, true>, DELTA_RUN);
    }
    return snap ? run(k_delta_scan_tc<DKP, SCAN_SAVE, false>, DELTA_RUN) : run(k_delta_scan_tc<DKP, SCAN_READ, false>, DELTA_RUN);
}

}  // namespace

namespace {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        cudaDriverEntryPointQueryResult found;
        void *fn = nullptr;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
        return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn) : nullptr;
    }();
    return encode;
}

cudaError_t encode_map(CUtensorMap *m, CUtensorMapDataType type, int rank, const void *p, const cuuint64_t *dim,
                       const cuuint64_t *strides, const cuuint32_t *box) {
    const auto encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return encode(m, type, rank, const_cast<void *>(p), dim, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t tc_tensor_map(CUtensorMap *m, const void *p, const long long *s, int B, int T, int heads, int D) {
    if (s[2] == 0) heads = 1;                                      // broadcast (tc_coord)
    if (s[0] == 0) B = 1;
    const cuuint64_t dim[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)B};
    // a dimension of one element is never stepped along: any stride will do
    auto bytes = [](long long stride, int n) { return (cuuint64_t)(n > 1 ? stride * 2 : 16); };
    const cuuint64_t str[3] = {bytes(s[2], heads), bytes(s[1], T), bytes(s[0], B)};
    const cuuint32_t box[4] = {64, 1, 64, 1};
    return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, p, dim, str, box);
}

cudaError_t tc_state_map(CUtensorMap *m, const void *p, long long slots, int rows, int columns, int box_rows) {
    const cuuint64_t dim[3] = {(cuuint64_t)columns, (cuuint64_t)rows, (cuuint64_t)slots};
    const cuuint64_t str[2] = {(cuuint64_t)columns * 4, (cuuint64_t)rows * columns * 4};
    const cuuint32_t box[3] = {32, (cuuint32_t)box_rows, 1};
    return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p, dim, str, box);
}

cudaError_t launch_delta_scan_tc(const DeltaDims &d, const DeltaIn &in, const DeltaLocal &w, float *state, void *o,
                                 float *snap, float *r, cudaStream_t st) {
    return d.Dk <= 64 ? scan_tc<64>(d, in, w, state, o, snap, r, st) : scan_tc<128>(d, in, w, state, o, snap, r, st);
}

}  // namespace sdm
