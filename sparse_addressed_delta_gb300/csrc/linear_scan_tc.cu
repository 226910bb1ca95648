// Linear attention's pass (linear_internal.cuh) over a head's chunks of 64 tokens on the 5th-generation tensor
// cores. Everything is transposed: 128 of the result's columns are the 128 lanes of tensor memory. With L the
// head's log-decay, i and j tokens of a chunk that begins with state S (a mirrored pass has i and j exchanged):
//   Z = (Q K^T) e^{L (i - j)} for j <= i, else 0          P (transposed), then planes in shared memory
//   o = e^{L (i + 1)} (S^T Q^T) + V^T Z^T                 OA and OB
//   S = e^{L n} S + V^T (e^{L (n - 1 - j)} K)              U, in one product with OB
// A float operand (S, Z, the decayed keys) goes in as three bfloat16 planes (24 bits), so results keep float32's
// accuracy and bfloat16 ones differ from float32 arithmetic's only where that rounds the other way. float32 inputs
// come as three planes too (NP = 3), with six of their products. The state stays in registers in float32; the
// tensor core only ever sums one chunk, from the smallest terms up (it cuts an accumulator's low bits at every
// step).
//
// S^T's planes are an A operand in tensor memory, V^T one in shared memory; Q, Z^T and the decayed keys are B operands
// there, the last two side by side: one product makes U and OB, and reads V^T once for both. Warps 0..15 compute (lanes
// 32 (warp % 4).., quarter warp / 4 of the tokens and of K), warp 16 issues the products, warp 17 loads and warp 18
// stores bfloat16 results, both by tensor copies. While the threads make the next chunk's decayed keys and Z the tensor
// core reads the state (OA) and makes P; while they store the results and split the new state it makes U and OB.
//
// What bounds it: shared memory. A 128 x 128 chunk moves 390 KB through it (copies in and out 80, the decayed keys 64,
// Z 24, operands of P 48, of U and OB 120, of OA 48), 3070 cycles of the 4000 that a chunk takes (2.0 us); the rest is
// the hand-over of U, keys and readings from one to the next. Measured: 128 blocks of 64 chunks 134 us, of 32 saving
// nothing 71, mirrored 72; float32 parts for shared heads 84 and 80 (64 bytes a lane's store; through shared memory 88 and
// 85). bfloat16 results stored by the threads themselves 151. U before OB, in products of their own, so that the keys could
// start earlier: 135, the operands read twice eat what it gains.
//
// Every wait is bounded: one that gives up sets SDM_ERR_TIMEOUT in the status block, and the block leaves after its
// copies and products in flight.
#include <type_traits>

#include "linear_tc.cuh"

namespace sdm {
namespace {

constexpr int kLinC = 64, kLinWarps = 16, kLinThreads = 32 * (kLinWarps + 3);

template <int KP, int NP>
struct LinScan {
    static constexpr int TILE = kLinC * 128, KT = KP / 64;         // 64 columns of 64 tokens; such tiles of Q or K
    static constexpr int Q = 0, K = Q + NP * KT * TILE, V = K + NP * KT * TILE, STAGE = V + NP * 2 * TILE;
    static constexpr int STAGES = NP == 3 ? 1 : 3;
    // planes of the decayed keys and, in the same rows behind them, of Z^T
    static constexpr int PLANE = (KT + 1) * TILE, KX = STAGES * STAGE, Z = KX + KT * TILE, AUX = KX + 3 * PLANE;
    static constexpr int POW = AUX, PAIR = POW + 4 * 80, BARS = PAIR + 4 * 128, BAD = BARS + 256, BYTES = BAD + 4 * 512 + 1024;
    static_assert(BYTES <= 227 * 1024, "shared memory");
    static constexpr int SP = 0, OA = 3 * (KP / 2), U = OA + kLinC, OB = U + KP, P = OB + kLinC;
    static_assert(P + kLinC <= 512, "tensor memory");
};

enum { B_FULL = 0, B_EMPTY = 3, B_PART = 6, B_ZK, B_U, B_UF, B_P, B_O, B_OF, B_S, B_OUT, B_DRAIN, B_COUNT };

struct LinArgs {
    LinearPass p;
    const float *g;
    const int32_t *valid;
    const float *starts;                 // [segs][B, H, Dk, Dv] states the segments begin with, in the pass's order
    DevStatus *status;
    long long heads[3];                  // head strides of the laid operands, 0: broadcast
    long long seqs[3];
    bool column;                         // columns with NaN or infinity are taken again (linear_column)
    Chain chain;
};

// One column of a segment by one warp, token by token from the state it begins with; the readings of tokens from
// t1 on are stored. For columns whose update in a chunk is not finite: in the chunk's products a NaN or infinity of
// one token meets the zeros that stand for the tokens before it (0 x inf is NaN), here it reaches the later ones alone.
template <typename T>
__device__ __noinline__ void linear_column(const LinearDims &d, const LinearPass &p, float fade, int b, int h, int col, int t0, int t1, int t2,
                                           const float *S) {
    constexpr int NR = kLinearMaxDk / 32;
    const int lane = threadIdx.x & 31;
    const T *q = static_cast<const T *>(p.q.p) + b * p.q.s[0] + h / p.q.share * p.q.s[2];
    const T *k = static_cast<const T *>(p.k.p) + b * p.k.s[0] + h / p.k.share * p.k.s[2];
    const T *v = static_cast<const T *>(p.v.p) + b * p.v.s[0] + h / p.v.share * p.v.s[2] + col;
    T *o = static_cast<T *>(p.out) + ((long long)b * d.T * d.H + h) * p.V + col;
    float s[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) s[i] = S && lane + 32 * i < p.K ? S[(lane + 32 * i) * p.sk] : 0.f;
#pragma unroll 1
    for (int t = t0; t < t2; ++t) {
        const float x = to_f32(v[t * p.v.s[1]]);
        float c = 0.f;
#pragma unroll
        for (int i = 0; i < NR; ++i)
            if (lane + 32 * i < p.K) {
                s[i] = fmaf(to_f32(k[t * p.k.s[1] + lane + 32 * i]), x, s[i] * fade);
                c = fmaf(to_f32(q[t * p.q.s[1] + lane + 32 * i]), s[i], c);
            }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) c += __shfl_xor_sync(~0u, c, m);
        if (lane == 0 && t >= t1) o[(long long)t * d.H * p.V] = from_f32<T>(p.from * c);
    }
}

template <int KP, int NP, bool REV, typename OT>
__global__ void __launch_bounds__(kLinThreads, 1)
    k_linear_scan(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo, const __grid_constant__ LinearDims d,
                  const __grid_constant__ LinArgs a) {
    using L = LinScan<KP, NP>;
    constexpr int C = kLinC, HD = KP / 4, ST = L::STAGES, KT = L::KT, TILE = L::TILE;
    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    auto bar = reinterpret_cast<unsigned long long *>(smem + L::BARS);
    volatile int *dead = reinterpret_cast<int *>(bar + B_COUNT);
    auto slot = reinterpret_cast<uint32_t *>(bar + B_COUNT + 1);
    float *pw = reinterpret_cast<float *>(smem + L::POW), *pair = reinterpret_cast<float *>(smem + L::PAIR);
    const LinearPass &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // this block's columns, part of K, head and segment
    unsigned at_block = blockIdx.x;
    const int tiles = (p.V + 127) / 128;
    const int tile = (int)(at_block % tiles);
    at_block /= tiles;
    const int kb = (int)(at_block % p.blocks);
    at_block /= p.blocks;
    const int h = (int)(at_block % d.H);
    at_block /= d.H;
    const int b = linear_longest_first(d, a.valid, (int)(at_block % d.B)), seg = (int)(at_block / d.B);   // seg: in the pass's order
    const long long bh = (long long)b * d.H + h;
    const int v0 = tile * 128, k0 = kb * 128, K = p.K - k0 < 128 ? p.K - k0 : 128;
    const int ntok = linear_valid(a.valid, b, d.T), chunks = (ntok + C - 1) / C;
    const int place = REV ? d.segs - 1 - seg : seg;
    const int n0 = linear_cut(chunks, place, d.segs), nch = linear_cut(chunks, place + 1, d.segs) - n0;
    const long long states = (long long)d.B * d.H * d.Dk * d.Dv, own = bh * d.Dk * d.Dv + k0 * p.sk;

    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(bar + B_FULL + i, 1);
            mbar_init(bar + B_EMPTY + i, sizeof(OT) == 2 ? 2 : 1);
        }
        for (int i = B_PART; i < B_COUNT; ++i)
            mbar_init(bar + i, i == B_ZK || i == B_UF || i == B_OF || i == B_S || i == B_OUT ? kLinWarps : 1);
        fence_mbar_init();
    }
    if (warp == kLinWarps) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid < 128) {
        // e^{L n} of n tokens; with the scale, of tokens n apart (0 before)
        const int n = tid < C ? C - tid : tid - C;
        const float x = linear_power(a.g[h], n);
        if (tid <= C) pw[n] = x;
        if (tid == C) pw[0] = 1.f;
        pair[tid] = tid < C ? 0.f : p.pair * x;
    }
    // blocks of Z^T that hold no pairs are never written again
    for (int i = tid; i < 3 * TILE / 16; i += kLinThreads)
        *reinterpret_cast<uint4 *>(smem + L::Z + i / (TILE / 16) * L::PLANE + i % (TILE / 16) * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    chain_begin(a.chain);
    if (tid == 0) *dead = tc_gives_up(d.spin) || __ldcg(&a.status->code) != 0;   // an earlier kernel of this call gave up
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *slot;
    auto chunk_at = [&](int it) { return REV ? n0 + nch - 1 - it : n0 + it; };
    int first = -1;                                                // iteration of the column's first update that is not finite
    float2 S[HD / 2];

    if (warp < kLinWarps) {
        const int part = warp >> 2, lane0 = 32 * (warp & 3), col = v0 + lane0 + lane, kk = part * HD;
        const bool mine = col < p.V;
        const uint32_t at = tm + ((uint32_t)lane0 << 16);
        const float *begin = d.segs > 1 ? a.starts + seg * states : p.first;
        if (begin) begin += own + kk * p.sk + col * p.sv;
        if (p.sk == 1 && ((uintptr_t)begin & 15) == 0) {           // transposed: K runs along the row
#pragma unroll
            for (int i = 0; i < HD / 4; ++i) {
                const float4 x = begin && mine && kk + 4 * i < K ? __ldcg(reinterpret_cast<const float4 *>(begin + 4 * i)) : make_float4(0.f, 0.f, 0.f, 0.f);
                S[2 * i] = make_float2(x.x, x.y);
                S[2 * i + 1] = make_float2(x.z, x.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < HD; ++i) reinterpret_cast<float *>(S)[i] = begin && mine && kk + i < K ? __ldcg(begin + i * p.sk) : 0.f;
        }
        auto planes_of_s = [&] {
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
                const uint32_t dst = at + L::SP + (kk + c) / 2;
                store_planes3(dst, dst + KP / 2, dst + KP, S + c / 2);
            }
            tc_wait_st();
        };
        auto arrive = [&](int which) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + which);
        };
        // The decayed keys, in units of 8 columns of 32 tokens, and Z^T (by lanes 0..63 of tensor memory, a key's row each)
        // of chunk `it`. A scheduler has every fourth warp, so those of the other lanes, and those whose block of Z^T holds
        // no pairs, take three of the units each, and those with a block off the diagonal one (a narrow state: half of that).
        // 32 heads x 256 chunks in four segments: all units by the other lanes' warps 145 us, so 137, three at once 134.
        const int ahead = REV ? lane0 - 16 * part - 15 : 16 * part - lane0 - 31;   // least tokens apart
        int unit0, unit1;
        {
            constexpr int UNITS = 2 * KP / 8;                      // 32 or 16
            // warps of lanes 64..: 3 of each 4; without pairs: 3; off the diagonal: 1; on it: none
            const bool other = (warp & 3) >= 2;
            const int none = REV ? (warp & 3) == 0 && part >= 2 : (warp & 3) == 1 && part < 2;
            const int off = REV ? (warp & 3) == 1 && part < 2 : (warp & 3) == 0 && part >= 2;
            const int at_other = part * 2 + (warp & 1), at_rest = part & 1;
            const int from = other ? 3 * at_other : none ? 24 + 3 * at_rest : off ? 30 + at_rest : 32, many = other || none ? 3 : off ? 1 : 0;
            unit0 = from * UNITS / 32;
            unit1 = (from + many) * UNITS / 32;
        }
        auto local = [&](int it) {
            const int n = chunk_at(it), nt = ntok - n * C < C ? ntok - n * C : C;
            if (!tc_warp_wait(bar + B_FULL + it % ST, it / ST & 1, dead, d.spin)) return false;
            const unsigned char *src = smem + it % ST * L::STAGE + L::K;
            auto one = [&](int i) {
                const int row = 32 * (i & 1) + lane, piece = i >> 1, off = (piece >> 3) * TILE + tc_at(row, piece & 7);
                const float w = row < nt ? p.to * pw[REV ? row + 1 : nt - 1 - row] : 0.f;
                float2 x[4];
                load_piece<NP, KT * TILE>(src + off, x);
                scale_piece(x, w, smem + L::KX + off, L::PLANE);
            };
            if (unit1 - unit0 == 3) {                          // side by side: one takes 500 cycles by itself
#pragma unroll
                for (int i = 0; i < 3; ++i) one(unit0 + i);
            } else {
                for (int i = unit0; i < unit1; ++i) one(i);
            }
            if ((warp & 3) < 2 && ahead >= -46) {
                if (!tc_warp_wait(bar + B_P, it & 1, dead, d.spin)) return false;
                tc_fence_after();
                const int row = lane0 + lane;
                float2 x[8];
                tc_load16(at + L::P + 16 * part, reinterpret_cast<float(&)[16]>(x));
                if (ahead >= 0) {                              // e^{L apart} = e^{L least} e^{L rest}, all of it before the diagonal
                    const float w = pair[C + (REV ? row - 16 * part - 15 : 16 * part - row)];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        x[i] = mul2(mul2(x[i], make_float2(w, w)), REV ? make_float2(pw[15 - 2 * i], pw[14 - 2 * i]) : make_float2(pw[2 * i], pw[2 * i + 1]));
                } else {
                    const int apart = REV ? row - 16 * part : 16 * part - row;   // of column 0; the others' step by step
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int a0 = REV ? apart - 2 * i : apart + 2 * i, a1 = REV ? a0 - 1 : a0 + 1;
                        const float2 y = mul2(x[i], make_float2(pair[C + a0], pair[C + a1]));
                        x[i] = make_float2(a0 >= 0 ? y.x : 0.f, a1 >= 0 ? y.y : 0.f);   // (a NaN past the diagonal stays out)
                    }
                }
                unsigned pl[3][8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    unsigned s[3];
                    split3(x[e].x, x[e].y, s);
                    pl[0][e] = s[0]; pl[1][e] = s[1]; pl[2][e] = s[2];
                }
#pragma unroll
                for (int m = 0; m < 3; ++m)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        *reinterpret_cast<uint4 *>(smem + L::Z + m * L::PLANE + tc_at(row, 2 * part + c)) =
                            make_uint4(pl[m][4 * c], pl[m][4 * c + 1], pl[m][4 * c + 2], pl[m][4 * c + 3]);
            }
            fence_proxy_async_smem();
            arrive(B_ZK);
            return true;
        };
        // bfloat16 results, 8 x 8 blocks stored transposed: block i of a store is 8 columns (i % 2) and 8 tokens (i / 2), a
        // lane's row one token; and what the state's readings are times, of a whole chunk
        const int orow = 16 * part + 8 * (lane >> 4) + (lane & 7), ocol = (lane0 >> 3) + ((lane >> 3) & 1);
        float reads[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 16 * part + 8 * (i >> 1) + 2 * (lane & 3) + (i & 1);
            reads[i] = p.from * pw[REV ? C - 1 - t : t + 1];
        }
        if (nch > 0) {
            planes_of_s();
            arrive(B_S);
        }
        bool ok = nch > 0 && local(0);
        for (int it = 0; ok && it < nch; ++it) {
            const unsigned par = it & 1;
            const int n = chunk_at(it), nt = ntok - n * C < C ? ntok - n * C : C;
            ok = tc_warp_wait(bar + B_U, par, dead, d.spin);
            if (!ok) break;
            tc_fence_after();
            const float whole = pw[nt];
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
                float2 x[8];
                tc_load16(at + L::U + kk + c, reinterpret_cast<float(&)[16]>(x));
                if (c == 0 && first < 0 && !(fabsf(x[0].x) <= 3.402823466e38f)) first = it;
#pragma unroll
                for (int i = 0; i < 8; ++i) S[c / 2 + i] = fma2(make_float2(whole, whole), S[c / 2 + i], x[i]);
            }
            arrive(B_UF);
            if (it + 1 < nch && !(ok = local(it + 1))) break;
            ok = tc_warp_wait(bar + B_O, par, dead, d.spin);
            if (!ok) break;
            tc_fence_after();
            if constexpr (sizeof(OT) == 2) {
                // in the place of the chunk's V, which warp 18 stores
                unsigned char *to = smem + it % ST * L::STAGE + L::V;
                float y[2][8], z[2][8];                        // 16 lanes of columns each
                tc_load_frag16(at + L::OA + 16 * part, at + L::OB + 16 * part, y[0], z[0]);
                tc_load_frag16(at + (16u << 16) + L::OA + 16 * part, at + (16u << 16) + L::OB + 16 * part, y[1], z[1]);
                arrive(B_OF);
#pragma unroll
                for (int l = 0; l < 2; ++l) {
                    if (nt == C) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) z[l][i] = fmaf(reads[(i >> 2) * 2 + (i & 1)], y[l][i], z[l][i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int t = 16 * part + 8 * (i >> 2) + 2 * (lane & 3) + (i & 1);
                            z[l][i] = t < nt ? fmaf(p.from * pw[REV ? nt - 1 - t : t + 1], y[l][i], z[l][i]) : 0.f;
                        }
                    }
                    unsigned r[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[i] = pack_bf16(z[l][2 * i], z[l][2 * i + 1]);
                    const int c = ocol + 2 * l;
                    stsm4t(smem_u32(to) + (c >> 3) * TILE + tc_at(orow, c & 7), r);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + B_OUT);
            } else {
                float x[16], y[16];
                tc_load16(at + L::OA + 16 * part, y);
                tc_load16(at + L::OB + 16 * part, x);
                arrive(B_OF);
                float *out = static_cast<float *>(p.out) + ((((long long)kb * d.B + b) * d.T + n * C + 16 * part) * d.H + h) * p.V + col;
                const int left = d.T - n * C - 16 * part;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int t = 16 * part + i;
                    const float r = t < nt ? fmaf(p.from * pw[REV ? nt - 1 - t : t + 1], y[i], x[i]) : 0.f;
                    if (mine && i < left) *out = r;
                    out += (long long)d.H * p.V;
                }
            }
            if (it + 1 < nch) {
                planes_of_s();
                arrive(B_S);
            }
        }
        reinterpret_cast<int *>(smem + L::BAD)[part * 128 + lane0 + lane] = first;
    } else if (warp == kLinWarps) {
        // ---- the products
        const uint32_t one = tc_elect(), tu = __shfl_sync(~0u, tm, 0), base = __shfl_sync(~0u, smem_u32(smem), 0);
        constexpr int KS = KP / 16;
        auto scores = [&](int it) {                                // K Q^T; lanes 64.. hold whatever follows K
            const uint32_t st = base + it % ST * L::STAGE, qd = tc_k_major(st + L::Q), kd = tc_k_major(st + L::K);
            bool add = false;
#pragma unroll
            for (int sum = NP - 1; sum >= 0; --sum)
#pragma unroll
                for (int m = sum; m >= 0; --m)
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const int off = ((ks >> 2) * TILE + 32 * (ks & 3)) / 16;
                        tc_mma_ss(one, tu + L::P, kd + m * KT * TILE / 16 + off, qd + (sum - m) * KT * TILE / 16 + off, tc_idesc<false>(C), add);
                        add = true;
                    }
            tc_commit_to(one, bar + B_P);
        };
        bool ok = nch > 0;
        if (ok) {
            ok = tc_warp_wait(bar + B_FULL, 0, dead, d.spin);
            tc_fence_after();
            if (ok) scores(0);
        }
        for (int it = 0; ok && it < nch; ++it) {
            const uint32_t st = base + it % ST * L::STAGE, qd = tc_k_major(st + L::Q), vm = tc_n_major(st + L::V, TILE);
            const uint32_t kx = tc_n_major(base + L::KX, TILE);
            const unsigned par = it & 1;
            ok = tc_warp_wait(bar + B_FULL + it % ST, it / ST & 1, dead, d.spin) && tc_warp_wait(bar + B_ZK, par, dead, d.spin);
            ok = ok && (it == 0 || (tc_warp_wait(bar + B_UF, par ^ 1, dead, d.spin) && tc_warp_wait(bar + B_OF, par ^ 1, dead, d.spin)));
            if (!ok) break;
            tc_fence_after();
            // U and, in the columns behind it, OB: V^T is read once for both
            bool add = false;
#pragma unroll
            for (int sum = 2; sum >= 0; --sum)
#pragma unroll
                for (int m = sum < NP - 1 ? sum : NP - 1; m >= 0; --m)
#pragma unroll
                    for (int ks = 0; ks < C / 16; ++ks) {
                        tc_mma_ss(one, tu + L::U, vm + (m * 2 * TILE + 2048 * ks) / 16, kx + ((sum - m) * L::PLANE + 2048 * ks) / 16,
                                  tc_idesc<true, true>(KP + C), add);
                        add = true;
                    }
            tc_commit_to(one, bar + B_U);
            if (ST > 1 && it + 1 < nch) {
                ok = tc_warp_wait(bar + B_FULL + (it + 1) % ST, (it + 1) / ST & 1, dead, d.spin);
                if (!ok) break;
                tc_fence_after();
                scores(it + 1);
            }
            ok = tc_warp_wait(bar + B_S, par, dead, d.spin);
            if (!ok) break;
            tc_fence_after();
            add = false;
#pragma unroll
            for (int sum = 2; sum >= 0; --sum)
#pragma unroll
                for (int m = sum < NP - 1 ? sum : NP - 1; m >= 0; --m)
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        tc_mma_ts(one, tu + L::OA, tu + L::SP + (sum - m) * (KP / 2) + 8 * ks,
                                  qd + (m * KT * TILE + (ks >> 2) * TILE + 32 * (ks & 3)) / 16, tc_idesc<false>(C), add);
                        add = true;
                    }
            tc_commit_to(one, bar + B_O);
            tc_commit_to(one, bar + B_EMPTY + it % ST);
            if (ST == 1 && it + 1 < nch) {
                ok = tc_warp_wait(bar + B_FULL, (it + 1) & 1, dead, d.spin);
                if (!ok) break;
                tc_fence_after();
                scores(it + 1);
            }
        }
        __syncwarp();
    } else if (warp == kLinWarps + 1) {
        // ---- the chunks' inputs
        linear_loads<ST>(smem, L::STAGE, bar + B_FULL, bar + B_EMPTY, bar + B_PART, nch, ntok, chunk_at, [&](unsigned char *st, int t0, unsigned long long *full) {
#pragma unroll
            for (int m = 0; m < NP; ++m) {
#pragma unroll
                for (int c = 0; c < KT; ++c) {
                    tc_tensor_load(st + L::Q + (m * KT + c) * TILE, &mq, k0 + 64 * c, tc_coord(a.heads[0], h / p.q.share), t0,
                                   tc_coord(a.seqs[0], b) + m * d.B, full);
                    tc_tensor_load(st + L::K + (m * KT + c) * TILE, &mk, k0 + 64 * c, tc_coord(a.heads[1], h / p.k.share), t0,
                                   tc_coord(a.seqs[1], b) + m * d.B, full);
                }
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    tc_tensor_load(st + L::V + (m * 2 + c) * TILE, &mv, v0 + 64 * c, tc_coord(a.heads[2], h / p.v.share), t0,
                                   tc_coord(a.seqs[2], b) + m * d.B, full);
            }
        }, dead, d.spin);
    } else if (sizeof(OT) == 2) {
        // ---- the bfloat16 results
        for (int it = 0; it < nch; ++it) {
            if (!tc_warp_wait(bar + B_OUT, it & 1, dead, d.spin)) break;
            if (lane == 0) {
                for (int c = 0; c < 2; ++c)
                    if (v0 + 64 * c < p.V)
                        tc_tensor_store(&mo, v0 + 64 * c, h, chunk_at(it) * C, b, smem + it % ST * L::STAGE + L::V + c * TILE);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                mbar_arrive(bar + B_EMPTY + it % ST);
            }
            __syncwarp();
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    if (*dead) {
        // the products issued so far are waited for (the copies were, by their own warp)
        if (tid == 32 * kLinWarps) {
            tc_commit_to(1, bar + B_DRAIN);
            mbar_wait_bounded(bar + B_DRAIN, 0);
            atomicCAS(&a.status->code, 0, (int)SDM_ERR_TIMEOUT);
        }
        __syncthreads();
    }
    tc_fence_before();
    const bool bad = __syncthreads_or(first >= 0);
    if (warp == kLinWarps) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512));
    chain_end(a.chain);
    if (*dead) return;
    if (bad && a.column) {
        const int *at = reinterpret_cast<int *>(smem + L::BAD);
        const float *begin = d.segs > 1 ? a.starts + seg * states : p.first;
        for (int c = warp; c < 128; c += kLinThreads / 32) {
            const int n = at[c], col = v0 + c;
            // a value's NaN leaves no row of the update finite
            if (n < 0 || col >= p.V || at[128 + c] != n || at[256 + c] != n || at[384 + c] != n) continue;
            const int t1 = (n0 + n) * C, t2 = t1 + C < ntok ? t1 + C : ntok;
            using IT = std::conditional_t<NP == 1, __nv_bfloat16, float>;
            linear_column<IT>(d, p, linear_power(a.g[h], 1), b, h, col, n0 * C, t1, t2, begin ? begin + own + col * p.sv : nullptr);
        }
        __syncthreads();
    }
    // Results behind the last chunk are 0: 16 bytes a thread, by all the sequence's segments in turn (one value a
    // thread by its last one: 4 of the 14 us of two sequences of up to 1003 tokens).
    constexpr int PIECE = 16 / (int)sizeof(OT);
    const int pieces = (p.V - v0 < 128 ? p.V - v0 : 128) / PIECE, rows = kLinThreads / pieces, row = tid / pieces;
    const long long step = (long long)d.H * p.V;
    OT *out = static_cast<OT *>(p.out) + (((long long)kb * d.B + b) * d.T * d.H + h) * p.V + v0 + tid % pieces * PIECE;
    if (row < rows)
        for (long long t = (long long)chunks * C + (long long)seg * rows + row; t < d.T; t += (long long)rows * d.segs)
            *reinterpret_cast<uint4 *>(out + t * step) = make_uint4(0, 0, 0, 0);
    float *end = seg + 1 == d.segs ? p.last : nullptr;
    if (warp < kLinWarps && end) {
        const int kk = (warp >> 2) * HD, col = v0 + 32 * (warp & 3) + lane;
        if (col < p.V)
#pragma unroll
            for (int i = 0; i < HD; ++i)
                if (kk + i < K) end[own + (kk + i) * p.sk + col * p.sv] = reinterpret_cast<float *>(S)[i];
    }
}

template <int KP, int NP, bool REV, typename OT>
cudaError_t scan(const LinearDims &d, const LinArgs &a, const CUtensorMap *m, Chain chain, cudaStream_t st) {
    auto kern = k_linear_scan<KP, NP, REV, OT>;
    using L = LinScan<KP, NP>;
    set_kernel_smem(kern, L::BYTES);
    const long long blocks = (long long)d.B * d.H * linear_tiles(a.p.V) * a.p.blocks * d.segs;
    return chain_launch(kern, (unsigned)blocks, kLinThreads, L::BYTES, st, m[0], m[1], m[2], m[3], d, a);
}

template <int KP, int NP>
cudaError_t scan_of(const LinearDims &d, const LinArgs &a, const CUtensorMap *m, Chain chain, cudaStream_t st) {
    using IT = std::conditional_t<NP == 1, __nv_bfloat16, float>;
    if constexpr (NP == 1)
        if (a.p.out_f32) return a.p.reverse ? scan<KP, NP, true, float>(d, a, m, chain, st) : scan<KP, NP, false, float>(d, a, m, chain, st);
    return a.p.reverse ? scan<KP, NP, true, IT>(d, a, m, chain, st) : scan<KP, NP, false, IT>(d, a, m, chain, st);
}

// the operands as the tensor copies take them: float32 ones as three bfloat16 planes, the others contiguous
struct LayTable {
    const void *src[4];
    __nv_bfloat16 *dst[4];
    long long s[4][3];
    int heads[4], width[4];
};
// The status block alone. A memset of it would not let the next launch start: 64 tokens of 16 heads 12.5 us in a graph, so 9.4,
// 200 tokens 18.6 and 15.2.
__global__ void k_linear_clear(DevStatus *status) {
    chain_next();
    if (threadIdx.x == 0) *status = DevStatus{};
}
template <typename T>
__global__ void __launch_bounds__(256) k_linear_lay(const __grid_constant__ LayTable t, int B, int T_, DevStatus *status) {
    chain_next();
    if (blockIdx.x + blockIdx.y + threadIdx.x == 0) *status = DevStatus{};
    const int w = blockIdx.y, heads = t.heads[w], width = t.width[w];
    const T *x = static_cast<const T *>(t.src[w]);
    const long long all = (long long)B * T_ * heads * (width / 8);
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
        const long long row = i / (width / 8), h = row % heads, bt = row / heads, at = bt % T_, b = bt / T_;
        const T *src = x + b * t.s[w][0] + at * t.s[w][1] + h * t.s[w][2] + i % (width / 8) * 8;
        if constexpr (sizeof(T) == 2) {
            reinterpret_cast<uint4 *>(t.dst[w])[i] = *reinterpret_cast<const uint4 *>(src);
        } else {
            float f[8];
            load_vec<float, 8, true>(src, f);
            unsigned pl[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                unsigned s[3];
                split_bf16<3>(f[2 * e], f[2 * e + 1], s);
                pl[0][e] = s[0]; pl[1][e] = s[1]; pl[2][e] = s[2];
            }
#pragma unroll
            for (int m = 0; m < 3; ++m)
                reinterpret_cast<uint4 *>(t.dst[w])[m * all + i] = make_uint4(pl[m][0], pl[m][1], pl[m][2], pl[m][3]);
        }
    }
}

}  // namespace

cudaError_t launch_linear_scan(const LinearDims &d, const LinearPass &p, const LinearIn &in, const LinearLaid (&laid)[3], const float *starts, void *status,
                               Chain chain, cudaStream_t st) {
    const int np = d.dtype == SDM_F32 ? 3 : 1;
    LinArgs a{p, in.g, in.valid, starts, static_cast<DevStatus *>(status), {}, {}, p.last != nullptr && !p.reverse, chain};
    CUtensorMap m[4];
    for (int i = 0; i < 3; ++i) {
        const cudaError_t e = tc_tensor_map(m + i, laid[i].p, laid[i].s, np * d.B, d.T, laid[i].heads, laid[i].width);
        if (e != cudaSuccess) return e;
        a.seqs[i] = laid[i].s[0];
        a.heads[i] = laid[i].s[2];
    }
    m[3] = m[2];                                                    // (of bfloat16 results alone)
    if (np == 1 && !p.out_f32) {
        const long long os[3] = {(long long)d.T * d.H * p.V, (long long)d.H * p.V, p.V};
        const cudaError_t e = tc_tensor_map(m + 3, p.out, os, d.B, d.T, d.H, p.V);
        if (e != cudaSuccess) return e;
    }
    const bool wide = p.K > 64;
    if (np == 1) return wide ? scan_of<128, 1>(d, a, m, chain, st) : scan_of<64, 1>(d, a, m, chain, st);
    return wide ? scan_of<128, 3>(d, a, m, chain, st) : scan_of<64, 3>(d, a, m, chain, st);
}

cudaError_t launch_linear_lay(const LinearDims &d, const LinearLay *lay, int n, DevStatus *status, cudaStream_t st) {
    if (n == 0) {
        k_linear_clear<<<1, 32, 0, st>>>(status);
        return cudaGetLastError();
    }
    LayTable t{};
    long long most = 0;
    for (int i = 0; i < n; ++i) {
        t.src[i] = lay[i].src;
        t.dst[i] = static_cast<__nv_bfloat16 *>(lay[i].dst);
        for (int j = 0; j < 3; ++j) t.s[i][j] = lay[i].s[j];
        t.heads[i] = lay[i].heads;
        t.width[i] = lay[i].width;
        const long long units = (long long)d.B * d.T * lay[i].heads * (lay[i].width / 8);
        most = units > most ? units : most;
    }
    const long long want = (most + 255) / 256;
    const dim3 grid((unsigned)(want < 8 * kRefSms ? want : 8 * kRefSms), n);
    if (d.dtype == SDM_F32) k_linear_lay<float><<<grid, 256, 0, st>>>(t, d.B, d.T, status);
    else k_linear_lay<__nv_bfloat16><<<grid, 256, 0, st>>>(t, d.B, d.T, status);
    return cudaGetLastError();
}

}  // namespace sdm
