// Linear attention's sequences in segments: what each segment adds to the state (a carry), and from that the states
// that they begin with (a join). With L the head's log-decay, over a chunk of n tokens
//   S = e^{L n} S + (e^{L (n - 1 - j)} K)^T V         (mirrored, for the gradient of the state: e^{L (j + 1)})
// on the 5th-generation tensor cores. The rows of the state are the lanes of tensor memory: the decayed keys, three
// bfloat16 planes, are an A operand there, which the threads of their lanes store; V is the B operand in shared memory.
// S stays in registers in float32. Two buffers of decayed keys and of products, four stages of inputs, float32 inputs as
// three planes with six of their products (NP = 3). Warps 0..15 compute (lanes 32 (warp % 4).., quarter warp / 4 of the
// tokens and of the columns), warp 16 issues the products, warp 17 loads.
//
// Bound by the threads' work (the issue of instructions is busy 59 % of its cycles, the tensor pipe 47 %): splitting the decayed
// keys in three planes and adding a product to the state, 0.86 us a chunk, near the copies' own time. 16384 tokens, 32 heads of 128 x 128, three of four segments:
// 55 us on 96 SMs, where the copies alone, as deep, take 42 (4.7 TB/s). Warps that take even and odd chunks instead of
// quarters of each 65.6 (63 then), the copies awaited one after the other 80.
#include <type_traits>

#include "linear_tc.cuh"

namespace sdm {
namespace {

constexpr int kCarC = 64, kCarWarps = 16, kCarThreads = 32 * (kCarWarps + 2);

template <int KP, int NP>
struct LinCarry {
    static constexpr int TILE = kCarC * 128, KT = KP / 64;
    static constexpr int K = 0, V = K + NP * KT * TILE, STAGE = V + NP * 2 * TILE, STAGES = NP == 1 ? 4 : 2;
    static constexpr int POW = STAGES * STAGE, WEIGHT = POW + 4 * 80, BARS = WEIGHT + 4 * 64, BYTES = BARS + 256 + 1024;
    static_assert(BYTES <= 227 * 1024, "shared memory");
    static constexpr int U = 0, KX = 256;                          // columns: two products of 128, two buffers of 3 x 32
};

enum { C_FULL = 0, C_EMPTY = 4, C_KX = 8, C_U = 10, C_UF = 12, C_PART = 14, C_DRAIN, C_COUNT };

struct CarryArgs {
    const float *g;
    const int32_t *valid;
    float *starts;                       // [segs][B, H, Dk, Dv]
    DevStatus *status;
    long long heads[2], seqs[2];         // of the laid keys and values, 0: broadcast
    int kshare, vshare, K, V;
    float to;
    Chain chain;
};

template <int KP, int NP, bool REV>
__global__ void __launch_bounds__(kCarThreads, 1)
    k_linear_carry(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const __grid_constant__ LinearDims d,
                   const __grid_constant__ CarryArgs a) {
    using L = LinCarry<KP, NP>;
    constexpr int C = kCarC, ST = L::STAGES, KT = L::KT, TILE = L::TILE;
    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    auto bar = reinterpret_cast<unsigned long long *>(smem + L::BARS);
    volatile int *dead = reinterpret_cast<int *>(bar + C_COUNT);
    auto slot = reinterpret_cast<uint32_t *>(bar + C_COUNT + 1);
    float *pw = reinterpret_cast<float *>(smem + L::POW);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    unsigned at_block = blockIdx.x;
    const int tiles = (a.V + 127) / 128;
    const int tile = (int)(at_block % tiles);
    at_block /= tiles;
    const int h = (int)(at_block % d.H);
    at_block /= d.H;
    const int b = linear_longest_first(d, a.valid, (int)(at_block % d.B)), seg = (int)(at_block / d.B);   // seg: in the pass's order
    const int v0 = tile * 128;
    const int ntok = linear_valid(a.valid, b, d.T), chunks = (ntok + C - 1) / C;
    const int place = REV ? d.segs - 1 - seg : seg;
    const int n0 = linear_cut(chunks, place, d.segs), nch = linear_cut(chunks, place + 1, d.segs) - n0;

    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(bar + C_FULL + i, 1);
            mbar_init(bar + C_EMPTY + i, 1);
        }
        for (int i = C_KX; i < C_COUNT; ++i) mbar_init(bar + i, i < C_U || i == C_UF || i == C_UF + 1 ? kCarWarps : 1);
        fence_mbar_init();
    }
    if (warp == kCarWarps) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    float *weight = reinterpret_cast<float *>(smem + L::WEIGHT);   // of a whole chunk's tokens
    if (tid <= C) {
        const float x = linear_power(a.g[h], tid);
        pw[tid] = x;
        if (REV ? tid > 0 : tid < C) weight[REV ? tid - 1 : C - 1 - tid] = a.to * x;
    }
    chain_begin(a.chain);
    if (tid == 0) *dead = tc_gives_up(d.spin) || __ldcg(&a.status->code) != 0;   // an earlier kernel of this call gave up
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *slot;
    auto chunk_at = [&](int it) { return REV ? n0 + nch - 1 - it : n0 + it; };

    if (warp < kCarWarps) {
        const int part = warp >> 2, lane0 = 32 * (warp & 3), row = lane0 + lane, col = v0 + 32 * part;
        const uint32_t at = tm + ((uint32_t)lane0 << 16);
        float2 S[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) S[i] = make_float2(0.f, 0.f);
        auto arrive = [&](int which) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + which);
        };
        // this lane's 16 decayed keys of chunk `it`; lanes past the keys' width (KP = 64) hold what is never looked at
        auto keys = [&](int it) {
            const int n = chunk_at(it), nt = ntok - n * C < C ? ntok - n * C : C;
            if (!tc_warp_wait(bar + C_FULL + it % ST, it / ST & 1, dead, d.spin)) return false;
            if (lane0 < KP) {
                // column `row` of the tile: 2 bytes of each token's 128, pieces of 8 exchanged by token (tc_at)
                const unsigned char *src = smem + it % ST * L::STAGE + L::K + (row >> 6) * TILE + 2 * (row & 7) + 16 * part * 128;
                const int piece = (row & 63) >> 3;
                float2 x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float y[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        y[e] = 0.f;
#pragma unroll
                        for (int m = NP - 1; m >= 0; --m) {
                            const float k = __uint_as_float((unsigned)*reinterpret_cast<const unsigned short *>(
                                                                src + m * KT * TILE + (2 * i + e) * 128 + ((piece ^ ((2 * i + e) & 7)) << 4)) << 16);
                            y[e] = m == NP - 1 ? k : y[e] + k;
                        }
                    }
                    x[i] = make_float2(y[0], y[1]);
                }
                if (nt == C) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 w = *reinterpret_cast<const float4 *>(weight + 16 * part + 4 * i);
                        x[2 * i] = mul2(x[2 * i], make_float2(w.x, w.y));
                        x[2 * i + 1] = mul2(x[2 * i + 1], make_float2(w.z, w.w));
                    }
                } else {
                    auto of = [&](int t) { return t < nt ? a.to * pw[REV ? t + 1 : nt - 1 - t] : 0.f; };
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], make_float2(of(16 * part + 2 * i), of(16 * part + 2 * i + 1)));
                }
                const uint32_t dst = at + L::KX + 96 * (it & 1) + 8 * part;
                store_planes3(dst, dst + 32, dst + 64, x);
                tc_wait_st();
            }
            arrive(C_KX + (it & 1));
            return true;
        };
        bool ok = nch > 0 && keys(0);
        for (int it = 0; ok && it < nch; ++it) {
            const int n = chunk_at(it), nt = ntok - n * C < C ? ntok - n * C : C;
            if (it + 1 < nch && !(ok = keys(it + 1))) break;
            if (!(ok = tc_warp_wait(bar + C_U + (it & 1), it >> 1 & 1, dead, d.spin))) break;
            tc_fence_after();
            const float whole = pw[nt];
#pragma unroll
            for (int c = 0; c < 32; c += 16) {
                float2 x[8];
                tc_load16(at + L::U + 128 * (it & 1) + 32 * part + c, reinterpret_cast<float(&)[16]>(x));
#pragma unroll
                for (int i = 0; i < 8; ++i) S[c / 2 + i] = fma2(make_float2(whole, whole), S[c / 2 + i], x[i]);
            }
            arrive(C_UF + (it & 1));
        }
        if (row < a.K && !*dead) {
            float *end = a.starts + (seg + 1) * ((long long)d.B * d.H * d.Dk * d.Dv) + (((long long)b * d.H + h) * d.Dk + row) * d.Dv + col;
#pragma unroll
            for (int i = 0; i < 8; ++i)                            // (the columns are a multiple of 16)
                if (col + 4 * i < a.V) *reinterpret_cast<float4 *>(end + 4 * i) = make_float4(S[2 * i].x, S[2 * i].y, S[2 * i + 1].x, S[2 * i + 1].y);
        }
    } else if (warp == kCarWarps) {
        // ---- the products
        const uint32_t one = tc_elect(), tu = __shfl_sync(~0u, tm, 0), base = __shfl_sync(~0u, smem_u32(smem), 0);
        for (int it = 0; it < nch; ++it) {
            const uint32_t vn = tc_n_major(base + it % ST * L::STAGE + L::V, TILE), kx = tu + L::KX + 96 * (it & 1);
            const bool ok = tc_warp_wait(bar + C_FULL + it % ST, it / ST & 1, dead, d.spin) &&
                            tc_warp_wait(bar + C_KX + (it & 1), it >> 1 & 1, dead, d.spin) &&
                            (it < 2 || tc_warp_wait(bar + C_UF + (it & 1), (it >> 1 & 1) ^ 1, dead, d.spin));
            if (!ok) break;
            tc_fence_after();
            // sums from their smallest terms up: the tensor core cuts an accumulator's low bits at every step
            bool add = false;
#pragma unroll
            for (int sum = 2; sum >= 0; --sum)
#pragma unroll
                for (int m = sum < NP - 1 ? sum : NP - 1; m >= 0; --m)
#pragma unroll
                    for (int ks = 0; ks < C / 16; ++ks) {
                        tc_mma_ts(one, tu + L::U + 128 * (it & 1), kx + 32 * (sum - m) + 8 * ks, vn + (m * 2 * TILE + 2048 * ks) / 16,
                                  tc_idesc<true>(128), add);
                        add = true;
                    }
            tc_commit_to(one, bar + C_U + (it & 1));
            tc_commit_to(one, bar + C_EMPTY + it % ST);
        }
        __syncwarp();
    } else {
        // ---- the chunks' inputs
        linear_loads<ST>(smem, L::STAGE, bar + C_FULL, bar + C_EMPTY, bar + C_PART, nch, ntok, chunk_at, [&](unsigned char *st, int t0, unsigned long long *full) {
#pragma unroll
            for (int m = 0; m < NP; ++m) {
#pragma unroll
                for (int c = 0; c < KT; ++c)
                    tc_tensor_load(st + L::K + (m * KT + c) * TILE, &mk, 64 * c, tc_coord(a.heads[0], h / a.kshare), t0,
                                   tc_coord(a.seqs[0], b) + m * d.B, full);
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    tc_tensor_load(st + L::V + (m * 2 + c) * TILE, &mv, v0 + 64 * c, tc_coord(a.heads[1], h / a.vshare), t0,
                                   tc_coord(a.seqs[1], b) + m * d.B, full);
            }
        }, dead, d.spin);
    }
    __syncthreads();
    if (*dead) {
        // the products issued so far are waited for (the copies were, by their own warp)
        if (tid == 32 * kCarWarps) {
            tc_commit_to(1, bar + C_DRAIN);
            mbar_wait_bounded(bar + C_DRAIN, 0);
            atomicCAS(&a.status->code, 0, (int)SDM_ERR_TIMEOUT);
        }
        __syncthreads();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kCarWarps) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512));
    chain_end(a.chain);
}

// starts [segs]: the state itself, then each segment's first state from the one before and what the carry left
__global__ void __launch_bounds__(256) k_linear_join(const __grid_constant__ LinearDims d, const float *g, const int32_t *valid, const float *first,
                                                     bool reverse, float *starts) {
    const long long cells = (long long)d.Dk * d.Dv, states = cells * d.B * d.H;
    const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= states) return;
    const long long bh = i / cells;
    const int b = (int)(bh / d.H), h = (int)(bh % d.H);
    const int ntok = linear_valid(valid, b, d.T), chunks = (ntok + d.C - 1) / d.C;
    auto bound = [&](int n) {
        const int t = linear_cut(chunks, n, d.segs) * d.C;
        return t < ntok ? t : ntok;
    };
    const float decay = g[h];
    chain_begin(Chain::behind);
    float4 s = first ? make_float4(first[i], first[i + 1], first[i + 2], first[i + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<float4 *>(starts + i) = s;
    // what the segments add is fetched eight at a time: one by one each waits for memory (16 segments 10 us)
    for (int m0 = 1; m0 < d.segs; m0 += 8) {
        float4 e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (m0 + j < d.segs) e[j] = *reinterpret_cast<const float4 *>(starts + (m0 + j) * states + i);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int m = m0 + j;
            if (m >= d.segs) break;
            const int place = reverse ? d.segs - m : m - 1;        // of the segment before
            const float w = linear_power(decay, bound(place + 1) - bound(place));
            s = make_float4(fmaf(w, s.x, e[j].x), fmaf(w, s.y, e[j].y), fmaf(w, s.z, e[j].z), fmaf(w, s.w, e[j].w));
            *reinterpret_cast<float4 *>(starts + m * states + i) = s;
        }
    }
}

template <int KP, int NP, bool REV>
cudaError_t carry(const LinearDims &d, const CarryArgs &a, const CUtensorMap *m, Chain chain, cudaStream_t st) {
    using L = LinCarry<KP, NP>;
    set_kernel_smem(k_linear_carry<KP, NP, REV>, L::BYTES);
    const long long blocks = (long long)d.B * d.H * linear_tiles(a.V) * (d.segs - 1);
    return chain_launch(k_linear_carry<KP, NP, REV>, (unsigned)blocks, kCarThreads, L::BYTES, st, m[0], m[1], d, a);
}

}  // namespace

// k, v: those of a pass along the state's rows (p.sv = 1)
cudaError_t launch_linear_carry(const LinearDims &d, const LinearPass &p, const LinearIn &in, const LinearLaid &k, const LinearLaid &v,
                                float *starts, void *status, Chain chain, cudaStream_t st) {
    const int np = d.dtype == SDM_F32 ? 3 : 1;
    const CarryArgs a{in.g, in.valid, starts, static_cast<DevStatus *>(status), {k.s[2], v.s[2]}, {k.s[0], v.s[0]}, p.k.share, p.v.share, p.K, p.V, p.to, chain};
    CUtensorMap m[2];
    cudaError_t e = tc_tensor_map(m, k.p, k.s, np * d.B, d.T, k.heads, k.width);
    if (e == cudaSuccess) e = tc_tensor_map(m + 1, v.p, v.s, np * d.B, d.T, v.heads, v.width);
    if (e != cudaSuccess) return e;
    auto go = [&](auto kp, auto planes) {
        constexpr int KP = decltype(kp)::value, NP = decltype(planes)::value;
        return p.reverse ? carry<KP, NP, true>(d, a, m, chain, st) : carry<KP, NP, false>(d, a, m, chain, st);
    };
    using std::integral_constant;
    if (np == 1) e = p.K > 64 ? go(integral_constant<int, 128>{}, integral_constant<int, 1>{}) : go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else e = p.K > 64 ? go(integral_constant<int, 128>{}, integral_constant<int, 3>{}) : go(integral_constant<int, 64>{}, integral_constant<int, 3>{});
    if (e != cudaSuccess) return e;
    const long long blocks = (linear_states(d) / 4 + 255) / 256;
    return chain_launch(k_linear_join, (unsigned)blocks, 256, 0, st, d, in.g, in.valid, p.first, p.reverse, starts);
}

}  // namespace sdm
