// The gradient of linear attention's decays. With G = dS / dL carried along beside a head's state S (L its
// log-decay), a chunk of n tokens that begins with (S, G) adds, with i, j its tokens,
//   sum_{j < i} (i - j) e^{L (i - j)} (q_i . k_j) (do_i . v_j) + <S, A'> + <G, A>
//   A  = sum_i e^{L (i + 1)} q_i do_i^T,   A' = sum_i (i + 1) e^{L (i + 1)} q_i do_i^T
// (times scale) and goes on with
//   G = e^{L n} (G + n S) + W',  W' = sum_j (n - 1 - j) e^{L (n - 1 - j)} k_j v_j^T
//   S = e^{L n} S + W,           W  = sum_j e^{L (n - 1 - j)} k_j v_j^T
// Every term carries its own decay, so none is a difference of larger ones. A segment begins with the state that
// the forward kept and G = 0, and ends with <G, R>, R the gradient of the state there.
//
// S and G stay in registers in float32, transposed: 128 of Dv's columns are the lanes of tensor memory. dO^T and V^T are
// A operands in shared memory, the queries and keys with both their weights, three bfloat16 planes each, one B operand:
// A and A' come from one product, W and W' from the next. All is bilinear in (Dk, Dv), so a block takes 64 columns of Dk
// and 128 of Dv for itself, the pairs' sums too: it has room for a buffer of queries and one of keys, so that the threads
// fill one (what they and the products take is shared memory's rate) while the other is multiplied. 64 heads of 128 x 128
// x 64 chunks: 139 us; 128 columns of Dk a block, with one buffer, 157; four products instead of two 188. A chunk takes
// 3450 cycles, of which shared memory is busy 3390 (operands of the products 2110, their buffers 900, copies 380).
// Warps as in linear_scan_tc.cu.
#include <type_traits>

#include "linear_tc.cuh"

namespace sdm {
namespace {

constexpr int kDecC = 64, kDecWarps = 16, kDecThreads = 32 * (kDecWarps + 2);

template <int NP>
struct LinDecay {
    static constexpr int KP = 64, TILE = kDecC * 128;
    // (a product's A operand of 128 rows reads on past the 64 of Q and dO: into what follows them)
    static constexpr int Q = 0, G = Q + NP * TILE, K = G + NP * 2 * TILE, V = K + NP * TILE, STAGE = V + NP * 2 * TILE;
    static constexpr int STAGES = NP == 1 ? 2 : 1, BUFS = NP == 1 ? 2 : 1;
    static constexpr int BUF = STAGES * STAGE, PLANE = 2 * TILE, BUFFER = 3 * PLANE, AUX = BUF + BUFS * BUFFER;   // [plane][weight]
    static constexpr int POW = AUX, PAIR = POW + 4 * 80, SUMS = PAIR + 4 * 128, BARS = SUMS + 8 * kDecWarps, BYTES = BARS + 256 + 1024;
    static_assert(BYTES <= 227 * 1024, "shared memory");
    static constexpr int A = 0, A1 = KP, W = 2 * KP, W1 = 3 * KP, PQ = 4 * KP, PG = PQ + 64;   // A', W' behind A and W; the pairs' products
};

enum { D_FULL = 0, D_EMPTY = 2, D_MUL = 4, D_CONV = 6, D_PAIR = 8, D_READ, D_PART, D_DRAIN, D_COUNT };

struct DecayArgs {
    const float *g;
    const int32_t *valid;
    const float *starts, *ends;          // [segs] states, in order; gradients of the ends, from the last (segs == 1: null: 0)
    double *part;
    DevStatus *status;
    long long heads[4], seqs[4];         // q, k, v, grad: strides of the laid operands, 0: broadcast
    int share, kblocks;
    Chain chain;
};

template <int NP>
__global__ void __launch_bounds__(kDecThreads, 1)
    k_linear_decay(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                   const __grid_constant__ CUtensorMap mg, const __grid_constant__ LinearDims d, const __grid_constant__ DecayArgs a) {
    using L = LinDecay<NP>;
    constexpr int C = kDecC, KP = L::KP, HD = KP / 4, ST = L::STAGES, TILE = L::TILE;
    constexpr bool TWO = L::BUFS == 2;
    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    auto bar = reinterpret_cast<unsigned long long *>(smem + L::BARS);
    volatile int *dead = reinterpret_cast<int *>(bar + D_COUNT);
    auto slot = reinterpret_cast<uint32_t *>(bar + D_COUNT + 1);
    float *pw = reinterpret_cast<float *>(smem + L::POW);
    double *sums = reinterpret_cast<double *>(smem + L::SUMS);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    unsigned at_block = blockIdx.x;
    const int tiles = (d.Dv + 127) / 128;
    const int tile = (int)(at_block % tiles);
    at_block /= tiles;
    const int kb = (int)(at_block % a.kblocks);
    at_block /= a.kblocks;
    const int seg = (int)(at_block % d.segs);
    const long long bh = at_block / d.segs;
    const int b = (int)(bh / d.H), h = (int)(bh % d.H);
    const int v0 = tile * 128, k0 = kb * KP;
    const int ntok = linear_valid(a.valid, b, d.T), chunks = (ntok + C - 1) / C;
    const int n0 = linear_cut(chunks, seg, d.segs), nch = linear_cut(chunks, seg + 1, d.segs) - n0;
    const long long states = (long long)d.B * d.H * d.Dk * d.Dv;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar + D_FULL + i, 1);
            mbar_init(bar + D_EMPTY + i, 1);
        }
        for (int i = D_MUL; i < D_COUNT; ++i)
            mbar_init(bar + i, (i >= D_CONV && i < D_PAIR) || i == D_READ ? kDecWarps : 1);
        fence_mbar_init();
    }
    if (warp == kDecWarps) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    float *pair = reinterpret_cast<float *>(smem + L::PAIR);
    if (tid < 128) {
        // e^{L n}, and n e^{L n} of tokens n apart (0 before)
        const int n = tid < C ? C - tid : tid - C;
        const float x = linear_power(a.g[h], n);
        pw[n] = x;
        if (tid == C) pw[0] = 1.f;
        pair[tid] = tid < C ? 0.f : (float)n * x;
    }
    chain_begin(a.chain);
    if (tid == 0) *dead = tc_gives_up(d.spin) || __ldcg(&a.status->code) != 0;   // an earlier kernel of this call gave up
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *slot;

    if (warp < kDecWarps) {
        const int part = warp >> 2, lane0 = 32 * (warp & 3), col = v0 + lane0 + lane, kk = part * HD;
        const bool mine = col < d.Dv;
        const uint32_t at = tm + ((uint32_t)lane0 << 16);
        const long long own = bh * d.Dk * d.Dv + (long long)(k0 + kk) * d.Dv + col;
        float S[HD], G[HD];
        // the sum so far and what its roundings lost: a double addition takes a warp 16 cycles of the SM
        float acc = 0.f, lost = 0.f;
        auto add = [&](float x) {
            const float sum = acc + x, of_x = sum - acc;
            lost += (acc - (sum - of_x)) + (x - of_x);
            acc = sum;
        };
        const float *begin = a.starts + seg * states + own;
#pragma unroll
        for (int i = 0; i < HD; ++i) {
            S[i] = mine && k0 + kk + i < d.Dk && nch > 0 ? __ldcg(begin + (long long)i * d.Dv) : 0.f;
            G[i] = 0.f;
        }
        auto arrive = [&](int which) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + which);
        };
        auto wait = [&](int which, int it) {
            const bool there = tc_warp_wait(bar + which, it & 1, dead, d.spin);
            tc_fence_after();
            return there;
        };
        // rows of Q or K times their two weights, as planes: a piece of 8 columns a thread
        static_assert(C * KP / 8 == 32 * kDecWarps, "one piece a thread");
        auto convert = [&](const unsigned char *src, unsigned char *dst, auto weights) {
            const int row = tid % C, off = tc_at(row, tid / C);
            const float2 w = weights(row);
            float2 x[4];
            load_piece<NP, TILE>(src + off, x);
            scale_piece(x, w.x, dst + off, L::PLANE);
            scale_piece(x, w.y, dst + TILE + off, L::PLANE);
            fence_proxy_async_smem();
        };
        // <this thread's part of the state, a product>
        auto dot = [&](int where, const float (&s)[HD]) {
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
                float x[16];
                tc_load16(at + where + kk + c, x);
#pragma unroll
                for (int i = 0; i < 16; ++i) sum = fmaf(s[c + i], x[i], sum);
            }
            if (mine) add(sum);
        };
        // s = w s + a product
        auto advance = [&](int where, float w, float (&s)[HD]) {
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
                float x[16];
                tc_load16(at + where + kk + c, x);
#pragma unroll
                for (int i = 0; i < 16; ++i) s[c + i] = fmaf(w, s[c + i], x[i]);
            }
        };
        float whole = 1.f;
        bool ok = true;
        unsigned char *buf = smem + L::BUF, *keys = buf + (TWO ? L::BUFFER : 0);
        for (int it = 0; it < nch; ++it) {
            const int nt = ntok - (n0 + it) * C < C ? ntok - (n0 + it) * C : C;
            const unsigned char *st = smem + it % ST * L::STAGE;
            ok = tc_warp_wait(bar + D_FULL + it % ST, it / ST & 1, dead, d.spin) && (TWO || it == 0 || wait(D_MUL + 1, it - 1));
            if (!ok) break;
            convert(st + L::Q, buf, [&](int t) {                   // (the product before from this buffer was waited for)
                const float w = t < nt ? d.scale * pw[t + 1] : 0.f;
                return make_float2(w, (float)(t + 1) * w);
            });
            arrive(D_CONV);
            if (it > 0) {
                if (TWO && !(ok = wait(D_MUL + 1, it - 1))) break;
                advance(L::W, whole, S);
                advance(L::W1, 1.f, G);
            }
            if (!TWO && !(ok = wait(D_MUL, it))) break;
            convert(st + L::K, keys, [&](int t) {
                const float w = t < nt ? pw[nt - 1 - t] : 0.f;
                return make_float2(w, (float)(nt - 1 - t) * w);
            });
            arrive(D_CONV + 1);
            // the pairs: a token's row each of lanes 0..63
            if (!(ok = wait(D_PAIR, it))) break;
            if ((warp & 3) < 2) {
                const float *apart = pair + C + lane0 + lane - 16 * part;
                float x[16], y[16], sum = 0.f;
                tc_load16(at + L::PQ + 16 * part, x);
                tc_load16(at + L::PG + 16 * part, y);
#pragma unroll
                for (int i = 0; i < 16; ++i) sum = fmaf(apart[-i] * x[i], y[i], sum);
                add(d.scale * sum);
            }
            arrive(D_READ);
            if (TWO && !(ok = wait(D_MUL, it))) break;
            dot(L::A, G);
            dot(L::A1, S);
            whole = pw[nt];
#pragma unroll
            for (int i = 0; i < HD; ++i) G[i] = whole * fmaf((float)nt, S[i], G[i]);
        }
        if (ok && nch > 0 && wait(D_MUL + 1, nch - 1)) {
            advance(L::W1, 1.f, G);
            if (a.ends && mine) {
                const float *end = a.ends + (d.segs - 1 - seg) * states + own;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < HD; ++i)
                    if (k0 + kk + i < d.Dk) sum = fmaf(G[i], __ldcg(end + (long long)i * d.Dv), sum);
                add(sum);
            }
        }
        double all = (double)acc + (double)lost;
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) all += __shfl_xor_sync(~0u, all, m);
        if (lane == 0) sums[warp] = all;
    } else if (warp == kDecWarps) {
        // ---- the products
        const uint32_t one = tc_elect(), tu = __shfl_sync(~0u, tm, 0), base = __shfl_sync(~0u, smem_u32(smem), 0);
        // [64 tokens] x [64 tokens] over `steps` of the width, NP planes each
        auto scores = [&](uint32_t dst, uint32_t x, uint32_t y, auto tiles_of) {
            constexpr int TL = decltype(tiles_of)::value;
            bool add = false;
#pragma unroll
            for (int sum = NP - 1; sum >= 0; --sum)
#pragma unroll
                for (int m = sum; m >= 0; --m)
#pragma unroll
                    for (int ks = 0; ks < 4 * TL; ++ks) {
                        const int off = ((ks >> 2) * TILE + 32 * (ks & 3)) / 16;
                        tc_mma_ss(one, dst, x + m * TL * TILE / 16 + off, y + (sum - m) * TL * TILE / 16 + off, tc_idesc<false>(C), add);
                        add = true;
                    }
        };
        auto pairs = [&](int it) {
            const uint32_t st = base + it % ST * L::STAGE;
            scores(tu + L::PQ, tc_k_major(st + L::Q), tc_k_major(st + L::K), std::integral_constant<int, 1>{});
            scores(tu + L::PG, tc_k_major(st + L::G), tc_k_major(st + L::V), std::integral_constant<int, 2>{});
            tc_commit_to(one, bar + D_PAIR);
        };
        auto product = [&](uint32_t dst, uint32_t vm, uint32_t kn) {
            bool add = false;
#pragma unroll
            for (int sum = 2; sum >= 0; --sum)
#pragma unroll
                for (int m = sum < NP - 1 ? sum : NP - 1; m >= 0; --m)
#pragma unroll
                    for (int ks = 0; ks < C / 16; ++ks) {
                        tc_mma_ss(one, dst, vm + (m * 2 * TILE + 2048 * ks) / 16, kn + ((sum - m) * L::PLANE + 2048 * ks) / 16,
                                  tc_idesc<true, true>(2 * KP), add);
                        add = true;
                    }
        };
        bool ok = nch > 0 && tc_warp_wait(bar + D_FULL, 0, dead, d.spin);
        tc_fence_after();
        if (ok) pairs(0);
        for (int it = 0; ok && it < nch; ++it) {
            const uint32_t st = base + it % ST * L::STAGE;
            const unsigned par = it & 1;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ok = ok && tc_warp_wait(bar + D_CONV + i, par, dead, d.spin);
                if (!ok) break;
                tc_fence_after();
                product(tu + (i == 0 ? L::A : L::W), tc_n_major(st + (i == 0 ? L::G : L::V), TILE), tc_n_major(base + L::BUF + (TWO ? i : 0) * L::BUFFER, TILE));
                tc_commit_to(one, bar + D_MUL + i);
            }
            if (!ok) break;
            tc_commit_to(one, bar + D_EMPTY + it % ST);
            if (it + 1 < nch) {
                ok = tc_warp_wait(bar + D_FULL + (it + 1) % ST, (it + 1) / ST & 1, dead, d.spin) && tc_warp_wait(bar + D_READ, par, dead, d.spin);
                if (!ok) break;
                tc_fence_after();
                pairs(it + 1);
            }
        }
        __syncwarp();
    } else {
        // ---- the chunks' inputs
        const int hk = h / a.share;
        linear_loads<ST>(smem, L::STAGE, bar + D_FULL, bar + D_EMPTY, bar + D_PART, nch, ntok, [&](int it) { return n0 + it; },
                         [&](unsigned char *st, int t0, unsigned long long *full) {
#pragma unroll
            for (int m = 0; m < NP; ++m) {
                tc_tensor_load(st + L::Q + m * TILE, &mq, k0, tc_coord(a.heads[0], hk), t0, tc_coord(a.seqs[0], b) + m * d.B, full);
                tc_tensor_load(st + L::K + m * TILE, &mk, k0, tc_coord(a.heads[1], hk), t0, tc_coord(a.seqs[1], b) + m * d.B, full);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    tc_tensor_load(st + L::G + (m * 2 + c) * TILE, &mg, v0 + 64 * c, tc_coord(a.heads[3], h), t0, tc_coord(a.seqs[3], b) + m * d.B, full);
                    tc_tensor_load(st + L::V + (m * 2 + c) * TILE, &mv, v0 + 64 * c, tc_coord(a.heads[2], h), t0, tc_coord(a.seqs[2], b) + m * d.B, full);
                }
            }
        }, dead, d.spin);
    }
    __syncthreads();
    if (*dead) {
        // the products issued so far are waited for (the copies were, by their own warp)
        if (tid == 32 * kDecWarps) {
            tc_commit_to(1, bar + D_DRAIN);
            mbar_wait_bounded(bar + D_DRAIN, 0);
            atomicCAS(&a.status->code, 0, (int)SDM_ERR_TIMEOUT);
        }
        __syncthreads();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kDecWarps) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512));
    if (tid == 0) {
        double s = 0.0;
        for (int i = 0; i < kDecWarps; ++i) s += sums[i];
        a.part[blockIdx.x] = s;
    }
    chain_end(a.chain);
}

// a head's parts of all sequences, in a fixed order; a warp a head
__global__ void __launch_bounds__(32) k_linear_decay_sum(const double *part, int B, int H, int each, float *out, Chain chain) {
    chain_begin(chain);
    const int h = blockIdx.x;
    double s = 0.0;
    for (long long i = threadIdx.x; i < (long long)B * each; i += 32) s += __ldcg(part + (i / each * H + h) * each + i % each);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(~0u, s, m);
    if (threadIdx.x == 0) out[h] = (float)s;
    chain_end(chain);
}

template <int NP>
cudaError_t decay(const LinearDims &d, const DecayArgs &a, const CUtensorMap *m, cudaStream_t st) {
    using L = LinDecay<NP>;
    set_kernel_smem(k_linear_decay<NP>, L::BYTES);
    return chain_launch(k_linear_decay<NP>, (unsigned)linear_decay_parts(d), kDecThreads, L::BYTES, st, m[0], m[1], m[2], m[3], d, a);
}

}  // namespace

cudaError_t launch_linear_decay(const LinearDims &d, const LinearIn &in, const LinearLaid (&laid)[4], const float *starts, const float *ends,
                                double *part, void *status, Chain chain, cudaStream_t st) {
    const int np = d.dtype == SDM_F32 ? 3 : 1;
    DecayArgs a{in.g, in.valid, starts, ends, part, static_cast<DevStatus *>(status), {}, {}, d.H / d.Hk, linear_decay_blocks(d), chain};
    CUtensorMap m[4];
    for (int i = 0; i < 4; ++i) {
        const cudaError_t e = tc_tensor_map(m + i, laid[i].p, laid[i].s, np * d.B, d.T, laid[i].heads, laid[i].width);
        if (e != cudaSuccess) return e;
        a.seqs[i] = laid[i].s[0];
        a.heads[i] = laid[i].s[2];
    }
    return np == 3 ? decay<3>(d, a, m, st) : decay<1>(d, a, m, st);
}

cudaError_t launch_linear_decay_sum(const LinearDims &d, const double *part, float *grad_decay, Chain chain, cudaStream_t st) {
    return chain_launch(k_linear_decay_sum, d.H, 32, 0, st, part, d.B, d.H, linear_decay_blocks(d) * linear_tiles(d.Dv) * d.segs, grad_decay, chain);
}

}  // namespace sdm
