// The gated delta rule token by token, for single tokens and short runs of them:
//   d = e^g S;  r = v - d^T k;  S' = d + beta k r^T;  o = scale S'^T q
// The state's columns are independent, and both sums over its rows can be taken from the decayed
// state in one pass: o = scale (d^T q + beta (q . k) r).
//
// Bound by memory: the state is read and written once a call (2 Dk Dv floats a head), held in
// registers over the call's tokens. A block owns SLICE = 4 LPR columns of one head; LPR lanes read
// a row's slice as 16-byte pieces, so 256 / LPR rows are read at once and every load of the state
// is issued before the first use. One block barrier a token: the rows' partial sums go through
// shared memory (two buffers in turn) and every thread adds them in warp order.
#include "delta_internal.cuh"

namespace sdm {
namespace {

constexpr int kStepThreads = 256, kStepWarps = kStepThreads / 32;

// 128 columns: two blocks an SM, their loads and stores in turn (256 x 32 heads of 128 x 128: 182 us, 89 %
// of the copy rate; 32 columns 246, 16 columns 342)
template <typename T, int LPR>
__global__ void __launch_bounds__(kStepThreads, LPR == 32 ? 2 : 4)
    k_delta_step(DeltaDims d, DeltaIn in, float *state, T *o) {
    constexpr int RP = kStepThreads / LPR;               // rows at once
    constexpr int NR = (kDeltaMaxDk + RP - 1) / RP;      // rows of a thread
    __shared__ float skq[2][2][kDeltaMaxDk];             // [buffer][k, q]
    __shared__ float4 part[2][kStepWarps][2][LPR];       // [buffer][warp][k, q sums][column piece]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cl = tid % LPR, r0 = tid / LPR;
    const int slices = d.Dv / (4 * LPR);
    const int sl = blockIdx.x % slices;
    const long long bh = blockIdx.x / slices;
    const int b = (int)(bh / d.H), h = (int)(bh % d.H), hk = h / (d.H / d.Hk);
    const int col = sl * 4 * LPR + 4 * cl;
    const int nt = delta_valid(in.valid, b, d.T);
    float *S = state + (bh * d.Dk) * d.Dv + col;
    const T *q = static_cast<const T *>(in.q) + b * d.qs[0] + hk * d.qs[2];
    const T *k = static_cast<const T *>(in.k) + b * d.ks[0] + hk * d.ks[2];
    const T *v = static_cast<const T *>(in.v) + b * d.vs[0] + h * d.vs[2] + col;
    const float *g = in.g + b * d.gs[0] + h * d.gs[2], *be = in.beta + b * d.bs[0] + h * d.bs[2];
    T *out = o + (((long long)b * d.T) * d.H + h) * d.Dv + col;
    const long long ostep = (long long)d.H * d.Dv;

    float4 s[NR];
    if (nt > 0) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int row = r0 + i * RP;
            s[i] = row < d.Dk ? *reinterpret_cast<const float4 *>(S + (size_t)row * d.Dv)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    for (int t = 0; t < nt; ++t) {
        const int buf = t & 1;
        if (tid < 2 * kDeltaMaxDk) {
            const int c = tid % kDeltaMaxDk, w = tid / kDeltaMaxDk;
            float x = 0.f;
            if (c < d.Dk) x = w ? to_f32(q[t * d.qs[1] + c]) : to_f32(k[t * d.ks[1] + c]);
            skq[buf][w][c] = x;
        }
        float vv[4];
        load_vec<T, 4, true>(v + t * d.vs[1], vv);
        const float fade = expf(delta_decay(g[t * d.gs[1]])), beta = be[t * d.bs[1]];
        __syncthreads();
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), c = a;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int row = r0 + i * RP;                 // rows past Dk: k, q and the state are 0
            const float kk = skq[buf][0][row], qq = skq[buf][1][row];
            s[i].x *= fade; s[i].y *= fade; s[i].z *= fade; s[i].w *= fade;
            a.x = fmaf(kk, s[i].x, a.x); a.y = fmaf(kk, s[i].y, a.y);
            a.z = fmaf(kk, s[i].z, a.z); a.w = fmaf(kk, s[i].w, a.w);
            c.x = fmaf(qq, s[i].x, c.x); c.y = fmaf(qq, s[i].y, c.y);
            c.z = fmaf(qq, s[i].z, c.z); c.w = fmaf(qq, s[i].w, c.w);
        }
#pragma unroll
        for (int m = LPR; m < 32; m *= 2) {              // the warp's rows
            a.x += __shfl_xor_sync(~0u, a.x, m); a.y += __shfl_xor_sync(~0u, a.y, m);
            a.z += __shfl_xor_sync(~0u, a.z, m); a.w += __shfl_xor_sync(~0u, a.w, m);
            c.x += __shfl_xor_sync(~0u, c.x, m); c.y += __shfl_xor_sync(~0u, c.y, m);
            c.z += __shfl_xor_sync(~0u, c.z, m); c.w += __shfl_xor_sync(~0u, c.w, m);
        }
        if (lane < LPR) {
            part[buf][warp][0][lane] = a;
            part[buf][warp][1][lane] = c;
        }
        float qk = 0.f;
#pragma unroll
        for (int i = 0; i < kDeltaMaxDk / 32; ++i)
            qk = fmaf(skq[buf][0][lane + 32 * i], skq[buf][1][lane + 32 * i], qk);
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) qk += __shfl_xor_sync(~0u, qk, m);
        __syncthreads();
        a = c = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kStepWarps; ++w) {
            const float4 x = part[buf][w][0][cl], y = part[buf][w][1][cl];
            a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
            c.x += y.x; c.y += y.y; c.z += y.z; c.w += y.w;
        }
        const float4 u = make_float4(beta * (vv[0] - a.x), beta * (vv[1] - a.y),
                                     beta * (vv[2] - a.z), beta * (vv[3] - a.w));
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const float kk = skq[buf][0][r0 + i * RP];
            s[i].x = fmaf(kk, u.x, s[i].x); s[i].y = fmaf(kk, u.y, s[i].y);
            s[i].z = fmaf(kk, u.z, s[i].z); s[i].w = fmaf(kk, u.w, s[i].w);
        }
        if (r0 == 0) {
            const float r[4] = {d.scale * fmaf(qk, u.x, c.x), d.scale * fmaf(qk, u.y, c.y),
                                d.scale * fmaf(qk, u.z, c.z), d.scale * fmaf(qk, u.w, c.w)};
            store_vec<T, 4>(out + t * ostep, r);
        }
    }
    if (nt > 0) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int row = r0 + i * RP;
            if (row < d.Dk) *reinterpret_cast<float4 *>(S + (size_t)row * d.Dv) = s[i];
        }
    }
    if (r0 == 0) {
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
        for (int t = nt; t < d.T; ++t) store_vec<T, 4>(out + t * ostep, zero);
    }
}

template <typename T>
cudaError_t launch_step(const DeltaDims &d, const DeltaIn &in, float *state, void *o,
                        cudaStream_t st) {
    const long long heads = (long long)d.B * d.H;
    T *out = static_cast<T *>(o);
    // whole rows of 128 columns once there is a block of them for every SM: fewer blocks read q and k. Fewer heads
    // in narrow slices, which spread a head over more SMs. 128, 32 and 16 columns, us (heads of 128 x 128, bfloat16):
    // 16 heads x 8 tokens 18.4, 16.4, 16.4; 96 x 1 10.2, 8.2, 12.3; 128 x 1 10.2, 10.2, 12.3; 256 x 1 12.3, 14.3, 18.4;
    // 512 x 1 18.4, 22.5, 28.7; 512 x 8 41, 57, 104. 32 and 16, 16 heads of 64 x 64 6.2, 6.1; 512 12.3, 16.4.
    if (d.Dv % 128 == 0 && heads * (d.Dv / 128) >= kRefSms)
        k_delta_step<T, 32><<<(unsigned)(heads * (d.Dv / 128)), kStepThreads, 0, st>>>(d, in, state, out);
    else if (d.Dv % 32 == 0 && heads * (d.Dv / 32) >= 2 * kRefSms)
        k_delta_step<T, 8><<<(unsigned)(heads * (d.Dv / 32)), kStepThreads, 0, st>>>(d, in, state, out);
    else
        k_delta_step<T, 4><<<(unsigned)(heads * (d.Dv / 16)), kStepThreads, 0, st>>>(d, in, state, out);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_step(const DeltaDims &d, const DeltaIn &in, float *state, void *o,
                              cudaStream_t st) {
    return d.dtype == SDM_BF16 ? launch_step<__nv_bfloat16>(d, in, state, o, st)
                               : launch_step<float>(d, in, state, o, st);
}

}  // namespace sdm
