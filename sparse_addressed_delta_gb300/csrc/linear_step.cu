// Linear attention token by token, for single tokens and short runs of them, and the sums of the gradients of
// heads that share a key head.
//   S = e^g S + k v^T;  o = scale S^T q
// Bound by memory: the state is read and written once a call (2 Dk Dv floats a head), held in registers over the
// call's tokens. A block owns SLICE = 4 LPR columns of one head; LPR lanes read a row's slice as 16-byte pieces, so
// 256 / LPR rows are read at once and every load of the state is issued before the first use. The columns' sums over
// the rows go through shared memory (two buffers in turn, one barrier a token) and are added in warp order.
#include <type_traits>

#include "linear_internal.cuh"

namespace sdm {
namespace {

constexpr int kStepThreads = 256, kStepWarps = kStepThreads / 32;

template <typename T, int LPR>
__global__ void __launch_bounds__(kStepThreads, LPR == 32 ? 2 : 4)
    k_linear_step(const __grid_constant__ LinearDims d, const void *qp, const void *kp, const void *vp, const float *g, const int32_t *valid,
                  float *state, T *o) {
    constexpr int RP = kStepThreads / LPR;               // rows at once
    constexpr int NR = (kLinearMaxDk + RP - 1) / RP;     // rows of a thread
    __shared__ float skq[2][2][kLinearMaxDk];            // [buffer][k, q]
    __shared__ float4 part[2][kStepWarps][LPR];          // [buffer][warp][column piece]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cl = tid % LPR, r0 = tid / LPR;
    const int slices = d.Dv / (4 * LPR);
    const int sl = blockIdx.x % slices;
    const long long bh = blockIdx.x / slices;
    const int b = (int)(bh / d.H), h = (int)(bh % d.H), hk = h / (d.H / d.Hk);
    const int col = sl * 4 * LPR + 4 * cl;
    const int nt = linear_valid(valid, b, d.T);
    float *S = state + (bh * d.Dk) * d.Dv + col;
    const T *q = static_cast<const T *>(qp) + b * d.qs[0] + hk * d.qs[2];
    const T *k = static_cast<const T *>(kp) + b * d.ks[0] + hk * d.ks[2];
    const T *v = static_cast<const T *>(vp) + b * d.vs[0] + h * d.vs[2] + col;
    T *out = o + (((long long)b * d.T) * d.H + h) * d.Dv + col;
    const long long ostep = (long long)d.H * d.Dv;

    float4 s[NR];
    if (nt > 0) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int row = r0 + i * RP;
            s[i] = row < d.Dk ? *reinterpret_cast<const float4 *>(S + (size_t)row * d.Dv) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    const float fade = linear_power(g[h], 1);
    for (int t = 0; t < nt; ++t) {
        const int buf = t & 1;
        if (tid < 2 * kLinearMaxDk) {
            const int c = tid % kLinearMaxDk, w = tid / kLinearMaxDk;
            float x = 0.f;
            if (c < d.Dk) x = w ? to_f32(q[t * d.qs[1] + c]) : to_f32(k[t * d.ks[1] + c]);
            skq[buf][w][c] = x;
        }
        float vv[4];
        load_vec<T, 4, true>(v + t * d.vs[1], vv);
        __syncthreads();
        float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int row = r0 + i * RP;
            if (row < kLinearMaxDk) {                    // rows past Dk: k and q are 0
                const float kk = skq[buf][0][row], qq = skq[buf][1][row];
                s[i].x = fmaf(kk, vv[0], s[i].x * fade); s[i].y = fmaf(kk, vv[1], s[i].y * fade);
                s[i].z = fmaf(kk, vv[2], s[i].z * fade); s[i].w = fmaf(kk, vv[3], s[i].w * fade);
                if (row < d.Dk) {                        // (a NaN of v must not meet them)
                    c.x = fmaf(qq, s[i].x, c.x); c.y = fmaf(qq, s[i].y, c.y);
                    c.z = fmaf(qq, s[i].z, c.z); c.w = fmaf(qq, s[i].w, c.w);
                }
            }
        }
#pragma unroll
        for (int m = LPR; m < 32; m *= 2) {              // the warp's rows
            c.x += __shfl_xor_sync(~0u, c.x, m); c.y += __shfl_xor_sync(~0u, c.y, m);
            c.z += __shfl_xor_sync(~0u, c.z, m); c.w += __shfl_xor_sync(~0u, c.w, m);
        }
        if (lane < LPR) part[buf][warp][lane] = c;
        __syncthreads();
        if (r0 == 0) {
            c = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kStepWarps; ++w) {
                const float4 x = part[buf][w][cl];
                c.x += x.x; c.y += x.y; c.z += x.z; c.w += x.w;
            }
            const float r[4] = {d.scale * c.x, d.scale * c.y, d.scale * c.z, d.scale * c.w};
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
cudaError_t launch_step(const LinearDims &d, const LinearIn &in, const void *q, const void *k, const void *v, float *state, void *o, cudaStream_t st) {
    const long long heads = (long long)d.B * d.H;
    auto go = [&](auto lpr) {
        constexpr int LPR = decltype(lpr)::value;
        k_linear_step<T, LPR><<<(unsigned)(heads * (d.Dv / (4 * LPR))), kStepThreads, 0, st>>>(d, q, k, v, in.g, in.valid, state, static_cast<T *>(o));
        return cudaGetLastError();
    };
    // Wide slices read whole rows, narrow ones give every SM a block. Heads of 128 x 128 in us, slices of 128 / 32 / 16
    // columns: 16 heads 3.7 / 2.6 / 2.5; 32 heads 3.7 / 2.6 / 2.9; 64 heads 3.8 / 3.1 / 4.0; 160 heads 5.3 / 5.2 / 6.8;
    // 256 heads 5.5 / 6.6 / 9.5; 8192 heads 173 / 205 / 273.
    if (d.Dv % 128 == 0 && heads * (d.Dv / 128) >= kRefSms) return go(std::integral_constant<int, 32>{});
    if (d.Dv % 32 == 0 && heads * (d.Dv / 32) >= kRefSms * 3 / 4) return go(std::integral_constant<int, 8>{});
    return go(std::integral_constant<int, 4>{});
}

// A thread takes 4 columns of four key heads' rows; a key head's heads lie one behind the other, `width` apart.
// 8192 tokens, 32 heads of 128 in pairs: 27 us, 6.2 TB/s.
constexpr int kSumRows = 4;
template <typename T>
__global__ void __launch_bounds__(256) k_linear_sum(const float *part, long long rows, int group, int blocks, int width, T *out, Chain chain) {
    chain_begin(chain);
    const int pieces = width / 4, rpb = 256 / pieces, sub = threadIdx.x / pieces, c = threadIdx.x % pieces * 4;
    if (sub >= rpb) return;                              // (not all of a block)
    const long long row = (long long)blockIdx.x * rpb * kSumRows + sub, plane = rows * group * width;
    float4 s[kSumRows] = {};
    for (int g = 0; g < group; ++g)
        for (int m = 0; m < blocks; ++m) {
            float4 x[kSumRows];
#pragma unroll
            for (int i = 0; i < kSumRows; ++i)
                if (row + i * rpb < rows)
                    x[i] = __ldcg(reinterpret_cast<const float4 *>(part + m * plane + ((row + i * rpb) * group + g) * width + c));
#pragma unroll
            for (int i = 0; i < kSumRows; ++i) {
                s[i].x += x[i].x; s[i].y += x[i].y; s[i].z += x[i].z; s[i].w += x[i].w;
            }
        }
#pragma unroll
    for (int i = 0; i < kSumRows; ++i)
        if (row + i * rpb < rows) {
            const float y[4] = {s[i].x, s[i].y, s[i].z, s[i].w};
            store_vec<T, 4>(out + (row + i * rpb) * width + c, y);
        }
    chain_end(chain);
}

}  // namespace

cudaError_t launch_linear_step(const LinearDims &d, const LinearIn &in, const void *q, const void *k, const void *v, float *state, void *o,
                               cudaStream_t st) {
    return d.dtype == SDM_BF16 ? launch_step<__nv_bfloat16>(d, in, q, k, v, state, o, st) : launch_step<float>(d, in, q, k, v, state, o, st);
}

cudaError_t launch_linear_sum(const LinearDims &d, const float *part, int blocks, int width, void *out, Chain chain, cudaStream_t st) {
    const long long rows = (long long)d.B * d.T * d.Hk, each = 256 / (width / 4) * kSumRows, grid = (rows + each - 1) / each;
    const int group = d.H / d.Hk;
    if (d.dtype == SDM_BF16)
        return chain_launch(k_linear_sum<__nv_bfloat16>, (unsigned)grid, 256, 0, st, part, rows, group, blocks, width, static_cast<__nv_bfloat16 *>(out), chain);
    return chain_launch(k_linear_sum<float>, (unsigned)grid, 256, 0, st, part, rows, group, blocks, width, static_cast<float *>(out), chain);
}

}  // namespace sdm
