// Linear attention token by token: one thread a column of the state, its rows in registers.
#include "linear_internal.cuh"

namespace sdm {
namespace {

constexpr int kTokThreads = 128;

template <typename T, typename OT>
__global__ void __launch_bounds__(kTokThreads) k_linear_tokens(LinearDims d, LinearPass p, LinearIn in) {
    __shared__ float sq[kLinearMaxDk], sk[kLinearMaxDk];
    const int tid = threadIdx.x, col = blockIdx.x * kTokThreads + tid, h = (int)(blockIdx.y % d.H), b = (int)(blockIdx.y / d.H);
    const int k0 = (int)blockIdx.z * 128, K = p.K - k0 < 128 ? p.K - k0 : 128;
    const bool mine = col < p.V;
    const T *q = static_cast<const T *>(p.q.p) + b * p.q.s[0] + h / p.q.share * p.q.s[2] + k0;
    const T *k = static_cast<const T *>(p.k.p) + b * p.k.s[0] + h / p.k.share * p.k.s[2] + k0;
    const T *v = static_cast<const T *>(p.v.p) + b * p.v.s[0] + h / p.v.share * p.v.s[2] + col;
    OT *out = static_cast<OT *>(p.out) + (((long long)blockIdx.z * d.B + b) * d.T * d.H + h) * p.V + col;
    const long long state = ((long long)b * d.H + h) * d.Dk * d.Dv + k0 * p.sk + col * p.sv;
    const int n = linear_valid(in.valid, b, d.T);
    const float fade = (float)linear_power(in.g[h], 1.0);
    float S[kLinearMaxDk];
#pragma unroll
    for (int i = 0; i < kLinearMaxDk; ++i) S[i] = p.first && mine && i < K ? p.first[state + i * p.sk] : 0.f;
    for (int i = 0; i < n; ++i) {
        const int t = p.reverse ? n - 1 - i : i;
        __syncthreads();
        sq[tid] = tid < K ? to_f32(q[t * p.q.s[1] + tid]) : 0.f;
        sk[tid] = tid < K ? to_f32(k[t * p.k.s[1] + tid]) : 0.f;
        __syncthreads();
        const float x = mine ? to_f32(v[t * p.v.s[1]]) * p.to : 0.f, f = p.reverse ? 1.f : fade;
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < kLinearMaxDk; ++r) {
            S[r] = fmaf(sk[r], x, f * S[r]);
            sum = fmaf(sq[r], S[r], sum);
        }
        if (p.reverse)
#pragma unroll
            for (int r = 0; r < kLinearMaxDk; ++r) S[r] *= fade;
        if (mine) out[(long long)t * d.H * p.V] = from_f32<OT>(sum * p.from);
    }
    if (!mine) return;
    for (int t = n; t < d.T; ++t) out[(long long)t * d.H * p.V] = from_f32<OT>(0.f);
    if (p.last)
#pragma unroll
        for (int i = 0; i < kLinearMaxDk; ++i)
            if (i < K) p.last[state + i * p.sk] = S[i];
}

// The decay's gradient by carrying G = dS / dg along: G = e^g (G + S_before), and <do, scale G^T q> at every token
template <typename T>
__global__ void __launch_bounds__(kTokThreads) k_linear_decay(LinearDims d, LinearIn in, LinearOperand oq, LinearOperand ok, LinearOperand ov,
                                                              LinearOperand og, const float *first, const float *final_grad, double *part) {
    extern __shared__ float G[];                                   // [Dk][threads]
    __shared__ float sq[kLinearMaxDk], sk[kLinearMaxDk];
    __shared__ double sum[kTokThreads];
    const int tid = threadIdx.x, col = blockIdx.x * kTokThreads + tid, h = (int)(blockIdx.y % d.H), b = (int)(blockIdx.y / d.H);
    const bool mine = col < d.Dv;
    const T *q = static_cast<const T *>(oq.p) + b * oq.s[0] + h / oq.share * oq.s[2];
    const T *k = static_cast<const T *>(ok.p) + b * ok.s[0] + h / ok.share * ok.s[2];
    const T *v = static_cast<const T *>(ov.p) + b * ov.s[0] + h / ov.share * ov.s[2] + col;
    const T *g = static_cast<const T *>(og.p) + b * og.s[0] + h / og.share * og.s[2] + col;
    const long long state = ((long long)b * d.H + h) * d.Dk * d.Dv + col;
    const int n = linear_valid(in.valid, b, d.T);
    const float fade = (float)linear_power(in.g[h], 1.0);
    float S[kLinearMaxDk];
#pragma unroll
    for (int i = 0; i < kLinearMaxDk; ++i) {
        S[i] = mine && i < d.Dk ? first[state + (long long)i * d.Dv] : 0.f;
        if (i < d.Dk) G[i * kTokThreads + tid] = 0.f;
    }
    double acc = 0.0;
    for (int t = 0; t < n; ++t) {
        __syncthreads();
        sq[tid] = tid < d.Dk ? to_f32(q[t * oq.s[1] + tid]) : 0.f;
        sk[tid] = tid < d.Dk ? to_f32(k[t * ok.s[1] + tid]) : 0.f;
        __syncthreads();
        const float x = mine ? to_f32(v[t * ov.s[1]]) : 0.f, got = mine ? to_f32(g[t * og.s[1]]) : 0.f;
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < kLinearMaxDk; ++r)
            if (r < d.Dk) {
                const float a = fade * (G[r * kTokThreads + tid] + S[r]);
                G[r * kTokThreads + tid] = a;
                S[r] = fmaf(sk[r], x, fade * S[r]);
                s = fmaf(sq[r], a, s);
            }
        acc += (double)(d.scale * s) * got;
    }
    if (final_grad && mine)
        for (int r = 0; r < d.Dk; ++r) acc += (double)G[r * kTokThreads + tid] * final_grad[state + (long long)r * d.Dv];
    sum[tid] = acc;
    __syncthreads();
    if (tid == 0) {
        for (int i = 1; i < kTokThreads; ++i) acc += sum[i];
        part[(long long)blockIdx.y * gridDim.x + blockIdx.x] = acc;
    }
}

__global__ void k_linear_decay_sum(const double *part, int B, int H, int tiles, float *out) {
    const int h = blockIdx.x * blockDim.x + threadIdx.x;
    if (h >= H) return;
    double s = 0.0;
    for (int b = 0; b < B; ++b)
        for (int i = 0; i < tiles; ++i) s += part[((long long)b * H + h) * tiles + i];
    out[h] = (float)s;
}

template <typename T>
__global__ void __launch_bounds__(256) k_linear_sum(const float *part, long long rows, int H, int group, int blocks, int width, T *out) {
    const int heads = H / group, pieces = width / 4;
    const long long all = rows * heads * pieces, plane = rows * H * width;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
        const long long row = i / pieces, bt = row / heads;
        const float *src = part + (bt * H + row % heads * group) * width + i % pieces * 4;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        for (int g = 0; g < group; ++g)
            for (int m = 0; m < blocks; ++m) {
                const float4 x = *reinterpret_cast<const float4 *>(src + m * plane + g * width);
                s[0] += x.x; s[1] += x.y; s[2] += x.z; s[3] += x.w;
            }
        store_vec<T, 4>(out + 4 * i, s);
    }
}

}  // namespace

cudaError_t launch_linear_tokens(const LinearDims &d, const LinearPass &p, const LinearIn &in, cudaStream_t st) {
    const dim3 grid(linear_tiles(p.V), d.B * d.H, p.blocks);
    if (d.dtype == SDM_F32) k_linear_tokens<float, float><<<grid, kTokThreads, 0, st>>>(d, p, in);
    else if (p.out_f32) k_linear_tokens<__nv_bfloat16, float><<<grid, kTokThreads, 0, st>>>(d, p, in);
    else k_linear_tokens<__nv_bfloat16, __nv_bfloat16><<<grid, kTokThreads, 0, st>>>(d, p, in);
    return cudaGetLastError();
}

cudaError_t launch_linear_sum(const LinearDims &d, const float *part, int blocks, int width, void *out, cudaStream_t st) {
    const long long rows = (long long)d.B * d.T, units = rows * d.Hk * (width / 4), want = (units + 255) / 256;
    const unsigned grid = (unsigned)(want < 8 * kRefSms ? want : 8 * kRefSms);
    if (d.dtype == SDM_BF16) k_linear_sum<<<grid, 256, 0, st>>>(part, rows, d.H, d.H / d.Hk, blocks, width, static_cast<__nv_bfloat16 *>(out));
    else k_linear_sum<<<grid, 256, 0, st>>>(part, rows, d.H, d.H / d.Hk, blocks, width, static_cast<float *>(out));
    return cudaGetLastError();
}

cudaError_t launch_linear_decay(const LinearDims &d, const LinearIn &in, const LinearOperand &q, const LinearOperand &k, const LinearOperand &v,
                                const LinearOperand &grad, const float *first, const float *final_grad, double *part, float *grad_decay,
                                cudaStream_t st) {
    const int tiles = linear_tiles(d.Dv);
    const size_t smem = (size_t)d.Dk * kTokThreads * 4;
    auto go = [&](auto kern) {
        set_kernel_smem(kern, smem);
        kern<<<dim3(tiles, d.B * d.H), kTokThreads, smem, st>>>(d, in, q, k, v, grad, first, final_grad, part);
        return cudaGetLastError();
    };
    const cudaError_t e = d.dtype == SDM_BF16 ? go(k_linear_decay<__nv_bfloat16>) : go(k_linear_decay<float>);
    if (e != cudaSuccess) return e;
    k_linear_decay_sum<<<(d.H + 63) / 64, 64, 0, st>>>(part, d.B, d.H, tiles, grad_decay);
    return cudaGetLastError();
}

}  // namespace sdm
