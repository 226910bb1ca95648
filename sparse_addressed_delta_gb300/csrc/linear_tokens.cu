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

}  // namespace sdm
