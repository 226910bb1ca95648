// Shared by the linear attention's kernels (linear*.cu). A head's state decays by the head's own factor at
// every token, is written and read:
//   S = e^g S + k v^T;   o = scale S^T q
// The backward's parts have the same form. With R the gradient of the state, run from the last token back,
//   dq = scale S do                   is the forward's with (do, v, k) for (q, k, v) and S transposed,
//   dk = R v,  dv = R^T k,  R += scale q do^T;  dk, dv are read, then R = e^g R
// are its mirror image with (v, do, q) and (k, q, do), so one kernel makes them all: a pass.
#pragma once

#include "chain.cuh"
#include "sdm_internal.cuh"

namespace sdm {

constexpr int kLinearMaxDk = 128, kLinearMaxDv = 512;
// Up to this many tokens go one by one. 12 tokens so and 13 in a chunk (128 x 128 bfloat16, in a graph): 2048 heads 135 and 133
// us (7.8 us a token more), 256 heads 15.2 and 19.0 (0.84 more), 16 heads 7.1 and 10.1 (0.4 more); float32, 16 heads 7.0 and
// 13.9. By the number of tokens alone, so that a sequence's results do not go by the batch it stands in: few heads would
// cross at 17 to 19 tokens.
constexpr int kLinearStepTokens = 12;
// A log-decay below this is taken as this: exp(-110) is 0 in float32, so the state is forgotten whole, and
// -inf (a hard reset at every token) has no 0 x inf among its powers.
constexpr float kLinearMinDecay = -110.f;

struct LinearDims {
    int B, T, H, Hk, Dk, Dv, dtype;
    int C, Nt;                           // chunk length, chunks a sequence
    int segs;                            // segments a sequence is cut into, run at once
    float scale;
    long long spin;                      // polls before a kernel's wait gives up (sdm_set_wait_limit)
    long long qs[3], ks[3], vs[3], os[3];   // element strides of (b, t, h); os: of the readings' gradient
};

// a tensor [B, T, heads, width] whose head h / share belongs to head h of a pass
struct LinearOperand {
    const void *p;
    long long s[3];
    int share;
};

struct LinearPass {
    LinearOperand q, k, v;
    int K, V;                            // widths of q and k, and of v and the result
    int blocks;                          // of K: each 128 columns, a result of its own
    bool reverse;
    float pair, from, to;                // scales: of q k, of what is read, of what is written
    const float *first;                  // state to begin with, null: 0
    float *last;                         // state to end with, or null
    long long sk, sv;                    // strides of a head's [Dk, Dv] state along K and V
    void *out;                           // [blocks][B, T, H, V] contiguous
    bool out_f32;                        // else of the inputs' type
};

struct LinearIn {
    const float *g;                      // [H]
    const int32_t *valid;                // may be null
};

__device__ __forceinline__ int linear_valid(const int32_t *valid, int b, int T) {
    const int v = valid ? valid[b] : T;
    return v < 0 ? 0 : (v > T ? T : v);
}
// floor(chunks n / segs), the chunk that segment n begins with, in 32 bits (segs is at most the SMs)
__device__ __forceinline__ int linear_cut(int chunks, int n, int segs) {
    const unsigned whole = (unsigned)chunks / (unsigned)segs, rest = (unsigned)chunks % (unsigned)segs;
    return (int)(whole * n + rest * n / segs);
}
// e^(g n) for whole n >= 0, within one unit in the last place. The powers multiply up along a sequence, and the
// rounding of g n itself would grow with n, so its low part is kept; the exponential is the argument reduction of Cody
// and Waite (n ln 2 in two parts, the first of few bits) and the Taylor series of the remainder. In 32 bits: a double
// exponential costs a block 2 us (the card has 2 lanes of doubles an SM).
__device__ __forceinline__ float linear_power(float g, int n) {
    if (g < kLinearMinDecay) g = kLinearMinDecay;
    const float m = (float)n, x = g * m, low = fmaf(g, m, -x);
    if (n == 0) return 1.f;
    if (!(x >= -110.f)) return x == x ? 0.f : x;
    if (x > 89.f) return __int_as_float(0x7f800000);
    const float k = rintf(x * 1.4426950408889634f);
    constexpr double kLn2 = 0.69314718055994530942;
    constexpr float kHigh = 0.693359375f, kLow = (float)(kLn2 - 0.693359375);   // 355 / 512: k times it is exact
    const float r = fmaf(k, -kHigh, x), r1 = r + fmaf(k, -kLow, low);
    float p = 1.f / 5040.f;
    p = fmaf(p, r1, 1.f / 720.f);
    p = fmaf(p, r1, 1.f / 120.f);
    p = fmaf(p, r1, 1.f / 24.f);
    p = fmaf(p, r1, 1.f / 6.f);
    p = fmaf(p, r1, 0.5f);
    return ldexpf(1.f + fmaf(p * r1, r1, r1), (int)k);
}

inline int linear_tiles(int columns) { return (columns + 127) / 128; }
inline long long linear_states(const LinearDims &d) { return (long long)d.B * d.H * d.Dk * d.Dv; }

// an operand as the tensor copies take it: bfloat16 [B, T, heads, width], float32 ones as three planes whose sum
// they are, [3 B, T, heads, width]
struct LinearLaid {
    const void *p;
    long long s[3];
    int heads, width;
};
// one to be laid out so: contiguous in dst
struct LinearLay {
    const void *src;
    long long s[3];
    int heads, width;
    void *dst;
};
// n of them, or none; clears the status block too
cudaError_t launch_linear_lay(const LinearDims &d, const LinearLay *lay, int n, DevStatus *status, cudaStream_t st);
cudaError_t launch_linear_scan(const LinearDims &d, const LinearPass &p, const LinearIn &in, const LinearLaid (&laid)[3], const float *starts,
                               void *status, Chain chain, cudaStream_t st);
// A sequence in segments (d.segs > 1): a first launch takes every segment but the pass's last from a state of zeros to
// what it adds, a join makes the states they begin with of that, and the scan runs all at once. k, v: the laid operands
// of a pass along the state's rows (sv = 1).
cudaError_t launch_linear_carry(const LinearDims &d, const LinearPass &p, const LinearIn &in, const LinearLaid &k, const LinearLaid &v, float *starts,
                                void *status, Chain chain, cudaStream_t st);

// up to kLinearStepTokens tokens (any number, but slowly)
cudaError_t launch_linear_step(const LinearDims &d, const LinearIn &in, const void *q, const void *k, const void *v, float *state, void *o,
                               cudaStream_t st);
// out [B, T, Hk, width] = the sum over a key head's heads, and over `blocks` parts, of part [blocks][B, T, H, width]
cudaError_t launch_linear_sum(const LinearDims &d, const float *part, int blocks, int width, void *out, Chain chain, cudaStream_t st);
// grad_decay [H] from the laid q, k, v and readings' gradient, the segments' first states and the gradients of the
// states they end with (from the last one; one segment: may be null)
inline int linear_decay_blocks(const LinearDims &d) { return (d.Dk + 63) / 64; }   // of Dk
inline long long linear_decay_parts(const LinearDims &d) { return (long long)d.B * d.H * d.segs * linear_decay_blocks(d) * linear_tiles(d.Dv); }
cudaError_t launch_linear_decay(const LinearDims &d, const LinearIn &in, const LinearLaid (&laid)[4], const float *starts, const float *ends,
                                double *part, void *status, Chain chain, cudaStream_t st);
// behind it: the parts' sums
cudaError_t launch_linear_decay_sum(const LinearDims &d, const double *part, float *grad_decay, Chain chain, cudaStream_t st);

}  // namespace sdm
