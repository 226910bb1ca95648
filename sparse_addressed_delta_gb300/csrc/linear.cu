// C ABI of linear attention with a decay for each head (declared and documented in include/sdm.h): argument
// checks and the launch sequence. Everything is queued on the caller's stream; nothing is allocated and
// nothing synchronizes.
#include "linear_internal.cuh"
#include "tcgen05.cuh"

namespace sdm {
namespace {

size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool off16(const void *p) { return (uintptr_t)p % 16 != 0; }

// How many segments a sequence is run in (launch_linear_carry): they pay where the heads alone leave SMs idle, one block
// an SM. By the times in microseconds measured: a chunk of the scan and of the carry, a block's start, the join and each
// of its steps. By shape and type alone: a saving forward's results are the plain one's, and a backward's segments its
// forward's, whatever the strides. Measured, forward,
// in segments and not: 16 heads of 128 x 128 x 128 chunks 70 and 259 us, x 16 29 and 42; 32 x 64 72 and 136; 64 x 64 117
// and 136; float32, 8 heads of 64 x 64 x 16 30 and 72, x 128 74 and 525.
void linear_segments(LinearDims &d) {
    const bool tensor = d.dtype == SDM_BF16;
    const double scan = tensor ? 2.0 : 4.5, carry = tensor ? 0.86 : 2.0, start = tensor ? 4.0 : 5.0, join = 5.0, step = 0.2;
    const long long blocks = (long long)d.B * d.H * linear_tiles(d.Dv);
    double best = start + scan * d.Nt;
    d.segs = 1;
    for (int s = 2; s <= d.Nt && blocks * s <= kRefSms; ++s) {
        const int chunks = (d.Nt + s - 1) / s;
        const double time = 2 * start + (scan + carry) * chunks + join + step * s;
        if (time < best) {
            best = time;
            d.segs = s;
        }
    }
}

// Checks the shape; fills d. Returns SDM_OK or a refusal (message set). A forward does not look at grad_stride.
int linear_check(const sdm_linear_shape *s, LinearDims &d, bool back) {
    if (!s) return set_error(SDM_ERR_INVALID, "linear attention: shape is NULL");
    if (s->B < 0 || s->T < 0)
        return set_error(SDM_ERR_INVALID, "linear attention: B and T must be >= 0, got %d, %d", s->B, s->T);
    if (s->H < 1 || s->Hk < 1 || s->H % s->Hk)
        return set_error(SDM_ERR_INVALID, "linear attention: H must be a multiple of Hk >= 1, got %d, %d", s->H, s->Hk);
    if (s->dtype != SDM_F32 && s->dtype != SDM_BF16)
        return set_error(SDM_ERR_INVALID, "linear attention: dtype must be SDM_F32 or SDM_BF16, got %d", s->dtype);
    if (s->Dk < 1 || s->Dv < 1)
        return set_error(SDM_ERR_INVALID, "linear attention: Dk and Dv must be >= 1, got %d, %d", s->Dk, s->Dv);
    if (s->Dk % 16 || s->Dk > kLinearMaxDk || s->Dv % 16 || s->Dv > kLinearMaxDv)
        return set_error(SDM_ERR_UNSUPPORTED, "linear attention: Dk (up to %d) and Dv (up to %d) must be multiples of 16, "
                         "got %d, %d", kLinearMaxDk, kLinearMaxDv, s->Dk, s->Dv);
    if (!(s->scale == s->scale)) return set_error(SDM_ERR_INVALID, "linear attention: scale is not a number");
    d.B = s->B; d.T = s->T; d.H = s->H; d.Hk = s->Hk; d.Dk = s->Dk; d.Dv = s->Dv;
    d.dtype = s->dtype;
    d.scale = s->scale;
    d.C = 64;
    if (s->T > INT32_MAX - d.C) return set_error(SDM_ERR_UNSUPPORTED, "linear attention: T must be at most 2^31 - 65, got %d", s->T);
    d.Nt = (s->T + d.C - 1) / d.C;
    d.spin = wait_limit();
    // blocks of a launch: one per head and 16 columns of the state
    if ((long long)s->B * s->H * (s->Dv / 16) >= (1LL << 31))
        return set_error(SDM_ERR_INVALID, "linear attention: B H Dv / 16 must be below 2^31");
    linear_segments(d);
    const int es = s->dtype == SDM_BF16 ? 2 : 4;
    for (int i = 0; i < 3; ++i) {
        d.qs[i] = s->q_stride[i]; d.ks[i] = s->k_stride[i]; d.vs[i] = s->v_stride[i]; d.os[i] = back ? s->grad_stride[i] : 0;
        if ((d.qs[i] * es) % 16 || (d.ks[i] * es) % 16 || (d.vs[i] * es) % 16 || (d.os[i] * es) % 16)
            return set_error(SDM_ERR_INVALID, "linear attention: the strides of q, k, v and the gradient must be multiples "
                             "of 16 bytes");
        if (d.qs[i] < 0 || d.ks[i] < 0 || d.vs[i] < 0 || d.os[i] < 0)
            return set_error(SDM_ERR_INVALID, "linear attention: negative stride");
    }
    if (d.dtype == SDM_BF16 && !(tc_tensor_fits(d.qs, d.B, d.T, d.Hk) && tc_tensor_fits(d.ks, d.B, d.T, d.Hk) &&
                                 tc_tensor_fits(d.vs, d.B, d.T, d.H) && tc_tensor_fits(d.os, d.B, d.T, d.H)))
        return set_error(SDM_ERR_UNSUPPORTED, "linear attention: bfloat16 strides must be below 2^39 elements");
    return SDM_OK;
}

int linear_check_inputs(const void *q, const void *k, const void *v, const float *g) {
    if (!q || !k || !v || !g) return set_error(SDM_ERR_INVALID, "linear attention: NULL pointer");
    if (off16(q) || off16(k) || off16(v))
        return set_error(SDM_ERR_INVALID, "linear attention: q, k and v must be 16-byte aligned");
    return SDM_OK;
}

int linear_check_ws(const char *what, const void *ws, size_t have, size_t need) {
    if (!ws || have < need || (uintptr_t)ws % kAlign)
        return set_error(SDM_ERR_WORKSPACE, "linear attention: %s NULL, too small (%zu of %zu bytes) or not %zu-byte aligned", what,
                         have, need, (size_t)kAlign);
    return SDM_OK;
}

int linear_status(cudaError_t e) {
    if (e == cudaSuccess) return SDM_OK;
    return set_error(SDM_ERR_CUDA, "linear attention: %s", cudaGetErrorString(e));
}

// the status block at a workspace's start
cudaError_t linear_clear(void *ws, size_t have, cudaStream_t st) {
    return ws && have >= kAlign ? cudaMemsetAsync(ws, 0, sizeof(DevStatus), st) : cudaSuccess;
}

// dq and dk are parts for each head and each 128 columns of Dv where there is more than one of them
bool linear_parts(const LinearDims &d) { return d.H != d.Hk || d.Dv > 128; }

// whether q, k, v or the gradient (i = 0 .. 3) has to be laid out for the tensor copies: float32, or bfloat16 and
// broadcast along the tokens (they step along them)
bool linear_lays(const LinearDims &d, int i) {
    return d.dtype == SDM_F32 || (d.T > 1 && (i == 0 ? d.qs : i == 1 ? d.ks : i == 2 ? d.vs : d.os)[1] == 0);
}

// Where a call's buffers lie in its workspace; `bytes` is their end.
struct LinearLayout {
    size_t laid[4];                      // q, k, v and the gradient where linear_lays
    size_t starts;                       // the segments' first states (a saving forward's are saved; a backward: of the gradient)
    size_t dq, dk, decay, bytes;
};

LinearLayout linear_layout(const LinearDims &d, bool back) {
    LinearLayout l{};
    size_t at = kAlign;                  // behind the status block
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += up(bytes);
        return here;
    };
    for (int i = 0; i < (back ? 4 : 3); ++i)
        l.laid[i] = take(linear_lays(d, i) ? (size_t)d.B * d.T * (i < 2 ? (size_t)d.Hk * d.Dk : (size_t)d.H * d.Dv) * (d.dtype == SDM_F32 ? 6 : 2) : 0);
    l.starts = take(d.segs > 1 ? d.segs * (size_t)linear_states(d) * 4 : 0);
    if (back) {
        const size_t part = linear_parts(d) ? (size_t)linear_tiles(d.Dv) * d.B * d.T * d.H * d.Dk * 4 : 0;
        l.dq = take(part);
        l.dk = take(part);
        l.decay = take((size_t)linear_decay_parts(d) * 8);
    }
    l.bytes = at;
    return l;
}

// what the saving forward keeps: the states its segments begin with, the initial one first
size_t linear_saved(const LinearDims &d) { return up(d.segs * (size_t)linear_states(d) * 4); }

// q, k, v (and with grad the readings' gradient) as the tensor copies take them; clears the status block
cudaError_t linear_lay(const LinearDims &d, const LinearLayout &l, unsigned char *ws, const void *const (&src)[4], LinearLaid (&laid)[4],
                       cudaStream_t st) {
    LinearLay lay[4];
    int n = 0;
    for (int i = 0; i < 4 && src[i]; ++i) {
        const long long *s = i == 0 ? d.qs : i == 1 ? d.ks : i == 2 ? d.vs : d.os;
        const int heads = i < 2 ? d.Hk : d.H, width = i < 2 ? d.Dk : d.Dv;
        laid[i] = LinearLaid{src[i], {s[0], s[1], s[2]}, heads, width};
        if (!linear_lays(d, i)) continue;
        lay[n++] = LinearLay{src[i], {s[0], s[1], s[2]}, heads, width, ws + l.laid[i]};
        laid[i] = LinearLaid{ws + l.laid[i], {(long long)d.T * heads * width, (long long)heads * width, width}, heads, width};
    }
    return launch_linear_lay(d, lay, n, reinterpret_cast<DevStatus *>(ws), st);
}

LinearOperand operand(const void *p, const long long *s, int share) { return LinearOperand{p, {s[0], s[1], s[2]}, share}; }

// sdm_linear_attention and, with `save`, sdm_linear_attention_save
int linear_forward(const sdm_linear_shape *shape, float *state, const void *q, const void *k, const void *v, const float *log_decay,
                   const int32_t *valid_tokens, void *readings, bool save, void *saved, size_t saved_bytes, void *workspace,
                   size_t workspace_bytes, void *stream) {
    LinearDims d;
    int rc = linear_check(shape, d, false);
    if (rc != SDM_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d.B == 0 || d.T == 0) return linear_status(linear_clear(workspace, workspace_bytes, st));
    rc = linear_check_inputs(q, k, v, log_decay);
    if (rc != SDM_OK) return rc;
    if (!state || !readings) return set_error(SDM_ERR_INVALID, "linear attention: NULL pointer");
    if (off16(state) || off16(readings))
        return set_error(SDM_ERR_INVALID, "linear attention: the state and the readings must be 16-byte aligned");
    const LinearIn in{log_decay, valid_tokens};
    const int group = d.H / d.Hk;
    const LinearPass p{operand(q, d.qs, group), operand(k, d.ks, group), operand(v, d.vs, 1), d.Dk, d.Dv, 1, false, d.scale, d.scale, 1.f,
                       state, state, d.Dv, 1, readings, false};
    if (!save && d.T <= kLinearStepTokens) {
        const cudaError_t e = linear_clear(workspace, workspace_bytes, st);
        return linear_status(e == cudaSuccess ? launch_linear_step(d, in, q, k, v, state, readings, st) : e);
    }
    const LinearLayout l = linear_layout(d, false);
    rc = linear_check_ws("workspace", workspace, workspace_bytes, l.bytes);
    if (rc == SDM_OK && save) rc = linear_check_ws("saved buffer", saved, saved_bytes, linear_saved(d));
    if (rc != SDM_OK) return rc;
    auto ws = static_cast<unsigned char *>(workspace);
    LinearLaid laid[4];
    cudaError_t e = cudaSuccess;
    if (save && d.segs == 1)
        e = cudaMemcpyAsync(saved, state, (size_t)linear_states(d) * 4, cudaMemcpyDeviceToDevice, st);
    if (e == cudaSuccess) e = linear_lay(d, l, ws, {q, k, v, nullptr}, laid, st);
    float *starts = save ? static_cast<float *>(saved) : reinterpret_cast<float *>(ws + l.starts);
    if (e == cudaSuccess && d.segs > 1) e = launch_linear_carry(d, p, in, laid[1], laid[2], starts, ws, Chain::behind, st);
    if (e == cudaSuccess) e = launch_linear_scan(d, p, in, {laid[0], laid[1], laid[2]}, starts, ws, Chain::behind, st);
    return linear_status(e);
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" {

size_t sdm_linear_attention_workspace_bytes(const sdm_linear_shape *shape) {
    LinearDims d;
    if (linear_check(shape, d, false) != SDM_OK) return 0;
    return linear_layout(d, false).bytes + kAlign;
}

int sdm_linear_attention(const sdm_linear_shape *shape, float *state, const void *q, const void *k, const void *v,
                         const float *log_decay, const int32_t *valid_tokens, void *readings, void *workspace,
                         size_t workspace_bytes, void *stream) {
    return linear_forward(shape, state, q, k, v, log_decay, valid_tokens, readings, false, nullptr, 0, workspace, workspace_bytes, stream);
}

size_t sdm_linear_attention_saved_bytes(const sdm_linear_shape *shape) {
    LinearDims d;
    if (linear_check(shape, d, false) != SDM_OK) return 0;
    return linear_saved(d) + kAlign;
}

int sdm_linear_attention_save(const sdm_linear_shape *shape, float *state, const void *q, const void *k, const void *v,
                              const float *log_decay, const int32_t *valid_tokens, void *readings, void *saved, size_t saved_bytes,
                              void *workspace, size_t workspace_bytes, void *stream) {
    return linear_forward(shape, state, q, k, v, log_decay, valid_tokens, readings, true, saved, saved_bytes, workspace, workspace_bytes,
                          stream);
}

size_t sdm_linear_attention_backward_workspace_bytes(const sdm_linear_shape *shape) {
    LinearDims d;
    if (linear_check(shape, d, true) != SDM_OK) return 0;
    return linear_layout(d, true).bytes + kAlign;
}

int sdm_linear_attention_backward(const sdm_linear_shape *shape, const void *q, const void *k, const void *v, const float *log_decay,
                                  const int32_t *valid_tokens, const void *saved, size_t saved_bytes, const void *grad_readings,
                                  const float *grad_final_state, float *grad_state, void *grad_q, void *grad_k, void *grad_v,
                                  float *grad_log_decay, void *workspace, size_t workspace_bytes, void *stream) {
    LinearDims d;
    int rc = linear_check(shape, d, true);
    if (rc != SDM_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t state_bytes = (size_t)linear_states(d) * 4;
    if (d.B == 0 || d.T == 0) {
        if (d.B && !grad_state) return set_error(SDM_ERR_INVALID, "linear attention: NULL pointer");
        cudaError_t e = linear_clear(workspace, workspace_bytes, st);
        if (e == cudaSuccess && grad_log_decay) e = cudaMemsetAsync(grad_log_decay, 0, (size_t)d.H * 4, st);
        if (e == cudaSuccess && d.B)         // the final state is the initial one
            e = !grad_final_state ? cudaMemsetAsync(grad_state, 0, state_bytes, st)
                : grad_final_state != grad_state ? cudaMemcpyAsync(grad_state, grad_final_state, state_bytes, cudaMemcpyDeviceToDevice, st)
                                                 : cudaSuccess;
        return linear_status(e);
    }
    rc = linear_check_inputs(q, k, v, log_decay);
    if (rc != SDM_OK) return rc;
    if (!grad_readings || !grad_state || !grad_q || !grad_k || !grad_v) return set_error(SDM_ERR_INVALID, "linear attention: NULL pointer");
    if (off16(grad_readings) || off16(grad_q) || off16(grad_k) || off16(grad_v))
        return set_error(SDM_ERR_INVALID, "linear attention: the gradients of q, k, v and the readings must be 16-byte aligned");
    const LinearLayout l = linear_layout(d, true);
    rc = linear_check_ws("workspace", workspace, workspace_bytes, l.bytes);
    if (rc == SDM_OK) rc = linear_check_ws("saved buffer", saved, saved_bytes, linear_saved(d));
    if (rc != SDM_OK) return rc;
    auto ws = static_cast<unsigned char *>(workspace);
    const LinearIn in{log_decay, valid_tokens};
    const int group = d.H / d.Hk, tiles = linear_tiles(d.Dv);
    const LinearOperand oq = operand(q, d.qs, group), ok = operand(k, d.ks, group), ov = operand(v, d.vs, 1), og = operand(grad_readings, d.os, 1);
    const bool parts = linear_parts(d);
    auto first = static_cast<const float *>(saved);
    void *dq = parts ? ws + l.dq : grad_q, *dk = parts ? ws + l.dk : grad_k;
    const LinearPass pq{og, ov, ok, d.Dv, d.Dk, tiles, false, d.scale, d.scale, 1.f, first, nullptr, 1, d.Dv, dq, parts};
    const LinearPass pk{ov, og, oq, d.Dv, d.Dk, tiles, true, d.scale, 1.f, d.scale, grad_final_state, nullptr, 1, d.Dv, dk, parts};
    const LinearPass pv{ok, oq, og, d.Dk, d.Dv, 1, true, d.scale, 1.f, d.scale, grad_final_state, grad_state, d.Dv, 1, grad_v, false};
    LinearLaid laid[4];
    const bool cut = d.segs > 1, decay = grad_log_decay != nullptr;
    auto part = reinterpret_cast<double *>(ws + l.decay);
    cudaError_t e = linear_lay(d, l, ws, {q, k, v, grad_readings}, laid, st);
    float *ends = reinterpret_cast<float *>(ws + l.starts);
    // The scans and the decays' gradient need only the segments' ends, and no other launch's results: they run beside each
    // other, as do the carry and dq's scan, and the sums of dq and what comes after them, so that a launch's idle SMs
    // have work (2 x 4096 tokens of 32 heads: 64 heads in two segments leave 24 of 152 idle; training 590 -> 534 us).
    if (e == cudaSuccess) e = launch_linear_scan(d, pq, in, {laid[3], laid[2], laid[1]}, first, ws, Chain::behind, st);
    if (e == cudaSuccess && cut) e = launch_linear_carry(d, pv, in, laid[0], laid[3], ends, ws, Chain::beside, st);
    if (e == cudaSuccess) e = launch_linear_scan(d, pk, in, {laid[2], laid[3], laid[0]}, ends, ws, cut ? Chain::behind : Chain::beside, st);
    if (e == cudaSuccess && decay) e = launch_linear_decay(d, in, laid, first, cut ? ends : grad_final_state, part, ws, Chain::beside, st);
    // (dq's scan has ended once dk's has passed a wait at its start)
    if (e == cudaSuccess && parts)
        e = launch_linear_sum(d, static_cast<const float *>(dq), tiles, d.Dk, grad_q, cut ? Chain::beside : Chain::behind, st);
    // (in one segment the others read the final state's gradient, which may be grad_state itself)
    if (e == cudaSuccess)
        e = launch_linear_scan(d, pv, in, {laid[1], laid[0], laid[3]}, ends, ws, !cut && grad_final_state == grad_state ? Chain::behind : Chain::beside, st);
    if (e == cudaSuccess && parts) e = launch_linear_sum(d, static_cast<const float *>(dk), tiles, d.Dk, grad_k, Chain::behind, st);
    if (e == cudaSuccess && decay) e = launch_linear_decay_sum(d, part, grad_log_decay, parts ? Chain::beside : Chain::behind, st);
    return linear_status(e);
}

}  // extern "C"
