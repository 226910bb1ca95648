// C ABI of the gated delta rule (declared and documented in include/sdm.h): argument checks and the
// launch sequence. Everything is queued on the caller's stream; nothing is allocated and nothing
// synchronizes.
#include <algorithm>

#include "tcgen05.cuh"

namespace sdm {
namespace {

// How many segments a sequence's scans take (DeltaBlock in delta_internal.cuh): two launches and a join,
// which pay when the heads alone leave SMs idle. By the times in microseconds measured: a chunk alone and
// beside twice as many blocks, a chunk of the first launch (the tensor-memory form at 128 x 128; the register
// form by its products), a block's start, the join and each of its steps. Measured, whole call, in segments
// and not, bfloat16 at 128 x 128: 32 heads x 256 chunks 637 and 1006 us, 16 x 64 139 and 250, 4 x 64 109 and
// 229 (backward 294 and 451, 169 and 336). Narrower heads are taken to cost the same: at 64 x 64, 16 heads x 64
// chunks 111 and 205, 4 x 64 84 and 184 (backward 242 and 359, 136 and 257); at 64 x 128, 32 x 64 170 and 225.
// float32 training, 8 heads of 64 x 64 x 32 chunks: 191 and 332. By shape and type alone: a saving forward's results
// are the plain one's, and a backward's segments its forward's, whatever the strides.
void delta_segments(DeltaDims &d) {
    constexpr double kStart = 8.0, kJoin = 8.0, kJoinStep = 4.0;
    const bool tensor = d.dtype == SDM_BF16;
    const int of = tensor ? 128 : 64;
    const double alone = tensor ? 2.6 : 0.5 * d.Dk / 16 + 1.0, beside = tensor ? 3.0 : alone, carry = tensor ? 2.3 : 0.36 * d.Dk / 16 + 0.6;
    const long long heads = (long long)d.B * d.H, blocks = heads * delta_tiles(d.Dv, of), units = heads * delta_tiles(d.Dk, of);
    const double startup = kStart / beside;                  // in chunks
    double best = (alone * d.Nt + kStart) * ((blocks + kRefSms - 1) / kRefSms);
    d.segs = d.first = 1;
    for (int s = 3; s <= d.Nt; ++s) {
        const long long busy = std::max((s - 2) * (blocks + units), (s - 1) * blocks);
        if (busy >= kRefSms) break;                          // segment 0 needs SMs beside the others
        // `rounds` blocks of segment 0 one after another take as long as one of the others
        const double rounds = (double)((blocks + kRefSms - busy - 1) / (kRefSms - busy));
        const double longer = std::min((d.Nt + startup * (1.0 - 1.0 / rounds)) / (s - 1 + 1.0 / rounds), d.Nt / (s - 1.0));
        const double time = (carry + beside) * longer + 2 * kStart + kJoin + kJoinStep * (s - 2);
        if (time < best) {
            best = time;
            d.segs = s;
            d.first = (int)(256.0 * (d.Nt - (s - 1) * longer) / longer);
        }
    }
}

// Checks the shape; fills d. Returns SDM_OK or a refusal (message set). A forward does not look at grad_stride.
int delta_check(const sdm_delta_shape *s, DeltaDims &d, bool back) {
    if (!s) return set_error(SDM_ERR_INVALID, "gated delta: shape is NULL");
    if (s->B < 0 || s->T < 0)
        return set_error(SDM_ERR_INVALID, "gated delta: B and T must be >= 0, got %d, %d", s->B, s->T);
    if (s->H < 1 || s->Hk < 1 || s->H % s->Hk)
        return set_error(SDM_ERR_INVALID, "gated delta: H must be a multiple of Hk >= 1, got %d, %d",
                         s->H, s->Hk);
    if (s->dtype != SDM_F32 && s->dtype != SDM_BF16)
        return set_error(SDM_ERR_INVALID, "gated delta: dtype must be SDM_F32 or SDM_BF16, got %d",
                         s->dtype);
    if (s->Dk < 1 || s->Dv < 1)
        return set_error(SDM_ERR_INVALID, "gated delta: Dk and Dv must be >= 1, got %d, %d", s->Dk, s->Dv);
    if (s->Dk % 16 || s->Dk > kDeltaMaxDk || s->Dv % 16 || s->Dv > kDeltaMaxDv)
        return set_error(SDM_ERR_UNSUPPORTED, "gated delta: Dk (up to %d) and Dv (up to %d) must be "
                         "multiples of 16, got %d, %d", kDeltaMaxDk, kDeltaMaxDv, s->Dk, s->Dv);
    if (!(s->scale == s->scale))
        return set_error(SDM_ERR_INVALID, "gated delta: scale is not a number");
    d.B = s->B; d.T = s->T; d.H = s->H; d.Hk = s->Hk; d.Dk = s->Dk; d.Dv = s->Dv;
    d.dtype = s->dtype;
    d.scale = s->scale;
    d.C = delta_chunk(s->dtype);
    d.back = back;
    d.spin = wait_limit();
    d.Nt = (int)(((long long)s->T + d.C - 1) / d.C);
    // blocks of a launch: one per chunk and head, or per head and 16 columns of the state
    if ((long long)s->B * s->H * d.Nt >= (1LL << 31) || (long long)s->B * s->H * (s->Dv / 16) >= (1LL << 31))
        return set_error(SDM_ERR_INVALID, "gated delta: B H ceil(T / %d) and B H Dv / 16 must be below 2^31", d.C);
    const int es = s->dtype == SDM_BF16 ? 2 : 4;
    for (int i = 0; i < 3; ++i) {
        d.qs[i] = s->q_stride[i]; d.ks[i] = s->k_stride[i]; d.vs[i] = s->v_stride[i];
        d.gs[i] = s->decay_stride[i]; d.bs[i] = s->beta_stride[i]; d.os[i] = back ? s->grad_stride[i] : 0;
        if ((d.qs[i] * es) % 16 || (d.ks[i] * es) % 16 || (d.vs[i] * es) % 16 || (d.os[i] * es) % 16)
            return set_error(SDM_ERR_INVALID, "gated delta: the strides of q, k, v and the gradient "
                             "must be multiples of 16 bytes");
        if (d.qs[i] < 0 || d.ks[i] < 0 || d.vs[i] < 0 || d.gs[i] < 0 || d.bs[i] < 0 || d.os[i] < 0)
            return set_error(SDM_ERR_INVALID, "gated delta: negative stride");
    }
    // bfloat16 inputs run on tcgen05, with narrow states too: 4096 tokens, 32 heads of 128 x 64 or 128 x 16 take 206
    // us, as three-plane products in registers they took 315 and 313
    d.tc = s->dtype == SDM_BF16;
    if (d.tc && !(tc_tensor_fits(d.qs, d.B, d.T, d.Hk) && tc_tensor_fits(d.ks, d.B, d.T, d.Hk) &&
                  tc_tensor_fits(d.vs, d.B, d.T, d.H) && tc_tensor_fits(d.os, d.B, d.T, d.H)))
        return set_error(SDM_ERR_UNSUPPORTED, "gated delta: bfloat16 strides must be below 2^39 elements");
    delta_segments(d);
    return SDM_OK;
}

bool off16(const void *p) { return (uintptr_t)p % 16 != 0; }

int delta_check_inputs(const void *q, const void *k, const void *v, const float *g,
                       const float *beta) {
    if (!q || !k || !v || !g || !beta) return set_error(SDM_ERR_INVALID, "gated delta: NULL pointer");
    if (off16(q) || off16(k) || off16(v))
        return set_error(SDM_ERR_INVALID, "gated delta: q, k and v must be 16-byte aligned");
    return SDM_OK;
}

int delta_status(cudaError_t e) {
    if (e == cudaSuccess) return SDM_OK;
    return set_error(SDM_ERR_CUDA, "gated delta: %s", cudaGetErrorString(e));
}

bool by_token(const DeltaDims &d) { return d.T <= kDeltaStepTokens; }

size_t delta_unit_bytes(const DeltaDims &d) { return d.segs > 1 ? (d.segs - 2) * (size_t)d.B * d.H * d.Dk * d.Dk * 4 : 0; }

// whether q, k, v or the gradient (i = 0 .. 3) is bfloat16 and broadcast along the tokens
bool delta_flat(const DeltaDims &d, int i) {
    return d.tc && d.T > 1 && (i == 0 ? d.qs : i == 1 ? d.ks : i == 2 ? d.vs : d.os)[1] == 0;
}

// Where the chunk form's buffers lie in a workspace; `bytes` is their end.
struct DeltaLayout {
    size_t q, k, x, p, aux;              // q, k: the planes of float32 inputs
    size_t flat[4];                      // bfloat16 q, k, v and gradient that are broadcast along the tokens
    size_t starts, units;                // the segments' (units: of a forward that saves nothing); a forward's own
    size_t ends, w, dq, dk;              // the backward's
    size_t bytes;
};

DeltaLayout delta_layout(const DeltaDims &d, bool backward) {
    DeltaLayout l{};
    size_t at = kAlign;                  // behind the status block
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += delta_up(bytes);
        return here;
    };
    const size_t tok = d.dtype == SDM_F32 ? (size_t)d.B * d.T * d.Hk * d.Dk * 3 * 2 : 0;
    l.q = take(tok);
    l.k = take(tok);
    l.x = take(delta_chunks(d) * 3 * delta_plane_bytes(d));
    l.p = take(delta_chunks(d) * 3 * delta_plane_bytes(d));
    l.aux = take(delta_chunks(d) * kDeltaAux * d.C * 4);
    // (a forward of one segment: where a column's state goes that delta_column takes again)
    l.starts = take(d.segs > 1 || !backward ? d.segs * (size_t)delta_states(d) * 4 : 0);
    if (!backward) l.units = take(delta_unit_bytes(d));
    if (backward) {
        l.ends = take(delta_chunks(d) * d.Dk * d.Dv * 4);
        l.w = take(delta_chunks(d) * d.C * d.Dv * 4);
        const size_t part = d.H != d.Hk && !(d.tc && d.Dv <= 128) ? (size_t)d.B * d.T * d.H * d.Dk * 4 : 0;
        l.dq = take(part);
        l.dk = take(part);
    }
    for (int i = 0; i < 4; ++i) l.flat[i] = take(delta_flat(d, i) && (i < 3 || backward) ? (size_t)d.B * d.T * (i < 2 ? (size_t)d.Hk * d.Dk : (size_t)d.H * d.Dv) * 2 : 0);
    l.bytes = at;
    return l;
}

// Tensor copies step along the tokens: bfloat16 inputs that do not (one token's for all) are laid out in the
// workspace first.
cudaError_t delta_unroll(DeltaDims &d, const DeltaLayout &l, unsigned char *ws, int i, const void *&x, cudaStream_t st) {
    if (!delta_flat(d, i)) return cudaSuccess;
    long long *s = i == 0 ? d.qs : i == 1 ? d.ks : i == 2 ? d.vs : d.os;
    const int heads = i < 2 ? d.Hk : d.H, width = i < 2 ? d.Dk : d.Dv;
    const cudaError_t e = launch_delta_unroll(d, x, s, heads, width, ws + l.flat[i], st);
    x = ws + l.flat[i];
    s[0] = (long long)d.T * heads * width;
    s[1] = (long long)heads * width;
    s[2] = width;
    return e;
}

// what the saving forward keeps: the state at every chunk's start and at the end, r, and the segments' units
size_t delta_saved_snap(const DeltaDims &d) {
    return delta_up((delta_chunks(d) + (size_t)d.B * d.H) * d.Dk * d.Dv * 4);
}
size_t delta_saved_units(const DeltaDims &d) { return delta_saved_snap(d) + delta_up(delta_chunks(d) * d.C * d.Dv * 4); }
size_t delta_saved(const DeltaDims &d) { return delta_saved_units(d) + delta_up(delta_unit_bytes(d)); }

DeltaPlanes delta_planes(const DeltaDims &d, const void *x, const long long *s, unsigned char *split) {
    DeltaPlanes p;
    if (d.dtype == SDM_BF16) {
        p.p = static_cast<const __nv_bfloat16 *>(x);
        p.plane = 0;
        for (int i = 0; i < 3; ++i) p.s[i] = s[i];
    } else {
        p.p = reinterpret_cast<const __nv_bfloat16 *>(split);
        p.plane = (long long)d.B * d.T * d.Hk * d.Dk;
        p.s[0] = (long long)d.T * d.Hk * d.Dk;
        p.s[1] = (long long)d.Hk * d.Dk;
        p.s[2] = d.Dk;
    }
    return p;
}

// the chunk-local work: planes of float32 keys and queries, X, P and the gates
cudaError_t delta_local(const DeltaDims &d, const DeltaIn &in, const DeltaLayout &l, unsigned char *ws,
                        DeltaPlanes &q, DeltaPlanes &k, DeltaLocal &w, cudaStream_t st) {
    q = delta_planes(d, in.q, d.qs, ws + l.q);
    k = delta_planes(d, in.k, d.ks, ws + l.k);
    w = DeltaLocal{ws + l.x, ws + l.p, reinterpret_cast<float *>(ws + l.aux), reinterpret_cast<DevStatus *>(ws),
                   reinterpret_cast<float *>(ws + l.starts), reinterpret_cast<float *>(ws + l.units)};
    if (d.dtype == SDM_F32) {
        const cudaError_t e = launch_delta_split(d, in.q, in.k, const_cast<__nv_bfloat16 *>(q.p), const_cast<__nv_bfloat16 *>(k.p), st);
        if (e != cudaSuccess) return e;
    }
    return launch_delta_local(d, in, q, k, w, st);
}

// The status block of a workspace that no kernel of this call clears (one too small to hold it is no workspace:
// such calls need none)
cudaError_t delta_clear(void *ws, size_t have, cudaStream_t st) {
    return ws && have >= kAlign ? cudaMemsetAsync(ws, 0, sizeof(DevStatus), st) : cudaSuccess;
}

int delta_check_ws(const char *what, const void *ws, size_t have, size_t need) {
    if (!ws || have < need || (uintptr_t)ws % kAlign)
        return set_error(SDM_ERR_WORKSPACE, "gated delta: %s NULL, too small (%zu of %zu bytes) "
                         "or not %zu-byte aligned", what, have, need, (size_t)kAlign);
    return SDM_OK;
}

}  // namespace
}  // namespace sdm

using namespace sdm;

namespace {

// sdm_gated_delta and, with `saved`, sdm_gated_delta_save
int delta_forward(const sdm_delta_shape *shape, float *state, const void *q, const void *k, const void *v,
                  const float *log_decay, const float *beta, const int32_t *valid_tokens, void *readings,
                  bool save, void *saved, size_t saved_bytes, void *workspace, size_t workspace_bytes,
                  void *stream) {
    DeltaDims d;
    int rc = delta_check(shape, d, false);
    if (rc != SDM_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d.B == 0 || d.T == 0) return delta_status(delta_clear(workspace, workspace_bytes, st));
    rc = delta_check_inputs(q, k, v, log_decay, beta);
    if (rc != SDM_OK) return rc;
    if (!state || !readings) return set_error(SDM_ERR_INVALID, "gated delta: NULL pointer");
    if (off16(state) || off16(readings))
        return set_error(SDM_ERR_INVALID, "gated delta: the state and the readings must be 16-byte aligned");
    DeltaIn in{q, k, v, log_decay, beta, valid_tokens};
    if (!save && by_token(d)) {
        const cudaError_t e = delta_clear(workspace, workspace_bytes, st);
        return delta_status(e == cudaSuccess ? launch_delta_step(d, in, state, readings, st) : e);
    }
    const DeltaLayout l = delta_layout(d, false);
    rc = delta_check_ws("workspace", workspace, workspace_bytes, l.bytes);
    if (rc == SDM_OK && save) rc = delta_check_ws("saved buffer", saved, saved_bytes, delta_saved(d));
    if (rc != SDM_OK) return rc;
    DeltaPlanes qp, kp;
    DeltaLocal w{};
    auto ws = static_cast<unsigned char *>(workspace);
    cudaError_t e = delta_unroll(d, l, ws, 0, in.q, st);
    if (e == cudaSuccess) e = delta_unroll(d, l, ws, 1, in.k, st);
    if (e == cudaSuccess) e = delta_unroll(d, l, ws, 2, in.v, st);
    if (e == cudaSuccess) e = delta_local(d, in, l, ws, qp, kp, w, st);
    if (save) w.units = reinterpret_cast<float *>(static_cast<unsigned char *>(saved) + delta_saved_units(d));
    float *snap = save ? static_cast<float *>(saved) : nullptr;
    float *r = save ? reinterpret_cast<float *>(static_cast<unsigned char *>(saved) + delta_saved_snap(d)) : nullptr;
    if (e == cudaSuccess)
        e = d.tc ? launch_delta_scan_tc(d, in, w, state, readings, snap, r, st)
                 : launch_delta_scan(d, in, qp, kp, w, state, readings, snap, r, st);
    return delta_status(e);
}

}  // namespace

extern "C" {

size_t sdm_gated_delta_workspace_bytes(const sdm_delta_shape *shape) {
    DeltaDims d;
    if (delta_check(shape, d, false) != SDM_OK) return 0;
    return delta_layout(d, false).bytes + kAlign;
}

int sdm_gated_delta(const sdm_delta_shape *shape, float *state, const void *q, const void *k,
                    const void *v, const float *log_decay, const float *beta,
                    const int32_t *valid_tokens, void *readings, void *workspace,
                    size_t workspace_bytes, void *stream) {
    return delta_forward(shape, state, q, k, v, log_decay, beta, valid_tokens, readings, false, nullptr, 0,
                         workspace, workspace_bytes, stream);
}

size_t sdm_gated_delta_saved_bytes(const sdm_delta_shape *shape) {
    DeltaDims d;
    if (delta_check(shape, d, false) != SDM_OK) return 0;
    return delta_saved(d) + kAlign;
}

int sdm_gated_delta_save(const sdm_delta_shape *shape, float *state, const void *q, const void *k,
                         const void *v, const float *log_decay, const float *beta,
                         const int32_t *valid_tokens, void *readings, void *saved,
                         size_t saved_bytes, void *workspace, size_t workspace_bytes, void *stream) {
    return delta_forward(shape, state, q, k, v, log_decay, beta, valid_tokens, readings, true, saved,
                         saved_bytes, workspace, workspace_bytes, stream);
}

size_t sdm_gated_delta_backward_workspace_bytes(const sdm_delta_shape *shape) {
    DeltaDims d;
    if (delta_check(shape, d, true) != SDM_OK) return 0;
    return delta_layout(d, true).bytes + kAlign;
}

int sdm_gated_delta_backward(const sdm_delta_shape *shape, const void *q, const void *k, const void *v,
                             const float *log_decay, const float *beta, const int32_t *valid_tokens,
                             const void *saved, size_t saved_bytes, const void *grad_readings,
                             const float *grad_final_state, float *grad_state, void *grad_q, void *grad_k,
                             void *grad_v, float *grad_log_decay, float *grad_beta, void *workspace,
                             size_t workspace_bytes, void *stream) {
    DeltaDims d;
    int rc = delta_check(shape, d, true);
    if (rc != SDM_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d.B == 0) return delta_status(delta_clear(workspace, workspace_bytes, st));
    if (!grad_state) return set_error(SDM_ERR_INVALID, "gated delta: NULL pointer");
    if (d.T == 0) {                      // the final state is the initial one
        const size_t bytes = (size_t)d.B * d.H * d.Dk * d.Dv * 4;
        const cudaError_t e = delta_clear(workspace, workspace_bytes, st);
        if (e != cudaSuccess) return delta_status(e);
        return delta_status(grad_final_state ? cudaMemcpyAsync(grad_state, grad_final_state, bytes, cudaMemcpyDeviceToDevice, st)
                                             : cudaMemsetAsync(grad_state, 0, bytes, st));
    }
    rc = delta_check_inputs(q, k, v, log_decay, beta);
    if (rc != SDM_OK) return rc;
    if (!grad_readings || !grad_q || !grad_k || !grad_v || !grad_log_decay || !grad_beta)
        return set_error(SDM_ERR_INVALID, "gated delta: NULL pointer");
    if (off16(grad_readings) || off16(grad_q) || off16(grad_k) || off16(grad_v))
        return set_error(SDM_ERR_INVALID, "gated delta: the gradients of q, k, v and the readings must be 16-byte aligned");
    const DeltaLayout l = delta_layout(d, true);
    rc = delta_check_ws("workspace", workspace, workspace_bytes, l.bytes);
    if (rc == SDM_OK) rc = delta_check_ws("saved buffer", saved, saved_bytes, delta_saved(d));
    if (rc != SDM_OK) return rc;
    auto ws = static_cast<unsigned char *>(workspace);
    DeltaIn in{q, k, v, log_decay, beta, valid_tokens};
    DeltaPlanes qp, kp;
    DeltaLocal w{};
    cudaError_t e = delta_unroll(d, l, ws, 0, in.q, st);
    if (e == cudaSuccess) e = delta_unroll(d, l, ws, 1, in.k, st);
    if (e == cudaSuccess) e = delta_unroll(d, l, ws, 2, in.v, st);
    if (e == cudaSuccess) e = delta_unroll(d, l, ws, 3, grad_readings, st);
    if (e == cudaSuccess) e = delta_local(d, in, l, ws, qp, kp, w, st);
    w.units = const_cast<float *>(reinterpret_cast<const float *>(static_cast<const unsigned char *>(saved) + delta_saved_units(d)));
    DeltaBack o;
    o.grad = grad_readings;
    o.state_in = grad_final_state;
    o.state_out = grad_state;
    o.grad_q = grad_q;
    o.grad_k = grad_k;
    o.grad_v = grad_v;
    o.grad_decay = grad_log_decay;
    o.grad_beta = grad_beta;
    o.snap = static_cast<const float *>(saved);
    o.r = reinterpret_cast<const float *>(static_cast<const unsigned char *>(saved) + delta_saved_snap(d));
    o.ends = reinterpret_cast<float *>(ws + l.ends);
    o.w = reinterpret_cast<float *>(ws + l.w);
    o.dq = reinterpret_cast<float *>(ws + l.dq);
    o.dk = reinterpret_cast<float *>(ws + l.dk);
    if (e == cudaSuccess) e = d.tc ? launch_delta_back_scan_tc(d, in, w, o, st) : launch_delta_back_scan(d, in, qp, kp, w, o, st);
    if (e == cudaSuccess) e = d.tc && d.Dv <= 128 ? launch_delta_back_local_tc(d, in, w, o, st) : launch_delta_back_local(d, in, qp, kp, w, o, st);
    return delta_status(e);
}

}  // extern "C"
