// The everyday calls of gated_delta, linear_attention, layer_norm and group_norm without the interpreter's share: a CPython module that
// reads the tensors' properties, allocates the results and calls libsdm.so's C ABI. It takes a call whose
// arguments are all in order (CUDA tensors of the current device, the right shapes and types, contiguous
// rows) and answers None for any other: the Python binding then does the same with its full checks and
// their messages. A call of a few microseconds' work costs the host 5 to 7 us this way, 13 to 19 by the
// interpreted checks and ctypes.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "sdm.h"

namespace {

PyObject *g_tensor, *g_parameter, *g_f32, *g_bf16, *g_i32, *g_u8, *g_empty, *g_empty_like, *g_device, *g_stream, *g_check;
PyObject *s_dtype, *s_shape, *s_device, *s_get_device, *s_is_contiguous, *s_stride, *s_data_ptr, *k_empty;
PyObject *s_grad_x, *s_grad_weight, *s_grad_bias, *s_grad_q, *s_grad_k, *s_grad_v, *s_grad_state, *s_grad_log_decay, *s_silu;

decltype(&sdm_gated_delta) f_delta;
decltype(&sdm_gated_delta_workspace_bytes) f_delta_bytes;
decltype(&sdm_layer_norm) f_norm;
decltype(&sdm_layer_norm_backward) f_norm_back;
decltype(&sdm_layer_norm_workspace_bytes) f_norm_bytes;
decltype(&sdm_linear_attention) f_linear;
decltype(&sdm_linear_attention_workspace_bytes) f_linear_bytes;
decltype(&sdm_linear_attention_save) f_linear_save;
decltype(&sdm_linear_attention_saved_bytes) f_linear_saved;
decltype(&sdm_linear_attention_backward) f_linear_back;
decltype(&sdm_linear_attention_backward_workspace_bytes) f_linear_back_bytes;
decltype(&sdm_group_norm) f_group;
decltype(&sdm_group_norm_workspace_bytes) f_group_bytes;
decltype(&sdm_group_norm_backward) f_group_back;
decltype(&sdm_group_norm_backward_workspace_bytes) f_group_back_bytes;
long g_step_tokens, g_linear_tokens;

constexpr int kDims = 8;

struct Arg {
    void *ptr;
    PyObject *dtype;                     // a torch.dtype is one object for good: compared, never used
    long device;
    Py_ssize_t dims;
    int64_t shape[kDims], stride[kDims], count;
    bool contiguous;
};

bool numbers(PyObject *tuple, Py_ssize_t n, int64_t *out) {
    if (!tuple || !PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) != n) return false;
    for (Py_ssize_t i = 0; i < n; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    return true;
}

// a plain tensor's properties; false (perhaps with an exception set) for anything else
bool read(PyObject *t, Arg &a) {
    if ((PyObject *)Py_TYPE(t) != g_tensor && (PyObject *)Py_TYPE(t) != g_parameter) return false;
    PyObject *x = PyObject_GetAttr(t, s_dtype);
    if (!x) return false;
    a.dtype = x;
    Py_DECREF(x);
    x = PyObject_CallMethodNoArgs(t, s_get_device);
    if (!x) return false;
    a.device = PyLong_AsLong(x);
    Py_DECREF(x);
    if (a.device < 0) return false;
    x = PyObject_GetAttr(t, s_shape);
    if (!x) return false;
    a.dims = PyTuple_Check(x) ? PyTuple_GET_SIZE(x) : kDims + 1;
    bool ok = a.dims <= kDims && numbers(x, a.dims, a.shape);
    Py_DECREF(x);
    if (!ok) return false;
    x = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!x) return false;
    a.contiguous = x == Py_True;
    Py_DECREF(x);
    a.count = 1;
    for (Py_ssize_t i = a.dims - 1; i >= 0; --i) {
        a.stride[i] = a.count;
        a.count *= a.shape[i];
    }
    if (!a.contiguous) {
        x = PyObject_CallMethodNoArgs(t, s_stride);
        ok = numbers(x, a.dims, a.stride);
        Py_XDECREF(x);
        if (!ok) return false;
    }
    x = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!x) return false;
    a.ptr = PyLong_AsVoidPtr(x);
    Py_DECREF(x);
    return !PyErr_Occurred();
}

bool is(const Arg &a, PyObject *dtype, long device, std::initializer_list<int64_t> shape) {
    if (a.dtype != dtype || a.device != device || a.dims != (Py_ssize_t)shape.size()) return false;
    Py_ssize_t i = 0;
    for (int64_t n : shape)
        if (a.shape[i++] != n) return false;
    return true;
}

PyObject *not_here() {
    PyErr_Clear();
    Py_RETURN_NONE;
}

// the current stream of the device, if that is the current one
bool stream_of(long device, void *&stream) {
    PyObject *x = PyObject_CallNoArgs(g_device);
    if (!x) return false;
    const long now = PyLong_AsLong(x);
    if (now == device) {
        PyObject *s = PyObject_CallOneArg(g_stream, x);
        if (s) stream = PyLong_AsVoidPtr(s);
        Py_XDECREF(s);
    }
    Py_DECREF(x);
    return now == device && !PyErr_Occurred();
}

// torch.empty(size, dtype, on t's device); steals size
PyObject *empty(PyObject *size, PyObject *dtype, PyObject *t) {
    PyObject *device = size ? PyObject_GetAttr(t, s_device) : nullptr;
    PyObject *args[3] = {size, dtype, device};
    PyObject *out = device ? PyObject_Vectorcall(g_empty, args, 1, k_empty) : nullptr;
    Py_XDECREF(device);
    Py_XDECREF(size);
    return out;
}

void *address(PyObject *t) {
    PyObject *x = PyObject_CallMethodNoArgs(t, s_data_ptr);
    void *p = x ? PyLong_AsVoidPtr(x) : nullptr;
    Py_XDECREF(x);
    return p;
}

// the library's answer: 0, or its error raised
bool accepted(int rc) {
    if (rc == 0) return true;
    PyObject *code = PyLong_FromLong(rc), *x = code ? PyObject_CallOneArg(g_check, code) : nullptr;
    Py_XDECREF(code);
    if (x) PyErr_SetString(PyExc_RuntimeError, "libsdm.so refused a call without a message");
    Py_XDECREF(x);
    return false;
}

int code_of(PyObject *dtype) { return dtype == g_bf16 ? SDM_BF16 : dtype == g_f32 ? SDM_F32 : -1; }

// (state, q, k, v, log_decay, beta, valid_tokens, scale, readings or None) -> readings, or None
PyObject *gated_delta(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 9) return not_here();
    Arg state, q, k, v, g, beta, valid{}, given;
    if (!read(args[3], v)) return not_here();
    const int code = code_of(v.dtype);
    if (code < 0 || v.dims != 4 || !read(args[1], q) || q.dims != 4) return not_here();
    const int64_t B = v.shape[0], T = v.shape[1], H = v.shape[2], Dv = v.shape[3], Hk = q.shape[2], Dk = q.shape[3];
    if (v.count == 0 || q.count == 0 || v.count > INT32_MAX || q.count > INT32_MAX) return not_here();
    if (!is(q, v.dtype, v.device, {B, T, Hk, Dk}) || !read(args[2], k) || !is(k, v.dtype, v.device, {B, T, Hk, Dk}) ||
        !read(args[4], g) || !is(g, g_f32, v.device, {B, T, H}) || !read(args[5], beta) || !is(beta, g_f32, v.device, {B, T, H}) ||
        !read(args[0], state) || !is(state, g_f32, v.device, {B, H, Dk, Dv}) || !state.contiguous)
        return not_here();
    if (args[8] != Py_None && (!read(args[8], given) || !is(given, v.dtype, v.device, {B, T, H, Dv}) || !given.contiguous)) return not_here();
    if (args[6] != Py_None && (!read(args[6], valid) || !is(valid, g_i32, v.device, {B}) || !valid.contiguous)) return not_here();
    const double scale = args[7] == Py_None ? pow((double)Dk, -0.5) : PyFloat_AsDouble(args[7]);
    if (PyErr_Occurred()) return not_here();
    sdm_delta_shape shape{(int32_t)B, (int32_t)T, (int32_t)H, (int32_t)Hk, (int32_t)Dk, (int32_t)Dv, code, (float)scale, {}, {}, {}, {}, {}, {}};
    const int64_t bytes = code == SDM_BF16 ? 2 : 4;
    auto strides = [&](const Arg &a, int64_t *out, bool rows) {
        int64_t all = 0;
        for (int i = 0; i < 3; ++i) {
            out[i] = a.shape[i] > 1 ? a.stride[i] : 0;             // a dimension of one is never stepped along
            all |= out[i];
        }
        return !rows || ((all * bytes | (int64_t)(intptr_t)a.ptr) % 16 == 0 && a.stride[3] == 1);
    };
    if (!strides(q, shape.q_stride, true) || !strides(k, shape.k_stride, true) || !strides(v, shape.v_stride, true) ||
        !strides(g, shape.decay_stride, false) || !strides(beta, shape.beta_stride, false))
        return not_here();
    void *stream;
    if (!stream_of(v.device, stream)) return not_here();
    PyObject *sizes = Py_BuildValue("(LLLL)", (long long)B, (long long)T, (long long)H, (long long)Dv);
    PyObject *out = args[8] != Py_None ? Py_NewRef(args[8]) : v.contiguous ? PyObject_CallOneArg(g_empty_like, args[3]) : empty(Py_XNewRef(sizes), v.dtype, args[3]);
    Py_XDECREF(sizes);
    if (!out) return nullptr;
    PyObject *ws = nullptr;
    size_t need = 0;
    bool ok = true;
    if (T > g_step_tokens) {
        need = f_delta_bytes(&shape);
        ok = need ? (ws = empty(PyLong_FromSize_t(need), g_u8, args[3])) != nullptr : accepted(SDM_ERR_INVALID);
    }
    if (ok) {
        void *o = address(out), *w = ws ? address(ws) : nullptr;
        int rc;
        Py_BEGIN_ALLOW_THREADS
        rc = f_delta(&shape, (float *)state.ptr, q.ptr, k.ptr, v.ptr, (float *)g.ptr, (float *)beta.ptr, (int32_t *)valid.ptr, o, w, need, stream);
        Py_END_ALLOW_THREADS
        ok = accepted(rc);
    }
    Py_XDECREF(ws);
    if (ok) return out;
    Py_DECREF(out);
    return nullptr;
}

// weight and bias of n columns, each None or a tensor: their type's code, or -1
int norm_params(const Arg &x, int64_t n, PyObject *weight, PyObject *bias, Arg &w, Arg &b) {
    PyObject *dtype = nullptr;
    for (int i = 0; i < 2; ++i) {
        PyObject *t = i ? bias : weight;
        Arg &a = i ? b : w;
        a.ptr = nullptr;
        if (t == Py_None) continue;
        if (!read(t, a) || (a.dtype != g_f32 && a.dtype != x.dtype) || (dtype && a.dtype != dtype) || !is(a, a.dtype, x.device, {n}) || !a.contiguous)
            return -1;
        dtype = a.dtype;
    }
    return dtype ? code_of(dtype) : SDM_F32;
}

bool norm_rows(const Arg &x, int &code, int64_t &n, int64_t &rows) {
    code = code_of(x.dtype);
    if (code < 0 || x.dims < 1 || !x.contiguous || x.count == 0) return false;
    n = x.shape[x.dims - 1];
    rows = x.count / n;
    return n <= INT32_MAX;
}

PyObject *stats_size(const Arg &x) {
    PyObject *size = PyTuple_New(x.dims);
    for (Py_ssize_t i = 0; size && i < x.dims; ++i) PyTuple_SET_ITEM(size, i, PyLong_FromLongLong(i + 1 < x.dims ? x.shape[i] : 2));
    return size;
}

// (x, weight, bias, eps, save) -> y, with save (y, stats), or None
PyObject *layer_norm(PyObject *, PyObject *const *args, Py_ssize_t count) {
    Arg x, w, b;
    int code;
    int64_t n, rows;
    if (count != 5 || !read(args[0], x) || !norm_rows(x, code, n, rows)) return not_here();
    const int wcode = norm_params(x, n, args[1], args[2], w, b);
    const double eps = PyFloat_AsDouble(args[3]);
    void *stream;
    if (wcode < 0 || PyErr_Occurred() || !stream_of(x.device, stream)) return not_here();
    PyObject *y = PyObject_CallOneArg(g_empty_like, args[0]);
    PyObject *stats = y && args[4] == Py_True ? empty(stats_size(x), g_f32, args[0]) : nullptr;
    bool ok = y && (stats || args[4] != Py_True);
    if (ok) {
        void *o = address(y);
        float *s = stats ? (float *)address(stats) : nullptr;
        int rc;
        Py_BEGIN_ALLOW_THREADS
        rc = f_norm(x.ptr, rows, (int)n, n, w.ptr, b.ptr, wcode, (float)eps, code, o, s, stream);
        Py_END_ALLOW_THREADS
        ok = accepted(rc);
    }
    PyObject *out = !ok ? nullptr : stats ? PyTuple_Pack(2, y, stats) : Py_NewRef(y);
    Py_XDECREF(y);
    Py_XDECREF(stats);
    return out;
}

// (grad, x, weight, stats, bias) -> {grad_x, grad_weight, grad_bias}, or None
PyObject *layer_norm_backward(PyObject *, PyObject *const *args, Py_ssize_t count) {
    Arg grad, x, w, none, stats;
    int code;
    int64_t n, rows;
    if (count != 5 || !read(args[1], x) || !norm_rows(x, code, n, rows) || !read(args[0], grad) || !grad.contiguous ||
        grad.dtype != x.dtype || grad.device != x.device || grad.dims != x.dims || !read(args[3], stats) || !stats.contiguous ||
        stats.dtype != g_f32 || stats.device != x.device || stats.dims != x.dims || stats.shape[x.dims - 1] != 2)
        return not_here();
    for (Py_ssize_t i = 0; i < x.dims; ++i)
        if (grad.shape[i] != x.shape[i] || (i + 1 < x.dims && stats.shape[i] != x.shape[i])) return not_here();
    const int wcode = norm_params(x, n, args[2], Py_None, w, none), bias = PyObject_IsTrue(args[4]);
    void *stream;
    if (wcode < 0 || bias < 0 || !stream_of(x.device, stream)) return not_here();
    const size_t need = f_norm_bytes(rows, (int)n);
    if (!need) return not_here();
    PyObject *gx = PyObject_CallOneArg(g_empty_like, args[1]), *gw = nullptr, *gb = nullptr, *ws = nullptr, *out = PyDict_New();
    bool ok = gx && out && PyDict_SetItem(out, s_grad_x, gx) == 0;
    if (ok && w.ptr) ok = (gw = empty(PyLong_FromLongLong(n), g_f32, args[1])) && PyDict_SetItem(out, s_grad_weight, gw) == 0;
    if (ok && bias) ok = (gb = empty(PyLong_FromLongLong(n), g_f32, args[1])) && PyDict_SetItem(out, s_grad_bias, gb) == 0;
    if (ok) ok = (ws = empty(PyLong_FromSize_t(need), g_u8, args[1])) != nullptr;
    if (ok) {
        void *px = address(gx), *pw = gw ? address(gw) : nullptr, *pb = gb ? address(gb) : nullptr, *s = address(ws);
        int rc;
        Py_BEGIN_ALLOW_THREADS
        rc = f_norm_back(grad.ptr, n, x.ptr, n, rows, (int)n, w.ptr, wcode, (float *)stats.ptr, code, px, (float *)pw, (float *)pb, s, need, stream);
        Py_END_ALLOW_THREADS
        ok = accepted(rc);
    }
    Py_XDECREF(gx);
    Py_XDECREF(gw);
    Py_XDECREF(gb);
    Py_XDECREF(ws);
    if (ok) return out;
    Py_XDECREF(out);
    return nullptr;
}

// An object held for the length of a call
struct Held {
    PyObject *p;
    explicit Held(PyObject *x = nullptr) : p(x) {}
    Held(const Held &) = delete;
    ~Held() { Py_XDECREF(p); }
    bool make(PyObject *x) {
        Py_XDECREF(p);
        p = x;
        return x != nullptr;
    }
    PyObject *give() {
        PyObject *x = p;
        p = nullptr;
        return x;
    }
    void *at() const { return p ? address(p) : nullptr; }
};

PyObject *sizes(std::initializer_list<int64_t> shape) {
    PyObject *t = PyTuple_New((Py_ssize_t)shape.size());
    Py_ssize_t i = 0;
    for (int64_t n : shape) {
        if (!t) break;
        PyTuple_SET_ITEM(t, i++, PyLong_FromLongLong(n));
    }
    return t;
}

// (b, t, h) strides of rows [B, T, heads, width]; whether they and the address are multiples of 16 bytes
bool row_strides(const Arg &a, int64_t bytes, int64_t *out) {
    int64_t all = 0;
    for (int i = 0; i < 3; ++i) {
        out[i] = a.shape[i] > 1 ? a.stride[i] : 0;                 // a dimension of one is never stepped along
        all |= out[i];
    }
    return (all * bytes | (int64_t)(intptr_t)a.ptr) % 16 == 0 && (a.stride[3] == 1 || a.shape[3] == 1);
}

// what linear attention's calls have in common: q, k, v, log_decay, valid_tokens, scale
struct Linear {
    Arg q, k, v, g, valid{};
    sdm_linear_shape shape{};
    int64_t B, T, H, Hk, Dk, Dv, bytes;
    void *stream;
    bool take(PyObject *pq, PyObject *pk, PyObject *pv, PyObject *pg, PyObject *pvalid, PyObject *pscale) {
        if (!read(pv, v)) return false;
        const int code = code_of(v.dtype);
        if (code < 0 || v.dims != 4 || !read(pq, q) || q.dims != 4) return false;
        B = v.shape[0], T = v.shape[1], H = v.shape[2], Dv = v.shape[3], Hk = q.shape[2], Dk = q.shape[3];
        if (v.count == 0 || q.count == 0 || v.count > INT32_MAX || q.count > INT32_MAX) return false;
        if (!is(q, v.dtype, v.device, {B, T, Hk, Dk}) || !read(pk, k) || !is(k, v.dtype, v.device, {B, T, Hk, Dk}) || !read(pg, g) ||
            !is(g, g_f32, v.device, {H}) || !g.contiguous)
            return false;
        if (pvalid != Py_None && (!read(pvalid, valid) || !is(valid, g_i32, v.device, {B}) || !valid.contiguous)) return false;
        const double scale = pscale == Py_None ? pow((double)Dk, -0.5) : PyFloat_AsDouble(pscale);
        if (PyErr_Occurred()) return false;
        bytes = code == SDM_BF16 ? 2 : 4;
        shape = sdm_linear_shape{(int32_t)B, (int32_t)T, (int32_t)H, (int32_t)Hk, (int32_t)Dk, (int32_t)Dv, code, (float)scale, {}, {}, {}, {}};
        return row_strides(q, bytes, shape.q_stride) && row_strides(k, bytes, shape.k_stride) && row_strides(v, bytes, shape.v_stride) &&
               stream_of(v.device, stream);
    }
    bool state(PyObject *t, Arg &a) const { return read(t, a) && is(a, g_f32, v.device, {B, H, Dk, Dv}) && a.contiguous; }
    // a new tensor [B, T, heads, width]
    PyObject *rows(PyObject *like, int64_t heads, int64_t width) const { return empty(sizes({B, T, heads, width}), v.dtype, like); }
};

// (state, q, k, v, log_decay, valid_tokens, scale, readings or None, save) -> readings, with save (readings, saved), or None
PyObject *linear_attention(PyObject *, PyObject *const *args, Py_ssize_t n) {
    Linear l;
    Arg state, given;
    if (n != 9 || !l.take(args[1], args[2], args[3], args[4], args[5], args[6]) || !l.state(args[0], state)) return not_here();
    if (args[7] != Py_None && (!read(args[7], given) || !is(given, l.v.dtype, l.v.device, {l.B, l.T, l.H, l.Dv}) || !given.contiguous))
        return not_here();
    const bool save = args[8] == Py_True;
    Held out(args[7] != Py_None ? Py_NewRef(args[7]) : l.rows(args[3], l.H, l.Dv)), ws, saved;
    if (!out.p) return nullptr;
    size_t need = 0, keep = 0;
    if (save || l.T > g_linear_tokens) {
        need = f_linear_bytes(&l.shape);
        if (!need) {
            accepted(SDM_ERR_INVALID);
            return nullptr;
        }
        if (!ws.make(empty(PyLong_FromSize_t(need), g_u8, args[3]))) return nullptr;
    }
    if (save) {
        keep = f_linear_saved(&l.shape);
        if (!saved.make(empty(PyLong_FromSize_t(keep), g_u8, args[3]))) return nullptr;
    }
    void *o = out.at(), *w = ws.at(), *s = saved.at();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = save ? f_linear_save(&l.shape, (float *)state.ptr, l.q.ptr, l.k.ptr, l.v.ptr, (float *)l.g.ptr, (int32_t *)l.valid.ptr, o, s, keep, w, need, l.stream)
              : f_linear(&l.shape, (float *)state.ptr, l.q.ptr, l.k.ptr, l.v.ptr, (float *)l.g.ptr, (int32_t *)l.valid.ptr, o, w, need, l.stream);
    Py_END_ALLOW_THREADS
    if (!accepted(rc)) return nullptr;
    return save ? PyTuple_Pack(2, out.p, saved.p) : out.give();
}

// (q, k, v, log_decay, valid_tokens, saved, grad_readings, grad_state, scale, decay) -> a dict of gradients, or None
PyObject *linear_attention_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    Linear l;
    Arg saved, grad, end{};
    if (n != 10 || !l.take(args[0], args[1], args[2], args[3], args[4], args[8])) return not_here();
    if (!read(args[5], saved) || saved.dtype != g_u8 || saved.device != l.v.device || !saved.contiguous || !read(args[6], grad) ||
        !is(grad, l.v.dtype, l.v.device, {l.B, l.T, l.H, l.Dv}) || !row_strides(grad, l.bytes, l.shape.grad_stride))
        return not_here();
    if (args[7] != Py_None && !l.state(args[7], end)) return not_here();
    const int decay = PyObject_IsTrue(args[9]);
    const size_t need = decay < 0 ? 0 : f_linear_back_bytes(&l.shape);
    if (!need) return not_here();
    Held dq(l.rows(args[2], l.Hk, l.Dk)), dk(l.rows(args[2], l.Hk, l.Dk)), dv(l.rows(args[2], l.H, l.Dv)),
        ds(empty(sizes({l.B, l.H, l.Dk, l.Dv}), g_f32, args[2])), dg, ws(empty(PyLong_FromSize_t(need), g_u8, args[2])), out(PyDict_New());
    if (!dq.p || !dk.p || !dv.p || !ds.p || !ws.p || !out.p || PyDict_SetItem(out.p, s_grad_q, dq.p) || PyDict_SetItem(out.p, s_grad_k, dk.p) ||
        PyDict_SetItem(out.p, s_grad_v, dv.p) || PyDict_SetItem(out.p, s_grad_state, ds.p))
        return nullptr;
    if (decay && (!dg.make(empty(PyLong_FromLongLong(l.H), g_f32, args[2])) || PyDict_SetItem(out.p, s_grad_log_decay, dg.p))) return nullptr;
    void *pq = dq.at(), *pk = dk.at(), *pv = dv.at(), *ps = ds.at(), *pg = dg.at(), *w = ws.at();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f_linear_back(&l.shape, l.q.ptr, l.k.ptr, l.v.ptr, (float *)l.g.ptr, (int32_t *)l.valid.ptr, saved.ptr, (size_t)saved.count, grad.ptr,
                       (float *)end.ptr, (float *)ps, pq, pk, pv, (float *)pg, w, need, l.stream);
    Py_END_ALLOW_THREADS
    return accepted(rc) ? out.give() : nullptr;
}

// x [N, ..., C] contiguous, its groups and activation
struct Group {
    Arg x;
    int code, act;
    int64_t N, L, C, G;
    void *stream;
    bool take(PyObject *px, PyObject *groups, PyObject *activation) {
        if (!read(px, x) || x.dims < 2 || !x.contiguous || x.count == 0 || (code = code_of(x.dtype)) < 0 || !PyLong_CheckExact(groups)) return false;
        N = x.shape[0], C = x.shape[x.dims - 1], L = x.count / N / C, G = PyLong_AsLongLong(groups);
        if (PyErr_Occurred() || C > INT32_MAX || G < 1 || C % G) return false;
        if (activation == Py_None) act = SDM_ACT_NONE;
        else if (PyUnicode_Check(activation) && PyUnicode_Compare(activation, s_silu) == 0) act = SDM_ACT_SILU;
        else return false;
        return stream_of(x.device, stream);
    }
};

// (x, groups, weight, bias, activation, eps, save) -> y, with save (y, stats), or None
PyObject *group_norm(PyObject *, PyObject *const *args, Py_ssize_t count) {
    Group g;
    Arg w, b;
    if (count != 7 || !g.take(args[0], args[1], args[4])) return not_here();
    const int wcode = norm_params(g.x, g.C, args[2], args[3], w, b);
    const double eps = PyFloat_AsDouble(args[5]);
    if (wcode < 0 || PyErr_Occurred()) return not_here();
    const bool save = args[6] == Py_True;
    const size_t need = f_group_bytes(g.N, g.L, (int)g.C, (int)g.G);
    if (!need) return not_here();
    Held y(PyObject_CallOneArg(g_empty_like, args[0])), stats, ws;
    if (!y.p || (save && !stats.make(empty(sizes({g.N, g.G, 2}), g_f32, args[0]))) ||
        (g.L > 1 || need > 256 ? !ws.make(empty(PyLong_FromSize_t(need), g_u8, args[0])) : false))
        return nullptr;
    void *o = y.at(), *s = stats.at(), *at = ws.at();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f_group(g.x.ptr, g.C, g.N, g.L, (int)g.C, (int)g.G, w.ptr, b.ptr, wcode, (float)eps, g.act, g.code, o, (float *)s, at, at ? need : 0, g.stream);
    Py_END_ALLOW_THREADS
    if (!accepted(rc)) return nullptr;
    return save ? PyTuple_Pack(2, y.p, stats.p) : y.give();
}

// (grad, x, groups, weight, bias, stats, activation) -> {grad_x, grad_weight, grad_bias}, or None
PyObject *group_norm_backward(PyObject *, PyObject *const *args, Py_ssize_t count) {
    Group g;
    Arg grad, w, b, stats;
    if (count != 7 || !g.take(args[1], args[2], args[6]) || !read(args[0], grad) || !grad.contiguous || grad.dtype != g.x.dtype ||
        grad.device != g.x.device || grad.dims != g.x.dims || !read(args[5], stats) || !is(stats, g_f32, g.x.device, {g.N, g.G, 2}) || !stats.contiguous)
        return not_here();
    for (Py_ssize_t i = 0; i < g.x.dims; ++i)
        if (grad.shape[i] != g.x.shape[i]) return not_here();
    const int wcode = norm_params(g.x, g.C, args[3], args[4], w, b);
    const size_t need = wcode < 0 ? 0 : f_group_back_bytes(g.N, g.L, (int)g.C, (int)g.G);
    if (!need) return not_here();
    Held gx(PyObject_CallOneArg(g_empty_like, args[1])), gw, gb, ws(empty(PyLong_FromSize_t(need), g_u8, args[1])), out(PyDict_New());
    if (!gx.p || !ws.p || !out.p || PyDict_SetItem(out.p, s_grad_x, gx.p)) return nullptr;
    if (w.ptr && (!gw.make(empty(PyLong_FromLongLong(g.C), g_f32, args[1])) || PyDict_SetItem(out.p, s_grad_weight, gw.p))) return nullptr;
    if (b.ptr && (!gb.make(empty(PyLong_FromLongLong(g.C), g_f32, args[1])) || PyDict_SetItem(out.p, s_grad_bias, gb.p))) return nullptr;
    void *px = gx.at(), *pw = gw.at(), *pb = gb.at(), *at = ws.at();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f_group_back(grad.ptr, g.C, g.x.ptr, g.C, g.N, g.L, (int)g.C, (int)g.G, w.ptr, b.ptr, wcode, g.act, (float *)stats.ptr, g.code, px,
                      (float *)pw, (float *)pb, at, need, g.stream);
    Py_END_ALLOW_THREADS
    return accepted(rc) ? out.give() : nullptr;
}

// the objects and the library's functions that the calls use
PyObject *setup(PyObject *, PyObject *args) {
    unsigned long long delta, delta_bytes, norm, norm_back, norm_bytes, lin[6], group[4];
    if (!PyArg_ParseTuple(args, "(OO)(OOOO)(OOOOO)ll(KKKKK)(KKKKKK)(KKKK)", &g_tensor, &g_parameter, &g_f32, &g_bf16, &g_i32, &g_u8, &g_empty,
                          &g_empty_like, &g_device, &g_stream, &g_check, &g_step_tokens, &g_linear_tokens, &delta, &delta_bytes,
                          &norm, &norm_back, &norm_bytes, lin, lin + 1, lin + 2, lin + 3, lin + 4, lin + 5, group, group + 1, group + 2, group + 3))
        return nullptr;
    for (PyObject *x : {g_tensor, g_parameter, g_f32, g_bf16, g_i32, g_u8, g_empty, g_empty_like, g_device, g_stream, g_check}) Py_INCREF(x);
    f_delta = (decltype(f_delta))(uintptr_t)delta;
    f_delta_bytes = (decltype(f_delta_bytes))(uintptr_t)delta_bytes;
    f_norm = (decltype(f_norm))(uintptr_t)norm;
    f_norm_back = (decltype(f_norm_back))(uintptr_t)norm_back;
    f_norm_bytes = (decltype(f_norm_bytes))(uintptr_t)norm_bytes;
    f_linear = (decltype(f_linear))(uintptr_t)lin[0];
    f_linear_bytes = (decltype(f_linear_bytes))(uintptr_t)lin[1];
    f_linear_save = (decltype(f_linear_save))(uintptr_t)lin[2];
    f_linear_saved = (decltype(f_linear_saved))(uintptr_t)lin[3];
    f_linear_back = (decltype(f_linear_back))(uintptr_t)lin[4];
    f_linear_back_bytes = (decltype(f_linear_back_bytes))(uintptr_t)lin[5];
    f_group = (decltype(f_group))(uintptr_t)group[0];
    f_group_bytes = (decltype(f_group_bytes))(uintptr_t)group[1];
    f_group_back = (decltype(f_group_back))(uintptr_t)group[2];
    f_group_back_bytes = (decltype(f_group_back_bytes))(uintptr_t)group[3];
    Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {{"setup", setup, METH_VARARGS, nullptr},
                          {"gated_delta", (PyCFunction)(void (*)(void))gated_delta, METH_FASTCALL, nullptr},
                          {"linear_attention", (PyCFunction)(void (*)(void))linear_attention, METH_FASTCALL, nullptr},
                          {"linear_attention_backward", (PyCFunction)(void (*)(void))linear_attention_backward, METH_FASTCALL, nullptr},
                          {"group_norm", (PyCFunction)(void (*)(void))group_norm, METH_FASTCALL, nullptr},
                          {"group_norm_backward", (PyCFunction)(void (*)(void))group_norm_backward, METH_FASTCALL, nullptr},
                          {"layer_norm", (PyCFunction)(void (*)(void))layer_norm, METH_FASTCALL, nullptr},
                          {"layer_norm_backward", (PyCFunction)(void (*)(void))layer_norm_backward, METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
    const struct { PyObject **at; const char *name; } names[] = {
        {&s_dtype, "dtype"}, {&s_shape, "shape"}, {&s_device, "device"}, {&s_get_device, "get_device"}, {&s_is_contiguous, "is_contiguous"},
        {&s_stride, "stride"}, {&s_data_ptr, "data_ptr"}, {&s_grad_x, "grad_x"}, {&s_grad_weight, "grad_weight"}, {&s_grad_bias, "grad_bias"},
        {&s_grad_q, "grad_q"}, {&s_grad_k, "grad_k"}, {&s_grad_v, "grad_v"}, {&s_grad_state, "grad_state"}, {&s_grad_log_decay, "grad_log_decay"},
        {&s_silu, "silu"}};
    for (const auto &n : names)
        if (!(*n.at = PyUnicode_InternFromString(n.name))) return nullptr;
    if (!(k_empty = PyTuple_Pack(2, s_dtype, s_device))) return nullptr;
    return PyModule_Create(&kModule);
}
