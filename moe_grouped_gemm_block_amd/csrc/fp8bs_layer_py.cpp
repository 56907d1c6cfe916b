// fp8bs_layer_py.cpp -- the short way from Python to the operators between the FP8 products: a CPython
// module that looks operands over and calls the library, for the calls of a decode step, whose host
// part is longer than their kernels.  Calls one after the other, by the binding's own checks and
// this way: norm of a row of 7168 8.0 us and 4.0, dispatch of 64 tokens of eight choices 9.6 and 4.9,
// combine 6.9 and 3.3, gated activation 7.7 and 3.8, columns of 200 x 416 6.2 and 4.0.
//
// Each function takes its operator's operands by position and answers the library's status, or -1 if
// anything is not as it should be -- a type, shape, device -- or needs more than a look (a workspace
// on another stream than the current one): nothing has been called then, and the binding's checks in
// layer.py say what is wrong, or make the call.  It never raises.
#include <Python.h>

#include <climits>

#include <ATen/ops/empty.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fp8bs.h"

namespace {

// Types of an operand, as sets.
enum : int { kF32 = 1, kBF16 = 2, kCode = 4, kI32 = 8, kI64 = 16, kByte = 32, kFloat = kF32 | kBF16 };

int type_of(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return kF32;
        case at::kBFloat16: return kBF16;
        case at::kByte: return kCode | kByte;
        case at::kFloat8_e4m3fn: return kCode;
        case at::kInt: return kI32;
        case at::kLong: return kI64;
        default: return 0;
    }
}
int code_of(int type) { return type & kF32 ? FP8BS_DTYPE_F32 : type & kBF16 ? FP8BS_DTYPE_BF16 : FP8BS_DTYPE_E4M3; }

// The library's functions and torch's current stream of a device, as the binding gives them.
decltype(&fp8bs_rms_norm) norm_fn;
decltype(&fp8bs_rms_norm_backward_workspace_size) norm_size_fn;
decltype(&fp8bs_rms_norm_backward) norm_backward_fn;
decltype(&fp8bs_moe_dispatch_workspace_size) dispatch_size_fn;
decltype(&fp8bs_moe_dispatch) dispatch_fn;
decltype(&fp8bs_moe_combine) combine_fn;
decltype(&fp8bs_moe_combine_backward) combine_backward_fn;
decltype(&fp8bs_gated_quantize) gated_fn;
decltype(&fp8bs_gated_quantize_backward) gated_backward_fn;
decltype(&fp8bs_quantize_128x1) columns_fn;
PyObject* raw_stream;

int64_t ld(int64_t rows) { return (rows + 3) & ~(int64_t)3; }

// Operands of a call, all on the device of the first, which must be the current one.
class Operands {
  public:
    explicit Operands(PyObject* first) {
        if (!THPVariable_CheckExact(first)) return;
        const at::Tensor& t = THPVariable_Unpack(first);
        if (!t.is_cuda()) return;
        index_ = t.get_device();
        ok_ = index_ == c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getDevice().index();
    }
    bool ok() const { return ok_; }
    // A dense tensor of one of `types`; nullptr, and not ok, if it is none.
    const at::Tensor* tensor(PyObject* o, int types) {
        if (ok_ && THPVariable_CheckExact(o)) {
            const at::Tensor& t = THPVariable_Unpack(o);
            if ((type_of(t) & types) && t.is_cuda() && t.get_device() == index_ &&
                t.layout() == at::kStrided && t.is_contiguous())
                return &t;
        }
        ok_ = false;
        return nullptr;
    }
    // ... of `dims` dimensions, whose sizes are ints
    const at::Tensor* tensor(PyObject* o, int types, int dims) {
        const at::Tensor* t = tensor(o, types);
        if (t && t->dim() == dims) {
            for (const int64_t n : t->sizes())
                if (n > INT_MAX) ok_ = false;
            if (ok_) return t;
        }
        ok_ = false;
        return nullptr;
    }
    // Address of an operand of a given shape; its type
    void* of(PyObject* o, int types, at::IntArrayRef shape, int* type = nullptr) {
        const at::Tensor* t = tensor(o, types);
        if (t && t->sizes() == shape) {
            if (type) *type = type_of(*t);
            return t->data_ptr();
        }
        ok_ = false;
        return nullptr;
    }
    // ... or None: nullptr
    void* optional(PyObject* o, int types, at::IntArrayRef shape, int* type = nullptr) {
        return o == Py_None ? nullptr : of(o, types, shape, type);
    }
    // float32 scales of a quantised operand; without one they are None
    float* scales(PyObject* o, bool wanted, int64_t count) {
        if (!wanted) {
            if (o != Py_None) ok_ = false;
            return nullptr;
        }
        const at::Tensor* t = tensor(o, kF32);
        if (t && t->numel() == count) return (float*)t->data_ptr();
        ok_ = false;
        return nullptr;
    }
    bool demand(bool what) { return ok_ = ok_ && what; }
    // The caller's workspace, or for None one of `bytes` (< 0: an error) from the current stream's memory
    // in `made`, which the caller keeps until the call has been made.
    const at::Tensor* workspace(PyObject* o, int64_t bytes, PyObject* stream, const at::Tensor& like,
                                at::Tensor& made) {
        if (o != Py_None) return tensor(o, kByte, 1);
        if (!demand(bytes == 0 || (bytes > 0 && stream == Py_None)) || bytes == 0) return nullptr;
        made = at::empty({bytes}, like.options().dtype(at::kByte));
        return &made;
    }
    // A stream's number, None: the current stream
    hipStream_t stream(PyObject* o) {
        if (!ok_) return nullptr;
        PyObject* own = nullptr;
        if (o == Py_None) {
            PyObject* index = PyLong_FromLong(index_);
            own = index ? PyObject_CallOneArg(raw_stream, index) : nullptr;
            Py_XDECREF(index);
            o = own;
        }
        void* p = o ? PyLong_AsVoidPtr(o) : nullptr;
        Py_XDECREF(own);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            ok_ = false;
        }
        return (hipStream_t)p;
    }

  private:
    int index_ = -1;
    bool ok_ = false;
};

int integer(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return -1;
    }
    return v < 0 || v > INT_MAX ? -1 : (int)v;
}

// x weight residual residual_out y q sfa rstd eps stream
int norm(PyObject* const* a) {
    Operands in(a[0]);
    const at::Tensor* x = in.tensor(a[0], kFloat, 2);
    if (!x) return -1;
    const int64_t rows = x->size(0), k = x->size(1);
    int wt = 0, rt = kBF16, ot = kBF16, yt = kBF16;
    const void* w = in.of(a[1], kFloat, {k}, &wt);
    const void* res = in.optional(a[2], kFloat, {rows, k}, &rt);
    void* out = in.optional(a[3], kFloat, {rows, k}, &ot);
    void* y = in.optional(a[4], kFloat, {rows, k}, &yt);
    void* q = in.optional(a[5], kCode, {rows, k});
    float* sfa = in.scales(a[6], a[5] != Py_None, k / 128 * ld(rows));
    float* rstd = (float*)in.optional(a[7], kF32, {rows});
    const double eps = PyFloat_AsDouble(a[8]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return -1;
    }
    in.demand((y || q || out) && (!res || !out || rt == ot));
    hipStream_t stream = in.stream(a[9]);
    if (!in.ok()) return -1;
    const int xt = type_of(*x);
    const void* xp = x->data_ptr();
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = norm_fn(xp, code_of(xt), res, out, code_of(res ? rt : ot), w, code_of(wt), y, code_of(yt), q, sfa,
                 rstd, (int)rows, (int)k, (float)eps, stream);
    Py_END_ALLOW_THREADS;
    return st;
}

// s rstd weight dy dx dresidual dweight accumulate workspace stream
int norm_backward(PyObject* const* a) {
    Operands in(a[0]);
    const at::Tensor* s = in.tensor(a[0], kFloat, 2);
    if (!s) return -1;
    const int64_t rows = s->size(0), k = s->size(1);
    const int type = type_of(*s);
    int wt = 0, gt = 0;
    const float* rstd = (const float*)in.of(a[1], kF32, {rows});
    const void* w = in.of(a[2], kFloat, {k}, &wt);
    const void* dy = in.of(a[3], kFloat, {rows, k}, &gt);
    void* dx = in.of(a[4], type, {rows, k});
    const void* dres = in.optional(a[5], type, {rows, k});
    float* dw = (float*)in.optional(a[6], kF32, {k});
    const int accumulate = PyObject_IsTrue(a[7]);
    if (accumulate < 0) PyErr_Clear();
    in.demand(accumulate >= 0);
    at::Tensor made;
    const at::Tensor* space =
        dw && in.ok() ? in.workspace(a[8], norm_size_fn(rows, (int)k), a[9], *s, made) : nullptr;
    hipStream_t stream = in.stream(a[9]);
    if (!in.ok()) return -1;
    const void* sp = s->data_ptr();
    void* wp = space ? space->data_ptr() : nullptr;
    const size_t bytes = space ? (size_t)space->numel() : 0;
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = norm_backward_fn(sp, code_of(type), rstd, w, code_of(wt), dy, code_of(gt), dres, dx, dw,
                          accumulate, (int)rows, (int)k, wp, bytes, stream);
    Py_END_ALLOW_THREADS;
    return st;
}

// ids x a group_data positions counts sfx sfa workspace stream
int dispatch(PyObject* const* a) {
    Operands in(a[0]);
    const at::Tensor* ids = in.tensor(a[0], kI32 | kI64, 2);
    const at::Tensor* x = in.tensor(a[1], kFloat | kCode, 2);
    const at::Tensor* counts = in.tensor(a[5], kI32, 1);
    if (!in.ok()) return -1;
    const int64_t tokens = ids->size(0), topk = ids->size(1), k = x->size(1), g = counts->size(0);
    const int type = type_of(*x);
    const bool codes = type & kCode;
    const at::Tensor* to = in.tensor(a[2], codes ? (int)kCode : type);
    if (!to || to->dim() < 2 || to->dim() > 3) return -1;
    const bool masked = to->dim() == 3;
    const int64_t m = to->size(masked ? 1 : 0);
    in.demand(x->size(0) == tokens && to->size(masked ? 2 : 1) == k && m <= INT_MAX &&
              (!masked || to->size(0) == g));
    int32_t* data = (int32_t*)in.of(a[3], kI32, {masked ? g : m});
    int32_t* positions = (int32_t*)in.of(a[4], kI32, ids->sizes());
    const float* sfx = in.scales(a[6], codes, k / 128 * ld(tokens));
    float* sfa = in.scales(a[7], codes, (masked ? g : 1) * (k / 128) * ld(m));
    if (!in.ok()) return -1;
    const int layout = masked ? FP8BS_LAYOUT_MASKED : FP8BS_LAYOUT_CONTIGUOUS;
    at::Tensor made;
    const at::Tensor* space = in.workspace(a[8], dispatch_size_fn(layout, tokens, (int)topk, (int)g, m), a[9],
                                           *x, made);
    hipStream_t stream = in.stream(a[9]);
    if (!in.ok()) return -1;
    const void *ip = ids->data_ptr(), *xp = x->data_ptr();
    void *ap = to->data_ptr(), *wp = space ? space->data_ptr() : nullptr;
    const size_t bytes = space ? (size_t)space->numel() : 0;
    int32_t* cp = (int32_t*)counts->data_ptr();
    const int id_bytes = (int)ids->element_size();
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = dispatch_fn(layout, ip, id_bytes, xp, code_of(type), sfx, ap, sfa, data, positions, cp, (int)tokens,
                     (int)topk, (int)g, (int)m, (int)k, wp, bytes, stream);
    Py_END_ALLOW_THREADS;
    return st;
}

// d positions y weights stream
int combine(PyObject* const* a) {
    Operands in(a[0]);
    const at::Tensor* d = in.tensor(a[0], kBF16);
    const at::Tensor* at = in.tensor(a[1], kI32, 2);
    const at::Tensor* y = in.tensor(a[2], kFloat, 2);
    if (!in.ok() || d->dim() < 2 || d->dim() > 3) return -1;
    const int64_t tokens = y->size(0), k = y->size(1), topk = at->size(1);
    in.demand(d->size(-1) == k && at->size(0) == tokens);
    const float* w = (const float*)in.optional(a[3], kF32, at->sizes());
    hipStream_t stream = in.stream(a[4]);
    if (!in.ok()) return -1;
    const int64_t rows = d->dim() == 3 ? d->size(0) * d->size(1) : d->size(0);
    const void* dp = d->data_ptr();
    const int32_t* pp = (const int32_t*)at->data_ptr();
    void* yp = y->data_ptr();
    const int type = code_of(type_of(*y));
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = combine_fn(dp, pp, w, yp, type, rows, (int)tokens, (int)topk, (int)k, stream);
    Py_END_ALLOW_THREADS;
    return st;
}

// dy positions d weights dd q sfa dweights stream
int combine_backward(PyObject* const* a) {
    Operands in(a[0]);
    const at::Tensor* dy = in.tensor(a[0], kFloat, 2);
    const at::Tensor* at = in.tensor(a[1], kI32, 2);
    PyObject* like = a[4] != Py_None ? a[4] : a[5] != Py_None ? a[5] : a[2];
    const at::Tensor* rows = in.tensor(like, kBF16 | kCode);
    if (!in.ok() || rows->dim() < 2 || rows->dim() > 3) return -1;
    const int64_t tokens = dy->size(0), k = dy->size(1), topk = at->size(1);
    const int64_t slots = rows->dim() == 3 ? rows->size(0) : 1, m = rows->size(-2);
    in.demand(rows->size(-1) == k && at->size(0) == tokens && slots <= INT_MAX && m <= INT_MAX);
    const void* d = in.optional(a[2], kBF16, rows->sizes());
    const float* w = (const float*)in.optional(a[3], kF32, at->sizes());
    void* dd = in.optional(a[4], kBF16, rows->sizes());
    void* q = in.optional(a[5], kCode, rows->sizes());
    float* sfa = in.scales(a[6], a[5] != Py_None, slots * (k / 128) * ld(m));
    float* dw = (float*)in.optional(a[7], kF32, at->sizes());
    in.demand((dd || q || dw) && (!dw || d));
    hipStream_t stream = in.stream(a[8]);
    if (!in.ok()) return -1;
    const void* gp = dy->data_ptr();
    const int32_t* pp = (const int32_t*)at->data_ptr();
    const int type = code_of(type_of(*dy));
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = combine_backward_fn(gp, type, d, pp, w, dd, q, sfa, dw, (int)slots, (int)m, (int)tokens, (int)topk,
                             (int)k, stream);
    Py_END_ALLOW_THREADS;
    return st;
}

// g hq sfh gq sfg grouped_layout masked_m activation stream
int gated(PyObject* const* a) {
    Operands in(a[0]);
    const bool masked = a[6] != Py_None, grouped = a[5] != Py_None;
    const at::Tensor* g = in.tensor(a[0], kBF16, masked ? 3 : 2);
    const int act = integer(a[7]);
    if (!g || act < 0 || (masked && grouped) || g->size(-1) % 2) return -1;
    const int64_t slots = masked ? g->size(0) : 1, m = g->size(-2), f = g->size(-1) / 2;
    int64_t shape[3] = {slots, m, f};
    void* hq = in.of(a[1], kCode, at::IntArrayRef(masked ? shape : shape + 1, masked ? 3 : 2));
    float* sfh = in.scales(a[2], true, slots * (f / 128) * ld(m));
    void* gq = in.optional(a[3], kCode, g->sizes());
    float* sfg = in.scales(a[4], a[3] != Py_None, slots * (2 * f / 128) * ld(m));
    const int32_t* data =
        (const int32_t*)(masked ? in.of(a[6], kI32, {slots}) : in.optional(a[5], kI32, {m}));
    hipStream_t stream = in.stream(a[8]);
    if (!in.ok()) return -1;
    const int layout = masked ? FP8BS_LAYOUT_MASKED : grouped ? FP8BS_LAYOUT_CONTIGUOUS : FP8BS_LAYOUT_DENSE;
    const void* gp = g->data_ptr();
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = gated_fn(layout, gp, hq, sfh, gq, sfg, data, (int)m, (int)f, (int)slots, act, stream);
    Py_END_ALLOW_THREADS;
    return st;
}

// g dh sfg d dq sfd dqt sfdt hqt sfht grouped_layout activation stream
int gated_backward(PyObject* const* a) {
    Operands in(a[0]);
    const at::Tensor* g = in.tensor(a[0], kBF16 | kCode, 2);
    const int act = integer(a[11]);
    if (!g || act < 0 || g->size(1) % 2) return -1;
    const int64_t m = g->size(0), f2 = g->size(1), f = f2 / 2, pad = (m + 127) / 128 * 128;
    const int type = type_of(*g);
    const void* dh = in.of(a[1], kBF16, {m, f});
    const float* sfg = in.scales(a[2], type & kCode, f2 / 128 * ld(m));
    void* d = in.optional(a[3], kBF16, {m, f2});
    void* dq = in.optional(a[4], kCode, {m, f2});
    float* sfd = in.scales(a[5], a[4] != Py_None, f2 / 128 * ld(m));
    void* dqt = in.optional(a[6], kCode, {pad, f2});
    float* sfdt = in.scales(a[7], a[6] != Py_None, pad / 128 * ld(f2));
    void* hqt = in.optional(a[8], kCode, {pad, f});
    float* sfht = in.scales(a[9], a[8] != Py_None, pad / 128 * ld(f));
    const int32_t* layout = (const int32_t*)in.optional(a[10], kI32, {m});
    in.demand(d || dq || dqt || hqt);
    hipStream_t stream = in.stream(a[12]);
    if (!in.ok()) return -1;
    const void* gp = g->data_ptr();
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = gated_backward_fn(gp, code_of(type), sfg, dh, d, dq, sfd, dqt, sfdt, hqt, sfht, layout, (int)m,
                           (int)f, act, stream);
    Py_END_ALLOW_THREADS;
    return st;
}

// x q sf sfx grouped_layout stream
int columns(PyObject* const* a) {
    Operands in(a[0]);
    const at::Tensor* x = in.tensor(a[0], kFloat | kCode, 2);
    if (!x) return -1;
    const int64_t rows = x->size(0), n = x->size(1), pad = (rows + 127) / 128 * 128;
    const int type = type_of(*x);
    void* q = in.of(a[1], kCode, {pad, n});
    float* sf = in.scales(a[2], true, pad / 128 * ld(n));
    const float* sfx = in.scales(a[3], type & kCode, n / 128 * ld(rows));
    const int32_t* layout = (const int32_t*)in.optional(a[4], kI32, {rows});
    hipStream_t stream = in.stream(a[5]);
    if (!in.ok()) return -1;
    const void* xp = x->data_ptr();
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = columns_fn(xp, code_of(type), sfx, q, sf, layout, (int)rows, (int)n, stream);
    Py_END_ALLOW_THREADS;
    return st;
}

template <int (*F)(PyObject* const*), Py_ssize_t N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t count) {
    int st = -1;
    if (count == N && raw_stream) {
        try {
            st = F(args);
        } catch (...) {                            // (torch's, of a tensor without memory of its own)
        }
    }
    return PyLong_FromLong(st);
}

// Addresses of the library's functions, in the order above, and the current stream's function.
PyObject* use(PyObject*, PyObject* args) {
    PyObject* p[11];
    if (!PyArg_UnpackTuple(args, "use", 11, 11, p, p + 1, p + 2, p + 3, p + 4, p + 5, p + 6, p + 7, p + 8, p + 9,
                           p + 10))
        return nullptr;
    void* fn[10];
    for (int i = 0; i < 10; ++i) fn[i] = PyLong_AsVoidPtr(p[i]);
    if (PyErr_Occurred()) return nullptr;
    norm_fn = (decltype(norm_fn))fn[0];
    norm_size_fn = (decltype(norm_size_fn))fn[1];
    norm_backward_fn = (decltype(norm_backward_fn))fn[2];
    dispatch_size_fn = (decltype(dispatch_size_fn))fn[3];
    dispatch_fn = (decltype(dispatch_fn))fn[4];
    combine_fn = (decltype(combine_fn))fn[5];
    combine_backward_fn = (decltype(combine_backward_fn))fn[6];
    gated_fn = (decltype(gated_fn))fn[7];
    gated_backward_fn = (decltype(gated_backward_fn))fn[8];
    columns_fn = (decltype(columns_fn))fn[9];
    Py_INCREF(p[10]);
    Py_XDECREF(raw_stream);
    raw_stream = p[10];
    Py_RETURN_NONE;
}

template <int (*F)(PyObject* const*), Py_ssize_t N>
constexpr PyMethodDef method(const char* name) {
    return {name, (PyCFunction)(void (*)())call<F, N>, METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<norm, 10>("rms_norm"),
                         method<norm_backward, 10>("rms_norm_backward"),
                         method<dispatch, 10>("moe_dispatch"),
                         method<combine, 5>("moe_combine"),
                         method<combine_backward, 9>("moe_combine_backward"),
                         method<gated, 9>("gated_quantize"),
                         method<gated_backward, 13>("gated_quantize_backward"),
                         method<columns, 6>("quantize_128x1"),
                         {"use", use, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "fp8bs_layer_py", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_fp8bs_layer_py() { return PyModule_Create(&module); }
