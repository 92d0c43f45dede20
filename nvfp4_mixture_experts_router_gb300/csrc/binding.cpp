// Python calls of the training operators (moe_nvfp4_train.h) on torch tensors:
// checks of types, shapes and strides, then the C entry point.
//
// The forward of the layer is bound with ctypes (api.py).  These operators are
// called several times a step on data of microseconds, and there the host time
// of a call counts: reading a tensor's type, shape, strides and address from
// Python took 4 us a call, from here 0.1 (GB300 host; the C entry and its
// launch take 2 to 3).  Each function returns the status code; api.py raises
// for it.  TypeError: a wrong element type or device; ValueError: a wrong shape.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <exception>
#include <initializer_list>
#include <string>

#include "../../include/moe_nvfp4_train.h"

namespace {

// A refused argument, thrown up to the entry.
struct Refused {
    PyObject* type;
    std::string what;
};
[[noreturn]] void wrong_type(const std::string& what) { throw Refused{PyExc_TypeError, what}; }
[[noreturn]] void wrong_value(const std::string& what) { throw Refused{PyExc_ValueError, what}; }

std::string text(std::initializer_list<int64_t> shape) {
    std::string s = "[";
    for (int64_t v : shape) s += (s.size() > 1 ? ", " : "") + std::to_string(v);
    return s + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) wrong_type(std::string(name) + " must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) wrong_type(std::string(name) + " must be a CUDA tensor");
    if (t.get_device() != c10::cuda::current_device()) wrong_value(std::string(name) + " is not on the current device");
    return t;
}

// Address of a contiguous tensor of the given type and shape; of None, where
// that is allowed: null.
void* flat(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape,
           bool or_none = false) {
    if (or_none && o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type) wrong_type(std::string(name) + " must be " + c10::toString(type));
    if (t.sizes() != at::IntArrayRef(shape) || !t.is_contiguous())
        wrong_value(std::string(name) + " must be contiguous " + text(shape));
    return t.data_ptr();
}
int32_t* flat_i32(PyObject* o, const char* name, std::initializer_list<int64_t> shape) {
    return static_cast<int32_t*>(flat(o, name, at::kInt, shape));
}
float* flat_f32(PyObject* o, const char* name, std::initializer_list<int64_t> shape, bool or_none = false) {
    return static_cast<float*>(flat(o, name, at::kFloat, shape, or_none));
}
// One device element of a 32-bit integer type, or None.
uint32_t* word(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.element_size() != 4 || c10::isFloatingType(t.scalar_type()) || t.numel() != 1)
        wrong_value(std::string(name) + " must be one 32-bit integer");
    return static_cast<uint32_t*>(t.data_ptr());
}

int dtype_of(const at::Tensor& t, const char* name) {
    if (t.scalar_type() == at::kBFloat16) return MOE_DTYPE_BF16;
    if (t.scalar_type() == at::kFloat) return MOE_DTYPE_F32;
    wrong_type(std::string(name) + " must be bfloat16 or float32");
}

// A [T, H] tensor with contiguous rows.
struct Rows {
    void* p;
    int T, H, dtype;
    int64_t stride;
    at::ScalarType type;
};
Rows rows2d(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 2) wrong_value(std::string(name) + " must be [T, H]");
    const int64_t T = t.size(0), H = t.size(1);
    if (T > INT32_MAX || H > INT32_MAX) wrong_value(std::string(name) + " is too large");
    if (T > 0 && H > 1 && t.stride(1) != 1) wrong_value(std::string(name) + " must have contiguous rows");
    // the stride of a single row, and of none, says nothing
    return Rows{t.data_ptr(), (int)T, (int)H, dtype_of(t, name), T > 1 ? t.stride(0) : H, t.scalar_type()};
}

struct Space {
    void* p;
    size_t bytes;
};
Space workspace(PyObject* o) {
    const at::Tensor& t = tensor(o, "the workspace");
    if (!t.is_contiguous()) wrong_value("the workspace must be contiguous");
    return Space{t.data_ptr(), t.nbytes()};
}

// The cudaStream_t of a torch.cuda.Stream, or of the current device's current one.
void* handle(PyObject* stream) {
    if (stream == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject* h = PyObject_GetAttrString(stream, "cuda_stream");
    if (!h) {
        PyErr_Clear();
        wrong_type("stream must be a torch.cuda.Stream or None");
    }
    void* p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        wrong_type("stream must be a torch.cuda.Stream or None");
    }
    return p;
}

double number(PyObject* o, const char* name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        wrong_type(std::string(name) + " must be a number");
    }
    return v;
}
int64_t integer(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        wrong_type(std::string(name) + " must be an integer");
    }
    return v;
}
int small(int64_t v, const char* name) {
    if (v < INT32_MIN || v > INT32_MAX) wrong_value(std::string(name) + " is out of range");
    return (int)v;
}

// Token rows, expert-ordered rows of the same type and row_of_route [T, K].
struct RowArgs {
    Rows tokens;
    void* rows;
    int64_t count;
    int K;
    const int32_t* row_of_route;
};
RowArgs row_args(PyObject* tokens, const char* name, PyObject* rows, PyObject* row_of_route) {
    RowArgs a;
    a.tokens = rows2d(tokens, name);
    const at::Tensor& r = tensor(rows, "the expert-ordered rows");
    if (r.dim() != 2) wrong_value("the expert-ordered rows must be [rows, H]");
    a.count = r.size(0);
    a.rows = flat(rows, "the expert-ordered rows", a.tokens.type, {a.count, a.tokens.H});
    const at::Tensor& m = tensor(row_of_route, "row_of_route");
    if (m.dim() != 2) wrong_value("row_of_route must be [T, K]");
    a.K = small(m.size(1), "K");
    a.row_of_route = flat_i32(row_of_route, "row_of_route", {a.tokens.T, a.K});
    return a;
}

// The C entry, without the interpreter's lock: a launch may wait for room in the
// device's queue, and other threads run meanwhile (0.05 us of a call's 2.2).
template <typename... P, typename... A>
int call(moe_status (*f)(P...), const A&... a) {
    PyThreadState* const thread = PyEval_SaveThread();
    const int status = f(static_cast<P>(a)...);      // the C entries throw nothing
    PyEval_RestoreThread(thread);
    return status;
}

int sort_routes(PyObject* const* a) {
    const int E = small(integer(a[0], "E"), "E");
    const at::Tensor& ids = tensor(a[1], "topk_ids");
    if (ids.dim() != 2) wrong_value("topk_ids must be [T, K]");
    const int64_t T = ids.size(0), K = ids.size(1);
    const Space ws = workspace(a[6]);
    return call(moe_nvfp4_sort_routes, small(T, "T"), E, small(K, "K"), flat_i32(a[1], "topk_ids", {T, K}),
                flat_i32(a[2], "count", {E}), flat_i32(a[3], "offsets", {(int64_t)E + 1}),
                flat_i32(a[4], "row_of_route", {T, K}), flat_i32(a[5], "route_of_row", {T * K}), ws.p, ws.bytes,
                handle(a[7]));
}

int dispatch(PyObject* const* a) {
    if (a[0] == Py_None && a[1] == Py_None) {        // no tokens
        const Rows r = rows2d(a[3], "the expert-ordered rows");
        void* p = flat(a[3], "the expert-ordered rows", r.type, {r.T, r.H});
        return call(moe_nvfp4_dispatch, 0, r.H, 1, r.T, r.dtype, nullptr, r.H, nullptr,
                    reinterpret_cast<int32_t*>(word(a[2], "rows_used")), p, handle(a[4]));
    }
    const RowArgs r = row_args(a[0], "x", a[3], a[1]);
    return call(moe_nvfp4_dispatch, r.tokens.T, r.tokens.H, r.K, r.count, r.tokens.dtype, r.tokens.p, r.tokens.stride,
                r.row_of_route, reinterpret_cast<int32_t*>(word(a[2], "rows_used")), r.rows, handle(a[4]));
}

int dispatch_backward(PyObject* const* a) {
    const RowArgs r = row_args(a[2], "dx", a[0], a[1]);
    return call(moe_nvfp4_dispatch_backward, r.tokens.T, r.tokens.H, r.K, r.count, r.tokens.dtype, r.rows,
                r.row_of_route, r.tokens.p, r.tokens.stride, handle(a[3]));
}

int combine(PyObject* const* a) {
    const RowArgs r = row_args(a[3], "y", a[0], a[1]);
    return call(moe_nvfp4_combine, r.tokens.T, r.tokens.H, r.K, r.count, r.tokens.dtype, r.rows, r.row_of_route,
                flat_f32(a[2], "topk_w", {r.tokens.T, r.K}), r.tokens.p, r.tokens.stride, handle(a[4]));
}

int combine_backward(PyObject* const* a) {
    const RowArgs r = row_args(a[0], "dy", a[1], a[2]);
    return call(moe_nvfp4_combine_backward, r.tokens.T, r.tokens.H, r.K, r.count, r.tokens.dtype, r.tokens.p,
                r.tokens.stride, r.rows, r.row_of_route, flat_f32(a[3], "topk_w", {r.tokens.T, r.K}),
                reinterpret_cast<int32_t*>(word(a[4], "rows_used")),
                flat(a[5], "do_rows", r.tokens.type, {r.count, r.tokens.H}), flat_f32(a[6], "dw", {r.tokens.T, r.K}),
                handle(a[7]));
}

// A rule is a tuple (api.RouteRule, api.AdamWRule).
PyObject* item(PyObject* rule, Py_ssize_t i, Py_ssize_t n) {
    if (!PyTuple_Check(rule) || PyTuple_GET_SIZE(rule) != n)
        wrong_type("the rule must be a tuple of " + std::to_string(n));
    return PyTuple_GET_ITEM(rule, i);
}
moe_route_rule route_rule(PyObject* o) {
    moe_route_rule r;
    r.score = small(integer(item(o, 0, 6), "score"), "score");
    r.groups = small(integer(item(o, 1, 6), "groups"), "groups");
    r.topk_groups = small(integer(item(o, 2, 6), "topk_groups"), "topk_groups");
    r.group_score = small(integer(item(o, 3, 6), "group_score"), "group_score");
    r.renormalize = small(integer(item(o, 4, 6), "renormalize"), "renormalize");
    r.scale = (float)number(item(o, 5, 6), "scale");
    return r;
}

// [T, K] of a tensor of two dimensions: K.
int slots(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 2) wrong_value(std::string(name) + " must be [T, K]");
    return small(t.size(1), "K");
}

int route_topk(PyObject* const* a) {
    const Rows l = rows2d(a[0], "logits");
    const int K = slots(a[3], "topk_ids");
    return call(moe_nvfp4_route_topk, l.T, l.H, K, l.dtype, l.p, l.stride, flat_f32(a[1], "bias", {l.H}, true),
                route_rule(a[2]), flat_i32(a[3], "topk_ids", {l.T, K}), flat_f32(a[4], "topk_w", {l.T, K}),
                handle(a[5]));
}

int route_topk_backward(PyObject* const* a) {
    const Rows l = rows2d(a[0], "logits"), d = rows2d(a[4], "dlogits");
    if (d.dtype != l.dtype) wrong_type("dlogits must have the type of the logits");
    if (d.T != l.T || d.H != l.H) wrong_value("dlogits must have the shape of the logits");
    const int K = slots(a[1], "topk_ids");
    return call(moe_nvfp4_route_topk_backward, l.T, l.H, K, l.dtype, l.p, l.stride,
                flat_i32(a[1], "topk_ids", {l.T, K}), flat_f32(a[2], "dw", {l.T, K}), route_rule(a[3]), d.p, d.stride,
                handle(a[5]));
}

using ExpertEntry = moe_status (*)(int64_t, int, int, int, const void*, const void*, const int32_t*, const int32_t*,
                                   void*, uint32_t*, void*);

// (first operand, second operand, count, offsets, output, status, stream); the
// weights, or their gradient, give E, N and K: argument `weights`.
int expert_product(PyObject* const* a, int weights, ExpertEntry entry, bool first_is_x, const char* const* names) {
    const at::Tensor& w = tensor(a[weights], names[weights == 1 ? 1 : 2]);
    if (w.dim() != 3) wrong_value(std::string(names[weights == 1 ? 1 : 2]) + " must be [E, N, K]");
    const int64_t E = w.size(0), N = w.size(1), K = w.size(2);
    const at::Tensor& rows = tensor(a[0], names[0]);
    if (rows.dim() != 2) wrong_value(std::string(names[0]) + " must have two dimensions");
    const int64_t R = rows.size(0);
    void* first = flat(a[0], names[0], at::kBFloat16, {R, first_is_x ? K : N});
    void *second, *out;
    if (weights == 1) {
        second = flat(a[1], names[1], at::kBFloat16, {E, N, K});
        out = flat(a[4], names[2], at::kBFloat16, {R, first_is_x ? N : K});
    } else {
        second = flat(a[1], names[1], at::kBFloat16, {R, K});
        out = flat(a[4], names[2], at::kBFloat16, {E, N, K});
    }
    const at::Tensor& offsets = tensor(a[3], "offsets");
    if (offsets.scalar_type() != at::kInt) wrong_type("offsets must be Int");
    if (offsets.dim() != 1 || offsets.size(0) < E || !offsets.is_contiguous())
        wrong_value("offsets must be contiguous [E] or longer");
    return call(entry, R, small(N, "N"), small(K, "K"), small(E, "E"), first, second, flat_i32(a[2], "count", {E}),
                static_cast<const int32_t*>(offsets.data_ptr()), out, word(a[5], "status"), handle(a[6]));
}

int expert_linear(PyObject* const* a) {
    static const char* const names[] = {"x_rows", "w", "y_rows"};
    return expert_product(a, 1, moe_nvfp4_expert_linear, true, names);
}
int expert_linear_dgrad(PyObject* const* a) {
    static const char* const names[] = {"dy_rows", "w", "dx_rows"};
    return expert_product(a, 1, moe_nvfp4_expert_linear_dgrad, false, names);
}
int expert_linear_wgrad(PyObject* const* a) {
    static const char* const names[] = {"dy_rows", "x_rows", "dw"};
    return expert_product(a, 4, moe_nvfp4_expert_linear_wgrad, false, names);
}

Rows same_rows(PyObject* o, const char* name, const Rows& x) {
    const Rows r = rows2d(o, name);
    if (r.dtype != x.dtype) wrong_type(std::string(name) + " must have the type of x");
    if (r.T != x.T || r.H != x.H) wrong_value(std::string(name) + " must have the shape of x");
    return r;
}

int layer_norm(PyObject* const* a) {
    const Rows x = rows2d(a[0], "x"), y = same_rows(a[4], "y", x);
    return call(moe_nvfp4_layer_norm, x.T, x.H, x.dtype, x.p, x.stride, flat_f32(a[1], "gamma", {x.H}),
                flat_f32(a[2], "beta", {x.H}, true), (float)number(a[3], "eps"), y.p, y.stride,
                flat_f32(a[5], "mean", {x.T}, true), flat_f32(a[6], "rstd", {x.T}, true), handle(a[7]));
}

int layer_norm_backward(PyObject* const* a) {
    const Rows x = rows2d(a[1], "x"), dy = same_rows(a[0], "dy", x), dx = same_rows(a[5], "dx", x);
    const Space ws = workspace(a[8]);
    return call(moe_nvfp4_layer_norm_backward, x.T, x.H, x.dtype, dy.p, dy.stride, x.p, x.stride,
                flat_f32(a[2], "gamma", {x.H}), flat_f32(a[3], "mean", {x.T}), flat_f32(a[4], "rstd", {x.T}), dx.p,
                dx.stride, flat_f32(a[6], "dgamma", {x.H}), flat_f32(a[7], "dbeta", {x.H}, true), ws.p, ws.bytes,
                handle(a[9]));
}

// Rows that may be None.
Rows rows_or_none(PyObject* o, const char* name, const Rows& x) {
    if (o != Py_None) return same_rows(o, name, x);
    Rows r = x;
    r.p = nullptr;
    return r;
}

int rms_norm(PyObject* const* a) {
    const Rows x = rows2d(a[0], "x"), res = rows_or_none(a[1], "residual", x), h = rows_or_none(a[4], "h", x),
               y = rows_or_none(a[5], "y", x);
    void* q = flat(a[6], "q", at::kFloat8_e4m3fn, {x.T, x.H}, true);
    void* scales = nullptr;
    int mode = MOE_SCALE_ROW;
    if (a[7] != Py_None) {
        const at::Tensor& s = tensor(a[7], "scales");
        if (s.scalar_type() != at::kFloat) {
            if (s.scalar_type() != at::kFloat8_e8m0fnu && s.scalar_type() != at::kByte)
                wrong_type("scales must be float32, float8_e8m0fnu or uint8");
            mode = MOE_SCALE_MX;
            scales = flat(a[7], "scales", s.scalar_type(), {x.T, (x.H + 31) / 32});
        } else if (s.dim() == 1) {
            scales = flat_f32(a[7], "scales", {x.T});
        } else {
            mode = MOE_SCALE_BLOCK128;
            scales = flat_f32(a[7], "scales", {x.T, (x.H + 127) / 128});
        }
    }
    if (x.T > 0 && (a[6] == Py_None) != (a[7] == Py_None)) wrong_value("q and scales go together");
    return call(moe_nvfp4_rms_norm, x.T, x.H, x.dtype, x.p, x.stride, res.p, res.stride, flat_f32(a[2], "gamma", {x.H}),
                (float)number(a[3], "eps"), h.p, h.stride, y.p, y.stride, q, scales, mode,
                flat_f32(a[8], "rstd", {x.T}, true), handle(a[9]));
}

int rms_norm_backward(PyObject* const* a) {
    const Rows h = rows2d(a[2], "h"), dy = same_rows(a[0], "dy", h), dh = rows_or_none(a[1], "dh", h),
               dx = same_rows(a[5], "dx", h);
    const Space ws = workspace(a[7]);
    return call(moe_nvfp4_rms_norm_backward, h.T, h.H, h.dtype, dy.p, dy.stride, dh.p, dh.stride, h.p, h.stride,
                flat_f32(a[3], "gamma", {h.H}), flat_f32(a[4], "rstd", {h.T}), dx.p, dx.stride,
                flat_f32(a[6], "dgamma", {h.H}), ws.p, ws.bytes, handle(a[8]));
}

template <typename T>
T* address(PyObject* o) {
    return reinterpret_cast<T*>(integer(o, "an array's address"));
}

// The list's length and device and its host arrays, as addresses, then the norm,
// which is on the current device: the list has to be there too.
int list_length(PyObject* const* a, PyObject* norm) {
    const int n = small(integer(a[0], "n"), "n");
    if (n > 0 && tensor(norm, "norm").get_device() != integer(a[1], "the gradients' device"))
        wrong_value("the gradients are not on the norm's device");
    return n;
}

int grad_norm(PyObject* const* a) {
    const Space ws = workspace(a[6]);
    return call(moe_nvfp4_grad_norm, list_length(a, a[5]), address<const void* const>(a[2]),
                address<const int64_t>(a[3]), address<const int32_t>(a[4]), flat_f32(a[5], "norm", {1}), ws.p,
                ws.bytes, handle(a[7]));
}

int grad_clip(PyObject* const* a) {
    return call(moe_nvfp4_grad_clip, list_length(a, a[6]), address<const void* const>(a[2]),
                address<void* const>(a[3]), address<const int64_t>(a[4]), address<const int32_t>(a[5]),
                flat_f32(a[6], "norm", {1}), (float)number(a[7], "max_norm"), (float)number(a[8], "eps"),
                handle(a[9]));
}

// (n, the list's device, its address, the rule, step, norm, lr_step, stream)
int adamw(PyObject* const* a) {
    const int n = small(integer(a[0], "n"), "n");
    if (n > 0 && integer(a[1], "the tensors' device") != c10::cuda::current_device())
        wrong_value("the tensors are not on the current device");
    moe_adamw_rule r;
    double* const to[] = {&r.lr, &r.beta1, &r.beta2, &r.eps, &r.weight_decay, &r.max_norm, &r.clip_eps};
    for (int i = 0; i < 7; ++i) *to[i] = number(item(a[3], i, 7), "the rule's entry");
    r.step = integer(a[4], "step");
    return call(moe_nvfp4_adamw, n, address<const moe_adamw_tensor>(a[2]), r, flat_f32(a[5], "norm", {1}, true),
                flat_f32(a[6], "lr_step", {2}, true), handle(a[7]));
}

// Runs one of the functions above on n arguments; no C++ exception leaves.
template <int (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    try {
        return PyLong_FromLong(F(args));
    } catch (const Refused& r) {
        PyErr_SetString(r.type, r.what.c_str());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

template <int (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
    return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<F, N>)), METH_FASTCALL,
                       nullptr};
}

PyMethodDef g_methods[] = {
    method<sort_routes, 8>("sort_routes"),
    method<dispatch, 5>("dispatch"),
    method<dispatch_backward, 4>("dispatch_backward"),
    method<combine, 5>("combine"),
    method<combine_backward, 8>("combine_backward"),
    method<expert_linear, 7>("expert_linear"),
    method<expert_linear_dgrad, 7>("expert_linear_dgrad"),
    method<expert_linear_wgrad, 7>("expert_linear_wgrad"),
    method<layer_norm, 8>("layer_norm"),
    method<layer_norm_backward, 10>("layer_norm_backward"),
    method<route_topk, 6>("route_topk"),
    method<route_topk_backward, 6>("route_topk_backward"),
    method<rms_norm, 10>("rms_norm"),
    method<rms_norm_backward, 9>("rms_norm_backward"),
    method<adamw, 8>("adamw"),
    method<grad_norm, 8>("grad_norm"),
    method<grad_clip, 10>("grad_clip"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    PyObject* m = PyModule_Create(&g_module);
    // the torch it was compiled for: another one's tensors may be laid out differently
    if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
