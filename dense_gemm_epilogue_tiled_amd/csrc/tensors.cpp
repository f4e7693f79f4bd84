// The tensor helpers of mx_ops.py and train_ops.py: checks of the tensors' types, shapes and
// pitches, new outputs and scratch, and the call of the C ABI.  In C++ because a
// decoding step calls them for microseconds of GPU work: the same steps took 11.5
// us for rms_norm in Python, 4 us of which were the launch, and take 5.3 here.
//
// Each function returns its tensors, or the C call's status if that is not GR_OK,
// and raises TypeError or ValueError for tensors that do not fit.  The caller has
// made the first tensor's device current and passes the stream's handle last.  That the
// tensors are on a GPU is checked after everything else that can be said of them.

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstdio>
#include <string>

#include "gemm_relu.h"

namespace {

using at::Tensor;

// A Python exception on its way out.
struct Raise {
    PyObject* type;
    std::string text;
};

[[noreturn]] void bad_value(const std::string& text) { throw Raise{PyExc_ValueError, text}; }
[[noreturn]] void bad_type(const std::string& text) { throw Raise{PyExc_TypeError, text}; }

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

// ---- arguments ----------------------------------------------------------------------

// These operators have no gradients: a tensor for which one is being recorded is refused,
// since its gradient would be lost without a word.
const Tensor& tensor_of(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) bad_type(std::string(what) + " must be a tensor");
    const Tensor& t = THPVariable_Unpack(o);
    if ((c10::GradMode::is_enabled() && t.requires_grad()) || t._fw_grad(0).defined())
        throw Raise{PyExc_RuntimeError, std::string(what) + " asks for a gradient, and this operator has no gradient: "
                                            "call it under torch.no_grad() or with a detached tensor"};
    return t;
}

// A tensor, or nullptr for None.
const Tensor* maybe_tensor(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor_of(o, what); }

int64_t int_of(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raise{nullptr, ""};
    return v;
}

void* stream_of(PyObject* o) {
    void* const p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Raise{nullptr, ""};
    return p;
}

// ---- tensors --------------------------------------------------------------------------

int format_of(at::ScalarType t) { return t == at::kBFloat16 ? GR_FMT_BF16 : (t == at::kHalf ? GR_FMT_F16 : -1); }

// Row pitch of a 2-D tensor with unit column stride.  Rows that share memory (an
// expanded tensor has the row stride 0) have no pitch.
int64_t pitch_of(const Tensor& t, const char* what) {
    const int64_t rows = t.size(0), cols = t.size(1);
    if (cols > 1 && rows > 0 && t.stride(1) != 1) bad_value(std::string(what) + " needs unit column stride");
    if (rows < 2 || cols == 0) return cols > 0 ? cols : 1;
    if (t.stride(0) < cols)
        bad_value(std::string(what) + " has rows that share memory: row stride " + std::to_string(t.stride(0)) + " for " +
                  std::to_string(cols) + " columns");
    return t.stride(0);
}

void on_gpu(const Tensor& t, const char* what) {
    if (!t.is_cuda()) bad_value(std::string(what) + " must be a GPU tensor");
}

template <typename T>
T* data_of(const Tensor& t) {
    return static_cast<T*>(t.data_ptr());
}

// A 16-bit matrix.
struct Matrix {
    const Tensor& t;
    int fmt;
    int64_t rows, cols, ld;
    uint16_t* data;

    Matrix(PyObject* o, const char* what) : t(tensor_of(o, what)) {
        fmt = format_of(t.scalar_type());
        if (fmt < 0) bad_type(std::string(what) + " must be float16 or bfloat16, got " + c10::toString(t.scalar_type()));
        if (t.dim() != 2) bad_value(std::string(what) + " must be 2-D");
        rows = t.size(0);
        cols = t.size(1);
        ld = pitch_of(t, what);
        data = data_of<uint16_t>(t);
    }
};

void check_place(const Tensor& t, const Tensor& like, const char* what) {
    if (t.device() != like.device()) bad_value(std::string(what) + " is on another device");
}

void check_kind(const Tensor& t, at::IntArrayRef shape, at::ScalarType kind, const char* what) {
    if (t.scalar_type() != kind || t.sizes() != shape)
        bad_value(std::string(what) + " must be " + shape_text(shape) + " of " + c10::toString(kind) + ", got " +
                  shape_text(t.sizes()) + " of " + c10::toString(t.scalar_type()));
}

// The pitch of t, which is rows x cols of `kind` next to `like`.
int64_t matching(const Tensor& t, const Tensor& like, int64_t rows, int64_t cols, at::ScalarType kind,
                 const char* what) {
    check_kind(t, {rows, cols}, kind, what);
    check_place(t, like, what);
    return pitch_of(t, what);
}

// The address of a contiguous vector of n values, nullptr for None.
template <typename T>
const T* vector_of(PyObject* o, const Tensor& like, int64_t n, at::ScalarType kind, const char* what) {
    const Tensor* t = maybe_tensor(o, what);
    if (!t) return nullptr;
    check_kind(*t, {n}, kind, what);
    if (n > 1 && t->stride(0) != 1) bad_value(std::string(what) + " must be contiguous");
    check_place(*t, like, what);
    return data_of<const T>(*t);
}

// A new tensor next to `like`, by the function behind torch.empty: some of these calls
// make three.
Tensor empty_like(const Tensor& like, at::IntArrayRef shape, at::ScalarType kind) {
    on_gpu(like, "the operand");
    return at::detail::empty_cuda(shape, kind, like.device(), c10::nullopt);
}

// The tensor given for an output, or a new one, and its pitch.
struct Output {
    Tensor t;
    int64_t ld;

    Output(PyObject* o, const Tensor& like, int64_t rows, int64_t cols, at::ScalarType kind, const char* what) {
        const Tensor* given = maybe_tensor(o, what);
        if (given) {
            t = *given;
            ld = matching(t, like, rows, cols, kind, what);
        } else {
            t = empty_like(like, {rows, cols}, kind);
            ld = cols > 0 ? cols : 1;
        }
    }
};

// Scratch of `need` bytes: new where the argument is True, a given tensor, or
// none (None).
struct Scratch {
    Tensor t;
    void* data = nullptr;
    int64_t bytes = 0;

    Scratch(PyObject* o, const Tensor& like, int64_t need) {
        if (o == Py_None) return;
        if (o == Py_True) {
            if (need == 0) return;
            t = empty_like(like, {need}, at::kByte);
        } else {
            t = tensor_of(o, "workspace");
            check_place(t, like, "workspace");
            if (!t.is_contiguous()) bad_value("workspace must be contiguous");
        }
        data = t.data_ptr();
        bytes = (int64_t)t.nbytes();
    }
};

// ---- results ----------------------------------------------------------------------------

PyObject* tuple_of(std::initializer_list<const Tensor*> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor* t : ts) {
        PyObject* o = Py_None;
        if (t && t->defined())
            o = THPVariable_Wrap(*t);
        else
            Py_INCREF(o);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// Every entry point: argument count, exceptions, and the GIL as torch holds it.
template <typename F>
PyObject* entry(Py_ssize_t given, Py_ssize_t wanted, F body) {
    if (given != wanted) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return body();
    } catch (const Raise& e) {
        if (e.type) PyErr_SetString(e.type, e.text.c_str());
    } catch (const std::bad_alloc&) {
        PyErr_NoMemory();
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// ---- norm and activation ------------------------------------------------------------------

// The output of rms_norm and gated_act and its scales.
struct Rounded {
    Tensor y, scale;
    int64_t ldy, ld_sy = 1;

    Rounded(PyObject* out, PyObject* scale_out, const Tensor& x, int code) {
        const int64_t M = x.size(0), N = x.size(1);
        if (code == GR_OUT_16) {
            if (scale_out != Py_None) bad_value("a 16-bit output has no scales");
            Output o(out, x, M, N, x.scalar_type(), "out");
            y = o.t;
            ldy = o.ld;
            return;
        }
        if (N % 32) bad_value("the columns must be a multiple of 32 for an MX output");
        Output o(out, x, M, code == GR_OUT_MXFP8 ? N : N / 2, code == GR_OUT_MXFP8 ? at::kFloat8_e4m3fn : at::kByte,
                 "out");
        Output s(scale_out, x, M, N / 32, at::kByte, "scale_out");
        y = o.t;
        ldy = o.ld;
        scale = s.t;
        ld_sy = s.ld;
    }
    uint8_t* scales() const { return scale.defined() ? data_of<uint8_t>(scale) : nullptr; }
};

// x, weight, residual, eps, out code, out, scale_out, sum_out, stream
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 9, [&]() -> PyObject* {
        const Matrix x(a[0], "x");
        const auto kind = x.t.scalar_type();
        const uint16_t* w = vector_of<uint16_t>(a[1], x.t, x.cols, kind, "weight");
        const Tensor* r = maybe_tensor(a[2], "residual");
        const double eps = PyFloat_AsDouble(a[3]);
        if (eps == -1.0 && PyErr_Occurred()) return nullptr;
        const int code = (int)int_of(a[4]);
        Tensor sum;
        int64_t ldr = 1, lds = 1;
        if (r) {
            ldr = matching(*r, x.t, x.rows, x.cols, kind, "residual");
            Output s(a[7], x.t, x.rows, x.cols, kind, "sum_out");
            sum = s.t;
            lds = s.ld;
        } else if (a[7] != Py_None) {
            bad_value("sum_out needs a residual");
        }
        const Rounded y(a[5], a[6], x.t, code);
        on_gpu(x.t, "x");
        const int st = rms_norm_mx(x.rows, x.cols, x.data, x.ld, r ? data_of<uint16_t>(*r) : nullptr, ldr, w,
                                   (float)eps, r ? data_of<uint16_t>(sum) : nullptr, lds, y.y.data_ptr(), y.ldy,
                                   y.scales(), y.ld_sy, x.fmt, code, stream_of(a[8]));
        return st == GR_OK ? tuple_of({&y.y, &y.scale, &sum}) : PyLong_FromLong(st);
    });
}

// gate, up, act, out code, out, scale_out, stream
PyObject* gated_act(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 7, [&]() -> PyObject* {
        const Matrix g(a[0], "gate");
        const Tensor* u = maybe_tensor(a[1], "up");
        const int64_t ldu = u ? matching(*u, g.t, g.rows, g.cols, g.t.scalar_type(), "up") : 1;
        const int act = (int)int_of(a[2]), code = (int)int_of(a[3]);
        const Rounded y(a[4], a[5], g.t, code);
        on_gpu(g.t, "gate");
        const int st = gated_act_mx(g.rows, g.cols, g.data, g.ld, u ? data_of<uint16_t>(*u) : nullptr, ldu, act,
                                    y.y.data_ptr(), y.ldy, y.scales(), y.ld_sy, g.fmt, code, stream_of(a[6]));
        return st == GR_OK ? tuple_of({&y.y, &y.scale}) : PyLong_FromLong(st);
    });
}

// ---- products -----------------------------------------------------------------------------

// An N x K MX fp4 matrix next to `like`.
struct Fp4 {
    int64_t rows, ld, ld_s;
    const uint8_t *data, *scale;

    Fp4(PyObject* wo, PyObject* so, const Tensor& like, int64_t K, const char* what) {
        const Tensor &w = tensor_of(wo, what), &s = tensor_of(so, "scale");
        if (w.scalar_type() != at::kByte || s.scalar_type() != at::kByte)
            bad_type(std::string(what) + " and its scales must be uint8 (E2M1 pairs, E8M0 codes)");
        if (K % 32) bad_value("K must be a multiple of 32");
        if (w.dim() != 2 || w.size(1) * 2 != K || s.dim() != 2 || s.size(0) != w.size(0) || s.size(1) != K / 32)
            bad_value(std::string(what) + " must be N x K/2 with N x K/32 scales for K = " + std::to_string(K));
        check_place(w, like, what);
        check_place(s, like, what);
        rows = w.size(0);
        ld = pitch_of(w, what);
        ld_s = pitch_of(s, what);
        data = data_of<const uint8_t>(w);
        scale = data_of<const uint8_t>(s);
    }
};

// x, weight, scale, bias, act, out, workspace, stream
PyObject* linear_mxfp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 8, [&]() -> PyObject* {
        const Matrix x(a[0], "x");
        const auto kind = x.t.scalar_type();
        const Fp4 w(a[1], a[2], x.t, x.cols, "weight");
        const uint16_t* bias = vector_of<uint16_t>(a[3], x.t, w.rows, kind, "bias");
        const int act = (int)int_of(a[4]);
        const Output c(a[5], x.t, x.rows, w.rows, kind, "out");
        on_gpu(x.t, "x");
        int64_t need = 0;
        int st = gemm_w4_bt_workspace_size(x.rows, w.rows, x.cols, &need);
        if (st != GR_OK) return PyLong_FromLong(st);
        const Scratch ws(a[6], x.t, need);
        st = gemm_w4_bt(x.rows, w.rows, x.cols, x.data, x.ld, w.data, w.ld, w.scale, w.ld_s, bias, act,
                        data_of<uint16_t>(c.t), c.ld, x.fmt, ws.data, ws.bytes, stream_of(a[7]));
        return st == GR_OK ? THPVariable_Wrap(c.t) : PyLong_FromLong(st);
    });
}

// a, scale_a, bt, scale_b, bias, act, output format, out, path (-1: the planner's), stream
PyObject* gemm_mxfp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 10, [&]() -> PyObject* {
        const Tensor& at_ = tensor_of(a[0], "a");
        if (at_.dim() != 2) bad_value("a must be 2-D");
        const int64_t K = at_.size(1) * 2;
        const Fp4 x(a[0], a[1], at_, K, "a"), w(a[2], a[3], at_, K, "bt");
        const int fmt = (int)int_of(a[6]);
        const auto kind = fmt == GR_FMT_BF16 ? at::kBFloat16 : at::kHalf;
        const uint16_t* bias = vector_of<uint16_t>(a[4], at_, w.rows, kind, "bias");
        const Output c(a[7], at_, x.rows, w.rows, kind, "out");
        const int act = (int)int_of(a[5]), path = (int)int_of(a[8]);
        on_gpu(at_, "a");
        uint16_t* const to = data_of<uint16_t>(c.t);
        const int st = path < 0 ? gemm_mxfp4_linear_bt(x.rows, w.rows, K, x.data, x.ld, x.scale, x.ld_s, w.data, w.ld, w.scale,
                                                w.ld_s, bias, act, to, c.ld, fmt, stream_of(a[9]))
                                : gemm_mxfp4_bt_forced(x.rows, w.rows, K, x.data, x.ld, x.scale, x.ld_s, w.data, w.ld,
                                                       w.scale, w.ld_s, bias, act, to, c.ld, fmt, stream_of(a[9]), path);
        return st == GR_OK ? THPVariable_Wrap(c.t) : PyLong_FromLong(st);
    });
}

// ---- mixture of experts -------------------------------------------------------------------

// x, router, topk, bias, renormalize, workspace, stream
PyObject* moe_route_(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 7, [&]() -> PyObject* {
        const Matrix x(a[0], "x");
        const Tensor& r = tensor_of(a[1], "router");
        if (r.dim() != 2) bad_value("router must be 2-D");
        const int64_t T = x.rows, H = x.cols, E = r.size(0), k = int_of(a[2]);
        const int64_t ldr = matching(r, x.t, E, H, x.t.scalar_type(), "router");
        const float* bias = vector_of<float>(a[3], x.t, E, at::kFloat, "bias");
        const int renorm = (int)int_of(a[4]);
        on_gpu(x.t, "x");
        int64_t need = 0;
        int st = moe_route_workspace_size(T, H, E, &need);
        if (st != GR_OK) return PyLong_FromLong(st);
        const Scratch ws(a[5], x.t, need);
        const int64_t cols = k > 0 && k <= E ? k : 0;
        const Tensor ids = empty_like(x.t, {T, cols}, at::kInt), weights = empty_like(x.t, {T, cols}, at::kFloat);
        st = moe_route(T, H, E, k, x.data, x.ld, data_of<uint16_t>(r), ldr, bias, renorm, data_of<int32_t>(ids),
                       data_of<float>(weights), x.fmt, ws.data, ws.bytes, stream_of(a[6]));
        return st == GR_OK ? tuple_of({&ids, &weights}) : PyLong_FromLong(st);
    });
}

// The address of a contiguous tensor of the experts, nullptr for None.
template <typename T>
const T* whole(PyObject* o, const Tensor& like, at::IntArrayRef shape, at::ScalarType kind, const char* what) {
    const Tensor* t = maybe_tensor(o, what);
    if (!t) return nullptr;
    check_kind(*t, shape, kind, what);
    check_place(*t, like, what);
    if (!t->is_contiguous()) bad_value(std::string(what) + " must be contiguous");
    return data_of<const T>(*t);
}

// x, ids, weights, w13, s13, w2, s2, b13, b2, act, out, workspace, stream
PyObject* moe_mxfp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 13, [&]() -> PyObject* {
        const Matrix x(a[0], "x");
        const auto kind = x.t.scalar_type();
        const Tensor &ids = tensor_of(a[1], "ids"), &w13 = tensor_of(a[3], "w13");
        for (int i : {2, 4, 5, 6}) tensor_of(a[i], "an operand of the experts");
        if (ids.dim() != 2) bad_value("ids must be 2-D");
        if (w13.dim() != 3 || w13.size(1) % 2) bad_value("w13 must be E x 2I x H/2");
        const int64_t T = x.rows, H = x.cols, k = ids.size(1), E = w13.size(0), I = w13.size(1) / 2;
        if (H % 32 || I % 32) bad_value("H and I must be multiples of 32");
        const int32_t* id = whole<int32_t>(a[1], x.t, {T, k}, at::kInt, "ids");
        const float* weight = whole<float>(a[2], x.t, {T, k}, at::kFloat, "weights");
        const uint8_t* d13 = whole<uint8_t>(a[3], x.t, {E, 2 * I, H / 2}, at::kByte, "w13");
        const uint8_t* c13 = whole<uint8_t>(a[4], x.t, {E, 2 * I, H / 32}, at::kByte, "s13");
        const uint8_t* d2 = whole<uint8_t>(a[5], x.t, {E, H, I / 2}, at::kByte, "w2");
        const uint8_t* c2 = whole<uint8_t>(a[6], x.t, {E, H, I / 32}, at::kByte, "s2");
        const uint16_t* b13 = whole<uint16_t>(a[7], x.t, {E, 2 * I}, kind, "b13");
        const uint16_t* b2 = whole<uint16_t>(a[8], x.t, {E, H}, kind, "b2");
        const int act = (int)int_of(a[9]);
        const Output c(a[10], x.t, T, H, kind, "out");
        on_gpu(x.t, "x");
        int64_t need = 0;
        int st = moe_w4_workspace_size(T, H, I, E, k, &need);
        if (st != GR_OK) return PyLong_FromLong(st);
        const Scratch ws(a[11], x.t, need);
        if (!ws.data && need > 0) return PyLong_FromLong(GR_ERR_SCRATCH);
        st = moe_w4(T, H, I, E, k, x.data, x.ld, id, weight, d13, c13, b13, d2, c2, b2, act, data_of<uint16_t>(c.t),
                    c.ld, x.fmt, ws.data, ws.bytes, stream_of(a[12]));
        return st == GR_OK ? THPVariable_Wrap(c.t) : PyLong_FromLong(st);
    });
}

// ---- training -----------------------------------------------------------------------------

double double_of(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raise{nullptr, ""};
    return v;
}

// A matrix next to `like`, of its type; nothing for None.
struct Maybe {
    int64_t ld = 1;
    uint16_t* data = nullptr;

    Maybe(PyObject* o, const Tensor& like, int64_t rows, int64_t cols, const char* what) {
        const Tensor* t = maybe_tensor(o, what);
        if (!t) {
            ld = cols > 0 ? cols : 1;
            return;
        }
        ld = matching(*t, like, rows, cols, like.scalar_type(), what);
        data = data_of<uint16_t>(*t);
    }
};

// An output that may not be wanted: new or given if `wanted`, else None must be given.
struct Wanted {
    Tensor t;
    int64_t ld = 1;
    uint16_t* data = nullptr;

    Wanted(PyObject* o, bool wanted, const Tensor& like, int64_t rows, int64_t cols, const char* what) {
        if (!wanted) {
            if (o != Py_None) bad_value(std::string(what) + " is given for what is not asked for");
            ld = cols > 0 ? cols : 1;
            return;
        }
        Output out(o, like, rows, cols, like.scalar_type(), what);
        t = out.t;
        ld = out.ld;
        data = data_of<uint16_t>(t);
    }
};

// A new vector of n values like `like`, if wanted.
Tensor vector_like(bool wanted, const Tensor& like, int64_t n) {
    return wanted ? empty_like(like, {n}, like.scalar_type()) : Tensor();
}
uint16_t* data_or_null(const Tensor& t) { return t.defined() ? data_of<uint16_t>(t) : nullptr; }

PyObject* failed(int st) { return PyLong_FromLong(st); }

// x, w13, b13, act, keep, out, gu_out, workspace, stream
PyObject* gated_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 9, [&]() -> PyObject* {
        const Matrix x(a[0], "x"), w(a[1], "w13");
        if (w.fmt != x.fmt) bad_type("w13 must have x's type");
        if (w.rows % 2 || w.cols != x.cols) bad_value("w13 must be 2I x " + std::to_string(x.cols) + ", got " + shape_text(w.t.sizes()));
        check_place(w.t, x.t, "w13");
        const int64_t I = w.rows / 2;
        const uint16_t* bias = vector_of<uint16_t>(a[2], x.t, 2 * I, x.t.scalar_type(), "b13");
        const int act = (int)int_of(a[3]);
        const bool keep = int_of(a[4]) != 0;
        const Wanted c(a[5], true, x.t, x.rows, I, "out"), gu(a[6], keep, x.t, x.rows, 2 * I, "gu_out");
        on_gpu(x.t, "x");
        int64_t need = 0;
        int st = gated_linear_workspace_size(x.rows, I, x.cols, &need);
        if (st != GR_OK) return failed(st);
        const Scratch ws(a[7], x.t, need);
        st = gated_linear_bt(x.rows, I, x.cols, x.data, x.ld, w.data, w.ld, bias, act, c.data, c.ld, gu.data, gu.ld, x.fmt,
                             ws.data, ws.bytes, stream_of(a[8]));
        return st == GR_OK ? tuple_of({&c.t, &gu.t}) : failed(st);
    });
}

// dy, x, weight, bias, input gradient, weight gradient, dx_out, dw_out, workspace, stream
PyObject* linear_backward_(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 10, [&]() -> PyObject* {
        const Matrix dy(a[0], "dy"), w(a[2], "weight");
        if (w.fmt != dy.fmt) bad_type("weight must have dy's type");
        if (w.rows != dy.cols) bad_value("weight must be " + std::to_string(dy.cols) + " x K, got " + shape_text(w.t.sizes()));
        check_place(w.t, dy.t, "weight");
        const int64_t M = dy.rows, N = dy.cols, K = w.cols;
        const bool bias = int_of(a[3]) != 0, want_x = int_of(a[4]) != 0, want_w = int_of(a[5]) != 0;
        if (want_w && a[1] == Py_None) bad_value("the weight's gradient needs x");
        const Maybe x(a[1], dy.t, M, K, "x");
        const Wanted dx(a[6], want_x, dy.t, M, K, "dx_out"), dw(a[7], want_w, dy.t, N, K, "dw_out");
        on_gpu(dy.t, "dy");
        const Tensor db = vector_like(bias, dy.t, N);
        int64_t need = 0;
        int st = linear_backward_workspace_size(M, N, K, dy.data, dy.ld, x.data, x.ld, w.data, w.ld, dx.data, dx.ld, dw.data,
                                                dw.ld, data_or_null(db), &need);
        if (st != GR_OK) return failed(st);
        const Scratch ws(a[8], dy.t, need);
        st = linear_backward(M, N, K, dy.data, dy.ld, x.data, x.ld, w.data, w.ld, dx.data, dx.ld, dw.data, dw.ld,
                             data_or_null(db), dy.fmt, ws.data, ws.bytes, stream_of(a[9]));
        return st == GR_OK ? tuple_of({&dx.t, &dw.t, &db}) : failed(st);
    });
}

// dh, x, w13, gu, act, bias, input gradient, weight gradient, dx_out, dw_out, workspace, stream
PyObject* gated_linear_backward_(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 12, [&]() -> PyObject* {
        const Matrix dh(a[0], "dh"), w(a[2], "w13");
        const int64_t M = dh.rows, I = dh.cols, H = w.cols;
        if (w.fmt != dh.fmt) bad_type("w13 must have dh's type");
        if (w.rows != 2 * I) bad_value("w13 must be " + std::to_string(2 * I) + " x H, got " + shape_text(w.t.sizes()));
        check_place(w.t, dh.t, "w13");
        const Matrix gu(a[3], "gu");
        const int64_t ldgu = matching(gu.t, dh.t, M, 2 * I, dh.t.scalar_type(), "gu");
        const int act = (int)int_of(a[4]);
        const bool bias = int_of(a[5]) != 0, want_x = int_of(a[6]) != 0, want_w = int_of(a[7]) != 0;
        if (want_w && a[1] == Py_None) bad_value("the weight's gradient needs x");
        const Maybe x(a[1], dh.t, M, H, "x");
        const Wanted dx(a[8], want_x, dh.t, M, H, "dx_out"), dw(a[9], want_w, dh.t, 2 * I, H, "dw_out");
        on_gpu(dh.t, "dh");
        const Tensor db = vector_like(bias, dh.t, 2 * I);
        int64_t need = 0;
        int st = gated_linear_backward_workspace_size(M, I, H, w.data, w.ld, dx.data, dx.ld, dw.data, data_or_null(db), &need);
        if (st != GR_OK) return failed(st);
        const Scratch ws(a[10], dh.t, need);
        st = gated_linear_backward(M, I, H, dh.data, dh.ld, x.data, x.ld, w.data, w.ld, gu.data, ldgu, act, dx.data, dx.ld,
                                   dw.data, dw.ld, data_or_null(db), dh.fmt, ws.data, ws.bytes, stream_of(a[11]));
        return st == GR_OK ? tuple_of({&dx.t, &dw.t, &db}) : failed(st);
    });
}

// The gates of a sandwich norm: N values, or G x N with G a divisor of the rows.
struct Gates {
    int64_t count = 0, ld = 1;
    const uint16_t* data = nullptr;
    bool flat = false;

    Gates(PyObject* o, const Tensor& like) {
        const Tensor* t = maybe_tensor(o, "gate");
        const int64_t M = like.size(0), N = like.size(1);
        ld = N > 0 ? N : 1;
        if (!t) return;
        flat = t->dim() == 1;
        if (flat) {
            data = vector_of<uint16_t>(o, like, N, like.scalar_type(), "gate");
            count = 1;
            return;
        }
        if (t->dim() != 2) bad_value("gate must be N values or G x N");
        count = t->size(0);
        ld = matching(*t, like, count, N, like.scalar_type(), "gate");
        if (count < 1 || M % count) bad_value("the rows must be a multiple of the gates: " + std::to_string(M) + " rows, " + std::to_string(count) + " gates");
        data = data_of<const uint16_t>(*t);
    }
};

// y, residual, weight, next_weight, gate, scale, eps, next norm, total_out, normed_out, stream
PyObject* sandwich_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 11, [&]() -> PyObject* {
        const Matrix y(a[0], "y");
        const auto kind = y.t.scalar_type();
        const int64_t M = y.rows, N = y.cols;
        const Tensor& res = tensor_of(a[1], "residual");
        const int64_t ldr = matching(res, y.t, M, N, kind, "residual");
        const uint16_t *w = vector_of<uint16_t>(a[2], y.t, N, kind, "weight"),
                       *next = vector_of<uint16_t>(a[3], y.t, N, kind, "next_weight");
        const Gates gate(a[4], y.t);
        const double scale = double_of(a[5]), eps = double_of(a[6]);
        const bool norm = int_of(a[7]) != 0;
        if (!norm && next) bad_value("next_weight is given for a norm that is not asked for");
        const Wanted total(a[8], true, y.t, M, N, "total_out"), normed(a[9], norm, y.t, M, N, "normed_out");
        on_gpu(y.t, "y");
        const int st = sandwich_norm_fwd(M, N, y.data, y.ld, data_of<uint16_t>(res), ldr, w, next, gate.data, gate.count, gate.ld,
                                         (float)scale, (float)eps, total.data, total.ld, normed.data, normed.ld, y.fmt,
                                         stream_of(a[10]));
        return st == GR_OK ? tuple_of({&total.t, &normed.t}) : failed(st);
    });
}

// y, dtotal, dnormed, total, weight, next_weight, gate, scale, eps, workspace, stream
PyObject* sandwich_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 11, [&]() -> PyObject* {
        const Matrix y(a[0], "y");
        const auto kind = y.t.scalar_type();
        const int64_t M = y.rows, N = y.cols;
        const Maybe dt(a[1], y.t, M, N, "dtotal"), dn(a[2], y.t, M, N, "dnormed");
        if (a[1] == Py_None && a[2] == Py_None) bad_value("dtotal or dnormed is needed");
        const Matrix total(a[3], "total");
        const int64_t ldt = matching(total.t, y.t, M, N, kind, "total");
        const uint16_t *w = vector_of<uint16_t>(a[4], y.t, N, kind, "weight"),
                       *next = vector_of<uint16_t>(a[5], y.t, N, kind, "next_weight");
        const Gates gate(a[6], y.t);
        const double scale = double_of(a[7]), eps = double_of(a[8]);
        on_gpu(y.t, "y");
        const Wanted dy(Py_None, true, y.t, M, N, "dy"), dr(Py_None, true, y.t, M, N, "dresidual");
        const Tensor dw = vector_like(a[4] != Py_None, y.t, N), dnext = vector_like(a[5] != Py_None && a[2] != Py_None, y.t, N);
        Tensor dgate;
        if (gate.flat) dgate = empty_like(y.t, {N}, kind);
        else if (gate.count > 0) dgate = empty_like(y.t, {gate.count, N}, kind);
        int64_t need = 0;
        int st = GR_OK;
        if (dw.defined() || dnext.defined() || dgate.defined()) {
            st = sandwich_norm_bwd_workspace_size(M, N, gate.count, &need);
            if (st != GR_OK) return failed(st);
        }
        const Scratch ws(a[9], y.t, need);
        st = sandwich_norm_bwd(M, N, dt.data, dt.ld, dn.data, dn.ld, y.data, y.ld, total.data, ldt, w, next, gate.data, gate.count,
                               gate.ld, (float)scale, (float)eps, dy.data, dy.ld, dr.data, dr.ld, data_or_null(dw),
                               data_or_null(dnext), data_or_null(dgate), N > 0 ? N : 1, y.fmt, ws.data, ws.bytes,
                               stream_of(a[10]));
        return st == GR_OK ? tuple_of({&dy.t, &dr.t, &dw, &dnext, &dgate}) : failed(st);
    });
}

// A batch of matrices (or one) with unit column stride: B x rows x cols.
struct Batch {
    int64_t count = 1, rows, cols, ld, stride;

    Batch(const Tensor& t, const char* what) {
        if (t.dim() != 2 && t.dim() != 3) bad_value(std::string(what) + " must be a matrix or a batch of matrices");
        const int d = (int)t.dim();
        rows = t.size(d - 2);
        cols = t.size(d - 1);
        if (cols > 1 && rows > 0 && t.stride(d - 1) != 1) bad_value(std::string(what) + " needs unit column stride");
        ld = cols > 0 ? cols : 1;
        if (rows > 1 && cols > 0) ld = t.stride(d - 2);
        const int64_t span = rows > 0 ? (rows - 1) * ld + cols : 0;
        stride = span;
        if (d == 3) {
            count = t.size(0);
            if (count > 1 && span > 0) stride = t.stride(0);
        }
        if (span > 0 && (ld < cols || stride < span)) bad_value(std::string(what) + " has rows or matrices that share memory");
    }
};

// update, steps, a, b, c, scale, eps, out, workspace, stream
PyObject* orthogonalize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 10, [&]() -> PyObject* {
        const Tensor& g = tensor_of(a[0], "update");
        const int fmt = g.scalar_type() == at::kFloat ? GR_FMT_F32 : format_of(g.scalar_type());
        if (fmt < 0) bad_type(std::string("update must be float16, bfloat16 or float32, got ") + c10::toString(g.scalar_type()));
        const Batch in(g, "update");
        const int64_t steps = int_of(a[1]);
        const float k[3] = {(float)double_of(a[2]), (float)double_of(a[3]), (float)double_of(a[4])};
        const double scale = double_of(a[5]), eps = double_of(a[6]);
        Tensor out;
        if (const Tensor* given = maybe_tensor(a[7], "out")) {
            check_kind(*given, g.sizes(), at::kBFloat16, "out");
            check_place(*given, g, "out");
            out = *given;
        } else {
            out = empty_like(g, g.sizes(), at::kBFloat16);
        }
        const Batch to(out, "out");
        on_gpu(g, "update");
        int64_t need = 0;
        int st = orthogonalize_workspace_size(in.count, in.rows, in.cols, &need);
        if (st != GR_OK) return failed(st);
        const Scratch ws(a[8], g, need);
        st = orthogonalize_update(in.count, in.rows, in.cols, g.data_ptr(), in.ld, in.stride, fmt, k,
                                  steps > 0 && steps < 1000 ? (int)steps : 0, (float)scale, (float)eps, data_of<uint16_t>(out),
                                  to.ld, to.stride, ws.data, ws.bytes, stream_of(a[9]));
        return st == GR_OK ? THPVariable_Wrap(out) : failed(st);
    });
}

#define CALL(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fn)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {CALL("rms_norm", rms_norm),         CALL("gated_act", gated_act),
                          CALL("linear_mxfp4", linear_mxfp4), CALL("gemm_mxfp4", gemm_mxfp4),
                          CALL("moe_route", moe_route_),      CALL("moe_mxfp4", moe_mxfp4),
                          CALL("gated_linear", gated_linear), CALL("linear_backward", linear_backward_),
                          CALL("gated_linear_backward", gated_linear_backward_),
                          CALL("sandwich_norm", sandwich_norm),
                          CALL("sandwich_norm_backward", sandwich_norm_backward),
                          CALL("orthogonalize", orthogonalize),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&kModule); }
