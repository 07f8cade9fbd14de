// The host side of the operators around the linears, for calls on the current
// stream: the same checks and allocations as the Python binding's, at less than half
// the cost.  One token's norm takes 2 us on the GPU and a call of it 15.5 us through
// Python (four outputs' allocation, a check per tensor, ctypes); 6 to 7 through here.
//
// Each function takes its Python counterpart's arguments in order (None where
// left out) and returns its result, or the C entry point's status as an int, or
// None where anything is not as the plain case has it: the binding then goes
// its own way, which raises the error or does the unusual.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/fp8blk.h"

namespace {

decltype(&fp8_add_rmsnorm_quantize_1x128) g_add_norm;
decltype(&fp8_rmsnorm_backward) g_norm_bwd;
decltype(&fp8_rmsnorm_backward_workspace_bytes) g_norm_bwd_bytes;
decltype(&fp8_token_logprobs) g_logprobs;
decltype(&fp8_token_logprobs_backward) g_logprobs_bwd;

using at::ScalarType;
using at::Tensor;
using Shape = c10::IntArrayRef;

constexpr int kRowwise = FP8_ROWWISE, kColwise = FP8_COLWISE;

// Arguments of one call.  `plain` turns false at the first that is not.
struct Call {
    PyObject* const* args;
    int dev = -1;
    bool plain = true;

    const Tensor* tensor(int i) {                          // or null for None
        PyObject* o = args[i];
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) {
            plain = false;
            return nullptr;
        }
        return &THPVariable_Unpack(o);
    }
    // the tensor whose device the call runs on
    const Tensor* first(int i) {
        const Tensor* t = tensor(i);
        if (!t || !t->is_cuda() || t->dim() != 2 || t->get_device() != c10::cuda::current_device()) {
            plain = false;
            return nullptr;
        }
        dev = static_cast<int>(t->get_device());
        return t;
    }
    bool fits(const Tensor& t, ScalarType type, Shape shape) const {
        return t.is_cuda() && t.get_device() == dev && t.scalar_type() == type && t.sizes() == shape && t.is_contiguous() &&
               (reinterpret_cast<uintptr_t>(t.data_ptr()) & 15u) == 0;     // (a slice that is not: the binding copies it)
    }
    // the data of a tensor that must be there, or may be None
    void* in(int i, ScalarType type, Shape shape, bool optional = false) {
        const Tensor* t = tensor(i);
        if (!t) {
            plain = plain && optional;
            return nullptr;
        }
        if (!fits(*t, type, shape)) plain = false;
        return t->data_ptr();
    }
    double number(int i) {
        const double v = PyFloat_AsDouble(args[i]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            plain = false;
        }
        return v;
    }
    long integer(int i) {
        const long v = PyLong_Check(args[i]) ? PyLong_AsLong(args[i]) : (plain = false, 0);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            plain = false;
        }
        return v;
    }
    void* stream() const { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }
};

// An output: the tensor given, or a new one.
struct Out {
    Tensor made;
    PyObject* given = nullptr;
    void* data = nullptr;

    // checks first, so that nothing is allocated in vain
    void check(Call& c, int i, ScalarType type, Shape shape) {
        if (c.args[i] == Py_None) return;
        given = c.args[i];
        data = c.in(i, type, shape);
    }
    void make(const Call& c, ScalarType type, Shape shape) {
        if (given) return;
        made = at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(c.dev)), std::nullopt);
        data = made.data_ptr();
    }
    PyObject* object() {                                   // a new reference; None for an output that was not asked for
        if (!given && !made.defined()) Py_RETURN_NONE;
        if (given) {
            Py_INCREF(given);
            return given;
        }
        return THPVariable_Wrap(std::move(made));
    }
};

template <int N>
PyObject* tuple_of(PyObject* (&items)[N]) {
    PyObject* t = PyTuple_New(N);
    for (int i = 0; i < N; ++i) {
        if (!t || !items[i]) {
            for (int j = i; j < N; ++j) Py_XDECREF(items[j]);
            Py_XDECREF(t);
            return nullptr;
        }
        PyTuple_SET_ITEM(t, i, items[i]);
    }
    return t;
}

bool count_is(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "takes %zd arguments, got %zd", want, n);
    return false;
}

// (x, gamma, residual, eps, mode, sum_out, rstd, q_row, s_row, q_colT, s_col)
PyObject* add_rmsnorm_quantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count_is(n, 11)) return nullptr;
    Call c{args};
    const Tensor* x = c.first(0);
    if (!x) Py_RETURN_NONE;
    const int64_t rows = x->size(0), cols = x->size(1);
    const Shape shape = x->sizes();
    if (!c.fits(*x, at::kBFloat16, shape)) Py_RETURN_NONE;
    void* gamma = c.in(1, at::kBFloat16, {cols});
    void* residual = c.in(2, at::kBFloat16, shape, true);
    const double eps = c.number(3);
    const long mode = c.integer(4);
    if (!c.plain || mode < 1 || mode > 3 || (!residual && args[2] == Py_None && args[5] != Py_None)) Py_RETURN_NONE;
    const bool add = args[2] != Py_None, row = mode & kRowwise, col = mode & kColwise;
    const int64_t s_row_shape[2] = {cols / 128, rows}, q_colT_shape[2] = {cols, rows}, s_col_shape[2] = {rows / 128, cols};
    Out sum, rstd, q_row, s_row, q_colT, s_col;
    if (add) sum.check(c, 5, at::kBFloat16, shape);
    rstd.check(c, 6, at::kFloat, {rows});
    if (row) {
        q_row.check(c, 7, at::kByte, shape);
        s_row.check(c, 8, at::kFloat, s_row_shape);
    }
    if (col) {
        q_colT.check(c, 9, at::kByte, q_colT_shape);
        s_col.check(c, 10, at::kFloat, s_col_shape);
    }
    if (!c.plain) Py_RETURN_NONE;
    if (add) sum.make(c, at::kBFloat16, shape);
    rstd.make(c, at::kFloat, {rows});
    if (row) {
        q_row.make(c, at::kByte, shape);
        s_row.make(c, at::kFloat, s_row_shape);
    }
    if (col) {
        q_colT.make(c, at::kByte, q_colT_shape);
        s_col.make(c, at::kFloat, s_col_shape);
    }
    const fp8_status st = g_add_norm(x->data_ptr(), residual, rows, cols, static_cast<float>(eps), gamma, static_cast<int>(mode),
                                     sum.data, static_cast<float*>(rstd.data), static_cast<uint8_t*>(q_row.data),
                                     static_cast<float*>(s_row.data), static_cast<uint8_t*>(q_colT.data),
                                     static_cast<float*>(s_col.data), c.stream());
    if (st != FP8_OK) return PyLong_FromLong(st);
    PyObject* s = add ? sum.object() : (Py_INCREF(args[0]), args[0]);
    PyObject* items[6] = {s, rstd.object(), q_row.object(), s_row.object(), q_colT.object(), s_col.object()};
    return tuple_of(items);
    END_HANDLE_TH_ERRORS
}

// (dy, s, rstd, gamma, dresidual, ds, dgamma, accumulate, workspace)
PyObject* rmsnorm_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count_is(n, 9)) return nullptr;
    Call c{args};
    const Tensor* s = c.first(1);
    if (!s) Py_RETURN_NONE;
    const int64_t rows = s->size(0), cols = s->size(1);
    const Shape shape = s->sizes();
    if (!c.fits(*s, at::kBFloat16, shape)) Py_RETURN_NONE;
    void* dy = c.in(0, at::kBFloat16, shape);
    void* rstd = c.in(2, at::kFloat, {rows});
    void* gamma = c.in(3, at::kBFloat16, {cols});
    void* dres = c.in(4, at::kBFloat16, shape, true);
    Out ds, dgamma;
    ds.check(c, 5, at::kBFloat16, shape);
    dgamma.check(c, 6, at::kFloat, {cols});
    const int accumulate = PyObject_IsTrue(args[7]);
    if (accumulate < 0) return nullptr;
    if (accumulate && !dgamma.given) c.plain = false;
    const Tensor* ws = c.tensor(8);
    if (ws && (!ws->is_cuda() || ws->get_device() != c.dev || !ws->is_contiguous())) c.plain = false;
    if (!c.plain) Py_RETURN_NONE;
    Tensor scratch;
    size_t bytes = 0;
    if (ws) {
        bytes = ws->nbytes();
    } else {
        const fp8_status st = g_norm_bwd_bytes(rows, cols, &bytes);
        if (st != FP8_OK) return PyLong_FromLong(st);
        scratch = at::detail::empty_cuda({static_cast<int64_t>(bytes)}, at::kByte, s->device(), std::nullopt);
        ws = &scratch;
    }
    ds.make(c, at::kBFloat16, shape);
    dgamma.make(c, at::kFloat, {cols});
    const fp8_status st = g_norm_bwd(dy, s->data_ptr(), static_cast<const float*>(rstd), gamma, dres, rows, cols, ds.data,
                                     static_cast<float*>(dgamma.data), accumulate, ws->data_ptr(), bytes, c.stream());
    if (st != FP8_OK) return PyLong_FromLong(st);
    PyObject* items[2] = {ds.object(), dgamma.object()};
    return tuple_of(items);
    END_HANDLE_TH_ERRORS
}

// A row-contiguous matrix of logits: its type's code and row stride.
bool logits_of(Call& c, const Tensor& t, int* code, int64_t* ld) {
    if (!t.is_cuda() || t.get_device() != c.dev || t.dim() != 2) return c.plain = false;
    const ScalarType type = t.scalar_type();
    *code = type == at::kBFloat16 ? FP8_BF16 : FP8_F32;
    const int64_t rows = t.size(0), vocab = t.size(1);
    *ld = rows <= 1 ? std::max(vocab, t.stride(0)) : t.stride(0);
    if ((type != at::kBFloat16 && type != at::kFloat) || (vocab > 1 && t.stride(1) != 1) || *ld < vocab) c.plain = false;
    return c.plain;
}

// (logits, targets, topk, logprob, entropy, stats, top_logprob, top_index)
PyObject* token_logprobs(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count_is(n, 8)) return nullptr;
    Call c{args};
    const Tensor* x = c.first(0);
    int code = 0;
    int64_t ld = 0;
    if (!x || !logits_of(c, *x, &code, &ld)) Py_RETURN_NONE;
    const int64_t rows = x->size(0), vocab = x->size(1);
    void* targets = c.in(1, at::kLong, {rows}, true);
    const bool with = args[1] != Py_None;
    const long topk = c.integer(2);
    if (!c.plain || topk < 0 || topk > FP8_MAX_TOPK) Py_RETURN_NONE;
    const int64_t two[2] = {rows, 2}, k[2] = {rows, topk};
    Out logprob, entropy, stats, top_lp, top_i;
    if (with) logprob.check(c, 3, at::kFloat, {rows});
    entropy.check(c, 4, at::kFloat, {rows});
    stats.check(c, 5, at::kFloat, two);
    if (topk) {
        top_lp.check(c, 6, at::kFloat, k);
        top_i.check(c, 7, at::kLong, k);
    }
    if (!c.plain) Py_RETURN_NONE;
    if (with) logprob.make(c, at::kFloat, {rows});
    entropy.make(c, at::kFloat, {rows});
    stats.make(c, at::kFloat, two);
    if (topk) {
        top_lp.make(c, at::kFloat, k);
        top_i.make(c, at::kLong, k);
    }
    const fp8_status st = g_logprobs(x->data_ptr(), code, rows, vocab, ld, static_cast<const int64_t*>(targets),
                                     static_cast<int>(topk), static_cast<float*>(logprob.data),
                                     static_cast<float*>(entropy.data), static_cast<float*>(stats.data),
                                     static_cast<float*>(top_lp.data), static_cast<int64_t*>(top_i.data), c.stream());
    if (st != FP8_OK) return PyLong_FromLong(st);
    PyObject* items[5] = {logprob.object(), entropy.object(), stats.object(), top_lp.object(), top_i.object()};
    return tuple_of(items);
    END_HANDLE_TH_ERRORS
}

// (logits, targets, stats, dlogprob, entropy, dentropy, dlogits)
PyObject* token_logprobs_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count_is(n, 7)) return nullptr;
    Call c{args};
    const Tensor* x = c.first(0);
    int code = 0, code_out = 0;
    int64_t ld = 0, ld_out = 0;
    if (!x || !logits_of(c, *x, &code, &ld)) Py_RETURN_NONE;
    const int64_t rows = x->size(0), vocab = x->size(1);
    void* targets = c.in(1, at::kLong, {rows}, true);
    void* stats = c.in(2, at::kFloat, {rows, 2});
    void* dlogprob = c.in(3, at::kFloat, {rows}, true);
    void* entropy = args[5] == Py_None ? nullptr : c.in(4, at::kFloat, {rows});
    void* dentropy = c.in(5, at::kFloat, {rows}, true);
    if (args[3] != Py_None && args[1] == Py_None) c.plain = false;
    Out out;
    if (const Tensor* d = c.tensor(6)) {
        if (d->scalar_type() != x->scalar_type() || d->sizes() != x->sizes() || !logits_of(c, *d, &code_out, &ld_out)) Py_RETURN_NONE;
        out.given = args[6];
        out.data = d->data_ptr();
    }
    if (!c.plain) Py_RETURN_NONE;
    if (!out.given) {
        out.make(c, x->scalar_type(), x->sizes());
        ld_out = vocab;
    }
    const fp8_status st = g_logprobs_bwd(x->data_ptr(), code, rows, vocab, ld, static_cast<const int64_t*>(targets),
                                         static_cast<const float*>(stats), static_cast<const float*>(dlogprob),
                                         static_cast<const float*>(entropy), static_cast<const float*>(dentropy), out.data,
                                         ld_out, c.stream());
    if (st != FP8_OK) return PyLong_FromLong(st);
    return out.object();
    END_HANDLE_TH_ERRORS
}

// The C entry points' addresses, in the order of the pointers above.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (!count_is(n, 5)) return nullptr;
    void* p[5];
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    g_add_norm = reinterpret_cast<decltype(g_add_norm)>(p[0]);
    g_norm_bwd = reinterpret_cast<decltype(g_norm_bwd)>(p[1]);
    g_norm_bwd_bytes = reinterpret_cast<decltype(g_norm_bwd_bytes)>(p[2]);
    g_logprobs = reinterpret_cast<decltype(g_logprobs)>(p[3]);
    g_logprobs_bwd = reinterpret_cast<decltype(g_logprobs_bwd)>(p[4]);
    Py_RETURN_NONE;
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind),           METHOD(add_rmsnorm_quantize),    METHOD(rmsnorm_backward),
                         METHOD(token_logprobs), METHOD(token_logprobs_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp8blk_host", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__fp8blk_host() { return PyModule_Create(&module); }
