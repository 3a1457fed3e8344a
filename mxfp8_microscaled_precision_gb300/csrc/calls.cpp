// calls.cpp -- the calls of libmxq that run in every decoding step (mxq.h, operators
// around the experts' products; MXFP4, and activations kept in 8 bits) as a CPython extension module: the checks of the
// tensors, the allocation of results and workspaces, the current stream and the call.
//
// For a single token the host's share is most of the time.  Through ctypes a call of 13 to 18
// arguments costs 2 to 3 us on the GB300's host, a tensor allocated from Python 1.7 to 2.6 us, five attributes
// of a tensor read from Python 0.25 us.  Through torch's C++ interface they cost a fraction of that.  Measured, a
// call with its results allocated, checks and allocations in Python before: layer norm 12.3 us to 6.5 us (2.7 us
// with results given), routing 9.5 us to 5.2 us, plan 9.6 us to 4.9 us, dispatch 7.9 us to 3.6 us; clipping 300
// gradients 155 us of host time to less than the kernels' 31 us.
//
// The library launches on the current device: a call's tensors all have to be there.
//
// Errors: ValueError for a tensor that a call cannot take, TypeError for an object that is none,
// the package's error class for a status of the library; a C++ exception (memory) becomes
// torch's own Python error.  Nothing leaves as an exception of C++.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>
#include <string>
#include <vector>

#include "mxq.h"

namespace {

struct Refused {   // ValueError
    std::string why;
};
struct PythonError {};   // set already

PyObject* raise_status = nullptr;   // (name, status): raises
PyObject* raw_stream = nullptr;     // the current stream of a device by its index, as an integer

// A new reference that is dropped at the end of its scope.
class Owned {
public:
    explicit Owned(PyObject* p) : p_(p) {
        if (p == nullptr) throw PythonError{};
    }
    Owned(const Owned&) = delete;
    Owned& operator=(const Owned&) = delete;
    ~Owned() { Py_XDECREF(p_); }
    PyObject* get() const { return p_; }
    PyObject* release() {
        PyObject* p = p_;
        p_ = nullptr;
        return p;
    }

private:
    PyObject* p_;
};

PyObject* wrapped(at::Tensor t) {
    PyObject* p = THPVariable_Wrap(std::move(t));
    if (p == nullptr) throw PythonError{};
    return p;
}

// ---- arguments ------------------------------------------------------------------------

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
        throw PythonError{};
    }
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}

// One out of the range of int32 must not come out valid: the library refuses INT32_MIN.
int32_t integer32(PyObject* o) {
    const int64_t v = integer(o);
    return v < INT32_MIN || v > INT32_MAX ? INT32_MIN : static_cast<int32_t>(v);
}

int32_t narrow(int64_t v) { return v < INT32_MIN || v > INT32_MAX ? INT32_MIN : static_cast<int32_t>(v); }

float number(PyObject* o) {
    const double d = PyFloat_AsDouble(o);
    if (d == -1.0 && PyErr_Occurred()) throw PythonError{};
    return static_cast<float>(d);
}

const char* name_of(at::ScalarType type) {
    switch (type) {
        case at::kBFloat16: return "bfloat16";
        case at::kFloat: return "float32";
        case at::kInt: return "int32";
        case at::kLong: return "int64";
        case at::kBool: return "bool";
        default: return "uint8";
    }
}

std::string shape_of(std::initializer_list<int64_t> shape) {
    std::string s = "[";
    for (int64_t n : shape) s += (s.size() > 1 ? ", " : "") + std::to_string(n);
    return s + "]";
}

// MXQ_BF16, MXQ_F32 or -1.
int code_of(const at::Tensor& t) {
    const at::ScalarType type = t.scalar_type();
    return type == at::kBFloat16 ? MXQ_BF16 : type == at::kFloat ? MXQ_F32 : -1;
}

// The device of the call's tensors, the first one's; -1 before it.
thread_local int call_device = -1;

// A call may run inside another one (a destructor that the interpreter runs meanwhile).
class OnDevice {
public:
    OnDevice() : outer_(call_device) { call_device = -1; }
    OnDevice(const OnDevice&) = delete;
    OnDevice& operator=(const OnDevice&) = delete;
    ~OnDevice() { call_device = outer_; }

private:
    int outer_;
};

// Every tensor passes here, a CUDA tensor as its type has been checked.
void same_device(const at::Tensor& t, const char* name) {
    const int device = t.get_device();
    if (call_device < 0) call_device = device;
    if (device != call_device)
        throw Refused{std::string(name) + " is on cuda:" + std::to_string(device) + ", another tensor of the call on cuda:" +
                      std::to_string(call_device)};
}

// A 2-D bf16 or fp32 CUDA tensor with unit last stride.  A single row has any stride (its own says nothing).
struct Matrix {
    void* data;
    mxq_dtype type;
    int64_t rows, cols, ld;
};
Matrix matrix(const at::Tensor& t, const char* name) {
    const int code = code_of(t);
    if (code < 0 || t.dim() != 2 || !t.is_cuda())
        throw Refused{std::string(name) + " must be a 2-D bfloat16 or float32 CUDA tensor"};
    same_device(t, name);
    const int64_t rows = t.size(0), cols = t.size(1), ld = t.stride(0);
    if (t.stride(1) != 1 && cols > 1) throw Refused{std::string(name) + " must have unit stride along its last axis"};
    return {t.data_ptr(), static_cast<mxq_dtype>(code), rows, cols, rows > 1 || ld > cols ? ld : cols};
}

// The address of a contiguous CUDA tensor of this type and shape.
void* dense(const at::Tensor& t, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
    if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape) || !t.is_cuda() || !t.is_contiguous())
        throw Refused{std::string(name) + " must be a contiguous " + name_of(type) + " CUDA tensor " + shape_of(shape)};
    same_device(t, name);
    return t.data_ptr();
}
void* dense(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
    return dense(tensor(o, name), name, type, shape);
}
void* dense_or_none(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
    return o == Py_None ? nullptr : dense(o, name, type, shape);
}

// An int32 matrix of slots.
struct Slots {
    int32_t* data;
    int64_t tokens, k;
};
Slots slots(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 2) throw Refused{std::string(name) + " must be 2-D"};
    return {static_cast<int32_t*>(dense(t, name, at::kInt, {t.size(0), t.size(1)})), t.size(0), t.size(1)};
}

// The current stream, of the current device, on which all tensors of the call have to be: t is one of them.
mxq_stream_t stream_of(const at::Tensor& t) {
    const int current = c10::impl::VirtualGuardImpl(at::kCUDA).getDevice().index();
    if (t.get_device() != current)
        throw Refused{"the tensors are on cuda:" + std::to_string(t.get_device()) + ", the current device is cuda:" +
                      std::to_string(current)};
    const Owned index(PyLong_FromLong(current));
    const Owned stream(PyObject_CallOneArg(raw_stream, index.get()));
    return reinterpret_cast<mxq_stream_t>(static_cast<intptr_t>(integer(stream.get())));
}

void check(mxq_status status, const char* name) {
    if (status == MXQ_OK) return;
    const Owned done(PyObject_CallFunction(raise_status, "si", name, static_cast<int>(status)));
    throw Refused{std::string(name) + " failed"};   // not reached: the call raises
}

// ---- results ----------------------------------------------------------------------------

at::Tensor fresh(const at::Tensor& like, at::IntArrayRef shape, at::ScalarType type) {
    return at::empty(shape, like.options().dtype(type));
}

// The results of a call, dropped unless it succeeds.
class Results {
public:
    Results() = default;
    Results(const Results&) = delete;
    Results& operator=(const Results&) = delete;
    ~Results() {
        for (PyObject* p : all_) Py_DECREF(p);
    }
    void* add(at::Tensor t) {
        void* data = t.data_ptr();
        all_.push_back(wrapped(std::move(t)));
        return data;
    }
    void add(PyObject* o) { all_.push_back(Py_NewRef(o)); }
    // given: checked against what the call writes, or None for a new tensor; *ld: its row stride.
    void* matrix(PyObject* given, const char* name, const at::Tensor& like, mxq_dtype type, int64_t rows, int64_t cols,
                 int64_t* ld) {
        *ld = cols;
        if (given == Py_None) return add(fresh(like, {rows, cols}, like.scalar_type()));
        const Matrix m = ::matrix(tensor(given, name), name);
        if (m.type != type || m.rows != rows || m.cols != cols)
            throw Refused{std::string(name) + " must be " + name_of(like.scalar_type()) + " " + shape_of({rows, cols})};
        *ld = m.ld;
        add(given);
        return m.data;
    }
    void* dense(PyObject* given, const char* name, const at::Tensor& like, at::ScalarType type,
                std::initializer_list<int64_t> shape) {
        if (given == Py_None) return add(fresh(like, shape, type));
        void* data = ::dense(given, name, type, shape);
        add(given);
        return data;
    }
    PyObject* one() {
        PyObject* p = all_.back();
        all_.pop_back();
        return p;
    }
    PyObject* tuple() {
        Owned t(PyTuple_New(static_cast<Py_ssize_t>(all_.size())));
        for (size_t i = 0; i < all_.size(); ++i) PyTuple_SET_ITEM(t.get(), static_cast<Py_ssize_t>(i), all_[i]);
        all_.clear();
        return t.release();
    }

private:
    std::vector<PyObject*> all_;
};

// The n objects of `out`, or n times None.
class Given {
public:
    Given(PyObject* out, Py_ssize_t n) {
        if (out == Py_None) return;
        fast_ = PySequence_Fast(out, "out must be a sequence of tensors");
        if (fast_ == nullptr) throw PythonError{};
        if (PySequence_Fast_GET_SIZE(fast_) != n) {
            Py_DECREF(fast_);
            throw Refused{"out must hold " + std::to_string(n) + " tensors"};
        }
    }
    Given(const Given&) = delete;
    Given& operator=(const Given&) = delete;
    ~Given() { Py_XDECREF(fast_); }
    PyObject* operator[](Py_ssize_t i) const { return fast_ == nullptr ? Py_None : PySequence_Fast_GET_ITEM(fast_, i); }

private:
    PyObject* fast_ = nullptr;
};

// ---- the calls ----------------------------------------------------------------------------
//
// Arguments as the functions of mxq.py list them; enums and truth values arrive as integers.

using Args = PyObject* const*;

// (logits, topk, score, bias, n_group, topk_group, group_score, renorm, scale, token_mask, out)
PyObject* route(Args a) {
    const at::Tensor& logits = tensor(a[0], "logits");
    const Matrix x = matrix(logits, "logits");
    const int64_t topk = integer(a[1]);
    const void* bias = dense_or_none(a[3], "bias", at::kFloat, {x.cols});
    const void* mask = nullptr;
    if (a[9] != Py_None) {
        const at::Tensor& m = tensor(a[9], "token_mask");
        mask = dense(m, "token_mask", m.scalar_type() == at::kBool ? at::kBool : at::kByte, {x.rows});
    }
    // before anything of that size is allocated
    if (topk < 1) throw Refused{"topk must be at least 1"};
    if (topk > MXQ_MAX_TOPK) check(topk > x.cols ? MXQ_ERR_INVALID_ARG : MXQ_ERR_UNSUPPORTED_SHAPE, "mxq_route");
    const Given out(a[10], 2);
    Results got;
    void* ids = got.dense(out[0], "ids", logits, at::kInt, {x.rows, topk});
    void* weights = got.dense(out[1], "weights", logits, at::kFloat, {x.rows, topk});
    check(mxq_route(x.data, x.type, x.rows, narrow(x.cols), x.ld, static_cast<const float*>(bias),
                    static_cast<const uint8_t*>(mask), static_cast<mxq_route_score>(integer32(a[2])), integer32(a[4]),
                    integer32(a[5]), static_cast<mxq_group_score>(integer32(a[6])),
                    narrow(topk), integer32(a[7]), number(a[8]), static_cast<int32_t*>(ids),
                    static_cast<float*>(weights), stream_of(logits)),
          "mxq_route");
    return got.tuple();
}

// (dweights, logits, ids, score, renorm, scale, out)
PyObject* route_backward(Args a) {
    const at::Tensor& logits = tensor(a[1], "logits");
    const Matrix x = matrix(logits, "logits");
    const Slots ids = slots(a[2], "ids");
    if (ids.tokens != x.rows) throw Refused{"ids and logits must have the same number of tokens"};
    const void* dweights = dense(a[0], "dweights", at::kFloat, {ids.tokens, ids.k});
    Results got;
    int64_t ld;
    void* out = got.matrix(a[6], "out", logits, x.type, x.rows, x.cols, &ld);
    check(mxq_route_backward(static_cast<const float*>(dweights), ids.data, x.data, x.type, x.rows, narrow(x.cols), x.ld,
                             static_cast<mxq_route_score>(integer32(a[3])), narrow(ids.k), integer32(a[4]), number(a[5]), out,
                             ld, stream_of(logits)),
          "mxq_route_backward");
    return got.one();
}

// (ids, experts, out)
PyObject* moe_plan(Args a) {
    const at::Tensor& like = tensor(a[0], "ids");
    const Slots ids = slots(a[0], "ids");
    const int64_t experts = integer(a[1]);
    if (experts < 1) check(MXQ_ERR_INVALID_ARG, "mxq_moe_plan");
    if (experts > MXQ_MAX_EXPERTS) check(MXQ_ERR_UNSUPPORTED_SHAPE, "mxq_moe_plan");   // before it is allocated
    const Given out(a[2], 2);
    Results got;
    void* offsets = got.dense(out[0], "offsets", like, at::kLong, {experts + 1});
    void* rows = got.dense(out[1], "rows", like, at::kInt, {ids.tokens, ids.k});
    check(mxq_moe_plan(ids.data, ids.tokens, narrow(ids.k), narrow(experts), static_cast<int64_t*>(offsets),
                       static_cast<int32_t*>(rows), stream_of(like)),
          "mxq_moe_plan");
    return got.tuple();
}

// (x, rows, out)
PyObject* moe_dispatch(Args a) {
    const at::Tensor& like = tensor(a[0], "x");
    const Matrix x = matrix(like, "x");
    const Slots rows = slots(a[1], "rows");
    if (rows.tokens != x.rows) throw Refused{"x and rows must have the same number of tokens"};
    Results got;
    int64_t ld;
    void* out = got.matrix(a[2], "out", like, x.type, rows.tokens * rows.k, x.cols, &ld);
    check(mxq_moe_dispatch(x.data, x.type, rows.tokens, narrow(rows.k), x.cols, x.ld, rows.data, out, ld, stream_of(like)),
          "mxq_moe_dispatch");
    return got.one();
}

// (y, rows, weights, out)
PyObject* moe_combine(Args a) {
    const at::Tensor& like = tensor(a[0], "y");
    const Matrix y = matrix(like, "y");
    const Slots rows = slots(a[1], "rows");
    if (y.rows != rows.tokens * rows.k) throw Refused{"y must have a row for every slot"};
    const void* weights = dense_or_none(a[2], "weights", at::kFloat, {rows.tokens, rows.k});
    Results got;
    int64_t ld;
    void* out = got.matrix(a[3], "out", like, y.type, rows.tokens, y.cols, &ld);
    check(mxq_moe_combine(y.data, y.type, rows.tokens, narrow(rows.k), y.cols, y.ld, rows.data,
                          static_cast<const float*>(weights), out, ld, stream_of(like)),
          "mxq_moe_combine");
    return got.one();
}

// (dout, y, rows, weights, out)
PyObject* moe_combine_backward(Args a) {
    const at::Tensor& like = tensor(a[1], "y");
    const Matrix y = matrix(like, "y");
    const Slots rows = slots(a[2], "rows");
    if (y.rows != rows.tokens * rows.k) throw Refused{"y must have a row for every slot"};
    const Matrix d = matrix(tensor(a[0], "dout"), "dout");
    if (d.type != y.type || d.rows != rows.tokens || d.cols != y.cols)
        throw Refused{std::string("dout must be ") + name_of(like.scalar_type()) + " " + shape_of({rows.tokens, y.cols})};
    const void* weights = dense(a[3], "weights", at::kFloat, {rows.tokens, rows.k});
    const Given out(a[4], 2);
    Results got;
    int64_t ld;
    void* dy = got.matrix(out[0], "dy", like, y.type, y.rows, y.cols, &ld);
    void* dweights = got.dense(out[1], "dweights", like, at::kFloat, {rows.tokens, rows.k});
    check(mxq_moe_combine_backward(d.data, y.data, y.type, rows.tokens, narrow(rows.k), y.cols, d.ld, y.ld, rows.data,
                                   static_cast<const float*>(weights), dy, ld, static_cast<float*>(dweights),
                                   stream_of(like)),
          "mxq_moe_combine_backward");
    return got.tuple();
}

// The address of a weight or shift [cols], null for None; *type: its dtype.
void* param(PyObject* o, const char* name, int64_t cols, int* type) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    *type = code_of(t);
    if (*type < 0) throw Refused{std::string(name) + " must be bfloat16 or float32"};
    return dense(t, name, t.scalar_type(), {cols});
}

// (x, weight, shift, eps, out)
PyObject* layer_norm(Args a) {
    const at::Tensor& like = tensor(a[0], "x");
    const Matrix x = matrix(like, "x");
    int type = MXQ_BF16, shift_type = 0;
    const void* weight = param(a[1], "weight", x.cols, &type);
    const void* shift = param(a[2], "shift", x.cols, &shift_type);
    if (a[2] != Py_None) {
        if (a[1] != Py_None && shift_type != type) throw Refused{"weight and shift must have the same dtype"};
        type = shift_type;
    }
    const Given out(a[4], 3);
    Results got;
    int64_t ld;
    void* y = got.matrix(out[0], "y", like, x.type, x.rows, x.cols, &ld);
    void* mean = got.dense(out[1], "mean", like, at::kFloat, {x.rows});
    void* rstd = got.dense(out[2], "rstd", like, at::kFloat, {x.rows});
    check(mxq_layer_norm(x.data, x.type, x.rows, x.cols, x.ld, weight, shift, static_cast<mxq_dtype>(type), number(a[3]),
                         y, ld, static_cast<float*>(mean), static_cast<float*>(rstd), stream_of(like)),
          "mxq_layer_norm");
    return got.tuple();
}

// (dy, x, weight, mean, rstd, out)
PyObject* layer_norm_backward(Args a) {
    const at::Tensor& like = tensor(a[1], "x");
    const Matrix x = matrix(like, "x");
    const Matrix dy = matrix(tensor(a[0], "dy"), "dy");
    if (dy.type != x.type || dy.rows != x.rows || dy.cols != x.cols)
        throw Refused{std::string("dy must be ") + name_of(like.scalar_type()) + " " + shape_of({x.rows, x.cols})};
    int type = MXQ_BF16;
    const void* weight = param(a[2], "weight", x.cols, &type);
    const void* mean = dense(a[3], "mean", at::kFloat, {x.rows});
    const void* rstd = dense(a[4], "rstd", at::kFloat, {x.rows});
    Results got;
    int64_t ld;
    void* dx = got.matrix(a[5], "dx", like, x.type, x.rows, x.cols, &ld);
    void* dweight = got.add(fresh(like, {x.cols}, at::kFloat));
    void* dshift = got.add(fresh(like, {x.cols}, at::kFloat));
    const size_t size = mxq_layer_norm_backward_workspace_size(x.rows, x.cols);
    const at::Tensor workspace = fresh(like, {static_cast<int64_t>(size)}, at::kByte);
    check(mxq_layer_norm_backward(dy.data, x.data, x.type, x.rows, x.cols, dy.ld, x.ld, weight,
                                  static_cast<mxq_dtype>(type), static_cast<const float*>(mean),
                                  static_cast<const float*>(rstd), dx, ld, static_cast<float*>(dweight),
                                  static_cast<float*>(dshift), workspace.data_ptr(), size, stream_of(like)),
          "mxq_layer_norm_backward");
    return got.tuple();
}

// The descriptor of a gradient and its output.
mxq_grad_desc grad_desc(const at::Tensor& g) {
    const int code = code_of(g);
    if (code < 0 || !g.is_cuda() || !g.is_contiguous())
        throw Refused{"gradients must be contiguous bfloat16 or float32 CUDA tensors"};
    same_device(g, "a gradient");
    mxq_grad_desc d{};
    d.grad = d.out = g.data_ptr();
    d.numel = g.numel();
    d.dtype = static_cast<mxq_dtype>(code);
    return d;
}

// The scalar for the norm and the workspace, on the gradients' device or the current one.
struct NormBuffers {
    at::Tensor norm, workspace;
    explicit NormBuffers(PyObject* grads) {
        at::TensorOptions on = at::TensorOptions().device(at::kCUDA);
        if (PyList_GET_SIZE(grads) > 0) on = tensor(PyList_GET_ITEM(grads, 0), "a gradient").options();
        norm = at::empty(at::IntArrayRef{}, on.dtype(at::kFloat));
        workspace = at::empty({static_cast<int64_t>(mxq_grad_norm_workspace_size(narrow(PyList_GET_SIZE(grads))))},
                              on.dtype(at::kByte));
    }
};

void want_list(PyObject* o) {
    if (PyList_Check(o)) return;
    PyErr_SetString(PyExc_TypeError, "a list of gradients is wanted");
    throw PythonError{};
}

// (grads: a list)
PyObject* grad_norm(Args a) {
    want_list(a[0]);
    const Py_ssize_t n = PyList_GET_SIZE(a[0]);
    std::vector<mxq_grad_desc> descs(static_cast<size_t>(n));
    for (Py_ssize_t i = 0; i < n; ++i) descs[i] = grad_desc(tensor(PyList_GET_ITEM(a[0], i), "a gradient"));
    const NormBuffers b(a[0]);
    check(mxq_grad_norm(descs.data(), narrow(n), static_cast<float*>(b.norm.data_ptr()), b.workspace.data_ptr(),
                        static_cast<size_t>(b.workspace.numel()), stream_of(b.norm)),
          "mxq_grad_norm");
    return wrapped(b.norm);
}

// (grads: a list, max_norm, eps, out: a list or None)
PyObject* clip_grad_norm(Args a) {
    want_list(a[0]);
    const Py_ssize_t n = PyList_GET_SIZE(a[0]);
    const bool fresh_out = a[3] == Py_None;
    Owned out(fresh_out ? PyList_New(n) : Py_NewRef(a[3]));
    want_list(out.get());
    if (PyList_GET_SIZE(out.get()) != n) throw Refused{"out must have a tensor for every gradient"};
    std::vector<mxq_grad_desc> descs(static_cast<size_t>(n));
    for (Py_ssize_t i = 0; i < n; ++i) {   // both lists are mxq.py's own: nobody else shortens them
        const at::Tensor& g = tensor(PyList_GET_ITEM(a[0], i), "a gradient");
        descs[i] = grad_desc(g);
        if (fresh_out) {
            at::Tensor t = at::empty_like(g);
            descs[i].out = t.data_ptr();
            PyList_SET_ITEM(out.get(), i, wrapped(std::move(t)));
            continue;
        }
        PyObject* o = PyList_GET_ITEM(out.get(), i);
        if (o == PyList_GET_ITEM(a[0], i)) continue;
        const at::Tensor& t = tensor(o, "an output");
        if (t.scalar_type() != g.scalar_type() || t.numel() != descs[i].numel || !t.is_cuda() || !t.is_contiguous())
            throw Refused{"every output must be a contiguous tensor like its gradient"};
        same_device(t, "an output");
        descs[i].out = t.data_ptr();
    }
    const NormBuffers b(a[0]);
    check(mxq_clip_grad_norm(descs.data(), narrow(n), number(a[1]), number(a[2]), static_cast<float*>(b.norm.data_ptr()),
                             b.workspace.data_ptr(), static_cast<size_t>(b.workspace.numel()), stream_of(b.norm)),
          "mxq_clip_grad_norm");
    const Owned norm(wrapped(b.norm));
    return PyTuple_Pack(2, norm.get(), out.get());
}

// ---- MXFP4, and activations kept in 8 bits ---------------------------------------------------

int64_t groups_of(int64_t cols) { return (cols + 31) / 32; }

int64_t scale_bytes(int64_t rows, int64_t cols, mxq_scale_layout layout) {
    return static_cast<int64_t>(mxq_scale_bytes(rows, 32 * groups_of(cols), layout));
}

// A contiguous uint8 CUDA tensor of this many bytes, whatever its shape.
void* bytes_of(PyObject* o, const char* name, int64_t size) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != at::kByte || !t.is_cuda() || !t.is_contiguous() || t.numel() != size)
        throw Refused{std::string(name) + " must be a contiguous uint8 CUDA tensor of " + std::to_string(size) + " bytes"};
    same_device(t, name);
    return t.data_ptr();
}

// A given matrix of this type and shape, or a new one.
void* matrix_out(Results& got, PyObject* given, const char* name, const at::Tensor& like, mxq_dtype type, int64_t rows,
                 int64_t cols, int64_t* ld) {
    const at::ScalarType scalar = type == MXQ_F32 ? at::kFloat : at::kBFloat16;
    if (given == Py_None) {
        *ld = cols;
        return got.add(fresh(like, {rows, cols}, scalar));
    }
    const Matrix m = matrix(tensor(given, name), name);
    if (m.type != type || m.rows != rows || m.cols != cols)
        throw Refused{std::string(name) + " must be " + name_of(scalar) + " " + shape_of({rows, cols})};
    *ld = m.ld;
    got.add(given);
    return m.data;
}

// A size that is an argument: what the library refuses is refused before memory is asked for.
int64_t size_arg(PyObject* o, const char* name) {
    const int64_t v = integer(o);
    if (v < 0) throw Refused{std::string(name) + " must not be negative"};
    if (v > (int64_t(1) << 31) - 4096) check(MXQ_ERR_UNSUPPORTED_SHAPE, name);
    return v;
}

mxq_scale_layout layout_of(PyObject* o) { return static_cast<mxq_scale_layout>(integer32(o)); }

// Payload and scales of one copy of `batch` matrices [rows, cols], as results.
struct Copy4 {
    void *q = nullptr, *s = nullptr;
    Copy4(Results& got, PyObject* q_out, PyObject* s_out, bool wanted, const char* q_name, const char* s_name,
          const at::Tensor& like, bool batched, int64_t batch, int64_t rows, int64_t cols, mxq_scale_layout layout) {
        if (!wanted) {
            if (q_out != Py_None || s_out != Py_None) throw Refused{std::string(q_name) + " is given and not asked for"};
            got.add(Py_None);
            got.add(Py_None);
            return;
        }
        const int64_t groups = groups_of(cols), size = scale_bytes(rows, cols, layout);
        if (batched) {
            q = got.dense(q_out, q_name, like, at::kByte, {batch, rows, 16 * groups});
            s = layout == MXQ_SCALE_ROWMAJOR ? got.dense(s_out, s_name, like, at::kByte, {batch, rows, groups})
                                             : got.dense(s_out, s_name, like, at::kByte, {batch, size});
        } else {
            q = got.dense(q_out, q_name, like, at::kByte, {rows, 16 * groups});
            s = layout == MXQ_SCALE_ROWMAJOR ? got.dense(s_out, s_name, like, at::kByte, {rows, groups})
                                             : got.dense(s_out, s_name, like, at::kByte, {size});
        }
    }
};

// (x, row, col, layout, out)
PyObject* quant_mxfp4(Args a) {
    const at::Tensor& x = tensor(a[0], "x");
    const int code = code_of(x);
    const bool batched = x.dim() == 3;
    if (code < 0 || (x.dim() != 2 && !batched) || !x.is_cuda())
        throw Refused{"x must be a 2-D or 3-D bfloat16 or float32 CUDA tensor"};
    same_device(x, "x");
    const int at0 = batched ? 1 : 0;
    const int64_t batch = batched ? x.size(0) : 1, rows = x.size(at0), cols = x.size(at0 + 1);
    if (x.stride(at0 + 1) != 1 && cols > 1) throw Refused{"x must have unit stride along its last axis"};
    const int64_t ld = rows > 1 || x.stride(at0) > cols ? x.stride(at0) : cols;
    const bool row = integer(a[1]) != 0, col = integer(a[2]) != 0;
    if (!row && !col) throw Refused{"neither copy is asked for"};
    const mxq_scale_layout layout = layout_of(a[3]);
    const Given out(a[4], 4);
    Results got;
    const Copy4 r(got, out[0], out[1], row, "q_row", "s_row", x, batched, batch, rows, cols, layout);
    const Copy4 c(got, out[2], out[3], col, "q_col", "s_col", x, batched, batch, cols, rows, layout);
    check(mxq_quant_mxfp4(x.data_ptr(), static_cast<mxq_dtype>(code), batch, rows, cols, ld, batched ? x.stride(0) : 0, r.q,
                          r.s, c.q, c.s, layout, stream_of(x)),
          "mxq_quant_mxfp4");
    return got.tuple();
}

// The experts' offsets [G + 1]; more experts than the library takes are refused before memory is asked for.
int32_t offsets_of(PyObject* o, const int64_t** data, const char* call) {
    const at::Tensor& t = tensor(o, "offsets");
    if (t.dim() != 1 || t.size(0) < 2) throw Refused{"offsets must be int64 [experts + 1]"};
    if (t.size(0) > 1025) check(MXQ_ERR_UNSUPPORTED_SHAPE, call);
    *data = static_cast<const int64_t*>(dense(t, "offsets", at::kLong, {t.size(0)}));
    return narrow(t.size(0) - 1);
}

// (x, offsets, out)
PyObject* quant_mxfp4_grouped(Args a) {
    const at::Tensor& like = tensor(a[0], "x");
    const Matrix x = matrix(like, "x");
    const int64_t* offsets;
    const int32_t G = offsets_of(a[1], &offsets, "mxq_quant_mxfp4_grouped");
    const int64_t bands = (x.rows + 127) / 128 + G;
    const Given out(a[2], 2);
    Results got;
    void* q = got.dense(out[0], "q", like, at::kByte, {x.rows, 16 * groups_of(x.cols)});
    void* s = got.dense(out[1], "s", like, at::kByte, {bands * ((x.cols + 127) / 128) * 512});
    check(mxq_quant_mxfp4_grouped(x.data, x.type, x.rows, x.cols, x.ld, offsets, G, bands, q, s, stream_of(like)),
          "mxq_quant_mxfp4_grouped");
    return got.tuple();
}

// (x, offsets, out)
PyObject* quant_mxfp4_cols_grouped(Args a) {
    const at::Tensor& like = tensor(a[0], "x");
    const Matrix x = matrix(like, "x");
    const int64_t* offsets;
    const int32_t G = offsets_of(a[1], &offsets, "mxq_quant_mxfp4_cols_grouped");
    const int64_t capacity = 128 * ((x.rows + 127) / 128 + G);
    const Given out(a[2], 2);
    Results got;
    void* q = got.dense(out[0], "q", like, at::kByte, {x.cols, capacity / 2});
    void* s = got.dense(out[1], "s", like, at::kByte, {scale_bytes(x.cols, capacity, MXQ_SCALE_MMA_TILED)});
    check(mxq_quant_mxfp4_cols_grouped(x.data, x.type, x.rows, x.cols, x.ld, offsets, G, capacity, q, s, stream_of(like)),
          "mxq_quant_mxfp4_cols_grouped");
    return got.tuple();
}

// (q, s, cols, element, layout, dtype, out)
PyObject* dequant_1x32(Args a) {
    const at::Tensor& q = tensor(a[0], "q");
    const at::Tensor& s = tensor(a[1], "s");
    if (q.scalar_type() != at::kByte || q.dim() != 2 || !q.is_cuda() || (q.stride(1) != 1 && q.size(1) > 1))
        throw Refused{"q must be a 2-D uint8 CUDA tensor with unit stride along its last axis"};
    same_device(q, "q");
    const int64_t rows = q.size(0), cols = size_arg(a[2], "cols"), groups = groups_of(cols);
    const mxq_element element = static_cast<mxq_element>(integer32(a[3]));
    const mxq_scale_layout layout = layout_of(a[4]);
    const mxq_dtype type = static_cast<mxq_dtype>(integer32(a[5]));
    const int64_t width = element == MXQ_ELEM_E2M1 ? 16 * groups : cols;
    if (q.size(1) != width) throw Refused{"q must have " + std::to_string(width) + " bytes a row"};
    int64_t lds = groups;
    const void* scales;
    if (layout == MXQ_SCALE_MMA_TILED) {
        scales = bytes_of(a[1], "s", scale_bytes(rows, cols, layout));
    } else {
        if (s.scalar_type() != at::kByte || s.dim() != 2 || !s.is_cuda() || s.size(0) != rows || s.size(1) != groups ||
            (s.stride(1) != 1 && groups > 1))
            throw Refused{"s must be a uint8 CUDA tensor " + shape_of({rows, groups}) + " with unit stride along its last axis"};
        same_device(s, "s");
        if (rows > 1) lds = s.stride(0);
        scales = s.data_ptr();
    }
    Results got;
    int64_t ld;
    void* out = matrix_out(got, a[6], "out", q, type, rows, cols, &ld);
    check(mxq_dequant_1x32(q.data_ptr(), scales, element, rows, cols, rows > 1 || q.stride(0) > width ? q.stride(0) : width,
                           lds, layout, out, type, ld, stream_of(q)),
          "mxq_dequant_1x32");
    return got.one();
}

// (a_q, a_s, b_q, b_s, M, N, K, out)
PyObject* gemm_mxfp4(Args a) {
    const at::Tensor& like = tensor(a[0], "a_q");
    const int64_t M = size_arg(a[4], "M"), N = size_arg(a[5], "N"), K = size_arg(a[6], "K"), row = 16 * groups_of(K);
    const void* a_q = bytes_of(a[0], "a_q", M * row);
    const void* a_s = bytes_of(a[1], "a_s", scale_bytes(M, K, MXQ_SCALE_MMA_TILED));
    const void* b_q = bytes_of(a[2], "b_q", N * row);
    const void* b_s = bytes_of(a[3], "b_s", scale_bytes(N, K, MXQ_SCALE_MMA_TILED));
    Results got;
    int64_t ld;
    void* y = matrix_out(got, a[7], "out", like, MXQ_BF16, M, N, &ld);
    check(mxq_gemm_mxfp4(a_q, a_s, b_q, b_s, M, N, K, y, ld, stream_of(like)), "mxq_gemm_mxfp4");
    return got.one();
}

// (a_q, a_s, b_q, b_s, offsets, N, K, out)
PyObject* grouped_gemm_mxfp4(Args a) {
    const at::Tensor& like = tensor(a[0], "a_q");
    if (like.dim() != 2) throw Refused{"a_q must be 2-D"};
    const int64_t M = like.size(0), N = size_arg(a[5], "N"), K = size_arg(a[6], "K"), row = 16 * groups_of(K);
    const int64_t* offsets;
    const int32_t G = offsets_of(a[4], &offsets, "mxq_grouped_gemm_mxfp4");
    const int64_t bands = (M + 127) / 128 + G;
    const void* a_q = bytes_of(a[0], "a_q", M * row);
    const void* a_s = bytes_of(a[1], "a_s", bands * ((K + 127) / 128) * 512);
    const void* b_q = bytes_of(a[2], "b_q", G * N * row);
    const void* b_s = bytes_of(a[3], "b_s", G * scale_bytes(N, K, MXQ_SCALE_MMA_TILED));
    Results got;
    int64_t ld;
    void* y = matrix_out(got, a[7], "out", like, MXQ_BF16, M, N, &ld);
    check(mxq_grouped_gemm_mxfp4(a_q, a_s, bands, b_q, b_s, offsets, G, M, N, K, y, ld, stream_of(like)),
          "mxq_grouped_gemm_mxfp4");
    return got.one();
}

// (a_q, a_s, b_q, b_s, offsets, M_total, out)
PyObject* grouped_gemm_mxfp4_wgrad(Args a) {
    const at::Tensor& like = tensor(a[0], "a_q");
    const at::Tensor& b = tensor(a[2], "b_q");
    if (like.dim() != 2 || b.dim() != 2) throw Refused{"a_q and b_q must be 2-D"};
    const int64_t M = like.size(0), N = b.size(0), rows = size_arg(a[5], "M_total");
    const int64_t* offsets;
    const int32_t G = offsets_of(a[4], &offsets, "mxq_grouped_gemm_mxfp4_wgrad");
    const int64_t capacity = 128 * ((rows + 127) / 128 + G);
    const void* a_q = bytes_of(a[0], "a_q", M * (capacity / 2));
    const void* a_s = bytes_of(a[1], "a_s", scale_bytes(M, capacity, MXQ_SCALE_MMA_TILED));
    const void* b_q = bytes_of(a[2], "b_q", N * (capacity / 2));
    const void* b_s = bytes_of(a[3], "b_s", scale_bytes(N, capacity, MXQ_SCALE_MMA_TILED));
    Results got;
    void* y = got.dense(a[6], "out", like, at::kBFloat16, {G, M, N});
    check(mxq_grouped_gemm_mxfp4_wgrad(a_q, a_s, b_q, b_s, offsets, G, rows, capacity, M, N, y, N, stream_of(like)),
          "mxq_grouped_gemm_mxfp4_wgrad");
    return got.one();
}

// (z, kind, gated, checkpoint, out)
PyObject* activation(Args a) {
    const at::Tensor& like = tensor(a[0], "z");
    const Matrix z = matrix(like, "z");
    const int32_t gated = integer32(a[2]);
    if (gated != 0 && z.cols % 2 != 0) throw Refused{"a gated z must have an even number of columns"};
    const bool keep = integer(a[3]) != 0;
    const int64_t parts = gated != 0 ? 2 : 1, inter = z.cols / parts;
    const Given out(a[4], 3);
    Results got;
    int64_t ld;
    void* y = got.matrix(out[0], "y", like, z.type, z.rows, inter, &ld);
    void *q = nullptr, *s = nullptr;
    if (keep) {
        q = got.dense(out[1], "q", like, at::kByte, {z.rows, z.cols});
        s = got.dense(out[2], "s", like, at::kByte, {z.rows, parts * groups_of(inter)});
    } else {
        if (out[1] != Py_None || out[2] != Py_None) throw Refused{"a checkpoint's tensor is given and none is asked for"};
        got.add(Py_None);
        got.add(Py_None);
    }
    check(mxq_activation(z.data, z.type, z.rows, inter, z.ld, static_cast<mxq_act>(integer32(a[1])), gated, y, ld, q, s,
                         stream_of(like)),
          "mxq_activation");
    return got.tuple();
}

// (dy, q, s, kind, gated, output, out)
PyObject* activation_backward(Args a) {
    const at::Tensor& like = tensor(a[0], "dy");
    const Matrix dy = matrix(like, "dy");
    const int32_t gated = integer32(a[4]);
    const int64_t parts = gated != 0 ? 2 : 1;
    const void* q = dense(a[1], "q", at::kByte, {dy.rows, parts * dy.cols});
    const void* s = dense(a[2], "s", at::kByte, {dy.rows, parts * groups_of(dy.cols)});
    const bool again = integer(a[5]) != 0;
    const Given out(a[6], 2);
    Results got;
    int64_t lddz, ldy = 0;
    void* dz = got.matrix(out[0], "dz", like, dy.type, dy.rows, parts * dy.cols, &lddz);
    void* y = nullptr;
    if (again) {
        y = got.matrix(out[1], "y", like, dy.type, dy.rows, dy.cols, &ldy);
    } else {
        if (out[1] != Py_None) throw Refused{"y is given and not asked for"};
        got.add(Py_None);
    }
    check(mxq_activation_backward(dy.data, dy.type, dy.ld, q, s, dy.rows, dy.cols, static_cast<mxq_act>(integer32(a[3])), gated,
                                  dz, lddz, y, ldy, stream_of(like)),
          "mxq_activation_backward");
    return got.tuple();
}

// ---- the module -----------------------------------------------------------------------------

// f(args) with every exception as a Python error.
template <PyObject* (*kCall)(Args), int kArgs>
PyObject* entry(PyObject*, Args args, Py_ssize_t given) {
    HANDLE_TH_ERRORS
    const OnDevice device;
    try {
        if (given != kArgs) {
            PyErr_Format(PyExc_TypeError, "%d arguments are wanted, not %zd", kArgs, given);
            return nullptr;
        }
        return kCall(args);
    } catch (const Refused& r) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, r.why.c_str());
        return nullptr;
    } catch (const PythonError&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// (raise_status)
PyObject* set_error(Args a) {
    Py_XSETREF(raise_status, Py_NewRef(a[0]));
    return Py_NewRef(Py_None);
}

#define ENTRY(name, n) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name, n>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {ENTRY(route, 11), ENTRY(route_backward, 7), ENTRY(moe_plan, 3), ENTRY(moe_dispatch, 3),
                         ENTRY(moe_combine, 4), ENTRY(moe_combine_backward, 5), ENTRY(layer_norm, 5),
                         ENTRY(layer_norm_backward, 6), ENTRY(grad_norm, 1), ENTRY(clip_grad_norm, 4),
                         ENTRY(quant_mxfp4, 5), ENTRY(quant_mxfp4_grouped, 3), ENTRY(dequant_1x32, 7),
                         ENTRY(quant_mxfp4_cols_grouped, 3), ENTRY(gemm_mxfp4, 8), ENTRY(grouped_gemm_mxfp4, 8),
                         ENTRY(grouped_gemm_mxfp4_wgrad, 7), ENTRY(activation, 5),
                         ENTRY(activation_backward, 7), ENTRY(set_error, 1), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mxqcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mxqcall() {
    PyObject* torch_c = PyImport_ImportModule("torch._C");
    if (torch_c == nullptr) return nullptr;
    raw_stream = PyObject_GetAttrString(torch_c, "_cuda_getCurrentRawStream");
    Py_DECREF(torch_c);
    if (raw_stream == nullptr) return nullptr;   // a torch without CUDA
    return PyModule_Create(&module);
}
