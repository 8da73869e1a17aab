// binding.cpp -- the Python binding of include/iq_layers.h, iq_fp4.h and iq_router.h:
// checks tensors, allocates the results that were not given and calls the C-ABI.
//
// It is compiled because the small calls of these operators are bound by the
// host: an operator on a few tokens runs for 3 to 6 us, and checking its
// tensors and allocating its result took 5 us from Python and takes 1.5 us
// here (a launch is 2.7 us).  The functions are positional; layers.py gives
// them names, defaults, documentation and their place in autograd's graph.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <c10/core/AutogradState.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/autograd/python_variable.h>

#include "iq_fp4.h"
#include "iq_layers.h"
#include "iq_router.h"

namespace {

// A refused argument: a Python TypeError or ValueError with this text.
struct Refused {
    PyObject* kind;
    std::string text;
};

[[noreturn]] void type_error(const std::string& text) { throw Refused{PyExc_TypeError, text}; }
[[noreturn]] void value_error(const std::string& text) { throw Refused{PyExc_ValueError, text}; }

std::string name_of(at::ScalarType t)
{
    switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kChar: return "torch.int8";
    case at::kByte: return "torch.uint8";
    default: return std::string("torch.") + c10::toString(t);
    }
}

// A non-zero status, raised as the package's IQError.
struct Failed {
    iq_status_t code;
    const char* where;
};

void check(iq_status_t code, const char* where)
{
    if (code != IQ_OK) throw Failed{code, where};
}

// The library call without the interpreter's lock: calls that report data
// errors by themselves wait for the GPU.
template <class Call>
iq_status_t unlocked(Call&& call)
{
    PyThreadState* state = PyEval_SaveThread();
    const iq_status_t code = call();
    PyEval_RestoreThread(state);
    return code;
}

const at::Tensor& gpu_tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) value_error(std::string(name) + " must be on the GPU");
    // Its memory holds the values with the other sign.
    if (t.is_neg()) value_error(std::string(name) + " is a negated view: call resolve_neg() on it");
    return t;
}

// What all tensors of a call share: the GPU of the first, which has to be the
// current device because that is where kernels are launched, and its current
// stream.
struct Call {
    int index;
    hipStream_t stream;
    Call(PyObject* first, const char* name)
    {
        index = gpu_tensor(first, name).get_device();
        if (index != c10::hip::current_device())
            value_error(std::string(name) + " is on cuda:" + std::to_string(index) +
                        ", which is not the current device");
        stream = c10::hip::getCurrentHIPStream((c10::DeviceIndex)index).stream();
    }
    at::TensorOptions options(at::ScalarType type) const
    {
        return at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)index));
    }
};

const at::Tensor& tensor(const Call& c, PyObject* o, const char* name)
{
    const at::Tensor& t = gpu_tensor(o, name);
    if (t.get_device() != c.index)
        value_error(std::string(name) + " must be on cuda:" + std::to_string(c.index));
    return t;
}

// iq_dtype_t of the values that these operators take.
bool value_type(at::ScalarType t, iq_dtype_t* out)
{
    if (t == at::kFloat)
        *out = IQ_DTYPE_F32;
    else if (t == at::kBFloat16)
        *out = IQ_DTYPE_BF16;
    else if (t == at::kHalf)
        *out = IQ_DTYPE_F16;
    else
        return false;
    return true;
}

void expect_type(const at::Tensor& t, at::ScalarType type, const char* name)
{
    if (t.scalar_type() != type)
        type_error(std::string(name) + " must be " + name_of(type) + ", got " + name_of(t.scalar_type()));
}

// A two-dimensional tensor with consecutive values in a row.
struct Matrix {
    const at::Tensor& t;
    int64_t rows, cols, ld;
    Matrix(const at::Tensor& m, const char* name) : t(m)
    {
        if (m.dim() != 2) value_error(std::string(name) + " must have two dimensions");
        rows = m.size(0);
        cols = m.size(1);
        ld = m.stride(0);
        if (m.stride(1) != 1 && cols != 1)
            value_error(std::string(name) + " must have consecutive values in a row");
    }
    void* data() const { return t.data_ptr(); }
};

Matrix values(const Call& c, PyObject* o, const char* name, iq_dtype_t* type)
{
    const at::Tensor& t = tensor(c, o, name);
    if (!value_type(t.scalar_type(), type))
        type_error(std::string(name) + " must be float32, bfloat16 or float16, got " +
                   name_of(t.scalar_type()));
    return Matrix(t, name);
}

Matrix codes(const Call& c, PyObject* o, const char* name)
{
    const at::Tensor& t = tensor(c, o, name);
    expect_type(t, at::kChar, name);
    return Matrix(t, name);
}

// Codes and scales of `groups` 4-bit groups of 32 to a row: bytes, `per_group` of
// them for each group.
Matrix group_bytes(const Call& c, PyObject* o, const char* name, int64_t per_group, int64_t groups)
{
    const at::Tensor& t = tensor(c, o, name);
    expect_type(t, at::kByte, name);
    const Matrix m(t, name);
    if (m.cols != per_group * groups)
        value_error(std::string(name) + " must have " + std::to_string(per_group * groups) + " columns");
    return m;
}

// A depth in groups.
int64_t groups_of(int64_t values, const char* name)
{
    if (values < IQ_GROUP || values % IQ_GROUP)
        value_error(std::string(name) + " must have a multiple of " + std::to_string(IQ_GROUP) + " columns");
    return values / IQ_GROUP;
}

// The same for each expert: [experts, channels, bytes] with consecutive bytes.
const at::Tensor& expert_bytes(const Call& c, PyObject* o, const char* name, int64_t bytes)
{
    const at::Tensor& t = tensor(c, o, name);
    expect_type(t, at::kByte, name);
    if (t.dim() != 3 || t.size(2) != bytes || (t.stride(2) != 1 && bytes != 1))
        value_error(std::string(name) + " must be [experts, channels, " + std::to_string(bytes) +
                    "] with consecutive bytes in a row");
    return t;
}

// A contiguous tensor of that type and shape.
template <class T>
T* array(const Call& c, PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape)
{
    const at::Tensor& t = tensor(c, o, name);
    expect_type(t, type, name);
    if (t.sizes() != shape || !t.is_contiguous()) {
        std::string text = std::string(name) + " must be a contiguous tensor of shape (";
        for (int64_t n : shape) text += std::to_string(n) + ", ";
        value_error(text + ")");
    }
    return static_cast<T*>(t.data_ptr());
}

// The status word, or null where the library is to wait and report by itself.
int32_t* status_word(const Call& c, PyObject* o)
{
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(c, o, "status");
    expect_type(t, at::kInt, "status");
    if (!t.is_contiguous() || t.numel() < 1) value_error("status must be a contiguous tensor");
    return static_cast<int32_t*>(t.data_ptr());
}

// The result: the caller's, which is returned as it is, or a new one.
struct Result {
    at::Tensor t;
    PyObject* given;
    int64_t ld;
    Result(const Call& c, PyObject* out, int64_t rows, int64_t cols, at::ScalarType type)
        : given(out == Py_None ? nullptr : out)
    {
        if (!given) {
            t = at::empty({rows, cols}, c.options(type));
            ld = cols;
            return;
        }
        t = tensor(c, out, "out");
        expect_type(t, type, "out");
        const Matrix m(t, "out");
        if (m.rows != rows || m.cols != cols)
            value_error("out must be [" + std::to_string(rows) + ", " + std::to_string(cols) + "]");
        ld = m.ld;
    }
    // For the call that writes it: a tensor of the caller's is a new version of
    // itself from then on, which autograd checks what it has saved by.  (Inference
    // tensors have no versions.)
    void* data() const
    {
        if (given && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
        return t.data_ptr();
    }
    PyObject* object() const
    {
        if (!given) return THPVariable_Wrap(t);
        Py_INCREF(given);
        return given;
    }
};

PyObject* tuple(std::initializer_list<at::Tensor> tensors)
{
    PyObject* result = PyTuple_New((Py_ssize_t)tensors.size());
    Py_ssize_t i = 0;
    for (const at::Tensor& t : tensors) PyTuple_SET_ITEM(result, i++, THPVariable_Wrap(t));
    return result;
}

// What expert_sort answers with.
struct Routing {
    int64_t tokens, top_k, experts;
    const int32_t *position, *offsets;
    Routing(const Call& c, PyObject* position_, PyObject* offsets_)
    {
        const at::Tensor& p = tensor(c, position_, "position");
        const at::Tensor& f = tensor(c, offsets_, "offsets");
        expect_type(p, at::kInt, "position");
        expect_type(f, at::kInt, "offsets");
        if (p.dim() != 2 || !p.is_contiguous())
            value_error("position must be a contiguous [tokens, top_k] tensor");
        if (f.dim() != 1 || f.size(0) < 2 || !f.is_contiguous())
            value_error("offsets must be a contiguous [num_experts + 1] tensor");
        tokens = p.size(0);
        top_k = p.size(1);
        experts = f.size(0) - 1;
        if (top_k > INT32_MAX || experts > INT32_MAX) value_error("too many choices or experts");
        position = static_cast<const int32_t*>(p.data_ptr());
        offsets = static_cast<const int32_t*>(f.data_ptr());
    }
};

void expect_rows(const Matrix& m, int64_t rows, const char* name)
{
    if (m.rows != rows) value_error(std::string(name) + " must have " + std::to_string(rows) + " rows");
}

// The type asked for, or that of a given result.
at::ScalarType result_type(PyObject* dtype, PyObject* out, iq_dtype_t* type)
{
    at::ScalarType t;
    if (out != Py_None) {
        if (!THPVariable_Check(out)) type_error("out must be a torch.Tensor");
        t = THPVariable_Unpack(out).scalar_type();
    } else {
        if (!THPDtype_Check(dtype)) type_error("dtype must be a torch.dtype");
        t = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
    }
    if (!value_type(t, type))
        type_error("dtype must be float32, bfloat16 or float16, got " + name_of(t));
    return t;
}

int32_t int32_of(PyObject* o, const char* name)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error(std::string(name) + " must be an integer");
    }
    if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " is out of range");
    return (int32_t)v;
}

// --- the calls, with the arguments of layers.py in their order -------------

PyObject* quantize_rows(PyObject* const* a)
{
    const Call c(a[0], "x");
    iq_dtype_t type;
    const Matrix x = values(c, a[0], "x", &type);
    int32_t* status = status_word(c, a[1]);
    at::Tensor q = at::empty({x.rows, x.cols}, c.options(at::kChar));
    at::Tensor scale = at::empty({x.rows}, c.options(at::kFloat));
    check(unlocked([&] {
        return iq_quantize_rows(type, x.data(), x.ld, x.rows, x.cols,
                                static_cast<int8_t*>(q.data_ptr()), x.cols,
                                static_cast<float*>(scale.data_ptr()), status, c.stream);
    }), "iq_quantize_rows");
    return tuple({q, scale});
}

PyObject* int8_matmul(PyObject* const* a)
{
    const Call c(a[0], "x");
    const Matrix x = codes(c, a[0], "x"), w = codes(c, a[2], "w");
    if (w.cols != x.cols) value_error("w must be [channels, " + std::to_string(x.cols) + "]");
    const float* xs = array<float>(c, a[1], "x_scale", at::kFloat, {x.rows});
    const float* ws = array<float>(c, a[3], "w_scale", at::kFloat, {w.rows});
    iq_dtype_t type;
    const at::ScalarType t = result_type(a[4], a[5], &type);
    const Result y(c, a[5], x.rows, w.rows, t);
    check(unlocked([&] {
        return iq_int8_matmul(static_cast<int8_t*>(x.data()), x.ld, xs,
                              static_cast<int8_t*>(w.data()), w.ld, ws, x.rows, w.rows, x.cols,
                              type, y.data(), y.ld, c.stream);
    }), "iq_int8_matmul");
    return y.object();
}

PyObject* int8_linear(PyObject* const* a)
{
    const Call c(a[0], "x");
    iq_dtype_t type;
    const Matrix x = values(c, a[0], "x", &type), w = codes(c, a[1], "w");
    if (w.cols != x.cols) value_error("w must be [channels, " + std::to_string(x.cols) + "]");
    const float* ws = array<float>(c, a[2], "w_scale", at::kFloat, {w.rows});
    const Result y(c, a[3], x.rows, w.rows, x.t.scalar_type());
    int32_t* status = status_word(c, a[4]);
    const int64_t need = iq_int8_linear_workspace(x.rows, w.rows, x.cols);
    at::Tensor work;
    if (need) work = at::empty({need}, c.options(at::kByte));
    check(unlocked([&] {
        return iq_int8_linear(type, x.data(), x.ld, static_cast<int8_t*>(w.data()), w.ld, ws,
                              x.rows, w.rows, x.cols, y.data(), y.ld,
                              need ? work.data_ptr() : nullptr, need, status, c.stream);
    }), "iq_int8_linear");
    return y.object();
}

PyObject* int8_expert_matmul(PyObject* const* a)
{
    const Call c(a[0], "x");
    const Matrix x = codes(c, a[0], "x");
    const at::Tensor& w = tensor(c, a[2], "w");
    expect_type(w, at::kChar, "w");
    if (w.dim() != 3 || w.size(2) != x.cols || (w.stride(2) != 1 && x.cols != 1))
        value_error("w must be [experts, channels, " + std::to_string(x.cols) +
                    "] with consecutive values in a row");
    const int64_t experts = w.size(0), channels = w.size(1);
    const int32_t top_k = int32_of(a[6], "top_k");
    const float* xs = array<float>(c, a[1], "x_scale", at::kFloat, {x.rows});
    const float* ws = array<float>(c, a[3], "w_scale", at::kFloat, {experts, channels});
    const int32_t* offsets = array<int32_t>(c, a[4], "offsets", at::kInt, {experts + 1});
    int64_t rows = x.rows;
    const int32_t* order = nullptr;
    if (a[5] != Py_None) {
        rows = x.rows * std::max(top_k, 0);
        order = array<int32_t>(c, a[5], "order", at::kInt, {rows});
    }
    iq_dtype_t type;
    const at::ScalarType t = result_type(a[7], a[8], &type);
    const Result y(c, a[8], rows, channels, t);
    if (experts > INT32_MAX) value_error("too many experts");
    check(unlocked([&] {
        return iq_int8_expert_matmul(static_cast<int8_t*>(x.data()), x.ld, xs, x.rows, order, top_k,
                                     offsets, (int32_t)experts, rows,
                                     static_cast<int8_t*>(w.data_ptr()), w.stride(1), w.stride(0),
                                     ws, channels, x.cols, type, y.data(), y.ld, c.stream);
    }), "iq_int8_expert_matmul");
    return y.object();
}

PyObject* quantize_groups(PyObject* const* a)
{
    const Call c(a[0], "w");
    iq_dtype_t type;
    const Matrix w = values(c, a[0], "w", &type);
    const int64_t groups = groups_of(w.cols, "w");
    int32_t* status = status_word(c, a[1]);
    at::Tensor codes = at::empty({w.rows, w.cols / 2}, c.options(at::kByte));
    at::Tensor scale = at::empty({w.rows, groups}, c.options(at::kByte));
    check(unlocked([&] {
        return iq_quantize_groups(type, w.data(), w.ld, w.rows, w.cols,
                                  static_cast<uint8_t*>(codes.data_ptr()), w.cols / 2,
                                  static_cast<uint8_t*>(scale.data_ptr()), groups, status, c.stream);
    }), "iq_quantize_groups");
    return tuple({codes, scale});
}

PyObject* dequantize_groups(PyObject* const* a)
{
    const Call c(a[0], "codes");
    const at::Tensor& t = tensor(c, a[0], "codes");
    expect_type(t, at::kByte, "codes");
    const Matrix codes(t, "codes");
    const int64_t groups = groups_of(2 * codes.cols, "the values of codes");
    const Matrix scale = group_bytes(c, a[1], "scale", 1, groups);
    expect_rows(scale, codes.rows, "scale");
    iq_dtype_t type;
    const at::ScalarType out = result_type(a[2], a[3], &type);
    const Result y(c, a[3], codes.rows, 2 * codes.cols, out);
    check(unlocked([&] {
        return iq_dequantize_groups(static_cast<uint8_t*>(codes.data()), codes.ld,
                                    static_cast<uint8_t*>(scale.data()), scale.ld, codes.rows,
                                    2 * codes.cols, type, y.data(), y.ld, c.stream);
    }), "iq_dequantize_groups");
    return y.object();
}

PyObject* fp4_linear(PyObject* const* a)
{
    const Call c(a[0], "x");
    iq_dtype_t type;
    const Matrix x = values(c, a[0], "x", &type);
    const int64_t groups = groups_of(x.cols, "x");
    const Matrix w = group_bytes(c, a[1], "w", IQ_GROUP / 2, groups);
    const Matrix scale = group_bytes(c, a[2], "w_scale", 1, groups);
    expect_rows(scale, w.rows, "w_scale");
    const Result y(c, a[3], x.rows, w.rows, x.t.scalar_type());
    const int64_t need = iq_fp4_linear_workspace(type, x.data(), x.ld, x.rows, w.rows, x.cols);
    at::Tensor work;
    if (need) work = at::empty({need}, c.options(at::kByte));
    check(unlocked([&] {
        return iq_fp4_linear(type, x.data(), x.ld, static_cast<uint8_t*>(w.data()), w.ld,
                             static_cast<uint8_t*>(scale.data()), scale.ld, x.rows, w.rows, x.cols,
                             y.data(), y.ld, need ? work.data_ptr() : nullptr, need, c.stream);
    }), "iq_fp4_linear");
    return y.object();
}

PyObject* fp4_expert_linear(PyObject* const* a)
{
    const Call c(a[0], "x");
    iq_dtype_t type;
    const Matrix x = values(c, a[0], "x", &type);
    const int64_t groups = groups_of(x.cols, "x");
    const at::Tensor& w = expert_bytes(c, a[1], "w", IQ_GROUP / 2 * groups);
    const at::Tensor& scale = expert_bytes(c, a[2], "w_scale", groups);
    const int64_t experts = w.size(0), channels = w.size(1);
    if (scale.size(0) != experts || scale.size(1) != channels)
        value_error("w_scale must be [" + std::to_string(experts) + ", " + std::to_string(channels) +
                    ", " + std::to_string(groups) + "]");
    const int32_t top_k = int32_of(a[5], "top_k");
    const int32_t* offsets = array<int32_t>(c, a[3], "offsets", at::kInt, {experts + 1});
    int64_t rows = x.rows;
    const int32_t* order = nullptr;
    if (a[4] != Py_None) {
        rows = x.rows * std::max(top_k, 0);
        order = array<int32_t>(c, a[4], "order", at::kInt, {rows});
    }
    const Result y(c, a[6], rows, channels, x.t.scalar_type());
    if (experts > INT32_MAX) value_error("too many experts");
    const int64_t need = iq_fp4_expert_linear_workspace(type, x.data(), x.ld, x.rows,
                                                        (int32_t)experts, rows, channels, x.cols);
    at::Tensor work;
    if (need) work = at::empty({need}, c.options(at::kByte));
    check(unlocked([&] {
        return iq_fp4_expert_linear(type, x.data(), x.ld, x.rows, order, top_k, offsets,
                                    (int32_t)experts, rows, static_cast<uint8_t*>(w.data_ptr()),
                                    w.stride(1), w.stride(0),
                                    static_cast<uint8_t*>(scale.data_ptr()), scale.stride(1),
                                    scale.stride(0), channels, x.cols, y.data(), y.ld,
                                    need ? work.data_ptr() : nullptr, need, c.stream);
    }), "iq_fp4_expert_linear");
    return y.object();
}

// [tokens, experts].
Matrix logits_of(const Call& c, PyObject* o, iq_dtype_t* type)
{
    const Matrix l = values(c, o, "logits", type);
    if (l.cols > INT32_MAX) value_error("too many experts");
    return l;
}

bool bool_of(PyObject* o, const char* name)
{
    if (!PyBool_Check(o)) type_error(std::string(name) + " must be True or False");
    return o == Py_True;
}

PyObject* expert_gate(PyObject* const* a)
{
    const Call c(a[0], "logits");
    iq_dtype_t type;
    const Matrix l = logits_of(c, a[0], &type);
    const int32_t top_k = int32_of(a[1], "top_k");
    const bool renormalize = bool_of(a[2], "renormalize");
    int32_t* status = status_word(c, a[3]);
    // The library refuses others, for which no room is made.
    const int64_t k = top_k > 0 && top_k <= l.cols ? top_k : 0;
    at::Tensor choice = at::empty({l.rows, k}, c.options(at::kInt));
    at::Tensor weights = at::empty({l.rows, k}, c.options(at::kFloat));
    check(unlocked([&] {
        return iq_expert_gate(type, l.data(), l.ld, l.rows, (int32_t)l.cols, top_k, renormalize,
                              static_cast<int32_t*>(choice.data_ptr()),
                              static_cast<float*>(weights.data_ptr()), status, c.stream);
    }), "iq_expert_gate");
    return tuple({choice, weights});
}

PyObject* expert_gate_backward(PyObject* const* a)
{
    const Call c(a[0], "grad");
    iq_dtype_t type;
    const Matrix l = logits_of(c, a[1], &type);
    const at::Tensor& t = tensor(c, a[2], "choice");
    if (t.dim() != 2 || t.size(0) != l.rows)
        value_error("choice must be a contiguous [tokens, top_k] tensor");
    const int64_t k = t.size(1);
    if (k > INT32_MAX) value_error("too many choices");
    const int32_t* choice = array<int32_t>(c, a[2], "choice", at::kInt, {l.rows, k});
    const float* weights = array<float>(c, a[3], "weights", at::kFloat, {l.rows, k});
    const float* grad = array<float>(c, a[0], "grad", at::kFloat, {l.rows, k});
    const bool renormalize = bool_of(a[4], "renormalize");
    at::Tensor out = at::empty({l.rows, l.cols}, c.options(l.t.scalar_type()));
    check(unlocked([&] {
        return iq_expert_gate_backward(type, grad, l.data(), l.ld, l.rows, (int32_t)l.cols, choice,
                                       weights, (int32_t)k, renormalize, out.data_ptr(), l.cols,
                                       c.stream);
    }), "iq_expert_gate_backward");
    return THPVariable_Wrap(out);
}

PyObject* expert_balance(PyObject* const* a)
{
    const Call c(a[0], "logits");
    iq_dtype_t type;
    const Matrix l = logits_of(c, a[0], &type);
    const at::Tensor& choice = tensor(c, a[1], "choice");
    if (choice.scalar_type() != at::kInt && choice.scalar_type() != at::kLong)
        type_error("choice must be int32 or int64, got " + name_of(choice.scalar_type()));
    if (choice.dim() != 2 || choice.size(0) != l.rows || !choice.is_contiguous())
        value_error("choice must be a contiguous [tokens, top_k] tensor");
    const int64_t k = choice.size(1);
    if (k > INT32_MAX) value_error("too many choices");
    int32_t* status = status_word(c, a[2]);
    at::Tensor loss = at::empty({}, c.options(at::kFloat));
    at::Tensor counts = at::empty({l.cols}, c.options(at::kInt));
    at::Tensor live = at::empty({}, c.options(at::kInt));
    const int64_t need = iq_expert_balance_workspace(l.rows, (int32_t)l.cols);
    at::Tensor work;
    if (need) work = at::empty({need}, c.options(at::kByte));
    check(unlocked([&] {
        return iq_expert_balance(type, l.data(), l.ld, l.rows, (int32_t)l.cols, choice.data_ptr(),
                                 (int32_t)choice.element_size(), (int32_t)k,
                                 static_cast<float*>(loss.data_ptr()),
                                 static_cast<int32_t*>(counts.data_ptr()),
                                 static_cast<int32_t*>(live.data_ptr()),
                                 need ? work.data_ptr() : nullptr, need, status, c.stream);
    }), "iq_expert_balance");
    return tuple({loss, counts, live});
}

PyObject* expert_balance_backward(PyObject* const* a)
{
    const Call c(a[0], "grad");
    iq_dtype_t type;
    const Matrix l = logits_of(c, a[1], &type);
    const at::Tensor& grad = tensor(c, a[0], "grad");
    expect_type(grad, at::kFloat, "grad");
    if (grad.numel() != 1) value_error("grad must have one value");
    const int32_t* counts = array<int32_t>(c, a[2], "counts", at::kInt, {l.cols});
    const int32_t* live = array<int32_t>(c, a[3], "live", at::kInt, {});
    at::Tensor out = at::empty({l.rows, l.cols}, c.options(l.t.scalar_type()));
    check(unlocked([&] {
        return iq_expert_balance_backward(type, static_cast<float*>(grad.data_ptr()), l.data(), l.ld,
                                          l.rows, (int32_t)l.cols, counts, live, out.data_ptr(),
                                          l.cols, c.stream);
    }), "iq_expert_balance_backward");
    return THPVariable_Wrap(out);
}

PyObject* expert_sort(PyObject* const* a)
{
    const Call c(a[0], "experts_of");
    const at::Tensor& choice = tensor(c, a[0], "experts_of");
    if (choice.scalar_type() != at::kInt && choice.scalar_type() != at::kLong)
        type_error("experts_of must be int32 or int64, got " + name_of(choice.scalar_type()));
    if (choice.dim() != 2 || !choice.is_contiguous())
        value_error("experts_of must be a contiguous [tokens, top_k] tensor");
    const int64_t tokens = choice.size(0), top_k = choice.size(1), n = tokens * top_k;
    const int32_t experts = int32_of(a[1], "num_experts");
    if (top_k > INT32_MAX) value_error("too many choices");
    int32_t* status = status_word(c, a[2]);
    const at::TensorOptions ints = c.options(at::kInt);
    at::Tensor order = at::empty({n}, ints), position = at::empty({tokens, top_k}, ints);
    at::Tensor offsets = at::empty({std::max<int64_t>(experts, 0) + 1}, ints);
    const int64_t need = iq_expert_sort_workspace(n, experts);
    at::Tensor work;
    if (need) work = at::empty({need}, c.options(at::kByte));
    check(unlocked([&] {
        return iq_expert_sort(choice.data_ptr(), (int32_t)choice.element_size(), tokens,
                              (int32_t)top_k, experts, static_cast<int32_t*>(order.data_ptr()),
                              static_cast<int32_t*>(position.data_ptr()),
                              static_cast<int32_t*>(offsets.data_ptr()),
                              need ? work.data_ptr() : nullptr, need, status, c.stream);
    }), "iq_expert_sort");
    return tuple({order, position, offsets});
}

PyObject* expert_dispatch(PyObject* const* a)
{
    const Call c(a[0], "x");
    iq_dtype_t type;
    const Matrix x = values(c, a[0], "x", &type);
    const Routing r(c, a[1], a[2]);
    expect_rows(x, r.tokens, "x");
    const Result y(c, a[3], r.tokens * r.top_k, x.cols, x.t.scalar_type());
    check(unlocked([&] {
        return iq_expert_dispatch(type, x.data(), x.ld, r.tokens, x.cols, r.position,
                                  (int32_t)r.top_k, r.offsets, (int32_t)r.experts, y.data(), y.ld,
                                  c.stream);
    }), "iq_expert_dispatch");
    return y.object();
}

PyObject* expert_dispatch_backward(PyObject* const* a)
{
    const Call c(a[0], "grad");
    iq_dtype_t type;
    const Matrix g = values(c, a[0], "grad", &type);
    const Routing r(c, a[1], a[2]);
    expect_rows(g, r.tokens * r.top_k, "grad");
    const Result y(c, a[3], r.tokens, g.cols, g.t.scalar_type());
    check(unlocked([&] {
        return iq_expert_dispatch_backward(type, g.data(), g.ld, r.tokens, g.cols, r.position,
                                           (int32_t)r.top_k, r.offsets, (int32_t)r.experts,
                                           y.data(), y.ld, c.stream);
    }), "iq_expert_dispatch_backward");
    return y.object();
}

PyObject* expert_combine(PyObject* const* a)
{
    const Call c(a[0], "y");
    iq_dtype_t type;
    const Matrix y = values(c, a[0], "y", &type);
    const Routing r(c, a[1], a[2]);
    expect_rows(y, r.tokens * r.top_k, "y");
    const float* weights = array<float>(c, a[3], "weights", at::kFloat, {r.tokens, r.top_k});
    const Result out(c, a[4], r.tokens, y.cols, y.t.scalar_type());
    check(unlocked([&] {
        return iq_expert_combine(type, y.data(), y.ld, r.tokens, y.cols, r.position,
                                 (int32_t)r.top_k, r.offsets, (int32_t)r.experts, weights,
                                 out.data(), out.ld, c.stream);
    }), "iq_expert_combine");
    return out.object();
}

PyObject* expert_combine_backward(PyObject* const* a)
{
    const Call c(a[0], "grad");
    iq_dtype_t type;
    const Matrix y = values(c, a[1], "y", &type);
    const at::Tensor& grad = tensor(c, a[0], "grad");
    expect_type(grad, y.t.scalar_type(), "grad");
    const Matrix g(grad, "grad");
    const Routing r(c, a[2], a[3]);
    expect_rows(y, r.tokens * r.top_k, "y");
    expect_rows(g, r.tokens, "grad");
    if (g.cols != y.cols) value_error("grad must have " + std::to_string(y.cols) + " columns");
    const float* weights = array<float>(c, a[4], "weights", at::kFloat, {r.tokens, r.top_k});
    at::Tensor y_grad = at::empty({y.rows, y.cols}, c.options(y.t.scalar_type()));
    at::Tensor w_grad = at::empty({r.tokens, r.top_k}, c.options(at::kFloat));
    check(unlocked([&] {
        return iq_expert_combine_backward(type, g.data(), g.ld, y.data(), y.ld, r.tokens, y.cols,
                                          r.position, (int32_t)r.top_k, r.offsets,
                                          (int32_t)r.experts, weights, y_grad.data_ptr(), y.cols,
                                          static_cast<float*>(w_grad.data_ptr()), c.stream);
    }), "iq_expert_combine_backward");
    return tuple({y_grad, w_grad});
}

// --- the module ------------------------------------------------------------

PyObject* iq_error = nullptr;         // the package's exception class

// Whether autograd records what is done with these arguments, or carries a tangent of one
// of them along (forward mode, which torch.no_grad() does not turn off).  The functions of the
// graph have no rule for tangents, and raise.
bool recorded(PyObject* const* args, Py_ssize_t count)
{
    const bool graph = at::GradMode::is_enabled();
    const bool tangents = c10::AutogradState::get_tls_state().get_fw_grad_mode();
    if (!graph && !tangents) return false;
    for (Py_ssize_t i = 0; i < count; ++i) {
        if (!THPVariable_Check(args[i])) continue;
        const at::Tensor& t = THPVariable_Unpack(args[i]);
        if ((graph && t.requires_grad()) || (tangents && t._fw_grad(/*level=*/0).defined())) return true;
    }
    return false;
}

// kGraph: results can be part of a graph.  A call that autograd records answers
// NotImplemented, and layers.py makes it again from a function of the graph.
template <PyObject* (*kCall)(PyObject* const*), int kArgs, bool kGraph>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    if (count != kArgs) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kArgs, count);
        return nullptr;
    }
    if (kGraph && recorded(args, count)) Py_RETURN_NOTIMPLEMENTED;
    try {
        return kCall(args);
    } catch (const Refused& r) {
        PyErr_SetString(r.kind, r.text.c_str());
    } catch (const Failed& f) {
        PyObject* e = PyObject_CallFunction(iq_error, "is", (int)f.code, f.where);
        if (e) {
            PyErr_SetObject(iq_error, e);
            Py_DECREF(e);
        }
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type)
{
    Py_INCREF(type);
    Py_XSETREF(iq_error, type);
    Py_RETURN_NONE;
}

template <PyObject* (*kCall)(PyObject* const*), int kArgs, bool kGraph>
PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<kCall, kArgs, kGraph>)),
            METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<quantize_rows, 2, false>("quantize_rows"),
    method<int8_matmul, 6, true>("int8_matmul"),
    method<int8_linear, 5, true>("int8_linear"),
    method<int8_expert_matmul, 9, true>("int8_expert_matmul"),
    method<quantize_groups, 2, false>("quantize_groups"),
    method<dequantize_groups, 4, true>("dequantize_groups"),
    method<fp4_linear, 4, true>("fp4_linear"),
    method<fp4_expert_linear, 7, true>("fp4_expert_linear"),
    method<expert_gate, 4, true>("expert_gate"),
    method<expert_gate_backward, 5, true>("expert_gate_backward"),
    method<expert_balance, 3, true>("expert_balance"),
    method<expert_balance_backward, 4, true>("expert_balance_backward"),
    method<expert_sort, 3, false>("expert_sort"),
    method<expert_dispatch, 4, true>("expert_dispatch"),
    method<expert_dispatch_backward, 4, true>("expert_dispatch_backward"),
    method<expert_combine, 5, true>("expert_combine"),
    method<expert_combine_backward, 5, true>("expert_combine_backward"),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layers", nullptr, -1, methods, nullptr, nullptr,
                      nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layers() { return PyModule_Create(&module); }
