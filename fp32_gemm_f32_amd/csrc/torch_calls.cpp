// torch_calls.cpp -- the tensor layer's short way into the C ABI: a Python extension (module
// _torch_calls) that takes torch tensors, allocates outputs and workspace and launches, at
// about the cost of a torch operator. It serves the ordinary case only: plain tensors of the
// right types and shapes on one GPU, rows of unit stride, outputs of its own. For anything else
// (also for what has to be refused) it returns None, and the Python layer takes over with its
// checks, copies and messages.
//
// A call of quantize_rows on 4 x 256 takes the host 10.8 us through ctypes with torch.empty, most
// of it argument handling; small products and single rows take the GPU less than that.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gemm_i8.h"
#include "sgemm_dtype.h"
#include "sgemm_f32.h"
#include "token_logprobs.h"

namespace {

const at::Tensor *plain(PyObject *o)
{
    return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

int dtype_code(at::ScalarType t)
{
    return t == at::kFloat      ? SGEMM_DTYPE_F32
           : t == at::kBFloat16 ? SGEMM_DTYPE_BF16
           : t == at::kHalf     ? SGEMM_DTYPE_F16
                                : -1;
}
at::ScalarType scalar_type(int code)
{
    return code == SGEMM_DTYPE_F32 ? at::kFloat : code == SGEMM_DTYPE_BF16 ? at::kBFloat16 : at::kHalf;
}

// A matrix the kernels can read: rows of unit-stride elements that do not overlap, at most
// 2^31 - 1 of either.
struct Matrix {
    int rows = 0, cols = 0;
    int64_t ld = 1;
    bool ok = false;
    explicit Matrix(const at::Tensor &t)
    {
        if (t.dim() != 2 || !t.is_cuda() || t.is_neg()) return;
        const int64_t r = t.size(0), c = t.size(1);
        if (r > INT_MAX || c > INT_MAX) return;
        if ((c > 1 && t.stride(1) != 1) || (r > 1 && t.stride(0) < c)) return;
        rows = int(r);
        cols = int(c);
        ld = std::max<int64_t>(r > 1 ? t.stride(0) : c, 1);
        ok = true;
    }
};

bool vector(const at::Tensor &t, int64_t n, at::ScalarType type, const at::Device &device)
{
    return t.scalar_type() == type && t.dim() == 1 && t.size(0) == n && (n < 2 || t.stride(0) == 1) &&
           t.device() == device && !t.is_neg();
}

// An optional vector of floats: None, or as vector() wants it.
struct MaybeVector {
    const at::Tensor *t = nullptr;
    bool ok = true;
    MaybeVector(PyObject *o, int64_t n, const at::Device &device)
    {
        if (o == Py_None) return;
        t = plain(o);
        ok = t != nullptr && vector(*t, n, at::kFloat, device);
    }
    float *data() const { return t ? static_cast<float *>(t->data_ptr()) : nullptr; }
};

at::Tensor empty(at::IntArrayRef size, at::ScalarType type, const at::Device &device)
{
    return at::detail::empty_cuda(size, type, device, std::nullopt);
}

// The launch's device and stream, for the time of a call.
struct Place {
    c10::hip::HIPGuard guard;
    void *stream;
    explicit Place(const at::Device &d)
        : guard(d.index()), stream(c10::hip::getCurrentHIPStream(d.index()).stream())
    {
    }
};

PyObject *none() { Py_RETURN_NONE; }

// quantize_rows(X) -> (Q, scales) or None
PyObject *quantize_rows(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const at::Tensor *x = n == 1 ? plain(args[0]) : nullptr;
    if (!x) return none();
    const Matrix m(*x);
    const int code = dtype_code(x->scalar_type());
    if (!m.ok || code < 0) return none();
    at::Tensor q, scales;
    int status;
    {
        pybind11::gil_scoped_release release;
        const Place place(x->device());
        q = empty({m.rows, m.cols}, at::kChar, x->device());
        scales = empty({m.rows}, at::kFloat, x->device());
        status = gemm_i8_quantize_rows(m.rows, m.cols, x->data_ptr(), code, m.ld,
                                       static_cast<int8_t *>(q.data_ptr()), std::max(m.cols, 1),
                                       static_cast<float *>(scales.data_ptr()), place.stream);
    }
    if (status != SGEMM_OK) return none();
    return PyTuple_Pack(2, py::reinterpret_steal<py::object>(THPVariable_Wrap(q)).ptr(),
                        py::reinterpret_steal<py::object>(THPVariable_Wrap(scales)).ptr());
    END_HANDLE_TH_ERRORS
}

// matmul_i8(A, a_scales, B, b_scales, bias or None, type of C) -> C or None
PyObject *matmul_i8(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 6) return none();
    const at::Tensor *a = plain(args[0]), *sa = plain(args[1]), *b = plain(args[2]), *sb = plain(args[3]);
    if (!a || !sa || !b || !sb || a->scalar_type() != at::kChar || b->scalar_type() != at::kChar)
        return none();
    const at::Device device = a->device();
    const Matrix ma(*a), mb(*b);
    const int code = int(PyLong_AsLong(args[5]));
    if (!ma.ok || !mb.ok || ma.cols != mb.cols || b->device() != device || code < 0 || code > 2 ||
        !vector(*sa, ma.rows, at::kFloat, device) || !vector(*sb, mb.rows, at::kFloat, device))
        return none();
    const MaybeVector bias(args[4], mb.rows, device);
    if (!bias.ok) return none();
    at::Tensor c, space;
    int status;
    {
        pybind11::gil_scoped_release release;
        const Place place(device);
        const int8_t *pa = static_cast<const int8_t *>(a->data_ptr());
        const int8_t *pb = static_cast<const int8_t *>(b->data_ptr());
        c = empty({ma.rows, mb.rows}, scalar_type(code), device);
        const size_t bytes = gemm_i8_workspace_size(ma.rows, mb.rows, ma.cols, pa, ma.ld, pb, mb.ld);
        if (bytes) space = empty({int64_t(bytes)}, at::kByte, device);
        status = gemm_i8(ma.rows, mb.rows, ma.cols, pa, ma.ld, static_cast<const float *>(sa->data_ptr()),
                         pb, mb.ld, static_cast<const float *>(sb->data_ptr()), bias.data(), c.data_ptr(),
                         code, std::max(mb.rows, 1), bytes ? space.data_ptr() : nullptr, bytes,
                         place.stream);
    }
    return status == SGEMM_OK ? THPVariable_Wrap(c) : none();
    END_HANDLE_TH_ERRORS
}

// The rows' tokens, int64 or int32; 0 bytes if they are neither.
int token_bytes(const at::Tensor &t, int64_t n, const at::Device &device)
{
    return vector(t, n, at::kLong, device) ? 8 : vector(t, n, at::kInt, device) ? 4 : 0;
}

// token_logprobs(logits, tokens, top, low) -> (logprobs, entropy, lse, values, indices, lse_low) or
// None; the last three are None where top, and low, are 0
PyObject *token_logprobs_(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 4 || !PyLong_Check(args[2])) return none();
    const at::Tensor *x = plain(args[0]), *tokens = plain(args[1]);
    const bool low = args[3] == Py_True;
    if (!x || !tokens) return none();
    const Matrix m(*x);
    const int code = dtype_code(x->scalar_type());
    const at::Device device = x->device();
    const long top = PyLong_AsLong(args[2]);
    // (a forward-mode tangent would be lost: the Python layer refuses it)
    if (!m.ok || code < 0 || top < 0 || top > TOKEN_LOGPROBS_MAX_TOP || x->_fw_grad(0).defined()) {
        PyErr_Clear();
        return none();
    }
    const int bytes_each = token_bytes(*tokens, m.rows, device);
    if (!bytes_each) return none();
    at::Tensor out[6], space;
    int status;
    {
        pybind11::gil_scoped_release release;
        const Place place(device);
        for (int i = 0; i < 3; ++i) out[i] = empty({m.rows}, at::kFloat, device);
        if (top) {
            out[3] = empty({m.rows, top}, at::kFloat, device);
            out[4] = empty({m.rows, top}, at::kLong, device);
        }
        if (low) out[5] = empty({m.rows}, at::kFloat, device);
        const size_t bytes = token_logprobs_workspace_size(m.rows, m.cols, code, int(top));
        if (bytes) space = empty({int64_t(bytes)}, at::kByte, device);
        float *f[4] = {};
        for (int i = 0; i < (top ? 4 : 3); ++i) f[i] = static_cast<float *>(out[i].data_ptr());
        status = token_logprobs_low(m.rows, m.cols, x->data_ptr(), code, m.ld, tokens->data_ptr(), bytes_each,
                                    f[0], f[1], f[2], low ? static_cast<float *>(out[5].data_ptr()) : nullptr,
                                    int(top), f[3], top ? static_cast<int64_t *>(out[4].data_ptr()) : nullptr,
                                    bytes ? space.data_ptr() : nullptr, bytes, place.stream);
    }
    if (status != SGEMM_OK) return none();
    PyObject *r = PyTuple_New(6);
    if (!r) return nullptr;
    for (int i = 0; i < 6; ++i)
        PyTuple_SET_ITEM(r, i, out[i].defined() ? THPVariable_Wrap(out[i]) : Py_NewRef(Py_None));
    return r;
    END_HANDLE_TH_ERRORS
}

// token_logprobs_backward(logits, tokens, lse, entropy, g_logprobs, g_entropy, g_lse, lse_low) ->
// gradient or None; each of the last five may be None
PyObject *token_logprobs_backward_(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 8) return none();
    const at::Tensor *x = plain(args[0]), *tokens = plain(args[1]);
    if (!x || !tokens) return none();
    const Matrix m(*x);
    const int code = dtype_code(x->scalar_type());
    const at::Device device = x->device();
    if (!m.ok || code < 0) return none();
    const int bytes_each = token_bytes(*tokens, m.rows, device);
    const MaybeVector lse(args[2], m.rows, device), entropy(args[3], m.rows, device),
        g0(args[4], m.rows, device), g1(args[5], m.rows, device), g2(args[6], m.rows, device),
        low(args[7], m.rows, device);
    if (!bytes_each || !lse.ok || !lse.t || !entropy.ok || !g0.ok || !g1.ok || !g2.ok || !low.ok ||
        (g1.t && !entropy.t))
        return none();
    at::Tensor grad;
    int status;
    {
        pybind11::gil_scoped_release release;
        const Place place(device);
        grad = empty({m.rows, m.cols}, x->scalar_type(), device);
        status = token_logprobs_backward_low(m.rows, m.cols, x->data_ptr(), code, m.ld, tokens->data_ptr(),
                                             bytes_each, lse.data(), low.data(), entropy.data(), g0.data(),
                                             g1.data(), g2.data(), grad.data_ptr(), std::max(m.cols, 1),
                                             place.stream);
    }
    return status == SGEMM_OK ? THPVariable_Wrap(grad) : none();
    END_HANDLE_TH_ERRORS
}

template <typename F> PyCFunction fast(F *f)
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef kMethods[] = {
    {"quantize_rows", fast(&quantize_rows), METH_FASTCALL, nullptr},
    {"matmul_i8", fast(&matmul_i8), METH_FASTCALL, nullptr},
    {"token_logprobs", fast(&token_logprobs_), METH_FASTCALL, nullptr},
    {"token_logprobs_backward", fast(&token_logprobs_backward_), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&kModule); }
