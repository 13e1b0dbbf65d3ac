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
#include <c10/core/GradMode.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "beam_search.h"
#include "gemm_i8.h"
#include "gemm_mx4.h"
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

// (a forward-mode tangent would be lost: the Python layer refuses it)
bool dual(const at::Tensor *t) { return t && t->_fw_grad(0).defined(); }

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
    if (!m.ok || code < 0 || top < 0 || top > TOKEN_LOGPROBS_MAX_TOP || dual(x)) {
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

// ---- 4-bit operands

// Rows of bytes as the Python layer's _padded allocates them: their distance.
int64_t padded(int64_t rows, int64_t cols) { return cols % 4 == 0 || rows < 2 ? std::max<int64_t>(cols, 1) : (cols + 15) / 16 * 16; }
at::Tensor empty_padded(int64_t rows, int64_t cols, const at::Device &device)
{
    const int64_t ld = padded(rows, cols);
    if (ld == cols || cols == 0) return empty({rows, cols}, at::kByte, device);
    return empty({rows, ld}, at::kByte, device).narrow(1, 0, cols);
}

// A packed matrix with its scales.
struct Packed {
    Matrix q, s;
    const uint8_t *data = nullptr, *scales = nullptr;
    bool ok;
    Packed(const at::Tensor &t, const at::Tensor &u) : q(t), s(u)
    {
        ok = q.ok && s.ok && t.scalar_type() == at::kByte && u.scalar_type() == at::kByte &&
             t.device() == u.device() && s.rows == q.rows && s.cols == (int64_t(q.cols) + 15) / 16 &&
             q.cols <= INT_MAX / 2;
        if (!ok) return;
        data = static_cast<const uint8_t *>(t.data_ptr());
        scales = static_cast<const uint8_t *>(u.data_ptr());
    }
};

int quantize_into(const at::Tensor &x, const Matrix &m, int code, const at::Tensor &q, const at::Tensor &scales,
                  void *stream)
{
    return gemm_mx4_quantize(m.rows, m.cols, x.data_ptr(), code, m.ld, static_cast<uint8_t *>(q.data_ptr()),
                             padded(m.rows, q.size(1)), static_cast<uint8_t *>(scales.data_ptr()),
                             padded(m.rows, scales.size(1)), stream);
}
int64_t packed_columns(int64_t k) { return (k + 1) / 2; }
int64_t packed_blocks(int64_t k) { return (k + 31) / 32; }

// quantize_mx4(X) -> (Q, scales) or None
PyObject *quantize_mx4(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const at::Tensor *x = n == 1 ? plain(args[0]) : nullptr;
    if (!x) return none();
    const Matrix m(*x);
    const int code = dtype_code(x->scalar_type());
    if (!m.ok || code < 0 || dual(x)) return none();
    at::Tensor q, scales;
    int status;
    {
        pybind11::gil_scoped_release release;
        const Place place(x->device());
        q = empty_padded(m.rows, packed_columns(m.cols), x->device());
        scales = empty_padded(m.rows, packed_blocks(m.cols), x->device());
        status = quantize_into(*x, m, code, q, scales, place.stream);
    }
    if (status != SGEMM_OK) return none();
    return PyTuple_Pack(2, py::reinterpret_steal<py::object>(THPVariable_Wrap(q)).ptr(),
                        py::reinterpret_steal<py::object>(THPVariable_Wrap(scales)).ptr());
    END_HANDLE_TH_ERRORS
}

// dequantize_mx4(Q, scales, type, columns or None) -> values or None
PyObject *dequantize_mx4(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 4 || !PyLong_CheckExact(args[2]) || (args[3] != Py_None && !PyLong_CheckExact(args[3]))) return none();
    const at::Tensor *q = plain(args[0]), *scales = plain(args[1]);
    if (!q || !scales) return none();
    const Packed p(*q, *scales);
    const int code = int(PyLong_AsLong(args[2]));
    const long columns = args[3] == Py_None ? 2L * p.q.cols : PyLong_AsLong(args[3]);
    if (PyErr_Occurred()) PyErr_Clear();
    if (!p.ok || code < 0 || code > 2) return none();
    if (columns < 0 || packed_columns(columns) != p.q.cols) return none();
    at::Tensor y;
    int status;
    {
        pybind11::gil_scoped_release release;
        const Place place(q->device());
        y = empty({p.q.rows, columns}, scalar_type(code), q->device());
        status = gemm_mx4_dequantize(p.q.rows, int(columns), p.data, p.q.ld, p.scales, p.s.ld, y.data_ptr(), code,
                                     std::max<int64_t>(columns, 1), place.stream);
    }
    return status == SGEMM_OK ? THPVariable_Wrap(y) : none();
    END_HANDLE_TH_ERRORS
}

// The product of packed A (given by its parts) and B into a new tensor.
int product_mx4(const uint8_t *a, int64_t lda, const uint8_t *sa, int64_t ldsa, int M, const Packed &b, int K,
                const MaybeVector &bias, int code, const at::Device &device, void *stream, at::Tensor &c)
{
    at::Tensor space;
    c = empty({M, b.q.rows}, scalar_type(code), device);
    const size_t bytes = gemm_mx4_workspace_size(M, b.q.rows, K, a, lda, sa, ldsa, b.data, b.q.ld, b.scales, b.s.ld);
    if (bytes) space = empty({int64_t(bytes)}, at::kByte, device);
    return gemm_mx4(M, b.q.rows, K, a, lda, sa, ldsa, b.data, b.q.ld, b.scales, b.s.ld, bias.data(), c.data_ptr(),
                    code, std::max(b.q.rows, 1), bytes ? space.data_ptr() : nullptr, bytes, stream);
}

// matmul_mx4(A, a_scales, B, b_scales, bias or None, type of C) -> C or None
PyObject *matmul_mx4(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 6) return none();
    const at::Tensor *a = plain(args[0]), *sa = plain(args[1]), *b = plain(args[2]), *sb = plain(args[3]);
    if (!a || !sa || !b || !sb) return none();
    const at::Device device = a->device();
    const Packed pa(*a, *sa), pb(*b, *sb);
    const int code = int(PyLong_AsLong(args[5]));
    if (!pa.ok || !pb.ok || pa.q.cols != pb.q.cols || b->device() != device || code < 0 || code > 2) return none();
    const MaybeVector bias(args[4], pb.q.rows, device);
    if (!bias.ok || dual(bias.t)) return none();
    at::Tensor c;
    int status;
    {
        pybind11::gil_scoped_release release;
        const Place place(device);
        status = product_mx4(pa.data, pa.q.ld, pa.scales, pa.s.ld, pa.q.rows, pb, 2 * pa.q.cols, bias, code, device,
                             place.stream, c);
    }
    return status == SGEMM_OK ? THPVariable_Wrap(c) : none();
    END_HANDLE_TH_ERRORS
}

// linear_mx4(X, B, b_scales, bias or None, type of C or -1) -> C or None
PyObject *linear_mx4(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 5) return none();
    const at::Tensor *x = plain(args[0]), *b = plain(args[1]), *sb = plain(args[2]);
    if (!x || !b || !sb) return none();
    const at::Device device = x->device();
    const Matrix m(*x);
    const Packed pb(*b, *sb);
    const int type = dtype_code(x->scalar_type());
    int code = int(PyLong_AsLong(args[4]));
    if (code == -1) code = type;
    if (!m.ok || !pb.ok || type < 0 || code < 0 || code > 2 || b->device() != device ||
        pb.q.cols != packed_columns(m.cols))
        return none();
    const MaybeVector bias(args[3], pb.q.rows, device);
    if (!bias.ok || dual(bias.t) || dual(x)) return none();
    at::Tensor q, scales, c;
    int status;
    {
        pybind11::gil_scoped_release release;
        const Place place(device);
        q = empty_padded(m.rows, pb.q.cols, device);
        scales = empty_padded(m.rows, pb.s.cols, device);
        status = quantize_into(*x, m, type, q, scales, place.stream);
        if (status == SGEMM_OK)
            status = product_mx4(static_cast<const uint8_t *>(q.data_ptr()), padded(m.rows, pb.q.cols),
                                 static_cast<const uint8_t *>(scales.data_ptr()), padded(m.rows, pb.s.cols), m.rows,
                                 pb, 2 * pb.q.cols, bias, code, device, place.stream, c);
    }
    return status == SGEMM_OK ? THPVariable_Wrap(c) : none();
    END_HANDLE_TH_ERRORS
}

// ---- beam search

// beam_step(logits, scores, top or None, finished or None, pad_token) -> (scores, beams, tokens) or None
PyObject *beam_step_(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 5 || (args[2] != Py_None && !PyLong_CheckExact(args[2])) || !PyLong_CheckExact(args[4])) return none();
    const at::Tensor *x = plain(args[0]), *scores = plain(args[1]);
    const at::Tensor *finished = args[3] == Py_None ? nullptr : plain(args[3]);
    if (!x || !scores || (args[3] != Py_None && !finished)) return none();
    const Matrix m(*x);
    const int code = dtype_code(x->scalar_type());
    const at::Device device = x->device();
    const auto per_beam = [&](const at::Tensor &t, at::ScalarType type) {
        return t.scalar_type() == type && t.dim() == 2 && t.is_contiguous() && t.device() == device && !t.is_neg() &&
               t.size(0) <= INT_MAX && t.size(1) <= BEAM_MAX;
    };
    long top = args[2] == Py_None ? 0 : PyLong_AsLong(args[2]);
    const long long pad_token = PyLong_AsLongLong(args[4]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return none();
    }
    if (!m.ok || code < 0 || !per_beam(*scores, at::kFloat) || dual(x) || dual(scores)) return none();
    const int64_t B = scores->size(0), W = scores->size(1);
    if (finished && (!per_beam(*finished, at::kBool) || finished->size(0) != B || finished->size(1) != W))
        return none();
    if (args[2] == Py_None) top = W;
    if (m.rows != B * W || W < 1 || top < 1 || top > BEAM_MAX) return none();
    at::Tensor out[3], space;
    int status;
    {
        pybind11::gil_scoped_release release;
        const Place place(device);
        out[0] = empty({B, top}, at::kFloat, device);
        out[1] = empty({B, top}, at::kLong, device);
        out[2] = empty({B, top}, at::kLong, device);
        const size_t bytes = beam_step_workspace_size(int(B), int(W), m.cols, code, int(top));
        if (bytes) space = empty({int64_t(bytes)}, at::kByte, device);
        status = beam_step(int(B), int(W), m.cols, x->data_ptr(), code, m.ld,
                           static_cast<const float *>(scores->data_ptr()),
                           finished ? static_cast<const uint8_t *>(finished->data_ptr()) : nullptr, pad_token, int(top),
                           static_cast<float *>(out[0].data_ptr()), static_cast<int64_t *>(out[1].data_ptr()),
                           static_cast<int64_t *>(out[2].data_ptr()), bytes ? space.data_ptr() : nullptr, bytes,
                           place.stream);
    }
    if (status != SGEMM_OK) return none();
    return PyTuple_Pack(3, py::reinterpret_steal<py::object>(THPVariable_Wrap(out[0])).ptr(),
                        py::reinterpret_steal<py::object>(THPVariable_Wrap(out[1])).ptr(),
                        py::reinterpret_steal<py::object>(THPVariable_Wrap(out[2])).ptr());
    END_HANDLE_TH_ERRORS
}

// beam_state's fields for two tensors of one shape; false where they have more than two dimensions of
// pieces.
bool state_of(const at::Tensor &src, const at::Tensor &dst, beam_state &s)
{
    const int64_t size = int64_t(src.element_size());
    struct Dim { int64_t n, src, dst; } dims[3];
    int count = 0;
    for (int64_t d = 1; d < src.dim(); ++d) {
        const int64_t n = src.size(d), a = src.stride(d) * size, b = dst.stride(d) * size;
        if (n == 1) continue;
        if (count > 0 && dims[count - 1].src == n * a && dims[count - 1].dst == n * b) {
            dims[count - 1] = {dims[count - 1].n * n, a, b};
        } else {
            if (count == 3) return false;
            dims[count++] = {n, a, b};
        }
    }
    s.run = size;
    if (count > 0 && dims[count - 1].src == size && dims[count - 1].dst == size) s.run *= dims[--count].n;
    if (count > 2) return false;
    const Dim none = {1, 0, 0};
    const Dim d1 = count == 2 ? dims[0] : none, d2 = count > 0 ? dims[count - 1] : none;
    s.src = src.data_ptr();
    s.dst = dst.data_ptr();
    s.src_row = src.size(0) > 1 ? src.stride(0) * size : 0;
    s.dst_row = src.size(0) > 1 ? dst.stride(0) * size : 0;
    s.count1 = d1.n; s.src_step1 = d1.src; s.dst_step1 = d1.dst;
    s.count2 = d2.n; s.src_step2 = d2.src; s.dst_step2 = d2.dst;
    return true;
}

// New tensors like the given ones. Small ones share an allocation (each of its own takes the host 0.5 us:
// 18 of 4 rows 16 us in all, the GPU 7), large ones have their own.
constexpr int64_t kShared = int64_t(64) << 20, kApart = 512;
std::vector<at::Tensor> empty_like_all(const std::vector<at::Tensor> &like, const at::Device &device)
{
    const auto room = [](const at::Tensor &t) {
        return (t.numel() * int64_t(t.element_size()) + kApart - 1) / kApart * kApart;
    };
    int64_t all = 0;
    for (const at::Tensor &t : like) all += room(t);
    std::vector<at::Tensor> out;
    out.reserve(like.size());
    if (all > kShared || like.size() < 2) {
        for (const at::Tensor &t : like) out.push_back(empty(t.sizes(), t.scalar_type(), device));
        return out;
    }
    const at::Tensor space = empty({all}, at::kByte, device);
    int64_t at_byte = 0;
    c10::SmallVector<int64_t, 8> strides;
    for (const at::Tensor &t : like) {
        strides.resize(size_t(t.dim()));
        int64_t step = 1;
        for (int64_t d = t.dim() - 1; d >= 0; --d) {
            strides[size_t(d)] = step;
            step *= std::max<int64_t>(t.size(d), 1);
        }
        at::Tensor o = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(space.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                                t.dtype());
        o.unsafeGetTensorImpl()->set_sizes_and_strides(t.sizes(), strides, at_byte / int64_t(t.element_size()));
        out.push_back(std::move(o));
        at_byte += room(t);
    }
    return out;
}

// reorder_beams(states, beams, out or None) -> out, or None: sequences of tensors only
PyObject *reorder_beams_(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 3) return none();
    const at::Tensor *beams = plain(args[1]);
    const auto listed = [](PyObject *o) { return PyList_CheckExact(o) || PyTuple_CheckExact(o); };
    if (!beams || !listed(args[0]) || (args[2] != Py_None && !listed(args[2]))) return none();
    if (beams->dim() != 2 || !beams->is_contiguous() || !beams->is_cuda() || beams->is_neg() ||
        beams->size(0) > INT_MAX || beams->size(1) > BEAM_MAX ||
        (beams->scalar_type() != at::kLong && beams->scalar_type() != at::kInt))
        return none();
    const at::Device device = beams->device();
    const int64_t rows = beams->size(0) * beams->size(1);
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(args[0]);
    const bool given = args[2] != Py_None;
    if (given && PySequence_Fast_GET_SIZE(args[2]) != count) return none();
    std::vector<at::Tensor> src, dst;
    std::vector<beam_state> states;
    src.reserve(size_t(count));
    dst.reserve(size_t(count));
    states.reserve(size_t(count));
    for (Py_ssize_t i = 0; i < count; ++i) {
        const at::Tensor *t = plain(PySequence_Fast_GET_ITEM(args[0], i));
        if (!t || t->device() != device || t->layout() != at::kStrided || t->dim() < 1 || t->size(0) != rows ||
            t->is_neg() || t->is_conj() || dual(t))
            return none();
        src.push_back(*t);
        if (!given) continue;
        const at::Tensor *o = plain(PySequence_Fast_GET_ITEM(args[2], i));
        if (!o || o->device() != device || o->layout() != at::kStrided || o->scalar_type() != t->scalar_type() ||
            o->sizes() != t->sizes() || o->is_neg() || o->is_conj() ||
            dual(o) || (o->requires_grad() && c10::GradMode::is_enabled()))
            return none();
        dst.push_back(*o);
    }
    int status;
    bool fits = true;
    {
        pybind11::gil_scoped_release release;
        const Place place(device);
        if (!given) dst = empty_like_all(src, device);
        for (Py_ssize_t i = 0; i < count; ++i) {
            beam_state s;
            if (src[i].numel() == 0) continue;
            if (!state_of(src[i], dst[i], s)) { fits = false; break; }
            states.push_back(s);
        }
        status = !fits ? int(SGEMM_EINVAL_DIM) : reorder_beams(int(beams->size(0)), int(beams->size(1)), beams->data_ptr(), int(beams->element_size()),
                               states.data(), int(states.size()), place.stream);
    }
    if (status != SGEMM_OK) return none();
    // (autograd refuses to use a saved tensor of another version)
    if (given)
        for (const at::Tensor &t : dst)
            if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    PyObject *r = PyList_New(count);
    if (!r) return nullptr;
    // (of given ones the objects that they have: the caller's list may be another one by now, for other
    // threads ran meanwhile)
    for (Py_ssize_t i = 0; i < count; ++i) PyList_SET_ITEM(r, i, THPVariable_Wrap(dst[size_t(i)]));
    return r;
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
    {"quantize_mx4", fast(&quantize_mx4), METH_FASTCALL, nullptr},
    {"dequantize_mx4", fast(&dequantize_mx4), METH_FASTCALL, nullptr},
    {"matmul_mx4", fast(&matmul_mx4), METH_FASTCALL, nullptr},
    {"linear_mx4", fast(&linear_mx4), METH_FASTCALL, nullptr},
    {"beam_step", fast(&beam_step_), METH_FASTCALL, nullptr},
    {"reorder_beams", fast(&reorder_beams_), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&kModule); }
