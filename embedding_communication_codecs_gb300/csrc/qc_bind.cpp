// qc_bind.cpp -- the 8-bit layer's calls on torch tensors, without Python between the
// tensors and the C ABI.
//
// Each function takes plainly right arguments (dense tensors of the expected types and
// shapes, all on one CUDA device), allocates the results and the workspace, and makes
// the C call with that device current, on that device's current stream.  It returns the results; None
// where an argument is anything else, for the caller to look closer; or the C call's
// status where that is not QC_OK.  A call of a few microseconds on the GPU costs the
// host about as much: through Python attributes and ctypes, a one-token product took
// 12.6 us to issue, of which the C call is 3.1.
#include <ATen/ATen.h>
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/qcodec.h"

namespace {

const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool dense(const at::Tensor &t, at::ScalarType type, int64_t dims) {
    return t.is_cuda() && t.dim() == dims && t.scalar_type() == type && t.is_contiguous();
}

// A dense fp32 or bf16 matrix.
bool rows(const at::Tensor *t) {
    return t && (dense(*t, at::kBFloat16, 2) || dense(*t, at::kFloat, 2));
}

// Two tensors on the same device.
bool together(const at::Tensor &a, const at::Tensor &b) { return a.device() == b.device(); }

// Row codes and their scales.
bool codes(const at::Tensor *c, const at::Tensor *s) {
    return c && s && dense(*c, at::kChar, 2) && dense(*s, at::kFloat, 1) && s->size(0) == c->size(0) && together(*c, *s);
}

qc_dtype type_of(const at::Tensor &t) { return t.scalar_type() == at::kFloat ? QC_DTYPE_F32 : QC_DTYPE_BF16; }

at::Tensor make(const at::Tensor &like, at::IntArrayRef shape, at::ScalarType type) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}

at::Tensor results(const at::Tensor &like, at::IntArrayRef shape, bool bf16) {
    return make(like, shape, bf16 ? at::kBFloat16 : at::kFloat);
}

qc_stream_t stream_of(const at::Tensor &t) {
    return reinterpret_cast<qc_stream_t>(c10::cuda::getCurrentCUDAStream(t.device().index()).stream());
}

PyObject *none() { Py_RETURN_NONE; }

PyObject *answer(qc_status st, const at::Tensor &result) {
    return st == QC_OK ? THPVariable_Wrap(result) : PyLong_FromLong(st);
}

// New references for PyTuple_Pack(), which takes its own.
struct Wrapped {
    PyObject *o;
    explicit Wrapped(at::Tensor t) : o(THPVariable_Wrap(std::move(t))) {}
    ~Wrapped() { Py_XDECREF(o); }
};

#define QC_GUARD_BEGIN try {
#define QC_GUARD_END                                             \
    }                                                            \
    catch (const std::exception &e) {                            \
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what()); \
        return nullptr;                                          \
    }

PyObject *rowwise_int8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    QC_GUARD_BEGIN
    const at::Tensor *x = n == 1 ? tensor(a[0]) : nullptr;
    if (!rows(x)) return none();
    const int64_t r = x->size(0), d = x->size(1);
    const c10::cuda::CUDAGuard current(x->device());
    const at::Tensor c = make(*x, {r, d}, at::kChar), s = make(*x, {r}, at::kFloat);
    const qc_status st = qc_rowwise_int8(x->data_ptr(), type_of(*x), d, r, d, c.data_ptr<int8_t>(), s.data_ptr<float>(), stream_of(*x));
    if (st != QC_OK) return PyLong_FromLong(st);
    const Wrapped wc(c), ws(s);
    return PyTuple_Pack(2, wc.o, ws.o);
    QC_GUARD_END
}

PyObject *rowwise_int8_dequant(PyObject *, PyObject *const *a, Py_ssize_t n) {
    QC_GUARD_BEGIN
    const at::Tensor *c = n == 3 ? tensor(a[0]) : nullptr, *s = n == 3 ? tensor(a[1]) : nullptr;
    if (!codes(c, s)) return none();
    const bool bf16 = a[2] == Py_True;
    const int64_t r = c->size(0), d = c->size(1);
    const c10::cuda::CUDAGuard current(c->device());
    const at::Tensor out = results(*c, {r, d}, bf16);
    return answer(qc_rowwise_int8_dequant(c->data_ptr<int8_t>(), s->data_ptr<float>(), r, d, out.data_ptr(),
                                          bf16 ? QC_DTYPE_BF16 : QC_DTYPE_F32, d, stream_of(*c)), out);
    QC_GUARD_END
}

// Scratch memory of a call, or none.
struct Workspace {
    at::Tensor t;
    size_t bytes;
    Workspace(const at::Tensor &like, size_t n) : bytes(n) {
        if (n) t = make(like, {static_cast<int64_t>(n)}, at::kByte);
    }
    void *p() const { return bytes ? t.data_ptr() : nullptr; }
};

PyObject *int8_matmul(PyObject *, PyObject *const *a, Py_ssize_t n) {
    QC_GUARD_BEGIN
    if (n != 6) return none();
    const at::Tensor *xc = tensor(a[0]), *xs = tensor(a[1]), *wc = tensor(a[2]), *ws = tensor(a[3]);
    const at::Tensor *bias = a[4] == Py_None ? nullptr : tensor(a[4]);
    if (!codes(xc, xs) || !codes(wc, ws) || xc->size(1) != wc->size(1) || !together(*xc, *wc)) return none();
    const int64_t T = xc->size(0), N = wc->size(0), K = xc->size(1);
    if (a[4] != Py_None && !(bias && dense(*bias, at::kFloat, 1) && bias->size(0) == N && together(*xc, *bias))) return none();
    const bool bf16 = a[5] == Py_True;
    const c10::cuda::CUDAGuard current(xc->device());
    const at::Tensor y = results(*xc, {T, N}, bf16);
    const Workspace w(*xc, qc_int8_matmul_codes_workspace(xc->data_ptr<int8_t>(), wc->data_ptr<int8_t>(), T, N, K));
    return answer(qc_int8_matmul(xc->data_ptr<int8_t>(), xs->data_ptr<float>(), wc->data_ptr<int8_t>(), ws->data_ptr<float>(),
                                 bias ? bias->data_ptr<float>() : nullptr, T, N, K, y.data_ptr(),
                                 bf16 ? QC_DTYPE_BF16 : QC_DTYPE_F32, N, w.p(), w.bytes, stream_of(*xc)), y);
    QC_GUARD_END
}

PyObject *int8_input_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
    QC_GUARD_BEGIN
    if (n != 4) return none();
    const at::Tensor *dy = tensor(a[0]), *wc = tensor(a[1]), *ws = tensor(a[2]);
    if (!dy || !dense(*dy, at::kBFloat16, 2) || !codes(wc, ws) || dy->size(1) != wc->size(0) || !together(*dy, *wc)) return none();
    const int64_t T = dy->size(0), N = wc->size(0), K = wc->size(1);
    const bool bf16 = a[3] == Py_True;
    const c10::cuda::CUDAGuard current(dy->device());
    const at::Tensor dx = results(*dy, {T, K}, bf16);
    const Workspace w(*dy, qc_int8_input_grad_workspace(T, N, K));
    return answer(qc_int8_input_grad(dy->data_ptr(), N, wc->data_ptr<int8_t>(), ws->data_ptr<float>(), T, N, K, dx.data_ptr(),
                                     bf16 ? QC_DTYPE_BF16 : QC_DTYPE_F32, K, w.p(), w.bytes, stream_of(*dy)), dx);
    QC_GUARD_END
}

PyObject *int8_weight_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
    QC_GUARD_BEGIN
    if (n != 5) return none();
    const at::Tensor *dy = tensor(a[0]), *xc = tensor(a[1]), *xs = tensor(a[2]);
    if (!dy || !dense(*dy, at::kBFloat16, 2) || !codes(xc, xs) || dy->size(0) != xc->size(0) || !together(*dy, *xc)) return none();
    const int64_t T = dy->size(0), N = dy->size(1), K = xc->size(1);
    const bool bf16 = a[3] == Py_True, with_bias = a[4] == Py_True;
    const c10::cuda::CUDAGuard current(dy->device());
    const at::Tensor dw = results(*dy, {N, K}, bf16), db = with_bias ? make(*dy, {N}, at::kFloat) : at::Tensor();
    const Workspace w(*dy, qc_int8_weight_grad_workspace(T, N, K));
    const qc_status st = qc_int8_weight_grad(dy->data_ptr(), N, xc->data_ptr<int8_t>(), xs->data_ptr<float>(), T, N, K,
                                             dw.data_ptr(), bf16 ? QC_DTYPE_BF16 : QC_DTYPE_F32,
                                             with_bias ? db.data_ptr<float>() : nullptr, 0, w.p(), w.bytes, stream_of(*dy));
    if (st != QC_OK) return PyLong_FromLong(st);
    const Wrapped wd(dw);
    if (!with_bias) return PyTuple_Pack(2, wd.o, Py_None);
    const Wrapped wb(db);
    return PyTuple_Pack(2, wd.o, wb.o);
    QC_GUARD_END
}

PyObject *swiglu_encode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    QC_GUARD_BEGIN
    const at::Tensor *x = n == 1 ? tensor(a[0]) : nullptr;
    if (!rows(x) || x->size(1) % 2) return none();
    const int64_t r = x->size(0), two = x->size(1), d = two / 2;
    const c10::cuda::CUDAGuard current(x->device());
    const at::Tensor hc = make(*x, {r, d}, at::kChar), hs = make(*x, {r}, at::kFloat), sc = make(*x, {r, two}, at::kChar),
                     ss = make(*x, {r, 2}, at::kFloat);
    const qc_status st = qc_swiglu_encode(x->data_ptr(), type_of(*x), two, r, d, hc.data_ptr<int8_t>(), hs.data_ptr<float>(),
                                          sc.data_ptr<int8_t>(), ss.data_ptr<float>(), stream_of(*x));
    if (st != QC_OK) return PyLong_FromLong(st);
    const Wrapped a0(hc), a1(hs), a2(sc), a3(ss);
    return PyTuple_Pack(4, a0.o, a1.o, a2.o, a3.o);
    QC_GUARD_END
}

PyObject *swiglu_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    QC_GUARD_BEGIN
    if (n != 3) return none();
    const at::Tensor *dh = tensor(a[0]), *sc = tensor(a[1]), *ss = tensor(a[2]);
    if (!rows(dh) || !sc || !ss || !dense(*sc, at::kChar, 2) || !dense(*ss, at::kFloat, 2)) return none();
    const int64_t r = dh->size(0), d = dh->size(1);
    if (sc->size(0) != r || sc->size(1) != 2 * d || ss->size(0) != r || ss->size(1) != 2) return none();
    if (!together(*dh, *sc) || !together(*dh, *ss)) return none();
    const c10::cuda::CUDAGuard current(dh->device());
    const at::Tensor out = make(*dh, {r, 2 * d}, dh->scalar_type());
    return answer(qc_swiglu_backward(dh->data_ptr(), type_of(*dh), d, sc->data_ptr<int8_t>(), ss->data_ptr<float>(), r, d,
                                     out.data_ptr(), 2 * d, stream_of(*dh)), out);
    QC_GUARD_END
}

#define QC_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {QC_METHOD(rowwise_int8),     QC_METHOD(rowwise_int8_dequant), QC_METHOD(int8_matmul),
                         QC_METHOD(int8_input_grad),  QC_METHOD(int8_weight_grad),     QC_METHOD(swiglu_encode),
                         QC_METHOD(swiglu_backward),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qcbind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qcbind() { return PyModule_Create(&module); }
