// Python module linear_layer_amd._call: the argument handling of the 4-bit
// products' and the residual norms' calls, which in Python takes longer than
// their small kernels run. Each function takes the tensors and numbers of the
// Python function of the same name, enqueues on the current stream of the
// tensors' device and returns the status of the C call, or None, with nothing
// enqueued, where an argument is not what the call takes: the Python function
// then finds and reports what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include "linear_layer.h"

namespace {

PyObject *g_current_device, *g_raw_stream;   // torch's getters, set by setup()

// What a call needs of its arguments so far.
struct Args {
    int device = -1;
    bool ok = true;

    const at::Tensor *tensor(PyObject *o)
    {
        if (!ok || !THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        const at::Tensor &t = THPVariable_Unpack(o);
        const int d = t.is_cuda() ? (int)t.get_device() : -1;
        if (device < 0)
            device = d;
        if (d < 0 || d != device) {
            ok = false;
            return nullptr;
        }
        return &t;
    }
    double number(PyObject *o)
    {
        const double v = ok ? PyFloat_AsDouble(o) : 0.0;
        if (ok && v == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return v;
    }
    // The current stream of the tensors' device, which has to be the current one.
    void *stream()
    {
        if (!ok || device < 0)
            return fail();
        PyObject *d = PyObject_CallNoArgs(g_current_device);
        const long now = d != nullptr ? PyLong_AsLong(d) : -1;
        Py_XDECREF(d);
        if (now != device || PyErr_Occurred())
            return fail();
        PyObject *index = PyLong_FromLong(now);
        PyObject *raw = index != nullptr ? PyObject_CallOneArg(g_raw_stream, index) : nullptr;
        Py_XDECREF(index);
        void *s = raw != nullptr ? PyLong_AsVoidPtr(raw) : nullptr;
        Py_XDECREF(raw);
        if (PyErr_Occurred())
            return fail();
        return s;
    }
    void *fail()
    {
        PyErr_Clear();
        ok = false;
        return nullptr;
    }
};

// A 2-D row-major matrix; rows, cols < 0 take the tensor's, else they have to match.
struct Mat {
    void *p = nullptr;
    int rows = 0, cols = 0, ld = 1;

    Mat() = default;
    Mat(Args &a, PyObject *o, at::ScalarType type, int64_t r = -1, int64_t c = -1, bool optional = false)
    {
        if (optional && o == Py_None) {
            ld = c > 1 ? (int)c : 1;
            return;
        }
        const at::Tensor *t = a.tensor(o);
        if (t == nullptr || t->scalar_type() != type || t->dim() != 2) {
            a.ok = false;
            return;
        }
        const int64_t m = t->size(0), n = t->size(1), step = t->stride(1), s = m > 1 ? t->stride(0) : n;
        if ((r >= 0 && m != r) || (c >= 0 && n != c) || (n > 1 && step != 1) || s < n || m > INT32_MAX || s > INT32_MAX) {
            a.ok = false;
            return;
        }
        p = t->data_ptr();
        rows = (int)m;
        cols = (int)n;
        ld = s > 1 ? (int)s : 1;
    }
};

// The type of a tensor of 32- or 16-bit floats as LL_TYPE_*.
int element_type(Args &a, PyObject *o, at::ScalarType &type)
{
    const at::Tensor *t = a.tensor(o);
    if (t == nullptr)
        return -1;
    type = t->scalar_type();
    if (type == at::kFloat)
        return LL_TYPE_F32;
    if (type == at::kHalf)
        return LL_TYPE_F16;
    if (type == at::kBFloat16)
        return LL_TYPE_BF16;
    a.ok = false;
    return -1;
}

// N contiguous fp32 values, or null for None.
float *vec(Args &a, PyObject *o, int64_t n)
{
    if (o == Py_None)
        return nullptr;
    const at::Tensor *t = a.tensor(o);
    if (t == nullptr || t->scalar_type() != at::kFloat || t->dim() != 1 || t->size(0) != n || (n > 1 && t->stride(0) != 1)) {
        a.ok = false;
        return nullptr;
    }
    return static_cast<float *>(t->data_ptr());
}

int64_t code_bytes(int64_t K) { return (K + 1) / 2; }
int64_t scale_bytes(int64_t K) { return (K + 31) / 32; }

// The workspace a product gains from, if any: memory of torch's allocator, in the
// order of the current stream, so that it may be given back at once.
at::Tensor scratch(const Args &a, PyObject *like, const Mat &A, const Mat &B, int64_t K, int form)
{
    const int64_t bytes = a.ok && A.rows > 0 && B.rows > 0 ? ll_mx4_workspace_size(A.rows, B.rows, (int)K, form) : 0;
    return bytes > 0 ? at::empty({bytes}, THPVariable_Unpack(like).options().dtype(at::kByte)) : at::Tensor();
}

template <class F>
PyObject *enqueue(const Args &a, F call)
{
    if (!a.ok)
        Py_RETURN_NONE;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = call();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

// A function of `n` arguments that lets no C++ exception out.
template <Py_ssize_t N, PyObject *(*F)(PyObject *const *)>
PyObject *guarded(PyObject *, PyObject *const *x, Py_ssize_t n)
{
    if (n != N) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return F(x);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

PyObject *setup(PyObject *const *x)
{
    Py_XDECREF(g_current_device);
    Py_XDECREF(g_raw_stream);
    Py_INCREF(x[0]);
    Py_INCREF(x[1]);
    g_current_device = x[0];
    g_raw_stream = x[1];
    Py_RETURN_NONE;
}

// X, codes, scales, trans
PyObject *quantize(PyObject *const *x)
{
    Args a;
    at::ScalarType type = at::kFloat;
    const int t = element_type(a, x[0], type);
    const Mat m(a, x[0], type);
    const int trans = PyObject_IsTrue(x[3]);
    const int64_t rows = trans ? m.cols : m.rows, K = trans ? m.rows : m.cols;
    const Mat q(a, x[1], at::kByte, rows, code_bytes(K)), s(a, x[2], at::kByte, rows, scale_bytes(K));
    void *stream = a.stream();
    return enqueue(a, [&] {
        return mx4_quantize(m.rows, m.cols, t, m.p, m.ld, trans, static_cast<uint8_t *>(q.p), q.ld,
                            static_cast<uint8_t *>(s.p), s.ld, stream);
    });
}

// codes, scales, Y
PyObject *dequantize(PyObject *const *x)
{
    Args a;
    at::ScalarType type = at::kFloat;
    const int t = element_type(a, x[2], type);
    const Mat y(a, x[2], type);
    const Mat q(a, x[0], at::kByte, y.rows, code_bytes(y.cols)), s(a, x[1], at::kByte, y.rows, scale_bytes(y.cols));
    void *stream = a.stream();
    return enqueue(a, [&] {
        return mx4_dequantize(y.rows, y.cols, static_cast<uint8_t *>(q.p), q.ld, static_cast<uint8_t *>(s.p), s.ld, t,
                              y.p, y.ld, stream);
    });
}

// A, SA, B, SB, C, alpha, beta, K or None
PyObject *gemm_mx4(PyObject *const *x)
{
    Args a;
    const Mat A(a, x[0], at::kByte);
    int64_t K = 2 * (int64_t)A.cols;
    if (x[7] != Py_None) {
        K = PyLong_AsLongLong(x[7]);
        if (PyErr_Occurred())
            a.fail();
    }
    if (K < 0 || K > INT32_MAX || code_bytes(K) != A.cols)
        a.ok = false;
    const Mat SA(a, x[1], at::kByte, A.rows, scale_bytes(K)), B(a, x[2], at::kByte, -1, code_bytes(K));
    const Mat SB(a, x[3], at::kByte, B.rows, scale_bytes(K)), C(a, x[4], at::kFloat, A.rows, B.rows);
    const float alpha = (float)a.number(x[5]), beta = (float)a.number(x[6]);
    void *stream = a.stream();
    const at::Tensor w = scratch(a, x[4], A, B, K, LL_A_MX4);
    return enqueue(a, [&] {
        return gemm_mx4f32_nt_ws(A.rows, B.rows, (int)K, alpha, static_cast<uint8_t *>(A.p), A.ld,
                              static_cast<uint8_t *>(SA.p), SA.ld, static_cast<uint8_t *>(B.p), B.ld,
                              static_cast<uint8_t *>(SB.p), SB.ld, beta, static_cast<float *>(C.p), C.ld,
                                 w.defined() ? w.data_ptr() : nullptr, w.defined() ? w.numel() : 0, stream);
    });
}

// A, B, SB, C, alpha, beta
template <bool BF16>
PyObject *gemm_16mx4(PyObject *const *x)
{
    Args a;
    const Mat A(a, x[0], BF16 ? at::kBFloat16 : at::kHalf), B(a, x[1], at::kByte, -1, code_bytes(A.cols));
    const Mat SB(a, x[2], at::kByte, B.rows, scale_bytes(A.cols)), C(a, x[3], at::kFloat, A.rows, B.rows);
    const float alpha = (float)a.number(x[4]), beta = (float)a.number(x[5]);
    void *stream = a.stream();
    const at::Tensor w = scratch(a, x[3], A, B, A.cols, BF16 ? LL_A_BF16 : LL_A_F16);
    return enqueue(a, [&] {
        return (BF16 ? gemm_bf16mx4f32_nt_ws : gemm_f16mx4f32_nt_ws)(
            A.rows, B.rows, A.cols, alpha, static_cast<uint16_t *>(A.p), A.ld, static_cast<uint8_t *>(B.p), B.ld,
            static_cast<uint8_t *>(SB.p), SB.ld, beta, static_cast<float *>(C.p), C.ld,
            w.defined() ? w.data_ptr() : nullptr, w.defined() ? w.numel() : 0, stream);
    });
}

// Y, w_post, gate, alpha, X, w_pre, XO, H, eps
PyObject *norm(PyObject *const *x)
{
    Args a;
    at::ScalarType type = at::kFloat;
    const int t = element_type(a, x[4], type);
    const Mat X(a, x[4], type);
    const int64_t M = X.rows, N = X.cols;
    const Mat Y(a, x[0], at::kFloat, M, N, true), XO(a, x[6], type, M, N, true), H(a, x[7], type, M, N, true);
    const float *w_post = vec(a, x[1], N), *gate = vec(a, x[2], N), *w_pre = vec(a, x[5], N);
    const float alpha = (float)a.number(x[3]), eps = (float)a.number(x[8]);
    void *stream = a.stream();
    return enqueue(a, [&] {
        return rmsnorm_residual(X.rows, X.cols, t, static_cast<float *>(Y.p), Y.ld, w_post, gate, alpha, X.p, X.ld, w_pre,
                                eps, XO.p, XO.ld, H.p, H.ld, stream);
    });
}

// DXO, DH, Y, w_post, gate, alpha, X, w_pre, DY, DX, dgate, dw_post, dw_pre, workspace, eps
PyObject *norm_grad(PyObject *const *x)
{
    Args a;
    at::ScalarType type = at::kFloat;
    const int t = element_type(a, x[6], type);
    const Mat X(a, x[6], type);
    const int64_t M = X.rows, N = X.cols;
    const Mat DXO(a, x[0], type, M, N, true), DH(a, x[1], type, M, N, true), Y(a, x[2], at::kFloat, M, N, true);
    const Mat DY(a, x[8], at::kFloat, M, N, true), DX(a, x[9], type, M, N, true);
    const float *w_post = vec(a, x[3], N), *gate = vec(a, x[4], N), *w_pre = vec(a, x[7], N);
    float *dgate = vec(a, x[10], N), *dw_post = vec(a, x[11], N), *dw_pre = vec(a, x[12], N);
    const float alpha = (float)a.number(x[5]), eps = (float)a.number(x[14]);
    void *ws = nullptr;
    int64_t bytes = 0;
    if (x[13] != Py_None) {
        const at::Tensor *w = a.tensor(x[13]);
        if (w == nullptr || !w->is_contiguous()) {
            a.ok = false;
        } else {
            ws = w->data_ptr();
            bytes = (int64_t)w->nbytes();
        }
    }
    void *stream = a.stream();
    return enqueue(a, [&] {
        return rmsnorm_residual_grad(X.rows, X.cols, t, DXO.p, DXO.ld, DH.p, DH.ld, static_cast<float *>(Y.p), Y.ld, w_post,
                                     gate, alpha, X.p, X.ld, w_pre, eps, static_cast<float *>(DY.p), DY.ld, DX.p, DX.ld,
                                     dgate, dw_post, dw_pre, ws, bytes, stream);
    });
}

#define LL_METHOD(name, n, f) \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&guarded<n, f>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    LL_METHOD("setup", 2, setup),
    LL_METHOD("mx4_quantize", 4, quantize),
    LL_METHOD("mx4_dequantize", 3, dequantize),
    LL_METHOD("gemm_mx4f32_nt", 8, gemm_mx4),
    LL_METHOD("gemm_f16mx4f32_nt", 6, gemm_16mx4<false>),
    LL_METHOD("gemm_bf16mx4f32_nt", 6, gemm_16mx4<true>),
    LL_METHOD("rmsnorm_residual", 9, norm),
    LL_METHOD("rmsnorm_residual_grad", 15, norm_grad),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__call() { return PyModule_Create(&module); }
