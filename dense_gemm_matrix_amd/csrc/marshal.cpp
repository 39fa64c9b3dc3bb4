// marshal.cpp -- the linear layer's entry points for Python: each function
// checks its torch tensors (type, shape, device, layout), reads their pointers
// and pitches and calls the C entry point of the same name (include/dgemm.h) on
// the tensors' device and stream.  Host code only, no arithmetic.
//
// Written against torch's C++ headers because of small calls: a token's norm or
// product runs 3-5 us on the GPU, a launch costs the host 3 us, and the same
// checks in Python cost another 4 (7.5 us per call, 3.9 this way).

#include <Python.h>

#include <c10/hip/HIPStream.h>
#include <hip/hip_runtime.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstring>

#include "dgemm.h"

namespace {

using at::ScalarType;

struct Raised {};  // a Python error is set

template <class... A>
[[noreturn]] void fail(PyObject* type, const char* fmt, A... a) {
    PyErr_Format(type, fmt, a...);
    throw Raised{};
}

// ------------------------------------------------------------------ arguments

// Values of a call's parameters by position: `npos` may be positional, the rest
// are keywords only; absent ones are NULL, None stays None.
template <int N>
void parse(const char* fn, const char* const (&names)[N], int npos, int nreq, PyObject* const* args,
           Py_ssize_t nargs, PyObject* kwnames, PyObject* (&out)[N]) {
    for (int i = 0; i < N; ++i) out[i] = nullptr;
    if (nargs > npos) fail(PyExc_TypeError, "%s() takes %d positional arguments", fn, npos);
    for (Py_ssize_t i = 0; i < nargs; ++i) out[i] = args[i];
    const Py_ssize_t nkw = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    for (Py_ssize_t k = 0; k < nkw; ++k) {
        PyObject* name = PyTuple_GET_ITEM(kwnames, k);
        int i = 0;
        while (i < N && PyUnicode_CompareWithASCIIString(name, names[i]) != 0) ++i;
        if (i == N) fail(PyExc_TypeError, "%s() got an unexpected keyword argument '%U'", fn, name);
        if (out[i]) fail(PyExc_TypeError, "%s() got multiple values for argument '%s'", fn, names[i]);
        out[i] = args[nargs + k];
    }
    for (int i = 0; i < nreq; ++i)
        if (!out[i]) fail(PyExc_TypeError, "%s() missing required argument '%s'", fn, names[i]);
}

bool given(PyObject* o) { return o && o != Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!o || !THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor", name);
    return THPVariable_Unpack(o);
}

int to_int(int64_t v) {
    if (v < 0 || v > INT_MAX) fail(PyExc_ValueError, "a size or row pitch exceeds 32 bits");
    return (int)v;
}

struct Mat {
    void* p = nullptr;
    int ld = 0;
    int rows = 0, cols = 0;
    ScalarType type = ScalarType::Undefined;
    int dev = -1;
};

// A row-major matrix.  One of at most one row never steps to a second, so its
// pitch is free: given as the row length rounded up to 16 bytes.
Mat matrix(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 2) fail(PyExc_ValueError, "operands must be 2-D");
    if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a device tensor", name);
    Mat m;
    m.rows = to_int(t.size(0));
    m.cols = to_int(t.size(1));
    m.type = t.scalar_type();
    m.dev = t.get_device();
    if (t.stride(1) != 1 && m.cols > 1 && m.rows > 0)
        fail(PyExc_ValueError, "operands must be row-major with unit inner stride");
    if (m.rows > 1) {
        m.ld = to_int(t.stride(0));
    } else {
        const int64_t per16 = 16 / (int64_t)t.element_size();
        m.ld = to_int(((m.cols > 1 ? m.cols : 1) + per16 - 1) / per16 * per16);
    }
    m.p = t.data_ptr();
    return m;
}

// An operand with the given size, type and device; absent: all zero.
Mat matrix_like(PyObject* o, const char* name, int rows, int cols, ScalarType type, int dev) {
    if (!given(o)) return Mat{};
    const Mat m = matrix(o, name);
    if (m.type != type) fail(PyExc_TypeError, "%s must be %s", name, c10::toString(type));
    if (m.rows != rows || m.cols != cols || m.dev != dev)
        fail(PyExc_ValueError, "%s must be a %d x %d matrix on device %d", name, rows, cols, dev);
    return m;
}

float* vec(PyObject* o, const char* name, int n, int dev) {
    if (!given(o)) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != ScalarType::Float || t.dim() != 1 || t.numel() != n || !t.is_contiguous() ||
        !t.is_cuda() || t.get_device() != dev)
        fail(PyExc_ValueError, "%s must be a contiguous float32 device vector of length %d", name, n);
    return (float*)t.data_ptr();
}

float* need_vec(PyObject* o, const char* name, int n, int dev) {
    if (!given(o)) fail(PyExc_ValueError, "%s is required", name);
    return vec(o, name, n, dev);
}

// A float32 matrix of block scales with any strides: block (i, b) at p[i * row + b * blk].
struct Scales {
    float* p = nullptr;
    int rows = 0, row = 0, blk = 0;
};

Scales scales(PyObject* o, const char* name, int blocks, int dev) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != ScalarType::Float || t.dim() != 2 || t.size(1) != blocks || !t.is_cuda() ||
        t.get_device() != dev)
        fail(PyExc_ValueError, "%s must be a float32 device matrix with %d columns", name, blocks);
    Scales s;
    s.p = (float*)t.data_ptr();
    s.rows = to_int(t.size(0));
    // A stride that is never stepped is free.
    s.row = s.rows > 1 ? to_int(t.stride(0)) : 1;
    s.blk = blocks > 1 ? to_int(t.stride(1)) : 1;
    return s;
}

int blocks_of(int n) { return (int)(((int64_t)n + DGEMM_F8_BLOCK - 1) / DGEMM_F8_BLOCK); }

struct Bytes {
    void* p = nullptr;
    size_t n = 0;
};

Bytes workspace(PyObject* o, int dev) {
    if (!given(o)) return Bytes{};
    const at::Tensor& t = tensor(o, "workspace");
    if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
        fail(PyExc_ValueError, "workspace must be a contiguous tensor on the output's device");
    return Bytes{t.data_ptr(), (size_t)t.nbytes()};
}

int act_code(PyObject* o) {
    static const char* const names[] = {"none", "relu", "gelu", "gelu_tanh", "silu"};
    if (!given(o)) return DGEMM_ACT_NONE;
    for (int i = 0; PyUnicode_Check(o) && i < 5; ++i)
        if (PyUnicode_CompareWithASCIIString(o, names[i]) == 0) return i;
    fail(PyExc_ValueError, "act must be one of none, relu, gelu, gelu_tanh, silu");
}

double number(PyObject* o, double otherwise) {
    if (!o) return otherwise;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
}

// DGEMM_IN_F32 / _BF16 / _F16 of a type, -1 for any other.
int fmt_of(ScalarType t) {
    return t == ScalarType::Float ? DGEMM_IN_F32 : t == ScalarType::BFloat16 ? DGEMM_IN_BF16
           : t == ScalarType::Half ? DGEMM_IN_F16 : -1;
}

int need_fmt(ScalarType t, const char* name) {
    const int f = fmt_of(t);
    if (f < 0) fail(PyExc_TypeError, "%s must be float32, bfloat16 or float16", name);
    return f;
}

// The input code of a product's operands and the output code of its results.
void formats(const Mat& A, const Mat& B, ScalarType c, PyObject* in_fmt, int& in, int& out) {
    const int own = fmt_of(A.type);
    in = own;
    if (given(in_fmt)) {
        static const char* const names[] = {"f32", "bf16", "f16", "f32x3"};
        in = -1;
        for (int i = 0; PyUnicode_Check(in_fmt) && i < 4; ++i)
            if (PyUnicode_CompareWithASCIIString(in_fmt, names[i]) == 0) in = i;
    }
    if (own < 0 || B.type != A.type || !(in == own || (in == DGEMM_IN_F32_3XBF16 && own == DGEMM_IN_F32)))
        fail(PyExc_TypeError, "unsupported input dtypes");
    if (c != ScalarType::Float && c != A.type)
        fail(PyExc_TypeError, "C must be float32 or the input dtype");
    out = c == ScalarType::Float ? DGEMM_OUT_F32 : DGEMM_OUT_SAME;
}

void conform(const Mat& A, const Mat& B, const Mat& C) {
    if (A.cols != B.rows || C.rows != A.rows || C.cols != B.cols)
        fail(PyExc_ValueError, "shapes (%d, %d) x (%d, %d) -> (%d, %d)", A.rows, A.cols, B.rows, B.cols,
             C.rows, C.cols);
    if (A.dev != C.dev || B.dev != C.dev)
        fail(PyExc_ValueError, "operands on different devices: %d, %d, %d", A.dev, B.dev, C.dev);
}

void* stream_of(PyObject* o, int dev) {
    if (!given(o)) return (void*)c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream();
    PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
    if (!h) throw Raised{};
    void* s = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Raised{};
    return s;
}

// Runs a C entry point with `dev` current and raises DgemmError for a status.
template <class F>
PyObject* call(int dev, F f) {
    int status = DGEMM_ERR_DEVICE;
    Py_BEGIN_ALLOW_THREADS
    int prev = -1;
    if (hipGetDevice(&prev) == hipSuccess) {
        if (prev == dev) {
            status = f();
        } else if (hipSetDevice(dev) == hipSuccess) {
            status = f();
            (void)hipSetDevice(prev);
        }
    }
    Py_END_ALLOW_THREADS
    if (status != DGEMM_OK) {
        PyObject* mod = PyImport_ImportModule("dense_gemm_matrix_amd._binding");
        PyObject* cls = mod ? PyObject_GetAttrString(mod, "DgemmError") : nullptr;
        PyObject* arg = cls ? PyLong_FromLong(status) : nullptr;
        if (arg) PyErr_SetObject(cls, arg);
        Py_XDECREF(arg);
        Py_XDECREF(cls);
        Py_XDECREF(mod);
        throw Raised{};
    }
    Py_RETURN_NONE;
}

template <class F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// ------------------------------------------------------------------ functions

PyObject* py_gemm_act(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    static const char* const names[] = {"A", "B", "C", "bias", "act", "residual", "preact", "workspace",
                                        "in_fmt", "stream"};
    return guarded([&] {
        PyObject* o[10];
        parse("gemm_act", names, 3, 3, args, nargs, kw, o);
        const Mat A = matrix(o[0], "A"), B = matrix(o[1], "B"), C = matrix(o[2], "C");
        conform(A, B, C);
        int in, out;
        formats(A, B, C.type, o[8], in, out);
        const float* bias = vec(o[3], "bias", C.cols, C.dev);
        const int act = act_code(o[4]);
        const Mat R = matrix_like(o[5], "residual", C.rows, C.cols, C.type, C.dev);
        const Mat Z = matrix_like(o[6], "preact", C.rows, C.cols, C.type, C.dev);
        const Bytes ws = workspace(o[7], C.dev);
        void* s = stream_of(o[9], C.dev);
        return call(C.dev, [&] {
            return gemm_act(in, out, C.rows, C.cols, A.cols, A.p, A.ld, B.p, B.ld, C.p, C.ld, bias, act,
                            R.p, R.ld, Z.p, Z.ld, ws.p, ws.n, s);
        });
    });
}

PyObject* py_gemm_act_bwd(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    static const char* const names[] = {"A", "B", "dC", "dA", "dB", "dbias", "preact", "act", "workspace",
                                        "in_fmt", "stream"};
    return guarded([&] {
        PyObject* o[11];
        parse("gemm_act_bwd", names, 3, 3, args, nargs, kw, o);
        const Mat A = matrix(o[0], "A"), B = matrix(o[1], "B"), dC = matrix(o[2], "dC");
        conform(A, B, dC);
        const int M = dC.rows, N = dC.cols, K = A.cols, dev = dC.dev;
        int in, out;
        formats(A, B, dC.type, o[9], in, out);
        const int act = act_code(o[7]);
        if (act != DGEMM_ACT_NONE && !given(o[6]))
            fail(PyExc_ValueError, "the gradient of an activation needs preact");
        const Mat dA = matrix_like(o[3], "dA", M, K, A.type, dev);
        const Mat dB = matrix_like(o[4], "dB", K, N, A.type, dev);
        float* dbias = vec(o[5], "dbias", N, dev);
        const Mat Z = act == DGEMM_ACT_NONE ? Mat{} : matrix_like(o[6], "preact", M, N, dC.type, dev);
        const Bytes ws = workspace(o[8], dev);
        void* s = stream_of(o[10], dev);
        return call(dev, [&] {
            return gemm_act_bwd(in, out, M, N, K, A.p, A.ld, B.p, B.ld, dC.p, dC.ld, Z.p, Z.ld, act, dA.p,
                                dA.ld, dB.p, dB.ld, dbias, ws.p, ws.n, s);
        });
    });
}

PyObject* py_gemm_f8(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    static const char* const names[] = {"A", "B", "C", "scale_a", "scale_b", "bias", "act", "residual",
                                        "workspace", "stream"};
    return guarded([&] {
        PyObject* o[10];
        parse("gemm_f8", names, 5, 5, args, nargs, kw, o);
        const Mat A = matrix(o[0], "A"), B = matrix(o[1], "B"), C = matrix(o[2], "C");
        if (A.cols != B.cols || C.rows != A.rows || C.cols != B.rows)
            fail(PyExc_ValueError, "shapes (%d, %d) x (%d, %d)^T -> (%d, %d)", A.rows, A.cols, B.rows,
                 B.cols, C.rows, C.cols);
        if (A.dev != C.dev || B.dev != C.dev)
            fail(PyExc_ValueError, "operands on different devices: %d, %d, %d", A.dev, B.dev, C.dev);
        if (A.type != ScalarType::Float8_e4m3fn || B.type != ScalarType::Float8_e4m3fn)
            fail(PyExc_TypeError, "A and B must be float8_e4m3fn");
        const int fmt = need_fmt(C.type, "C");
        const float* sa = need_vec(o[3], "scale_a", C.rows, C.dev);
        const float* sb = need_vec(o[4], "scale_b", C.cols, C.dev);
        const float* bias = vec(o[5], "bias", C.cols, C.dev);
        const int act = act_code(o[6]);
        const Mat R = matrix_like(o[7], "residual", C.rows, C.cols, C.type, C.dev);
        const Bytes ws = workspace(o[8], C.dev);
        void* s = stream_of(o[9], C.dev);
        return call(C.dev, [&] {
            return gemm_f8(fmt, C.rows, C.cols, A.cols, A.p, A.ld, B.p, B.ld, C.p, C.ld, sa, sb, bias, act,
                           R.p, R.ld, ws.p, ws.n, s);
        });
    });
}

PyObject* py_rmsnorm(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    static const char* const names[] = {"X", "weight", "Y", "residual", "total", "scale", "rstd", "eps",
                                        "stream"};
    return guarded([&] {
        PyObject* o[9];
        parse("rmsnorm", names, 3, 3, args, nargs, kw, o);
        const Mat X = matrix(o[0], "X");
        const int M = X.rows, N = X.cols, dev = X.dev, fmt = need_fmt(X.type, "X");
        const float* w = need_vec(o[1], "weight", N, dev);
        const bool f8 = tensor(o[2], "Y").scalar_type() == ScalarType::Float8_e4m3fn;
        if (f8 != given(o[5])) fail(PyExc_ValueError, "a float8_e4m3fn Y takes a scale, and only that");
        const Mat Y = matrix_like(o[2], "Y", M, N, f8 ? ScalarType::Float8_e4m3fn : X.type, dev);
        const Mat R = matrix_like(o[3], "residual", M, N, X.type, dev);
        const Mat S = matrix_like(o[4], "total", M, N, X.type, dev);
        int out = f8 ? DGEMM_ROWS_F8 : DGEMM_ROWS_SAME;
        float* scale = nullptr;
        if (f8 && tensor(o[5], "scale").dim() == 2) {
            out = DGEMM_ROWS_F8_BLOCK;
            const Scales sc = scales(o[5], "scale", blocks_of(N), dev);
            if (sc.rows != M || (M > 1 && sc.row != 1) || (N > DGEMM_F8_BLOCK && sc.blk != M))
                fail(PyExc_ValueError, "scale must be the transpose of a contiguous (%d, %d) matrix", blocks_of(N), M);
            scale = sc.p;
        } else {
            scale = vec(o[5], "scale", M, dev);
        }
        float* rstd = vec(o[6], "rstd", M, dev);
        const double eps = number(o[7], 1e-6);
        void* s = stream_of(o[8], dev);
        return call(dev, [&] {
            return rmsnorm(fmt, out, M, N, X.p, X.ld, R.p, R.ld, S.p, S.ld,
                           w, (float)eps, Y.p, Y.ld, scale, rstd, s);
        });
    });
}

PyObject* py_rmsnorm_bwd(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    static const char* const names[] = {"dY", "total", "weight", "rstd", "dX", "dtotal", "dweight",
                                        "workspace", "stream"};
    return guarded([&] {
        PyObject* o[9];
        parse("rmsnorm_bwd", names, 5, 5, args, nargs, kw, o);
        const Mat dY = matrix(o[0], "dY");
        const int M = dY.rows, N = dY.cols, dev = dY.dev, fmt = need_fmt(dY.type, "dY");
        const Mat S = matrix_like(o[1], "total", M, N, dY.type, dev);
        const float* w = need_vec(o[2], "weight", N, dev);
        const float* rstd = need_vec(o[3], "rstd", M, dev);
        const Mat dX = matrix_like(o[4], "dX", M, N, dY.type, dev);
        const Mat dS = matrix_like(o[5], "dtotal", M, N, dY.type, dev);
        float* dw = vec(o[6], "dweight", N, dev);
        const Bytes ws = workspace(o[7], dev);
        void* s = stream_of(o[8], dev);
        return call(dev, [&] {
            return rmsnorm_bwd(fmt, M, N, dY.p, dY.ld, S.p, S.ld, w, rstd, dS.p, dS.ld, dX.p, dX.ld, dw,
                               ws.p, ws.n, s);
        });
    });
}

PyObject* py_quant_f8(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    static const char* const names[] = {"X", "Q", "scale", "transpose", "stream"};
    return guarded([&] {
        PyObject* o[5];
        parse("quant_f8", names, 3, 3, args, nargs, kw, o);
        const Mat X = matrix(o[0], "X");
        const int fmt = need_fmt(X.type, "X");
        const int tr = o[3] ? PyObject_IsTrue(o[3]) : 0;
        if (tr < 0) throw Raised{};
        const int rows = tr ? X.cols : X.rows, cols = tr ? X.rows : X.cols;
        if (!given(o[1])) fail(PyExc_ValueError, "Q is required");
        const Mat Q = matrix_like(o[1], "Q", rows, cols, ScalarType::Float8_e4m3fn, X.dev);
        float* scale = need_vec(o[2], "scale", rows, X.dev);
        void* s = stream_of(o[4], X.dev);
        return call(X.dev, [&] {
            return quant_f8(fmt, tr, X.rows, X.cols, X.p, X.ld, Q.p, Q.ld, scale, s);
        });
    });
}

PyObject* py_gemm_f8_block(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    static const char* const names[] = {"A", "B", "C", "scale_a", "scale_b", "bias", "act", "residual",
                                        "workspace", "stream"};
    return guarded([&] {
        PyObject* o[10];
        parse("gemm_f8_block", names, 5, 5, args, nargs, kw, o);
        const Mat A = matrix(o[0], "A"), B = matrix(o[1], "B"), C = matrix(o[2], "C");
        if (A.cols != B.cols || C.rows != A.rows || C.cols != B.rows)
            fail(PyExc_ValueError, "shapes (%d, %d) x (%d, %d)^T -> (%d, %d)", A.rows, A.cols, B.rows,
                 B.cols, C.rows, C.cols);
        if (A.dev != C.dev || B.dev != C.dev)
            fail(PyExc_ValueError, "operands on different devices: %d, %d, %d", A.dev, B.dev, C.dev);
        if (A.type != ScalarType::Float8_e4m3fn || B.type != ScalarType::Float8_e4m3fn)
            fail(PyExc_TypeError, "A and B must be float8_e4m3fn");
        const int fmt = need_fmt(C.type, "C"), kb = blocks_of(A.cols);
        const Scales sa = scales(o[3], "scale_a", kb, C.dev), sb = scales(o[4], "scale_b", kb, C.dev);
        if (sa.rows != C.rows) fail(PyExc_ValueError, "scale_a must have a row per row of A");
        const bool each = sb.rows == C.cols;
        if (!each && sb.rows != blocks_of(C.cols))
            fail(PyExc_ValueError, "scale_b must have a row per row of B, or per %d of them", DGEMM_F8_BLOCK);
        const float* bias = vec(o[5], "bias", C.cols, C.dev);
        const int act = act_code(o[6]);
        const Mat R = matrix_like(o[7], "residual", C.rows, C.cols, C.type, C.dev);
        const Bytes ws = workspace(o[8], C.dev);
        void* s = stream_of(o[9], C.dev);
        return call(C.dev, [&] {
            return gemm_f8_block(fmt, each ? 1 : DGEMM_F8_BLOCK, C.rows, C.cols, A.cols, A.p, A.ld, B.p, B.ld,
                                 C.p, C.ld, sa.p, sa.row, sa.blk, sb.p, sb.row, sb.blk, bias, act, R.p, R.ld,
                                 ws.p, ws.n, s);
        });
    });
}

PyObject* py_quant_f8_block(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    static const char* const names[] = {"X", "Q", "scale", "transpose", "stream"};
    return guarded([&] {
        PyObject* o[5];
        parse("quant_f8_block", names, 3, 3, args, nargs, kw, o);
        const Mat X = matrix(o[0], "X");
        const int fmt = need_fmt(X.type, "X");
        const int tr = o[3] ? PyObject_IsTrue(o[3]) : 0;
        if (tr < 0) throw Raised{};
        const int rows = tr ? X.cols : X.rows, cols = tr ? X.rows : X.cols;
        if (!given(o[1])) fail(PyExc_ValueError, "Q is required");
        const Mat Q = matrix_like(o[1], "Q", rows, cols, ScalarType::Float8_e4m3fn, X.dev);
        const Scales sc = scales(o[2], "scale", blocks_of(cols), X.dev);
        if (sc.rows != rows && sc.rows != blocks_of(rows))
            fail(PyExc_ValueError, "scale must have a row per row of Q, or per %d of them", DGEMM_F8_BLOCK);
        void* s = stream_of(o[4], X.dev);
        return call(X.dev, [&] {
            return quant_f8_block(fmt, sc.rows == rows ? 1 : DGEMM_F8_BLOCK, tr, X.rows, X.cols, X.p, X.ld, Q.p,
                                  Q.ld, sc.p, sc.row, sc.blk, s);
        });
    });
}

PyObject* py_layernorm(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    static const char* const names[] = {"X", "weight", "bias", "Y", "residual", "total", "scale", "mean", "rstd",
                                        "eps", "stream"};
    return guarded([&] {
        PyObject* o[11];
        parse("layernorm", names, 4, 4, args, nargs, kw, o);
        const Mat X = matrix(o[0], "X");
        const int M = X.rows, N = X.cols, dev = X.dev, fmt = need_fmt(X.type, "X");
        const float* w = need_vec(o[1], "weight", N, dev);
        const float* b = vec(o[2], "bias", N, dev);
        const bool f8 = tensor(o[3], "Y").scalar_type() == ScalarType::Float8_e4m3fn;
        if (f8 != given(o[6])) fail(PyExc_ValueError, "a float8_e4m3fn Y takes a scale, and only that");
        const Mat Y = matrix_like(o[3], "Y", M, N, f8 ? ScalarType::Float8_e4m3fn : X.type, dev);
        const Mat R = matrix_like(o[4], "residual", M, N, X.type, dev);
        const Mat S = matrix_like(o[5], "total", M, N, X.type, dev);
        int out = f8 ? DGEMM_ROWS_F8 : DGEMM_ROWS_SAME;
        Scales sc;
        if (f8 && tensor(o[6], "scale").dim() == 2) {
            out = DGEMM_ROWS_F8_BLOCK;
            sc = scales(o[6], "scale", blocks_of(N), dev);
            if (sc.rows != M) fail(PyExc_ValueError, "scale must have a row per row of Y");
        } else {
            sc.p = vec(o[6], "scale", M, dev);
        }
        float* mean = vec(o[7], "mean", M, dev);
        float* rstd = vec(o[8], "rstd", M, dev);
        const double eps = number(o[9], 1e-5);
        void* s = stream_of(o[10], dev);
        return call(dev, [&] {
            return layernorm(fmt, out, M, N, X.p, X.ld, R.p, R.ld, S.p, S.ld, w, b, (float)eps, Y.p, Y.ld, sc.p,
                             sc.row, sc.blk, mean, rstd, s);
        });
    });
}

PyObject* py_layernorm_bwd(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    static const char* const names[] = {"dY", "total", "weight", "mean", "rstd", "dX", "dtotal", "dweight",
                                        "dbias", "workspace", "stream"};
    return guarded([&] {
        PyObject* o[11];
        parse("layernorm_bwd", names, 6, 6, args, nargs, kw, o);
        const Mat dY = matrix(o[0], "dY");
        const int M = dY.rows, N = dY.cols, dev = dY.dev, fmt = need_fmt(dY.type, "dY");
        const Mat S = matrix_like(o[1], "total", M, N, dY.type, dev);
        const float* w = need_vec(o[2], "weight", N, dev);
        const float* mean = need_vec(o[3], "mean", M, dev);
        const float* rstd = need_vec(o[4], "rstd", M, dev);
        const Mat dX = matrix_like(o[5], "dX", M, N, dY.type, dev);
        const Mat dS = matrix_like(o[6], "dtotal", M, N, dY.type, dev);
        float* dw = vec(o[7], "dweight", N, dev);
        float* db = vec(o[8], "dbias", N, dev);
        const Bytes ws = workspace(o[9], dev);
        void* s = stream_of(o[10], dev);
        return call(dev, [&] {
            return layernorm_bwd(fmt, M, N, dY.p, dY.ld, S.p, S.ld, w, mean, rstd, dS.p, dS.ld, dX.p, dX.ld, dw,
                                 db, ws.p, ws.n, s);
        });
    });
}

// The second weight of a gated layer, like the first; a row pitch of its own.
Mat second_weight(PyObject* o, const Mat& first) {
    if (!given(o)) fail(PyExc_ValueError, "Bu is required");
    return matrix_like(o, "Bu", first.rows, first.cols, first.type, first.dev);
}

PyObject* py_gemm_gated(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    static const char* const names[] = {"A", "Bg", "Bu", "C", "bias_g", "bias_u", "act", "gate", "up", "workspace",
                                        "stream"};
    return guarded([&] {
        PyObject* o[11];
        parse("gemm_gated", names, 4, 4, args, nargs, kw, o);
        const Mat A = matrix(o[0], "A"), Bg = matrix(o[1], "Bg"), Bu = second_weight(o[2], Bg), C = matrix(o[3], "C");
        conform(A, Bg, C);
        int in, out;
        formats(A, Bg, C.type, nullptr, in, out);
        const float* bg = vec(o[4], "bias_g", C.cols, C.dev);
        const float* bu = vec(o[5], "bias_u", C.cols, C.dev);
        const int act = o[6] ? act_code(o[6]) : DGEMM_ACT_SILU;
        const Mat G = matrix_like(o[7], "gate", C.rows, C.cols, C.type, C.dev);
        const Mat U = matrix_like(o[8], "up", C.rows, C.cols, C.type, C.dev);
        const Bytes ws = workspace(o[9], C.dev);
        void* s = stream_of(o[10], C.dev);
        return call(C.dev, [&] {
            return gemm_gated(in, out, C.rows, C.cols, A.cols, A.p, A.ld, Bg.p, Bg.ld, Bu.p, Bu.ld, C.p, C.ld, bg, bu,
                              act, G.p, G.ld, U.p, U.ld, ws.p, ws.n, s);
        });
    });
}

PyObject* py_gemm_gated_bwd(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
    static const char* const names[] = {"A", "Bg", "Bu", "dC", "gate", "up", "act", "dA", "dBg", "dBu", "dbias_g",
                                        "dbias_u", "workspace", "stream"};
    return guarded([&] {
        PyObject* o[14];
        parse("gemm_gated_bwd", names, 6, 6, args, nargs, kw, o);
        const Mat A = matrix(o[0], "A"), Bg = matrix(o[1], "Bg"), Bu = second_weight(o[2], Bg);
        const Mat dC = matrix(o[3], "dC");
        conform(A, Bg, dC);
        const int M = dC.rows, N = dC.cols, K = A.cols, dev = dC.dev;
        int in, out;
        formats(A, Bg, dC.type, nullptr, in, out);
        if (!given(o[4]) || !given(o[5])) fail(PyExc_ValueError, "gate and up are required");
        const Mat G = matrix_like(o[4], "gate", M, N, dC.type, dev), U = matrix_like(o[5], "up", M, N, dC.type, dev);
        const int act = o[6] ? act_code(o[6]) : DGEMM_ACT_SILU;
        const Mat dA = matrix_like(o[7], "dA", M, K, A.type, dev);
        const Mat dBg = matrix_like(o[8], "dBg", K, N, A.type, dev), dBu = matrix_like(o[9], "dBu", K, N, A.type, dev);
        float* dbg = vec(o[10], "dbias_g", N, dev);
        float* dbu = vec(o[11], "dbias_u", N, dev);
        const Bytes ws = workspace(o[12], dev);
        void* s = stream_of(o[13], dev);
        return call(dev, [&] {
            return gemm_gated_bwd(in, out, M, N, K, A.p, A.ld, Bg.p, Bg.ld, Bu.p, Bu.ld, dC.p, dC.ld, G.p, G.ld, U.p,
                                  U.ld, act, dA.p, dA.ld, dBg.p, dBg.ld, dBu.p, dBu.ld, dbg, dbu, ws.p, ws.n, s);
        });
    });
}

#define FN(name, doc) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL | METH_KEYWORDS, doc}
PyMethodDef methods[] = {
    FN(gemm_act,
       "gemm_act(A, B, C, *, bias=None, act='none', residual=None, preact=None, workspace=None,\n"
       "         in_fmt=None, stream=None)\n\n"
       "C = act(A @ B + bias) + residual; preact (optional) = A @ B + bias.\n\n"
       "`residual` and `preact` have C's shape and dtype; `residual` may be C itself.  `act` is none,\n"
       "relu, gelu, gelu_tanh or silu; `workspace` and `in_fmt` as in gemm_ex."),
    FN(gemm_act_bwd,
       "gemm_act_bwd(A, B, dC, *, dA=None, dB=None, dbias=None, preact=None, act='none',\n"
       "             workspace=None, in_fmt=None, stream=None)\n\n"
       "Gradients of gemm_act: dA (A's shape and dtype), dB (B's) and dbias (float32), each\n"
       "written if given; `preact` as gemm_act stored it (not needed with act 'none').  The\n"
       "workspace holds at least gemm_act_bwd_workspace's required bytes."),
    FN(gemm_f8,
       "gemm_f8(A, B, C, scale_a, scale_b, *, bias=None, act='none', residual=None,\n"
       "        workspace=None, stream=None)\n\n"
       "C = act(scale_a[:, None] * scale_b * (A @ B.T) + bias) + residual for float8_e4m3fn\n"
       "A [M, K] and B [N, K]; C (and residual) float32, bfloat16 or float16."),
    FN(rmsnorm,
       "rmsnorm(X, weight, Y, *, residual=None, total=None, scale=None, rstd=None, eps=1e-6,\n"
       "        stream=None)\n\n"
       "Y = s * rstd * weight row by row, s = X + residual, rstd = (mean s^2 + eps)^-1/2.\n\n"
       "Y has X's dtype, or is float8_e4m3fn with a float32 `scale` per row (gemm_f8's A and\n"
       "scale_a), or per row and block of 128 columns (gemm_f8_block's: the transpose of a\n"
       "contiguous (blocks, rows) tensor).  `total` (X's dtype) receives s and `rstd` (float32, one per row) its root\n"
       "where given: what rmsnorm_bwd reads.  `total` and Y may be X or residual themselves."),
    FN(rmsnorm_bwd,
       "rmsnorm_bwd(dY, total, weight, rstd, dX, *, dtotal=None, dweight=None, workspace=None,\n"
       "            stream=None)\n\n"
       "Gradients of rmsnorm: dX (the residual's too) and, where given, dweight (float32; needs\n"
       "rmsnorm_bwd_workspace's bytes).  `total` and `rstd` as rmsnorm stored them (total is X\n"
       "where there was no residual); `dtotal` is the gradient that reaches total by other ways.\n"
       "dX may be dY or dtotal itself."),
    FN(quant_f8,
       "quant_f8(X, Q, scale, *, transpose=False, stream=None)\n\n"
       "Q, scale = X's rows in 8 bits (float8_e4m3fn, one float32 scale per row); with transpose\n"
       "its columns, Q being X.T's shape: gemm_f8's B from a [K, N] weight."),
    FN(gemm_gated,
       "gemm_gated(A, Bg, Bu, C, *, bias_g=None, bias_u=None, act='silu', gate=None, up=None,\n"
       "           workspace=None, stream=None)\n\n"
       "C = act(G) * U with G = A @ Bg + bias_g and U = A @ Bu + bias_u, stored in `gate` and `up`\n"
       "(C's shape and dtype) where given.  float32, bfloat16 or float16; C has A's dtype or is\n"
       "float32.  `act` is silu, gelu, gelu_tanh, relu or none; `workspace` as in gemm_ex."),
    FN(gemm_gated_bwd,
       "gemm_gated_bwd(A, Bg, Bu, dC, gate, up, *, act='silu', dA=None, dBg=None, dBu=None,\n"
       "               dbias_g=None, dbias_u=None, workspace=None, stream=None)\n\n"
       "Gradients of gemm_gated: dA, dBg and dBu (shapes and dtype of A, Bg and Bu), dbias_g and\n"
       "dbias_u (float32), each written if given; `gate` and `up` as gemm_gated stored them.  The\n"
       "workspace holds at least gemm_gated_bwd_workspace's required bytes."),
    FN(gemm_f8_block,
       "gemm_f8_block(A, B, C, scale_a, scale_b, *, bias=None, act='none', residual=None,\n"
       "              workspace=None, stream=None)\n\n"
       "C = act(a @ b.T + bias) + residual, a and b being float8_e4m3fn A [M, K] and B [N, K] with\n"
       "each block of 128 columns scaled: scale_a [M, blocks] by row, scale_b [N, blocks] by row or\n"
       "[ceil(N / 128), blocks] by 128 rows (float32, any strides).  C (and residual) float32,\n"
       "bfloat16 or float16; `residual` may be C itself."),
    FN(quant_f8_block,
       "quant_f8_block(X, Q, scale, *, transpose=False, stream=None)\n\n"
       "Q, scale = X (with transpose X.T) in 8 bits, float8_e4m3fn, with a float32 scale per block of\n"
       "128 columns of Q and one or 128 of its rows, as scale's shape says: gemm_f8_block's operands."),
    FN(layernorm,
       "layernorm(X, weight, bias, Y, *, residual=None, total=None, scale=None, mean=None, rstd=None,\n"
       "          eps=1e-5, stream=None)\n\n"
       "Y = (s - mean) * rstd * weight + bias row by row, s = X + residual; bias may be None.\n\n"
       "Y has X's dtype, or is float8_e4m3fn with a float32 `scale` per row (gemm_f8's A and scale_a)\n"
       "or per row and block of 128 columns (gemm_f8_block's; any strides).  `total` (X's dtype)\n"
       "receives s, `mean` and `rstd` (float32, one per row) its moments where given: what\n"
       "layernorm_bwd reads.  `total` and Y may be X or residual themselves."),
    FN(layernorm_bwd,
       "layernorm_bwd(dY, total, weight, mean, rstd, dX, *, dtotal=None, dweight=None, dbias=None,\n"
       "              workspace=None, stream=None)\n\n"
       "Gradients of layernorm: dX (the residual's too) and, where given, dweight and dbias (float32;\n"
       "either needs layernorm_bwd_workspace's bytes).  `total`, `mean` and `rstd` as layernorm stored\n"
       "them (total is X where there was no residual); `dtotal` is the gradient that reaches total by\n"
       "other ways.  dX may be dY or dtotal itself."),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal",
                      "The linear layer's entry points for torch tensors (csrc/marshal.cpp).", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
