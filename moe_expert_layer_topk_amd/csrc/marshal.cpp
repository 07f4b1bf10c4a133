// Argument marshalling of the dense operators for Python, as a CPython module.
//
// Their smallest calls take 4 us on the GPU; looking at five tensors from
// Python and passing them through ctypes took 8 us of host time per call.
// Here a call checks its tensors, allocates the outputs that were not passed
// and calls the C ABI on the current stream of the tensors' device: no
// arithmetic, and the same checks and errors for every caller.
//
// Outputs come from torch's allocator past its dispatcher, which takes longer
// than the allocator: dispatch modes (and the filling of new tensors that
// torch's deterministic mode does) do not see them. Like the rest of the
// library these calls have no gradient; an input that requires one is read, and
// the outputs require none.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/EmptyTensor.h>
#include <ATen/hip/impl/HIPCachingAllocatorMasqueradingAsCUDA.h>
#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <c10/hip/HIPFunctions.h>

#include <string>

#include "../../include/moe.h"

namespace {

PyObject* g_error = nullptr;          // MoeError

[[noreturn]] void refuse(const std::string& what) {
    PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, what.c_str());
    throw python_error();
}

std::string said(const at::Tensor& t) {
    std::string s = std::string(c10::toString(t.scalar_type())) + " (";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + ") on " + t.device().str();
}

void count(Py_ssize_t got, Py_ssize_t want, const char* f) {
    if (got != want) refuse(std::string(f) + ": " + std::to_string(want) + " arguments");
}

// the tensor in o; undefined for None
const at::Tensor& tensor(PyObject* o, const char* name) {
    static const at::Tensor none;
    if (o == Py_None) return none;
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

bool plain(const at::Tensor& t, at::ScalarType type) {
    return t.is_cuda() && t.scalar_type() == type && t.layout() == at::kStrided && t.is_contiguous() && !t.is_neg() &&
           !t.is_conj();
}

// a device made current, and the one before it again at the end
struct Current {
    c10::DeviceIndex before, now;
    explicit Current(c10::Device d) : before(c10::hip::current_device()), now(d.index()) {
        if (now != before) c10::hip::set_device(now);
    }
    ~Current() {
        if (now != before) (void)hipSetDevice(before);
    }
    Current(const Current&) = delete;
};

struct Matrix {
    const at::Tensor& t;
    int rows, cols;
    c10::Device dev;
};

// a non-empty contiguous matrix in device memory
Matrix matrix(PyObject* o, at::ScalarType type, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (!t.defined()) refuse(std::string(name) + " must be a tensor");
    if (!plain(t, type) || t.dim() != 2 || t.numel() == 0 || t.size(0) > INT32_MAX || t.size(1) > INT32_MAX)
        refuse(std::string(name) + " must be a non-empty contiguous " + c10::toString(type) + " matrix on the device, got " +
               said(t));
    return {t, (int)t.size(0), (int)t.size(1), t.device()};
}

// address of a contiguous tensor of exactly this shape (cols < 0: a vector) and type beside m (null for None)
void* beside(const at::Tensor& t, const Matrix& m, int64_t rows, int64_t cols, at::ScalarType type, const char* name) {
    if (!t.defined()) return nullptr;
    const bool shape = cols < 0 ? t.dim() == 1 && t.size(0) == rows : t.dim() == 2 && t.size(0) == rows && t.size(1) == cols;
    if (!shape || !plain(t, type) || t.device() != m.dev)
        refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor of shape (" + std::to_string(rows) +
               (cols < 0 ? "" : ", " + std::to_string(cols)) + ") on " + m.dev.str() + ", got " + said(t));
    return t.data_ptr();
}
void* needed(PyObject* o, const Matrix& m, int64_t rows, int64_t cols, at::ScalarType type, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (!t.defined()) refuse(std::string(name) + " must be a tensor");
    return beside(t, m, rows, cols, type, name);
}
void* given(PyObject* o, const Matrix& m, int64_t rows, int64_t cols, at::ScalarType type, const char* name) {
    return beside(tensor(o, name), m, rows, cols, type, name);
}

// an output: the tensor passed, or a new one
struct Out {
    at::Tensor t;
    void* p = nullptr;
    Out() = default;
    Out(PyObject* o, const Matrix& m, int64_t rows, int64_t cols, at::ScalarType type, const char* name) {
        t = tensor(o, name);
        if (t.defined()) {
            p = beside(t, m, rows, cols, type, name);
            return;
        }
        // (past the dispatcher, which takes longer than the allocator; m's device is current)
        const int64_t size[2] = {rows, cols};
        t = at::detail::empty_generic(at::IntArrayRef(size, cols < 0 ? 1 : 2),
                                      c10::hip::HIPCachingAllocatorMasqueradingAsCUDA::get(),
                                      c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt);
        p = t.data_ptr();
    }
};

// the call on the (current) device's current stream; the GIL is free meanwhile
template <typename F>
void run(const Matrix& m, F call) {
    int status, hip = 0;
    void* stream = (void*)c10::hip::getCurrentHIPStreamMasqueradingAsCUDA(m.dev.index()).stream();
    Py_BEGIN_ALLOW_THREADS
    status = call(stream);
    if (status != MOE_OK) hip = moe_last_hip_error();
    Py_END_ALLOW_THREADS
    if (status != MOE_OK)
        refuse(std::string("libmoe: ") + moe_strerror(status) + " (status " + std::to_string(status) + ", hip error " +
               std::to_string(hip) + ")");
}

long integer(PyObject* o, const char* name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " is out of range");
    return v;
}

PyObject* wrap(const at::Tensor& t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
template <typename... T>
PyObject* tuple(const T&... t) {
    PyObject* r = PyTuple_New(sizeof...(t));
    if (!r) throw python_error();
    Py_ssize_t i = 0;
    (PyTuple_SET_ITEM(r, i++, wrap(t)), ...);
    return r;
}

constexpr auto BF16 = at::kBFloat16, F32 = at::kFloat, I8 = at::kChar, U8 = at::kByte;

// (x, weight, eps, res, q_mode, with_y, sum, y, codes, scales) -> (y, sum, codes, scales)
PyObject* py_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 10, "norm");
    const Matrix x = matrix(a[0], BF16, "x");
    const Current on(x.dev);
    const int T = x.rows, H = x.cols;
    const float* w = (const float*)given(a[1], x, H, -1, F32, "weight");
    const double eps = PyFloat_AsDouble(a[2]);
    if (eps == -1.0 && PyErr_Occurred()) throw python_error();
    const void* res = given(a[3], x, T, H, BF16, "res");
    const int q = (int)integer(a[4], "q_mode");
    const int with_y = PyObject_IsTrue(a[5]);
    if (with_y < 0) throw python_error();
    Out sum, y, codes, scales;
    if (res || a[6] != Py_None) sum = Out(a[6], x, T, H, BF16, "sum");
    if (with_y) y = Out(a[7], x, T, H, BF16, "y");
    else if (a[7] != Py_None) refuse("y is written only with with_y");
    if (q == MOE_Q_FP8_G128_POW2) {
        codes = Out(a[8], x, T, H, U8, "codes");
        scales = Out(a[9], x, T, H / 128, U8, "scales");
    } else if (q != MOE_Q_NONE) {
        codes = Out(a[8], x, T, H, I8, "codes");
        scales = Out(a[9], x, T, -1, F32, "scales");
    } else if (a[8] != Py_None || a[9] != Py_None) refuse("codes and scales are written only with a q_mode");
    run(x, [&](void* st) {
        return moe_norm((const uint16_t*)x.t.data_ptr(), (const uint16_t*)res, w, (float)eps, T, H, q, (uint16_t*)sum.p,
                        (uint16_t*)y.p, (uint8_t*)codes.p, scales.p, st);
    });
    return tuple(y.t, sum.t, codes.t, scales.t);
    END_HANDLE_TH_ERRORS
}

// (x, codes, scales) -> (codes, scales)
PyObject* py_quant_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 3, "quant_rows");
    const Matrix x = matrix(a[0], BF16, "x");
    const Current on(x.dev);
    const Out codes(a[1], x, x.rows, x.cols, I8, "codes"), scales(a[2], x, x.rows, -1, F32, "scales");
    run(x, [&](void* st) {
        return moe_quant_rows((const uint16_t*)x.t.data_ptr(), x.rows, x.cols, (int8_t*)codes.p, (float*)scales.p, st);
    });
    return tuple(codes.t, scales.t);
    END_HANDLE_TH_ERRORS
}

// (codes, scales, out) -> out
PyObject* py_dequant_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 3, "dequant_rows");
    const at::Tensor& t = tensor(a[0], "codes");
    const bool i8 = t.defined() && t.scalar_type() == I8;
    const Matrix c = matrix(a[0], i8 ? I8 : U8, "codes");
    const Current on(c.dev);
    const void* scales = i8 ? needed(a[1], c, c.rows, -1, F32, "scales") : needed(a[1], c, c.rows, c.cols / 128, U8, "scales");
    const Out out(a[2], c, c.rows, c.cols, BF16, "out");
    run(c, [&](void* st) {
        return moe_dequant_rows((const uint8_t*)c.t.data_ptr(), scales, c.rows, c.cols,
                                i8 ? MOE_Q_I8_ROW : MOE_Q_FP8_G128_POW2, (uint16_t*)out.p, st);
    });
    return wrap(out.t);
    END_HANDLE_TH_ERRORS
}

// a and b of a product: as many columns, on one device
void fit(const Matrix& a, const Matrix& b, const char* name) {
    if (b.cols != a.cols || b.dev != a.dev) refuse(std::string("a ") + said(a.t) + " and " + name + " " + said(b.t) + " do not fit");
}

// (a, sa, b, sb, bias, add, out, out_dtype) -> out
PyObject* py_gemm_i8(PyObject*, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 8, "gemm_i8");
    const Matrix a = matrix(v[0], I8, "a"), b = matrix(v[2], I8, "b");
    fit(a, b, "b");
    const Current on(a.dev);
    at::ScalarType ot = BF16;
    if (v[7] != Py_None) {
        if (!THPDtype_Check(v[7])) refuse("out_dtype must be a dtype");
        ot = reinterpret_cast<THPDtype*>(v[7])->scalar_type;
    } else if (v[6] != Py_None) ot = tensor(v[6], "out").scalar_type();
    if (ot != BF16 && ot != F32) refuse(std::string("out must be bfloat16 or float32, got ") + c10::toString(ot));
    const int M = a.rows, N = b.rows;
    const void* sa = needed(v[1], a, M, -1, F32, "sa");
    const void* sb = needed(v[3], a, N, -1, F32, "sb");
    const void* bias = given(v[4], a, N, -1, F32, "bias");
    const void* add = given(v[5], a, M, N, ot, "add");
    const Out out(v[6], a, M, N, ot, "out");
    run(a, [&](void* st) {
        return moe_gemm_i8((const int8_t*)a.t.data_ptr(), (const float*)sa, (const int8_t*)b.t.data_ptr(), (const float*)sb,
                           (const float*)bias, add, M, N, a.cols, ot == F32 ? MOE_OUT_F32 : MOE_OUT_BF16, out.p, st);
    });
    return wrap(out.t);
    END_HANDLE_TH_ERRORS
}

// (a, sa, w13, s13, out) -> out
PyObject* py_glu_i8(PyObject*, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 5, "glu_i8");
    const Matrix a = matrix(v[0], I8, "a"), w = matrix(v[2], I8, "w13");
    fit(a, w, "w13");
    const Current on(a.dev);
    if (w.rows % 2) refuse("w13 holds gate and up rows, as many of each: got " + std::to_string(w.rows) + " rows");
    const int M = a.rows, I = w.rows / 2;
    const void* sa = needed(v[1], a, M, -1, F32, "sa");
    const void* s13 = needed(v[3], a, w.rows, -1, F32, "s13");
    const Out out(v[4], a, M, I, BF16, "out");
    run(a, [&](void* st) {
        return moe_glu_i8((const int8_t*)a.t.data_ptr(), (const float*)sa, (const int8_t*)w.t.data_ptr(), (const float*)s13, M,
                          I, a.cols, (uint16_t*)out.p, st);
    });
    return wrap(out.t);
    END_HANDLE_TH_ERRORS
}

// (MoeError,): the exception that refusals raise
PyObject* py_set_error(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 1, "set_error");
    Py_INCREF(a[0]);
    Py_XDECREF(g_error);
    g_error = a[0];
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, (PyCFunction)(void (*)(void))F, METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<py_norm>("norm"), method<py_quant_rows>("quant_rows"),
                           method<py_dequant_rows>("dequant_rows"), method<py_gemm_i8>("gemm_i8"),
                           method<py_glu_i8>("glu_i8"), method<py_set_error>("set_error"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&g_module); }
