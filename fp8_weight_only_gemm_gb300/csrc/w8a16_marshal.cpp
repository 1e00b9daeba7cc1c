// Python-side marshalling of the short calls: the paged cache's append and attention and the
// 4-bit product run for a few microseconds on the GPU, and asking some ten tensors for
// pointers, shapes and strides from Python takes longer than that (an append call: 11.6 us,
// 3 of them the launch). This module asks them directly, makes the checks that only tensors
// allow (types, devices, shapes, contiguity), and calls the C entry that binding.py has
// given it. Everything else is checked by the library.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "w8a16.h"

namespace {

decltype(&w8a16_kv_append) g_append;
decltype(&w8a16_kv_attention) g_attention;
decltype(&w8a16_gemm_w4) g_w4;

const at::Tensor* tensor(PyObject* o, const char* name) {
    if (THPVariable_Check(o)) return &THPVariable_Unpack(o);
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
    return nullptr;
}

bool on(const at::Tensor& t, long index, const char* name) {
    if (t.is_cuda() && t.get_device() == index) return true;
    PyErr_Format(PyExc_ValueError, "all tensors must be on one CUDA device (cuda:%ld); %s is on %s", index, name, t.device().str().c_str());
    return false;
}

// An activation tensor's W8A16_ACT_*, or -1 with an error.
int act_type(const at::Tensor& t, const char* name) {
    if (t.scalar_type() == at::kBFloat16) return W8A16_ACT_BF16;
    if (t.scalar_type() == at::kHalf) return W8A16_ACT_F16;
    PyErr_Format(PyExc_TypeError, "%s must be bfloat16 or float16", name);
    return -1;
}

bool heads(PyObject* o, const char* name, int64_t rows, int64_t dim, at::ScalarType type, long index, w8a16_heads_t* out) {
    const at::Tensor* t = tensor(o, name);
    if (!t) return false;
    if (t->dim() != 3 || t->size(0) != rows || t->size(2) != dim || t->stride(2) != 1) {
        PyErr_Format(PyExc_ValueError, "%s must be [%lld, heads, %lld] with unit stride along the head", name, (long long)rows, (long long)dim);
        return false;
    }
    if (t->scalar_type() != type) {
        PyErr_Format(PyExc_TypeError, "%s must have the type of the others", name);
        return false;
    }
    if (!on(*t, index, name)) return false;
    *out = {t->data_ptr(), t->stride(0), t->stride(1), static_cast<uint32_t>(t->size(1))};
    return true;
}

bool ints(const at::Tensor& t, int64_t n, long index, const char* name) {
    if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s must be contiguous int32 [%lld]", name, (long long)n);
        return false;
    }
    return on(t, index, name);
}

bool batch(PyObject* table_o, PyObject* lens_o, PyObject* cu_o, PyObject* max_q_o, int64_t rows, long index, w8a16_kv_batch_t* out) {
    const at::Tensor *table = tensor(table_o, "page_table"), *lens = table ? tensor(lens_o, "lens") : nullptr;
    if (!lens) return false;
    if (table->dim() != 2 || table->scalar_type() != at::kInt || table->stride(1) != 1) {
        PyErr_SetString(PyExc_ValueError, "page_table must be int32 [batch, max_pages] with contiguous rows");
        return false;
    }
    const int64_t B = table->size(0);
    if (!on(*table, index, "page_table") || !ints(*lens, B, index, "lens")) return false;
    const int32_t* cu = nullptr;
    int64_t max_q = 0;
    if (cu_o != Py_None) {
        const at::Tensor* t = tensor(cu_o, "cu_q");
        if (!t || !ints(*t, B + 1, index, "cu_q")) return false;
        cu = t->const_data_ptr<int32_t>();
        if (max_q_o == Py_None) {
            PyErr_SetString(PyExc_ValueError, "cu_q needs max_q, the most rows of one sequence");
            return false;
        }
    }
    if (max_q_o != Py_None) {
        max_q = PyLong_AsLongLong(max_q_o);
        if (max_q == -1 && PyErr_Occurred()) return false;
        if (max_q < 0 || max_q > 0xFFFFFFFFll) {
            PyErr_SetString(PyExc_ValueError, "max_q is out of range");
            return false;
        }
    } else if (B == 0 || rows % B) {
        PyErr_Format(PyExc_ValueError, "%lld rows do not divide among %lld sequences: pass cu_q and max_q", (long long)rows, (long long)B);
        return false;
    } else {
        max_q = rows / B;
    }
    if (rows > 0xFFFFFFFFll || B > 0xFFFFFFFFll || table->size(1) > 0xFFFFFFFFll) {
        PyErr_SetString(PyExc_ValueError, "too many rows, sequences or pages");
        return false;
    }
    *out = {table->const_data_ptr<int32_t>(), lens->const_data_ptr<int32_t>(), cu, table->stride(0), static_cast<uint32_t>(table->size(1)),
            static_cast<uint32_t>(B), static_cast<uint32_t>(rows), static_cast<uint32_t>(max_q)};
    return true;
}

// The stream of a call: the given handle, or the device's current one.
bool stream_of(PyObject* o, long index, w8a16_stream_t* out) {
    if (o == Py_None) {
        *out = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
        return true;
    }
    *out = static_cast<w8a16_stream_t>(PyLong_AsVoidPtr(o));
    return !PyErr_Occurred();
}

// Runs `f` on device `index` without the interpreter lock; C++ errors become Python's. The lock is back
// before an exception is, whoever throws it.
struct Unlocked {
    PyThreadState* const state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F>
PyObject* run(long index, F&& f) {
    int rc = 0;
    try {
        c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
        Unlocked unlocked;
        rc = f();
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
    return PyLong_FromLong(rc);
}

bool count(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}

// Tensor methods throw on what they do not support; no exception crosses into Python.
template <PyObject* (*F)(PyObject* const*)>
PyObject* guarded(PyObject* const* a) {
    try {
        return F(a);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// (cache address, device, head_dim, k, v, page_table, lens, cu_q, max_q, q, q_out, cos, sin, interleaved, stream)
PyObject* kv_append_impl(PyObject* const* a) {
    const auto* cache = static_cast<const w8a16_kv_cache_t*>(PyLong_AsVoidPtr(a[0]));
    const long index = PyLong_AsLong(a[1]), dim = PyLong_AsLong(a[2]);
    if (PyErr_Occurred()) return nullptr;
    if ((a[11] == Py_None) != (a[12] == Py_None)) {
        PyErr_SetString(PyExc_ValueError, "cos and sin go together: one of them is None");
        return nullptr;
    }
    const int interleaved = PyObject_IsTrue(a[13]);
    if (interleaved < 0) return nullptr;
    const at::Tensor* k = tensor(a[3], "k");
    if (!k) return nullptr;
    const int act = act_type(*k, "k");
    if (act < 0) return nullptr;
    const at::ScalarType type = k->scalar_type();
    const int64_t rows = k->dim() ? k->size(0) : 0;
    w8a16_kv_batch_t b;
    w8a16_heads_t kd, vd, qd{}, od{};
    if (!batch(a[5], a[6], a[7], a[8], rows, index, &b) || !heads(a[3], "k", rows, dim, type, index, &kd) ||
        !heads(a[4], "v", rows, dim, type, index, &vd))
        return nullptr;
    const bool with_q = a[9] != Py_None;
    if (with_q && (!heads(a[9], "q", rows, dim, type, index, &qd) || !heads(a[10], "q_out", rows, dim, type, index, &od))) return nullptr;
    w8a16_rope_t rope{nullptr, nullptr, 0, 0, 0};
    if (a[11] != Py_None) {
        const at::Tensor *c = tensor(a[11], "cos"), *s = c ? tensor(a[12], "sin") : nullptr;
        if (!s) return nullptr;
        if (c->dim() != 2 || s->sizes() != c->sizes() || c->scalar_type() != at::kFloat || s->scalar_type() != at::kFloat ||
            !c->is_contiguous() || !s->is_contiguous()) {
            PyErr_SetString(PyExc_ValueError, "cos and sin must be contiguous float32 [positions, rotary_dim / 2]");
            return nullptr;
        }
        if (!on(*c, index, "cos") || !on(*s, index, "sin")) return nullptr;
        rope = {c->const_data_ptr<float>(), s->const_data_ptr<float>(), static_cast<uint32_t>(c->size(0)), static_cast<uint32_t>(2 * c->size(1)),
                interleaved ? 1u : 0u};
    }
    w8a16_stream_t stream;
    if (!stream_of(a[14], index, &stream)) return nullptr;
    return run(index, [&] {
        return g_append(cache, &b, static_cast<uint32_t>(act), &kd, &vd, with_q ? &qd : nullptr, with_q ? &od : nullptr, &rope, stream);
    });
}

// (cache address, device, head_dim, q, out, page_table, lens, cu_q, max_q, softmax_scale, workspace, stream)
PyObject* kv_attention_impl(PyObject* const* a) {
    const auto* cache = static_cast<const w8a16_kv_cache_t*>(PyLong_AsVoidPtr(a[0]));
    const long index = PyLong_AsLong(a[1]), dim = PyLong_AsLong(a[2]);
    const double scale = PyFloat_AsDouble(a[9]);
    if (PyErr_Occurred()) return nullptr;
    const at::Tensor* q = tensor(a[3], "q");
    if (!q) return nullptr;
    const int act = act_type(*q, "q");
    if (act < 0) return nullptr;
    const int64_t rows = q->dim() ? q->size(0) : 0;
    w8a16_kv_batch_t b;
    w8a16_heads_t qd, od;
    if (!batch(a[5], a[6], a[7], a[8], rows, index, &b) || !heads(a[3], "q", rows, dim, q->scalar_type(), index, &qd) ||
        !heads(a[4], "out", rows, dim, q->scalar_type(), index, &od))
        return nullptr;
    const at::Tensor* ws = tensor(a[10], "workspace");
    if (!ws) return nullptr;
    if (ws->scalar_type() != at::kByte || !ws->is_contiguous()) {
        PyErr_SetString(PyExc_ValueError, "workspace must be a contiguous uint8 tensor");
        return nullptr;
    }
    if (!on(*ws, index, "workspace")) return nullptr;
    w8a16_stream_t stream;
    if (!stream_of(a[11], index, &stream)) return nullptr;
    void* const ws_ptr = ws->data_ptr();
    const uint64_t ws_bytes = static_cast<uint64_t>(ws->numel());
    return run(index, [&] { return g_attention(cache, &b, static_cast<uint32_t>(act), &qd, &od, static_cast<float>(scale), ws_ptr, ws_bytes, stream); });
}

// (A, W, scale, C, zeros, flags, stream)
PyObject* gemm_w4_impl(PyObject* const* a) {
    const at::Tensor *A = tensor(a[0], "A"), *W = A ? tensor(a[1], "W") : nullptr, *S = W ? tensor(a[2], "scale") : nullptr,
                     *C = S ? tensor(a[3], "C") : nullptr, *Z = C && a[4] != Py_None ? tensor(a[4], "zeros") : nullptr;
    if (!C || (a[4] != Py_None && !Z)) return nullptr;
    const int act = act_type(*A, "A");
    if (act < 0) return nullptr;
    const auto refuse = [](PyObject* type, const char* what) -> PyObject* {
        PyErr_SetString(type, what);
        return nullptr;
    };
    if (A->dim() != 2 || A->stride(1) != 1) return refuse(PyExc_ValueError, "A must be [M, K] with contiguous rows");
    const int64_t M = A->size(0), K = A->size(1);
    if (W->dim() != 2 || W->scalar_type() != at::kByte || !W->is_contiguous() || W->size(1) * 2 != K)
        return refuse(PyExc_ValueError, "W must be contiguous uint8 [N, K/2] (two codes a byte)");
    const int64_t N = W->size(0);
    if (S->dim() != 2 || S->size(0) != N || S->size(1) < 1 || K % S->size(1) || !S->is_contiguous())
        return refuse(PyExc_ValueError, "scale must be contiguous [N, K/group]");
    if (S->scalar_type() != at::kFloat && S->scalar_type() != A->scalar_type())
        return refuse(PyExc_TypeError, "scale must be float32 or of A's type");
    if (Z && (Z->scalar_type() != at::kByte || Z->sizes() != S->sizes() || !Z->is_contiguous()))
        return refuse(PyExc_ValueError, "zeros must be contiguous uint8 of scale's shape");
    if (C->scalar_type() != A->scalar_type() || C->dim() != 2 || C->stride(1) != 1 || C->size(0) != M || C->size(1) < N)
        return refuse(PyExc_ValueError, "C must be [M, >=N] of A's type with contiguous rows");
    if (!A->is_cuda()) return refuse(PyExc_ValueError, "all tensors must be on a CUDA device");
    const long index = A->get_device();
    if (!on(*W, index, "W") || !on(*S, index, "scale") || !on(*C, index, "C") || (Z && !on(*Z, index, "zeros"))) return nullptr;
    if (M > 0xFFFFFFFFll || N > 0xFFFFFFFFll || K > 0xFFFFFFFFll || A->stride(0) > 0xFFFFFFFFll || C->stride(0) > 0xFFFFFFFFll)
        return refuse(PyExc_ValueError, "sizes and row pitches must be below 2^32");
    const unsigned long flags = PyLong_AsUnsignedLong(a[5]);
    w8a16_stream_t stream;
    if (PyErr_Occurred() || !stream_of(a[6], index, &stream)) return nullptr;
    const void *const Ap = A->data_ptr(), *const Wp = W->data_ptr(), *const Sp = S->data_ptr(), *const Zp = Z ? Z->data_ptr() : nullptr;
    void* const Cp = C->data_ptr();
    return run(index, [&] {
        return g_w4(Ap, static_cast<uint32_t>(A->stride(0)), static_cast<uint32_t>(act), Wp, Sp,
                    S->scalar_type() == at::kFloat ? W8A16_W4_SCALE_F32 : W8A16_W4_SCALE_ACT, Zp, static_cast<uint32_t>(K / S->size(1)), Cp,
                    static_cast<uint32_t>(C->stride(0)), static_cast<uint32_t>(M), static_cast<uint32_t>(N), static_cast<uint32_t>(K),
                    static_cast<uint32_t>(flags), stream);
    });
}

PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) { return count(n, 15) ? guarded<kv_append_impl>(a) : nullptr; }
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t n) { return count(n, 12) ? guarded<kv_attention_impl>(a) : nullptr; }
PyObject* gemm_w4(PyObject*, PyObject* const* a, Py_ssize_t n) { return count(n, 7) ? guarded<gemm_w4_impl>(a) : nullptr; }

// The addresses of w8a16_kv_append, w8a16_kv_attention and w8a16_gemm_w4.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count(n, 3)) return nullptr;
    g_append = reinterpret_cast<decltype(g_append)>(PyLong_AsVoidPtr(a[0]));
    g_attention = reinterpret_cast<decltype(g_attention)>(PyLong_AsVoidPtr(a[1]));
    g_w4 = reinterpret_cast<decltype(g_w4)>(PyLong_AsVoidPtr(a[2]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
                         {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_append)), METH_FASTCALL, nullptr},
                         {"kv_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_attention)), METH_FASTCALL, nullptr},
                         {"gemm_w4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gemm_w4)), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "w8a16_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_w8a16_marshal() { return PyModule_Create(&module); }
