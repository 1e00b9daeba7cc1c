// Python-side marshalling of the short calls: the paged cache's append and attention, the
// 4-bit product and the norms run for a few microseconds on the GPU, and asking some ten tensors for
// pointers, shapes and strides from Python takes longer than that (an append call: 11.6 us,
// 3 of them the launch). This module asks them directly, makes the checks that only tensors
// allow (types, devices, shapes, contiguity), and calls the C entry that binding.py has
// given it. Everything else is checked by the library.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "w8a16.h"

namespace {

decltype(&w8a16_kv_append) g_append;
decltype(&w8a16_kv_append_axes) g_append_axes;
decltype(&w8a16_kv_attention) g_attention;
decltype(&w8a16_kv_attention_ex) g_attention_ex;
decltype(&w8a16_gemm_w4) g_w4;
decltype(&w8a16_norm_residual) g_norm;

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

// (cache address, device, head_dim, k, v, page_table, lens, cu_q, max_q, q, q_out, cos, sin, interleaved, stream), and with
// AXES (positions, axes, pairs, address of pair_axis) behind them
template <bool AXES>
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
    if constexpr (AXES) {
        const at::Tensor* const pos = tensor(a[15], "positions");
        if (!pos) return nullptr;
        const long axes = PyLong_AsLong(a[16]), pairs = PyLong_AsLong(a[17]);
        const auto* const of = static_cast<const uint8_t*>(PyLong_AsVoidPtr(a[18]));
        if (PyErr_Occurred()) return nullptr;
        if (rope.rotary_dim != 2 * static_cast<uint64_t>(pairs)) {
            PyErr_Format(PyExc_ValueError, "axes are of %ld rotary pairs, cos and sin of %u", pairs, rope.rotary_dim / 2);
            return nullptr;
        }
        if (pos->scalar_type() != at::kInt || pos->dim() != 2 || pos->size(0) < axes || pos->size(1) != rows || pos->stride(1) != 1) {
            PyErr_Format(PyExc_ValueError, "positions must be int32 [%ld, %lld] with contiguous rows", axes, (long long)rows);
            return nullptr;
        }
        if (!on(*pos, index, "positions")) return nullptr;
        w8a16_rope_axes_t x;
        x.positions = pos->const_data_ptr<int32_t>(), x.axes = static_cast<uint32_t>(axes);
        x.axis_stride = axes > 1 ? pos->stride(0) : rows;
        std::memcpy(x.pair_axis, of, sizeof x.pair_axis);
        return run(index, [&] {
            return g_append_axes(cache, &b, static_cast<uint32_t>(act), &kd, &vd, with_q ? &qd : nullptr, with_q ? &od : nullptr, &rope, &x, stream);
        });
    }
    return run(index, [&] {
        return g_append(cache, &b, static_cast<uint32_t>(act), &kd, &vd, with_q ? &qd : nullptr, with_q ? &od : nullptr, &rope, stream);
    });
}

// (cache address, device, head_dim, q, out, page_table, lens, cu_q, max_q, softmax_scale, workspace, stream), and with SPAN
// (window, sinks, prefix_pages, prefix_len) behind them
template <bool SPAN>
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
    if constexpr (SPAN) {
        w8a16_kv_span_t span{0, 0, nullptr, 0, 0};
        const auto number = [&](PyObject* o, const char* name, uint32_t* to) {
            const long long v = PyLong_AsLongLong(o);
            if (v == -1 && PyErr_Occurred()) return false;
            if (v < 0 || v > 0xFFFFFFFFll) {
                PyErr_Format(PyExc_ValueError, "%s is out of range", name);
                return false;
            }
            *to = static_cast<uint32_t>(v);
            return true;
        };
        if (!number(a[12], "window", &span.window) || !number(a[13], "sinks", &span.sinks) || !number(a[15], "prefix_len", &span.prefix_len)) return nullptr;
        if (a[14] != Py_None) {
            const at::Tensor* const pages = tensor(a[14], "prefix_pages");
            if (!pages) return nullptr;
            if (pages->scalar_type() != at::kInt || pages->dim() != 1 || pages->size(0) < 1 || pages->size(0) > 0xFFFFFFFFll || !pages->is_contiguous()) {
                PyErr_SetString(PyExc_ValueError, "prefix_pages must be contiguous int32 [pages]");
                return nullptr;
            }
            if (!on(*pages, index, "prefix_pages")) return nullptr;
            span.prefix_pages = pages->const_data_ptr<int32_t>(), span.num_prefix_pages = static_cast<uint32_t>(pages->size(0));
        }
        return run(index, [&] {
            return g_attention_ex(cache, &b, static_cast<uint32_t>(act), &qd, &od, &span, static_cast<float>(scale), ws_ptr, ws_bytes, stream);
        });
    }
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

// (x, residual, out, out_scale, residual_out, weight, bias, post_weight, post_bias, gate, scale, eps, kind, flags, stream)
PyObject* norm_residual_impl(PyObject* const* a) {
    const auto refuse = [](PyObject* type, const char* what) -> PyObject* {
        PyErr_SetString(type, what);
        return nullptr;
    };
    const at::Tensor* x = tensor(a[0], "x");
    if (!x) return nullptr;
    const int act = act_type(*x, "x");
    if (act < 0) return nullptr;
    if (x->dim() != 2 || x->stride(1) != 1) return refuse(PyExc_ValueError, "x must be [M, H] with contiguous rows");
    if (!x->is_cuda()) return refuse(PyExc_ValueError, "all tensors must be on a CUDA device");
    const int64_t M = x->size(0), H = x->size(1);
    const long index = x->get_device();
    if (M > 0xFFFFFFFFll || H > 0xFFFFFFFFll) return refuse(PyExc_ValueError, "sizes must be below 2^32");
    // An optional tensor; false with an error set.
    const auto optional = [&](int i, const char* name, const at::Tensor** t) {
        *t = nullptr;
        if (a[i] == Py_None) return true;
        *t = tensor(a[i], name);
        return *t != nullptr && on(**t, index, name);
    };
    const at::Tensor *r, *y, *ys, *h, *w, *b, *pw, *pb, *g;
    if (!optional(1, "residual", &r) || !optional(2, "out", &y) || !optional(3, "out_scale", &ys) || !optional(4, "residual_out", &h) ||
        !optional(5, "weight", &w) || !optional(6, "bias", &b) || !optional(7, "post_weight", &pw) || !optional(8, "post_bias", &pb) ||
        !optional(9, "gate", &g))
        return nullptr;
    const auto rows = [&](const at::Tensor* t) { return !t || (t->dim() == 2 && t->size(0) == M && t->size(1) == H && t->stride(1) == 1); };
    if (!rows(r) || !rows(h)) return refuse(PyExc_ValueError, "residual and residual_out must be [M, H] with contiguous rows");
    const auto act_or_f32 = [&](const at::Tensor* t) { return !t || t->scalar_type() == at::kFloat || t->scalar_type() == x->scalar_type(); };
    if (!act_or_f32(r) || !act_or_f32(h)) return refuse(PyExc_TypeError, "residual and residual_out must be float32 or of x's type");
    if (r && h && r->scalar_type() != h->scalar_type()) return refuse(PyExc_TypeError, "residual and residual_out must have one type");
    if (ys) {
        if (!y || (y->scalar_type() != at::kByte && y->scalar_type() != at::kFloat8_e4m3fn))
            return refuse(PyExc_TypeError, "quantised, out must be E4M3 codes (uint8 or float8_e4m3fn)");
        // (an H that is no multiple of 128 is the library's to report; it knows a quantised call by the pointer)
        if (ys->scalar_type() != at::kFloat || ys->dim() != 2 || (H % 128 == 0 && ys->size(0) * 128 != H) || ys->size(1) < M ||
            ys->stride(1) != 1 || ys->data_ptr() == nullptr)
            return refuse(PyExc_ValueError, "out_scale must be float32 [H/128, >=M] with contiguous rows");
    } else if (y && y->scalar_type() != x->scalar_type()) {
        return refuse(PyExc_TypeError, "out must be of x's type");
    }
    if (!rows(y)) return refuse(PyExc_ValueError, "out must be [M, H] with contiguous rows");
    const at::Tensor* const weights[4] = {w, b, pw, pb};
    const at::Tensor* first = nullptr;
    for (const at::Tensor* t : weights) {
        if (!t) continue;
        if (t->dim() != 1 || t->size(0) != H || !t->is_contiguous()) return refuse(PyExc_ValueError, "weights and biases must be contiguous [H]");
        if (!act_or_f32(t) || (first && first->scalar_type() != t->scalar_type()))
            return refuse(PyExc_TypeError, "weights and biases must have one type, float32 or x's");
        first = t;
    }
    // (without rows its pointer would be NULL, which is a call without a gate)
    if (g && (g->dim() != 2 || g->size(0) < 1 || g->size(1) != H || g->stride(1) != 1 || g->size(0) > 0xFFFFFFFFll || g->scalar_type() != x->scalar_type()))
        return refuse(PyExc_ValueError, "gate must be [rows, H] of x's type with contiguous rows");
    const double scale = PyFloat_AsDouble(a[10]), eps = PyFloat_AsDouble(a[11]);
    const unsigned long kind = PyLong_AsUnsignedLong(a[12]), flags = PyLong_AsUnsignedLong(a[13]);
    w8a16_stream_t stream;
    if (PyErr_Occurred() || !stream_of(a[14], index, &stream)) return nullptr;
    const auto ptr = [](const at::Tensor* t) { return t ? t->data_ptr() : nullptr; };
    // a single row's pitch is not used: of a [1, H] view it may be anything
    const auto pitch = [](const at::Tensor* t, int64_t every) {
        return !t ? 0 : t->size(0) > 1 ? t->stride(0) : (t->size(1) + every - 1) / every * every;
    };
    w8a16_norm_t n;
    n.x = ptr(x), n.residual = ptr(r), n.residual_out = ptr(h), n.out = ptr(y), n.out_scale = static_cast<float*>(ptr(ys));
    n.weight = ptr(w), n.bias = ptr(b), n.post_weight = ptr(pw), n.post_bias = ptr(pb), n.gate = ptr(g);
    n.x_stride = pitch(x, 8), n.residual_stride = pitch(r, 8), n.residual_out_stride = pitch(h, 8), n.out_stride = pitch(y, 16);
    n.out_scale_stride = ys ? (ys->size(0) > 1 ? ys->stride(0) : (M + 3) / 4 * 4) : 0, n.gate_stride = pitch(g, 8);
    n.M = static_cast<uint32_t>(M), n.H = static_cast<uint32_t>(H), n.gate_rows = g ? static_cast<uint32_t>(g->size(0)) : 0;
    n.act_dtype = static_cast<uint32_t>(act), n.residual_f32 = (r ? r : h) && (r ? r : h)->scalar_type() == at::kFloat;
    n.weight_f32 = first && first->scalar_type() == at::kFloat, n.kind = static_cast<uint32_t>(kind);
    n.eps = static_cast<float>(eps), n.scale = static_cast<float>(scale);
    return run(index, [&] { return g_norm(&n, static_cast<uint32_t>(flags), stream); });
}

PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) { return count(n, 15) ? guarded<kv_append_impl<false>>(a) : nullptr; }
PyObject* kv_append_axes(PyObject*, PyObject* const* a, Py_ssize_t n) { return count(n, 19) ? guarded<kv_append_impl<true>>(a) : nullptr; }
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t n) { return count(n, 12) ? guarded<kv_attention_impl<false>>(a) : nullptr; }
PyObject* kv_attention_ex(PyObject*, PyObject* const* a, Py_ssize_t n) { return count(n, 16) ? guarded<kv_attention_impl<true>>(a) : nullptr; }
PyObject* gemm_w4(PyObject*, PyObject* const* a, Py_ssize_t n) { return count(n, 7) ? guarded<gemm_w4_impl>(a) : nullptr; }
PyObject* norm_residual(PyObject*, PyObject* const* a, Py_ssize_t n) { return count(n, 15) ? guarded<norm_residual_impl>(a) : nullptr; }

// The addresses of w8a16_kv_append, w8a16_kv_attention, w8a16_gemm_w4, w8a16_norm_residual, w8a16_kv_append_axes and
// w8a16_kv_attention_ex.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count(n, 6)) return nullptr;
    g_append = reinterpret_cast<decltype(g_append)>(PyLong_AsVoidPtr(a[0]));
    g_attention = reinterpret_cast<decltype(g_attention)>(PyLong_AsVoidPtr(a[1]));
    g_w4 = reinterpret_cast<decltype(g_w4)>(PyLong_AsVoidPtr(a[2]));
    g_norm = reinterpret_cast<decltype(g_norm)>(PyLong_AsVoidPtr(a[3]));
    g_append_axes = reinterpret_cast<decltype(g_append_axes)>(PyLong_AsVoidPtr(a[4]));
    g_attention_ex = reinterpret_cast<decltype(g_attention_ex)>(PyLong_AsVoidPtr(a[5]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
                         {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_append)), METH_FASTCALL, nullptr},
                         {"kv_append_axes", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_append_axes)), METH_FASTCALL, nullptr},
                         {"kv_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_attention)), METH_FASTCALL, nullptr},
                         {"kv_attention_ex", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_attention_ex)), METH_FASTCALL, nullptr},
                         {"gemm_w4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gemm_w4)), METH_FASTCALL, nullptr},
                         {"norm_residual", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm_residual)), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "w8a16_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_w8a16_marshal() { return PyModule_Create(&module); }
