// calls.cpp -- the host side of the rotary positions' and the paged cache's calls, as a Python module: checks of
// tensors, outputs and workspaces from PyTorch's allocator, and the C entry points of include/tsa_cache.h.
//
// These calls serve single tokens, whose kernels take 3 to 20 us: marshalled in Python (ctypes) a call took 18 to
// 25 us of the host, here it takes 7 to 9.  The rotation's gradient is a C++ node of the autograd graph, so that a
// backward pass runs it without the interpreter: a training step's call and gradient took 250 us with a Python
// node, 150 to 160 here, where PyTorch's own x * 2 and its gradient take 100.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cmath>
#include <stdexcept>
#include <string>

#include "tsa_cache.h"

namespace {

using at::Tensor;

// What a call of the library returned, where it was not TSA_OK.
struct StatusError : std::runtime_error {
    tsa_status status;
    std::string where;
    StatusError(tsa_status s, const char *w)
        : std::runtime_error(std::string(w) + ": " + tsa_status_string(s)), status(s), where(w) {}
};

void check(tsa_status s, const char *where) {
    if (s != TSA_OK) throw StatusError(s, where);
}

tsa_stream_t stream_of(const Tensor &t) {
    return reinterpret_cast<tsa_stream_t>(c10::cuda::getCurrentCUDAStream(t.device().index()).stream());
}

tsa_dtype dtype_of(const Tensor &t) {
    const auto type = t.scalar_type();
    TORCH_CHECK_TYPE(type == at::kHalf || type == at::kBFloat16, "expected float16 or bfloat16, got ", type);
    return type == at::kHalf ? TSA_F16 : TSA_BF16;
}

// A tensor [B, heads, tokens, D] of contiguous rows; of `like`'s type, device, batch, tokens and D.
void check_rows(const char *name, const Tensor &t, const Tensor *like = nullptr) {
    TORCH_CHECK_VALUE(t.dim() == 4 && t.is_cuda() && (t.stride(3) == 1 || t.size(3) == 1), name,
                      " must be a CUDA tensor [B, heads, tokens, D] with contiguous rows");
    if (like) {
        TORCH_CHECK_VALUE(t.scalar_type() == like->scalar_type() && t.device() == like->device() &&
                              t.size(0) == like->size(0) && t.size(2) == like->size(2) && t.size(3) == like->size(3),
                          name, " must have the type, device, batch, tokens and row length of the others");
    }
}

// A tensor that a call writes in place: there is no gradient of that.
void check_written(const char *name, const Tensor &t) {
    TORCH_CHECK_VALUE(!t.defined() || !t.requires_grad() || !c10::GradMode::is_enabled(), name,
                      " requires a gradient, and is written in place, without one");
}

// It was written: autograd will notice if it had kept it for a backward pass.  (Inference tensors keep no versions.)
void written_to(const Tensor &t) {
    if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// `t`, or a new contiguous tensor shaped as `like`.
Tensor rows_out(const char *name, const Tensor &t, const Tensor &like) {
    if (!t.defined()) return at::empty(like.sizes(), like.options());
    check_rows(name, t, &like);
    check_written(name, t);
    TORCH_CHECK_VALUE(t.sizes() == like.sizes(), name, " must have the shape ", like.sizes());
    return t;
}

const int32_t *check_list(const char *name, const Tensor &t, at::IntArrayRef shape, const Tensor &like) {
    TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.sizes() == shape && t.device() == like.device() && t.is_contiguous(), name,
                      " must be a contiguous int32 tensor of shape ", shape, " on the inputs' device");
    return t.const_data_ptr<int32_t>();
}

void put_strides(int64_t *to, const Tensor &t) {
    for (int i = 0; i < 3; ++i) to[i] = t.defined() ? t.stride(i) : 0;
}

const void *data(const Tensor &t) { return t.defined() ? t.const_data_ptr() : nullptr; }
void *written(const Tensor &t) { return t.defined() ? t.mutable_data_ptr() : nullptr; }

struct Frequencies {
    const double *values;
    int64_t n;
};

// --- rotary positions ---

std::array<Tensor, 2> rotary(const Tensor &Q, const Tensor &K, Frequencies f, const Tensor &positions, bool interleaved,
                             double magnitude, bool inverse, const Tensor &out, const Tensor &out_k) {
    check_rows("Q", Q);
    const int64_t B = Q.size(0), S = Q.size(2);
    if (K.defined()) check_rows("K", K, &Q);
    TORCH_CHECK_VALUE(K.defined() || !out_k.defined(), "out_k without K");
    if (positions.defined()) {
        TORCH_CHECK_VALUE(positions.scalar_type() == at::kInt && positions.device() == Q.device() && positions.is_contiguous() &&
                              (positions.sizes() == at::IntArrayRef{S} || positions.sizes() == at::IntArrayRef{B, S}),
                          "positions must be a contiguous int32 tensor [S] or [B, S] on the inputs' device");
    }
    const tsa_dtype dtype = dtype_of(Q);
    const Tensor q = rows_out("out", out, Q), k = K.defined() ? rows_out("out_k", out_k, K) : Tensor();
    int64_t strides[12];
    put_strides(strides, Q);
    put_strides(strides + 3, K);
    put_strides(strides + 6, q);
    put_strides(strides + 9, k);
    check(tsa_rotary(Q.const_data_ptr(), data(K), strides, static_cast<const int32_t *>(data(positions)),
                     positions.defined() && positions.dim() == 2 ? B : 1, f.values, 2 * f.n, interleaved, (float)magnitude,
                     inverse, written(q), written(k), dtype, B, Q.size(1),
                     K.defined() ? K.size(1) : 0, S, Q.size(3), stream_of(Q)),
          "tsa_rotary");
    written_to(out);
    written_to(out_k);
    return {q, k};
}

// `t` as the rotation reads it: whole rows, multiples of 16 bytes apart and from such a boundary on.  (The
// gradient that reaches a backward pass may be any view.)
Tensor readable(const Tensor &t) {
    bool fine = t.stride(3) == 1 && reinterpret_cast<uintptr_t>(t.const_data_ptr()) % 16 == 0;
    for (int i = 0; i < 3; ++i) fine = fine && (t.size(i) == 1 || t.stride(i) % 8 == 0);
    return fine ? t : t.clone(at::MemoryFormat::Contiguous);
}

// Whether `t` is dense with tokens before heads, which is then its gradient's layout too.
bool tokens_first(const Tensor &t) {
    const int64_t B = t.size(0), H = t.size(1), S = t.size(2), D = t.size(3);
    return t.dim() == 4 && t.stride(3) == 1 && t.stride(1) == D && t.stride(2) == H * D && (B == 1 || t.stride(0) == S * H * D);
}

struct Rotary : torch::autograd::Function<Rotary> {
    static torch::autograd::variable_list forward(torch::autograd::AutogradContext *ctx, const Tensor &Q,
                                                  const std::optional<Tensor> &K, const std::optional<Tensor> &positions,
                                                  const std::vector<double> &f, bool interleaved, double magnitude,
                                                  bool inverse) {
        const Tensor k = K.has_value() ? *K : Tensor(), at = positions.has_value() ? *positions : Tensor();
        check_rows("Q", Q);
        if (k.defined()) check_rows("K", k, &Q);
        // the frequencies are a copy, and a change of positions in place before the backward is noticed
        ctx->saved_data["f"] = f;
        ctx->saved_data["interleaved"] = interleaved;
        ctx->saved_data["magnitude"] = magnitude;
        ctx->saved_data["inverse"] = inverse;
        ctx->saved_data["layouts"] = (int64_t)tokens_first(Q) | (int64_t)(k.defined() && tokens_first(k)) << 1;
        ctx->saved_data["both"] = k.defined();
        ctx->saved_data["positions"] = at.defined();
        if (at.defined()) ctx->save_for_backward({at});
        ctx->set_materialize_grads(false);
        const auto r = rotary(readable(Q), k.defined() ? readable(k) : k, {f.data(), (int64_t)f.size()}, at, interleaved,
                              magnitude, inverse, Tensor(), Tensor());
        return k.defined() ? torch::autograd::variable_list{r[0], r[1]} : torch::autograd::variable_list{r[0]};
    }

    // The rotation back, which is one of these itself where its own gradient is wanted.
    static torch::autograd::variable_list backward(torch::autograd::AutogradContext *ctx,
                                                   torch::autograd::variable_list grads) {
        const std::vector<double> f = ctx->saved_data["f"].toDoubleVector();
        const bool interleaved = ctx->saved_data["interleaved"].toBool(), inverse = !ctx->saved_data["inverse"].toBool();
        const double magnitude = ctx->saved_data["magnitude"].toDouble();
        const int64_t layouts = ctx->saved_data["layouts"].toInt();
        const Tensor at = ctx->saved_data["positions"].toBool() ? ctx->get_saved_variables()[0] : Tensor();
        torch::autograd::variable_list back(7);  // one per argument of forward
        int wanted[2], n = 0;
        for (int i = 0; i < (ctx->saved_data["both"].toBool() ? 2 : 1); ++i)
            if (grads[i].defined() && ctx->needs_input_grad(i)) wanted[n++] = i;
        if (n == 0) return back;
        if (c10::GradMode::is_enabled()) {
            // (a copy of a gradient in another layout is part of the graph)
            const auto r = Rotary::apply(readable(grads[wanted[0]]),
                                         n == 2 ? std::optional<Tensor>(readable(grads[wanted[1]])) : std::nullopt,
                                         at.defined() ? std::optional<Tensor>(at) : std::nullopt, f, interleaved, magnitude,
                                         inverse);
            for (int i = 0; i < n; ++i) back[wanted[i]] = r[i];
            return back;
        }
        Tensor g[2], out[2];
        for (int i = 0; i < n; ++i) {
            g[i] = readable(grads[wanted[i]]);
            if (layouts >> wanted[i] & 1)
                out[i] = at::empty({g[i].size(0), g[i].size(2), g[i].size(1), g[i].size(3)}, g[i].options()).transpose(1, 2);
        }
        const auto r = rotary(g[0], g[1], {f.data(), (int64_t)f.size()}, at, interleaved, magnitude, inverse, out[0], out[1]);
        for (int i = 0; i < n; ++i) back[wanted[i]] = r[i];
        return back;
    }
};

// --- the paged cache ---

struct Pages {
    int64_t pages, size, k_stride, v_stride, most;
    const int32_t *table, *lens;
};

Pages check_pages(const Tensor &Kc, const Tensor &Vc, const Tensor &table, const Tensor &lens, int64_t B, int64_t HK, int64_t D,
                  const Tensor &like) {
    TORCH_CHECK_VALUE(Kc.dim() == 4 && Kc.size(1) == HK && Kc.size(3) == D, "K_cache must be [pages, ", HK, ", page_size, ", D, "]");
    const int64_t size = Kc.size(2);
    for (const Tensor *t : {&Kc, &Vc}) {
        TORCH_CHECK_VALUE(t->sizes() == Kc.sizes() && t->scalar_type() == like.scalar_type() && t->device() == like.device() &&
                              (HK == 1 || t->stride(1) == size * D) && t->stride(2) == D && t->stride(3) == 1,
                          t == &Kc ? "K_cache" : "V_cache",
                          " must be a [pages, HK, page_size, D] tensor of the inputs' type and device, its pages contiguous");
    }
    TORCH_CHECK_VALUE(table.dim() == 2, "page_table must be a contiguous int32 tensor [B, pages] on the inputs' device");
    Pages p = {Kc.size(0), size, Kc.stride(0), Vc.stride(0), table.size(1), nullptr, nullptr};
    p.table = check_list("page_table", table, {B, p.most}, like);
    p.lens = check_list("seq_lens", lens, {B}, like);
    return p;
}

Tensor paged_append(const Tensor &Q, const Tensor &K, const Tensor &V, const Tensor &Kc, const Tensor &Vc, const Tensor &table,
                    const Tensor &lens, const Tensor &counts, const Frequencies *f, bool interleaved, double magnitude,
                    const Tensor &out) {
    check_rows("K", K);
    check_rows("V", V, &K);
    TORCH_CHECK_VALUE(V.size(1) == K.size(1), "V must have K's shape");
    const int64_t B = K.size(0), HK = K.size(1), T = K.size(2), D = K.size(3);
    if (Q.defined()) {
        check_rows("Q", Q, &K);
        TORCH_CHECK_VALUE(f, "Q is there to be rotated: frequencies are missing");
    } else {
        TORCH_CHECK_VALUE(!out.defined(), "out without Q");
    }
    const Pages p = check_pages(Kc, Vc, table, lens, B, HK, D, K);
    check_written("K_cache", Kc);
    check_written("V_cache", Vc);
    const int32_t *const fresh = counts.defined() ? check_list("counts", counts, {B}, K) : nullptr;
    const tsa_dtype dtype = dtype_of(K);
    const Tensor q = Q.defined() ? rows_out("out", out, Q) : Tensor();
    int64_t strides[12];
    put_strides(strides, Q);
    put_strides(strides + 3, K);
    put_strides(strides + 6, V);
    put_strides(strides + 9, q);
    check(tsa_paged_append(data(Q), K.const_data_ptr(), V.const_data_ptr(), strides, written(Kc),
                           written(Vc), p.pages, p.size, p.k_stride, p.v_stride, p.table, p.most, p.lens, fresh,
                           f ? f->values : nullptr, f ? 2 * f->n : 0, interleaved, (float)magnitude, written(q),
                           dtype, B, Q.defined() ? Q.size(1) : 0, HK, T, D, stream_of(K)),
          "tsa_paged_append");
    for (const Tensor *t : {&Kc, &Vc, &out}) written_to(*t);
    return q;
}

Tensor paged_decode(const Tensor &Q, const Tensor &Kc, const Tensor &Vc, const Tensor &table, const Tensor &lens,
                    const Tensor &row_ptr, const Tensor &col_idx, const double *scale, int64_t block, const Tensor &out,
                    const Tensor &workspace) {
    TORCH_CHECK_VALUE(Q.dim() == 3 && Q.is_cuda() && Q.is_contiguous(), "Q must be a contiguous CUDA tensor [B, H, D]");
    const int64_t B = Q.size(0), H = Q.size(1), D = Q.size(2), HK = Kc.dim() == 4 ? Kc.size(1) : 0;
    const Pages p = check_pages(Kc, Vc, table, lens, B, HK, D, Q);
    TORCH_CHECK_VALUE(row_ptr.defined() == col_idx.defined(), "row_ptr and col_idx go together");
    const int32_t *rows = nullptr, *blocks = nullptr;
    int64_t nnz = 0;
    Tensor none;
    if (row_ptr.defined()) {
        TORCH_CHECK_VALUE(row_ptr.numel() == B + 1, "row_ptr must hold ", B + 1, " entries");
        rows = check_list("row_ptr", row_ptr, row_ptr.sizes(), Q);
        blocks = check_list("col_idx", col_idx, col_idx.sizes(), Q);
        nnz = col_idx.numel();
        if (nnz == 0) {
            none = at::zeros({1}, col_idx.options());
            blocks = none.const_data_ptr<int32_t>();
            nnz = 1;
        }
    }
    const tsa_dtype dtype = dtype_of(Q);
    if (out.defined()) {
        TORCH_CHECK_VALUE(out.sizes() == Q.sizes() && out.scalar_type() == Q.scalar_type() && out.device() == Q.device() &&
                              out.is_contiguous(),
                          "out must be a contiguous tensor of Q's type, shape and device");
        check_written("out", out);
    }
    const Tensor o = out.defined() ? out : at::empty(Q.sizes(), Q.options());
    const size_t need = tsa_paged_attention_decode_workspace_bytes(B, H, HK, D, p.size, p.most, block, nnz);
    Tensor w = workspace;
    if (w.defined()) {
        TORCH_CHECK_VALUE(w.scalar_type() == at::kByte && w.device() == Q.device() && w.is_contiguous(),
                          "workspace must be a contiguous uint8 tensor on the inputs' device");
    } else if (need > 0) {
        w = at::empty({(int64_t)need}, Q.options().dtype(at::kByte));
    }
    check(tsa_paged_attention_decode(Q.const_data_ptr(), data(Kc), data(Vc), p.pages, p.size, p.k_stride, p.v_stride, p.table,
                                     p.most, p.lens, rows, blocks, nnz, written(o), dtype, B, H, HK, D, block,
                                     (float)(scale ? *scale : 1.0 / std::sqrt((double)D)), written(w),
                                     w.defined() ? (size_t)w.numel() : 0, stream_of(Q)),
          "tsa_paged_attention_decode");
    written_to(out);
    return o;
}

// --- Python ---

PyObject *g_error = nullptr;  // TsaError(status, where)

// A call's arguments: positional, None for what is not given.
struct Args {
    PyObject *const *a;
    const char *call;

    Args(PyObject *const *args, Py_ssize_t given, Py_ssize_t n, const char *name) : a(args), call(name) {
        TORCH_CHECK_TYPE(given == n, name, " takes ", n, " arguments, got ", given);
    }
    bool none(int i) const { return a[i] == Py_None; }
    const Tensor &tensor(int i) const {
        static const Tensor undefined;
        if (none(i)) return undefined;
        TORCH_CHECK_TYPE(THPVariable_Check(a[i]), call, " takes tensors, got ", Py_TYPE(a[i])->tp_name);
        return THPVariable_Unpack(a[i]);
    }
    const Tensor &given(int i, const char *name) const {
        TORCH_CHECK_TYPE(!none(i), call, ": ", name, " is missing");
        return tensor(i);
    }
    bool truth(int i) const {
        const int v = PyObject_IsTrue(a[i]);
        if (v < 0) throw python_error();
        return v == 1;
    }
    double number(int i) const {
        const double v = PyFloat_AsDouble(a[i]);
        if (v == -1.0 && PyErr_Occurred()) throw python_error();
        return v;
    }
    int64_t integer(int i) const {
        const long long v = PyLong_AsLongLong(a[i]);
        if (v == -1 && PyErr_Occurred()) throw python_error();
        return v;
    }
};

// A host array of binary64.
struct Array {
    Py_buffer view = {};
    Frequencies f = {nullptr, 0};

    Array(const Args &a, int i) {
        if (a.none(i)) return;
        if (PyObject_GetBuffer(a.a[i], &view, PyBUF_CONTIG_RO | PyBUF_FORMAT) != 0) throw python_error();
        if (!view.format || std::string(view.format) != "d") {
            PyBuffer_Release(&view);
            TORCH_CHECK_TYPE(false, a.call, ": frequencies must be binary64");
        }
        f = {static_cast<const double *>(view.buf), (int64_t)(view.len / 8)};
    }
    Array(const Array &) = delete;
    ~Array() {
        if (view.obj) PyBuffer_Release(&view);
    }
    const Frequencies &needed(const Args &a) const {
        TORCH_CHECK_TYPE(f.values, a.call, ": frequencies are missing");
        return f;
    }
};

// The interpreter is not needed while the library checks and launches (a launch may wait for room in its queue).
struct WithoutGil {
    PyThreadState *state = PyEval_SaveThread();
    ~WithoutGil() { PyEval_RestoreThread(state); }
};

PyObject *wrap(const Tensor &t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

PyObject *wrap(const Tensor &q, const Tensor &k) {
    if (!k.defined()) return wrap(q);
    PyObject *x = wrap(q), *y = wrap(k);
    PyObject *r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

template <class Call>
PyObject *answered(Call call) {
    HANDLE_TH_ERRORS
    try {
        return call();
    } catch (const StatusError &e) {
        PyObject *v = PyObject_CallFunction(g_error, "is", (int)e.status, e.where.c_str());
        if (v) {
            PyErr_SetObject(g_error, v);
            Py_DECREF(v);
        }
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *py_rotary(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return answered([&]() -> PyObject * {
        const Args a(args, n, 9, "tsa_rotary");
        const Tensor &Q = a.given(0, "Q"), &K = a.tensor(1), &positions = a.tensor(3), &out = a.tensor(7), &out_k = a.tensor(8);
        const Array f(a, 2);
        const Frequencies &values = f.needed(a);
        const bool interleaved = a.truth(4), inverse = a.truth(6);
        const double magnitude = a.number(5);
        std::array<Tensor, 2> r;
        {
            WithoutGil gil;
            r = rotary(Q, K, values, positions, interleaved, magnitude, inverse, out, out_k);
        }
        return wrap(r[0], r[1]);
    });
}

PyObject *py_rotary_autograd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return answered([&]() -> PyObject * {
        const Args a(args, n, 6, "rotary");
        const Tensor &Q = a.given(0, "Q"), &K = a.tensor(1), &positions = a.tensor(3);
        std::vector<double> values;
        {
            const Array f(a, 2);
            values.assign(f.needed(a).values, f.f.values + f.f.n);
        }
        const bool interleaved = a.truth(4);
        const double magnitude = a.number(5);
        torch::autograd::variable_list r;
        {
            WithoutGil gil;
            r = Rotary::apply(Q, K.defined() ? std::optional<Tensor>(K) : std::nullopt,
                              positions.defined() ? std::optional<Tensor>(positions) : std::nullopt, values, interleaved,
                              magnitude, false);
        }
        return wrap(r[0], r.size() == 2 ? r[1] : Tensor());
    });
}

PyObject *py_paged_append(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return answered([&]() -> PyObject * {
        const Args a(args, n, 12, "tsa_paged_append");
        const Tensor &Q = a.tensor(0), &K = a.given(1, "K"), &V = a.given(2, "V"), &Kc = a.given(3, "K_cache"),
                     &Vc = a.given(4, "V_cache"), &table = a.given(5, "page_table"), &lens = a.given(6, "seq_lens"),
                     &counts = a.tensor(7), &out = a.tensor(11);
        const Array f(a, 8);
        const bool interleaved = a.truth(9);
        const double magnitude = a.number(10);
        Tensor r;
        {
            WithoutGil gil;
            r = paged_append(Q, K, V, Kc, Vc, table, lens, counts, a.none(8) ? nullptr : &f.f, interleaved, magnitude, out);
        }
        return wrap(r);
    });
}

PyObject *py_paged_decode(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return answered([&]() -> PyObject * {
        const Args a(args, n, 11, "tsa_paged_attention_decode");
        const Tensor &Q = a.given(0, "Q"), &Kc = a.given(1, "K_cache"), &Vc = a.given(2, "V_cache"),
                     &table = a.given(3, "page_table"), &lens = a.given(4, "seq_lens"), &row_ptr = a.tensor(5),
                     &col_idx = a.tensor(6), &out = a.tensor(9), &workspace = a.tensor(10);
        const double scale = a.none(7) ? 0.0 : a.number(7);
        const int64_t block = a.integer(8);
        Tensor r;
        {
            WithoutGil gil;
            r = paged_decode(Q, Kc, Vc, table, lens, row_ptr, col_idx, a.none(7) ? nullptr : &scale, block, out, workspace);
        }
        return wrap(r);
    });
}

// The class of the errors that the library's status codes become.
PyObject *py_set_error(PyObject *, PyObject *cls) {
    Py_INCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

template <class F>
PyCFunction method(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f));
}

PyMethodDef g_methods[] = {{"rotary", method(py_rotary), METH_FASTCALL, nullptr},
                           {"rotary_autograd", method(py_rotary_autograd), METH_FASTCALL, nullptr},
                           {"paged_append", method(py_paged_append), METH_FASTCALL, nullptr},
                           {"paged_decode", method(py_paged_decode), METH_FASTCALL, nullptr},
                           {"set_error", py_set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "tsa_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_tsa_calls() { return PyModule_Create(&g_module); }
