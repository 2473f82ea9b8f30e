// The paged calls' argument marshalling for Python, for calls that need no
// word of explanation: tensors are checked and read through torch's C++ side,
// some nanoseconds each where Python takes half a microsecond (thirteen of
// them in an attention call: 7.5 us of a call whose kernels take 7).
//
// Each function takes the address of the library's entry and the arguments of
// the Python call in order, and returns the library's status, or -1 where
// anything is not as the call wants it: the caller then looks again in Python,
// which says what is wrong (or makes the call, with another device current).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>

#include "qsa.h"

namespace {

using at::ScalarType;
using Args = PyObject *const *;

struct No {};  // the arguments are not as the call wants them

const at::Tensor &tensor(PyObject *o) {
    if (!THPVariable_Check(o)) throw No{};
    return THPVariable_Unpack(o);
}
void want(bool fine) {
    if (!fine) throw No{};
}
int small(int64_t v) {
    want(v >= 0 && v <= INT_MAX);
    return (int)v;
}

// The device and checks of one call's tensors.
struct Call {
    c10::Device dev;
    explicit Call(const at::Tensor &t) : dev(t.device()) {
        want(dev.is_cuda() && c10::cuda::current_device() == dev.index());
    }
    void *in(const at::Tensor &t, ScalarType type, at::IntArrayRef shape) const {
        want(t.scalar_type() == type && t.device() == dev && t.layout() == at::kStrided && t.sizes() == shape && t.is_contiguous());
        return t.data_ptr();
    }
    template <class T>
    T *in(PyObject *o, ScalarType type, at::IntArrayRef shape) const {
        return static_cast<T *>(in(tensor(o), type, shape));
    }
    template <class T>
    T *opt(PyObject *o, ScalarType type, at::IntArrayRef shape) const {
        return o == Py_None ? nullptr : in<T>(o, type, shape);
    }
    unsigned *err(PyObject *o) const {
        if (o == Py_None) return nullptr;
        const at::Tensor &t = tensor(o);
        want(t.scalar_type() == at::kInt && t.device() == dev && t.layout() == at::kStrided && t.numel() >= 1);
        return static_cast<unsigned *>(t.data_ptr());
    }
    void *scratch(PyObject *o, size_t &bytes) const {
        const at::Tensor &t = tensor(o);
        want(t.device() == dev && t.layout() == at::kStrided && t.is_contiguous());
        bytes = (size_t)t.numel() * t.element_size();
        return t.data_ptr();
    }
    // A cache: codes [..., Hkv, D], scales [..., Hkv, 4].
    template <class A>
    void cache(A &a, Args o) const {
        const at::Tensor &kq = tensor(o[0]);
        c10::DimVector scales(kq.sizes());
        want(!scales.empty());
        scales.back() = 4;
        a.kq = static_cast<int8_t *>(in(kq, at::kChar, kq.sizes()));
        a.vq = in<int8_t>(o[1], at::kChar, kq.sizes());
        a.ksc = in<uint16_t>(o[2], at::kHalf, scales);
        a.vsc = in<uint16_t>(o[3], at::kHalf, scales);
    }
    void *stream(PyObject *o) const {
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev.index()).stream();
        PyObject *index = PyObject_GetAttrString(o, "device_index"), *raw = PyObject_GetAttrString(o, "cuda_stream");
        const long on = index ? PyLong_AsLong(index) : -1;
        void *s = raw ? PyLong_AsVoidPtr(raw) : nullptr;
        Py_XDECREF(index);
        Py_XDECREF(raw);
        want(!PyErr_Occurred() && on == dev.index());
        return s;
    }
};

int dtype_code(ScalarType t) {
    return t == at::kFloat ? QSA_F32 : t == at::kHalf ? QSA_F16 : t == at::kBFloat16 ? QSA_BF16 : -1;
}
float number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    want(!(v == -1.0 && PyErr_Occurred()));
    return (float)v;
}

template <class A>
int run(PyObject *entry, const A &a, void *stream) {
    const auto fn = reinterpret_cast<qsa_status (*)(const A *, void *)>(PyLong_AsVoidPtr(entry));
    want(fn != nullptr);
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = fn(&a, stream);
    Py_END_ALLOW_THREADS;
    return status;
}

// q_in k_in v_in positions slots kq vq ksc vsc q_out q_norm_w k_norm_w inv_freq interleaved eps rope_mscale err stream
int prep(PyObject *entry, Args o) {
    const at::Tensor &q = tensor(o[0]), &kq = tensor(o[5]), &out = tensor(o[9]);
    const Call c(q);
    want(q.dim() == 3 && kq.dim() >= 3);
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2), hkv = kq.size(-2);
    want(kq.size(-1) == D && hkv > 0 && D > 0);
    qsa_paged_prep_args a{};
    a.ntok = small(T), a.n_q_heads = small(H), a.n_kv_heads = small(hkv), a.head_dim = small(D), a.group = a.head_dim / 4;
    a.cache_cells = small(kq.numel() / (hkv * D));
    a.in_dtype = dtype_code(q.scalar_type()), a.q_out_dtype = dtype_code(out.scalar_type());
    want(a.in_dtype >= 0 && (a.q_out_dtype == QSA_F16 || a.q_out_dtype == QSA_BF16));
    const void **in[3] = {&a.q_in, &a.k_in, &a.v_in};
    int64_t *stride[3] = {&a.q_stride, &a.k_stride, &a.v_stride};
    for (int i = 0; i < 3; ++i) {
        const at::Tensor &t = tensor(o[i]);
        const int64_t h = i ? hkv : H;
        want(t.scalar_type() == q.scalar_type() && t.device() == c.dev && t.layout() == at::kStrided && t.dim() == 3 && t.size(0) == T &&
             t.size(1) == h && t.size(2) == D);
        want(t.numel() == 0 || (t.stride(2) == 1 && (h <= 1 || t.stride(1) == D)));
        *in[i] = t.data_ptr();
        *stride[i] = t.stride(0);
    }
    if (o[12] != Py_None) {
        const at::Tensor &f = tensor(o[12]);
        want(f.dim() == 1);
        a.inv_freq = static_cast<const float *>(c.in(f, at::kFloat, f.sizes()));
        a.rope_dims = small(2 * f.size(0));
    }
    c.cache(a, o + 5);
    a.interleaved = PyObject_IsTrue(o[13]);
    want(a.interleaved >= 0);
    a.eps = number(o[14]), a.rope_mscale = number(o[15]);
    a.q_norm_w = c.opt<float>(o[10], at::kFloat, {D}), a.k_norm_w = c.opt<float>(o[11], at::kFloat, {D});
    a.positions = c.in<int32_t>(o[3], at::kInt, {T}), a.slots = c.in<int32_t>(o[4], at::kInt, {T});
    a.q_out = c.in(out, out.scalar_type(), {T, H, D});
    a.err = c.err(o[16]);
    return run(entry, a, c.stream(o[17]));
}

// kq vq ksc vsc ids k_out v_out rows page_table err stream
int gather(PyObject *entry, Args o) {
    const at::Tensor &kq = tensor(o[0]), &ids = tensor(o[4]), &out = tensor(o[5]);
    const Call c(kq);
    want(kq.dim() >= 3);
    const int64_t hkv = kq.size(-2), D = kq.size(-1), n = ids.numel();
    want(hkv > 0 && D > 0);
    qsa_paged_gather_args a{};
    a.n_ids = small(n), a.n_kv_heads = small(hkv), a.head_dim = small(D), a.group = a.head_dim / 4;
    a.cache_cells = small(kq.numel() / (hkv * D));
    a.out_dtype = dtype_code(out.scalar_type());
    want(a.out_dtype >= 0 && (o[7] == Py_None) == (o[8] == Py_None));
    if (o[8] != Py_None) {
        const at::Tensor &table = tensor(o[8]);
        want(kq.dim() == 4 && table.dim() == 2);
        a.page_size = small(kq.size(1)), a.n_rows = small(table.size(0)), a.max_pages = small(table.size(1));
        a.page_table = static_cast<const int32_t *>(c.in(table, at::kInt, table.sizes()));
        a.rows = c.in<int32_t>(o[7], at::kInt, {n});
    }
    c.cache(a, o);
    a.ids = static_cast<const int32_t *>(c.in(ids, at::kInt, {n}));
    a.k_out = c.in(out, out.scalar_type(), {n, hkv, D}), a.v_out = c.in<void>(o[6], out.scalar_type(), {n, hkv, D});
    a.err = c.err(o[9]);
    return run(entry, a, c.stream(o[10]));
}

// q kq vq ksc vsc page_table seq_lens out workspace rows softmax_scale gate lse err stream
int attn(PyObject *entry, Args o) {
    const at::Tensor &q = tensor(o[0]), &kq = tensor(o[1]), &table = tensor(o[5]);
    const Call c(q);
    want(q.dim() == 3 && kq.dim() == 4 && table.dim() == 2);
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
    want(kq.size(3) == D && (q.scalar_type() == at::kHalf || q.scalar_type() == at::kBFloat16));
    qsa_paged_attn_args a{};
    a.n_tokens = small(T), a.n_q_heads = small(H), a.n_kv_heads = small(kq.size(2)), a.head_dim = small(D), a.group = a.head_dim / 4;
    a.page_size = small(kq.size(1)), a.n_pages = small(kq.size(0)), a.n_rows = small(table.size(0)), a.max_pages = small(table.size(1));
    a.dtype = dtype_code(q.scalar_type());
    c.cache(a, o + 1);
    a.q = c.in(q, q.scalar_type(), {T, H, D});
    a.page_table = static_cast<const int32_t *>(c.in(table, at::kInt, table.sizes()));
    a.seq_lens = c.in<int32_t>(o[6], at::kInt, {T}), a.rows = c.opt<int32_t>(o[9], at::kInt, {T});
    a.softmax_scale = o[10] == Py_None ? (float)std::pow((double)D, -0.5) : number(o[10]);
    a.gate = c.opt<float>(o[11], at::kFloat, {T, H, D}), a.lse = c.opt<float>(o[12], at::kFloat, {T, H});
    a.out = c.in<void>(o[7], q.scalar_type(), {T, H, D});
    a.workspace = c.scratch(o[8], a.workspace_bytes);
    a.err = c.err(o[13]);
    return run(entry, a, c.stream(o[14]));
}

// Shape of a pool, or of one layer of it.
template <class A>
void pool(A &a, const at::Tensor &kq, const at::Tensor &table) {
    want((kq.dim() == 4 || kq.dim() == 5) && table.dim() == 2);
    const at::IntArrayRef s = kq.sizes().slice(kq.dim() - 4);
    a.n_layers = kq.dim() == 5 ? small(kq.size(0)) : 1;
    a.n_pages = small(s[0]), a.page_size = small(s[1]), a.n_kv_heads = small(s[2]), a.head_dim = small(s[3]), a.group = a.head_dim / 4;
    a.max_pages = small(table.size(1));
}

// page_table seq_lens src n_new kq vq ksc vsc page_table_out seq_lens_out refs slots positions workspace err stream
int update(PyObject *entry, Args o) {
    const at::Tensor &table = tensor(o[0]), &n_new = tensor(o[3]), &kq = tensor(o[4]), &slots = tensor(o[11]);
    const Call c(kq);
    qsa_page_update_args a{};
    pool(a, kq, table);
    const int64_t rows_in = table.size(0), rows = n_new.numel(), n = slots.numel();
    a.n_rows_in = small(rows_in), a.n_rows = small(rows), a.n_slots = small(n);
    c.cache(a, o + 4);
    a.page_table = static_cast<const int32_t *>(c.in(table, at::kInt, table.sizes()));
    a.seq_lens = c.in<int32_t>(o[1], at::kInt, {rows_in}), a.src = c.opt<int32_t>(o[2], at::kInt, {rows});
    a.n_new = static_cast<const int32_t *>(c.in(n_new, at::kInt, {rows}));
    a.page_table_out = c.in<int32_t>(o[8], at::kInt, {rows, a.max_pages}), a.seq_lens_out = c.in<int32_t>(o[9], at::kInt, {rows});
    a.refs = c.in<int32_t>(o[10], at::kInt, {a.n_pages});
    a.slots = static_cast<int32_t *>(c.in(slots, at::kInt, {n})), a.positions = c.in<int32_t>(o[12], at::kInt, {n});
    a.workspace = c.scratch(o[13], a.workspace_bytes);
    a.err = c.err(o[14]);
    return run(entry, a, c.stream(o[15]));
}

// page_table seq_lens kq vq ksc vsc page_table_out refs page_map n_live workspace err stream
int compact(PyObject *entry, Args o) {
    const at::Tensor &table = tensor(o[0]), &kq = tensor(o[2]);
    const Call c(kq);
    qsa_page_compact_args a{};
    pool(a, kq, table);
    const int64_t rows = table.size(0);
    a.n_rows = small(rows);
    c.cache(a, o + 2);
    a.page_table = static_cast<const int32_t *>(c.in(table, at::kInt, table.sizes()));
    a.seq_lens = c.in<int32_t>(o[1], at::kInt, {rows});
    a.page_table_out = c.in<int32_t>(o[6], at::kInt, table.sizes());
    a.refs = c.in<int32_t>(o[7], at::kInt, {a.n_pages}), a.page_map = c.in<int32_t>(o[8], at::kInt, {a.n_pages});
    a.n_live = c.in<int32_t>(o[9], at::kInt, {1});
    a.workspace = c.scratch(o[10], a.workspace_bytes);
    a.err = c.err(o[11]);
    return run(entry, a, c.stream(o[12]));
}

// Page bounds: codes [pages, Hkv, D], scales [pages, Hkv, 4].
template <class A>
void bounds_of(A &a, const Call &c, Args o, int64_t pages, int64_t hkv, int64_t D) {
    a.hi_q = c.in<int8_t>(o[0], at::kChar, {pages, hkv, D}), a.lo_q = c.in<int8_t>(o[1], at::kChar, {pages, hkv, D});
    a.hi_sc = c.in<uint16_t>(o[2], at::kHalf, {pages, hkv, 4}), a.lo_sc = c.in<uint16_t>(o[3], at::kHalf, {pages, hkv, 4});
}
int whole(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    want(!(v == -1 && PyErr_Occurred()) && v >= INT_MIN && v <= INT_MAX);
    return (int)v;
}

// page_table seq_lens kq ksc hi_q lo_q hi_sc lo_sc n_new err stream
int bounds(PyObject *entry, Args o) {
    const at::Tensor &table = tensor(o[0]), &kq = tensor(o[2]);
    const Call c(kq);
    want(kq.dim() == 4 && table.dim() == 2);
    const int64_t pages = kq.size(0), page = kq.size(1), hkv = kq.size(2), D = kq.size(3), rows = table.size(0);
    qsa_page_bounds_args a{};
    a.n_rows = small(rows), a.max_pages = small(table.size(1)), a.n_pages = small(pages), a.page_size = small(page);
    a.n_kv_heads = small(hkv), a.head_dim = small(D), a.group = a.head_dim / 4;
    a.page_table = static_cast<const int32_t *>(c.in(table, at::kInt, table.sizes()));
    a.seq_lens = c.in<int32_t>(o[1], at::kInt, {rows}), a.n_new = c.opt<int32_t>(o[8], at::kInt, {rows});
    a.kq = static_cast<const int8_t *>(c.in(kq, at::kChar, kq.sizes()));
    a.ksc = c.in<uint16_t>(o[3], at::kHalf, {pages, page, hkv, 4});
    bounds_of(a, c, o + 4, pages, hkv, D);
    a.err = c.err(o[9]);
    return run(entry, a, c.stream(o[10]));
}

// q hi_q lo_q hi_sc lo_sc page_table seq_lens scores page_size rows err stream
int score(PyObject *entry, Args o) {
    const at::Tensor &q = tensor(o[0]), &hi = tensor(o[1]), &table = tensor(o[5]), &scores = tensor(o[7]);
    const Call c(q);
    want(q.dim() == 3 && hi.dim() == 3 && table.dim() == 2 && scores.dim() == 3);
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2), hkv = hi.size(1);
    want(hi.size(2) == D && (q.scalar_type() == at::kHalf || q.scalar_type() == at::kBFloat16));
    qsa_page_score_args a{};
    a.n_tokens = small(T), a.n_q_heads = small(H), a.n_kv_heads = small(hkv), a.head_dim = small(D), a.group = a.head_dim / 4;
    a.page_size = whole(o[8]), a.n_pages = small(hi.size(0)), a.n_rows = small(table.size(0)), a.max_pages = small(table.size(1));
    a.dtype = dtype_code(q.scalar_type());
    a.q = c.in(q, q.scalar_type(), {T, H, D});
    bounds_of(a, c, o + 1, hi.size(0), hkv, D);
    a.page_table = static_cast<const int32_t *>(c.in(table, at::kInt, table.sizes()));
    a.seq_lens = c.in<int32_t>(o[6], at::kInt, {T}), a.rows = c.opt<int32_t>(o[9], at::kInt, {T});
    a.scores = static_cast<float *>(c.in(scores, at::kFloat, {T, hkv, scores.size(2)})), a.ld = scores.size(2);
    a.err = c.err(o[10]);
    return run(entry, a, c.stream(o[11]));
}

// scores seq_lens pages counts page_size budget sink local err stream
int select(PyObject *entry, Args o) {
    const at::Tensor &scores = tensor(o[0]), &pages = tensor(o[2]);
    const Call c(scores);
    want(scores.dim() == 3 && pages.dim() == 3);
    const int64_t T = scores.size(0), hkv = scores.size(1), w = pages.size(2);
    qsa_page_select_args a{};
    a.n_tokens = small(T), a.n_kv_heads = small(hkv), a.page_size = whole(o[4]), a.width = small(w);
    a.budget = whole(o[5]), a.sink = whole(o[6]), a.local = whole(o[7]);
    a.scores = static_cast<const float *>(c.in(scores, at::kFloat, scores.sizes())), a.ld = scores.size(2);
    a.seq_lens = c.in<int32_t>(o[1], at::kInt, {T});
    a.pages = static_cast<int32_t *>(c.in(pages, at::kInt, {T, hkv, w})), a.counts = c.in<int32_t>(o[3], at::kInt, {T, hkv});
    a.err = c.err(o[8]);
    return run(entry, a, c.stream(o[9]));
}

// What the two calls below have in common: q kq vq ksc vsc page_table; out
// workspace rows softmax_scale gate lse err
template <class A>
Call attn_parts(A &a, Args first, Args last) {
    const at::Tensor &q = tensor(first[0]), &kq = tensor(first[1]), &table = tensor(first[5]);
    const Call c(q);
    want(q.dim() == 3 && kq.dim() == 4 && table.dim() == 2);
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
    want(kq.size(3) == D && (q.scalar_type() == at::kHalf || q.scalar_type() == at::kBFloat16));
    a.n_tokens = small(T), a.n_q_heads = small(H), a.n_kv_heads = small(kq.size(2)), a.head_dim = small(D), a.group = a.head_dim / 4;
    a.page_size = small(kq.size(1)), a.n_pages = small(kq.size(0)), a.n_rows = small(table.size(0)), a.max_pages = small(table.size(1));
    a.dtype = dtype_code(q.scalar_type());
    c.cache(a, first + 1);
    a.q = c.in(q, q.scalar_type(), {T, H, D});
    a.page_table = static_cast<const int32_t *>(c.in(table, at::kInt, table.sizes()));
    a.out = c.in<void>(last[0], q.scalar_type(), {T, H, D});
    a.workspace = c.scratch(last[1], a.workspace_bytes);
    a.rows = c.opt<int32_t>(last[2], at::kInt, {T});
    a.softmax_scale = last[3] == Py_None ? (float)std::pow((double)D, -0.5) : number(last[3]);
    a.gate = c.opt<float>(last[4], at::kFloat, {T, H, D}), a.lse = c.opt<float>(last[5], at::kFloat, {T, H});
    a.err = c.err(last[6]);
    return c;
}

// q kq vq ksc vsc page_table seq_lens pages counts out workspace rows softmax_scale gate lse err stream
int sparse_attn(PyObject *entry, Args o) {
    qsa_paged_sparse_attn_args a{};
    const Call c = attn_parts(a, o, o + 9);
    const at::Tensor &pages = tensor(o[7]);
    want(pages.dim() == 3);
    const int64_t T = a.n_tokens, hkv = a.n_kv_heads;
    a.width = small(pages.size(2));
    a.seq_lens = c.in<int32_t>(o[6], at::kInt, {T});
    a.pages = static_cast<const int32_t *>(c.in(pages, at::kInt, {T, hkv, pages.size(2)}));
    a.counts = c.in<int32_t>(o[8], at::kInt, {T, hkv});
    return run(entry, a, c.stream(o[16]));
}

// q kq vq ksc vsc page_table prefix_lens mask out workspace rows softmax_scale gate lse err stream
int tree_attn(PyObject *entry, Args o) {
    qsa_paged_tree_attn_args a{};
    const Call c = attn_parts(a, o, o + 8);
    const at::Tensor &mask = tensor(o[7]);
    want(mask.dim() == 2);
    a.words = small(mask.size(1));
    a.prefix_lens = c.in<int32_t>(o[6], at::kInt, {a.n_tokens});
    a.mask = static_cast<const int32_t *>(c.in(mask, at::kInt, {a.n_tokens, mask.size(1)}));
    return run(entry, a, c.stream(o[15]));
}

// What is thrown here is said again by Python.
template <int (*F)(PyObject *, Args), int N>
PyObject *entry(PyObject *, Args o, Py_ssize_t n) {
    int status = -1;
    try {
        if (n == N + 1) status = F(o[0], o + 1);
    } catch (...) {
    }
    PyErr_Clear();
    return PyLong_FromLong(status);
}
#define QSA_METHOD(name, n) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(entry<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {QSA_METHOD(prep, 18),   QSA_METHOD(gather, 11),  QSA_METHOD(attn, 15),
                         QSA_METHOD(update, 16), QSA_METHOD(compact, 13), QSA_METHOD(bounds, 11),
                         QSA_METHOD(score, 12),  QSA_METHOD(select, 10),  QSA_METHOD(sparse_attn, 17),
                         QSA_METHOD(tree_attn, 16), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// With the torch and the interpreter that it was compiled for: tensors are read
// by the layout in that torch's headers.
PyMODINIT_FUNC PyInit__paged_binding() {
    PyObject *m = PyModule_Create(&module);
    if (m && (PyModule_AddStringConstant(m, "torch_version", QSA_TORCH_VERSION) < 0 ||
              PyModule_AddStringConstant(m, "abi_tag", QSA_ABI_TAG) < 0))
        Py_CLEAR(m);
    return m;
}
