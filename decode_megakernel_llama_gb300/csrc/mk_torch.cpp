// mk_torch.cpp — the Python binding's quick way into the drafted-tree operators
// (mk_rope_append, mk_tree_attention, mk_kv_compact, mk_kv_reorder).
//
// These calls take ten tensors and a few microseconds on the GPU; checking and
// packing the tensors' types, shapes and addresses in Python takes 3 to 5 us,
// here 0.3. Each function makes the checks of its namesake in _lib.py on torch's
// own tensor objects, calls the C ABI and returns its status; where anything is
// not as it should be, or the call wants another device or a stream of its own
// for its workspace, it does nothing and returns 1, and the Python function says
// what is wrong or goes the long way. The C ABI's addresses come from the library
// that _lib.py loaded (bind). Its file is named after the torch and Python it was
// compiled against (build.py).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mk.h"

namespace {

constexpr long kNotHere = 1;  // for the Python function to deal with

struct {
    decltype(&mk_rope_append) rope;
    decltype(&mk_tree_attention) tree;
    decltype(&mk_tree_attention_workspace) tree_work;
    decltype(&mk_kv_compact) compact;
    decltype(&mk_kv_reorder) reorder;
} mk;

const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A dense tensor of type t on the CUDA device d with the shape given.
bool dense(const at::Tensor *x, at::ScalarType t, int d, at::IntArrayRef shape) {
    return x && x->scalar_type() == t && x->is_cuda() && x->get_device() == d && x->sizes() == shape &&
           x->is_contiguous();
}

// The same, or None.
bool dense_or_none(PyObject *o, const at::Tensor **x, at::ScalarType t, int d, at::IntArrayRef shape) {
    *x = nullptr;
    if (o == Py_None) return true;
    *x = tensor(o);
    return dense(*x, t, d, shape);
}

const void *address(const at::Tensor *x) { return x ? x->const_data_ptr() : nullptr; }

// The device's current stream, if it is the current device.
bool stream_of(int d, PyObject *given, void **s) {
    if (given != Py_None || c10::cuda::current_device() != d) return false;
    *s = c10::cuda::getCurrentCUDAStream(d).stream();
    return true;
}

int io_type(const at::Tensor &x) {
    return x.scalar_type() == at::kFloat ? MK_F32 : x.scalar_type() == at::kBFloat16 ? MK_BF16 : -1;
}

// qkv, q_out, k_cache, v_cache, positions, rows, inv_freq, slots, q_norm, k_norm, eps, mscale, interleaved, stream
long rope_append(PyObject *const *o, Py_ssize_t n_args) {
    if (n_args != 14) return kNotHere;
    const at::Tensor *qkv = tensor(o[0]), *q = tensor(o[1]), *k = tensor(o[2]), *v = tensor(o[3]), *f = tensor(o[6]);
    if (!qkv || !q || !k || !v || !f || !qkv->is_cuda() || !q->is_cuda()) return kNotHere;
    if (qkv->dim() != 2 || q->dim() != 3 || k->dim() != 4 || f->dim() != 1) return kNotHere;
    const int d = qkv->get_device(), type = io_type(*qkv);
    const int64_t n = q->size(0), Hq = q->size(1), Hkv = k->size(1), hd = k->size(3), half = f->size(0);
    const int64_t width = (Hq + 2 * Hkv) * hd;
    const at::Tensor *slots, *qn, *kn;
    void *s;
    if (type < 0 || n < 1 || n > INT32_MAX || q->size(2) != hd || q->scalar_type() != qkv->scalar_type() ||
        q->get_device() != d || qkv->size(0) != n || qkv->size(1) != width || half > hd ||
        !dense(k, at::kBFloat16, d, k->sizes()) || !dense(v, at::kBFloat16, d, k->sizes()) ||
        !dense(tensor(o[4]), at::kInt, d, {n}) || !dense(tensor(o[5]), at::kInt, d, {n}) ||
        !dense(f, at::kDouble, d, {half}) || !dense_or_none(o[7], &slots, at::kInt, d, {n}) ||
        !dense_or_none(o[8], &qn, at::kBFloat16, d, {hd}) || !dense_or_none(o[9], &kn, at::kBFloat16, d, {hd}) ||
        qkv->stride(1) != 1 || q->stride(2) != 1 || (Hq > 1 && q->stride(1) != hd) || Hq > INT32_MAX ||
        k->size(0) > INT32_MAX || Hkv > INT32_MAX || k->size(2) > INT32_MAX || !stream_of(d, o[13], &s))
        return kNotHere;
    const int inter = PyObject_IsTrue(o[12]);
    mk_rope_args a{};
    a.n = n, a.n_heads = Hq, a.n_kv_heads = Hkv, a.head_dim = hd, a.rot = 2 * half, a.interleaved = inter;
    a.dtype = type, a.slots = k->size(0), a.max_seq = k->size(2);
    a.eps = PyFloat_AsDouble(o[10]), a.mscale = PyFloat_AsDouble(o[11]);
    if (inter < 0 || PyErr_Occurred()) {
        PyErr_Clear();
        return kNotHere;
    }
    a.qkv_stride = n > 1 ? qkv->stride(0) : width, a.q_stride = n > 1 ? q->stride(0) : Hq * hd;
    a.qkv = address(qkv), a.q_out = q->data_ptr(), a.k_cache = k->data_ptr(), a.v_cache = v->data_ptr();
    a.positions = static_cast<const int32_t *>(address(tensor(o[4])));
    a.rows = static_cast<const int32_t *>(address(tensor(o[5])));
    a.slot_of = static_cast<const int32_t *>(address(slots));
    a.inv_freq = static_cast<const double *>(address(f));
    a.q_norm = address(qn), a.k_norm = address(kn);
    return mk.rope(&a, s);
}

// q, k_cache, v_cache, lengths, masks, out, scale (None: 1 / sqrt(hd)), counts, slots, max_len, status, stream, wait_ns
long tree_attention(PyObject *const *o, Py_ssize_t n_args) {
    if (n_args != 13) return kNotHere;
    const at::Tensor *q = tensor(o[0]), *k = tensor(o[1]), *v = tensor(o[2]), *out = tensor(o[5]);
    if (!q || !k || !v || !out || !q->is_cuda() || !out->is_cuda() || q->dim() != 4 || k->dim() != 4) return kNotHere;
    const int d = q->get_device(), type = io_type(*q);
    const int64_t B = q->size(0), T = q->size(1), Hq = q->size(2), hd = q->size(3), S = k->size(2), row = Hq * hd;
    const at::Tensor *counts, *slots, *status;
    void *s;
    if (type < 0 || B < 1 || T < 1 || B > INT32_MAX || T > INT32_MAX || Hq < 1 || Hq > INT32_MAX ||
        out->sizes() != q->sizes() || out->scalar_type() != q->scalar_type() || out->get_device() != d ||
        k->size(3) != hd || !dense(k, at::kBFloat16, d, k->sizes()) || !dense(v, at::kBFloat16, d, k->sizes()) ||
        !dense(tensor(o[3]), at::kInt, d, {B}) || !dense(tensor(o[4]), at::kLong, d, {B, T}) ||
        !dense_or_none(o[7], &counts, at::kInt, d, {B}) || !dense_or_none(o[8], &slots, at::kInt, d, {B}) ||
        !dense_or_none(o[10], &status, at::kInt, d, {1}) || (!slots && B > k->size(0)) || q->stride(3) != 1 ||
        out->stride(3) != 1 || (Hq > 1 && (q->stride(2) != hd || out->stride(2) != hd)) || k->size(0) > INT32_MAX ||
        k->size(1) > INT32_MAX || S > INT32_MAX || !stream_of(d, o[11], &s))
        return kNotHere;
    mk_tree_args a{};
    const double scale = o[6] == Py_None ? 1.0 / std::sqrt((double)hd) : PyFloat_AsDouble(o[6]);
    const long max_len = PyLong_AsLong(o[9]);
    const long long wait_ns = PyLong_AsLongLong(o[12]);
    if (PyErr_Occurred() || max_len < 0 || max_len > INT32_MAX) {
        PyErr_Clear();
        return kNotHere;
    }
    a.batch = B, a.nodes = T, a.n_heads = Hq, a.n_kv_heads = k->size(1), a.head_dim = hd, a.dtype = type;
    a.slots = k->size(0), a.max_seq = S, a.max_len = max_len;
    a.scale = scale, a.wait_ns = wait_ns;
    a.q_batch_stride = B > 1 ? q->stride(0) : 0, a.q_token_stride = T > 1 ? q->stride(1) : row;
    a.out_batch_stride = B > 1 ? out->stride(0) : 0, a.out_token_stride = T > 1 ? out->stride(1) : row;
    a.q = address(q), a.out = out->data_ptr(), a.k_cache = address(k), a.v_cache = address(v);
    a.lengths = static_cast<const int32_t *>(address(tensor(o[3])));
    a.masks = static_cast<const uint64_t *>(address(tensor(o[4])));
    a.counts = static_cast<const int32_t *>(address(counts));
    a.slot_of = static_cast<const int32_t *>(address(slots));
    a.status = status ? static_cast<int32_t *>(status->data_ptr()) : nullptr;
    at::Tensor work;
    const int64_t bytes = mk.tree_work(&a);
    if (bytes < 0) return bytes;
    if (bytes > 0) {
        work = at::empty({bytes}, k->options().dtype(at::kByte));
        a.workspace = work.data_ptr();
        a.workspace_bytes = bytes;
    }
    return mk.tree(&a, s);
}

// Two whole caches, k and v.
const at::Tensor *caches(PyObject *ko, PyObject *vo) {
    const at::Tensor *k = tensor(ko);
    if (!k || !k->is_cuda() || k->dim() != 5) return nullptr;
    const int d = k->get_device();
    for (int i = 0; i < 5; ++i)
        if (k->size(i) > INT32_MAX) return nullptr;
    return dense(k, at::kBFloat16, d, k->sizes()) && dense(tensor(vo), at::kBFloat16, d, k->sizes()) ? k : nullptr;
}

// k, v, starts, nodes, counts, stream
long kv_compact(PyObject *const *o, Py_ssize_t n_args) {
    const at::Tensor *k = n_args == 6 ? caches(o[0], o[1]) : nullptr, *nodes = k ? tensor(o[3]) : nullptr;
    if (!nodes || nodes->dim() != 2) return kNotHere;
    const int d = k->get_device();
    const int64_t B = k->size(1), n = nodes->size(1);
    void *s;
    if (n > INT32_MAX || !dense(tensor(o[2]), at::kInt, d, {B}) || !dense(nodes, at::kInt, d, {B, n}) ||
        !dense(tensor(o[4]), at::kInt, d, {B}) || !stream_of(d, o[5], &s))
        return kNotHere;
    return mk.compact(k->data_ptr(), tensor(o[1])->data_ptr(), k->size(0), B, k->size(2), k->size(3), k->size(4), n,
                      static_cast<const int32_t *>(address(tensor(o[2]))), static_cast<const int32_t *>(address(nodes)),
                      static_cast<const int32_t *>(address(tensor(o[4]))), s);
}

// k, v, sources, lengths, stream
long kv_reorder(PyObject *const *o, Py_ssize_t n_args) {
    const at::Tensor *k = n_args == 5 ? caches(o[0], o[1]) : nullptr;
    if (!k) return kNotHere;
    const int d = k->get_device();
    const int64_t B = k->size(1);
    void *s;
    if (!dense(tensor(o[2]), at::kInt, d, {B}) || !dense(tensor(o[3]), at::kInt, d, {B}) || !stream_of(d, o[4], &s))
        return kNotHere;
    return mk.reorder(k->data_ptr(), tensor(o[1])->data_ptr(), k->size(0), B, k->size(2), k->size(3), k->size(4),
                      static_cast<const int32_t *>(address(tensor(o[2]))),
                      static_cast<const int32_t *>(address(tensor(o[3]))), s);
}

template <long (*F)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    long rc = kNotHere;
    try {
        rc = F(args, n);
    } catch (...) {  // the Python function meets the same error and words it
        rc = kNotHere;
    }
    return PyLong_FromLong(rc);
}

// The addresses of mk_rope_append, mk_tree_attention, mk_tree_attention_workspace, mk_kv_compact, mk_kv_reorder.
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
    void *p[5];
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
        return nullptr;
    }
    for (int i = 0; i < 5; ++i)
        if (!(p[i] = PyLong_AsVoidPtr(args[i]))) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a NULL address");
            return nullptr;
        }
    mk.rope = reinterpret_cast<decltype(mk.rope)>(p[0]);
    mk.tree = reinterpret_cast<decltype(mk.tree)>(p[1]);
    mk.tree_work = reinterpret_cast<decltype(mk.tree_work)>(p[2]);
    mk.compact = reinterpret_cast<decltype(mk.compact)>(p[3]);
    mk.reorder = reinterpret_cast<decltype(mk.reorder)>(p[4]);
    Py_RETURN_NONE;
}

#define MK_ENTRY(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"bind", MK_ENTRY(&bind)},
                         {"rope_append", MK_ENTRY(&entry<rope_append>)},
                         {"tree_attention", MK_ENTRY(&entry<tree_attention>)},
                         {"kv_compact", MK_ENTRY(&entry<kv_compact>)},
                         {"kv_reorder", MK_ENTRY(&entry<kv_reorder>)},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "mk_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_mk_torch(void) { return PyModule_Create(&module); }
