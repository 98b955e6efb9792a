// marshal.cpp -- the serving operators' calls from Python without the cost of
// asking every tensor in Python for its shape, strides, type, device and
// address (about 1 us a tensor, 10 us a call, where the kernels of a small step
// take 3).  Each function fills the C argument struct from the tensors and makes
// the call.  It knows the regular case only: anything that the binding would
// refuse makes it return None before any call, and the binding's own Python code
// then says what is wrong.

#define PY_SSIZE_T_CLEAN
#define __HIP_PLATFORM_AMD__ 1

#include <Python.h>

#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>

#include "xpress_argmax.h"

namespace {

using at::Tensor;

PyObject* none() { Py_RETURN_NONE; }

// A tensor argument, null for None; *ok falls for anything else.
const Tensor* tensor(PyObject* o, bool* ok)
{
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) {
        *ok = false;
        return nullptr;
    }
    return &THPVariable_Unpack(o);
}

int64_t code_of(const Tensor& t)
{
    switch (t.scalar_type()) {
        case at::kBFloat16: return XPRESS_BF16;
        case at::kHalf: return XPRESS_FP16;
        case at::kFloat8_e4m3fn: return XPRESS_E4M3;
        default: return -1;
    }
}

bool on(const Tensor& t, int64_t dev) { return t.is_cuda() && t.get_device() == dev; }

// The library works on the current device, whose stream the binding takes too.
bool on_current(int64_t dev)
{
    return c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getDevice().index() == dev;
}

bool has_shape(const Tensor& t, std::initializer_list<int64_t> shape)
{
    return t.sizes() == at::IntArrayRef(shape);
}

// A contiguous tensor of this type and shape, or None.
bool plain(const Tensor* t, at::ScalarType type, std::initializer_list<int64_t> shape, int64_t dev)
{
    return !t || (t->scalar_type() == type && has_shape(*t, shape) && t->is_contiguous() && on(*t, dev));
}

// Unit stride along the last dimension.
bool rows(const Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape, int64_t dev)
{
    return t.scalar_type() == type && has_shape(t, shape) && on(t, dev) &&
           (t.stride(-1) == 1 || t.size(-1) <= 1);
}

template <typename T>
T* address(const Tensor* t)
{
    return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

bool cache(const Tensor* k, const Tensor* v, const Tensor* table, const Tensor* ks, const Tensor* vs,
           xpress_kv_cache* c)
{
    if (!k || !v || !table || k->dim() != 4 || !k->is_cuda() || v->sizes() != k->sizes() ||
        v->strides() != k->strides() || v->scalar_type() != k->scalar_type()) {
        return false;
    }
    const int64_t dev = k->get_device();
    c->dtype = code_of(*k);
    c->pages = k->size(0);
    c->heads = k->size(1);
    c->page_size = k->size(2);
    c->dim = k->size(3);
    if (c->dtype < 0 || (k->stride(3) != 1 && c->dim > 1) || !on(*v, dev) || !on(*table, dev) ||
        table->dim() != 2 || table->scalar_type() != at::kInt || (table->size(1) > 1 && table->stride(1) != 1) ||
        !plain(ks, at::kFloat, {c->heads}, dev) || !plain(vs, at::kFloat, {c->heads}, dev)) {
        return false;
    }
    if (!on_current(dev)) return false;
    c->k = k->data_ptr();
    c->v = v->data_ptr();
    c->k_scale = address<const float>(ks);
    c->v_scale = address<const float>(vs);
    c->page_table = address<const int32_t>(table);
    c->stride_page = k->stride(0);
    c->stride_head = k->stride(1);
    c->stride_token = k->stride(2);
    c->seqs = table->size(0);
    c->table_width = table->size(1);
    c->stride_table = table->stride(0);
    return true;
}

// The C entry point with these arguments and the stream.
template <typename... Args>
PyObject* call(PyObject* entry, PyObject* stream, Args... args)
{
    void* fn = PyLong_AsVoidPtr(entry);
    if (!fn && PyErr_Occurred()) return nullptr;
    void* st = PyLong_AsVoidPtr(stream);
    if (!st && PyErr_Occurred()) return nullptr;
    int status = 0;
    Py_BEGIN_ALLOW_THREADS
    status = reinterpret_cast<int (*)(Args..., hipStream_t)>(fn)(args..., static_cast<hipStream_t>(st));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

// Whole numbers from a on; false where one is none (or, with an error set, too large).
template <size_t K>
bool whole(PyObject* const* a, int64_t (&to)[K])
{
    for (size_t i = 0; i < K; ++i) {
        if (!PyLong_Check(a[i])) return false;
        to[i] = PyLong_AsLongLong(a[i]);
        if (to[i] == -1 && PyErr_Occurred()) return false;
    }
    return true;
}

bool expect(Py_ssize_t have, Py_ssize_t want)
{
    if (have == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, have);
    return false;
}

// entry, stream, q, k, v, q_out, k_cache, v_cache, page_table, positions, cos_sin,
// seq_of, k_scale, v_scale, interleaved, and of kv_append_at places
template <bool AT>
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (!expect(n, AT ? 16 : 15)) return nullptr;
    try {
        bool ok = true;
        const Tensor* t[12];
        for (int i = 0; i < 12; ++i) t[i] = tensor(a[2 + i], &ok);
        const Tensor *q = t[0], *k = t[1], *v = t[2], *q_out = t[3], *pos = t[7], *cs = t[8], *seq = t[9];
        xpress_kv_append_args x = {};
        if (!ok || !k || !v || !pos || (q != nullptr) != (q_out != nullptr) || k->dim() != 3 ||
            !cache(t[4], t[5], t[6], t[10], t[11], &x.cache)) {
            Py_RETURN_NONE;
        }
        const int64_t dev = t[4]->get_device(), T = k->size(0), heads = x.cache.heads, dim = x.cache.dim;
        const at::ScalarType type = k->scalar_type();
        x.dtype = code_of(*k);
        if (x.dtype < 0 || !rows(*k, type, {T, heads, dim}, dev) || !rows(*v, type, {T, heads, dim}, dev) ||
            !plain(pos, at::kInt, {T}, dev) || !plain(seq, at::kInt, {T}, dev)) {
            Py_RETURN_NONE;
        }
        if (q) {
            if (q->dim() != 3) Py_RETURN_NONE;
            x.Hq = q->size(1);
            if (!rows(*q, type, {T, x.Hq, dim}, dev) || !rows(*q_out, type, {T, x.Hq, dim}, dev)) Py_RETURN_NONE;
            x.q = q->data_ptr();
            x.q_out = q_out->data_ptr();
            x.stride_q_t = q->stride(0);
            x.stride_q_h = q->stride(1);
            x.stride_o_t = q_out->stride(0);
            x.stride_o_h = q_out->stride(1);
        }
        x.max_pos = 0x7FFFFFFFll;
        if (cs) {
            if (cs->dim() != 2 || !plain(cs, at::kFloat, {cs->size(0), cs->size(1)}, dev)) Py_RETURN_NONE;
            x.max_pos = cs->size(0);
            x.rot_dim = cs->size(1);
            x.cos_sin = address<const float>(cs);
        }
        x.k = k->data_ptr();
        x.v = v->data_ptr();
        x.positions = address<const int32_t>(pos);
        x.seq_of = address<const int32_t>(seq);
        x.T = T;
        const int in = PyObject_IsTrue(a[14]);
        if (in < 0) return nullptr;
        x.interleaved = in;
        x.stride_k_t = k->stride(0);
        x.stride_k_h = k->stride(1);
        x.stride_v_t = v->stride(0);
        x.stride_v_h = v->stride(1);
        if constexpr (AT) {
            const Tensor* at = tensor(a[15], &ok);
            if (!ok || !at || !plain(at, at::kInt, {T}, dev)) Py_RETURN_NONE;
            return call<const xpress_kv_append_args*, const int32_t*>(a[0], a[1], &x, address<const int32_t>(at));
        }
        return call<const xpress_kv_append_args*>(a[0], a[1], &x);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// entry, stream, q, k_cache, v_cache, page_table, lens, out, lse, k_scale, v_scale,
// max_len, window, scale (None: 1 / sqrt(dim)), and of the sparse forms sinks, of the
// tree's the tree
enum class Form { kDense, kSinks, kTree };

template <Form FORM>
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (!expect(n, 14 + (int)FORM)) return nullptr;
    try {
        bool ok = true;
        const Tensor* t[9];
        for (int i = 0; i < 9; ++i) t[i] = tensor(a[2 + i], &ok);
        const Tensor *q = t[0], *lens = t[4], *out = t[5], *lse = t[6];
        xpress_paged_attention_args x = {};
        if (!ok || !q || !lens || !out || q->dim() != 4 || !cache(t[1], t[2], t[3], t[7], t[8], &x.cache)) {
            Py_RETURN_NONE;
        }
        const int64_t dev = t[1]->get_device(), N = x.cache.seqs, Q = q->size(1), Hq = q->size(2),
                      dim = x.cache.dim;
        const at::ScalarType type = q->scalar_type();
        x.dtype = code_of(*q);
        if (x.dtype < 0 || !rows(*q, type, {N, Q, Hq, dim}, dev) || !rows(*out, type, {N, Q, Hq, dim}, dev) ||
            !plain(lse, at::kFloat, {N, Q, Hq}, dev) || !plain(lens, at::kInt, {N}, dev) ||
            !PyLong_Check(a[11]) || !PyLong_Check(a[12])) {
            Py_RETURN_NONE;
        }
        x.max_len = PyLong_AsLongLong(a[11]);
        x.window = PyLong_AsLongLong(a[12]);
        x.scale = a[13] == Py_None ? 1.0 / std::sqrt((double)dim) : PyFloat_AsDouble(a[13]);
        if (PyErr_Occurred()) return nullptr;
        x.q = q->data_ptr();
        x.out = out->data_ptr();
        x.lse = address<float>(lse);
        x.lens = address<const int32_t>(lens);
        x.Q = Q;
        x.Hq = Hq;
        x.stride_q_n = q->stride(0);
        x.stride_q_i = q->stride(1);
        x.stride_q_h = q->stride(2);
        x.stride_o_n = out->stride(0);
        x.stride_o_i = out->stride(1);
        x.stride_o_h = out->stride(2);
        using Args = const xpress_paged_attention_args*;
        if constexpr (FORM == Form::kDense) {
            return call<Args>(a[0], a[1], &x);
        } else {
            int64_t sinks[1];
            if (!whole(a + 14, sinks)) return PyErr_Occurred() ? nullptr : none();
            if constexpr (FORM == Form::kSinks) return call<Args, int64_t>(a[0], a[1], &x, sinks[0]);
            if constexpr (FORM == Form::kTree) {
                const Tensor* tree = tensor(a[15], &ok);
                if (!ok || !tree || tree->dim() != 3 || !rows(*tree, at::kInt, {N, Q, (Q + 31) / 32}, dev)) {
                    Py_RETURN_NONE;
                }
                return call<Args, const int32_t*, int64_t, int64_t, int64_t>(
                    a[0], a[1], &x, address<const int32_t>(tree), tree->stride(0), tree->stride(1), sinks[0]);
            }
        }
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// Logits: bf16, or their bits in 16-bit integers, with unit stride along the last
// dimension, in a storage that holds `bytes` from the first element on.  The rows'
// places come from the call's strides.
bool logits(const Tensor* t, int64_t bytes, int64_t dev)
{
    if (!t) return true;
    const at::ScalarType type = t->scalar_type();
    return (type == at::kBFloat16 || type == at::kShort || type == at::kUInt16) && on(*t, dev) &&
           (t->dim() == 0 || t->size(-1) <= 1 || t->stride(-1) == 1) && t->has_storage() &&
           (int64_t)t->storage().nbytes() - t->storage_offset() * 2 >= bytes;
}

// At least n numbers of this type, one after the other.
bool numbers(const Tensor* t, at::ScalarType type, int64_t n, int64_t dev)
{
    return t->scalar_type() == type && on(*t, dev) && t->is_contiguous() && t->numel() >= n;
}

// entry, stream, base, bias, blk, prob, temperature, top_k, top_p, min_p, u, N, B,
// V, stride_base_r, stride_bias_r
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    using In = const void*;
    using Out = void*;
    if (!expect(n, 16)) return nullptr;
    try {
        bool ok = true;
        const Tensor* t[9];
        for (int i = 0; i < 9; ++i) t[i] = tensor(a[2 + i], &ok);
        int64_t d[5];
        for (int i = 0; i < 5; ++i) {
            if (!PyLong_Check(a[11 + i])) Py_RETURN_NONE;
            d[i] = PyLong_AsLongLong(a[11 + i]);
        }
        if (PyErr_Occurred()) return nullptr;
        const int64_t most = 0x7FFFFFFFll, N = d[0], B = d[1], V = d[2];
        if (!ok || !t[0] || !t[2] || N < 0 || B < 1 || N > most / B || V < 1 || V > most || d[3] < V ||
            d[3] > (most << 16) || d[4] < 0 || d[4] > (most << 16)) {
            Py_RETURN_NONE;
        }
        const int64_t rows = N * (B - 1);
        const unsigned __int128 base = ((unsigned __int128)(rows - (rows > 0)) * d[3] + V) * 2u,
                                bias = ((unsigned __int128)(rows - (rows > 0)) * d[4] + V) * 2u,
                                far = (unsigned __int128)1 << 62;
        if (rows == 0 || base > far || bias > far || !t[0]->is_cuda()) Py_RETURN_NONE;
        const int64_t dev = t[0]->get_device();
        if (!logits(t[0], (int64_t)base, dev) || !logits(t[1], (int64_t)bias, dev) ||
            !numbers(t[2], at::kLong, N * B, dev) || !on_current(dev)) {
            Py_RETURN_NONE;
        }
        for (int i = 3; i < 9; ++i) {
            const at::ScalarType type = i == 5 ? at::kInt : at::kFloat;   // top_k; the others
            if (t[i] ? !numbers(t[i], type, rows, dev) : i != 3) Py_RETURN_NONE;
        }
        return call<In, In, Out, Out, In, In, In, In, In, int64_t, int64_t, int64_t, int64_t, int64_t>(
            a[0], a[1], address<void>(t[0]), address<void>(t[1]), address<void>(t[2]), address<void>(t[3]),
            address<void>(t[4]), address<void>(t[5]), address<void>(t[6]), address<void>(t[7]), address<void>(t[8]),
            N, B, V, d[3], d[4]);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// The counts of a pool's pages on the current device; *dev is the device.
bool counts(const Tensor* t, int64_t* dev)
{
    if (!t || t->dim() != 1 || t->scalar_type() != at::kInt || !t->is_cuda() || !t->is_contiguous()) return false;
    *dev = t->get_device();
    return on_current(*dev);
}

// An int32 table [rows, width].
bool table(const Tensor* t, int64_t dev)
{
    return t && t->dim() == 2 && rows(*t, at::kInt, {t->size(0), t->size(1)}, dev);
}

// n int32 numbers one after the other, in any shape.
bool flat(const Tensor* t, int64_t n, int64_t dev)
{
    return t && t->scalar_type() == at::kInt && t->is_contiguous() && on(*t, dev) && t->numel() == n;
}

using Ints = const int32_t*;
using IntsOut = int32_t*;

// entry, stream, refs, table, lens, src, new_refs, new_table, copies, missing, page_size
PyObject* kv_fork(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (!expect(n, 11)) return nullptr;
    try {
        bool ok = true;
        const Tensor* t[8];
        for (int i = 0; i < 8; ++i) t[i] = tensor(a[2 + i], &ok);
        int64_t dev = 0, page[1];
        if (!whole(a + 10, page)) return PyErr_Occurred() ? nullptr : none();
        if (!ok || !counts(t[0], &dev) || !table(t[1], dev) || !table(t[5], dev)) Py_RETURN_NONE;
        const int64_t pages = t[0]->size(0), N = t[1]->size(0), W = t[1]->size(1), M = t[5]->size(0);
        if (t[5]->size(1) != W || !t[2] || !plain(t[2], at::kInt, {N}, dev) || !flat(t[3], M, dev) || !t[4] ||
            !plain(t[4], at::kInt, {pages}, dev) || !t[6] || !plain(t[6], at::kInt, {M, 3}, dev) ||
            !plain(t[7], at::kInt, {1}, dev)) {
            Py_RETURN_NONE;
        }
        return call<Ints, int64_t, Ints, int64_t, Ints, int64_t, Ints, int64_t, int64_t, int64_t, IntsOut, IntsOut,
                    int64_t, IntsOut, IntsOut>(
            a[0], a[1], address<const int32_t>(t[0]), pages, address<const int32_t>(t[1]), t[1]->stride(0),
            address<const int32_t>(t[2]), N, address<const int32_t>(t[3]), M, W, page[0], address<int32_t>(t[4]),
            address<int32_t>(t[5]), t[5]->stride(0), address<int32_t>(t[6]), address<int32_t>(t[7]));
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// A cache without its table.
bool pool(const Tensor* k, const Tensor* v, xpress_kv_cache* c)
{
    if (!k || !v || k->dim() != 4 || !k->is_cuda() || v->sizes() != k->sizes() || v->strides() != k->strides() ||
        v->scalar_type() != k->scalar_type()) {
        return false;
    }
    c->dtype = code_of(*k);
    c->pages = k->size(0);
    c->heads = k->size(1);
    c->page_size = k->size(2);
    c->dim = k->size(3);
    if (c->dtype < 0 || (k->stride(3) != 1 && c->dim > 1) || !on(*v, k->get_device()) || !on_current(k->get_device())) {
        return false;
    }
    c->k = k->data_ptr();
    c->v = v->data_ptr();
    c->stride_page = k->stride(0);
    c->stride_head = k->stride(1);
    c->stride_token = k->stride(2);
    return true;
}

// entry, stream, k_cache, v_cache, copies
PyObject* kv_copy(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (!expect(n, 5)) return nullptr;
    try {
        bool ok = true;
        const Tensor* t[3];
        for (int i = 0; i < 3; ++i) t[i] = tensor(a[2 + i], &ok);
        xpress_kv_cache c = {};
        if (!ok || !t[2] || t[2]->dim() != 2 || !pool(t[0], t[1], &c) ||
            !plain(t[2], at::kInt, {t[2]->size(0), 3}, t[0]->get_device())) {
            Py_RETURN_NONE;
        }
        return call<const xpress_kv_cache*, Ints, int64_t>(a[0], a[1], &c, address<const int32_t>(t[2]),
                                                           t[2]->size(0));
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// entry, stream, refs, table, have, want, missing, page_size
PyObject* kv_grow(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (!expect(n, 8)) return nullptr;
    try {
        bool ok = true;
        const Tensor* t[5];
        for (int i = 0; i < 5; ++i) t[i] = tensor(a[2 + i], &ok);
        int64_t dev = 0, page[1];
        if (!whole(a + 7, page)) return PyErr_Occurred() ? nullptr : none();
        if (!ok || !counts(t[0], &dev) || !table(t[1], dev)) Py_RETURN_NONE;
        const int64_t N = t[1]->size(0);
        if (!t[2] || !plain(t[2], at::kInt, {N}, dev) || !t[3] || !plain(t[3], at::kInt, {N}, dev) ||
            !plain(t[4], at::kInt, {1}, dev)) {
            Py_RETURN_NONE;
        }
        return call<IntsOut, int64_t, IntsOut, int64_t, int64_t, int64_t, int64_t, Ints, Ints, IntsOut>(
            a[0], a[1], address<int32_t>(t[0]), t[0]->size(0), address<int32_t>(t[1]), t[1]->stride(0), N,
            t[1]->size(1), page[0], address<const int32_t>(t[2]), address<const int32_t>(t[3]),
            address<int32_t>(t[4]));
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// entry, stream, refs, table, lens, page_size, window, sinks
PyObject* kv_free(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (!expect(n, 8)) return nullptr;
    try {
        bool ok = true;
        const Tensor* t[3];
        for (int i = 0; i < 3; ++i) t[i] = tensor(a[2 + i], &ok);
        int64_t dev = 0, d[3];
        if (!whole(a + 5, d)) return PyErr_Occurred() ? nullptr : none();
        if (!ok || !counts(t[0], &dev) || !table(t[1], dev) || !t[2] ||
            !plain(t[2], at::kInt, {t[1]->size(0)}, dev)) {
            Py_RETURN_NONE;
        }
        return call<IntsOut, int64_t, IntsOut, int64_t, int64_t, int64_t, int64_t, Ints, int64_t, int64_t>(
            a[0], a[1], address<int32_t>(t[0]), t[0]->size(0), address<int32_t>(t[1]), t[1]->stride(0),
            t[1]->size(0), t[1]->size(1), d[0], address<const int32_t>(t[2]), d[1], d[2]);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// entry, stream, k_cache, v_cache, page_table, start, path, count
PyObject* kv_compact(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (!expect(n, 8)) return nullptr;
    try {
        bool ok = true;
        const Tensor* t[6];
        for (int i = 0; i < 6; ++i) t[i] = tensor(a[2 + i], &ok);
        xpress_kv_cache c = {};
        if (!ok || !cache(t[0], t[1], t[2], nullptr, nullptr, &c)) Py_RETURN_NONE;
        const int64_t dev = t[0]->get_device(), N = c.seqs;
        if (!table(t[4], dev) || t[4]->size(0) != N || !t[3] || !plain(t[3], at::kInt, {N}, dev) || !t[5] ||
            !plain(t[5], at::kInt, {N}, dev)) {
            Py_RETURN_NONE;
        }
        return call<const xpress_kv_cache*, Ints, Ints, int64_t, Ints, int64_t>(
            a[0], a[1], &c, address<const int32_t>(t[3]), address<const int32_t>(t[4]), t[4]->stride(0),
            address<const int32_t>(t[5]), t[4]->size(1));
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// entry, stream, base, bias, scores, best, rows, ids, N, beams, V, K, stride_base_r,
// stride_bias_r
PyObject* beam_select(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (!expect(n, 14)) return nullptr;
    try {
        bool ok = true;
        const Tensor* t[6];
        for (int i = 0; i < 6; ++i) t[i] = tensor(a[2 + i], &ok);
        int64_t d[6];
        if (!whole(a + 8, d)) return PyErr_Occurred() ? nullptr : none();
        const int64_t most = 0x7FFFFFFFll, N = d[0], beams = d[1], V = d[2], K = d[3];
        if (!ok || !t[0] || !t[2] || !t[3] || !t[4] || !t[5] || N < 1 || beams < 1 || N > most / beams || V < 1 ||
            V > most || K < 1 || K > most || d[4] < V || d[4] > (most << 16) || d[5] < 0 || d[5] > (most << 16) ||
            N > most / K || !t[0]->is_cuda()) {
            Py_RETURN_NONE;
        }
        const int64_t R = N * beams, dev = t[0]->get_device();
        const unsigned __int128 base = ((unsigned __int128)(R - 1) * d[4] + V) * 2u,
                                bias = ((unsigned __int128)(R - 1) * d[5] + V) * 2u,
                                far = (unsigned __int128)1 << 62;
        if (base > far || bias > far || !logits(t[0], (int64_t)base, dev) || !logits(t[1], (int64_t)bias, dev) ||
            !numbers(t[2], at::kFloat, R, dev) || !numbers(t[3], at::kFloat, N * K, dev) ||
            !numbers(t[4], at::kInt, N * K, dev) || !numbers(t[5], at::kLong, N * K, dev) || !on_current(dev)) {
            Py_RETURN_NONE;
        }
        return call<const void*, const void*, const float*, float*, int32_t*, void*, int64_t, int64_t, int64_t,
                    int64_t, int64_t, int64_t>(
            a[0], a[1], address<const void>(t[0]), address<const void>(t[1]), address<const float>(t[2]),
            address<float>(t[3]), address<int32_t>(t[4]), address<void>(t[5]), N, beams, V, K, d[4], d[5]);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// Rows behind the first dimension, each one after the other in memory, which holds the
// values themselves (not those whose conjugate or negative the tensor stands for).
bool whole_rows(const Tensor& t)
{
    if (t.is_conj() || t.is_neg()) return false;
    int64_t step = 1;
    for (int64_t i = t.dim() - 1; i > 0; --i) {
        if (t.size(i) != 1 && t.stride(i) != step) return false;
        step *= t.size(i);
    }
    return true;
}

// entry, stream, states, src
PyObject* beam_reorder(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (!expect(n, 4)) return nullptr;
    constexpr Py_ssize_t kMost = 64;
    if ((!PyList_CheckExact(a[2]) && !PyTuple_CheckExact(a[2])) || Py_SIZE(a[2]) > kMost) Py_RETURN_NONE;
    try {
        bool ok = true;
        const Tensor* src = tensor(a[3], &ok);
        if (!ok || !src || !src->is_cuda()) Py_RETURN_NONE;
        const int64_t dev = src->get_device(), M = src->numel();
        if (!flat(src, M, dev) || !on_current(dev)) Py_RETURN_NONE;
        xpress_beam_state x[kMost];
        const Py_ssize_t count = Py_SIZE(a[2]);
        int64_t N = 0;
        for (Py_ssize_t i = 0; i < count; ++i) {
            PyObject* pair = PySequence_Fast_GET_ITEM(a[2], i);
            if (!PyTuple_CheckExact(pair) || Py_SIZE(pair) != 2) Py_RETURN_NONE;
            const Tensor *from = tensor(PyTuple_GET_ITEM(pair, 0), &ok), *to = tensor(PyTuple_GET_ITEM(pair, 1), &ok);
            if (!ok || !from || !to || from->dim() < 1 || from->dim() != to->dim() ||
                from->sizes().slice(1) != to->sizes().slice(1) || from->scalar_type() != to->scalar_type() ||
                to->size(0) != M || (i > 0 && from->size(0) != N) || !on(*from, dev) || !on(*to, dev) ||
                !whole_rows(*from) || !whole_rows(*to)) {
                Py_RETURN_NONE;
            }
            N = from->size(0);
            const int64_t e = from->element_size();
            int64_t row = e;
            for (int64_t d = 1; d < from->dim(); ++d) row *= from->size(d);
            x[i] = xpress_beam_state{from->data_ptr(), to->data_ptr(), from->stride(0) * e, to->stride(0) * e, row};
        }
        return call<const xpress_beam_state*, int64_t, Ints, int64_t, int64_t>(
            a[0], a[1], x, (int64_t)count, address<const int32_t>(src), N, M);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);

PyMethodDef method(const char* name, PyCFunction f)
{
    return {name, f, METH_FASTCALL,
            "the C entry point of this name from tensors: its status, or None where the arguments are not regular"};
}

PyCFunction of(Fast f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {
    method("kv_append", of(append<false>)),
    method("kv_append_at", of(append<true>)),
    method("paged_attention", of(attention<Form::kDense>)),
    method("sink_attention", of(attention<Form::kSinks>)),
    method("tree_attention", of(attention<Form::kTree>)),
    method("sample", of(sample)),
    method("kv_fork", of(kv_fork)),
    method("kv_copy", of(kv_copy)),
    method("kv_grow", of(kv_grow)),
    method("kv_free", of(kv_free)),
    method("kv_compact", of(kv_compact)),
    method("beam_select", of(beam_select)),
    method("beam_reorder", of(beam_reorder)),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
