// calls.cpp -- the argument side of the per-layer calls, natively: checks of the tensors (type,
// device, shape, contiguity) and the C-ABI call.  A decode step makes these calls once per layer,
// and reading the same properties from Python costs more than the launch itself (8.6 against 4 us
// for paged_norm_rope_append on a Grace core).  Each function takes the pool's handle and the
// arguments of the Python function of its name in order, raises ValueError for a tensor that does
// not fit, and returns the call's kv_status.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <initializer_list>

#include "kv_paged.h"

namespace {

// A positional argument list being read; the first failure sets a Python error.
struct Args {
    PyObject* const* a;
    bool ok = true;
    int device = -1;                                // of the CUDA tensors

    void fail(PyObject* type, const char* name, const char* what)
    {
        if (ok) PyErr_Format(type, "%s must be %s", name, what);
        ok = false;
    }
    int64_t integer(int i)
    {
        if (!ok) return 0;
        const long long v = PyLong_AsLongLong(a[i]);
        if (v == -1 && PyErr_Occurred()) ok = false;
        return v;
    }
    int small(int i, const char* name)
    {
        const int64_t v = integer(i);
        if (v < INT32_MIN || v > INT32_MAX) fail(PyExc_ValueError, name, "a 32-bit integer");
        return static_cast<int>(v);
    }
    // A size that the C ABI takes as an int.
    void fits(int64_t n, const char* name)
    {
        if (n > INT32_MAX) fail(PyExc_ValueError, name, "of fewer than 2^31 entries per dimension");
    }
    float real(int i)
    {
        if (!ok) return 0.f;
        const double v = PyFloat_AsDouble(a[i]);
        if (v == -1.0 && PyErr_Occurred()) ok = false;
        return static_cast<float>(v);
    }
    bool truth(int i)
    {
        const int v = ok ? PyObject_IsTrue(a[i]) : 0;
        if (v < 0) ok = false;
        return v > 0;
    }
    kv_pool* pool(int i)
    {
        if (ok && a[i] == Py_None) {
            PyErr_SetString(PyExc_RuntimeError, "pool was destroyed");
            ok = false;
        }
        return reinterpret_cast<kv_pool*>(integer(i));
    }
    // Null for None where that is allowed, and after a failure.
    const at::Tensor* tensor(int i, const char* name, bool optional = false)
    {
        if (!ok || (optional && a[i] == Py_None)) return nullptr;
        if (!THPVariable_Check(a[i])) {
            fail(PyExc_ValueError, name, "a tensor");
            return nullptr;
        }
        return &THPVariable_Unpack(a[i]);
    }
    // Address of a tensor's first number.  A fake tensor has a CUDA device and no memory: its null
    // address would pass for an optional argument that is not there.
    void* address(const at::Tensor& t, const char* name)
    {
        void* p = t.numel() > 0 ? t.data_ptr() : nullptr;
        if (p == nullptr && t.numel() > 0) fail(PyExc_ValueError, name, "a tensor with memory");
        return p;
    }
    // The CUDA tensors at these places lie on one device (an address of another one is not for the
    // kernels to read; what is not a CUDA tensor is refused by name, below).  Only places of tensors:
    // asking a number whether it is one takes 50 ns.
    void one_device(std::initializer_list<int> places)
    {
        for (const int i : places) {
            if (!ok || a[i] == Py_None || !THPVariable_Check(a[i])) continue;
            const at::Tensor& t = THPVariable_Unpack(a[i]);
            if (!t.is_cuda()) continue;
            const int dev = static_cast<int>(t.get_device());
            if (device >= 0 && dev != device) fail(PyExc_ValueError, "the tensors", "on one device");
            device = dev;
        }
    }
    // And that is the pool's.
    bool on_device_of(const kv_pool* p)
    {
        int dev = -1;
        if (ok && kv_pool_shape(p, nullptr, nullptr, nullptr, nullptr, nullptr, &dev) == KV_OK && dev != device)
            fail(PyExc_ValueError, "the tensors", "on the pool's device");
        return ok;
    }
    // Address of a contiguous CUDA tensor of n numbers (n < 0: any).
    template <typename T = void>
    T* data(int i, at::ScalarType type, int64_t n, const char* name, bool optional = false)
    {
        const at::Tensor* t = tensor(i, name, optional);
        if (t == nullptr) return nullptr;
        if (t->scalar_type() != type || !t->is_cuda() || !t->is_contiguous() || (n >= 0 && t->numel() != n)) {
            if (ok)
                PyErr_Format(PyExc_ValueError, "%s must be a contiguous CUDA tensor of %s%s%lld numbers, got %s on %s, %lld numbers",
                             name, c10::toString(type), n >= 0 ? ", " : ", any ", static_cast<long long>(n < 0 ? 0 : n),
                             c10::toString(t->scalar_type()), t->is_cuda() ? "CUDA" : "another device",
                             static_cast<long long>(t->numel()));
            ok = false;
            return nullptr;
        }
        return static_cast<T*>(address(*t, name));
    }
    // A [tokens, heads, d] bf16 tensor whose token rows are contiguous: address and token stride.
    const void* rows(int i, int64_t n, int64_t heads, int64_t d, const char* name, int64_t* stride)
    {
        const at::Tensor* t = tensor(i, name);
        if (t == nullptr) return nullptr;
        if (t->scalar_type() != at::kBFloat16 || !t->is_cuda() || t->dim() != 3 || t->size(0) != n || t->size(1) != heads ||
            t->size(2) != d || t->stride(2) != 1 || (heads > 1 && t->stride(1) != d)) {
            if (ok)
                PyErr_Format(PyExc_ValueError, "%s must be a CUDA bf16 tensor [%lld, %lld, %lld] with the heads of a token contiguous",
                             name, static_cast<long long>(n), static_cast<long long>(heads), static_cast<long long>(d));
            ok = false;
            return nullptr;
        }
        *stride = n > 1 ? t->stride(0) : heads * d;
        return address(*t, name);
    }
};

PyObject* status(const Args& a, kv_status s) { return a.ok ? PyLong_FromLong(s) : nullptr; }

bool count(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want) PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", n, want);
    return n == want;
}

// Queries [batch, heads, q_len, d] or [batch, heads, d] with their block tables.
struct Queries {
    int64_t batch = 0, heads = 0, q_len = 1, max_blocks = 0, rows = 0;
    const void* q = nullptr;
    const int32_t* tables = nullptr;
    Queries(Args& a, int qi, int ti, int64_t d)
    {
        const at::Tensor* t = a.tensor(qi, "q");
        const at::Tensor* b = a.tensor(ti, "block_tables");
        if (!a.ok) return;
        if ((t->dim() != 3 && t->dim() != 4) || t->size(-1) != d || b->dim() != 2 || b->size(0) != t->size(0)) {
            a.fail(PyExc_ValueError, "q",
                   "[batch, q_heads, head_dim] or [batch, q_heads, q_len, head_dim], with one row of block_tables per sequence");
            return;
        }
        batch = t->size(0);
        heads = t->size(1);
        q_len = t->dim() == 4 ? t->size(2) : 1;
        max_blocks = b->size(1);
        for (const int64_t n : {batch, heads, q_len}) a.fits(n, "q");
        a.fits(max_blocks, "block_tables");
        if (!a.ok) return;
        rows = batch * heads * q_len;
        q = a.data(qi, at::kBFloat16, rows * d, "q");
        tables = a.data<const int32_t>(ti, at::kInt, batch * max_blocks, "block_tables");
    }
};

// (pool, head_dim, kv_heads, q, k, v, block_tables, context_lens, q_weight, k_weight, eps, rope_table,
//  interleaved, q_len, token_seq, token_pos, out, stream)
PyObject* norm_rope_append(PyObject*, PyObject* const* args, Py_ssize_t nargs)
{
    if (!count(nargs, 18)) return nullptr;
    Args a{args};
    kv_pool* pool = a.pool(0);
    const int64_t d = a.integer(1), kv = a.integer(2);
    const bool interleaved = a.truth(12);
    a.one_device({3, 4, 5, 6, 7, 8, 9, 11, 14, 15, 16});
    const at::Tensor* q = a.tensor(3, "q");
    const at::Tensor* tab = a.tensor(6, "block_tables");
    const at::Tensor* rope = a.tensor(11, "rope_table", true);
    if (a.ok && q->dim() != 3) a.fail(PyExc_ValueError, "q", "[tokens, q_heads, head_dim]");
    if (a.ok && tab->dim() != 2) a.fail(PyExc_ValueError, "block_tables", "[batch, max_blocks]");
    // (an empty table has no address, and none means no rotation)
    if (a.ok && rope != nullptr && (rope->dim() != 2 || rope->numel() == 0))
        a.fail(PyExc_ValueError, "rope_table", "[positions, rope_dim], of one position at least");
    if (!a.ok) return nullptr;
    const int64_t n = q->size(0), heads = q->size(1), batch = tab->size(0), max_blocks = tab->size(1);
    const int64_t positions = rope != nullptr ? rope->size(0) : 0, rope_dim = rope != nullptr ? rope->size(1) : 0;
    for (const int64_t m : {n, heads}) a.fits(m, "q");
    for (const int64_t m : {batch, max_blocks}) a.fits(m, "block_tables");
    a.fits(positions, "rope_table");
    a.fits(rope_dim, "rope_table");
    const int q_len = a.small(13, "q_len");
    if (a.ok && (q_len < 1 || n % q_len != 0)) a.fail(PyExc_ValueError, "the tokens", "q_len per sequence");
    int64_t qs = 0, ks = 0, vs = 0;
    const void* qp = a.rows(3, n, heads, d, "q", &qs);
    const void* kp = a.rows(4, n, kv, d, "k", &ks);
    const void* vp = a.rows(5, n, kv, d, "v", &vs);
    const int32_t* tables = a.data<const int32_t>(6, at::kInt, batch * max_blocks, "block_tables");
    const int32_t* ctx = a.data<const int32_t>(7, at::kInt, batch, "context_lens", true);
    const float* qw = a.data<const float>(8, at::kFloat, d, "q_weight", true);
    const float* kw = a.data<const float>(9, at::kFloat, d, "k_weight", true);
    const float eps = a.real(10);
    const float* table = a.data<const float>(11, at::kFloat, positions * rope_dim, "rope_table", true);
    const int32_t* seq = a.data<const int32_t>(14, at::kInt, n, "token_seq", true);
    const int32_t* pos = a.data<const int32_t>(15, at::kInt, n, "token_pos", true);
    void* out = a.data(16, at::kBFloat16, n * heads * d, "out");
    const int64_t stream = a.integer(17);
    if (!a.on_device_of(pool)) return nullptr;
    return status(a, paged_norm_rope_append(pool, qp, qs, kp, ks, vp, vs, static_cast<int>(heads), static_cast<int>(n), qw, kw,
                                            eps, table, static_cast<int>(positions), static_cast<int>(rope_dim),
                                            interleaved ? KV_ROPE_INTERLEAVED : KV_ROPE_HALF, seq, pos, tables,
                                            static_cast<int>(max_blocks), ctx, static_cast<int>(batch), q_len, out,
                                            reinterpret_cast<void*>(stream)));
}

// (pool, head_dim, q, block_tables, context_lens, scale, softcap, window, alibi_slopes, first_keys,
//  prefix_lens, kv_split_tokens, workspace, out, lse, stream)
PyObject* attention_masked(PyObject*, PyObject* const* args, Py_ssize_t nargs)
{
    if (!count(nargs, 16)) return nullptr;
    Args a{args};
    kv_pool* pool = a.pool(0);
    const int64_t d = a.integer(1);
    a.one_device({2, 3, 4, 8, 9, 10, 12, 13, 14});
    const Queries q(a, 2, 3, d);
    const int32_t* ctx = a.data<const int32_t>(4, at::kInt, q.batch, "context_lens");
    const float scale = a.real(5);
    kv_attention_mask m = {};
    m.softcap = a.real(6);
    m.window = a.small(7, "window");
    m.alibi_slopes = a.data<const float>(8, at::kFloat, q.heads, "alibi_slopes", true);
    m.first_keys = a.data<const int32_t>(9, at::kInt, q.batch, "first_keys", true);
    m.prefix_lens = a.data<const int32_t>(10, at::kInt, q.batch, "prefix_lens", true);
    const int split = a.small(11, "kv_split_tokens");
    void* ws = a.data(12, at::kByte, -1, "workspace", true);
    const size_t ws_bytes = ws != nullptr ? static_cast<size_t>(THPVariable_Unpack(args[12]).numel()) : 0;
    void* out = a.data(13, at::kBFloat16, q.rows * d, "out");
    float* lse = a.data<float>(14, at::kFloat, q.rows, "lse", true);
    const int64_t stream = a.integer(15);
    if (!a.on_device_of(pool)) return nullptr;
    return status(a, paged_attention_masked(pool, q.q, static_cast<int>(q.heads), static_cast<int>(q.q_len), q.tables,
                                            static_cast<int>(q.max_blocks), ctx, static_cast<int>(q.batch), scale, &m, split, ws,
                                            ws_bytes, out, lse, reinterpret_cast<void*>(stream)));
}

// (pool, head_dim, q, block_tables, context_lens, group_offsets, group_blocks, scale, kv_split_tokens,
//  workspace, out, lse, stream)
PyObject* shared_prefix_attention(PyObject*, PyObject* const* args, Py_ssize_t nargs)
{
    if (!count(nargs, 13)) return nullptr;
    Args a{args};
    kv_pool* pool = a.pool(0);
    const int64_t d = a.integer(1);
    a.one_device({2, 3, 4, 5, 6, 9, 10, 11});
    const Queries q(a, 2, 3, d);
    const int32_t* ctx = a.data<const int32_t>(4, at::kInt, q.batch, "context_lens");
    const at::Tensor* blk = a.tensor(6, "group_blocks");
    const int64_t groups = blk != nullptr ? blk->numel() : 0;
    a.fits(groups, "group_blocks");
    const int32_t* offsets = a.data<const int32_t>(5, at::kInt, groups + 1, "group_offsets");
    const int32_t* blocks = a.data<const int32_t>(6, at::kInt, groups, "group_blocks");
    const float scale = a.real(7);
    const int split = a.small(8, "kv_split_tokens");
    void* ws = a.data(9, at::kByte, -1, "workspace", true);
    const size_t ws_bytes = ws != nullptr ? static_cast<size_t>(THPVariable_Unpack(args[9]).numel()) : 0;
    void* out = a.data(10, at::kBFloat16, q.rows * d, "out");
    float* lse = a.data<float>(11, at::kFloat, q.rows, "lse", true);
    const int64_t stream = a.integer(12);
    if (!a.on_device_of(pool)) return nullptr;
    return status(a, paged_shared_prefix_attention(pool, q.q, static_cast<int>(q.heads), static_cast<int>(q.q_len), q.tables,
                                                   static_cast<int>(q.max_blocks), ctx, static_cast<int>(q.batch), offsets, blocks,
                                                   static_cast<int>(groups), scale, split, ws, ws_bytes, out, lse,
                                                   reinterpret_cast<void*>(stream)));
}

// The C entry: torch throws where a tensor has no strides or no memory (sparse, meta).
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t nargs)
{
    try {
        return F(self, args, nargs);
    } catch (const std::exception& e) {
        if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "a tensor without plain memory: %s", e.what());
    } catch (...) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a tensor without plain memory");
    }
    return nullptr;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<F>)); }

PyMethodDef methods[] = {
    {"norm_rope_append", fast<norm_rope_append>(), METH_FASTCALL, "paged_norm_rope_append"},
    {"attention_masked", fast<attention_masked>(), METH_FASTCALL, "paged_attention_masked"},
    {"shared_prefix_attention", fast<shared_prefix_attention>(), METH_FASTCALL, "paged_shared_prefix_attention"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "Native argument checks of the per-layer calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
