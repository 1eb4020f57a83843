// pkv_torch.cpp -- the Python side of the 8-bit and 4-bit caches' and the
// block selection's calls: takes torch tensors, checks them, calls the C
// functions of libpkv.so.  A decode step makes these calls once per layer; checked and
// converted in Python they cost 6 us each, more than most of their kernels.
//
// The module does not link to libpkv.so: bind() receives the addresses of the
// functions from the library that the package has loaded.  Every call returns
// a pkv_status (0 or negative), or, where the caller gave no workspace and one
// is needed, its size in bytes: the package allocates it and calls again.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdint>

#include "../../include/pkv.h"

namespace {

// The bound functions, in the order of the names that the package passes.
enum {
    kAppend, kSummarize, kSelect, kSelectBytes, kDecodeQ8, kDecodeSelected, kListBytes,
    kWriteQ4, kGatherQ4, kDecodeQ4, kQ4Bytes, kFunctions
};
void *g_function[kFunctions];

using T = const at::Tensor *;

// One call's arguments; the first failed check sets the Python error, and
// everything after it does nothing.
struct Call {
    PyObject *const *args;
    bool ok = true;
    T first = nullptr;
    int index = 0;

    explicit Call(PyObject *const *a) : args(a) {}

    bool value_error(const char *what)
    {
        if (ok)
            PyErr_SetString(PyExc_ValueError, what);
        return ok = false;
    }

    // Tensor argument i: contiguous, on the CUDA device of the first one.
    // `rows`: of three dimensions, of which the first may have any stride.
    T tensor(int i, const char *name, bool optional = false, bool rows = false)
    {
        PyObject *o = args[i];
        if (!ok || (optional && o == Py_None))
            return nullptr;
        if (!THPVariable_Check(o)) {
            PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
            ok = false;
            return nullptr;
        }
        T t = &THPVariable_Unpack(o);
        const bool laid_out = !rows ? t->is_contiguous()
                              : t->dim() == 3 && (t->numel() == 0 || ((t->size(2) == 1 || t->stride(2) == 1) &&
                                                                      (t->size(1) == 1 || t->stride(1) == t->size(2))));
        if (!t->is_cuda() || !laid_out) {
            PyErr_Format(PyExc_ValueError, rows ? "%s must be a CUDA tensor of three dimensions, contiguous but for the first"
                                                : "%s must be a contiguous CUDA tensor", name);
            ok = false;
            return nullptr;
        }
        if (!first) {
            first = t;
            index = t->device().index();
        } else if (t->device().index() != index) {
            PyErr_Format(PyExc_ValueError, "%s is on cuda:%d, other arguments on cuda:%d", name, (int)t->device().index(), index);
            ok = false;
            return nullptr;
        }
        return t;
    }

    int64_t integer(int i)
    {
        if (!ok)
            return 0;
        const long long v = PyLong_AsLongLong(args[i]);
        if (v == -1 && PyErr_Occurred())
            ok = false;
        return v;
    }

    double real(int i)
    {
        if (!ok)
            return 0;
        const double v = PyFloat_AsDouble(args[i]);
        if (v == -1.0 && PyErr_Occurred())
            ok = false;
        return v;
    }

    int narrow(int64_t v)
    {
        if (v < INT_MIN || v > INT_MAX)
            value_error("a size does not fit in 32 bits");
        return (int)v;
    }

    // The stream argument: None, an object with cuda_stream, or a number.
    void *stream(int i)
    {
        PyObject *o = args[i];
        if (!ok)
            return nullptr;
        if (o == Py_None)
            return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
        PyObject *s = PyObject_GetAttrString(o, "cuda_stream");
        if (!s) {
            PyErr_Clear();
            s = PyNumber_Index(o);
        }
        if (!s) {
            ok = false;
            return nullptr;
        }
        void *p = PyLong_AsVoidPtr(s);
        Py_DECREF(s);
        if (!p && PyErr_Occurred())
            ok = false;
        return p;
    }

    uint32_t *status(int i)
    {
        T t = tensor(i, "device_status", true);
        if (t && (t->numel() < 1 || t->element_size() != 4 || t->is_floating_point()))
            value_error("device_status must be an int32 or uint32 tensor");
        return ok && t ? static_cast<uint32_t *>(t->data_ptr()) : nullptr;
    }

    // Tables [B, MB] and lengths [B] -> MB.
    int tables(T block_tables, T context_lens, int64_t B)
    {
        if (!ok)
            return 0;
        if (block_tables->scalar_type() != at::kInt || context_lens->scalar_type() != at::kInt)
            value_error("block_tables and context_lens must be int32");
        else if (block_tables->dim() != 2 || block_tables->size(0) != B || context_lens->dim() != 1 || context_lens->size(0) != B)
            value_error("block_tables must be [B, MB] and context_lens [B]");
        return ok ? narrow(block_tables->size(1)) : 0;
    }

    void scales(T s, int64_t NB, int64_t Hk)
    {
        if (ok && (s->scalar_type() != at::kFloat || s->dim() != 2 || s->size(0) != NB || s->size(1) != (Hk + 3) / 4 * 4))
            value_error("scales must be float32 [num_blocks, num_kv_heads rounded up to a multiple of 4]");
    }

    void new_tokens(T query_start, int64_t B, int64_t tokens)
    {
        if (!ok)
            return;
        if (!query_start) {
            if (tokens != B)
                value_error("without query_start every sequence has one new token");
        } else if (query_start->scalar_type() != at::kInt || query_start->dim() != 1 || query_start->size(0) != B + 1) {
            value_error("query_start must be int32 [B + 1]");
        }
    }

    bool dims(T t, int64_t n, const char *what) { return !ok || t->dim() == n || value_error(what); }
};

// pkv_dtype of a tensor; -1: none.
int dtype(T t)
{
    switch (t->scalar_type()) {
    case at::kFloat: return PKV_F32;
    case at::kHalf: return PKV_F16;
    case at::kBFloat16: return PKV_BF16;
    case at::kFloat8_e4m3fn: return PKV_E4M3;
    default: return -1;
    }
}
bool floating(T t) { return dtype(t) >= 0 && dtype(t) != PKV_E4M3; }

void *address(T t) { return t ? t->data_ptr() : nullptr; }
template <typename P> P *as(T t) { return static_cast<P *>(address(t)); }

// Elements from one row [H, D] of t to the next.
int64_t row_stride(T t) { return t->size(0) > 1 ? t->stride(0) : t->size(1) * t->size(2); }

// Makes the tensors' device current while a call runs.
struct Device {
    int before;
    bool changed;
    explicit Device(int index) : before(c10::cuda::current_device()), changed(before != index)
    {
        if (changed)
            c10::cuda::set_device((c10::DeviceIndex)index);
    }
    ~Device()
    {
        if (changed)
            c10::cuda::set_device((c10::DeviceIndex)before);
    }
};

bool arguments(Py_ssize_t have, Py_ssize_t want)
{
    if (!g_function[0]) {
        PyErr_SetString(PyExc_RuntimeError, "the library's functions are not bound");
        return false;
    }
    if (have != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return false;
    }
    return true;
}

// Runs a call and turns what torch throws into a Python error.
template <typename F>
PyObject *guarded(F f)
{
    try {
        return f();
    } catch (const std::exception &e) {
        if (!PyErr_Occurred())
            PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// bind(addresses): one number per function.
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != kFunctions) {
        PyErr_SetString(PyExc_TypeError, "wrong number of functions");
        return nullptr;
    }
    for (int i = 0; i < kFunctions; ++i) {
        g_function[i] = PyLong_AsVoidPtr(args[i]);
        if (!g_function[i]) {
            if (!PyErr_Occurred())
                PyErr_SetString(PyExc_ValueError, "a function has no address");
            g_function[0] = nullptr;
            return nullptr;
        }
    }
    Py_RETURN_NONE;
}

// append(key, value, k_cache, v_cache, k_scales, v_scales, block_tables,
//        context_lens, query_start, device_status, stream)
PyObject *append(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    if (!arguments(nargs, 11))
        return nullptr;
    return guarded([&]() -> PyObject * {
        Call c(args);
        T key = c.tensor(0, "key"), value = c.tensor(1, "value"), k = c.tensor(2, "k_cache"), v = c.tensor(3, "v_cache");
        T ks = c.tensor(4, "k_scales"), vs = c.tensor(5, "v_scales"), bt = c.tensor(6, "block_tables");
        T cl = c.tensor(7, "context_lens"), qs = c.tensor(8, "query_start", true);
        uint32_t *status = c.status(9);
        if (!c.ok || !c.dims(key, 3, "shape mismatch") || !c.dims(k, 4, "shape mismatch"))
            return nullptr;
        const int64_t tokens = key->size(0), Hk = key->size(1), D = key->size(2), NB = k->size(0), bs = k->size(2);
        if (k->size(1) != Hk || k->size(3) != D || value->sizes() != key->sizes() || v->sizes() != k->sizes())
            c.value_error("shape mismatch");
        else if (!floating(key) || value->scalar_type() != key->scalar_type())
            c.value_error("key and value must share a floating dtype");
        else if (dtype(k) != PKV_E4M3 || dtype(v) != PKV_E4M3)
            c.value_error("k_cache and v_cache must be float8_e4m3fn");
        c.scales(ks, NB, Hk);
        c.scales(vs, NB, Hk);
        const int64_t B = cl->numel();
        const int MB = c.tables(bt, cl, B);
        c.new_tokens(qs, B, tokens);
        void *stream = c.stream(10);
        const int n[5] = {c.narrow(B), c.narrow(tokens), c.narrow(Hk), c.narrow(D), c.narrow(bs)};
        if (!c.ok)
            return nullptr;
        const Device device(c.index);
        return PyLong_FromLong(reinterpret_cast<decltype(&pkv_append_cache_q8)>(g_function[kAppend])(
            address(key), address(value), dtype(key), address(k), address(v), as<float>(ks), as<float>(vs), as<int32_t>(bt), MB,
            as<int32_t>(cl), as<int32_t>(qs), n[0], n[1], n[2], n[3], n[4], NB, status, stream));
    });
}

// summarize(k_cache, summaries, block_tables, context_lens, query_start,
//           num_tokens or None, k_scales, device_status, stream)
PyObject *summarize(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    if (!arguments(nargs, 9))
        return nullptr;
    return guarded([&]() -> PyObject * {
        Call c(args);
        T k = c.tensor(0, "k_cache"), sums = c.tensor(1, "summaries"), bt = c.tensor(2, "block_tables");
        T cl = c.tensor(3, "context_lens"), qs = c.tensor(4, "query_start", true), ks = c.tensor(6, "k_scales", true);
        uint32_t *status = c.status(7);
        if (!c.ok || !c.dims(k, 4, "shape mismatch"))
            return nullptr;
        const int64_t NB = k->size(0), Hk = k->size(1), bs = k->size(2), D = k->size(3);
        const bool q8 = dtype(k) == PKV_E4M3;
        if (dtype(k) < 0)
            c.value_error("k_cache must be float16, bfloat16 or float8_e4m3fn");
        else if (q8 != (ks != nullptr))
            c.value_error("k_scales go with a float8_e4m3fn cache");
        else if (q8)
            c.scales(ks, NB, Hk);
        if (c.ok && (sums->dim() != 4 || sums->size(0) != NB || sums->size(1) != Hk || sums->size(2) != 2 || sums->size(3) != D ||
                     dtype(sums) != (q8 ? PKV_BF16 : dtype(k))))
            c.value_error("summaries must be [NB, Hk, 2, D] of the cache's dtype (bfloat16 for an 8-bit cache)");
        const int64_t B = cl->numel();
        const int MB = c.tables(bt, cl, B);
        int64_t tokens = B;
        if (args[5] != Py_None)
            tokens = c.integer(5);
        else if (c.ok && qs)
            c.value_error("query_start needs num_tokens");
        c.new_tokens(qs, B, tokens);
        void *stream = c.stream(8);
        const int n[5] = {c.narrow(B), c.narrow(tokens), c.narrow(Hk), c.narrow(D), c.narrow(bs)};
        if (!c.ok)
            return nullptr;
        const Device device(c.index);
        return PyLong_FromLong(reinterpret_cast<decltype(&pkv_summarize_blocks)>(g_function[kSummarize])(
            address(k), dtype(k), as<float>(ks), address(sums), dtype(sums), as<int32_t>(bt), MB, as<int32_t>(cl), as<int32_t>(qs),
            n[0], n[1], n[2], n[3], n[4], NB, status, stream));
    });
}

// A workspace argument, or what the call needs if it is None.
struct Workspace {
    void *at = nullptr;
    size_t bytes = 0;
    bool given;
    Workspace(Call &c, int i)
    {
        T t = c.tensor(i, "workspace", true);
        given = t != nullptr;
        at = address(t);
        bytes = t ? (size_t)t->numel() * t->element_size() : 0;
    }
};

// select(selected, q, summaries, block_tables, context_lens, block_size,
//        keep_first, keep_last, max_context_len or None, workspace,
//        device_status, stream)
PyObject *select(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    if (!arguments(nargs, 12))
        return nullptr;
    return guarded([&]() -> PyObject * {
        Call c(args);
        T sel = c.tensor(0, "selected"), q = c.tensor(1, "q"), sums = c.tensor(2, "summaries"), bt = c.tensor(3, "block_tables");
        T cl = c.tensor(4, "context_lens");
        const int64_t bs = c.integer(5), first = c.integer(6), last = c.integer(7);
        Workspace ws(c, 9);
        uint32_t *status = c.status(10);
        if (!c.ok || !c.dims(q, 3, "shape mismatch") || !c.dims(sums, 4, "shape mismatch") || !c.dims(sel, 3, "shape mismatch"))
            return nullptr;
        const int64_t B = q->size(0), H = q->size(1), D = q->size(2), NB = sums->size(0), Hk = sums->size(1);
        if (sums->size(2) != 2 || sums->size(3) != D || sel->size(0) != B || sel->size(1) != Hk)
            c.value_error("shape mismatch");
        else if (sel->scalar_type() != at::kInt || !floating(q) || !floating(sums))
            c.value_error("selected must be int32, q and summaries floating");
        const int MB = c.tables(bt, cl, B);
        const int64_t most = args[8] == Py_None ? (int64_t)MB * c.narrow(bs) : c.integer(8);
        void *stream = c.stream(11);
        const int n[9] = {c.narrow(B), c.narrow(H), c.narrow(Hk), c.narrow(D), c.narrow(bs), c.narrow(most), c.narrow(sel->size(2)),
                          c.narrow(first), c.narrow(last)};
        if (!c.ok)
            return nullptr;
        const Device device(c.index);
        if (!ws.given) {
            const size_t need = reinterpret_cast<decltype(&pkv_select_blocks_workspace_bytes)>(g_function[kSelectBytes])(n[0], n[2], n[5], n[4]);
            if (need)
                return PyLong_FromSize_t(need);
        }
        return PyLong_FromLong(reinterpret_cast<decltype(&pkv_select_blocks)>(g_function[kSelect])(
            as<int32_t>(sel), address(q), dtype(q), address(sums), dtype(sums), as<int32_t>(bt), MB, as<int32_t>(cl), n[0], n[1], n[2],
            n[3], n[4], NB, n[5], n[6], n[7], n[8], ws.at, ws.bytes, status, stream));
    });
}

// decode(out, q, k_cache, v_cache, k_scales, v_scales, block_tables,
//        context_lens, selected, scale, max_context_len or None,
//        partition_size, workspace, device_status, stream): over the selected
// blocks unless `selected` is None
PyObject *decode(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    if (!arguments(nargs, 15))
        return nullptr;
    return guarded([&]() -> PyObject * {
        Call c(args);
        const bool select = args[8] != Py_None;
        T out = c.tensor(0, "out"), q = c.tensor(1, "q"), k = c.tensor(2, "k_cache"), v = c.tensor(3, "v_cache");
        T ks = c.tensor(4, "k_scales", select), vs = c.tensor(5, "v_scales", select), bt = c.tensor(6, "block_tables");
        T cl = c.tensor(7, "context_lens"), sel = c.tensor(8, "selected", true);
        const double scale = c.real(9);
        const int64_t partition = c.integer(11);
        Workspace ws(c, 12);
        uint32_t *status = c.status(13);
        if (!c.ok || !c.dims(q, 3, "shape mismatch") || !c.dims(k, 4, "shape mismatch"))
            return nullptr;
        const int64_t B = q->size(0), H = q->size(1), D = q->size(2), NB = k->size(0), Hk = k->size(1), bs = k->size(2);
        const bool q8 = dtype(k) == PKV_E4M3;
        if (k->size(3) != D || v->sizes() != k->sizes() || out->sizes() != q->sizes())
            c.value_error("shape mismatch");
        else if (!floating(out) || !floating(q))
            c.value_error("q and out must be floating");
        else if (!select && (!q8 || dtype(v) != PKV_E4M3))
            c.value_error("k_cache and v_cache must be float8_e4m3fn");
        else if (v->scalar_type() != k->scalar_type() || (!q8 && k->scalar_type() != q->scalar_type()))
            c.value_error("q, k_cache and v_cache must share a dtype, or the caches be float8_e4m3fn");
        else if ((ks != nullptr) != q8 || (vs != nullptr) != q8)
            c.value_error("k_scales and v_scales go with float8_e4m3fn caches");
        if (c.ok && q8) {
            c.scales(ks, NB, Hk);
            c.scales(vs, NB, Hk);
        }
        if (c.ok && select && (sel->scalar_type() != at::kInt || sel->dim() != 3 || sel->size(0) != B || sel->size(1) != Hk))
            c.value_error("selected must be int32 [B, Hk, K]");
        const int MB = c.tables(bt, cl, B);
        const int64_t most = args[10] == Py_None ? (int64_t)MB * c.narrow(bs) : c.integer(10);
        void *stream = c.stream(14);
        const int K = select && c.ok ? c.narrow(sel->size(2)) : 0;
        const int n[7] = {c.narrow(B), c.narrow(H), c.narrow(Hk), c.narrow(D), c.narrow(bs), c.narrow(most), c.narrow(partition)};
        if (!c.ok)
            return nullptr;
        const Device device(c.index);
        if (!ws.given && bs > 0) {
            const size_t need = reinterpret_cast<decltype(&pkv_paged_attention_list_workspace_bytes)>(g_function[kListBytes])(
                n[0], n[1], n[2], n[3], n[4], select ? K : (int)((most + bs - 1) / bs), n[6]);
            if (need)
                return PyLong_FromSize_t(need);
        }
        if (select)
            return PyLong_FromLong(reinterpret_cast<decltype(&pkv_paged_attention_decode_selected)>(g_function[kDecodeSelected])(
                address(out), dtype(out), address(q), dtype(q), address(k), address(v), dtype(k), as<float>(ks), as<float>(vs),
                as<int32_t>(bt), MB, as<int32_t>(cl), as<int32_t>(sel), K, n[0], n[1], n[2], n[3], n[4], NB, n[5], (float)scale, n[6],
                ws.at, ws.bytes, status, stream));
        return PyLong_FromLong(reinterpret_cast<decltype(&pkv_paged_attention_decode_q8)>(g_function[kDecodeQ8])(
            address(out), dtype(out), address(q), dtype(q), address(k), address(v), as<float>(ks), as<float>(vs), as<int32_t>(bt), MB,
            as<int32_t>(cl), n[0], n[1], n[2], n[3], n[4], NB, n[5], (float)scale, n[6], ws.at, ws.bytes, status, stream));
    });
}

// What the 4-bit cache's calls ask of their caches: uint8 [NB, Hk, bs, D / 2 + D / 16].
void q4_caches(Call &c, T k, T v, int64_t Hk, int64_t D)
{
    if (!c.ok)
        return;
    if (k->scalar_type() != at::kByte || v->scalar_type() != at::kByte)
        c.value_error("k_cache and v_cache must be uint8");
    else if (k->dim() != 4 || v->sizes() != k->sizes() || k->size(1) != Hk || D % 16 || k->size(3) != D / 2 + D / 16)
        c.value_error("k_cache and v_cache must be [NB, Hk, bs, D / 2 + D / 16]");
}

void slots(Call &c, T mapping, int64_t tokens)
{
    if (c.ok && (mapping->scalar_type() != at::kLong || mapping->dim() != 1 || mapping->size(0) != tokens))
        c.value_error("slot_mapping must be int64 [T]");
}

// write_q4(key, value, k_cache, v_cache, slot_mapping, device_status, stream)
PyObject *write_q4(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    if (!arguments(nargs, 7))
        return nullptr;
    return guarded([&]() -> PyObject * {
        Call c(args);
        T key = c.tensor(0, "key", false, true), value = c.tensor(1, "value", false, true);
        T k = c.tensor(2, "k_cache"), v = c.tensor(3, "v_cache"), at = c.tensor(4, "slot_mapping");
        uint32_t *status = c.status(5);
        if (!c.ok)
            return nullptr;
        const int64_t tokens = key->size(0), Hk = key->size(1), D = key->size(2);
        if (value->sizes() != key->sizes())
            c.value_error("shape mismatch");
        else if (!floating(key) || value->scalar_type() != key->scalar_type())
            c.value_error("key and value must share a floating dtype");
        q4_caches(c, k, v, Hk, D);
        slots(c, at, tokens);
        void *stream = c.stream(6);
        const int n[3] = {c.narrow(tokens), c.narrow(Hk), c.narrow(D)};
        const int bs = c.ok ? c.narrow(k->size(2)) : 0;
        if (!c.ok)
            return nullptr;
        const Device device(c.index);
        return PyLong_FromLong(reinterpret_cast<decltype(&pkv_reshape_and_cache_q4)>(g_function[kWriteQ4])(
            address(key), row_stride(key), address(value), row_stride(value), dtype(key), address(k), address(v), as<int64_t>(at), n[0],
            n[1], n[2], bs, k->size(0), status, stream));
    });
}

// gather_q4(key, value, k_cache, v_cache, slot_mapping, cache's pkv_dtype or
//           None: key's, device_status, stream)
PyObject *gather_q4(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    if (!arguments(nargs, 8))
        return nullptr;
    return guarded([&]() -> PyObject * {
        Call c(args);
        T key = c.tensor(0, "key", false, true), value = c.tensor(1, "value", false, true);
        T k = c.tensor(2, "k_cache"), v = c.tensor(3, "v_cache"), at = c.tensor(4, "slot_mapping");
        uint32_t *status = c.status(6);
        if (!c.ok)
            return nullptr;
        const int64_t tokens = key->size(0), Hk = key->size(1), D = key->size(2);
        if (value->sizes() != key->sizes())
            c.value_error("shape mismatch");
        else if (!floating(key) || value->scalar_type() != key->scalar_type())
            c.value_error("key and value must share a floating dtype");
        q4_caches(c, k, v, Hk, D);
        slots(c, at, tokens);
        const int kind = !c.ok ? 0 : args[5] == Py_None ? dtype(key) : c.narrow(c.integer(5));
        void *stream = c.stream(7);
        const int n[3] = {c.narrow(tokens), c.narrow(Hk), c.narrow(D)};
        const int bs = c.ok ? c.narrow(k->size(2)) : 0;
        if (!c.ok)
            return nullptr;
        const Device device(c.index);
        return PyLong_FromLong(reinterpret_cast<decltype(&pkv_gather_cache_q4)>(g_function[kGatherQ4])(
            address(key), row_stride(key), address(value), row_stride(value), dtype(key), address(k), address(v), kind,
            as<int64_t>(at), n[0], n[1], n[2], bs, k->size(0), status, stream));
    });
}

// decode_q4(out, q, k_cache, v_cache, block_tables, context_lens, scale,
//           max_context_len or None, partition_size, workspace, device_status,
//           stream)
PyObject *decode_q4(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    if (!arguments(nargs, 12))
        return nullptr;
    return guarded([&]() -> PyObject * {
        Call c(args);
        T out = c.tensor(0, "out"), q = c.tensor(1, "q", false, true), k = c.tensor(2, "k_cache"), v = c.tensor(3, "v_cache");
        T bt = c.tensor(4, "block_tables"), cl = c.tensor(5, "context_lens");
        const double scale = c.real(6);
        const int64_t partition = c.integer(8);
        Workspace ws(c, 9);
        uint32_t *status = c.status(10);
        if (!c.ok || !c.dims(k, 4, "shape mismatch"))
            return nullptr;
        const int64_t B = q->size(0), H = q->size(1), D = q->size(2), NB = k->size(0), Hk = k->size(1), bs = k->size(2);
        if (out->sizes() != q->sizes())
            c.value_error("shape mismatch");
        else if (!floating(out) || !floating(q))
            c.value_error("q and out must be floating");
        q4_caches(c, k, v, Hk, D);
        const int MB = c.tables(bt, cl, B);
        const int64_t most = args[7] == Py_None ? (int64_t)MB * c.narrow(bs) : c.integer(7);
        void *stream = c.stream(11);
        const int n[7] = {c.narrow(B), c.narrow(H), c.narrow(Hk), c.narrow(D), c.narrow(bs), c.narrow(most), c.narrow(partition)};
        if (!c.ok)
            return nullptr;
        const Device device(c.index);
        if (!ws.given) {
            const size_t need = reinterpret_cast<decltype(&pkv_paged_attention_q4_workspace_bytes)>(g_function[kQ4Bytes])(
                n[0], n[1], n[2], n[3], n[4], n[5], n[6]);
            if (need)
                return PyLong_FromSize_t(need);
        }
        return PyLong_FromLong(reinterpret_cast<decltype(&pkv_paged_attention_decode_q4)>(g_function[kDecodeQ4])(
            address(out), dtype(out), address(q), row_stride(q), dtype(q), address(k), address(v), as<int32_t>(bt), MB,
            as<int32_t>(cl), n[0], n[1], n[2], n[3], n[4], NB, n[5], (float)scale, n[6], ws.at, ws.bytes, status, stream));
    });
}

PyMethodDef g_methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"summarize", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(summarize)), METH_FASTCALL, nullptr},
    {"select", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(select)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode)), METH_FASTCALL, nullptr},
    {"write_q4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(write_q4)), METH_FASTCALL, nullptr},
    {"gather_q4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gather_q4)), METH_FASTCALL, nullptr},
    {"decode_q4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode_q4)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_pkv_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pkv_torch(void) { return PyModule_Create(&g_module); }
