// ds41_binding.cpp - the Python side of the dense attention's calls as an extension
// module: their checks of tensors, new outputs and the call itself.
//
// What bounds the smallest of these calls is the host: a call through ctypes spends
// 20 us on attributes of tensors and conversions of 30 arguments in front of a kernel
// of 5 us.  Here the same checks take 1 us.  The entry points themselves come as
// addresses from the library that ds41.py has loaded (bind); nothing is linked to it.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

#include "ds41.h"

namespace {

using at::Tensor;

decltype(&ds41_kv_cache_write) g_write;
decltype(&ds41_kv_cache_read) g_read;
decltype(&ds41_prompt_attn_fwd) g_prompt;
decltype(&ds41_tree_attn_fwd) g_tree;
decltype(&ds41_tree_attn_workspace_bytes) g_tree_ws;
PyObject* g_failed;  // failed(name, code) raises

// An exception that a Python call has set.
void python_ok(bool ok) {
    if (!ok) throw python_error();
}
int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    python_ok(v != -1 || !PyErr_Occurred());
    return v;
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    python_ok(v != -1.0 || !PyErr_Occurred());
    return (float)v;
}
const Tensor& tensor(const char* name, PyObject* o) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, ": expected a tensor, got ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}
std::optional<Tensor> maybe(const char* name, PyObject* o) {
    if (o == Py_None) return std::nullopt;
    return tensor(name, o);
}

// The call runs on the current device's stream: the tensors are there.
at::Device here(const Tensor& t) {
    const at::Device dev = t.device();
    TORCH_CHECK_VALUE(dev.is_cuda(), "expected CUDA tensors, got one on ", dev);
    const int cur = c10::cuda::current_device();
    TORCH_CHECK_VALUE(dev.index() == cur, "the tensors are on ", dev,
                      ", the current device is cuda:", cur, ": the call runs on its stream");
    return dev;
}
// The pointer of a contiguous tensor of this shape and type on this device.
void* data(const char* name, const Tensor& t, at::Device dev, at::IntArrayRef shape,
           at::ScalarType type) {
    TORCH_CHECK_VALUE(t.device() == dev, name, " is on ", t.device(), ", expected ", dev);
    TORCH_CHECK_VALUE(t.sizes() == shape && t.scalar_type() == type, name, ": expected ", type, " ",
                      shape, ", got ", t.scalar_type(), " ", t.sizes());
    TORCH_CHECK_VALUE(t.is_contiguous(), name, ": expected a contiguous tensor");
    return t.data_ptr();
}
void* data_or_null(const char* name, PyObject* o, at::Device dev, at::IntArrayRef shape,
                   at::ScalarType type) {
    return o == Py_None ? nullptr : data(name, tensor(name, o), dev, shape, type);
}
int64_t length(const char* name, const Tensor& t) {
    TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) >= 1, name, ": expected [B + 1], got ", t.sizes());
    return t.size(0) - 1;
}

// A bf16 tensor [tokens, heads, hd] whose last dimension is dense (with `dense`: the
// heads too): pointer, and strides between tokens and heads.
struct Heads {
    const ds41_bf16* p;
    int64_t tok, head;
};
Heads heads(const char* name, const Tensor& t, at::Device dev, int64_t hd, bool dense = false) {
    TORCH_CHECK_VALUE(t.dim() == 3 && t.scalar_type() == at::kBFloat16 && t.size(2) == hd, name,
                      ": expected bfloat16 [tokens, heads, ", hd, "], got ", t.scalar_type(), " ",
                      t.sizes());
    TORCH_CHECK_VALUE(t.device() == dev, name, " is on ", t.device(), ", expected ", dev);
    const int64_t n = t.size(0), h = t.size(1);
    int64_t tok = t.stride(0), head = t.stride(1);
    if (h == 1 || n == 0) head = hd;  // strides that no address depends on
    if (n <= 1) tok = head == hd ? h * hd : hd;
    TORCH_CHECK_VALUE((t.stride(2) == 1 || hd <= 1) && (!dense || head == hd), name, ": strides ",
                      t.strides(), ": the last dimension", dense ? " and the heads" : "",
                      " must be dense");
    return {static_cast<const ds41_bf16*>(t.data_ptr()), tok, head};
}

struct Cache {
    void *k, *v;
    float *ks, *vs;
    int fmt;
    int64_t n_pages, kvh, page, hd;
};
Cache cache_of(PyObject* o, at::Device dev) {
    TORCH_CHECK_TYPE(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 4,
                     "cache: expected a KvCache, got ", Py_TYPE(o)->tp_name);
    const Tensor& k = tensor("cache.k", PyTuple_GET_ITEM(o, 0));
    const Tensor& v = tensor("cache.v", PyTuple_GET_ITEM(o, 1));
    PyObject *ks = PyTuple_GET_ITEM(o, 2), *vs = PyTuple_GET_ITEM(o, 3);
    TORCH_CHECK_VALUE(k.dim() == 4, "cache: expected [n_pages, kvh, page, hd], got ", k.sizes());
    const at::ScalarType type = k.scalar_type();
    const bool e4m3 = type == at::kFloat8_e4m3fn;
    TORCH_CHECK_VALUE(e4m3 || type == at::kBFloat16,
                      "cache: expected bfloat16 or float8_e4m3fn, got ", type);
    TORCH_CHECK_VALUE(e4m3 == (ks != Py_None) && e4m3 == (vs != Py_None),
                      "cache: an e4m3 cache has k_scales and v_scales, a bf16 cache none");
    Cache c{};
    c.n_pages = k.size(0);
    c.kvh = k.size(1);
    c.page = k.size(2);
    c.hd = k.size(3);
    c.fmt = e4m3 ? DS41_KV_E4M3 : DS41_KV_BF16;
    c.k = data("cache.k", k, dev, k.sizes(), type);
    c.v = data("cache.v", v, dev, k.sizes(), type);
    const at::IntArrayRef rows = k.sizes().slice(0, 3);
    c.ks = (float*)data_or_null("cache.k_scales", ks, dev, rows, at::kFloat);
    c.vs = (float*)data_or_null("cache.v_scales", vs, dev, rows, at::kFloat);
    return c;
}
const int32_t* pages(const Tensor& t, at::Device dev, int64_t B) {
    TORCH_CHECK_VALUE(t.dim() == 2, "page_table: expected [B, max_pages], got ", t.sizes());
    return (const int32_t*)data("page_table", t, dev, {B, t.size(1)}, at::kInt);
}
// The output given, or a new one.
Tensor output(const char* name, PyObject* o, at::Device dev, at::IntArrayRef shape) {
    if (o == Py_None)
        return at::empty(shape, at::TensorOptions().dtype(at::kBFloat16).device(dev));
    const Tensor& t = tensor(name, o);
    data(name, t, dev, shape, at::kBFloat16);
    return t;
}
ds41_stream_t stream_of(at::Device dev) {
    return (ds41_stream_t)c10::cuda::getCurrentCUDAStream(dev.index()).stream();
}
template <typename Call>
void run(const char* name, Call call) {
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = call();
    Py_END_ALLOW_THREADS;
    if (rc == DS41_OK) return;
    PyObject* r = PyObject_CallFunction(g_failed, "si", name, rc);
    Py_XDECREF(r);
    throw python_error();
}
PyObject* given_or(PyObject* o, const Tensor& t) {
    return o == Py_None ? THPVariable_Wrap(t) : Py_NewRef(o);
}
void count(Py_ssize_t n, Py_ssize_t want) {
    TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n);
}

// kv_cache_write(cache, k, v, slots)
PyObject* kv_cache_write(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    count(n_args, 4);
    const Tensor &k = tensor("k", a[1]), &v = tensor("v", a[2]);
    const at::Device dev = here(k);
    const Cache c = cache_of(a[0], dev);
    TORCH_CHECK_VALUE(k.dim() == 3 && k.size(1) == c.kvh && k.size(2) == c.hd &&
                          v.sizes() == k.sizes(),
                      "k, v: expected [n, ", c.kvh, ", ", c.hd, "], got ", k.sizes(), ", ",
                      v.sizes());
    const int64_t n = k.size(0);
    const Heads kh = heads("k", k, dev, c.hd, true), vh = heads("v", v, dev, c.hd, true);
    auto slots = (const int64_t*)data("slots", tensor("slots", a[3]), dev, {n}, at::kLong);
    const ds41_stream_t st = stream_of(dev);
    run("ds41_kv_cache_write", [&] {
        return g_write(kh.p, kh.tok, vh.p, vh.tok, slots, c.k, c.v, c.ks, c.vs, c.fmt, c.n_pages,
                       c.page, c.kvh, c.hd, n, st);
    });
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// kv_cache_read(cache, page_table, cu_k, rows, starts, k, v) -> (k, v)
PyObject* kv_cache_read(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    count(n_args, 7);
    const Tensor &table = tensor("page_table", a[1]), &cu = tensor("cu_k", a[2]);
    const at::Device dev = here(cu);
    const Cache c = cache_of(a[0], dev);
    const int64_t B = length("cu_k", cu), rows = integer(a[3]);
    TORCH_CHECK_VALUE(rows >= 0, "rows=", rows);
    const int32_t* pt = pages(table, dev, B);
    auto cup = (const int32_t*)data("cu_k", cu, dev, {B + 1}, at::kInt);
    auto starts = (const int32_t*)data_or_null("starts", a[4], dev, {B}, at::kInt);
    const int64_t shape[3] = {rows, c.kvh, c.hd};
    const Tensor k = output("k", a[5], dev, shape), v = output("v", a[6], dev, shape);
    auto kp = (ds41_bf16*)k.data_ptr(), vp = (ds41_bf16*)v.data_ptr();
    const ds41_stream_t st = stream_of(dev);
    run("ds41_kv_cache_read", [&] {
        return g_read(c.k, c.v, c.ks, c.vs, c.fmt, c.n_pages, c.page, c.kvh, c.hd, pt,
                      table.size(1), cup, starts, B, kp, vp, rows, st);
    });
    PyObject* both = PyTuple_New(2);
    python_ok(both != nullptr);
    PyTuple_SET_ITEM(both, 0, given_or(a[5], k));
    PyTuple_SET_ITEM(both, 1, given_or(a[6], v));
    return both;
    END_HANDLE_TH_ERRORS
}

// prompt_attn_fwd(q, k, v, cu_q, cu_k, max_q, scale, sink, window, o, lse) -> o
PyObject* prompt_attn_fwd(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    count(n_args, 11);
    const Tensor &q = tensor("q", a[0]), &k = tensor("k", a[1]), &v = tensor("v", a[2]);
    const Tensor &cu_q = tensor("cu_q", a[3]), &cu_k = tensor("cu_k", a[4]);
    const at::Device dev = here(q);
    TORCH_CHECK_VALUE(q.dim() == 3 && k.dim() == 3, "q, k: expected [tokens, heads, hd], got ",
                      q.sizes(), ", ", k.sizes());
    const int64_t Tq = q.size(0), nh = q.size(1), hd = q.size(2), Tk = k.size(0), kvh = k.size(1);
    const Heads qh = heads("q", q, dev, hd), kh = heads("k", k, dev, hd);
    const Heads vh = heads("v", v, dev, hd);
    TORCH_CHECK_VALUE(v.sizes() == k.sizes(), "v: expected ", k.sizes(), ", got ", v.sizes());
    const int64_t B = length("cu_q", cu_q), max_q = integer(a[5]), window = integer(a[8]);
    auto cq = (const int32_t*)data("cu_q", cu_q, dev, {B + 1}, at::kInt);
    auto ck = (const int32_t*)data("cu_k", cu_k, dev, {B + 1}, at::kInt);
    const float scale = real(a[6]);
    auto sink = (const float*)data_or_null("sink", a[7], dev, {nh}, at::kFloat);
    auto lse = (float*)data_or_null("lse", a[10], dev, {Tq, nh}, at::kFloat);
    const Tensor o = output("o", a[9], dev, q.sizes());
    auto op = (ds41_bf16*)o.data_ptr();
    const ds41_stream_t st = stream_of(dev);
    run("ds41_prompt_attn_fwd", [&] {
        return g_prompt(qh.p, qh.tok, qh.head, kh.p, kh.tok, kh.head, vh.p, vh.tok, vh.head, cq, ck,
                        B, Tq, Tk, max_q, nh, kvh, hd, scale, window, sink, op, lse, st);
    });
    return given_or(a[9], o);
    END_HANDLE_TH_ERRORS
}

// tree_attn_fwd(q, cache, page_table, lens, cu_q, max_q, max_len, scale, mask, sink,
// window, o, lse, ws) -> o
PyObject* tree_attn_fwd(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    count(n_args, 14);
    const Tensor &q = tensor("q", a[0]), &table = tensor("page_table", a[2]),
                 &lens = tensor("lens", a[3]), &cu_q = tensor("cu_q", a[4]);
    const at::Device dev = here(q);
    const Cache c = cache_of(a[1], dev);
    const Heads qh = heads("q", q, dev, c.hd);
    const int64_t Tq = q.size(0), nh = q.size(1), B = length("cu_q", cu_q);
    const int64_t max_q = integer(a[5]), max_len = integer(a[6]), window = integer(a[10]);
    const float scale = real(a[7]);
    const int32_t* pt = pages(table, dev, B);
    auto lp = (const int32_t*)data("lens", lens, dev, {B}, at::kInt);
    auto cq = (const int32_t*)data("cu_q", cu_q, dev, {B + 1}, at::kInt);
    int64_t words = 0;
    const int64_t* mask = nullptr;
    if (a[8] != Py_None) {
        const Tensor& m = tensor("mask", a[8]);
        TORCH_CHECK_VALUE(m.dim() == 2, "mask: expected [Tq, words], got ", m.sizes());
        words = m.size(1);
        mask = (const int64_t*)data("mask", m, dev, {Tq, words}, at::kLong);
    }
    auto sink = (const float*)data_or_null("sink", a[9], dev, {nh}, at::kFloat);
    auto lse = (float*)data_or_null("lse", a[12], dev, {Tq, nh}, at::kFloat);
    const Tensor o = output("o", a[11], dev, q.sizes());
    auto op = (ds41_bf16*)o.data_ptr();
    const size_t need = g_tree_ws(B, Tq, max_q, max_len, nh, c.kvh, c.hd, window, c.fmt);
    std::optional<Tensor> ws = maybe("ws", a[13]);
    if (ws) {
        TORCH_CHECK_VALUE(ws->device() == dev && ws->is_contiguous() && ws->nbytes() >= need,
                          "ws: expected a contiguous tensor of at least ", need, " bytes on ", dev);
    } else if (need > 0) {
        ws = at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(dev));
    }
    void* wp = ws && need > 0 ? ws->data_ptr() : nullptr;
    const ds41_stream_t st = stream_of(dev);
    run("ds41_tree_attn_fwd", [&] {
        return g_tree(qh.p, qh.tok, qh.head, c.k, c.v, c.ks, c.vs, c.fmt, c.n_pages, c.page, pt,
                      table.size(1), lp, cq, mask, words, B, Tq, max_q, max_len, nh, c.kvh, c.hd,
                      scale, window, sink, op, lse, wp, need, st);
    });
    return given_or(a[11], o);
    END_HANDLE_TH_ERRORS
}

// bind(write, read, prompt, tree, tree_workspace_bytes, failed): the addresses of the
// entry points, and what raises for a code that is not DS41_OK
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    count(n_args, 6);
    g_write = (decltype(g_write))integer(a[0]);
    g_read = (decltype(g_read))integer(a[1]);
    g_prompt = (decltype(g_prompt))integer(a[2]);
    g_tree = (decltype(g_tree))integer(a[3]);
    g_tree_ws = (decltype(g_tree_ws))integer(a[4]);
    Py_XSETREF(g_failed, Py_NewRef(a[5]));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define DS41_FAST(f) {#f, (PyCFunction)(void (*)())f, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {DS41_FAST(kv_cache_write), DS41_FAST(kv_cache_read),
                           DS41_FAST(prompt_attn_fwd), DS41_FAST(tree_attn_fwd), DS41_FAST(bind),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ds41_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ds41_binding(void) { return PyModule_Create(&g_module); }
