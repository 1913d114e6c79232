// ds41_binding.cpp - the Python side of the calls of the dense attention, its pages and
// blocks, and of beam search as an extension module: their checks of tensors, new outputs
// and the call itself.
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
#include <type_traits>

#include "ds41.h"

namespace {

using at::Tensor;

decltype(&ds41_kv_cache_write) g_write;
decltype(&ds41_kv_cache_read) g_read;
decltype(&ds41_prompt_attn_fwd) g_prompt;
decltype(&ds41_tree_attn_fwd) g_tree;
decltype(&ds41_tree_attn_workspace_bytes) g_tree_ws;
decltype(&ds41_kv_pages_take) g_take;
decltype(&ds41_kv_pages_free) g_free;
decltype(&ds41_kv_pages_fork) g_fork;
decltype(&ds41_kv_pages_fork_workspace_bytes) g_fork_ws;
decltype(&ds41_kv_pages_copy) g_copy;
decltype(&ds41_kv_pages_compact) g_compact;
decltype(&ds41_kv_pages_compact_workspace_bytes) g_compact_ws;
decltype(&ds41_beam_select) g_beam;
decltype(&ds41_beam_select_workspace_bytes) g_beam_ws;
decltype(&ds41_kv_block_keys) g_keys;
decltype(&ds41_block_select) g_select;
decltype(&ds41_block_attn_fwd) g_blocks;
decltype(&ds41_block_prompt_attn_fwd) g_block_prompt;
decltype(&ds41_block_prompt_attn_workspace_bytes) g_block_prompt_ws;
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
Tensor output(const char* name, PyObject* o, at::Device dev, at::IntArrayRef shape,
              at::ScalarType type = at::kBFloat16) {
    if (o == Py_None) return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
    const Tensor& t = tensor(name, o);
    data(name, t, dev, shape, type);
    return t;
}
// The scratch of a call: what is given, or new.
struct Scratch {
    std::optional<Tensor> t;
    void* p = nullptr;
    Scratch(PyObject* o, at::Device dev, size_t need) : t(maybe("ws", o)) {
        if (t) {
            TORCH_CHECK_VALUE(t->device() == dev && t->is_contiguous() && t->nbytes() >= need,
                              "ws: expected a contiguous tensor of at least ", need, " bytes on ",
                              dev);
        } else if (need > 0) {
            t = at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(dev));
        }
        if (t && need > 0) p = t->data_ptr();
    }
};
// A cache's block keys, or none.
struct Keys {
    int8_t* codes = nullptr;
    float* scales = nullptr;
};
Keys keys_of(PyObject* o, at::Device dev, int64_t n_pages, int64_t kvh, int64_t hd) {
    if (o == Py_None) return {};
    TORCH_CHECK_TYPE(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 2,
                     "keys: expected BlockKeys, got ", Py_TYPE(o)->tp_name);
    return {(int8_t*)data("keys.codes", tensor("keys.codes", PyTuple_GET_ITEM(o, 0)), dev,
                          {n_pages, kvh, hd}, at::kChar),
            (float*)data("keys.scales", tensor("keys.scales", PyTuple_GET_ITEM(o, 1)), dev,
                         {n_pages, kvh}, at::kFloat)};
}
const int32_t* ints(const char* name, PyObject* o, at::Device dev, int64_t n) {
    return (const int32_t*)data(name, tensor(name, o), dev, {n}, at::kInt);
}
int64_t count_of(const char* name, const Tensor& t) {
    TORCH_CHECK_VALUE(t.dim() == 1, name, ": expected one dimension, got ", t.sizes());
    return t.size(0);
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
    const Scratch ws(a[13], dev, need);
    const ds41_stream_t st = stream_of(dev);
    run("ds41_tree_attn_fwd", [&] {
        return g_tree(qh.p, qh.tok, qh.head, c.k, c.v, c.ks, c.vs, c.fmt, c.n_pages, c.page, pt,
                      table.size(1), lp, cq, mask, words, B, Tq, max_q, max_len, nh, c.kvh, c.hd,
                      scale, window, sink, op, lse, ws.p, need, st);
    });
    return given_or(a[11], o);
    END_HANDLE_TH_ERRORS
}

// kv_pages_take(refs, page_table, lens, new_lens, page, ws)
PyObject* kv_pages_take(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    count(n_args, 6);
    const Tensor &refs = tensor("refs", a[0]), &table = tensor("page_table", a[1]);
    const at::Device dev = here(refs);
    const int64_t n_pages = count_of("refs", refs), page = integer(a[4]);
    const int64_t B = count_of("lens", tensor("lens", a[2]));
    auto rp = (int32_t*)ints("refs", a[0], dev, n_pages);
    auto pt = (int32_t*)pages(table, dev, B);
    auto lp = ints("lens", a[2], dev, B), np = ints("new_lens", a[3], dev, B);
    const Scratch ws(a[5], dev, (size_t)n_pages * 4);
    const ds41_stream_t st = stream_of(dev);
    run("ds41_kv_pages_take", [&] {
        return g_take(rp, n_pages, page, pt, table.size(1), lp, np, B, ws.p, (size_t)n_pages * 4,
                      st);
    });
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// kv_pages_free(refs, page_table, lens, page)
PyObject* kv_pages_free(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    count(n_args, 4);
    const Tensor &refs = tensor("refs", a[0]), &table = tensor("page_table", a[1]);
    const at::Device dev = here(refs);
    const int64_t n_pages = count_of("refs", refs), page = integer(a[3]);
    const int64_t B = count_of("lens", tensor("lens", a[2]));
    auto rp = (int32_t*)ints("refs", a[0], dev, n_pages);
    const int32_t* pt = pages(table, dev, B);
    auto lp = ints("lens", a[2], dev, B);
    const ds41_stream_t st = stream_of(dev);
    run("ds41_kv_pages_free",
        [&] { return g_free(rp, n_pages, page, pt, table.size(1), lp, B, st); });
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// kv_pages_fork(cache, refs, page_table, lens, parents, table_out, lens_out, replace,
// keys, ws) -> (table_out, lens_out)
PyObject* kv_pages_fork(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    count(n_args, 10);
    const Tensor &refs = tensor("refs", a[1]), &table = tensor("page_table", a[2]);
    const at::Device dev = here(refs);
    const Cache c = cache_of(a[0], dev);
    const int64_t B = count_of("lens", tensor("lens", a[3]));
    const int64_t n = count_of("parents", tensor("parents", a[4]));
    auto rp = (int32_t*)ints("refs", a[1], dev, c.n_pages);
    const int32_t* pt = pages(table, dev, B);
    auto lp = ints("lens", a[3], dev, B), pp = ints("parents", a[4], dev, n);
    const int64_t max_pages = table.size(1);
    const Tensor out = output("table_out", a[5], dev, {n, max_pages}, at::kInt);
    const Tensor out_lens = output("lens_out", a[6], dev, {n}, at::kInt);
    const int replace = PyObject_IsTrue(a[7]);
    python_ok(replace >= 0);
    const Keys keys = keys_of(a[8], dev, c.n_pages, c.kvh, c.hd);
    const size_t need = g_fork_ws(c.n_pages, B, n);
    const Scratch ws(a[9], dev, need);
    const ds41_stream_t st = stream_of(dev);
    run("ds41_kv_pages_fork", [&] {
        return g_fork(c.k, c.v, c.ks, c.vs, c.fmt, c.n_pages, c.page, c.kvh, c.hd, keys.codes,
                      keys.scales, rp, pt, max_pages, lp, B, pp, n, replace,
                      (int32_t*)out.data_ptr(), (int32_t*)out_lens.data_ptr(), ws.p, need, st);
    });
    PyObject* both = PyTuple_New(2);
    python_ok(both != nullptr);
    PyTuple_SET_ITEM(both, 0, given_or(a[5], out));
    PyTuple_SET_ITEM(both, 1, given_or(a[6], out_lens));
    return both;
    END_HANDLE_TH_ERRORS
}

// kv_pages_copy(cache, src, dst, rows, keys)
PyObject* kv_pages_copy(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    count(n_args, 5);
    const Tensor& src = tensor("src", a[1]);
    const at::Device dev = here(src);
    const Cache c = cache_of(a[0], dev);
    const int64_t n = count_of("src", src);
    auto sp = ints("src", a[1], dev, n), dp = ints("dst", a[2], dev, n);
    auto rp = (const int32_t*)data_or_null("rows", a[3], dev, {n}, at::kInt);
    const Keys keys = keys_of(a[4], dev, c.n_pages, c.kvh, c.hd);
    const ds41_stream_t st = stream_of(dev);
    run("ds41_kv_pages_copy", [&] {
        return g_copy(c.k, c.v, c.ks, c.vs, c.fmt, c.n_pages, c.page, c.kvh, c.hd, keys.codes,
                      keys.scales, sp, dp, rp, n, st);
    });
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// kv_pages_compact(cache, refs, page_table, lens, keys, live, ws) -> live
PyObject* kv_pages_compact(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    count(n_args, 7);
    const Tensor &refs = tensor("refs", a[1]), &table = tensor("page_table", a[2]);
    const at::Device dev = here(refs);
    const Cache c = cache_of(a[0], dev);
    const int64_t B = count_of("lens", tensor("lens", a[3]));
    auto rp = (int32_t*)ints("refs", a[1], dev, c.n_pages);
    auto pt = (int32_t*)pages(table, dev, B);
    auto lp = ints("lens", a[3], dev, B);
    const Keys keys = keys_of(a[4], dev, c.n_pages, c.kvh, c.hd);
    const Tensor live = output("live", a[5], dev, {1}, at::kInt);
    const size_t need = g_compact_ws(c.n_pages);
    const Scratch ws(a[6], dev, need);
    const ds41_stream_t st = stream_of(dev);
    run("ds41_kv_pages_compact", [&] {
        return g_compact(c.k, c.v, c.ks, c.vs, c.fmt, c.n_pages, c.page, c.kvh, c.hd, keys.codes,
                         keys.scales, rp, pt, table.size(1), lp, B, (int32_t*)live.data_ptr(),
                         ws.p, need, st);
    });
    return given_or(a[5], live);
    END_HANDLE_TH_ERRORS
}

// beam_select(logits, scores, k, ended, end_token, out_scores, parents, tokens, ws)
// -> (out_scores, parents, tokens)
PyObject* beam_select(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    count(n_args, 9);
    const Tensor& x = tensor("logits", a[0]);
    const at::Device dev = here(x);
    const bool bf16 = x.scalar_type() == at::kBFloat16;
    TORCH_CHECK_VALUE(x.dim() == 3 && (bf16 || x.scalar_type() == at::kFloat),
                      "logits: expected float32 or bfloat16 [B, W, V], got ", x.scalar_type(), " ",
                      x.sizes());
    const int64_t B = x.size(0), W = x.size(1), V = x.size(2), k = integer(a[2]);
    TORCH_CHECK_VALUE(x.stride(2) == 1 || V <= 1, "logits: strides ", x.strides(),
                      ": the vocabulary must be dense");
    auto sp = (const float*)data("scores", tensor("scores", a[1]), dev, {B, W}, at::kFloat);
    const uint8_t* ended = nullptr;
    if (a[3] != Py_None) {
        const Tensor& e = tensor("ended", a[3]);
        ended = (const uint8_t*)data(
            "ended", e, dev, {B, W}, e.scalar_type() == at::kByte ? at::kByte : at::kBool);
    }
    const int64_t end_token = integer(a[4]);
    TORCH_CHECK_VALUE(k >= 1 && k <= 128, "k=", k, " (1 .. 128)");
    const int64_t shape[2] = {B, k};
    const Tensor out = output("out_scores", a[5], dev, shape, at::kFloat);
    const Tensor parents = output("parents", a[6], dev, shape, at::kInt);
    const Tensor tokens = output("tokens", a[7], dev, shape, at::kInt);
    const size_t need = g_beam_ws(B, W, V, k);
    const Scratch ws(a[8], dev, need);
    const ds41_stream_t st = stream_of(dev);
    run("ds41_beam_select", [&] {
        return g_beam(x.data_ptr(), bf16 ? DS41_LOGITS_BF16 : DS41_LOGITS_F32, x.stride(0),
                      x.stride(1), sp, ended, end_token, B, W, V, k, (float*)out.data_ptr(),
                      (int32_t*)parents.data_ptr(), (int32_t*)tokens.data_ptr(), ws.p, need, st);
    });
    PyObject* all = PyTuple_New(3);
    python_ok(all != nullptr);
    PyTuple_SET_ITEM(all, 0, given_or(a[5], out));
    PyTuple_SET_ITEM(all, 1, given_or(a[6], parents));
    PyTuple_SET_ITEM(all, 2, given_or(a[7], tokens));
    return all;
    END_HANDLE_TH_ERRORS
}

// kv_block_keys(cache, keys, page_table, lens, max_new, starts)
PyObject* kv_block_keys(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    count(n_args, 6);
    const Tensor &table = tensor("page_table", a[2]), &lens = tensor("lens", a[3]);
    const at::Device dev = here(lens);
    const Cache c = cache_of(a[0], dev);
    TORCH_CHECK_TYPE(a[1] != Py_None, "keys: expected BlockKeys");
    const Keys keys = keys_of(a[1], dev, c.n_pages, c.kvh, c.hd);
    const int64_t B = count_of("lens", lens), max_new = integer(a[4]);
    const int32_t* pt = pages(table, dev, B);
    auto lp = ints("lens", a[3], dev, B);
    auto starts = (const int32_t*)data_or_null("starts", a[5], dev, {B}, at::kInt);
    const ds41_stream_t st = stream_of(dev);
    run("ds41_kv_block_keys", [&] {
        return g_keys(c.k, c.ks, c.fmt, c.n_pages, c.page, c.kvh, c.hd, pt, table.size(1), lp,
                      starts, B, max_new, keys.codes, keys.scales, st);
    });
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// block_select(q, keys, page, page_table, lens, cu_q, max_q, max_len, topk, first, local,
// idx) -> idx
PyObject* block_select(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    count(n_args, 12);
    const Tensor &q = tensor("q", a[0]), &table = tensor("page_table", a[3]),
                 &cu_q = tensor("cu_q", a[5]);
    const at::Device dev = here(q);
    TORCH_CHECK_TYPE(PyTuple_Check(a[1]) && PyTuple_GET_SIZE(a[1]) == 2,
                     "keys: expected BlockKeys, got ", Py_TYPE(a[1])->tp_name);
    const Tensor& codes = tensor("keys.codes", PyTuple_GET_ITEM(a[1], 0));
    TORCH_CHECK_VALUE(codes.dim() == 3, "keys.codes: expected [n_pages, kvh, hd], got ",
                      codes.sizes());
    const int64_t n_pages = codes.size(0), kvh = codes.size(1), hd = codes.size(2);
    const Keys keys = keys_of(a[1], dev, n_pages, kvh, hd);
    const Heads qh = heads("q", q, dev, hd);
    const int64_t Tq = q.size(0), nh = q.size(1), B = length("cu_q", cu_q), page = integer(a[2]);
    const int64_t max_q = integer(a[6]), max_len = integer(a[7]), topk = integer(a[8]);
    const int64_t first = integer(a[9]), local = integer(a[10]);
    const int32_t* pt = pages(table, dev, B);
    auto lp = ints("lens", a[4], dev, B), cq = ints("cu_q", a[5], dev, B + 1);
    TORCH_CHECK_VALUE(topk >= 1 && topk <= 1024, "topk=", topk, " (1 .. 1024)");
    const Tensor idx = output("idx", a[11], dev, {Tq, kvh, topk}, at::kInt);
    const ds41_stream_t st = stream_of(dev);
    run("ds41_block_select", [&] {
        return g_select(qh.p, qh.tok, qh.head, keys.codes, keys.scales, n_pages, page, kvh, hd, pt,
                        table.size(1), lp, cq, B, Tq, max_q, max_len, nh, topk, first, local,
                        (int32_t*)idx.data_ptr(), st);
    });
    return given_or(a[11], idx);
    END_HANDLE_TH_ERRORS
}

// [Tq, kvh, topk]
const int32_t* lists(PyObject* o, at::Device dev, int64_t Tq, int64_t kvh, int64_t& topk) {
    const Tensor& t = tensor("idx", o);
    TORCH_CHECK_VALUE(t.dim() == 3, "idx: expected [Tq, kvh, topk], got ", t.sizes());
    topk = t.size(2);
    return (const int32_t*)data("idx", t, dev, {Tq, kvh, topk}, at::kInt);
}

// block_attn_fwd(q, cache, page_table, lens, cu_q, max_q, idx, scale, sink, o, lse) -> o
PyObject* block_attn_fwd(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    count(n_args, 11);
    const Tensor &q = tensor("q", a[0]), &table = tensor("page_table", a[2]),
                 &cu_q = tensor("cu_q", a[4]);
    const at::Device dev = here(q);
    const Cache c = cache_of(a[1], dev);
    const Heads qh = heads("q", q, dev, c.hd);
    const int64_t Tq = q.size(0), nh = q.size(1), B = length("cu_q", cu_q), max_q = integer(a[5]);
    const int32_t* pt = pages(table, dev, B);
    auto lp = ints("lens", a[3], dev, B), cq = ints("cu_q", a[4], dev, B + 1);
    int64_t topk;
    const int32_t* idx = lists(a[6], dev, Tq, c.kvh, topk);
    const float scale = real(a[7]);
    auto sink = (const float*)data_or_null("sink", a[8], dev, {nh}, at::kFloat);
    auto lse = (float*)data_or_null("lse", a[10], dev, {Tq, nh}, at::kFloat);
    const Tensor o = output("o", a[9], dev, q.sizes());
    const ds41_stream_t st = stream_of(dev);
    run("ds41_block_attn_fwd", [&] {
        return g_blocks(qh.p, qh.tok, qh.head, c.k, c.v, c.ks, c.vs, c.fmt, c.n_pages, c.page, pt,
                        table.size(1), lp, cq, idx, topk, B, Tq, max_q, nh, c.kvh, c.hd, scale,
                        sink, (ds41_bf16*)o.data_ptr(), lse, st);
    });
    return given_or(a[9], o);
    END_HANDLE_TH_ERRORS
}

// block_prompt_attn_fwd(q, k, v, cu_q, cu_k, max_q, max_k, idx, block, scale, sink, o, lse,
// ws) -> o
PyObject* block_prompt_attn_fwd(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    count(n_args, 14);
    const Tensor &q = tensor("q", a[0]), &k = tensor("k", a[1]), &v = tensor("v", a[2]);
    const Tensor& cu_q = tensor("cu_q", a[3]);
    const at::Device dev = here(q);
    TORCH_CHECK_VALUE(q.dim() == 3 && k.dim() == 3, "q, k: expected [tokens, heads, hd], got ",
                      q.sizes(), ", ", k.sizes());
    const int64_t Tq = q.size(0), nh = q.size(1), hd = q.size(2), Tk = k.size(0), kvh = k.size(1);
    const Heads qh = heads("q", q, dev, hd), kh = heads("k", k, dev, hd);
    const Heads vh = heads("v", v, dev, hd);
    TORCH_CHECK_VALUE(v.sizes() == k.sizes(), "v: expected ", k.sizes(), ", got ", v.sizes());
    const int64_t B = length("cu_q", cu_q), max_q = integer(a[5]), max_k = integer(a[6]);
    auto cq = ints("cu_q", a[3], dev, B + 1), ck = ints("cu_k", a[4], dev, B + 1);
    int64_t topk;
    const int32_t* idx = lists(a[7], dev, Tq, kvh, topk);
    const int64_t block = integer(a[8]);
    const float scale = real(a[9]);
    auto sink = (const float*)data_or_null("sink", a[10], dev, {nh}, at::kFloat);
    auto lse = (float*)data_or_null("lse", a[12], dev, {Tq, nh}, at::kFloat);
    const Tensor o = output("o", a[11], dev, q.sizes());
    const size_t need = g_block_prompt_ws(B, Tq, max_q, max_k, topk, block, nh, kvh);
    const Scratch ws(a[13], dev, need);
    const ds41_stream_t st = stream_of(dev);
    run("ds41_block_prompt_attn_fwd", [&] {
        return g_block_prompt(qh.p, qh.tok, qh.head, kh.p, kh.tok, kh.head, vh.p, vh.tok, vh.head,
                              cq, ck, idx, topk, block, B, Tq, Tk, max_q, max_k, nh, kvh, hd,
                              scale, sink, (ds41_bf16*)o.data_ptr(), lse, ws.p, need, st);
    });
    return given_or(a[11], o);
    END_HANDLE_TH_ERRORS
}

// bind(failed, the entry points' addresses in this order ...): failed raises for a code that is
// not DS41_OK
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    count(n_args, 20);
    int i = 0;
    auto next = [&](auto& f) { f = (std::remove_reference_t<decltype(f)>)integer(a[++i]); };
    next(g_write);
    next(g_read);
    next(g_prompt);
    next(g_tree);
    next(g_tree_ws);
    next(g_take);
    next(g_free);
    next(g_fork);
    next(g_fork_ws);
    next(g_copy);
    next(g_compact);
    next(g_compact_ws);
    next(g_beam);
    next(g_beam_ws);
    next(g_keys);
    next(g_select);
    next(g_blocks);
    next(g_block_prompt);
    next(g_block_prompt_ws);
    Py_XSETREF(g_failed, Py_NewRef(a[0]));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define DS41_FAST(f) {#f, (PyCFunction)(void (*)())f, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {DS41_FAST(kv_cache_write),   DS41_FAST(kv_cache_read),
                           DS41_FAST(prompt_attn_fwd),  DS41_FAST(tree_attn_fwd),
                           DS41_FAST(kv_pages_take),    DS41_FAST(kv_pages_free),
                           DS41_FAST(kv_pages_fork),    DS41_FAST(kv_pages_copy),
                           DS41_FAST(kv_pages_compact), DS41_FAST(beam_select),
                           DS41_FAST(kv_block_keys),    DS41_FAST(block_select),
                           DS41_FAST(block_attn_fwd),   DS41_FAST(block_prompt_attn_fwd),
                           DS41_FAST(bind),             {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ds41_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ds41_binding(void) { return PyModule_Create(&g_module); }
