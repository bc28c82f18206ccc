// CPython module behind awq_int4_moe_gb300/decoder.py and prompt.py: takes the tensors of a
// call apart, checks what the C call cannot see (types, shapes, devices,
// dense rows), calls the entry point of include/awq_decoder.h or awq_prompt.h on
// the current stream and returns its status. No computation, no state. In Python alone
// these checks cost several times what the smallest calls take on the device.
#include <Python.h>

#include <algorithm>
#include <cmath>
#include <sstream>
#include <string>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/awq_prompt.h"

namespace {

struct Bad {
    PyObject *type;
    std::string text;
};

[[noreturn]] void bad_value(const std::string &text) { throw Bad{PyExc_ValueError, text}; }
[[noreturn]] void bad_type(const std::string &text) { throw Bad{PyExc_TypeError, text}; }

std::string shape_text(at::IntArrayRef s)
{
    std::ostringstream o;
    o << "(";
    for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
    o << (s.size() == 1 ? ",)" : ")");
    return o.str();
}

const char *type_name(at::ScalarType t)
{
    switch (t) {
    case at::kHalf: return "float16";
    case at::kBFloat16: return "bfloat16";
    case at::kFloat: return "float32";
    case at::kInt: return "int32";
    case at::kLong: return "int64";
    case at::kFloat8_e4m3fn: return "float8_e4m3fn";
    default: return c10::toString(t);
    }
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) bad_type(std::string(name) + ": expected a tensor, got " + Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

int act_code(at::ScalarType t) { return t == at::kHalf ? AWQ_DTYPE_F16 : t == at::kBFloat16 ? AWQ_DTYPE_BF16 : -1; }

// The arguments of one call: the first tensor gives the device that all others
// have to be on, and the stream; the device is the current one while the call
// lives.
struct Call {
    c10::DeviceIndex device = -1;
    c10::cuda::OptionalCUDAGuard guard;

    void check(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape)
    {
        if (t.scalar_type() != type)
            bad_type(std::string(name) + ": expected " + type_name(type) + ", got " + type_name(t.scalar_type()));
        if (t.sizes() != shape)
            bad_value(std::string(name) + ": expected shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
        check_device(t, name);
    }

    void check_device(const at::Tensor &t, const char *name)
    {
        if (!t.is_cuda()) bad_value(std::string(name) + ": must be a CUDA device tensor, got one on " + t.device().str());
        if (device < 0) device = t.device().index();
        if (t.device().index() != device)
            bad_value(std::string(name) + ": on another device (" + t.device().str() + ") than the call's first tensor");
    }

    // An activation: its type's code.
    int activation(const at::Tensor &t, const char *name, int dims)
    {
        const int code = act_code(t.scalar_type());
        if (code < 0) bad_type(std::string(name) + ": expected float16 or bfloat16, got " + type_name(t.scalar_type()));
        if (t.dim() != dims)
            bad_value(std::string(name) + ": expected " + std::to_string(dims) + " dimensions, got shape " + shape_text(t.sizes()));
        check_device(t, name);
        return code;
    }

    // 2D with dense rows; NULL for None where that is allowed. A single row's
    // stride carries no information and may be anything.
    void *rows(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, int64_t *ld, bool optional = false)
    {
        *ld = 0;
        if (optional && o == Py_None) return nullptr;
        const at::Tensor &t = tensor(o, name);
        check(t, name, type, shape);
        if (t.stride(1) != 1 && shape[1] > 1) strides(t, name);
        *ld = shape[0] > 1 ? t.stride(0) : std::max(t.stride(0), shape[1]);
        return t.data_ptr();
    }

    // Contiguous; NULL for None where that is allowed.
    void *dense(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, bool optional = false)
    {
        if (optional && o == Py_None) return nullptr;
        const at::Tensor &t = tensor(o, name);
        check(t, name, type, shape);
        if (!t.is_contiguous()) strides(t, name);
        return t.data_ptr();
    }

    awq_heads heads(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape)
    {
        const at::Tensor &t = tensor(o, name);
        check(t, name, type, shape);
        if (t.stride(2) != 1 && shape[2] > 1) strides(t, name);
        return awq_heads{t.data_ptr(), t.stride(0), t.stride(1)};
    }

    // [pages][page size][KV heads][head dim], any strides but the last.
    awq_kv_cache cache(PyObject *ko, PyObject *vo, double k_scale, double v_scale, at::ScalarType act)
    {
        const at::Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache");
        if (k.scalar_type() != v.scalar_type())
            bad_type(std::string("v_cache: expected ") + type_name(k.scalar_type()) + ", got " + type_name(v.scalar_type()));
        if (k.scalar_type() != at::kFloat8_e4m3fn && k.scalar_type() != act)
            bad_type(std::string("k_cache: expected ") + type_name(act) + " or float8_e4m3fn, got " + type_name(k.scalar_type()));
        if (k.dim() != 4 || k.sizes() != v.sizes())
            bad_value("k_cache, v_cache: expected one shape [pages][page size][heads][dim], got " + shape_text(k.sizes()) + " and " +
                      shape_text(v.sizes()));
        check_device(k, "k_cache");
        check_device(v, "v_cache");
        if (k.size(3) > 1) {
            if (k.stride(3) != 1) strides(k, "k_cache");
            if (v.stride(3) != 1) strides(v, "v_cache");
        }
        for (int i = 0; i < 4; ++i)
            if (k.size(i) > 0x7fffffff) bad_value("k_cache: sizes are limited to 2^31 - 1, got " + shape_text(k.sizes()));
        awq_kv_cache c;
        c.k = {k.data_ptr(), k.stride(0), k.stride(1), k.stride(2), static_cast<float>(k_scale)};
        c.v = {v.data_ptr(), v.stride(0), v.stride(1), v.stride(2), static_cast<float>(v_scale)};
        c.dtype = k.scalar_type() == at::kFloat8_e4m3fn ? AWQ_DTYPE_E4M3 : act_code(act);
        c.num_pages = static_cast<int32_t>(k.size(0));
        c.page_size = static_cast<int32_t>(k.size(1));
        c.num_heads = static_cast<int32_t>(k.size(2));
        c.head_dim = static_cast<int32_t>(k.size(3));
        return c;
    }

    int32_t *status(PyObject *o)
    {
        const at::Tensor &t = tensor(o, "dev_status");
        if (t.scalar_type() != at::kInt || t.numel() < 1)
            bad_type(std::string("dev_status: expected int32 and at least 1 element, got ") + type_name(t.scalar_type()) + " of shape " +
                     shape_text(t.sizes()));
        check_device(t, "dev_status");
        return static_cast<int32_t *>(t.data_ptr());
    }

    // Where the sequences of a packed batch begin, and the last one's end.
    void *bounds(PyObject *o, int32_t *batch)
    {
        const at::Tensor &t = tensor(o, "cu_seqlens");
        if (t.dim() != 1 || t.size(0) < 1 || t.size(0) > 0x7fffffff)
            bad_value("cu_seqlens: expected shape (batch + 1,), got " + shape_text(t.sizes()));
        *batch = static_cast<int32_t>(t.size(0) - 1);
        return dense(o, "cu_seqlens", at::kInt, t.sizes());
    }

    const at::Tensor &scratch(PyObject *o)
    {
        const at::Tensor &t = tensor(o, "workspace");
        check_device(t, "workspace");
        if (!t.is_contiguous()) strides(t, "workspace");
        return t;
    }

    // A stream handle, or None for the device's current stream.
    void *stream(PyObject *o)
    {
        // (asking costs 0.1 us; with one device there is nothing to ask)
        if (c10::cuda::device_count() > 1 && c10::cuda::current_device() != device) guard.set_index(device);
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device).stream();
        void *p = PyLong_AsVoidPtr(o);
        if (PyErr_Occurred()) throw Bad{nullptr, ""};
        return p;
    }

    [[noreturn]] static void strides(const at::Tensor &t, const char *name)
    {
        bad_value(std::string(name) + ": needs dense rows, got strides " + shape_text(t.strides()));
    }
};

double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Bad{nullptr, ""};
    return v;
}

bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Bad{nullptr, ""};
    return v;
}

// The factor of a score: 1 / sqrt(dim) for None.
float score_scale(PyObject *o, int64_t dim)
{
    return static_cast<float>(o == Py_None ? 1.0 / std::sqrt(static_cast<double>(std::max<int64_t>(dim, 1))) : number(o));
}

// A size as the C ABI's int32.
int32_t size32(int64_t n, const char *name)
{
    if (n > 0x7fffffff) bad_value(std::string(name) + ": sizes are limited to 2^31 - 1, got " + std::to_string(n));
    return static_cast<int32_t>(n);
}

int64_t groups(int64_t n) { return (n + AWQ_FP8_BLOCK - 1) / AWQ_FP8_BLOCK; }

// x, weight, eps, residual, residual_out, out, out_q, out_scales, stream
awq_status add_rmsnorm(PyObject *const *a)
{
    Call c;
    const at::Tensor &x = tensor(a[0], "x");
    const int code = c.activation(x, "x", 2);
    const at::ScalarType type = x.scalar_type();
    const at::IntArrayRef shape = x.sizes();
    int64_t ldx, ldr, ldro, ldo, ldq;
    void *px = c.rows(a[0], "x", type, shape, &ldx);
    void *pr = c.rows(a[3], "residual", type, shape, &ldr, true);
    void *pro = c.rows(a[4], "residual_out", type, shape, &ldro, true);
    void *po = c.rows(a[5], "out", type, shape, &ldo, true), *pq = c.rows(a[6], "out_q", at::kFloat8_e4m3fn, shape, &ldq, true);
    void *ps = c.dense(a[7], "out_scales", at::kFloat, {shape[0], groups(shape[1])}, true);
    void *pw = c.dense(a[1], "weight", type, {shape[1]});
    return awq_add_rmsnorm(px, ldx, pr, ldr, pro, ldro, pw, static_cast<float>(number(a[2])), po, ldo, static_cast<uint8_t *>(pq),
                           ldq, static_cast<float *>(ps), size32(shape[0], "x"), size32(shape[1], "x"), code, c.stream(a[8]));
}

// x, out_q, out_scales, stream
awq_status quantize_fp8(PyObject *const *a)
{
    Call c;
    const at::Tensor &x = tensor(a[0], "x");
    const int code = c.activation(x, "x", 2);
    const at::IntArrayRef shape = x.sizes();
    int64_t ldx, ldq;
    void *px = c.rows(a[0], "x", x.scalar_type(), shape, &ldx), *pq = c.rows(a[1], "out_q", at::kFloat8_e4m3fn, shape, &ldq);
    void *ps = c.dense(a[2], "out_scales", at::kFloat, {shape[0], groups(shape[1])});
    return awq_quantize_fp8(px, ldx, static_cast<uint8_t *>(pq), ldq, static_cast<float *>(ps), size32(shape[0], "x"),
                            size32(shape[1], "x"), code, c.stream(a[3]));
}

// q, k, v, positions, cos_sin, slots, k_cache, v_cache, dev_status, q_out, interleaved, k_scale, v_scale, stream
awq_status rope_append(PyObject *const *a)
{
    Call c;
    const at::Tensor &q = tensor(a[0], "q");
    const int code = c.activation(q, "q", 3);
    const at::ScalarType type = q.scalar_type();
    const at::IntArrayRef shape = q.sizes();
    const awq_kv_cache cache = c.cache(a[6], a[7], number(a[11]), number(a[12]), type);
    if (shape[2] != cache.head_dim)
        bad_value("q: head size " + std::to_string(shape[2]) + ", the cache's is " + std::to_string(cache.head_dim));
    const awq_heads hq = c.heads(a[0], "q", type, shape), ho = a[9] == Py_None ? hq : c.heads(a[9], "q_out", type, shape);
    const int64_t kv_shape[3] = {shape[0], cache.num_heads, shape[2]};
    const awq_heads hk = c.heads(a[1], "k", type, kv_shape), hv = c.heads(a[2], "v", type, kv_shape);
    const at::Tensor &table = tensor(a[4], "cos_sin");
    if (table.dim() != 2) bad_value("cos_sin: expected 2 dimensions, got shape " + shape_text(table.sizes()));
    void *pt = c.dense(a[4], "cos_sin", at::kFloat, table.sizes());
    void *pp = c.dense(a[3], "positions", at::kInt, {shape[0]}), *ps = c.dense(a[5], "slots", at::kLong, {shape[0]});
    return awq_rope_append(&hq, &ho, &hk, &hv, static_cast<int32_t *>(pp), static_cast<float *>(pt), size32(table.size(0), "cos_sin"),
                           size32(table.size(1), "cos_sin"), truth(a[10]), static_cast<int64_t *>(ps), &cache,
                           size32(shape[0], "q"), size32(shape[1], "q"), code, c.status(a[8]), c.stream(a[13]));
}

// q, k_cache, v_cache, page_table, seq_lens, out, workspace, dev_status, scale, lse, k_scale, v_scale, stream
awq_status paged_attention(PyObject *const *a)
{
    Call c;
    const at::Tensor &q = tensor(a[0], "q");
    const int code = c.activation(q, "q", 3);
    const at::ScalarType type = q.scalar_type();
    const at::IntArrayRef shape = q.sizes();
    const awq_kv_cache cache = c.cache(a[1], a[2], number(a[10]), number(a[11]), type);
    if (shape[2] != cache.head_dim)
        bad_value("q: head size " + std::to_string(shape[2]) + ", the cache's is " + std::to_string(cache.head_dim));
    const awq_heads hq = c.heads(a[0], "q", type, shape), ho = c.heads(a[5], "out", type, shape);
    const at::Tensor &table = tensor(a[3], "page_table");
    if (table.dim() != 2) bad_value("page_table: expected 2 dimensions, got shape " + shape_text(table.sizes()));
    const int64_t pages = table.size(1);
    int64_t ldt;
    void *pt = c.rows(a[3], "page_table", at::kInt, {shape[0], pages}, &ldt);
    void *pl = c.dense(a[4], "seq_lens", at::kInt, {shape[0]});
    void *ps = c.dense(a[9], "lse", at::kFloat, {shape[0], shape[1]}, true);
    const at::Tensor &ws = tensor(a[6], "workspace");
    c.check_device(ws, "workspace");
    if (!ws.is_contiguous()) Call::strides(ws, "workspace");
    const double scale = a[8] == Py_None ? 1.0 / std::sqrt(static_cast<double>(std::max<int64_t>(shape[2], 1))) : number(a[8]);
    return awq_paged_attention(&hq, &cache, static_cast<int32_t *>(pt), ldt, size32(pages, "page_table"), static_cast<int32_t *>(pl),
                               size32(shape[0], "q"), size32(shape[1], "q"), code, static_cast<float>(scale), &ho,
                               static_cast<float *>(ps), ws.data_ptr(), ws.nbytes(), c.status(a[7]), c.stream(a[12]));
}

// a, a_scales, b, b_scales, out, dev_status, stream
awq_status fp8_gemm(PyObject *const *a)
{
    Call c;
    const at::Tensor &out = tensor(a[4], "out"), &ta = tensor(a[0], "a");
    const int code = c.activation(out, "out", 2);
    if (ta.dim() != 2) bad_value("a: expected 2 dimensions, got shape " + shape_text(ta.sizes()));
    const int64_t m = out.size(0), n = out.size(1), k = ta.size(1);
    int64_t lda, ldb, ldo;
    void *pa = c.rows(a[0], "a", at::kFloat8_e4m3fn, {m, k}, &lda), *pb = c.rows(a[2], "b", at::kFloat8_e4m3fn, {n, k}, &ldb);
    void *po = c.rows(a[4], "out", out.scalar_type(), {m, n}, &ldo);
    void *sa = c.dense(a[1], "a_scales", at::kFloat, {m, groups(k)}), *sb = c.dense(a[3], "b_scales", at::kFloat, {groups(n), groups(k)});
    return awq_fp8_gemm(static_cast<uint8_t *>(pa), lda, static_cast<float *>(sa), static_cast<uint8_t *>(pb), ldb,
                        static_cast<float *>(sb), po, ldo, size32(m, "a"), size32(n, "b"), size32(k, "a"), code, c.status(a[5]),
                        c.stream(a[6]));
}

// q, k, v, cu_seqlens, out, workspace, dev_status, scale, lse, stream
awq_status prompt_attention(PyObject *const *a)
{
    Call c;
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
    const int code = c.activation(q, "q", 3);
    const at::ScalarType type = q.scalar_type();
    const at::IntArrayRef shape = q.sizes();
    if (k.dim() != 3) bad_value("k: expected 3 dimensions, got shape " + shape_text(k.sizes()));
    const int64_t kv_shape[3] = {shape[0], k.size(1), shape[2]};
    const awq_heads hq = c.heads(a[0], "q", type, shape), ho = c.heads(a[4], "out", type, shape);
    const awq_heads hk = c.heads(a[1], "k", type, kv_shape), hv = c.heads(a[2], "v", type, kv_shape);
    int32_t batch;
    void *pc = c.bounds(a[3], &batch);
    void *pl = c.dense(a[8], "lse", at::kFloat, {shape[0], shape[1]}, true);
    const at::Tensor &ws = c.scratch(a[5]);
    return awq_prompt_attention(&hq, &hk, &hv, static_cast<int32_t *>(pc), batch, size32(shape[0], "q"), size32(shape[1], "q"),
                                size32(kv_shape[1], "k"), size32(shape[2], "q"), code, score_scale(a[7], shape[2]), &ho,
                                static_cast<float *>(pl), ws.data_ptr(), ws.nbytes(), c.status(a[6]), c.stream(a[9]));
}

// q, k_cache, v_cache, page_table, cu_seqlens, seq_lens, out, workspace, dev_status, scale, lse, k_scale, v_scale, stream
awq_status chunk_attention(PyObject *const *a)
{
    Call c;
    const at::Tensor &q = tensor(a[0], "q");
    const int code = c.activation(q, "q", 3);
    const at::ScalarType type = q.scalar_type();
    const at::IntArrayRef shape = q.sizes();
    const awq_kv_cache cache = c.cache(a[1], a[2], number(a[11]), number(a[12]), type);
    if (shape[2] != cache.head_dim)
        bad_value("q: head size " + std::to_string(shape[2]) + ", the cache's is " + std::to_string(cache.head_dim));
    const awq_heads hq = c.heads(a[0], "q", type, shape), ho = c.heads(a[6], "out", type, shape);
    int32_t batch;
    void *pc = c.bounds(a[4], &batch);
    const at::Tensor &table = tensor(a[3], "page_table");
    if (table.dim() != 2) bad_value("page_table: expected 2 dimensions, got shape " + shape_text(table.sizes()));
    const int64_t pages = table.size(1);
    int64_t ldt;
    void *pt = c.rows(a[3], "page_table", at::kInt, {batch, pages}, &ldt);
    void *pl = c.dense(a[5], "seq_lens", at::kInt, {batch});
    void *ps = c.dense(a[10], "lse", at::kFloat, {shape[0], shape[1]}, true);
    const at::Tensor &ws = c.scratch(a[7]);
    return awq_chunk_attention(&hq, &cache, static_cast<int32_t *>(pt), ldt, size32(pages, "page_table"), static_cast<int32_t *>(pc),
                               static_cast<int32_t *>(pl), batch, size32(shape[0], "q"), size32(shape[1], "q"), code,
                               score_scale(a[9], shape[2]), &ho, static_cast<float *>(ps), ws.data_ptr(), ws.nbytes(),
                               c.status(a[8]), c.stream(a[13]));
}

// q, k, v, q_weight, k_weight, eps, positions, cos_sin, slots, k_cache, v_cache, dev_status, q_out, interleaved, k_scale,
// v_scale, stream
awq_status qk_norm_rope_append(PyObject *const *a)
{
    Call c;
    const at::Tensor &q = tensor(a[0], "q");
    const int code = c.activation(q, "q", 3);
    const at::ScalarType type = q.scalar_type();
    const at::IntArrayRef shape = q.sizes();
    const awq_kv_cache cache = c.cache(a[9], a[10], number(a[14]), number(a[15]), type);
    if (shape[2] != cache.head_dim)
        bad_value("q: head size " + std::to_string(shape[2]) + ", the cache's is " + std::to_string(cache.head_dim));
    const awq_heads hq = c.heads(a[0], "q", type, shape), ho = a[12] == Py_None ? hq : c.heads(a[12], "q_out", type, shape);
    const int64_t kv_shape[3] = {shape[0], cache.num_heads, shape[2]};
    const awq_heads hk = c.heads(a[1], "k", type, kv_shape), hv = c.heads(a[2], "v", type, kv_shape);
    void *pqw = c.dense(a[3], "q_weight", type, {shape[2]}), *pkw = c.dense(a[4], "k_weight", type, {shape[2]});
    const at::Tensor &table = tensor(a[7], "cos_sin");
    if (table.dim() != 2) bad_value("cos_sin: expected 2 dimensions, got shape " + shape_text(table.sizes()));
    void *pt = c.dense(a[7], "cos_sin", at::kFloat, table.sizes());
    void *pp = c.dense(a[6], "positions", at::kInt, {shape[0]}), *ps = c.dense(a[8], "slots", at::kLong, {shape[0]});
    return awq_qk_norm_rope_append(&hq, &ho, &hk, &hv, pqw, pkw, static_cast<float>(number(a[5])), static_cast<int32_t *>(pp),
                                   static_cast<float *>(pt), size32(table.size(0), "cos_sin"), size32(table.size(1), "cos_sin"),
                                   truth(a[13]), static_cast<int64_t *>(ps), &cache, size32(shape[0], "q"),
                                   size32(shape[1], "q"), code, c.status(a[11]), c.stream(a[16]));
}

// One entry of the module: N positional arguments in, the status out.
template <awq_status (*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return PyLong_FromLong(F(args));
    } catch (const Bad &e) {
        if (e.type) PyErr_SetString(e.type, e.text.c_str());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <awq_status (*F)(PyObject *const *), Py_ssize_t N>
constexpr PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<add_rmsnorm, 9>("add_rmsnorm"),       method<quantize_fp8, 4>("quantize_fp8"),
                         method<rope_append, 14>("rope_append"),      method<paged_attention, 13>("paged_attention"),
                         method<fp8_gemm, 7>("fp8_gemm"),             method<prompt_attention, 10>("prompt_attention"),
                         method<chunk_attention, 14>("chunk_attention"),
                         method<qk_norm_rope_append, 17>("qk_norm_rope_append"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind(void) { return PyModule_Create(&module); }
