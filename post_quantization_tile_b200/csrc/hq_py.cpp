// hq_py.cpp -- the Python side of the 8-bit operators: checks of torch tensors, output and scratch
// allocation, the tensors' stream, and the C calls of include/hq.h.
//
// A decoding step calls these operators on a few tokens, where the GPU needs two to ten microseconds and the
// same marshalling in Python took about as long again; here it takes one to two.  Wrong arguments raise
// ValueError before anything is launched, a status other than HQ_OK raises the package's HQError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/MemoryOverlap.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>
#include <utility>

#include "../../include/hq.h"

namespace {

PyObject* g_error = nullptr;  // HQError(code, where)

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};
[[noreturn]] void refuse(const std::string& why) { throw Refused(why); }

std::string shape_text(at::IntArrayRef s)
{
    std::string t = "[";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// a tensor on CUDA device `dev` of this type and shape, with a contiguous last dimension or as a whole
enum Layout { kWhole, kRows };
const at::Tensor& on(PyObject* o, const char* name, int dev, at::ScalarType type, at::IntArrayRef shape, Layout layout)
{
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.sizes() != shape)
        refuse(std::string(name) + " must be " + c10::toString(type) + " " + shape_text(shape) + " on cuda:" + std::to_string(dev) +
               ", got " + c10::toString(t.scalar_type()) + " " + shape_text(t.sizes()) + " on " + t.device().str());
    if (layout == kWhole && !t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    if (layout == kRows && t.size(-1) > 1 && t.stride(-1) != 1) refuse(std::string(name) + " needs a contiguous last dimension");
    return t;
}

int device_of(const at::Tensor& t, const char* name)
{
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor (no CPU path)");
    return t.get_device();
}

hq_dtype_t dense_type(at::ScalarType t)
{
    if (t == at::kBFloat16) return HQ_BF16;
    if (t == at::kFloat) return HQ_F32;
    refuse("dense tensors must be bfloat16 or float32");
}

at::Tensor make(int dev, at::ScalarType type, at::IntArrayRef shape)
{
    return at::Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt));
}

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

// a call's workspace: the caller's Workspace, or scratch that returns to torch's allocator (which keeps it
// to this stream, or to the graph under capture) when the call has been issued
struct Scratch {
    at::Tensor buf;
    void* ptr = nullptr;
    size_t bytes = 0;
};
Scratch scratch(PyObject* ws, int dev, size_t need)
{
    Scratch s;
    if (ws != Py_None) {
        PyObject* b = PyObject_GetAttrString(ws, "buf");
        if (!b) {
            PyErr_Clear();
            refuse("ws must be a Workspace");
        }
        if (THPVariable_Check(b)) s.buf = THPVariable_Unpack(b);
        Py_DECREF(b);
        if (!s.buf.defined() || !s.buf.is_cuda() || s.buf.get_device() != dev) refuse("ws lies on another device");
    } else if (need) {
        s.buf = make(dev, at::kByte, {(int64_t)need});
    } else {
        return s;
    }
    s.ptr = s.buf.data_ptr();
    s.bytes = (size_t)s.buf.numel();
    return s;
}

int64_t whole(PyObject* o, const char* name)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(name) + " must be a whole number");
    }
    return v;
}

// strides of the leading dimensions; those of dimensions of length one, which any stride describes, as 0
void strides(const at::Tensor& t, int64_t* to, int n)
{
    for (int i = 0; i < n; ++i) to[i] = t.size(i) == 1 ? 0 : t.stride(i);
}

// an output whose rows are distinct: an expanded one would be written by several rows at once
const at::Tensor& output(const at::Tensor& t, const char* name)
{
    if (at::has_internal_overlap(t) == at::MemOverlap::Yes) refuse(std::string(name) + " is expanded: its rows share memory");
    return t;
}

// whether rows of la elements from 0 and of lb elements from d, both repeated n[k] times at strides s[k] (the
// largest first, each spanning the ones behind it), have an element in common
bool rows_meet(int64_t d, const int64_t* s, const int64_t* n, int dims, int64_t la, int64_t lb)
{
    if (dims == 0) return d < la && d > -lb;
    if (n[0] == 1 || s[0] < 1) return rows_meet(d, s + 1, n + 1, dims - 1, la, lb);
    const int64_t i = d / s[0];
    for (int64_t j = i - 1; j <= i + 1; ++j)
        if (j > -n[0] && j < n[0] && rows_meet(d - j * s[0], s + 1, n + 1, dims - 1, la, lb)) return true;
    return false;
}
// an output may not share memory with an input that other rows still read; the very same view is left to the caller
void apart(const at::Tensor& out, const at::Tensor& in, const char* names)
{
    if (!out.is_alias_of(in)) return;
    const int dims = (int)out.dim() - 1;
    const int64_t d = in.storage_offset() - out.storage_offset();
    bool same = true;
    int64_t s[3], n[3];
    for (int i = 0; i < dims; ++i) {
        s[i] = out.size(i) == 1 ? 0 : out.stride(i);
        n[i] = out.size(i);
        same = same && out.size(i) == in.size(i) && (n[i] == 1 || s[i] == in.stride(i));
    }
    if (same && d == 0 && out.sizes() == in.sizes()) return;
    bool meet;
    if (same) {
        for (int i = 1; i < dims; ++i)
            for (int j = i; j > 0 && s[j] > s[j - 1]; --j) std::swap(s[j], s[j - 1]), std::swap(n[j], n[j - 1]);
        meet = rows_meet(d, s, n, dims, out.size(dims), in.size(dims));
    } else {
        meet = at::get_overlap_status(out, in) == at::MemOverlapStatus::Partial;
    }
    if (meet) refuse(std::string(names) + " overlap");
}

struct Cache {
    hq_kv8_t c;
    int dev;
};
Cache cache_of(PyObject* const* a)
{
    const at::Tensor& k = tensor(a[0], "cache.k");
    Cache r;
    r.dev = device_of(k, "the cache");
    if (k.dim() != 4) refuse("cache.k must be [pages, heads, page, dim]");
    const at::IntArrayRef all = k.sizes(), pages = all.slice(0, 2);
    if (pages[0] > INT32_MAX || all[1] > INT32_MAX || all[2] > INT32_MAX || all[3] > INT32_MAX) refuse("the cache is too large");
    r.c.k = (uint8_t*)on(a[0], "cache.k", r.dev, at::kFloat8_e4m3fn, all, kWhole).data_ptr();
    r.c.v = (uint8_t*)on(a[1], "cache.v", r.dev, at::kFloat8_e4m3fn, all, kWhole).data_ptr();
    r.c.k_scale = (float*)on(a[2], "cache.k_scale", r.dev, at::kFloat, pages, kWhole).data_ptr();
    r.c.v_scale = (float*)on(a[3], "cache.v_scale", r.dev, at::kFloat, pages, kWhole).data_ptr();
    r.c.pages = all[0];
    r.c.heads = (int32_t)all[1];
    r.c.page = (int32_t)all[2];
    r.c.dim = (int32_t)all[3];
    return r;
}

struct Table {
    const int32_t* ptr;
    int64_t stride, pages;
};
Table table_of(PyObject* o, const char* name, int dev, int64_t B)
{
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != B ||
        (t.size(1) > 1 && t.stride(1) != 1))
        refuse(std::string(name) + " must be int32 [" + std::to_string(B) + ", pages] on cuda:" + std::to_string(dev) + " with contiguous rows");
    return Table{(const int32_t*)t.data_ptr(), B > 1 ? t.stride(0) : t.size(1), t.size(1)};
}

const int32_t* ints(PyObject* o, const char* name, int dev, int64_t B)
{
    return o == Py_None ? nullptr : (const int32_t*)on(o, name, dev, at::kInt, {B}, kWhole).data_ptr();
}

bool failed(hq_status_t s, const char* where)
{
    if (s == HQ_OK) return false;
    PyObject* e = PyObject_CallFunction(g_error, "is", (int)s, where);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return true;
}

template <typename F>
PyObject* guarded(F f)
{
    try {
        return f();
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(PyExc_MemoryError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

bool arity(Py_ssize_t n, Py_ssize_t want)
{
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments wanted, got %zd", want, n);
    return false;
}

// fp8_quantize(x, block, data | None, scale | None, ws) -> (data, scale)
PyObject* fp8_quantize(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (!arity(n, 5)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor& x = tensor(a[0], "x");
        const int dev = device_of(x, "x");
        if (x.dim() != 2 || (x.size(1) > 1 && x.stride(1) != 1)) refuse("x must be 2-D [rows, cols] with contiguous rows");
        const int64_t block = whole(a[1], "block"), rows = x.size(0), cols = x.size(1);
        if (block != 1 && block != 128) refuse("block must be 1 or 128");
        const int64_t ld = (cols + 15) / 16 * 16, kb = (cols + 127) / 128, rb = (rows + block - 1) / block;
        at::Tensor q = a[2] == Py_None ? make(dev, at::kFloat8_e4m3fn, {rows, ld}) : on(a[2], "out.data", dev, at::kFloat8_e4m3fn, {rows, ld}, kWhole);
        at::Tensor s = a[3] == Py_None ? make(dev, at::kFloat, {kb, rb}) : on(a[3], "out.scale", dev, at::kFloat, {kb, rb}, kWhole);
        const Scratch w = scratch(a[4], dev, 0);
        if (failed(hq_fp8_quantize(x.data_ptr(), dense_type(x.scalar_type()), rows, cols, rows > 1 ? x.stride(0) : cols, (int32_t)block,
                                   (uint8_t*)q.data_ptr(), ld, (float*)s.data_ptr(), w.ptr, w.bytes, stream_of(dev)),
                   "hq_fp8_quantize"))
            return nullptr;
        PyObject* r = PyTuple_New(2);
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(q)));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(s)));
        return r;
    });
}

// gemm_fp8(M, K, a.data, a.scale, N, w.data, w.scale, dtype, out | None, ws) -> out
PyObject* gemm_fp8(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (!arity(n, 10)) return nullptr;
    return guarded([&]() -> PyObject* {
        const int64_t M = whole(a[0], "a.rows"), K = whole(a[1], "a.cols"), N = whole(a[4], "w.rows");
        if (M < 1 || N < 1 || K < 1) refuse("a and w need rows and columns");
        const int dev = device_of(tensor(a[2], "a.data"), "a");
        const int64_t ld = (K + 15) / 16 * 16, kb = (K + 127) / 128;
        const at::Tensor &A = on(a[2], "a.data", dev, at::kFloat8_e4m3fn, {M, ld}, kWhole), &sa = on(a[3], "a.scale", dev, at::kFloat, {kb, M}, kWhole);
        const at::Tensor &W = on(a[5], "w.data", dev, at::kFloat8_e4m3fn, {N, ld}, kWhole),
                         &sw = on(a[6], "w.scale", dev, at::kFloat, {kb, (N + 127) / 128}, kWhole);
        at::Tensor y;
        if (a[8] == Py_None) {
            if (!THPDtype_Check(a[7])) refuse("dtype must be a torch dtype");
            const at::ScalarType type = reinterpret_cast<THPDtype*>(a[7])->scalar_type;
            dense_type(type);
            y = make(dev, type, {M, N});
        } else {
            y = tensor(a[8], "out");
            dense_type(y.scalar_type());
            on(a[8], "out", dev, y.scalar_type(), {M, N}, kWhole);
        }
        const Scratch w = scratch(a[9], dev, 0);
        if (failed(hq_gemm_fp8((const uint8_t*)A.data_ptr(), ld, (const float*)sa.data_ptr(), M, (const uint8_t*)W.data_ptr(), ld,
                               (const float*)sw.data_ptr(), N, K, y.data_ptr(), dense_type(y.scalar_type()), w.ptr, w.bytes, stream_of(dev)),
                   "hq_gemm_fp8"))
            return nullptr;
        return THPVariable_Wrap(std::move(y));
    });
}

// kv8_append(cache k, v, k_scale, v_scale, k, v, table, lens, n_new | None, ws)
PyObject* kv8_append(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (!arity(n, 10)) return nullptr;
    return guarded([&]() -> PyObject* {
        const Cache c = cache_of(a);
        const at::Tensor& k = tensor(a[4], "k");
        if (k.dim() != 4 || k.size(1) != c.c.heads || k.size(3) != c.c.dim)
            refuse("k and v must be [B, " + std::to_string(c.c.heads) + ", S, " + std::to_string(c.c.dim) + "]");
        const at::IntArrayRef shape = k.sizes();
        hq_kv8_append_t p;
        p.cache = c.c;
        p.dtype = dense_type(k.scalar_type());
        p.k = on(a[4], "k", c.dev, k.scalar_type(), shape, kRows).data_ptr();
        const at::Tensor& v = on(a[5], "v", c.dev, k.scalar_type(), shape, kRows);
        p.v = v.data_ptr();
        p.B = shape[0];
        p.S = shape[2];
        strides(k, p.k_stride, 3);
        strides(v, p.v_stride, 3);
        const Table t = table_of(a[6], "table", c.dev, p.B);
        p.table = t.ptr;
        p.table_stride = t.stride;
        p.max_pages = t.pages;
        p.lens = (const int32_t*)on(a[7], "lens", c.dev, at::kInt, {p.B}, kWhole).data_ptr();
        p.n_new = ints(a[8], "n_new", c.dev, p.B);
        const Scratch w = scratch(a[9], c.dev, 0);
        if (failed(hq_kv8_append(&p, w.ptr, w.bytes, stream_of(c.dev)), "hq_kv8_append")) return nullptr;
        Py_RETURN_NONE;
    });
}

// kv8_attend(cache k, v, k_scale, v_scale, q, table, lens, q_lens | None, scale | None, causal, out | None,
//            lse | None, weights | None, weights_in | None, ws) -> out
PyObject* kv8_attend(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (!arity(n, 15)) return nullptr;
    return guarded([&]() -> PyObject* {
        const Cache c = cache_of(a);
        const at::Tensor& q = tensor(a[4], "q");
        if (q.dim() != 4 || q.size(3) != c.c.dim) refuse("q must be [B, Hq, Sq, " + std::to_string(c.c.dim) + "]");
        const at::IntArrayRef shape = q.sizes();
        hq_kv8_attend_t p;
        p.cache = c.c;
        p.q = on(a[4], "q", c.dev, at::kBFloat16, shape, kRows).data_ptr();
        at::Tensor out = a[10] == Py_None ? make(c.dev, at::kBFloat16, shape) : on(a[10], "out", c.dev, at::kBFloat16, shape, kRows);
        p.out = output(out, "out").data_ptr();
        apart(out, q, "out and q");
        p.B = shape[0];
        p.Hq = shape[1];
        p.Sq = shape[2];
        strides(q, p.q_stride, 3);
        strides(out, p.out_stride, 3);
        const Table t = table_of(a[5], "table", c.dev, p.B);
        p.table = t.ptr;
        p.table_stride = t.stride;
        p.max_pages = t.pages;
        p.lens = (const int32_t*)on(a[6], "lens", c.dev, at::kInt, {p.B}, kWhole).data_ptr();
        p.q_lens = ints(a[7], "q_lens", c.dev, p.B);
        const double scale = a[8] == Py_None ? 1.0 / std::sqrt((double)c.c.dim) : PyFloat_AsDouble(a[8]);
        if (PyErr_Occurred()) return nullptr;
        p.scale = (float)scale;
        p.causal = PyObject_IsTrue(a[9]);
        if (p.causal < 0) return nullptr;
        p.lse = p.weights = nullptr;
        p.weights_in = nullptr;
        p.lse_stride[0] = p.lse_stride[1] = 0;
        for (int i = 0; i < 2; ++i) p.win_stride[i] = p.w_stride[i] = 0;
        p.L = 0;
        if (a[11] != Py_None) {
            const at::Tensor& x = output(on(a[11], "lse", c.dev, at::kFloat, shape.slice(0, 3), kRows), "lse");
            p.lse = (float*)x.data_ptr();
            p.lse_stride[0] = x.stride(0);
            p.lse_stride[1] = x.stride(1);
        }
        if (a[12] != Py_None) {
            const at::Tensor& x = tensor(a[12], "weights");
            p.L = x.dim() == 3 ? x.size(2) : 0;
            p.weights = (float*)output(on(a[12], "weights", c.dev, at::kFloat, {p.B, c.c.heads, p.L}, kRows), "weights").data_ptr();
            p.w_stride[0] = x.stride(0);
            p.w_stride[1] = x.stride(1);
            if (a[13] != Py_None) {
                const at::Tensor& y = on(a[13], "weights_in", c.dev, at::kFloat, {p.B, c.c.heads, p.L}, kRows);
                apart(x, y, "weights and weights_in");
                p.weights_in = (const float*)y.data_ptr();
                p.win_stride[0] = y.stride(0);
                p.win_stride[1] = y.stride(1);
            }
        } else if (a[13] != Py_None) {
            refuse("weights_in without weights");
        }
        const size_t need = a[14] != Py_None ? 0 : hq_kv8_attend_workspace_need(&p);
        const Scratch w = scratch(a[14], c.dev, need);
        if (failed(hq_kv8_attend(&p, w.ptr, w.bytes, stream_of(c.dev)), "hq_kv8_attend")) return nullptr;
        return THPVariable_Wrap(std::move(out));
    });
}

// kv8_evict(cache k, v, k_scale, v_scale, table, lens, weights, budget, recent, to_table, out_lens | None,
//           out_weights | None, ws) -> (out_lens, out_weights)
PyObject* kv8_evict(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (!arity(n, 13)) return nullptr;
    return guarded([&]() -> PyObject* {
        const Cache c = cache_of(a);
        const at::Tensor& x = tensor(a[6], "weights");
        if (x.dim() != 3) refuse("weights must be [B, heads, slots]");
        hq_kv8_evict_t p;
        p.cache = c.c;
        p.B = x.size(0);
        p.L = x.size(2);
        p.weights = (const float*)on(a[6], "weights", c.dev, at::kFloat, {p.B, c.c.heads, p.L}, kRows).data_ptr();
        p.w_stride[0] = x.stride(0);
        p.w_stride[1] = x.stride(1);
        const Table t = table_of(a[4], "table", c.dev, p.B), to = table_of(a[9], "to_table", c.dev, p.B);
        p.table = t.ptr;
        p.table_stride = t.stride;
        p.max_pages = t.pages;
        p.to_table = to.ptr;
        p.to_stride = to.stride;
        p.to_pages = to.pages;
        p.lens = (const int32_t*)on(a[5], "lens", c.dev, at::kInt, {p.B}, kWhole).data_ptr();
        p.budget = whole(a[7], "budget");
        p.recent = whole(a[8], "recent");
        if (p.budget < 1 || p.recent < 0) refuse("budget must be at least 1 and recent at least 0");
        at::Tensor lens = a[10] == Py_None ? make(c.dev, at::kInt, {p.B}) : on(a[10], "out_lens", c.dev, at::kInt, {p.B}, kWhole);
        apart(lens, tensor(a[5], "lens"), "out_lens and lens");
        at::Tensor ow;
        if (a[11] == Py_None) {
            ow = at::zeros({p.B, c.c.heads, p.budget}, x.options());
        } else {
            ow = tensor(a[11], "out_weights");
            if (ow.dim() != 3 || ow.size(2) < p.budget) refuse("out_weights needs room for the budget");
            output(on(a[11], "out_weights", c.dev, at::kFloat, {p.B, c.c.heads, ow.size(2)}, kRows), "out_weights");
            apart(ow, x, "out_weights and weights");
        }
        p.out_lens = (int32_t*)lens.data_ptr();
        p.out_weights = (float*)ow.data_ptr();
        p.ow_stride[0] = ow.stride(0);
        p.ow_stride[1] = ow.stride(1);
        const Scratch w = scratch(a[12], c.dev, a[12] != Py_None ? 0 : hq_kv8_evict_workspace_bytes(p.B, c.c.heads, p.budget));
        if (failed(hq_kv8_evict(&p, w.ptr, w.bytes, stream_of(c.dev)), "hq_kv8_evict")) return nullptr;
        PyObject* r = PyTuple_New(2);
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(lens)));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(ow)));
        return r;
    });
}

// the exception class that a status other than HQ_OK raises
PyObject* set_error(PyObject*, PyObject* type)
{
    Py_INCREF(type);
    Py_XSETREF(g_error, type);
    Py_RETURN_NONE;
}

#define HQ_FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {HQ_FAST(fp8_quantize), HQ_FAST(gemm_fp8), HQ_FAST(kv8_append), HQ_FAST(kv8_attend), HQ_FAST(kv8_evict),
                         {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hq8", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__hq8(void) { return PyModule_Create(&module); }
