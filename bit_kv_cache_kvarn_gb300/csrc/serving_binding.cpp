// Python entry of the serving-step calls: checks of the tensors and the C calls, in compiled code.
//
// A decode step's kernels run for 3 to 10 microseconds; checking and passing their 15 to 30 arguments in
// Python and ctypes took 21 microseconds a call on the Grace cores, so these three calls come through the
// CPython interface.  Each function takes its arguments by position and returns the kvarn_status; a
// wrong tensor raises ValueError naming it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <initializer_list>
#include <limits>
#include <stdexcept>
#include <string>

#include "../../include/kvarn.h"

namespace {

struct PythonError {};  // a Python exception is already set

std::string text(at::IntArrayRef v) {
    std::string s = "(";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + ")";
}

[[noreturn]] void bad(const std::string& what) { throw std::invalid_argument(what); }

const at::Tensor* tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}
const at::Tensor* tensor_or_null(PyObject* o, const char* name) { return o == Py_None ? nullptr : tensor(o, name); }

struct Checker {
    int dev;

    void device(const at::Tensor& t, const char* name) const {
        if (!t.is_cuda() || t.get_device() != dev)
            bad(std::string(name) + " must be a tensor of the current CUDA device");
    }
    void type(const at::Tensor& t, at::ScalarType dt, const char* name) const {
        if (t.scalar_type() != dt)
            bad(std::string(name) + " must be " + c10::toString(dt) + ", got " + c10::toString(t.scalar_type()));
    }
    // data pointer of a contiguous tensor of this type and shape (-1: any size)
    template <typename P>
    P* array(const at::Tensor& t, at::ScalarType dt, std::initializer_list<int64_t> shape, const char* name) const {
        device(t, name);
        type(t, dt, name);
        bool same = t.dim() == (int64_t)shape.size();
        int i = 0;
        for (int64_t want : shape) {
            if (!same) break;
            same = want < 0 || t.size(i) == want;
            ++i;
        }
        if (!same) bad(std::string(name) + " has shape " + text(t.sizes()) + ", needs " + text(at::IntArrayRef(shape.begin(), shape.size())));
        if (!t.is_contiguous()) bad(std::string(name) + " must be contiguous");
        return static_cast<P*>(t.data_ptr());
    }
    int32_t* ints(PyObject* o, std::initializer_list<int64_t> shape, const char* name) const {
        return array<int32_t>(*tensor(o, name), at::kInt, shape, name);
    }
    int32_t* ints_or_null(PyObject* o, std::initializer_list<int64_t> shape, const char* name) const {
        return o == Py_None ? nullptr : ints(o, shape, name);
    }
    float* floats_or_null(PyObject* o, std::initializer_list<int64_t> shape, const char* name) const {
        return o == Py_None ? nullptr : array<float>(*tensor(o, name), at::kFloat, shape, name);
    }
};

int narrow(int64_t v, const char* name) {
    if (v < INT_MIN || v > INT_MAX) bad(std::string(name) + " = " + std::to_string(v) + " does not fit 32 bits");
    return (int)v;
}
int as_int(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError();
    return narrow(v, name);
}
float as_float(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError();
    return (float)v;
}
// the same, but only 0 itself becomes 0
float as_float_or_zero(PyObject* o) {
    const float v = as_float(o);
    return v == 0.f && PyFloat_AsDouble(o) != 0.0 ? std::numeric_limits<float>::denorm_min() : v;
}
int as_bool(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PythonError();
    return v;
}
kvarn_stream_t as_stream(PyObject* o, int dev) {
    if (o == Py_None) return (kvarn_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw PythonError();
    return (kvarn_stream_t)p;
}
kvarn_dtype as_dtype(at::ScalarType t, const char* name) {
    if (t == at::kBFloat16) return KVARN_DTYPE_BF16;
    if (t == at::kHalf) return KVARN_DTYPE_FP16;
    if (t == at::kFloat) return KVARN_DTYPE_FP32;
    bad(std::string("unsupported type of ") + name + ": " + c10::toString(t));
}

// [tokens, heads, 128] view with contiguous channels; the stride of an axis of one entry is never used
// and given as 0
struct Rows {
    void* p = nullptr;
    int64_t token = 0, head = 0;
};
Rows rows(const Checker& c, const at::Tensor& t, at::ScalarType dt, int64_t tokens, int64_t heads, const char* name) {
    c.device(t, name);
    c.type(t, dt, name);
    if (t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads || t.size(2) != KVARN_HEAD_DIM)
        bad(std::string(name) + " has shape " + text(t.sizes()) + ", needs " + text({tokens, heads, KVARN_HEAD_DIM}));
    if (t.stride(2) != 1) bad(std::string(name) + ": the channels must be contiguous");
    Rows r;
    r.p = t.data_ptr();
    r.token = tokens > 1 ? t.stride(0) : 0;
    r.head = heads > 1 ? t.stride(1) : 0;
    return r;
}

// [n_pages, Hkv, page_size, 128] views of one layout
struct Cache {
    void* k = nullptr;
    void* v = nullptr;
    int64_t n_pages = 0, heads = 0, page_stride = 0, head_stride = 0, token_stride = 0;
    int page_size = 1;
};
Cache cache(const Checker& c, const at::Tensor& k, const at::Tensor& v, at::ScalarType dt) {
    c.device(k, "k_cache");
    c.type(k, dt, "k_cache");
    c.device(v, "v_cache");
    c.type(v, dt, "v_cache");
    if (k.dim() != 4 || k.size(3) != KVARN_HEAD_DIM || k.stride(3) != 1)
        bad("k_cache must be [n_pages, Hkv, page_size, 128] with contiguous channels");
    if (!k.sizes().equals(v.sizes()) || !k.strides().equals(v.strides()))
        bad("v_cache must have k_cache's shape and strides");
    Cache r;
    r.k = k.data_ptr();
    r.v = v.data_ptr();
    r.n_pages = k.size(0);
    r.heads = k.size(1);
    r.page_size = narrow(k.size(2), "page_size");
    r.page_stride = k.stride(0);
    r.head_stride = k.stride(1);
    r.token_stride = k.stride(2);
    return r;
}

kvarn_status step_tables(PyObject* const* x) {
    const Checker c = {(int)c10::cuda::current_device()};
    const at::Tensor& table = *tensor(x[3], "page_table");
    if (table.dim() != 2) bad("page_table must be [B, max_pages]");
    const int64_t B = table.size(0), width = table.size(1);
    const at::Tensor& free_pages = *tensor(x[4], "free_pages");
    const at::Tensor& positions = *tensor(x[11], "positions");
    if (free_pages.dim() != 1 || positions.dim() != 1) bad("free_pages and positions must have one axis");
    const int64_t cap = free_pages.size(0), n_rows = positions.size(0);
    int64_t hkv = 0;
    int32_t* blocks = nullptr;
    if (const at::Tensor* t = tensor_or_null(x[14], "block_table")) {
        if (t->dim() != 3) bad("block_table must be [B, Hkv, max_pages]");
        hkv = t->size(1);
        blocks = c.array<int32_t>(*t, at::kInt, {B, hkv, width}, "block_table");
    }
    return kvarn_step_tables(
        narrow(B, "B"), narrow(width, "max_pages"), as_int(x[6], "page_size"), c.ints(x[0], {B}, "seq_lens"),
        c.ints(x[1], {B}, "n_new"), c.ints(x[2], {B}, "page_counts"), c.ints(x[3], {B, width}, "page_table"),
        c.ints(x[4], {cap}, "free_pages"), c.ints(x[5], {1}, "free_count"), narrow(cap, "free_capacity"),
        c.ints(x[7], {B}, "kv_lens"), c.ints(x[8], {B}, "page_counts_out"), c.ints(x[9], {1}, "free_count_out"),
        c.ints(x[10], {B + 1}, "cu_tokens"), c.ints(x[11], {n_rows}, "positions"), c.ints(x[12], {n_rows}, "slot_map"),
        narrow(n_rows, "n_rows"), blocks, narrow(hkv, "Hkv"), c.ints(x[13], {1}, "status"), as_stream(x[15], c.dev));
}

kvarn_status rope_qkv(PyObject* const* x) {
    const Checker c = {(int)c10::cuda::current_device()};
    const at::Tensor* q = tensor_or_null(x[0], "q");
    const at::Tensor* k = tensor_or_null(x[1], "k");
    const at::Tensor* v = tensor_or_null(x[2], "v");
    const at::Tensor& positions = *tensor(x[3], "positions");
    const at::Tensor* freq = tensor_or_null(x[4], "inv_freq");
    const at::Tensor* q_out = tensor_or_null(x[5], "q_out");
    const at::Tensor* k_cache = tensor_or_null(x[6], "k_cache");
    const at::Tensor* v_cache = tensor_or_null(x[7], "v_cache");
    if (!q != !q_out || !k != !v || !k != !k_cache || !k != !v_cache)
        bad("q goes with q_out, and k with v, k_cache and v_cache");
    if (!q && !k) bad("neither queries nor keys are given");
    if (positions.dim() != 1) bad("positions must have one axis");
    const int64_t T = positions.size(0);
    const at::ScalarType xt = q ? q->scalar_type() : k->scalar_type(), ot = q ? q_out->scalar_type() : k_cache->scalar_type();
    int64_t hq = 0, hkv = 0;
    Rows rq, ro, rk, rv;
    Cache kv;
    if (q) {
        if (q->dim() != 3) bad("q must be [T, Hq, 128]");
        hq = q->size(1);
        rq = rows(c, *q, xt, T, hq, "q");
        ro = rows(c, *q_out, ot, T, hq, "q_out");
    }
    if (k) {
        if (k->dim() != 3) bad("k must be [T, Hkv, 128]");
        hkv = k->size(1);
        rk = rows(c, *k, xt, T, hkv, "k");
        rv = rows(c, *v, xt, T, hkv, "v");
        if (rk.token != rv.token || rk.head != rv.head) bad("k and v must have the same strides");
        kv = cache(c, *k_cache, *v_cache, ot);
        if (kv.heads != hkv) bad("the cache has " + std::to_string(kv.heads) + " heads, k has " + std::to_string(hkv));
    }
    const int64_t pairs = freq ? freq->numel() : 0;
    return kvarn_rope_qkv(
        as_dtype(xt, "q, k, v"), as_dtype(ot, "q_out and the cache"), narrow(T, "T"), narrow(hq, "Hq"), narrow(hkv, "Hkv"), rq.p,
        rq.token, rq.head, rk.p, rv.p, rk.token, rk.head, c.ints(x[3], {T}, "positions"),
        freq ? c.array<double>(*freq, at::kDouble, {pairs}, "inv_freq") : nullptr, narrow(2 * pairs, "rot_dim"),
        as_bool(x[13]), as_float(x[12]), c.floats_or_null(x[9], {KVARN_HEAD_DIM}, "q_weight"),
        c.floats_or_null(x[10], {KVARN_HEAD_DIM}, "k_weight"), as_float(x[11]), ro.p, ro.token, ro.head, kv.k, kv.v, kv.n_pages,
        kv.page_size, kv.page_stride, kv.head_stride, kv.token_stride, c.ints_or_null(x[8], {T}, "slot_map"),
        as_stream(x[14], c.dev));
}

kvarn_status paged_attention(PyObject* const* x) {
    const Checker c = {(int)c10::cuda::current_device()};
    const at::Tensor& q = *tensor(x[0], "q");
    if (q.dim() != 3) bad("q must be [B, Hq, 128]");
    const int64_t B = q.size(0), hq = q.size(1);
    const at::ScalarType dt = q.scalar_type();
    const Rows rq = rows(c, q, dt, B, hq, "q");
    const Cache kv = cache(c, *tensor(x[1], "k_cache"), *tensor(x[2], "v_cache"), dt);
    const at::Tensor& table = *tensor(x[3], "page_table");
    if (table.dim() != 2) bad("page_table must be [B, max_pages]");
    const int64_t width = table.size(1);
    const at::Tensor& out = *tensor(x[5], "out");
    const at::Tensor& ws = *tensor(x[7], "workspace");
    c.device(ws, "workspace");
    if (!ws.is_contiguous()) bad("workspace must be contiguous");
    return kvarn_paged_attention(
        as_dtype(dt, "q"), narrow(B, "B"), narrow(hq, "Hq"), narrow(kv.heads, "Hkv"), rq.p, rq.token, rq.head, kv.k, kv.v,
        kv.n_pages, kv.page_size, kv.page_stride, kv.head_stride, kv.token_stride, c.ints(x[3], {B, width}, "page_table"),
        narrow(width, "max_pages"), c.ints(x[4], {B}, "kv_lens"), c.ints_or_null(x[11], {B}, "kv_starts"),
        as_int(x[10], "window"), as_float(x[6]), as_float_or_zero(x[8]), c.floats_or_null(x[9], {hq}, "slopes"), ws.data_ptr(),
        (size_t)ws.nbytes(), as_dtype(out.scalar_type(), "out"),
        c.array<void>(out, out.scalar_type(), {B, hq, KVARN_HEAD_DIM}, "out"), c.floats_or_null(x[12], {B, hq}, "lse"),
        as_stream(x[13], c.dev));
}

// No C++ exception leaves through the interpreter.
template <kvarn_status (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return PyLong_FromLong((long)F(args));
    } catch (const PythonError&) {
    } catch (const std::invalid_argument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <kvarn_status (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<step_tables, 16>("step_tables"), method<rope_qkv, 15>("rope_qkv"),
                         method<paged_attention, 14>("paged_attention"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving(void) { return PyModule_Create(&module); }
