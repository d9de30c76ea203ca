// The serving calls' way from Python to the C ABI in one step: takes tensors, checks them and calls.
//
// A decoding step is bound by its host: ten tensors' attributes cost the interpreter some 6 us a call, the kernel
// behind it 2 to 8.  Reading them here costs 0.3 us.
//
// A function accepts a call or returns None: whatever it does not recognise (another type, shape, stride or
// device, an object that is not a plain tensor) is left to the checks in Python, which say what is wrong.  So no
// refusal is worded here, and nothing here is needed for a call to work.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <cstring>

#include "../../include/xsattn.h"

namespace {

decltype(&xs_rope_fwd) rope_fwd;
decltype(&xs_rope_append_paged) append_fwd;
decltype(&xs_paged_step) step_fwd;
decltype(&xs_attn_paged_plan) plan_fwd;
decltype(&xs_attn_paged_fwd) attn_fwd;
decltype(&xs_rope_append_paged8) append8_fwd;
decltype(&xs_paged_read8) read8_fwd;
decltype(&xs_attn_paged8_plan) plan8_fwd;
decltype(&xs_attn_paged8_fwd) attn8_fwd;

struct NotAccepted {};

void need(bool ok) {
    if (!ok) throw NotAccepted{};
}

const at::Tensor& tensor(PyObject* o) {
    need(THPVariable_CheckExact(o));
    const at::Tensor& t = THPVariable_Unpack(o);
    need(t.is_cuda() && t.layout() == at::kStrided);
    return t;
}

long long integer(PyObject* o, long long lo, long long hi) {
    need(PyLong_Check(o));
    int overflow = 0;
    const long long x = PyLong_AsLongLongAndOverflow(o, &overflow);
    need(overflow == 0 && x >= lo && x <= hi);
    return x;
}

int int32(PyObject* o) { return static_cast<int>(integer(o, INT_MIN, INT_MAX)); }

void* address(PyObject* o) { return reinterpret_cast<void*>(static_cast<uintptr_t>(integer(o, 0, LLONG_MAX))); }

int extent(const at::Tensor& t, int i) {
    const int64_t x = t.size(i);
    need(x <= INT_MAX);
    return static_cast<int>(x);
}

int dtype_of(const at::Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return XS_DTYPE_BF16;
    need(t.scalar_type() == at::kHalf);
    return XS_DTYPE_FP16;
}

// The device that a call runs on: its first tensor's, if that is the current one.
int device_of(const at::Tensor& t) {
    const int dev = t.get_device();
    need(dev == c10::cuda::current_device());
    return dev;
}

// None: the current stream of the device
void* stream_of(PyObject* o, int dev) {
    return o == Py_None ? c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream() : address(o);
}

template <typename T>
T* vec(PyObject* o, at::ScalarType type, int64_t n, int dev) {
    const at::Tensor& t = tensor(o);
    need(t.scalar_type() == type && t.dim() == 1 && t.numel() == n && t.is_contiguous() && t.get_device() == dev);
    return static_cast<T*>(t.data_ptr());
}

int* ints(PyObject* o, int64_t n, int dev) { return vec<int>(o, at::kInt, n, dev); }

// A [T, H, D] tensor whose heads are contiguous.
struct Rows {
    void* p;
    int T, H;
    long long stride;
};

Rows rows(const at::Tensor& t, at::ScalarType type, int64_t D, int dev) {
    need(t.scalar_type() == type && t.dim() == 3 && t.size(2) == D && t.get_device() == dev);
    Rows r{t.data_ptr(), extent(t, 0), extent(t, 1), 0};
    need(t.stride(2) == 1 && (r.H <= 1 || t.stride(1) == D));
    r.stride = r.T > 1 ? t.stride(0) : static_cast<long long>(r.H) * D;
    return r;
}

xs_paged_cache cache_of(PyObject* ko, PyObject* vo, at::ScalarType type, int dtype, int dev) {
    const at::Tensor &k = tensor(ko), &v = tensor(vo);
    need(k.dim() == 4 && k.scalar_type() == type && k.get_device() == dev && k.stride(3) == 1);
    need(v.scalar_type() == type && v.get_device() == dev && v.sizes() == k.sizes() && v.stride(3) == 1);
    xs_paged_cache c;
    std::memset(&c, 0, sizeof c);
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    for (int i = 0; i < 3; ++i) {
        c.k_strides[i] = k.stride(i);
        c.v_strides[i] = v.stride(i);
    }
    c.n_pages = extent(k, 0);
    c.page_size = extent(k, 1);
    c.Hkv = extent(k, 2);
    c.D = extent(k, 3);
    c.dtype = dtype;
    return c;
}

// A cache of e4m3 numbers, and its scales (e8m0, or their bytes).
xs_paged_cache8 cache8_of(PyObject* ko, PyObject* vo, PyObject* kso, PyObject* vso, int dtype, int dev) {
    const at::Tensor &k = tensor(ko), &v = tensor(vo), &ks = tensor(kso), &vs = tensor(vso);
    need(k.dim() == 4 && k.scalar_type() == at::kFloat8_e4m3fn && k.get_device() == dev && k.stride(3) == 1);
    need(v.scalar_type() == at::kFloat8_e4m3fn && v.get_device() == dev && v.sizes() == k.sizes() && v.stride(3) == 1);
    xs_paged_cache8 c;
    std::memset(&c, 0, sizeof c);
    c.n_pages = extent(k, 0);
    c.page_size = extent(k, 1);
    c.Hkv = extent(k, 2);
    c.D = extent(k, 3);
    for (const at::Tensor* t : {&ks, &vs}) {
        need(t->scalar_type() == at::kFloat8_e8m0fnu || t->scalar_type() == at::kByte);
        need(t->dim() == 3 && t->size(0) == c.n_pages && t->size(2) == c.Hkv && t->size(1) == ks.size(1) && t->get_device() == dev);
    }
    need(ks.size(1) >= 1 && c.page_size % ks.size(1) == 0);
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.k_scales = ks.data_ptr();
    c.v_scales = vs.data_ptr();
    for (int i = 0; i < 3; ++i) {
        c.k_strides[i] = k.stride(i);
        c.v_strides[i] = v.stride(i);
        c.k_scale_strides[i] = ks.stride(i);
        c.v_scale_strides[i] = vs.stride(i);
    }
    c.block = static_cast<int>(c.page_size / ks.size(1));
    c.dtype = dtype;
    return c;
}

template <typename F>
PyObject* call(F&& f) {
    int code;
    Py_BEGIN_ALLOW_THREADS
    code = f();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(code);
}

// No C++ exception leaves this file.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n == N) {
        try {
            return F(args);
        } catch (...) {
            PyErr_Clear();
        }
    }
    Py_RETURN_NONE;
}

// x, positions, out, rope, D, grad, stream
PyObject* rope(PyObject* const* a) {
    const at::Tensor &x = tensor(a[0]), &out = tensor(a[2]);
    const int dtype = dtype_of(x), dev = device_of(x), D = int32(a[4]), grad = int32(a[5]);
    const Rows xr = rows(x, x.scalar_type(), D, dev), o = rows(out, x.scalar_type(), D, dev);
    need(xr.T == o.T && xr.H == o.H);
    const int* positions = ints(a[1], xr.T, dev);
    const xs_rope* r = static_cast<const xs_rope*>(address(a[3]));
    void* stream = stream_of(a[6], dev);
    return call([&] { return rope_fwd(xr.p, positions, o.p, xr.T, xr.H, xr.stride, o.stride, dtype, grad, r, stream); });
}

// q, k, v, positions, slots, q_out, k_cache, v_cache, rope, D, stream
PyObject* append(PyObject* const* a) {
    const at::Tensor& q = tensor(a[0]);
    const at::ScalarType type = q.scalar_type();
    const int dtype = dtype_of(q), dev = device_of(q), D = int32(a[9]);
    const Rows qr = rows(q, type, D, dev), k = rows(tensor(a[1]), type, D, dev), v = rows(tensor(a[2]), type, D, dev),
               o = rows(tensor(a[5]), type, D, dev);
    xs_rope_append_args g;
    std::memset(&g, 0, sizeof g);
    g.cache = cache_of(a[6], a[7], type, dtype, dev);
    need(qr.T == k.T && qr.T == v.T && qr.T == o.T && qr.H == o.H && k.H == v.H && g.cache.Hkv == k.H && g.cache.D == D);
    g.q = qr.p;
    g.k = k.p;
    g.v = v.p;
    g.positions = ints(a[3], qr.T, dev);
    g.slots = vec<long long>(a[4], at::kLong, qr.T, dev);
    g.q_out = o.p;
    g.rope = static_cast<const xs_rope*>(address(a[8]));
    g.q_stride = qr.stride;
    g.k_stride = k.stride;
    g.v_stride = v.stride;
    g.q_out_stride = o.stride;
    g.T = qr.T;
    g.H = qr.H;
    void* stream = stream_of(a[10], dev);
    return call([&] { return append_fwd(&g, stream); });
}

// cache_lens, new_lens, block_table, free_pages, free_count, page_size, kv_lens, cu_q, positions, slots,
// free_count_out, status, stream
PyObject* step(PyObject* const* a) {
    const at::Tensor& table = tensor(a[2]);
    need(table.dim() == 2 && table.scalar_type() == at::kInt && table.is_contiguous());
    const int dev = device_of(table), n = extent(table, 0), width = extent(table, 1), page_size = int32(a[5]);
    const int64_t pages = tensor(a[3]).numel(), rows = tensor(a[8]).numel();
    need(pages <= INT_MAX && rows <= INT_MAX);
    int* const table_p = static_cast<int*>(table.data_ptr());
    const int *cached = ints(a[0], n, dev), *fresh = ints(a[1], n, dev), *count = ints(a[4], 1, dev);
    int *free_pages = ints(a[3], pages, dev), *kv = ints(a[6], n, dev), *cu = ints(a[7], int64_t(n) + 1, dev),
        *positions = ints(a[8], rows, dev), *count_out = ints(a[10], 1, dev), *status = ints(a[11], n, dev);
    long long* slots = vec<long long>(a[9], at::kLong, rows, dev);
    void* stream = stream_of(a[12], dev);
    return call([&] {
        return step_fwd(cached, fresh, table_p, free_pages, count, n, width, static_cast<int>(pages), page_size,
                        static_cast<int>(rows), kv, cu, positions, slots, count_out, status, stream);
    });
}

// A workspace: its buffer, and (n, H, Hkv, D, address, bytes).
struct Work {
    int n, H, Hkv, D;
    void* p;
    size_t bytes;
};

Work work_of(PyObject* buffer, PyObject* dims, int dev) {
    need(tensor(buffer).get_device() == dev && PyTuple_CheckExact(dims) && PyTuple_GET_SIZE(dims) == 6);
    auto at = [&](int i) { return PyTuple_GET_ITEM(dims, i); };
    return Work{int32(at(0)), int32(at(1)), int32(at(2)), int32(at(3)), address(at(4)),
                static_cast<size_t>(integer(at(5), 0, LLONG_MAX))};
}

// cu_q, kv_lens, max_q, buffer, dims, causal, window, stream
PyObject* plan_with(decltype(&xs_attn_paged_plan) f, PyObject* const* a) {
    const int dev = device_of(tensor(a[0]));
    const Work w = work_of(a[3], a[4], dev);
    const int *cu = ints(a[0], int64_t(w.n) + 1, dev), *kv = ints(a[1], w.n, dev);
    const int max_q = int32(a[2]), causal = int32(a[5]), window = int32(a[6]);
    void* stream = stream_of(a[7], dev);
    return call([&] { return f(cu, kv, w.n, w.H, w.Hkv, w.D, max_q, causal, window, w.p, w.bytes, stream); });
}

PyObject* plan(PyObject* const* a) { return plan_with(plan_fwd, a); }
PyObject* plan8(PyObject* const* a) { return plan_with(plan8_fwd, a); }

// The arguments of an attention beside q and the cache, from `a` = block_table, layout, outs, scale, buffer, dims,
// planned, lse.
template <typename Args>
void fill_attn(Args& g, const at::Tensor& q, PyObject* const* a, int dev) {
    const at::Tensor& table = tensor(a[0]);
    const at::ScalarType type = q.scalar_type();
    const Work w = work_of(a[4], a[5], dev);
    const Rows qr = rows(q, type, w.D, dev);
    need(qr.H == w.H && g.cache.Hkv == w.Hkv && g.cache.D == w.D);
    need(table.dim() == 2 && table.scalar_type() == at::kInt && table.size(0) == w.n && table.get_device() == dev);
    g.table_width = extent(table, 1);
    need(table.stride(1) == 1 || g.table_width <= 1);
    g.layout = int32(a[1]);
    need(PyList_CheckExact(a[2]) || PyTuple_CheckExact(a[2]));
    const Py_ssize_t P = PySequence_Fast_GET_SIZE(a[2]);
    need(P >= 1 && P <= XS_MAX_P);
    const bool one = g.layout == XS_LAYOUT_CONTIGUOUS, shards = g.layout == XS_LAYOUT_A2A;
    const int64_t out_T = shards ? qr.T / P : qr.T, out_H = one || shards ? qr.H : qr.H / P;
    for (Py_ssize_t i = 0; i < P; ++i) {
        const at::Tensor& o = tensor(PySequence_Fast_GET_ITEM(a[2], i));
        need(o.dim() == 3 && o.size(0) == out_T && o.size(1) == out_H && o.size(2) == w.D && o.scalar_type() == type &&
             o.is_contiguous() && o.get_device() == dev);
        g.outs[i] = o.data_ptr();
    }
    need(PyFloat_CheckExact(a[3]));
    const double scale = PyFloat_AS_DOUBLE(a[3]);
    need(std::fabs(scale) <= FLT_MAX);
    need(PyTuple_CheckExact(a[6]) && PyTuple_GET_SIZE(a[6]) == 3);
    if (a[7] != Py_None) {
        const at::Tensor& z = tensor(a[7]);
        need(z.scalar_type() == at::kFloat && z.dim() == 2 && z.size(0) == qr.T && z.size(1) == qr.H && z.is_contiguous() &&
             z.get_device() == dev);
        g.lse = static_cast<float*>(z.data_ptr());
    }
    g.q = qr.p;
    g.block_table = static_cast<const int*>(table.data_ptr());
    g.workspace = w.p;
    g.workspace_bytes = w.bytes;
    g.q_stride = qr.stride;
    g.table_stride = table.stride(0);
    g.P = static_cast<int>(P);
    g.T = qr.T;
    g.H = qr.H;
    g.n = w.n;
    g.max_q = int32(PyTuple_GET_ITEM(a[6], 0));
    g.causal = int32(PyTuple_GET_ITEM(a[6], 1));
    g.window = int32(PyTuple_GET_ITEM(a[6], 2));
    g.scale = static_cast<float>(scale);
}

// q, k_cache, v_cache, block_table, layout, outs, scale, buffer, dims, planned, lse, stream
PyObject* attn(PyObject* const* a) {
    const at::Tensor& q = tensor(a[0]);
    const int dtype = dtype_of(q), dev = device_of(q);
    xs_attn_paged_args g;
    std::memset(&g, 0, sizeof g);
    g.cache = cache_of(a[1], a[2], q.scalar_type(), dtype, dev);
    fill_attn(g, q, a + 3, dev);
    void* stream = stream_of(a[11], dev);
    return call([&] { return attn_fwd(&g, stream); });
}

// q, k_cache, v_cache, k_scales, v_scales, block_table, layout, outs, scale, buffer, dims, planned, lse, stream
PyObject* attn8(PyObject* const* a) {
    const at::Tensor& q = tensor(a[0]);
    const int dtype = dtype_of(q), dev = device_of(q);
    xs_attn_paged8_args g;
    std::memset(&g, 0, sizeof g);
    g.cache = cache8_of(a[1], a[2], a[3], a[4], dtype, dev);
    fill_attn(g, q, a + 5, dev);
    void* stream = stream_of(a[13], dev);
    return call([&] { return attn8_fwd(&g, stream); });
}

// q, k, v, positions, slots, q_out, k_cache, v_cache, k_scales, v_scales, rope, D, stream
PyObject* append8(PyObject* const* a) {
    const at::Tensor& q = tensor(a[0]);
    const at::ScalarType type = q.scalar_type();
    const int dtype = dtype_of(q), dev = device_of(q), D = int32(a[11]);
    const Rows qr = rows(q, type, D, dev), k = rows(tensor(a[1]), type, D, dev), v = rows(tensor(a[2]), type, D, dev),
               o = rows(tensor(a[5]), type, D, dev);
    xs_rope_append8_args g;
    std::memset(&g, 0, sizeof g);
    g.cache = cache8_of(a[6], a[7], a[8], a[9], dtype, dev);
    need(qr.T == k.T && qr.T == v.T && qr.T == o.T && qr.H == o.H && k.H == v.H && g.cache.Hkv == k.H && g.cache.D == D);
    g.q = qr.p;
    g.k = k.p;
    g.v = v.p;
    g.positions = ints(a[3], qr.T, dev);
    g.slots = vec<long long>(a[4], at::kLong, qr.T, dev);
    g.q_out = o.p;
    g.rope = static_cast<const xs_rope*>(address(a[10]));
    g.q_stride = qr.stride;
    g.k_stride = k.stride;
    g.v_stride = v.stride;
    g.q_out_stride = o.stride;
    g.T = qr.T;
    g.H = qr.H;
    void* stream = stream_of(a[12], dev);
    return call([&] { return append8_fwd(&g, stream); });
}

// k_cache, v_cache, k_scales, v_scales, block_table, cu_rows, first, k_out, v_out, stream
PyObject* read8(PyObject* const* a) {
    const at::Tensor &ko = tensor(a[7]), &table = tensor(a[4]);
    const int dtype = dtype_of(ko), dev = device_of(ko);
    xs_paged_read8_args g;
    std::memset(&g, 0, sizeof g);
    g.cache = cache8_of(a[0], a[1], a[2], a[3], dtype, dev);
    const Rows k = rows(ko, ko.scalar_type(), g.cache.D, dev), v = rows(tensor(a[8]), ko.scalar_type(), g.cache.D, dev);
    need(k.T == v.T && k.H == v.H && k.H == g.cache.Hkv);
    need(table.dim() == 2 && table.scalar_type() == at::kInt && table.get_device() == dev);
    g.n = extent(table, 0);
    g.table_width = extent(table, 1);
    need(table.stride(1) == 1 || g.table_width <= 1);
    g.block_table = static_cast<const int*>(table.data_ptr());
    g.cu_rows = ints(a[5], int64_t(g.n) + 1, dev);
    g.first = a[6] == Py_None ? nullptr : ints(a[6], g.n, dev);
    g.k_out = k.p;
    g.v_out = v.p;
    g.k_stride = k.stride;
    g.v_stride = v.stride;
    g.table_stride = table.stride(0);
    g.T = k.T;
    void* stream = stream_of(a[9], dev);
    return call([&] { return read8_fwd(&g, stream); });
}

// The addresses of the nine entry points, in the order below.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    unsigned long long p[9];
    for (Py_ssize_t i = 0; i < 9; ++i) {
        p[i] = n == 9 ? PyLong_AsUnsignedLongLong(args[i]) : 0;
        if (PyErr_Occurred()) return nullptr;
        if (p[i] == 0) {
            PyErr_SetString(PyExc_ValueError, "nine addresses");
            return nullptr;
        }
    }
    rope_fwd = reinterpret_cast<decltype(rope_fwd)>(p[0]);
    append_fwd = reinterpret_cast<decltype(append_fwd)>(p[1]);
    step_fwd = reinterpret_cast<decltype(step_fwd)>(p[2]);
    plan_fwd = reinterpret_cast<decltype(plan_fwd)>(p[3]);
    attn_fwd = reinterpret_cast<decltype(attn_fwd)>(p[4]);
    append8_fwd = reinterpret_cast<decltype(append8_fwd)>(p[5]);
    read8_fwd = reinterpret_cast<decltype(read8_fwd)>(p[6]);
    plan8_fwd = reinterpret_cast<decltype(plan8_fwd)>(p[7]);
    attn8_fwd = reinterpret_cast<decltype(attn8_fwd)>(p[8]);
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F* f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f));
}

PyMethodDef methods[] = {
    {"bind", fast(bind), METH_FASTCALL, "addresses of the C ABI's entry points"},
    {"rope", fast(entry<rope, 7>), METH_FASTCALL, "xs_rope_fwd"},
    {"append", fast(entry<append, 11>), METH_FASTCALL, "xs_rope_append_paged"},
    {"step", fast(entry<step, 13>), METH_FASTCALL, "xs_paged_step"},
    {"plan", fast(entry<plan, 8>), METH_FASTCALL, "xs_attn_paged_plan"},
    {"attn", fast(entry<attn, 12>), METH_FASTCALL, "xs_attn_paged_fwd"},
    {"append8", fast(entry<append8, 13>), METH_FASTCALL, "xs_rope_append_paged8"},
    {"read8", fast(entry<read8, 10>), METH_FASTCALL, "xs_paged_read8"},
    {"plan8", fast(entry<plan8, 8>), METH_FASTCALL, "xs_attn_paged8_plan"},
    {"attn8", fast(entry<attn8, 14>), METH_FASTCALL, "xs_attn_paged8_fwd"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Serving calls on tensors.", -1, methods, nullptr, nullptr, nullptr,
                      nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    PyObject* m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
