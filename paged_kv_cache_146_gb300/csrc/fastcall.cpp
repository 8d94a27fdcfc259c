// Compiled form of the binding's argument checks for the calls that a decode step
// makes once per layer (rotated append, windowed and block-scaled attention,
// read-back): a call of a few rows spends most of its time on the host, and there
// most of it on reading tensor fields from Python.  Measured back to back: a rotated
// append of 57 tokens 10.8 us through Python's checks and ctypes, 3.1 here; windowed
// decode of 3 sequences 8.5 and 4.1.
//
// Each function makes the same checks as the Python binding, and calls the
// library when all of them hold.  When one does not (or the tensors sit on
// another device than the current one) it returns None without calling anything,
// and the binding's own checks say what is wrong.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "pagedkv.h"

namespace {

// Entry points of the library, set once by bind().
decltype(&paged_decode_attention_window) decode_window = nullptr;
decltype(&paged_decode_attention_b8) decode_b8 = nullptr;
decltype(&kv_cache_write_rope) write_rope = nullptr;
decltype(&kv_dequantize_blocks) dequantize = nullptr;
decltype(&paged_prefill_attention_window) prefill_window = nullptr;

// The library is called without the interpreter lock, like through ctypes: a launch
// waits while the driver's queue is full.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// A check that did not hold.
struct Refused {};
inline void want(bool ok)
{
    if (!ok) throw Refused{};
}

// (handle, blocks, kv heads, block size, head_dim, bf16 rows, record bytes)
struct Pool {
    const pkv_pool *handle;
    int64_t blocks, heads, block_size, dim, record;
    at::ScalarType rows;
};

int64_t integer(PyObject *o)
{
    want(PyLong_Check(o));
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused{};
    }
    return v;
}

Pool pool_of(PyObject *o)
{
    want(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 7);
    Pool p;
    p.handle = reinterpret_cast<const pkv_pool *>(integer(PyTuple_GET_ITEM(o, 0)));
    p.blocks = integer(PyTuple_GET_ITEM(o, 1));
    p.heads = integer(PyTuple_GET_ITEM(o, 2));
    p.block_size = integer(PyTuple_GET_ITEM(o, 3));
    p.dim = integer(PyTuple_GET_ITEM(o, 4));
    p.rows = integer(PyTuple_GET_ITEM(o, 5)) ? at::kBFloat16 : at::kHalf;
    p.record = integer(PyTuple_GET_ITEM(o, 6));
    return p;
}

const at::Tensor &tensor(PyObject *o)
{
    want(THPVariable_Check(o));
    return THPVariable_Unpack(o);
}

// A contiguous tensor of the call; its address.
void *dense(PyObject *o, at::IntArrayRef sizes, at::ScalarType type, c10::DeviceIndex dev)
{
    const at::Tensor &t = tensor(o);
    want(t.is_cuda() && t.get_device() == dev && t.scalar_type() == type && t.sizes() == sizes &&
         t.is_contiguous());
    return t.data_ptr();
}

void *status_word(PyObject *o, c10::DeviceIndex dev)
{
    const at::Tensor &t = tensor(o);
    want(t.is_cuda() && t.get_device() == dev && t.scalar_type() == at::kInt && t.numel() >= 1);
    return t.data_ptr();
}

// Rows [T][H][D] with any token stride; their address and stride.
void *rows(const at::Tensor &t, int64_t T, int64_t H, int64_t D, at::ScalarType type,
           c10::DeviceIndex dev, int64_t *stride)
{
    want(t.is_cuda() && t.get_device() == dev && t.scalar_type() == type && t.dim() == 3 &&
         t.size(0) == T && t.size(1) == H && t.size(2) == D);
    want(T == 0 || H == 0 || (t.stride(2) == 1 && (t.stride(1) == D || H == 1)));
    *stride = H * D;
    if (T > 1) {
        *stride = t.stride(0);
        want(*stride >= H * D && *stride % 8 == 0);
    }
    return t.data_ptr();
}

struct Pools {
    void *a, *b;
};

// K and V pools, or the record pool (second object ignored).
Pools pools_of(const Pool &p, PyObject *a, PyObject *b, c10::DeviceIndex dev)
{
    if (p.record) {
        const int64_t sizes[3] = {p.blocks, p.heads, p.record};
        return {dense(a, sizes, at::kByte, dev), nullptr};
    }
    const int64_t sizes[4] = {p.blocks, p.heads, p.block_size, p.dim};
    return {dense(a, sizes, p.rows, dev), dense(b, sizes, p.rows, dev)};
}

// The call's stream on the current device.
void *stream_of(PyObject *o, c10::DeviceIndex dev)
{
    want(c10::cuda::current_device() == dev);
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev).stream();
    return reinterpret_cast<void *>(integer(o));
}

template <typename F>
PyObject *guarded(F &&call)
{
    try {
        return PyLong_FromLong(call());
    } catch (const Refused &) {
    } catch (const std::exception &) {     // from a tensor field: the binding says which
    }
    Py_RETURN_NONE;
}

// (pool, q, out, tables, lens, scale, window, sinks, status, k_pool or records, v_pool, stream)
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> long {
        want(n == 12 && decode_window);
        const Pool p = pool_of(a[0]);
        const at::Tensor &q = tensor(a[1]);
        want(q.is_cuda() && q.dim() == 3 && q.scalar_type() == p.rows && q.is_contiguous());
        const auto dev = static_cast<c10::DeviceIndex>(q.get_device());
        const int64_t S = q.size(0), hq = q.size(1);
        want(q.size(2) == p.dim && hq % p.heads == 0 && S <= INT32_MAX && hq <= INT32_MAX);
        void *out = dense(a[2], q.sizes(), p.rows, dev);
        const at::Tensor &tables = tensor(a[3]);
        want(tables.dim() == 2 && tables.size(1) <= INT32_MAX);
        const int64_t maxb = tables.size(1), ts[2] = {S, maxb}, ls[1] = {S};
        const auto *tp = static_cast<const int32_t *>(dense(a[3], ts, at::kInt, dev));
        const auto *lp = static_cast<const int32_t *>(dense(a[4], ls, at::kInt, dev));
        want(PyFloat_Check(a[5]));
        const float scale = static_cast<float>(PyFloat_AS_DOUBLE(a[5]));
        const int64_t window = integer(a[6]), sinks = integer(a[7]);
        auto *status = static_cast<int32_t *>(status_word(a[8], dev));
        const Pools pools = pools_of(p, a[9], a[10], dev);
        void *stream = stream_of(a[11], dev);
        const Unlocked unlocked;
        if (p.record)
            return decode_b8(p.handle, out, q.data_ptr(), pools.a, tp, (int32_t)maxb, lp, (int32_t)S,
                             (int32_t)hq, scale, (int32_t)window, (int32_t)sinks, status, stream);
        return decode_window(p.handle, out, q.data_ptr(), pools.a, pools.b, tp, (int32_t)maxb, lp,
                             (int32_t)S, (int32_t)hq, scale, (int32_t)window, (int32_t)sinks, status,
                             stream);
    });
}

// (pool, k_new, v_new, positions, cos_sin, slots, status, q, q_out, interleaved, k_pool or
// records, v_pool, stream); q and q_out None: no queries
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> long {
        want(n == 13 && write_rope);
        const Pool p = pool_of(a[0]);
        const at::Tensor &k = tensor(a[1]), &v = tensor(a[2]);
        want(k.is_cuda());
        const auto dev = static_cast<c10::DeviceIndex>(k.get_device());
        const at::Tensor &slots = tensor(a[5]), &table = tensor(a[4]);
        want(slots.dim() == 1 && table.dim() == 2 && slots.size(0) <= INT32_MAX &&
             table.size(0) <= INT32_MAX && table.size(1) <= INT32_MAX);
        const int64_t T = slots.size(0), one[1] = {T};
        const auto *sp = static_cast<const int64_t *>(dense(a[5], one, at::kLong, dev));
        const auto *pp = static_cast<const int32_t *>(dense(a[3], one, at::kInt, dev));
        const auto *cs = static_cast<const float *>(dense(a[4], table.sizes(), at::kFloat, dev));
        int64_t ks, vs, qs = 0, os = 0, hq = 0;
        const void *kp = rows(k, T, p.heads, p.dim, p.rows, dev, &ks);
        const void *vp = rows(v, T, p.heads, p.dim, p.rows, dev, &vs);
        const void *qp = nullptr;
        void *op = nullptr;
        if (a[7] != Py_None) {
            const at::Tensor &q = tensor(a[7]);
            want(q.dim() == 3 && q.size(1) <= INT32_MAX);
            hq = q.size(1);
            qp = rows(q, T, hq, p.dim, p.rows, dev, &qs);
            op = rows(tensor(a[8]), T, hq, p.dim, p.rows, dev, &os);
            want(qp != op || qs == os);
        } else {
            want(a[8] == Py_None);
        }
        auto *status = static_cast<int32_t *>(status_word(a[6], dev));
        const Pools pools = pools_of(p, a[10], a[11], dev);
        const bool interleaved = integer(a[9]) != 0;
        void *stream = stream_of(a[12], dev);
        const Unlocked unlocked;
        return write_rope(p.handle, op, os, qp, qs, (int32_t)hq, kp, ks, vp, vs, pp, cs,
                          (int32_t)table.size(0), (int32_t)table.size(1), interleaved, sp,
                          (int32_t)T, pools.a, pools.b, status, stream);
    });
}

// (pool, ids, k_out, v_out, status, records, stream)
PyObject *dequant(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> long {
        want(n == 7 && dequantize);
        const Pool p = pool_of(a[0]);
        const at::Tensor &ids = tensor(a[1]);
        want(p.record && ids.is_cuda() && ids.dim() == 1 && ids.size(0) <= INT32_MAX);
        const auto dev = static_cast<c10::DeviceIndex>(ids.get_device());
        const int64_t m = ids.size(0), one[1] = {m}, sizes[4] = {m, p.heads, 16, p.dim};
        const auto *ip = static_cast<const int32_t *>(dense(a[1], one, at::kInt, dev));
        void *k = dense(a[2], sizes, p.rows, dev), *v = dense(a[3], sizes, p.rows, dev);
        auto *status = static_cast<int32_t *>(status_word(a[4], dev));
        const Pools pools = pools_of(p, a[5], Py_None, dev);
        void *stream = stream_of(a[6], dev);
        const Unlocked unlocked;
        return dequantize(p.handle, ip, (int32_t)m, pools.a, k, v, status, stream);
    });
}

// (pool, q, out, tables, query_start, lens, scale, window, sinks, workspace, status, k_pool,
// v_pool, stream)
PyObject *prefill(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> long {
        want(n == 14 && prefill_window);
        const Pool p = pool_of(a[0]);
        const at::Tensor &q = tensor(a[1]);
        want(!p.record && q.is_cuda() && q.dim() == 3 && q.scalar_type() == p.rows &&
             q.is_contiguous());
        const auto dev = static_cast<c10::DeviceIndex>(q.get_device());
        const int64_t T = q.size(0), hq = q.size(1);
        want(q.size(2) == p.dim && hq % p.heads == 0 && T <= INT32_MAX && hq <= INT32_MAX);
        void *out = dense(a[2], q.sizes(), p.rows, dev);
        const at::Tensor &tables = tensor(a[3]), &ws = tensor(a[9]);
        want(tables.dim() == 2 && tables.size(0) < INT32_MAX && tables.size(1) <= INT32_MAX &&
             ws.dim() == 1);
        const int64_t S = tables.size(0), maxb = tables.size(1);
        const int64_t ts[2] = {S, maxb}, ls[1] = {S}, qs[1] = {S + 1};
        const auto *tp = static_cast<const int32_t *>(dense(a[3], ts, at::kInt, dev));
        const auto *sp = static_cast<const int32_t *>(dense(a[4], qs, at::kInt, dev));
        const auto *lp = static_cast<const int32_t *>(dense(a[5], ls, at::kInt, dev));
        want(PyFloat_Check(a[6]));
        const float scale = static_cast<float>(PyFloat_AS_DOUBLE(a[6]));
        void *wp = dense(a[9], ws.sizes(), at::kByte, dev);
        auto *status = static_cast<int32_t *>(status_word(a[10], dev));
        const Pools pools = pools_of(p, a[11], a[12], dev);
        const int64_t window = integer(a[7]), sinks = integer(a[8]);
        void *stream = stream_of(a[13], dev);
        const Unlocked unlocked;
        return prefill_window(p.handle, out, q.data_ptr(), pools.a, pools.b, tp, (int32_t)maxb, sp, lp,
                              (int32_t)S, (int32_t)T, (int32_t)hq, scale, (int32_t)window,
                              (int32_t)sinks, wp, (size_t)ws.numel(), status, stream);
    });
}

// Addresses of the library's entry points, in the order of the variables above.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
        return nullptr;
    }
    void *p[5];
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
            return nullptr;
        }
    }
    decode_window = reinterpret_cast<decltype(decode_window)>(p[0]);
    decode_b8 = reinterpret_cast<decltype(decode_b8)>(p[1]);
    write_rope = reinterpret_cast<decltype(write_rope)>(p[2]);
    dequantize = reinterpret_cast<decltype(dequantize)>(p[3]);
    prefill_window = reinterpret_cast<decltype(prefill_window)>(p[4]);
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<decode>("decode"), method<rope>("rope"), method<dequant>("dequantize"),
                         method<prefill>("prefill"), method<bind>("bind"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall(void)
{
    // what the binding compares before it takes the module
    PyObject *m = PyModule_Create(&module);
    if (m && (PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0 ||
              PyModule_AddIntConstant(m, "python_version", PY_MAJOR_VERSION * 100 + PY_MINOR_VERSION) < 0 ||
              PyModule_AddStringConstant(m, "interface", PKV_INTERFACE) < 0)) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
