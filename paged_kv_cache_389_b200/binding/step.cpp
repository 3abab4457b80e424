// The serving-step calls for Python: checks of tensors, device and stream, then the call
// into the library (include/pa.h).
//
// Why compiled: these calls take 4 to 10 us on the GPU, and the same checks written in Python
// with a ctypes call took 10 us on the host (0.6 us a tensor, 2 us for the 15 to 18 converted
// arguments), so a loop of them was bound by the binding.
//
// Every function takes its tensors, numbers, the error flag (or None) and the stream (or
// None: the current one of the tensors' device) by position and returns the pa_status.  A wrong
// tensor raises AssertionError, a pool of another type TypeError; no C++ exception leaves.
#include <Python.h>

#include <initializer_list>
#include <string>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pa.h"

namespace {

struct Refused {
    PyObject *type;   // borrowed (a static exception type); nullptr: an error is set already
    std::string what;
};

std::string list(at::IntArrayRef x) {
    std::string s = "(";
    for (size_t i = 0; i < x.size(); ++i) s += (i ? ", " : "") + std::to_string(x[i]);
    return s + ")";
}

const at::Tensor &tensor(PyObject *o, const char *what) {
    if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(what) + ": a tensor wanted"};
    return THPVariable_Unpack(o);
}

const at::Tensor &tensor_of(PyObject *o, int64_t dims, const char *what) {
    const at::Tensor &t = tensor(o, what);
    if (t.dim() != dims)
        throw Refused{PyExc_AssertionError, std::string(what) + ": " + std::to_string(dims) + " dimensions wanted, got shape " +
                                                list(t.sizes())};
    return t;
}

int device_of(const at::Tensor &t) { return t.is_cuda() ? (int)t.get_device() : -1; }

// Address of a contiguous tensor of this type and shape on device `dev`.
template <typename T = void>
T *ptr(PyObject *o, at::ScalarType type, std::initializer_list<int64_t> shape, int dev, const char *what) {
    const at::Tensor &t = tensor(o, what);
    if (t.scalar_type() != type || !t.sizes().equals(at::IntArrayRef(shape)) || device_of(t) != dev || !t.is_contiguous())
        throw Refused{PyExc_AssertionError,
                      std::string(what) + ": contiguous " + c10::toString(type) + " of shape " + list(at::IntArrayRef(shape)) +
                          " on device " + std::to_string(dev) + " wanted, got " + c10::toString(t.scalar_type()) + " " +
                          list(t.sizes()) + " on " + t.device().str() + (t.is_contiguous() ? "" : ", strided")};
    return static_cast<T *>(t.data_ptr());
}

int32_t *i32(PyObject *o, std::initializer_list<int64_t> shape, int dev, const char *what) {
    return ptr<int32_t>(o, at::kInt, shape, dev, what);
}

int32_t *flag(PyObject *o, int dev) { return o == Py_None ? nullptr : i32(o, {1}, dev, "err_flag"); }

int32_t narrow(int64_t x, const char *what) {
    if (x < 0 || x > INT32_MAX) throw Refused{PyExc_AssertionError, std::string(what) + ": out of 32 bits"};
    return (int32_t)x;
}

int32_t integer(PyObject *o, const char *what) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Refused{nullptr, {}};
    if (x < INT32_MIN || x > INT32_MAX) throw Refused{PyExc_AssertionError, std::string(what) + ": out of 32 bits"};
    return (int32_t)x;
}

float number(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Refused{nullptr, {}};
    return (float)x;
}

// bf16 [tokens, heads, d] whose heads and dims are contiguous; the tokens may be further apart.
struct Rows {
    void *p;
    int64_t stride;   // elements between tokens
    Rows(PyObject *o, int64_t tokens, int64_t heads, int64_t d, int dev, const char *what) {
        const at::Tensor &t = tensor(o, what);
        if (t.scalar_type() != at::kBFloat16 || !t.sizes().equals({tokens, heads, d}) || device_of(t) != dev ||
            t.stride(2) != 1 || (heads > 1 && t.stride(1) != d))
            throw Refused{PyExc_AssertionError,
                          std::string(what) + ": bf16 " + list({tokens, heads, d}) +
                              " with contiguous heads and dims on device " + std::to_string(dev) + " wanted, got " +
                              c10::toString(t.scalar_type()) + " " + list(t.sizes()) + " with strides " + list(t.strides()) +
                              " on " + t.device().str()};
        p = t.data_ptr();
        stride = tokens > 1 ? t.stride(0) : heads * d;
    }
};

// 8-bit pools with a scale per (block, kv head).
struct Pool {
    int dev;
    pa_cache_desc desc;
    void *kc, *vc;
    float *ks, *vs;
    Pool(PyObject *key, PyObject *value, PyObject *key_scales, PyObject *value_scales) {
        const at::Tensor &t = tensor_of(key, 4, "key_cache");
        const at::ScalarType type = t.scalar_type();
        if (type != at::kFloat8_e4m3fn && type != at::kChar)
            throw Refused{PyExc_TypeError, std::string("unsupported dtype ") + c10::toString(type)};
        dev = device_of(t);
        const int64_t nb = t.size(0), h = t.size(1), bs = t.size(2), d = t.size(3);
        kc = ptr(key, type, {nb, h, bs, d}, dev, "key_cache");
        vc = ptr(value, type, {nb, h, bs, d}, dev, "value_cache");
        ks = ptr<float>(key_scales, at::kFloat, {nb, h}, dev, "key_scales");
        vs = ptr<float>(value_scales, at::kFloat, {nb, h}, dev, "value_scales");
        desc = pa_cache_desc{narrow(nb, "key_cache"), narrow(h, "key_cache"), narrow(bs, "key_cache"), narrow(d, "key_cache"),
                             type == at::kChar ? PA_INT8 : PA_FP8_E4M3, 1.f, 1.f};
    }
};

struct Workspace {
    void *p;
    size_t bytes;
    Workspace(PyObject *o, int dev) {
        const at::Tensor &t = tensor(o, "workspace");
        if (device_of(t) != dev || !t.is_contiguous())
            throw Refused{PyExc_AssertionError, "workspace: contiguous and on the other tensors' device"};
        p = t.data_ptr();
        bytes = t.nbytes();
    }
};

// Makes `dev` the current device for the call and gives the stream to launch on.  While it lives
// the interpreter lock is free, as ctypes leaves it for the library's other calls: a launch that
// waits for room in a full queue does not hold up the program's other threads.
class Launch {
public:
    Launch(int dev, PyObject *stream) {
        if (dev < 0) throw Refused{PyExc_AssertionError, "tensors passed to the library must be on a CUDA device"};
        if (stream == Py_None) {
            s_ = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
        } else {
            PyObject *h = PyObject_GetAttrString(stream, "cuda_stream");
            if (!h) throw Refused{nullptr, {}};
            s_ = PyLong_AsVoidPtr(h);
            Py_DECREF(h);
            if (PyErr_Occurred()) throw Refused{nullptr, {}};
        }
        guard_.set_index((c10::DeviceIndex)dev);
        state_ = PyEval_SaveThread();
    }
    ~Launch() { PyEval_RestoreThread(state_); }
    Launch(const Launch &) = delete;
    Launch &operator=(const Launch &) = delete;
    void *stream() const { return s_; }

private:
    c10::cuda::OptionalCUDAGuard guard_;
    void *s_;
    PyThreadState *state_;
};

using Args = PyObject *const *;

pa_status step_plan(Args a) {
    const at::Tensor &counts = tensor_of(a[0], 1, "counts"), &tables = tensor_of(a[2], 2, "block_tables");
    const int dev = device_of(counts);
    const int64_t S = counts.size(0), mb = tables.size(1), N = tensor_of(a[3], 1, "free_blocks").size(0),
                  cap = tensor_of(a[5], 1, "slot_mapping").size(0);
    int32_t *cnt = i32(a[0], {S}, dev, "counts"), *lens = i32(a[1], {S}, dev, "context_lens");
    int32_t *tab = i32(a[2], {S, mb}, dev, "block_tables"), *stack = i32(a[3], {N}, dev, "free_blocks");
    int32_t *height = i32(a[4], {1}, dev, "num_free");
    int64_t *slots = ptr<int64_t>(a[5], at::kLong, {cap}, dev, "slot_mapping");
    int32_t *starts = i32(a[6], {S + 1}, dev, "seq_starts");
    int32_t *new_lens = a[7] == Py_None ? lens : i32(a[7], {S}, dev, "new_context_lens");
    int32_t *new_height = a[8] == Py_None ? height : i32(a[8], {1}, dev, "new_num_free");
    int32_t *err = flag(a[9], dev);
    const Launch on(dev, a[10]);
    return pa_step_plan(cnt, lens, narrow(S, "counts"), tab, narrow(mb, "block_tables"), stack, narrow(N, "free_blocks"),
                        height, slots, narrow(cap, "slot_mapping"), starts, new_lens, new_height, err, on.stream());
}

pa_status step_release(Args a) {
    const at::Tensor &finished = tensor_of(a[0], 1, "finished"), &tables = tensor_of(a[2], 2, "block_tables");
    const int dev = device_of(finished);
    const int64_t S = finished.size(0), mb = tables.size(1), N = tensor_of(a[3], 1, "free_blocks").size(0);
    int32_t *fin = i32(a[0], {S}, dev, "finished"), *lens = i32(a[1], {S}, dev, "context_lens");
    int32_t *tab = i32(a[2], {S, mb}, dev, "block_tables"), *stack = i32(a[3], {N}, dev, "free_blocks");
    int32_t *height = i32(a[4], {1}, dev, "num_free");
    int32_t *new_lens = a[5] == Py_None ? lens : i32(a[5], {S}, dev, "new_context_lens");
    int32_t *new_height = a[6] == Py_None ? height : i32(a[6], {1}, dev, "new_num_free");
    int32_t *err = flag(a[7], dev);
    const Launch on(dev, a[8]);
    return pa_step_release(fin, lens, narrow(S, "finished"), tab, narrow(mb, "block_tables"), stack, narrow(N, "free_blocks"),
                           height, new_lens, new_height, err, on.stream());
}

pa_status cache_write_scaled(Args a) {
    const Pool pool(a[3], a[4], a[5], a[6]);
    const int64_t T = tensor_of(a[0], 3, "key").size(0), h = pool.desc.num_kv_heads, d = pool.desc.head_dim;
    const Rows k(a[0], T, h, d, pool.dev, "key"), v(a[1], T, h, d, pool.dev, "value");
    int64_t *slots = ptr<int64_t>(a[2], at::kLong, {T}, pool.dev, "slot_mapping");
    int32_t *err = flag(a[7], pool.dev);
    const Launch on(pool.dev, a[8]);
    return pa_cache_write_scaled(k.p, v.p, k.stride, v.stride, slots, narrow(T, "key"), pool.kc, pool.vc, pool.ks, pool.vs,
                                 &pool.desc, err, on.stream());
}

pa_status copy_blocks_scaled(Args a) {
    const Pool pool(a[0], a[1], a[2], a[3]);
    const int64_t n = tensor_of(a[4], 2, "src_dst_pairs").size(0);
    int32_t *pairs = i32(a[4], {n, 2}, pool.dev, "src_dst_pairs"), *err = flag(a[5], pool.dev);
    const Launch on(pool.dev, a[6]);
    return pa_copy_blocks_scaled(pool.kc, pool.vc, pool.ks, pool.vs, pairs, narrow(n, "src_dst_pairs"), &pool.desc, err,
                                 on.stream());
}

// query, key_cache, value_cache, key_scales, value_scales, block_tables, context_lens, max_context_len,
// scale, out, workspace, err_flag, stream
pa_status decode_scaled(Args a) {
    const Pool pool(a[1], a[2], a[3], a[4]);
    const at::Tensor &q = tensor_of(a[0], 3, "query");
    const int64_t S = q.size(0), hq = q.size(1), d = pool.desc.head_dim, mb = tensor_of(a[5], 2, "block_tables").size(1);
    void *query = ptr(a[0], at::kBFloat16, {S, hq, d}, pool.dev, "query");
    int32_t *tab = i32(a[5], {S, mb}, pool.dev, "block_tables"), *lens = i32(a[6], {S}, pool.dev, "context_lens");
    void *out = ptr(a[9], at::kBFloat16, {S, hq, d}, pool.dev, "out");
    const Workspace ws(a[10], pool.dev);
    int32_t *err = flag(a[11], pool.dev);
    const int32_t most = integer(a[7], "max_context_len");
    const float scale = number(a[8]);
    const Launch on(pool.dev, a[12]);
    return pa_decode_scaled(query, pool.kc, pool.vc, pool.ks, pool.vs, tab, narrow(mb, "block_tables"), lens, most,
                            narrow(S, "query"), narrow(hq, "query"), scale, ws.p, ws.bytes, out, &pool.desc, err, on.stream());
}

// query, key, value, seq_starts, max_seq_len, scale, out, workspace, err_flag, stream
pa_status prefill_packed(Args a) {
    const at::Tensor &q = tensor_of(a[0], 3, "query");
    const int dev = device_of(q);
    const int64_t T = q.size(0), hq = q.size(1), d = q.size(2), hkv = tensor_of(a[1], 3, "key").size(1),
                  S = tensor_of(a[3], 1, "seq_starts").size(0) - 1;
    const Rows query(a[0], T, hq, d, dev, "query"), k(a[1], T, hkv, d, dev, "key"), v(a[2], T, hkv, d, dev, "value");
    if (S < 0) throw Refused{PyExc_AssertionError, "seq_starts: one more than the sequences wanted"};
    int32_t *starts = i32(a[3], {S + 1}, dev, "seq_starts");
    const int32_t most = integer(a[4], "max_seq_len");
    const float scale = number(a[5]);
    void *out = ptr(a[6], at::kBFloat16, {T, hq, d}, dev, "out");
    const Workspace ws(a[7], dev);
    int32_t *err = flag(a[8], dev);
    const Launch on(dev, a[9]);
    return pa_prefill_packed(query.p, k.p, v.p, query.stride, k.stride, v.stride, starts, narrow(S, "seq_starts"),
                             narrow(T, "query"), most, narrow(hq, "query"), narrow(hkv, "key"), narrow(d, "query"), scale, ws.p,
                             ws.bytes, out, err, on.stream());
}

template <pa_status (*kCall)(Args), int kArgs>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "%d arguments wanted, got %zd", kArgs, n);
        return nullptr;
    }
    try {
        return PyLong_FromLong((long)kCall(args));
    } catch (const Refused &r) {
        if (r.type) PyErr_SetString(r.type, r.what.c_str());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <pa_status (*kCall)(Args), int kArgs>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&entry<kCall, kArgs>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<step_plan, 11>("step_plan"),
                         method<step_release, 9>("step_release"),
                         method<cache_write_scaled, 9>("cache_write_scaled"),
                         method<copy_blocks_scaled, 7>("copy_blocks_scaled"),
                         method<decode_scaled, 13>("decode_scaled"),
                         method<prefill_packed, 10>("prefill_packed"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_step", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step() { return PyModule_Create(&module); }
