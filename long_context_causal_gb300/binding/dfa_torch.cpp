// dfa_torch.cpp -- the calls whose latency counts, marshalled in C++.
//
// A short windowed-attention or checkpoint call runs for a few microseconds on
// the GPU, and reading a tensor's sizes, checking it and allocating outputs
// from Python costs several times that (a decode step: 20 us in Python, 8 here).
// These functions do for the calls of include/dfa.h what dfa.py does for the
// others: check the tensors, allocate what the caller did not give, and hand
// pointers and the stream to the library.  No arithmetic.  The library's entry
// points come from bind(), so both sides use the same libdfa.so.
//
// Each returns its tensors, or the library's status as an int where that is
// not DFA_OK; bad tensors raise ValueError or TypeError here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <string>

#include "../../include/dfa.h"

namespace {

struct Entry {
    decltype(&dfa_attn_fwd_sink) fwd;
    decltype(&dfa_attn_bwd_sink) bwd;
    decltype(&dfa_attn_bwd_sink_workspace_size) bwd_bytes;
    decltype(&dfa_attn_decode_sink) decode;
    decltype(&dfa_attn_decode_sink_workspace_size) decode_bytes;
    decltype(&dfa_ckpt8_save) save;
    decltype(&dfa_ckpt8_restore) restore;
    decltype(&dfa_ckpt8_size) ckpt_bytes;
    decltype(&dfa_attn_bwd_ckpt8) bwd_ckpt;
    decltype(&dfa_attn_bwd_ckpt8_workspace_size) bwd_ckpt_bytes;
} g;

struct ValueErr {
    std::string what;
};
struct TypeErr {
    std::string what;
};
struct Raised {};   // a Python error is set

// The library call and the allocations may block (a full launch queue, a
// cudaMalloc): other Python threads run meanwhile, as with ctypes.
struct NoGil {
    PyThreadState* save = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(save); }
};
template <typename F, typename... A>
dfa_status without_gil(F entry, A... args) {
    const NoGil released;
    return entry(args...);
}

std::string shape_of(const at::Tensor& t) {
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw TypeErr{std::string(name) + " must be a tensor"};
    return THPVariable_Unpack(o);
}

int number(PyObject* o, const char* name) {
    const long x = PyLong_AsLong(o);
    if (x == -1 && PyErr_Occurred()) throw Raised{};
    if (x < INT_MIN || x > INT_MAX) throw ValueErr{std::string(name) + " does not fit a 32-bit integer"};
    return (int)x;
}

// None: 1 / sqrt(D).
float scale_of(PyObject* o, int64_t D) {
    if (o == Py_None) return (float)(1.0 / std::sqrt((double)D));
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Raised{};
    return (float)x;
}

dfa_dtype dtype_of(const at::Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return DFA_BF16;
    if (t.scalar_type() == at::kFloat) return DFA_F32;
    throw TypeErr{std::string("unsupported dtype ") + c10::toString(t.scalar_type()) + " (float32 or bfloat16)"};
}

// Every tensor lies on the current CUDA device: the library launches there, on
// the pointers it is given.
int on_gpu(std::initializer_list<const at::Tensor*> ts) {
    const int now = (*ts.begin())->is_cuda() ? (int)c10::cuda::current_device() : -1;
    for (const at::Tensor* t : ts)
        if (!t->is_cuda() || t->get_device() != (*ts.begin())->get_device())
            throw ValueErr{"the tensors must be CUDA tensors on one device, got one on " + t->device().str()};
    if ((*ts.begin())->get_device() != now)
        throw ValueErr{"the tensors are on " + (*ts.begin())->device().str() + ", the current device is cuda:" + std::to_string(now)};
    return now;
}

// A tensor the caller hands over must be dense and of exactly this shape, type
// and device: a smaller one would be written past its end.
at::Tensor given(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, const at::Device& dev) {
    const at::Tensor& t = tensor(o, name);
    if (!t.is_contiguous()) throw ValueErr{std::string(name) + " must be contiguous (BSHD dense)"};
    if (t.sizes() != shape || t.scalar_type() != type || t.device() != dev) {
        std::string want = "(";
        for (size_t i = 0; i < shape.size(); ++i) want += (i ? ", " : "") + std::to_string(shape[i]);
        throw ValueErr{std::string(name) + " must be a " + c10::toString(type) + " tensor of shape " + want + ") on " +
                       dev.str() + ", got " + c10::toString(t.scalar_type()) + " " + shape_of(t) + " on " + t.device().str()};
    }
    return t;
}

struct Stream {
    void* handle;
    bool other;      // not the current one
};
Stream stream_of(PyObject* o, int dev) {
    void* const now = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    if (o == Py_None) return Stream{now, false};
    PyObject* n = nullptr;
    if (PyLong_Check(o)) {
        n = o;
        Py_INCREF(n);
    } else {
        n = PyObject_GetAttrString(o, "cuda_stream");
        if (!n) throw Raised{};
    }
    void* h = PyLong_AsVoidPtr(n);
    Py_DECREF(n);
    if (PyErr_Occurred()) throw Raised{};
    return Stream{h, h != now};
}

c10::cuda::CUDAStream torch_stream(const Stream& s, const at::Device& dev) {
    return c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(s.handle), dev.index());
}

// A new tensor is owned by the stream the call runs on: the allocator hands out
// its memory again only behind the call's kernels, and took it from no work that
// another stream has still to do.
at::Tensor allocate(at::IntArrayRef shape, at::ScalarType type, const at::Device& dev, const Stream& s) {
    const auto opt = at::TensorOptions().dtype(type).device(dev);
    const NoGil released;
    if (!s.other) return at::empty(shape, opt);
    c10::cuda::CUDAStreamGuard guard(torch_stream(s, dev));
    return at::empty(shape, opt);
}

// An output made here is the caller's, who uses it on the current stream: that
// is waited for as well before its memory is handed out again.
at::Tensor result(at::IntArrayRef shape, at::ScalarType type, const at::Device& dev, const Stream& s) {
    at::Tensor t = allocate(shape, type, dev, s);
    if (s.other) t.record_stream(c10::cuda::getCurrentCUDAStream(dev.index()));
    return t;
}
at::Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, const at::Device& dev,
                  const Stream& s) {
    return o == Py_None ? result(shape, type, dev, s) : given(o, name, shape, type, dev);
}

// The caller may drop a tensor as soon as the call returns, and another stream
// than its own may still use it then.
void hold(const Stream& s, std::initializer_list<const at::Tensor*> ts) {
    if (!s.other) return;
    for (const at::Tensor* t : ts) t->record_stream(torch_stream(s, t->device()));
}

// A caller's byte buffer, or one for this call.
at::Tensor bytes(PyObject* o, const char* name, size_t n, const at::Device& dev, const Stream& s) {
    if (o != Py_None) {
        const at::Tensor& t = tensor(o, name);
        if (t.scalar_type() != at::kByte || !t.is_contiguous() || t.device() != dev)
            throw ValueErr{std::string(name) + " must be a contiguous uint8 tensor on " + dev.str()};
        return t;
    }
    return allocate({n ? (int64_t)n : 16}, at::kByte, dev, s);
}

struct Sequence {
    int B, S, H, Hkv, D;
};
int small(int64_t x) {
    if (x > INT_MAX) throw ValueErr{"tensor size does not fit a 32-bit integer"};
    return (int)x;
}
Sequence sequence(const at::Tensor& q, const at::Tensor& k, const at::Tensor& v) {
    if (q.dim() != 4 || k.dim() != 4 || k.sizes() != v.sizes() || k.size(0) != q.size(0) || k.size(1) != q.size(1) ||
        k.size(3) != q.size(3))
        throw ValueErr{"q must be [B, S, H, D] and k, v [B, S, H_kv, D], got " + shape_of(q) + ", " + shape_of(k) + ", " +
                       shape_of(v)};
    if (k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type())
        throw ValueErr{"q, k and v must have the same dtype"};
    if (!q.is_contiguous() || !k.is_contiguous() || !v.is_contiguous())
        throw ValueErr{"q, k and v must be contiguous (BSHD dense)"};
    return Sequence{small(q.size(0)), small(q.size(1)), small(q.size(2)), small(k.size(2)), small(q.size(3))};
}

PyObject* pack(std::initializer_list<at::Tensor> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) throw Raised{};
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
    return r;
}

// ---------------------------------------------------------------- the calls
PyObject* fwd(PyObject* const* a) {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const Sequence z = sequence(q, k, v);
    const int d = on_gpu({&q, &k, &v});
    const at::Device dev = q.device();
    const Stream s = stream_of(a[8], d);
    at::Tensor O = output(a[6], "O", q.sizes(), q.scalar_type(), dev, s);
    at::Tensor lse = output(a[7], "lse", {z.B, z.H, z.S}, at::kFloat, dev, s);
    hold(s, {&q, &k, &v, &O, &lse});
    const int window = number(a[3], "window"), n_sink = number(a[4], "n_sink");
    const dfa_status st = without_gil(g.fwd, q.data_ptr(), k.data_ptr(), v.data_ptr(), dtype_of(q), z.B, z.H, z.Hkv, z.S,
                                      z.D, window, n_sink, scale_of(a[5], z.D), O.data_ptr(),
                                      static_cast<float*>(lse.data_ptr()), s.handle);
    return st ? PyLong_FromLong(st) : pack({std::move(O), std::move(lse)});
}

PyObject* bwd(PyObject* const* a) {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const Sequence z = sequence(q, k, v);
    const int d = on_gpu({&q, &k, &v});
    const at::Device dev = q.device();
    const auto type = q.scalar_type();
    const at::Tensor O = given(a[3], "O", q.sizes(), type, dev);
    const at::Tensor lse = given(a[4], "lse", {z.B, z.H, z.S}, at::kFloat, dev);
    const at::Tensor dO = given(a[5], "dO", q.sizes(), type, dev);
    const int window = number(a[6], "window"), n_sink = number(a[7], "n_sink");
    const Stream s = stream_of(a[13], d);
    at::Tensor dQ = output(a[9], "dQ", q.sizes(), type, dev, s);
    at::Tensor dK = output(a[10], "dK", k.sizes(), type, dev, s);
    at::Tensor dV = output(a[11], "dV", k.sizes(), type, dev, s);
    const at::Tensor ws = bytes(a[12], "workspace_buf",
                                a[12] == Py_None ? g.bwd_bytes(z.B, z.H, z.Hkv, z.S, z.D, window, n_sink) : 0, dev, s);
    hold(s, {&q, &k, &v, &O, &lse, &dO, &dQ, &dK, &dV, &ws});
    const dfa_status st = without_gil(g.bwd, q.data_ptr(), k.data_ptr(), v.data_ptr(), O.data_ptr(),
                                      static_cast<const float*>(lse.data_ptr()), dO.data_ptr(), dtype_of(q), z.B, z.H,
                                      z.Hkv, z.S, z.D, window, n_sink, scale_of(a[8], z.D), dQ.data_ptr(), dK.data_ptr(),
                                      dV.data_ptr(), ws.data_ptr(), (size_t)ws.numel(), s.handle);
    return st ? PyLong_FromLong(st) : pack({std::move(dQ), std::move(dK), std::move(dV)});
}

PyObject* decode(PyObject* const* a) {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    if (q.dim() != 3 || k.dim() != 4 || k.sizes() != v.sizes() || k.size(0) != q.size(0) || k.size(3) != q.size(2))
        throw ValueErr{"q must be [B, H, D] and k, v [B, S_max, H_kv, D], got " + shape_of(q) + ", " + shape_of(k) + ", " +
                       shape_of(v)};
    if (k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type())
        throw ValueErr{"q, k and v must have the same dtype"};
    if (k.strides() != v.strides() || k.stride(3) != 1)
        throw ValueErr{"k and v must share their strides, with the head dimension contiguous"};
    if (!q.is_contiguous()) throw ValueErr{"q must be contiguous ([B, H, D] dense)"};
    const int d = on_gpu({&q, &k, &v});
    const at::Device dev = q.device();
    const int B = small(q.size(0)), H = small(q.size(1)), D = small(q.size(2)), S = small(k.size(1)), Hkv = small(k.size(2));
    const at::Tensor len = given(a[3], "kv_len", {B}, at::kInt, dev);
    const Stream s = stream_of(a[10], d);
    at::Tensor O = output(a[7], "O", q.sizes(), q.scalar_type(), dev, s);
    at::Tensor lse = output(a[8], "lse", {B, H}, at::kFloat, dev, s);
    const at::Tensor ws = bytes(a[9], "workspace_buf", a[9] == Py_None ? g.decode_bytes(B, H, Hkv, D) : 0, dev, s);
    hold(s, {&q, &k, &v, &len, &O, &lse, &ws});
    const int64_t strides[3] = {k.stride(0), k.stride(1), k.stride(2)};
    const dfa_status st = without_gil(g.decode, q.data_ptr(), k.data_ptr(), v.data_ptr(), dtype_of(q), B, H, Hkv, S, D,
                                      static_cast<const int64_t*>(strides), static_cast<const int32_t*>(len.data_ptr()),
                                      number(a[4], "window"), number(a[5], "n_sink"), scale_of(a[6], D), O.data_ptr(),
                                      static_cast<float*>(lse.data_ptr()), ws.data_ptr(), (size_t)ws.numel(), s.handle);
    return st ? PyLong_FromLong(st) : pack({std::move(O), std::move(lse)});
}

PyObject* save(PyObject* const* a) {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const Sequence z = sequence(q, k, v);
    const int d = on_gpu({&q, &k, &v});
    const at::Device dev = q.device();
    const at::Tensor O = given(a[3], "O", q.sizes(), q.scalar_type(), dev);
    const Stream s = stream_of(a[5], d);
    at::Tensor ckpt = a[4] == Py_None ? result({(int64_t)g.ckpt_bytes(z.B, z.H, z.Hkv, z.S, z.D)}, at::kByte, dev, s)
                                      : bytes(a[4], "ckpt", 0, dev, s);
    hold(s, {&q, &k, &v, &O, &ckpt});
    const dfa_status st = without_gil(g.save, q.data_ptr(), k.data_ptr(), v.data_ptr(), O.data_ptr(), dtype_of(q), z.B, z.H,
                                      z.Hkv, z.S, z.D, ckpt.data_ptr(), (size_t)ckpt.numel(), s.handle);
    return st ? PyLong_FromLong(st) : THPVariable_Wrap(std::move(ckpt));
}

PyObject* restore(PyObject* const* a) {
    const at::Tensor& given_ckpt = tensor(a[0], "ckpt");
    const int d = on_gpu({&given_ckpt});
    const at::Device dev = given_ckpt.device();
    const Stream s = stream_of(a[10], d);
    const at::Tensor ckpt = bytes(a[0], "ckpt", 0, dev, s);
    const int B = number(a[1], "B"), H = number(a[2], "H"), Hkv = number(a[3], "H_kv"), S = number(a[4], "S"),
              D = number(a[5], "D");
    if (B < 0 || H < 0 || Hkv < 0 || S < 0 || D < 0) throw ValueErr{"sizes must not be negative"};
    at::Tensor q = output(a[6], "q", {B, S, H, D}, at::kBFloat16, dev, s);
    at::Tensor k = output(a[7], "k", {B, S, Hkv, D}, at::kBFloat16, dev, s);
    at::Tensor v = output(a[8], "v", {B, S, Hkv, D}, at::kBFloat16, dev, s);
    at::Tensor O = output(a[9], "O", {B, S, H, D}, at::kBFloat16, dev, s);
    hold(s, {&ckpt, &q, &k, &v, &O});
    const dfa_status st = without_gil(g.restore, ckpt.data_ptr(), (size_t)ckpt.numel(), DFA_BF16, B, H, Hkv, S, D,
                                      q.data_ptr(), k.data_ptr(), v.data_ptr(), O.data_ptr(), s.handle);
    return st ? PyLong_FromLong(st) : pack({std::move(q), std::move(k), std::move(v), std::move(O)});
}

PyObject* bwd_ckpt(PyObject* const* a) {
    const at::Tensor &ck = tensor(a[0], "ckpt"), &dO = tensor(a[2], "dO");
    if (dO.dim() != 4 || !dO.is_contiguous())
        throw ValueErr{"dO must be a contiguous [B, S, H, D] tensor, got " + shape_of(dO)};
    const int d = on_gpu({&dO, &ck});
    const at::Device dev = dO.device();
    const Stream s = stream_of(a[11], d);
    const at::Tensor ckpt = bytes(a[0], "ckpt", 0, dev, s);
    const int B = small(dO.size(0)), S = small(dO.size(1)), H = small(dO.size(2)), D = small(dO.size(3));
    const int Hkv = number(a[3], "H_kv");
    if (Hkv < 0) throw ValueErr{"H_kv must not be negative"};
    const at::Tensor lse = given(a[1], "lse", {B, H, S}, at::kFloat, dev);
    const int window = a[4] == Py_None ? std::max(S, 1) : number(a[4], "window"), n_sink = number(a[5], "n_sink");
    at::Tensor dQ = output(a[7], "dQ", dO.sizes(), dO.scalar_type(), dev, s);
    at::Tensor dK = output(a[8], "dK", {B, S, Hkv, D}, dO.scalar_type(), dev, s);
    at::Tensor dV = output(a[9], "dV", {B, S, Hkv, D}, dO.scalar_type(), dev, s);
    const at::Tensor ws = bytes(a[10], "workspace_buf",
                                a[10] == Py_None ? g.bwd_ckpt_bytes(B, H, Hkv, S, D, window, n_sink) : 0, dev, s);
    hold(s, {&ckpt, &lse, &dO, &dQ, &dK, &dV, &ws});
    const dfa_status st = without_gil(g.bwd_ckpt, ckpt.data_ptr(), (size_t)ckpt.numel(),
                                      static_cast<const float*>(lse.data_ptr()), dO.data_ptr(), dtype_of(dO), B, H, Hkv, S, D,
                                      window, n_sink, scale_of(a[6], D), dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(),
                                      ws.data_ptr(), (size_t)ws.numel(), s.handle);
    return st ? PyLong_FromLong(st) : pack({std::move(dQ), std::move(dK), std::move(dV)});
}

// ---------------------------------------------------------------- module
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    HANDLE_TH_ERRORS
    at::AutoDispatchBelowAutograd no_autograd;
    try {
        return F(a);
    } catch (const ValueErr& e) {
        PyErr_SetString(PyExc_ValueError, e.what.c_str());
    } catch (const TypeErr& e) {
        PyErr_SetString(PyExc_TypeError, e.what.c_str());
    } catch (const Raised&) {
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

// bind(address of each entry point, in the order of Entry)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* p[10];
    if (n != 10) {
        PyErr_SetString(PyExc_TypeError, "bind takes ten addresses");
        return nullptr;
    }
    for (int i = 0; i < 10; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null entry point");
            return nullptr;
        }
    }
    static_assert(sizeof(Entry) == sizeof(p), "one pointer each");
    memcpy(&g, p, sizeof(p));
    Py_RETURN_NONE;
}

#define FAST(f) (PyCFunction)(void (*)(void))(f), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"bind", FAST(bind)},
                         {"fwd_sink", FAST((call<fwd, 9>))},
                         {"bwd_sink", FAST((call<bwd, 14>))},
                         {"decode_sink", FAST((call<decode, 11>))},
                         {"ckpt8_save", FAST((call<save, 6>))},
                         {"ckpt8_restore", FAST((call<restore, 11>))},
                         {"bwd_ckpt8", FAST((call<bwd_ckpt, 12>))},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dfa_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dfa_torch() { return PyModule_Create(&module); }
