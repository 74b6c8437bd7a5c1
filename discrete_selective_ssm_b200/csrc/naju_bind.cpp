// Argument marshalling of the vector-state scan, the 4-bit projections and the
// 8-bit state cache for Python: what the ctypes functions of _native.py do
// (checks, outputs allocated with torch, raw pointers and the current stream
// into the C ABI), compiled, because at a few microseconds a kernel the
// interpreter's share of a call was two to five times the kernel's.  No
// arithmetic, no kernel: the entry points come as addresses from the loaded
// libnaju.so.
#include <ATen/ATen.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <stdexcept>
#include <string>

#include "naju.h"

namespace {

typedef at::IntArrayRef Shape;

PyObject* g_error = nullptr;  // NajuError
decltype(&naju_vscan_workspace_bytes) g_ws_bytes;
decltype(&naju_vscan_fwd) g_vscan_fwd;
decltype(&naju_vscan_bwd) g_vscan_bwd;
decltype(&naju_vscan_step) g_vscan_step;
decltype(&naju_w4_linear) g_w4_linear;
decltype(&naju_state_store) g_state_store;
decltype(&naju_state_load) g_state_load;

struct Raised {};  // a Python exception is set

[[noreturn]] void raise(PyObject* type, const std::string& what) {
    PyErr_SetString(type, what.c_str());
    throw Raised{};
}
void check(naju_status st, const char* where) {
    if (st == NAJU_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", (int)st, where);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

const at::Tensor* opt(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}
const at::Tensor& need(PyObject* o, const char* name) {
    const at::Tensor* t = opt(o, name);
    if (!t) raise(PyExc_TypeError, std::string(name) + " must be a tensor");
    return *t;
}
int device_of(const at::Tensor& t, const char* name) {
    if (!t.is_cuda())
        raise(PyExc_ValueError, std::string(name) + " must be a CUDA tensor, got " + t.device().str());
    return t.get_device();
}
int dtype_of(const at::Tensor& t) {
    if (t.scalar_type() == at::kFloat) return NAJU_F32;
    if (t.scalar_type() == at::kBFloat16) return NAJU_BF16;
    raise(PyExc_TypeError, std::string("unsupported dtype ") + at::toString(t.scalar_type()));
}
at::ScalarType type_of(int code) { return code == NAJU_F32 ? at::kFloat : at::kBFloat16; }

std::string text(Shape s) {
    std::ostringstream o;
    o << s;
    return o.str();
}
// Data pointer of an argument that must be a contiguous `dt` tensor of `shape`
// on CUDA device `dev`.
void* ptr(const at::Tensor& t, const char* name, Shape shape, at::ScalarType dt, int dev) {
    if (!t.is_cuda() || t.get_device() != dev)
        raise(PyExc_ValueError, std::string(name) + " must be a CUDA tensor on device " +
                                    std::to_string(dev) + ", got " + t.device().str());
    if (t.scalar_type() != dt)
        raise(PyExc_TypeError, std::string(name) + " must be " + at::toString(dt) + ", got " +
                                   at::toString(t.scalar_type()));
    if (t.sizes() != shape)
        raise(PyExc_ValueError, std::string(name) + " must have shape " + text(shape) + ", got " +
                                    text(t.sizes()));
    if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
    return t.data_ptr();
}
void* ptr(const at::Tensor* t, const char* name, Shape shape, at::ScalarType dt, int dev) {
    return t ? ptr(*t, name, shape, dt, dev) : nullptr;
}
// The device and stream of a call: the device's current stream unless one is
// given.  A given one is the current one meanwhile, so that what the call
// allocates is that stream's memory (memory of the caller's stream could still
// be in use there, and could be handed out again before the kernel has run).
// Tensors of one stream that the other works on are held by the allocator
// until that work is done, should they be dropped before.
class Call {
public:
    Call(PyObject* given, int dev)
        : guard_((c10::DeviceIndex)dev), caller_(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev)),
          stream_(caller_) {
        if (given == Py_None) return;
        PyObject* h = PyObject_GetAttrString(given, "cuda_stream");
        if (!h) throw Raised{};
        void* s = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (!s && PyErr_Occurred()) throw Raised{};
        if (s == (void*)cudaStreamLegacy) s = nullptr;
        if (s == (void*)caller_.stream()) return;
        stream_ = c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(s), (c10::DeviceIndex)dev);
        on_.reset_stream(stream_);
        other_ = true;
    }
    void* stream() const { return stream_.stream(); }
    // An argument that the kernel reads or writes.
    void uses(const at::Tensor* t) const {
        if (other_ && t && t->defined()) hold(*t, stream_);
    }
    void uses(const at::Tensor& t) const { uses(&t); }
    // A result that the caller takes back: allocated here, or an argument.
    void gives(const at::Tensor& t) const {
        if (!other_ || !t.defined()) return;
        hold(t, stream_);
        hold(t, caller_);
    }

private:
    static void hold(const at::Tensor& t, c10::cuda::CUDAStream s) {
        c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), s);
    }
    c10::cuda::CUDAGuard guard_;
    c10::cuda::OptionalCUDAStreamGuard on_;
    c10::cuda::CUDAStream caller_, stream_;
    bool other_ = false;
};
long long integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v != 0;
}
PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
void arity(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) raise(PyExc_TypeError, "wrong number of arguments");
}

naju_dims vdims(const at::Tensor& h, PyObject* out_dtype) {
    if (h.dim() != 3)
        raise(PyExc_ValueError, "h must be [batch, seqlen, d_inner], got " + text(h.sizes()));
    naju_dims d{};
    d.batch = h.size(0);
    d.seqlen = h.size(1);
    d.d_inner = h.size(2);
    d.d_state = 1;
    d.dtype = dtype_of(h);
    d.out_dtype = out_dtype == Py_None ? d.dtype : (int32_t)integer(out_dtype);
    return d;
}
at::Tensor workspace(const naju_dims& d, const at::Tensor& like) {
    const size_t n = g_ws_bytes(&d);
    if (n == 0) check(NAJU_ERR_INVALID_ARG, "naju_vscan_workspace_bytes");
    at::Tensor ws = at::empty({(int64_t)n}, like.options().dtype(at::kByte));
    const uintptr_t off = -(uintptr_t)ws.data_ptr() & 255;
    if (off) {  // (an allocator that aligns less than CUDA's)
        ws = at::empty({(int64_t)n + 256}, like.options().dtype(at::kByte));
        ws = ws.narrow(0, (int64_t)(-(uintptr_t)ws.data_ptr() & 255), (int64_t)n);
    }
    return ws;
}
void* ws_ptr(const at::Tensor& ws, int dev) {
    if (ws.scalar_type() != at::kByte || !ws.is_cuda() || ws.get_device() != dev ||
        !ws.is_contiguous())
        raise(PyExc_ValueError, "workspace must be a contiguous uint8 tensor on CUDA device " +
                                    std::to_string(dev));
    return ws.data_ptr();
}

// h, a, b, z, x0, out_dtype, workspace, want_final, y, x_final, stream
PyObject* vscan_fwd(PyObject* const* v, Py_ssize_t n) {
    arity(n, 11);
    const at::Tensor& h = need(v[0], "h");
    const naju_dims d = vdims(h, v[5]);
    const int dev = device_of(h, "h");
    const at::ScalarType dt = h.scalar_type(), ot = type_of(d.out_dtype);
    const Shape act = h.sizes();
    const int64_t st[2] = {d.batch, d.d_inner};
    const at::Tensor &a = need(v[1], "a"), *b = opt(v[2], "b"), *z = opt(v[3], "z"),
                     *x0 = opt(v[4], "x0"), *ws0 = opt(v[6], "workspace"), *y0 = opt(v[8], "y"),
                     *xf0 = opt(v[9], "x_final");
    const Call call(v[10], dev);
    void *ph = ptr(h, "h", act, dt, dev), *pa = ptr(a, "a", act, dt, dev),
         *pb = ptr(b, "b", act, dt, dev), *pz = ptr(z, "z", act, dt, dev);
    void* px0 = ptr(x0, "x0", st, at::kFloat, dev);
    const at::Tensor ws = ws0 ? *ws0 : workspace(d, h);
    const at::Tensor y = y0 ? *y0 : at::empty(act, h.options().dtype(ot));
    const bool final = xf0 || truth(v[7]);
    const at::Tensor xf = xf0 ? *xf0 : final ? at::empty(st, h.options().dtype(at::kFloat)) : at::Tensor();
    check(g_vscan_fwd(&d, ph, pa, pb, pz, static_cast<float*>(px0), ptr(y, "y", act, ot, dev),
                      final ? static_cast<float*>(ptr(xf, "x_final", st, at::kFloat, dev)) : nullptr,
                      ws_ptr(ws, dev), (size_t)ws.numel(), call.stream()),
          "naju_vscan_fwd");
    for (const at::Tensor* t : {&h, &a, b, z, x0}) call.uses(t);
    for (const at::Tensor* t : {&ws, &y, &xf}) call.gives(*t);
    PyObject* xo = final ? wrap(xf) : Py_NewRef(Py_None);
    return Py_BuildValue("(NNN)", wrap(y), xo, wrap(ws));
}

// dy, h, a, b, workspace, z, dx_final, out_dtype, want_dx0, grads (dict or None), stream
PyObject* vscan_bwd(PyObject* const* v, Py_ssize_t n) {
    arity(n, 11);
    const at::Tensor& h = need(v[1], "h");
    const naju_dims d = vdims(h, v[7]);
    const int dev = device_of(h, "h");
    const at::ScalarType dt = h.scalar_type(), ot = type_of(d.out_dtype);
    const Shape act = h.sizes();
    const int64_t st[2] = {d.batch, d.d_inner};
    const at::Tensor &dy = need(v[0], "dy"), &a = need(v[2], "a"), *b = opt(v[3], "b"),
                     &ws = need(v[4], "workspace"), *z = opt(v[5], "z"),
                     *dxf = opt(v[6], "dx_final");
    const Call call(v[10], dev);
    void *ph = ptr(h, "h", act, dt, dev), *pa = ptr(a, "a", act, dt, dev),
         *pb = ptr(b, "b", act, dt, dev), *pz = ptr(z, "z", act, dt, dev),
         *pdy = ptr(dy, "dy", act, dt, dev);
    void* pdxf = ptr(dxf, "dx_final", st, at::kFloat, dev);
    static const char* names[5] = {"dh", "da", "db", "dz", "dx0"};
    PyObject* grads = v[9];
    at::Tensor g[5];
    const bool own = grads == Py_None;
    for (int i = 0; i < 5; ++i) {
        if (own) {
            const bool want = i < 2 || (i == 2 && b) || (i == 3 && z) ||
                              (i == 4 && truth(v[8]));
            if (!want) continue;
            g[i] = i == 4 ? at::empty(st, h.options().dtype(at::kFloat))
                          : at::empty(act, h.options().dtype(ot));
        } else {
            PyObject* o = PyDict_GetItemString(grads, names[i]);
            const at::Tensor* t = o ? opt(o, names[i]) : nullptr;
            if (t) g[i] = *t;
        }
    }
    const auto out = [&](int i) {
        if (!g[i].defined()) return (void*)nullptr;
        return i == 4 ? ptr(g[i], names[i], st, at::kFloat, dev) : ptr(g[i], names[i], act, ot, dev);
    };
    check(g_vscan_bwd(&d, ph, pa, pb, pz, pdy, static_cast<float*>(pdxf), out(0), out(1), out(2),
                      out(3), static_cast<float*>(out(4)), ws_ptr(ws, dev), (size_t)ws.numel(),
                      call.stream()),
          "naju_vscan_bwd");
    for (const at::Tensor* t : {&h, &a, b, z, &dy, dxf, &ws}) call.uses(t);
    for (const at::Tensor& t : g) call.gives(t);
    if (!own) return Py_NewRef(grads);
    PyObject* r = PyDict_New();
    if (!r) throw Raised{};
    for (int i = 0; i < 5; ++i) {
        PyObject* o = g[i].defined() ? wrap(g[i]) : Py_NewRef(Py_None);
        PyDict_SetItemString(r, names[i], o);
        Py_DECREF(o);
    }
    return r;
}

// state, h, a, b, z, y, stream
PyObject* vscan_step(PyObject* const* v, Py_ssize_t n) {
    arity(n, 7);
    const at::Tensor &state = need(v[0], "state"), &h = need(v[1], "h"), &a = need(v[2], "a"),
                     *b = opt(v[3], "b"), *z = opt(v[4], "z"), *y0 = opt(v[5], "y");
    const Shape sh = h.sizes();
    if (sh.size() != 2) raise(PyExc_ValueError, "h must be [batch, d_inner], got " + text(sh));
    const int dev = device_of(h, "h"), code = dtype_of(h);
    const at::ScalarType dt = h.scalar_type();
    const Call call(v[6], dev);
    const at::Tensor y = y0 ? *y0 : at::empty(sh, h.options());
    check(g_vscan_step(sh[0], sh[1], code, ptr(h, "h", sh, dt, dev), ptr(a, "a", sh, dt, dev),
                       ptr(b, "b", sh, dt, dev), ptr(z, "z", sh, dt, dev),
                       static_cast<float*>(ptr(state, "state", sh, at::kFloat, dev)),
                       ptr(y, "y", sh, dt, dev), call.stream()),
          "naju_vscan_step");
    for (const at::Tensor* t : {&state, &h, &a, b, z}) call.uses(t);
    call.gives(y);
    return wrap(y);
}

// x, wq, scales, group, bias, residual, y, stream
PyObject* w4_linear(PyObject* const* v, Py_ssize_t n) {
    arity(n, 8);
    const at::Tensor &x = need(v[0], "x"), &wq = need(v[1], "wq"), &sc = need(v[2], "scales"),
                     *bias = opt(v[4], "bias"), *res = opt(v[5], "residual"), *y0 = opt(v[6], "y");
    const long long group = integer(v[3]);
    if (group != 32 && group != 64 && group != 128)
        check(NAJU_ERR_UNSUPPORTED, "4-bit projection with this group size");
    if (x.dim() < 1 || wq.dim() != 2)
        raise(PyExc_ValueError, "x must have at least one and wq two dimensions");
    const int dev = device_of(x, "x"), code = dtype_of(x);
    const at::ScalarType dt = x.scalar_type();
    const int64_t K = x.size(-1), O = wq.size(0), m = K ? x.numel() / K : 0;
    c10::DimVector out(x.sizes().begin(), x.sizes().end());
    out.back() = O;
    const int64_t ws[2] = {O, (K + 127) / 128 * 64}, ss[2] = {O, (K + group - 1) / group}, bs[1] = {O};
    const Call call(v[7], dev);
    void *px = ptr(x, "x", x.sizes(), dt, dev), *pw = ptr(wq, "wq", ws, at::kByte, dev),
         *ps = ptr(sc, "scales", ss, at::kBFloat16, dev);
    void *pb = ptr(bias, "bias", bs, at::kFloat, dev), *pr = ptr(res, "residual", out, dt, dev);
    const at::Tensor y = y0 ? *y0 : at::empty(out, x.options());
    check(g_w4_linear(m, K, O, (int32_t)group, code, px, pw, ps, static_cast<float*>(pb), pr,
                      ptr(y, "y", out, dt, dev), call.stream()),
          "naju_w4_linear");
    for (const at::Tensor* t : {&x, &wq, &sc, bias, res}) call.uses(t);
    call.gives(y);
    return wrap(y);
}

struct Cache {
    int64_t shape[3], n, slots;
    int dev;
    int8_t* q;
    float* scale;
    int32_t* at;
    const at::Tensor* given[3];  // the pool's two tensors and the slots
};
Cache cache_args(PyObject* pool_q, PyObject* pool_scale, PyObject* slots) {
    const at::Tensor &q = need(pool_q, "pool_q"), &sc = need(pool_scale, "pool_scale"),
                     &sl = need(slots, "slots");
    if (q.dim() != 3)
        raise(PyExc_ValueError, "pool_q must be [n_slots, d_inner, d_state], got " + text(q.sizes()));
    if (sl.dim() != 1) raise(PyExc_ValueError, "slots must be [n], got " + text(sl.sizes()));
    Cache c;
    c.dev = device_of(q, "pool_q");
    c.n = sl.size(0);
    c.slots = q.size(0);
    c.shape[0] = c.n;
    c.shape[1] = q.size(1);
    c.shape[2] = q.size(2);
    const int64_t ss[2] = {q.size(0), q.size(1)}, ls[1] = {c.n};
    c.q = static_cast<int8_t*>(ptr(q, "pool_q", q.sizes(), at::kChar, c.dev));
    c.scale = static_cast<float*>(ptr(sc, "pool_scale", ss, at::kFloat, c.dev));
    c.at = static_cast<int32_t*>(ptr(sl, "slots", ls, at::kInt, c.dev));
    c.given[0] = &q;
    c.given[1] = &sc;
    c.given[2] = &sl;
    return c;
}

// state, slots, pool_q, pool_scale, stream
PyObject* state_store(PyObject* const* v, Py_ssize_t n) {
    arity(n, 5);
    const at::Tensor& state = need(v[0], "state");
    const Cache c = cache_args(v[2], v[3], v[1]);
    const Call call(v[4], c.dev);
    check(g_state_store(c.n, c.shape[1], c.shape[2], c.slots,
                        static_cast<float*>(ptr(state, "state", Shape(c.shape, 3), at::kFloat, c.dev)),
                        c.at, c.q, c.scale, call.stream()),
          "naju_state_store");
    call.uses(state);
    for (const at::Tensor* t : c.given) call.uses(t);
    Py_RETURN_NONE;
}

// pool_q, pool_scale, slots, state, stream
PyObject* state_load(PyObject* const* v, Py_ssize_t n) {
    arity(n, 5);
    const Cache c = cache_args(v[0], v[1], v[2]);
    const at::Tensor* s0 = opt(v[3], "state");
    const Call call(v[4], c.dev);
    const at::Tensor state = s0 ? *s0
                                : at::empty(Shape(c.shape, 3),
                                            need(v[1], "pool_scale").options());
    check(g_state_load(c.n, c.shape[1], c.shape[2], c.slots, c.q, c.scale, c.at,
                       static_cast<float*>(ptr(state, "state", Shape(c.shape, 3), at::kFloat, c.dev)),
                       call.stream()),
          "naju_state_load");
    for (const at::Tensor* t : c.given) call.uses(t);
    call.gives(state);
    return s0 ? Py_NewRef(v[3]) : wrap(state);
}

// NajuError, then the addresses of the C ABI's functions in the order below
PyObject* bind(PyObject* const* v, Py_ssize_t n) {
    arity(n, 8);
    void* f[7];
    for (int i = 0; i < 7; ++i) {
        f[i] = PyLong_AsVoidPtr(v[i + 1]);
        if (!f[i]) raise(PyExc_ValueError, "null entry point");
    }
    g_ws_bytes = reinterpret_cast<decltype(g_ws_bytes)>(f[0]);
    g_vscan_fwd = reinterpret_cast<decltype(g_vscan_fwd)>(f[1]);
    g_vscan_bwd = reinterpret_cast<decltype(g_vscan_bwd)>(f[2]);
    g_vscan_step = reinterpret_cast<decltype(g_vscan_step)>(f[3]);
    g_w4_linear = reinterpret_cast<decltype(g_w4_linear)>(f[4]);
    g_state_store = reinterpret_cast<decltype(g_state_store)>(f[5]);
    g_state_load = reinterpret_cast<decltype(g_state_load)>(f[6]);
    Py_XDECREF(g_error);
    g_error = Py_NewRef(v[0]);
    Py_RETURN_NONE;
}

// No C++ exception leaves a function that Python calls.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* v, Py_ssize_t n) {
    try {
        return F(v, n);
    } catch (const Raised&) {
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* type = nullptr;
        if (PyObject* torch = PyImport_ImportModule("torch")) {
            type = PyObject_GetAttrString(torch, "OutOfMemoryError");
            Py_DECREF(torch);
        }
        PyErr_SetString(type ? type : PyExc_RuntimeError, e.what_without_backtrace());
        Py_XDECREF(type);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define NAJU_METHOD(f) \
    {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<f>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {NAJU_METHOD(bind),        NAJU_METHOD(vscan_fwd),  NAJU_METHOD(vscan_bwd),
                         NAJU_METHOD(vscan_step),  NAJU_METHOD(w4_linear),  NAJU_METHOD(state_store),
                         NAJU_METHOD(state_load),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_naju_bind", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__naju_bind(void) { return PyModule_Create(&module); }
