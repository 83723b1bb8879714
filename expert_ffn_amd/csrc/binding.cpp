// Python binding of the operators around the expert FFN (the module
// expert_ffn_amd._binding; expert_ffn_amd re-exports its functions).
//
// Argument marshalling only, as the ctypes binding of the other entry points: it
// checks shapes, types and devices, passes pointers, sizes and torch's current
// stream to the C entry point of the same name, and raises MoeError on a non-OK
// status.  It is compiled because these calls are short: in a decode step they
// run kernels of 3 to 7 us, and ctypes with the same checks in Python took 6.6 us
// of host time for a norm and 10.9 for the end of a block, where a launch alone
// takes 3.
#include <Python.h>

#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>
#include <exception>

#include "../../include/expert_ffn.h"

namespace {

struct Raised {};   // a Python exception is set

[[noreturn]] void raise(PyObject* type, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    PyErr_FormatV(type, fmt, ap);
    va_end(ap);
    throw Raised{};
}

// "(2, 64)" of a tensor's sizes
std::string sizes(const at::Tensor& t) {
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + (t.dim() == 1 ? ",)" : ")");
}

// Arguments of one call, in the order of the names (null where not given).
constexpr int MAX_ARGS = 20;
struct Signature {
    const char* fn;
    int n, required;
    const char* names[MAX_ARGS];
    PyObject* interned[MAX_ARGS];
};

void take(Signature& S, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames, PyObject** out) {
    if (nargs > S.n) raise(PyExc_TypeError, "%s() takes %d arguments, %zd were given", S.fn, S.n, nargs);
    for (int i = 0; i < S.n; ++i) out[i] = i < nargs ? args[i] : nullptr;
    const Py_ssize_t nkw = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    for (Py_ssize_t k = 0; k < nkw; ++k) {
        PyObject* name = PyTuple_GET_ITEM(kwnames, k);
        int at = -1;
        for (int i = 0; i < S.n && at < 0; ++i)
            if (S.interned[i] == name) at = i;
        for (int i = 0; i < S.n && at < 0; ++i)
            if (PyUnicode_Compare(S.interned[i], name) == 0) at = i;
        if (at < 0) raise(PyExc_TypeError, "%s() got an unexpected keyword argument '%U'", S.fn, name);
        if (out[at]) raise(PyExc_TypeError, "%s() got multiple values for argument '%s'", S.fn, S.names[at]);
        out[at] = args[nargs + k];
    }
    for (int i = 0; i < S.required; ++i)
        if (!out[i]) raise(PyExc_TypeError, "%s() is missing its argument '%s'", S.fn, S.names[i]);
}

bool given(PyObject* o) { return o && o != Py_None; }

int32_t to_int(PyObject* o, const char* name, int32_t def) {
    if (!o) return def;
    PyObject* i = PyNumber_Index(o);
    if (!i) throw Raised{};
    const long v = PyLong_AsLong(i);
    Py_DECREF(i);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v < INT32_MIN || v > INT32_MAX) raise(PyExc_OverflowError, "%s does not fit 32 bits", name);
    return static_cast<int32_t>(v);
}
float to_float(PyObject* o, float def) {
    if (!o) return def;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return static_cast<float>(v);
}

// type codes: the public ones, and those of whole numbers
enum Kind { ANY = -1, F32 = MOE_F32, BF16 = MOE_BF16, I8 = 16, I32 = 17, OTHER = 18 };
Kind kind_of(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return F32;
        case at::kBFloat16: return BF16;
        case at::kChar: return I8;
        case at::kInt: return I32;
        default: return OTHER;
    }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!o || !THPVariable_Check(o)) raise(PyExc_TypeError, "%s is not a tensor", name);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided) raise(PyExc_TypeError, "%s is not a dense tensor", name);
    return t;
}
// the type code of t, which has to be `want` (ANY: fp32 or bf16)
int32_t check_kind(const at::Tensor& t, const char* name, Kind want) {
    const Kind k = kind_of(t);
    if (want == ANY ? (k != F32 && k != BF16) : k != want)
        raise(PyExc_TypeError, "unsupported dtype %s of %s", c10::toString(t.scalar_type()), name);
    return k;
}
void check_device(const at::Tensor& t, const char* name, int dev) {
    if (!t.is_cuda() || t.get_device() != dev)
        raise(PyExc_ValueError, "%s is on %s, expected GPU %d", name, t.device().str().c_str(), dev);
}

struct Mat {   // rows at any stride, their elements contiguous
    void* p = nullptr;
    int32_t dt = MOE_F32;
    int64_t ld = 0;
    int32_t rows = 0, cols = 0;
};
int32_t size32(int64_t n, const char* name) {
    if (n > INT32_MAX) raise(PyExc_ValueError, "%s is too large", name);
    return static_cast<int32_t>(n);
}
// the matrix whose shape the others follow
Mat first(PyObject* o, const char* name, Kind want, int* dev) {
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda()) raise(PyExc_ValueError, "%s is on %s: a GPU is needed", name, t.device().str().c_str());
    if (t.dim() != 2) raise(PyExc_ValueError, "%s has %d dimensions, expected 2", name, static_cast<int>(t.dim()));
    *dev = static_cast<int>(t.get_device());
    Mat m;
    m.rows = size32(t.size(0), name);
    m.cols = size32(t.size(1), name);
    m.dt = check_kind(t, name, want);
    if (t.stride(1) != 1 && m.cols > 1) raise(PyExc_ValueError, "the elements of a row of %s are not contiguous", name);
    m.p = t.data_ptr();
    m.ld = m.rows > 1 ? t.stride(0) : m.cols;
    return m;
}
Mat mat(PyObject* o, const char* name, int64_t rows, int64_t cols, int dev, Kind want) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
        raise(PyExc_ValueError, "%s has shape %s, expected (%lld, %lld)", name, sizes(t).c_str(), static_cast<long long>(rows),
              static_cast<long long>(cols));
    check_device(t, name, dev);
    Mat m;
    m.dt = check_kind(t, name, want);
    if (t.stride(1) != 1 && cols > 1) raise(PyExc_ValueError, "the elements of a row of %s are not contiguous", name);
    m.p = t.data_ptr();
    m.ld = rows > 1 ? t.stride(0) : cols;
    m.rows = static_cast<int32_t>(rows);
    m.cols = static_cast<int32_t>(cols);
    return m;
}
// n contiguous elements, whatever the shape
void* vec(PyObject* o, const char* name, int64_t n, int dev, Kind want, int32_t* dt = nullptr) {
    const at::Tensor& t = tensor(o, name);
    if (t.numel() != n)
        raise(PyExc_ValueError, "%s has %lld elements, expected %lld", name, static_cast<long long>(t.numel()),
              static_cast<long long>(n));
    check_device(t, name, dev);
    const int32_t k = check_kind(t, name, want);
    if (dt) *dt = k;
    if (!t.is_contiguous()) raise(PyExc_ValueError, "%s is not contiguous", name);
    return t.data_ptr();
}
template <typename T>
T* vec_or_null(PyObject* o, const char* name, int64_t n, int dev, Kind want, int32_t* dt = nullptr) {
    return given(o) ? static_cast<T*>(vec(o, name, n, dev, want, dt)) : nullptr;
}

// the stream to launch on: `o` (a torch stream of GPU dev), or the GPU's current one
void* stream_of(PyObject* o, int dev) {
    if (!given(o)) return c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(dev)).stream();
    PyObject* i = PyObject_GetAttrString(o, "device_index");
    if (!i) throw Raised{};
    const long d = PyLong_AsLong(i);
    Py_DECREF(i);
    if (d == -1 && PyErr_Occurred()) throw Raised{};
    if (d != dev) raise(PyExc_ValueError, "the stream belongs to GPU %ld, the tensors are on GPU %d", d, dev);
    PyObject* s = PyObject_GetAttrString(o, "cuda_stream");
    if (!s) throw Raised{};
    void* p = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    if (!p && PyErr_Occurred()) throw Raised{};
    return p;
}

// Runs f with GPU dev current and the interpreter lock released; raises on a status.
template <typename F>
void on_device(int dev, F f) {
    const int cur = c10::hip::current_device();
    moe_status st;
    if (cur != dev) c10::hip::set_device(static_cast<c10::DeviceIndex>(dev));
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    if (cur != dev) c10::hip::set_device(static_cast<c10::DeviceIndex>(cur));
    if (st == MOE_OK) return;
    PyObject* pkg = PyImport_ImportModule("expert_ffn_amd");
    PyObject* type = pkg ? PyObject_GetAttrString(pkg, "MoeError") : nullptr;
    PyObject* e = type ? PyObject_CallFunction(type, "is", static_cast<int>(st), moe_last_error()) : nullptr;
    if (e) PyErr_SetObject(type, e);
    Py_XDECREF(e);
    Py_XDECREF(type);
    Py_XDECREF(pkg);
    throw Raised{};
}

template <typename F>
PyObject* guarded(F f) {
    try {
        f();
        Py_RETURN_NONE;
    } catch (const Raised&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define BOUND(name) PyObject* name(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames)
#define TAKE(S) \
    PyObject* a[MAX_ARGS]; \
    take(S, args, nargs, kwnames, a)

Signature S_route = {"route_score_topk", 12, 4,
                     {"logits", "k", "topk_ids", "topk_w", "score", "bias", "n_group", "topk_group", "group_rank", "renorm",
                      "scale", "stream"}, {}};
BOUND(route_score_topk) {
    return guarded([&] {
        TAKE(S_route);
        int dev;
        const Mat l = first(a[0], "logits", ANY, &dev);
        const int32_t k = to_int(a[1], "k", 0);
        const int64_t R = static_cast<int64_t>(l.rows) * k;
        const float* bias = vec_or_null<float>(a[5], "bias", l.cols, dev, F32);
        int32_t* ids = static_cast<int32_t*>(vec(a[2], "topk_ids", R, dev, I32));
        float* w = static_cast<float*>(vec(a[3], "topk_w", R, dev, F32));
        const int32_t score = to_int(a[4], "score", MOE_SCORE_SOFTMAX), G = to_int(a[6], "n_group", 1),
                      keep = to_int(a[7], "topk_group", 1), rank = to_int(a[8], "group_rank", MOE_GROUP_MAX),
                      renorm = to_int(a[9], "renorm", 1);
        const float scale = to_float(a[10], 1.0f);
        void* s = stream_of(a[11], dev);
        on_device(dev, [&] {
            return moe_route_score_topk(l.p, l.dt, l.ld, bias, l.rows, l.cols, k, score, G, keep, rank, renorm, scale, ids, w, s);
        });
    });
}

Signature S_router = {"router_score_topk", 15, 7,
                      {"x", "w_router", "k", "logits", "ws", "topk_ids", "topk_w", "score", "bias", "n_group", "topk_group",
                       "group_rank", "renorm", "scale", "stream"}, {}};
BOUND(router_score_topk) {
    return guarded([&] {
        TAKE(S_router);
        int dev;
        const Mat x = first(a[0], "x", ANY, &dev);
        if (x.ld != x.cols) raise(PyExc_ValueError, "x is not contiguous");
        const at::Tensor& wr = tensor(a[1], "w_router");
        if (wr.dim() != 2) raise(PyExc_ValueError, "w_router has %d dimensions, expected 2", static_cast<int>(wr.dim()));
        const int32_t E = size32(wr.size(0), "w_router"), T = x.rows, k = to_int(a[2], "k", 0);
        const float* w = static_cast<float*>(vec(a[1], "w_router", static_cast<int64_t>(E) * x.cols, dev, F32));
        float* lg = static_cast<float*>(vec(a[3], "logits", static_cast<int64_t>(T) * E, dev, F32));
        const float* bias = vec_or_null<float>(a[8], "bias", E, dev, F32);
        int32_t* ids = static_cast<int32_t*>(vec(a[5], "topk_ids", static_cast<int64_t>(T) * k, dev, I32));
        float* tw = static_cast<float*>(vec(a[6], "topk_w", static_cast<int64_t>(T) * k, dev, F32));
        const at::Tensor& ws = tensor(a[4], "ws");
        check_device(ws, "ws", dev);
        if (!ws.is_contiguous()) raise(PyExc_ValueError, "ws is not contiguous");
        void* wp = ws.data_ptr();
        const size_t wb = static_cast<size_t>(ws.numel()) * ws.element_size();
        const int32_t score = to_int(a[7], "score", MOE_SCORE_SOFTMAX), G = to_int(a[9], "n_group", 1),
                      keep = to_int(a[10], "topk_group", 1), rank = to_int(a[11], "group_rank", MOE_GROUP_MAX),
                      renorm = to_int(a[12], "renorm", 1);
        const float scale = to_float(a[13], 1.0f);
        void* s = stream_of(a[14], dev);
        on_device(dev, [&] {
            return moe_router_score_topk(x.p, x.dt, T, x.cols, w, E, k, bias, score, G, keep, rank, renorm, scale, lg, wp, wb,
                                         ids, tw, s);
        });
    });
}

// x, xq and xq_scale of a norm
struct Outs {
    Mat x, q;
    float* scale = nullptr;
};
Outs norm_outputs(PyObject* x, PyObject* xq, PyObject* xs, const Mat& h, int dev) {
    Outs o;
    if (given(x)) o.x = mat(x, "x", h.rows, h.cols, dev, ANY);
    if (given(xq) != given(xs)) raise(PyExc_ValueError, "xq and xq_scale go together");
    if (given(xq)) {
        o.q = mat(xq, "xq", h.rows, h.cols, dev, I8);
        o.scale = static_cast<float*>(vec(xs, "xq_scale", h.rows, dev, F32));
    }
    return o;
}

Signature S_norm_in = {"norm_in", 8, 3, {"h", "w", "eps", "x", "xq", "xq_scale", "w_offset", "stream"}, {}};
BOUND(norm_in) {
    return guarded([&] {
        TAKE(S_norm_in);
        int dev;
        const Mat h = first(a[0], "h", ANY, &dev);
        int32_t wdt = MOE_F32;
        const void* w = vec_or_null<void>(a[1], "w", h.cols, dev, ANY, &wdt);
        const float eps = to_float(a[2], 0.0f), off = to_float(a[6], 0.0f);
        const Outs o = norm_outputs(a[3], a[4], a[5], h, dev);
        void* s = stream_of(a[7], dev);
        on_device(dev, [&] {
            return moe_norm_in(h.p, h.dt, h.ld, h.rows, h.cols, w, wdt, off, eps, o.x.p, o.x.dt, o.x.ld,
                               static_cast<int8_t*>(o.q.p), o.q.ld, o.scale, s);
        });
    });
}

Signature S_quant = {"quantize_tokens", 4, 3, {"x", "xq", "xq_scale", "stream"}, {}};
BOUND(quantize_tokens) {
    return guarded([&] {
        TAKE(S_quant);
        int dev;
        const Mat x = first(a[0], "x", ANY, &dev);
        const Mat q = mat(a[1], "xq", x.rows, x.cols, dev, I8);
        float* sc = static_cast<float*>(vec(a[2], "xq_scale", x.rows, dev, F32));
        void* s = stream_of(a[3], dev);
        on_device(dev, [&] {
            return moe_quantize_tokens(x.p, x.dt, x.ld, x.rows, x.cols, static_cast<int8_t*>(q.p), q.ld, sc, s);
        });
    });
}

Signature S_norm_out = {"norm_out", 17, 4,
                        {"h", "h_out", "w_post", "eps", "out_routes", "topk_w", "route_pos", "y", "gate", "block_scale",
                         "res_scale", "w_next", "x", "xq", "xq_scale", "w_offset", "stream"}, {}};
BOUND(norm_out) {
    return guarded([&] {
        TAKE(S_norm_out);
        if (!given(a[4]) && (given(a[5]) || given(a[6]))) raise(PyExc_ValueError, "topk_w and route_pos need out_routes");
        int dev;
        const Mat h = first(a[0], "h", ANY, &dev);
        const int32_t T = h.rows, H = h.cols;
        const Mat ho = mat(a[1], "h_out", T, H, dev, static_cast<Kind>(h.dt));
        Mat routes, y;
        float* tw = nullptr;
        int32_t* pos = nullptr;
        int32_t k = 0;
        if (given(a[4])) {
            if (!given(a[5]) || !given(a[6])) raise(PyExc_ValueError, "out_routes needs topk_w and route_pos");
            const int64_t R = tensor(a[6], "route_pos").numel();
            k = T ? static_cast<int32_t>(R / T) : 0;
            if (static_cast<int64_t>(k) * T != R)
                raise(PyExc_ValueError, "route_pos has %lld elements, not a multiple of T=%d", static_cast<long long>(R), T);
            routes = mat(a[4], "out_routes", R, H, dev, ANY);
            if (routes.ld != H) raise(PyExc_ValueError, "out_routes is not contiguous");
            tw = static_cast<float*>(vec(a[5], "topk_w", R, dev, F32));
            pos = static_cast<int32_t*>(vec(a[6], "route_pos", R, dev, I32));
        }
        if (given(a[7])) y = mat(a[7], "y", T, H, dev, ANY);
        int32_t wdt = MOE_F32, ndt = MOE_F32;
        const void* wp = vec_or_null<void>(a[2], "w_post", H, dev, ANY, &wdt);
        const void* wn = vec_or_null<void>(a[11], "w_next", H, dev, ANY, &ndt);
        if (wp && wn && wdt != ndt) raise(PyExc_TypeError, "w_post and w_next have different dtypes");
        if (wn) wdt = ndt;
        const void* gate = nullptr;
        int32_t gdt = MOE_F32;
        int64_t gst = 0, gsh = 0;
        if (given(a[8])) {   // broadcasts to [T, H]
            const at::Tensor& g = tensor(a[8], "gate");
            const int64_t nd = g.dim(), gr = nd == 2 ? g.size(0) : 1, gc = nd >= 1 ? g.size(nd - 1) : 1;
            if (nd > 2 || (gr != 1 && gr != T) || (gc != 1 && gc != H))
                raise(PyExc_ValueError, "gate has shape %s, which does not broadcast to (%d, %d)", sizes(g).c_str(), T, H);
            check_device(g, "gate", dev);
            gdt = check_kind(g, "gate", ANY);
            if (gr > 1) gst = g.stride(0);
            if (gc > 1) gsh = g.stride(nd - 1);
            gate = g.data_ptr();
        }
        const Outs o = norm_outputs(a[12], a[13], a[14], h, dev);
        const int32_t next = given(a[12]) || given(a[13]);
        if (wn && !next) raise(PyExc_ValueError, "w_next is given, but neither x nor xq to write the next norm into");
        const float eps = to_float(a[3], 0.0f), bs = to_float(a[9], 1.0f), rs = to_float(a[10], 1.0f), off = to_float(a[15], 0.0f);
        void* s = stream_of(a[16], dev);
        on_device(dev, [&] {
            return moe_norm_out(routes.p, routes.dt, tw, pos, k, y.p, y.dt, y.ld, T, H, wp, wdt, off, eps, gate, gdt, gst, gsh,
                                bs, rs, h.p, h.dt, h.ld, ho.p, ho.ld, next, wn, o.x.p, o.x.dt, o.x.ld,
                                static_cast<int8_t*>(o.q.p), o.q.ld, o.scale, s);
        });
    });
}

Signature S_mm = {"matmul_i8", 7, 5, {"xq", "x_scale", "wq", "w_scale", "out", "bias", "stream"}, {}};
BOUND(matmul_i8) {
    return guarded([&] {
        TAKE(S_mm);
        int dev;
        const Mat x = first(a[0], "xq", I8, &dev);
        const at::Tensor& wt = tensor(a[2], "wq");
        const int32_t N = wt.dim() == 2 ? size32(wt.size(0), "wq") : 0;
        const Mat w = mat(a[2], "wq", N, x.cols, dev, I8);
        const Mat o = mat(a[4], "out", x.rows, N, dev, ANY);
        const float* sx = static_cast<float*>(vec(a[1], "x_scale", x.rows, dev, F32));
        const float* sw = static_cast<float*>(vec(a[3], "w_scale", N, dev, F32));
        const float* bias = vec_or_null<float>(a[5], "bias", N, dev, F32);
        void* s = stream_of(a[6], dev);
        on_device(dev, [&] {
            return moe_matmul_i8(static_cast<int8_t*>(x.p), x.ld, sx, static_cast<int8_t*>(w.p), w.ld, sw, bias, x.rows, N, x.cols,
                                 o.p, o.dt, o.ld, s);
        });
    });
}

Signature S_gmm = {"gated_matmul_i8", 7, 6, {"xq", "x_scale", "wq", "w_scale", "act", "out", "stream"}, {}};
BOUND(gated_matmul_i8) {
    return guarded([&] {
        TAKE(S_gmm);
        int dev;
        const Mat x = first(a[0], "xq", I8, &dev);
        const at::Tensor& wt = tensor(a[2], "wq");
        const int32_t N2 = wt.dim() == 2 ? size32(wt.size(0), "wq") : 0, F = N2 / 2;
        if (N2 % 2) raise(PyExc_ValueError, "wq has %d rows: gate and up rows come in pairs", N2);
        const Mat w = mat(a[2], "wq", N2, x.cols, dev, I8);
        const Mat o = mat(a[5], "out", x.rows, F, dev, ANY);
        const float* sx = static_cast<float*>(vec(a[1], "x_scale", x.rows, dev, F32));
        const float* sw = static_cast<float*>(vec(a[3], "w_scale", N2, dev, F32));
        const int32_t act = to_int(a[4], "act", -1);
        void* s = stream_of(a[6], dev);
        on_device(dev, [&] {
            return moe_gated_matmul_i8(static_cast<int8_t*>(x.p), x.ld, sx, static_cast<int8_t*>(w.p), w.ld, sw, x.rows, F, x.cols,
                                       act, o.p, o.dt, o.ld, s);
        });
    });
}

// a pool of adapters: [n, ...] of the given sizes, each adapter contiguous
const at::Tensor& pool(PyObject* o, const char* name, int dev, int64_t* stride) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() < 3) raise(PyExc_ValueError, "%s has shape %s, expected a pool of matrices", name, sizes(t).c_str());
    check_device(t, name, dev);
    check_kind(t, name, BF16);
    int64_t each = 1;
    for (int64_t i = t.dim() - 1; i > 0; each *= t.size(i--))
        if (t.size(i) > 1 && t.stride(i) != each) raise(PyExc_ValueError, "an adapter of %s is not contiguous", name);
    *stride = t.size(0) > 1 ? t.stride(0) : each;
    return t;
}
struct Adapters {   // of a product: s, adapter_ids, b and ranks (or none of them)
    Mat s;
    int32_t *ids = nullptr, *ranks = nullptr, n = 0, R = 0;
    const void* b = nullptr;
    int64_t stride = 0;
};
Adapters adapters(PyObject* s, PyObject* ids, PyObject* b, PyObject* ranks, const Mat& x, int32_t rows, int32_t halves, int dev) {
    Adapters A;
    if (!given(s)) {
        if (given(ids) || given(b) || given(ranks)) raise(PyExc_ValueError, "adapter_ids, b and ranks go with s");
        return A;
    }
    const at::Tensor& t = pool(b, "b", dev, &A.stride);
    if (t.dim() != 3 || t.size(1) != rows)
        raise(PyExc_ValueError, "b has shape %s, expected (n, %d, R)", sizes(t).c_str(), rows);
    A.n = size32(t.size(0), "b");
    A.R = size32(t.size(2), "b");
    A.b = t.data_ptr();
    A.s = mat(s, "s", x.rows, static_cast<int64_t>(halves) * A.R, dev, BF16);
    A.ids = static_cast<int32_t*>(vec(ids, "adapter_ids", x.rows, dev, I32));
    A.ranks = vec_or_null<int32_t>(ranks, "ranks", A.n, dev, I32);
    return A;
}
// a weight matrix [rows, K] whose row count the call takes from it
Mat weights(PyObject* o, const char* name, int64_t K, int dev) {
    const at::Tensor& t = tensor(o, name);
    return mat(o, name, t.dim() == 2 ? size32(t.size(0), name) : 0, K, dev, BF16);
}
int32_t half_of(const Mat& w, const char* name) {
    if (w.rows % 2) raise(PyExc_ValueError, "%s has %d rows: gate and up rows come in pairs", name, w.rows);
    return w.rows / 2;
}

Signature S_mmb = {"matmul_bf16", 8, 3, {"x", "w", "out", "s", "adapter_ids", "b", "ranks", "stream"}, {}};
BOUND(matmul_bf16) {
    return guarded([&] {
        TAKE(S_mmb);
        int dev;
        const Mat x = first(a[0], "x", BF16, &dev);
        const Mat w = weights(a[1], "w", x.cols, dev);
        const Mat o = mat(a[2], "out", x.rows, w.rows, dev, ANY);
        const Adapters A = adapters(a[3], a[4], a[5], a[6], x, w.rows, 1, dev);
        void* s = stream_of(a[7], dev);
        on_device(dev, [&] {
            return moe_matmul_bf16(x.p, x.ld, w.p, w.ld, x.rows, w.rows, x.cols, o.p, o.dt, o.ld, A.s.p, A.s.ld, A.ids, A.b, A.stride,
                                   A.ranks, A.n, A.R, s);
        });
    });
}

Signature S_gmmb = {"gated_matmul_bf16", 10, 4, {"x", "w", "act", "out", "pre", "s", "adapter_ids", "b", "ranks", "stream"}, {}};
BOUND(gated_matmul_bf16) {
    return guarded([&] {
        TAKE(S_gmmb);
        int dev;
        const Mat x = first(a[0], "x", BF16, &dev);
        const Mat w = weights(a[1], "w", x.cols, dev);
        const int32_t F = half_of(w, "w"), act = to_int(a[2], "act", -1);
        const Mat o = mat(a[3], "out", x.rows, F, dev, ANY);
        const Mat pre = given(a[4]) ? mat(a[4], "pre", x.rows, w.rows, dev, BF16) : Mat{};
        const Adapters A = adapters(a[5], a[6], a[7], a[8], x, w.rows, 2, dev);
        void* s = stream_of(a[9], dev);
        on_device(dev, [&] {
            return moe_gated_matmul_bf16(x.p, x.ld, w.p, w.ld, x.rows, F, x.cols, act, o.p, o.dt, o.ld, pre.p, pre.ld, A.s.p, A.s.ld,
                                         A.ids, A.b, A.stride, A.ranks, A.n, A.R, s);
        });
    });
}

Signature S_shrink = {"adapter_shrink", 7, 5, {"x", "adapter_ids", "a", "scale", "s", "ranks", "stream"}, {}};
BOUND(adapter_shrink) {
    return guarded([&] {
        TAKE(S_shrink);
        int dev;
        const Mat x = first(a[0], "x", BF16, &dev);
        int64_t stride;
        const at::Tensor& t = pool(a[2], "a", dev, &stride);
        const int64_t nd = t.dim();
        if (nd > 4 || t.size(nd - 1) != x.cols || (nd == 4 && t.size(1) != 1 && t.size(1) != 2))
            raise(PyExc_ValueError, "a has shape %s, expected (n, R, %d) or (n, 2, R, %d)", sizes(t).c_str(), x.cols, x.cols);
        const int32_t n = size32(t.size(0), "a"), R = size32(t.size(nd - 2), "a"), halves = nd == 4 ? static_cast<int32_t>(t.size(1)) : 1;
        const Mat o = mat(a[4], "s", x.rows, static_cast<int64_t>(halves) * R, dev, BF16);
        const int32_t* ids = static_cast<int32_t*>(vec(a[1], "adapter_ids", x.rows, dev, I32));
        const float* scale = vec_or_null<float>(a[3], "scale", n, dev, F32);
        const int32_t* ranks = vec_or_null<int32_t>(a[5], "ranks", n, dev, I32);
        const void* pa = t.data_ptr();
        void* s = stream_of(a[6], dev);
        on_device(dev, [&] {
            return moe_adapter_shrink(x.p, x.ld, x.rows, x.cols, ids, pa, stride, n, R, halves, scale, ranks, o.p, o.ld, s);
        });
    });
}

Signature S_mmbg = {"matmul_bf16_backward", 6, 3, {"x", "w", "dout", "dx", "dw", "stream"}, {}};
BOUND(matmul_bf16_backward) {
    return guarded([&] {
        TAKE(S_mmbg);
        int dev;
        const Mat x = first(a[0], "x", BF16, &dev);
        const Mat w = weights(a[1], "w", x.cols, dev);
        const Mat d = mat(a[2], "dout", x.rows, w.rows, dev, BF16);
        const Mat dx = given(a[3]) ? mat(a[3], "dx", x.rows, x.cols, dev, ANY) : Mat{};
        const Mat dw = given(a[4]) ? mat(a[4], "dw", w.rows, x.cols, dev, ANY) : Mat{};
        if (!given(a[3]) && !given(a[4])) raise(PyExc_ValueError, "neither dx nor dw is given");
        if (x.rows == 0 && !given(a[4])) return;   // dx has no rows
        void* s = stream_of(a[5], dev);
        on_device(dev, [&] {
            return moe_matmul_bf16_backward(x.p, x.ld, w.p, w.ld, d.p, d.ld, x.rows, w.rows, x.cols, dx.p, dx.dt, dx.ld, dw.p, dw.dt,
                                            dw.ld, s);
        });
    });
}

Signature S_gmmbg = {"gated_matmul_bf16_backward", 9, 6, {"x", "w", "act", "pre", "dout", "dpre", "dx", "dw", "stream"}, {}};
BOUND(gated_matmul_bf16_backward) {
    return guarded([&] {
        TAKE(S_gmmbg);
        int dev;
        const Mat x = first(a[0], "x", BF16, &dev);
        const Mat w = weights(a[1], "w", x.cols, dev);
        const int32_t F = half_of(w, "w"), act = to_int(a[2], "act", -1);
        const Mat pre = mat(a[3], "pre", x.rows, w.rows, dev, BF16);
        const Mat d = mat(a[4], "dout", x.rows, F, dev, BF16);
        const Mat dp = mat(a[5], "dpre", x.rows, w.rows, dev, BF16);
        const Mat dx = given(a[6]) ? mat(a[6], "dx", x.rows, x.cols, dev, ANY) : Mat{};
        const Mat dw = given(a[7]) ? mat(a[7], "dw", w.rows, x.cols, dev, ANY) : Mat{};
        void* s = stream_of(a[8], dev);
        on_device(dev, [&] {
            return moe_gated_matmul_bf16_backward(x.p, x.ld, w.p, w.ld, act, pre.p, pre.ld, d.p, d.ld, x.rows, F, x.cols, dp.p, dp.ld,
                                                  dx.p, dx.dt, dx.ld, dw.p, dw.dt, dw.ld, s);
        });
    });
}

#define METHOD(name, doc) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL | METH_KEYWORDS, doc}
PyMethodDef methods[] = {
    METHOD(route_score_topk,
           "route_score_topk(logits, k, topk_ids, topk_w, score=0, bias=None, n_group=1, topk_group=1, group_rank=0, "
           "renorm=1, scale=1.0, stream=None)\n--\n\n"
           "Top-k of softmax or sigmoid scores (SCORE_SOFTMAX, SCORE_SIGMOID) of logits [T, E] plus a bias [E] that\n"
           "counts for the choice only, inside the topk_group best of n_group expert groups (GROUP_MAX, GROUP_TOP2);\n"
           "ids int32 and weights fp32 [T, k]."),
    METHOD(router_score_topk,
           "router_score_topk(x, w_router, k, logits, ws, topk_ids, topk_w, score=0, bias=None, n_group=1, topk_group=1, "
           "group_rank=0, renorm=1, scale=1.0, stream=None)\n--\n\n"
           "fp32 router product of x [T, H] with w_router [E, H] (logits [T, E] out, ws as for router_topk), then\n"
           "route_score_topk on the logits."),
    METHOD(norm_in,
           "norm_in(h, w, eps, x=None, xq=None, xq_scale=None, w_offset=0.0, stream=None)\n--\n\n"
           "RMS norm of the rows of h [T, H] with weight w_offset + w [H] (w None: 1), into x (fp32 or bf16), as int8\n"
           "codes xq with one fp32 scale per row (xq_scale [T]), or both."),
    METHOD(quantize_tokens,
           "quantize_tokens(x, xq, xq_scale, stream=None)\n--\n\n"
           "int8 codes and the scale of each row of x [T, K]: codes rint(x / s), s = max |x| / 127."),
    METHOD(norm_out,
           "norm_out(h, h_out, w_post, eps, out_routes=None, topk_w=None, route_pos=None, y=None, gate=None, "
           "block_scale=1.0, res_scale=1.0, w_next=None, x=None, xq=None, xq_scale=None, w_offset=0.0, stream=None)\n--\n\n"
           "End of a block: h_out = res_scale * h + block_scale * gate * norm(b; w_post), where b is the weighted combine\n"
           "of out_routes (topk_w, route_pos [T, k] as for combine) plus y [T, H]; then, when x or xq is given, the next\n"
           "block's norm of h_out (w_next) into them.  w_post None: b is not normed.  gate broadcasts to [T, H].  h_out\n"
           "may be h."),
    METHOD(matmul_i8,
           "matmul_i8(xq, x_scale, wq, w_scale, out, bias=None, stream=None)\n--\n\n"
           "out [T, N] = (xq [T, K] . wq [N, K]) * x_scale [T] * w_scale [N] (+ bias [N] fp32): int8 codes, exact int32\n"
           "sums, out fp32 or bf16."),
    METHOD(gated_matmul_i8,
           "gated_matmul_i8(xq, x_scale, wq, w_scale, act, out, stream=None)\n--\n\n"
           "out [T, F] = act(gate) * up of the int8 product of xq [T, K] with wq [2F, K] (gate rows, then up rows, as an\n"
           "expert's w13)."),
    METHOD(matmul_bf16,
           "matmul_bf16(x, w, out, s=None, adapter_ids=None, b=None, ranks=None, stream=None)\n--\n\n"
           "out [T, N] = x [T, K] . w [N, K] in bf16, fp32 sums, out fp32 or bf16.  With s [T, R] (adapter_shrink), token t\n"
           "adds s[t] . b[adapter_ids[t]] of its request's low-rank adapter: b [n, N, R], ranks int32 [n] (None: R), ids\n"
           "int32 [T], outside [0, n): none."),
    METHOD(gated_matmul_bf16,
           "gated_matmul_bf16(x, w, act, out, pre=None, s=None, adapter_ids=None, b=None, ranks=None, stream=None)\n--\n\n"
           "out [T, F] = act(gate) * up of the bf16 product of x [T, K] with w [2F, K] (gate rows, then up rows, as an\n"
           "expert's w13); pre [T, 2F] takes the sums for the backward pass (without adapters).  Adapters as for\n"
           "matmul_bf16, before the activation: s [T, 2R] and b [n, 2F, R], gate's then up's."),
    METHOD(adapter_shrink,
           "adapter_shrink(x, adapter_ids, a, scale, s, ranks=None, stream=None)\n--\n\n"
           "s[t] = scale[i] * (x[t] . a[i]), i = adapter_ids[t]: the first product of the tokens' low-rank adapters, zeros\n"
           "without one and past a rank.  a [n, R, K] with s [T, R], or [n, 2, R, K] (gate and up) with s [T, 2R]; scale\n"
           "fp32 [n] or None.  s is bf16: out carries its rounding in fp32 too."),
    METHOD(matmul_bf16_backward,
           "matmul_bf16_backward(x, w, dout, dx=None, dw=None, stream=None)\n--\n\n"
           "dx [T, K] = dout [T, N] . w, dw [N, K] = dout^T . x, each fp32 or bf16 or None."),
    METHOD(gated_matmul_bf16_backward,
           "gated_matmul_bf16_backward(x, w, act, pre, dout, dpre, dx=None, dw=None, stream=None)\n--\n\n"
           "From pre [T, 2F] of a forward pass without adapters and dout [T, F]: dpre [T, 2F] (may be pre), dx [T, K] =\n"
           "dpre . w, dw [2F, K] = dpre^T . x.  dpre is bf16: dx and dw carry its rounding in fp32 too."),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Operators around the expert FFN (see expert_ffn_amd).", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    for (Signature* s : {&S_route, &S_router, &S_norm_in, &S_quant, &S_norm_out, &S_mm, &S_gmm, &S_mmb, &S_gmmb, &S_shrink, &S_mmbg, &S_gmmbg})
        for (int i = 0; i < s->n; ++i)
            if (!(s->interned[i] = PyUnicode_InternFromString(s->names[i]))) return nullptr;
    return PyModule_Create(&module);
}
