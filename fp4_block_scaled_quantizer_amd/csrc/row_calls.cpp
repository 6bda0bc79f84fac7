// row_calls.cpp -- argument marshalling of the row-wise operators for the
// Python binding, compiled: a decoding step makes these calls on a few
// kilobytes each, and reading a tensor's attributes from Python costs more
// than the launch.  Checks that every tensor has the shape, type, strides and
// device that the call gives the library, allocates the outputs not given,
// and calls libfp4q through the addresses that bind() gets from the ctypes
// layer.  No computation.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/StreamGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/fp4q.h"

namespace {

struct Library {
    decltype(&::fp4_dropout) dropout;
    decltype(&::fp4_norm) norm;
    decltype(&::fp4q_norm_grad_workspace_bytes) norm_grad_workspace;
    decltype(&::fp4_norm_grad) norm_grad;
    decltype(&::fp4_swiglu_grad_bf16) swiglu_grad;
    decltype(&::fp4_rotary) rotary;
    decltype(&::fp4_pack8) pack8;
    decltype(&::fp4_unpack8) unpack8;
    decltype(&::fp4_norm_pack8) norm_pack8;
    decltype(&::fp4_norm_grad_pack8) norm_grad_pack8;
    decltype(&::fp4_swiglu_grad_pack8) swiglu_grad_pack8;
    decltype(&::fp4_matvec_mx) matvec_mx;
    decltype(&::fp4_matvec_mx_pack8) matvec_mx_pack8;
    decltype(&::fp4_matvec_nv) matvec_nv;
    PyObject *error;          // Fp4qError
    PyObject *current, *raw, *external;  // torch's current device, its current stream, a stream of a handle
} lib{};

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct PythonError {};  // set already

// ---- Python values

const at::Tensor *tensor_or_null(PyObject *o, const char *name)
{
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}
const at::Tensor &tensor(PyObject *o, const char *name)
{
    const at::Tensor *t = tensor_or_null(o, name);
    if (!t) throw Refused(std::string(name) + " must be a tensor");
    return *t;
}
int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError();
    return v;
}
uint64_t bits64(PyObject *o)  // a key: any integer, its low 64 bits
{
    const unsigned long long v = PyLong_AsUnsignedLongLongMask(o);
    if (v == (unsigned long long)-1 && PyErr_Occurred()) throw PythonError();
    return v;
}
double real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError();
    return v;
}
bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PythonError();
    return v != 0;
}

// ---- tensors

int type_of(const at::Tensor &t)  // -1: neither
{
    switch (t.scalar_type()) {
    case at::kFloat: return FP4Q_OUT_F32;
    case at::kBFloat16: return FP4Q_OUT_BF16;
    default: return -1;
    }
}

struct Matrix {
    void *p = nullptr;
    int64_t ld = 0;
};
Matrix rows_of(const at::Tensor &t, const char *name)
{
    const int64_t rows = t.size(0), cols = t.size(1);
    const int64_t ld = rows <= 1 ? cols : t.stride(0);
    if (ld < cols || (t.stride(1) != 1 && cols > 1))
        throw Refused(std::string(name) + " must have unit column stride and rows that do not overlap");
    return Matrix{t.data_ptr(), ld};
}

// While a call runs, the `stream` it names is torch's current one. What the
// call makes is then that stream's memory, which is given out again in the
// order of its work; from the caller's stream it could hold what kernels
// queued there still use, and be given out there while this call's kernels
// still write. Outputs are recorded on the caller's stream as well, where they
// are read next: they may be let go of there without more ado.
class OnStream {
public:
    OnStream(PyObject *stream, const at::Tensor &t)
    {
        if (stream == Py_None || !t.is_cuda()) return;
        PyObject *own = nullptr;
        if (!PyObject_HasAttrString(stream, "stream_id")) {  // a handle of another library's
            PyObject *h = PyObject_GetAttrString(stream, "cuda_stream");
            own = h ? PyObject_CallOneArg(lib.external, h) : nullptr;
            Py_XDECREF(h);
            if (!own) throw PythonError();
            stream = own;
        }
        const int64_t id = member(stream, "stream_id"), index = member(stream, "device_index"),
                      type = member(stream, "device_type");
        Py_XDECREF(own);
        if (PyErr_Occurred()) throw PythonError();
        if (type != (int64_t)at::kCUDA) throw Refused("stream must be a GPU stream");
        guard_.reset_stream(c10::Stream::unpack3(id, (c10::DeviceIndex)index, at::kCUDA));
    }
    at::Tensor empty(at::IntArrayRef sizes, const at::TensorOptions &o)
    {
        at::Tensor t = at::empty(sizes, o);
        if (guard_.original_stream()) made_.push_back(t);
        return t;
    }
    void done() const
    {
        if (const auto caller = guard_.original_stream())
            for (const at::Tensor &t : made_) t.record_stream(*caller);
    }

private:
    static int64_t member(PyObject *o, const char *name)
    {
        PyObject *v = PyErr_Occurred() ? nullptr : PyObject_GetAttrString(o, name);
        const int64_t k = v ? PyLong_AsLongLong(v) : -1;
        Py_XDECREF(v);
        return k;
    }
    c10::OptionalStreamGuard guard_;
    std::vector<at::Tensor> made_;
};

// A call's first matrix, and others of its shape, type and device.
struct Like {
    const at::Tensor &t;
    int type;
    int64_t rows, cols;
    Like(PyObject *o, const char *name) : t(tensor(o, name)), type(type_of(t))
    {
        if (type < 0 || t.dim() != 2) throw Refused(std::string(name) + " must be a 2-D fp32 or bf16 tensor");
        rows = t.size(0);
        cols = t.size(1);
    }
    Matrix matrix(const at::Tensor &o, const char *name) const
    {
        if (o.dim() != 2 || o.size(0) != rows || o.size(1) != cols || o.scalar_type() != t.scalar_type() ||
            o.device() != t.device())
            throw Refused(std::string(name) + " must be a tensor of the first one's shape, type and device");
        return rows_of(o, name);
    }
    // given, made here, or (neither wanted nor given) none; `keep` holds it
    Matrix output(OnStream &on, PyObject *o, const char *name, bool wanted, at::Tensor &keep) const
    {
        const at::Tensor *g = tensor_or_null(o, name);
        if (g) {
            keep = *g;
            return matrix(*g, name);
        }
        if (!wanted) return Matrix{};
        keep = on.empty({rows, cols}, t.options());
        return Matrix{keep.data_ptr(), cols};
    }
    Matrix input(PyObject *o, const char *name) const
    {
        const at::Tensor *g = tensor_or_null(o, name);
        return g ? matrix(*g, name) : Matrix{};
    }
    void *vector(const at::Tensor &o, const char *name, int64_t n, at::ScalarType type) const
    {
        if (o.numel() != n || o.scalar_type() != type || o.device() != t.device() || !o.is_contiguous())
            throw Refused(std::string(name) + " must be " + std::to_string(n) + " contiguous " + at::toString(type) +
                          " elements on the same device");
        return o.data_ptr();
    }
    float *floats(OnStream &on, PyObject *o, const char *name, int64_t n, bool wanted, at::Tensor &keep) const
    {
        const at::Tensor *g = tensor_or_null(o, name);
        if (g)
            keep = *g;
        else if (wanted)
            keep = on.empty({n}, t.options().dtype(at::kFloat));
        else
            return nullptr;
        return static_cast<float *>(vector(keep, name, n, at::kFloat));
    }
    const void *weight(PyObject *o, const char *name, int &type) const
    {
        const at::Tensor *g = tensor_or_null(o, name);
        if (!g) return nullptr;
        const int k = type_of(*g);
        if (k < 0) throw Refused(std::string(name) + " must be fp32 or bf16");
        if (type >= 0 && k != type) throw Refused("gamma and beta must have the same type");
        type = k;
        return vector(*g, name, cols, g->scalar_type());
    }
};

// A dense tensor of `type` with exactly these sizes on `like`'s device.
void *dense(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef sizes, const at::Tensor &like)
{
    if (t.scalar_type() != type || t.sizes() != sizes || t.device() != like.device() || !t.is_contiguous()) {
        std::string shape;
        for (const int64_t n : sizes) shape += (shape.empty() ? "" : ", ") + std::to_string(n);
        throw Refused(std::string(name) + " must be a contiguous " + at::toString(type) + " tensor of shape (" + shape +
                      ") on the same device");
    }
    return t.data_ptr();
}

// 8-bit rows: codes [rows, cols] and scales [rows, cols / 32], given or (an
// output's) made.
struct Packed {
    void *codes, *scales;
};
Packed packed(PyObject *codes, PyObject *scales, const char *names[2], int64_t rows, int64_t cols, const at::Tensor &like,
              OnStream *on = nullptr, at::Tensor *keep = nullptr)
{
    const at::Tensor *c = tensor_or_null(codes, names[0]), *s = tensor_or_null(scales, names[1]);
    if (on) {
        const auto bytes = like.options().dtype(at::kByte);
        keep[0] = c ? *c : on->empty({rows, cols}, bytes);
        keep[1] = s ? *s : on->empty({rows, cols / 32}, bytes);
        c = &keep[0];
        s = &keep[1];
    }
    if (!c || !s) throw Refused(std::string(names[0]) + " and " + names[1] + " must be tensors");
    return Packed{dense(*c, names[0], at::kByte, {rows, cols}, like), dense(*s, names[1], at::kByte, {rows, cols / 32}, like)};
}

// The handle of the current stream.  The library launches on the current GPU,
// which the tensors have to be on.
void *stream_of(const at::Tensor &t)
{
    PyObject *dev = t.is_cuda() ? PyObject_CallNoArgs(lib.current) : nullptr;
    if (t.is_cuda() && !dev) throw PythonError();
    const int64_t d = dev ? PyLong_AsLongLong(dev) : -1;
    if (!dev || d != t.get_device()) {
        Py_XDECREF(dev);
        throw Refused("the tensors must be on the current GPU");
    }
    PyObject *h = PyObject_CallOneArg(lib.raw, dev);
    Py_DECREF(dev);
    if (!h) throw PythonError();
    void *s = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!s && PyErr_Occurred()) throw PythonError();
    return s;
}

void done(const char *fn, fp4q_status status)
{
    if (status == FP4Q_OK) return;
    PyObject *e = PyObject_CallFunction(lib.error, "si", fn, (int)status);
    if (e) {
        PyErr_SetObject(lib.error, e);
        Py_DECREF(e);
    }
    throw PythonError();
}

PyObject *result(const at::Tensor &t)
{
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
PyObject *results(std::initializer_list<const at::Tensor *> ts)
{
    PyObject *out = PyTuple_New((Py_ssize_t)ts.size());
    if (!out) throw PythonError();
    Py_ssize_t i = 0;
    for (const at::Tensor *t : ts) {
        PyObject *v = result(*t);
        if (!v) {
            Py_DECREF(out);
            throw PythonError();
        }
        PyTuple_SET_ITEM(out, i++, v);
    }
    return out;
}

// ---- the calls

const char *kCodes[2] = {"codes", "scales"}, *kCodes8[2] = {"codes8", "scales8"};

PyObject *dropout(PyObject *const *a)
{
    enum { X, P, SEED, STREAM_ID, RES, Y, STREAM };
    const Like x(a[X], "x");
    OnStream on(a[STREAM], x.t);
    const Matrix mx = x.matrix(x.t, "x"), mr = x.input(a[RES], "residual");
    at::Tensor y;
    const Matrix my = x.output(on, a[Y], "y", true, y);
    const double p = real(a[P]);
    void *st = stream_of(x.t);
    done("fp4_dropout", lib.dropout(mx.p, x.rows, x.cols, mx.ld, x.type, mr.p, mr.ld, (float)p, bits64(a[SEED]),
                                    (uint32_t)bits64(a[STREAM_ID]), my.p, my.ld, st));
    on.done();
    return result(y);
}

template <bool kPack8>
PyObject *norm(PyObject *const *a)
{
    enum {
        X, GAMMA, BETA, KIND, EPS, RES, P, SEED, STREAM_ID, SAVE, WANT_Y, LAYOUT, Y, H, MEAN, RSTD, CODES, SCALES, STREAM,
        CODES8, SCALES8
    };
    const Like x(a[X], "x");
    OnStream on(a[STREAM], x.t);
    const Matrix mx = x.matrix(x.t, "x"), mr = x.input(a[RES], "residual");
    const double p = real(a[P]);
    const int kind = (int)integer(a[KIND]);
    const bool save = truth(a[SAVE]);
    at::Tensor y, h, mean, rstd, keep8[2];
    const Matrix mh = x.output(on, a[H], "h", a[RES] != Py_None || p > 0, h), my = x.output(on, a[Y], "y", truth(a[WANT_Y]), y);
    float *pm = x.floats(on, a[MEAN], "mean", x.rows, save && kind == FP4Q_NORM_LAYER, mean);
    float *ps = x.floats(on, a[RSTD], "rstd", x.rows, save, rstd);
    int wt = -1;
    const void *pg = x.weight(a[GAMMA], "gamma", wt), *pb = x.weight(a[BETA], "beta", wt);
    const at::Tensor *codes = tensor_or_null(a[CODES], "codes"), *scales = tensor_or_null(a[SCALES], "scales");
    Packed p8{};
    if (kPack8) p8 = packed(a[CODES8], a[SCALES8], kCodes8, x.rows, x.cols, x.t, &on, keep8);
    void *st = stream_of(x.t);
    const auto call = [&](auto *fn, auto... more) {
        return fn(mx.p, x.rows, x.cols, mx.ld, x.type, mr.p, mr.ld, (float)p, bits64(a[SEED]),
                  (uint32_t)bits64(a[STREAM_ID]), mh.p, mh.ld, kind, pg, pb, wt < 0 ? FP4Q_OUT_F32 : wt,
                  (float)real(a[EPS]), my.p, my.ld, pm, ps, codes ? codes->data_ptr() : nullptr,
                  scales ? scales->data_ptr() : nullptr, (int)integer(a[LAYOUT]), more..., st);
    };
    if constexpr (kPack8) {
        done("fp4_norm_pack8", call(lib.norm_pack8, p8.codes, p8.scales));
        on.done();
        return results({&y, &h, &mean, &rstd, &keep8[0], &keep8[1]});
    } else {
        done("fp4_norm", call(lib.norm));
        on.done();
        return results({&y, &h, &mean, &rstd});
    }
}

// H: the normed rows, or with kPack8 their codes (and SCALES).
template <bool kPack8>
PyObject *norm_grad(PyObject *const *a)
{
    enum {
        DY, H, GAMMA, KIND, MEAN, RSTD, DRES, P, SEED, STREAM_ID, WEIGHTS, DH, DX, DGAMMA, DBETA, WORKSPACE, STREAM,
        SCALES
    };
    const Like x(a[DY], "dy");
    OnStream on(a[STREAM], x.t);
    const Matrix my = x.matrix(x.t, "dy"), mr = x.input(a[DRES], "dres");
    Matrix mh;
    Packed h8{};
    if constexpr (kPack8)
        h8 = packed(a[H], a[SCALES], kCodes, x.rows, x.cols, x.t);
    else
        mh = x.matrix(tensor(a[H], "h"), "h");
    const double p = real(a[P]);
    const int kind = (int)integer(a[KIND]);
    const bool weights = truth(a[WEIGHTS]);
    at::Tensor dh, dx, dgamma, dbeta, mean, rstd, ws;
    const Matrix md = x.output(on, a[DH], "dh", true, dh), mx = x.output(on, a[DX], "dx", p > 0, dx);
    float *pg = x.floats(on, a[DGAMMA], "dgamma", x.cols, weights, dgamma);
    float *pb = x.floats(on, a[DBETA], "dbeta", x.cols, weights && kind == FP4Q_NORM_LAYER, dbeta);
    int wt = -1;
    const void *gamma = x.weight(a[GAMMA], "gamma", wt);
    const float *pm = x.floats(on, a[MEAN], "mean", x.rows, false, mean);
    const float *ps = static_cast<float *>(x.vector(tensor(a[RSTD], "rstd"), "rstd", x.rows, at::kFloat));
    void *st = stream_of(x.t);
    size_t bytes = 0;
    if (const at::Tensor *w = tensor_or_null(a[WORKSPACE], "workspace")) {
        if (w->device() != x.t.device() || !w->is_contiguous())
            throw Refused("workspace must be a contiguous tensor on dy's device");
        ws = *w;
        bytes = (size_t)w->numel() * w->element_size();
    } else if (pg || pb) {
        bytes = lib.norm_grad_workspace(x.rows, x.cols);
        if (bytes) ws = at::empty({(int64_t)bytes}, x.t.options().dtype(at::kByte));
    }
    const auto rest = [&](auto *fn, auto... h) {
        return fn(my.p, x.rows, x.cols, my.ld, x.type, h..., mr.p, mr.ld, kind, gamma, wt < 0 ? FP4Q_OUT_F32 : wt, pm, ps,
                  (float)p, bits64(a[SEED]), (uint32_t)bits64(a[STREAM_ID]), md.p, md.ld, mx.p, mx.ld, pg, pb,
                  bytes ? ws.data_ptr() : nullptr, bytes, st);
    };
    if constexpr (kPack8)
        done("fp4_norm_grad_pack8", rest(lib.norm_grad_pack8, h8.codes, h8.scales));
    else
        done("fp4_norm_grad", rest(lib.norm_grad, mh.p, mh.ld));
    on.done();
    return results({&dh, &dx, &dgamma, &dbeta});
}

// C: the gate/up output, or with kPack8 its codes (and SCALES).
template <bool kPack8>
PyObject *swiglu_grad(PyObject *const *a)
{
    enum { DH, C, PAIR, WANT_H, DC, H, STREAM, SCALES };
    const Like x(a[DH], "dh");
    OnStream on(a[STREAM], x.t);
    const Matrix mi = x.matrix(x.t, "dh");
    const int64_t M = x.rows, F = x.cols;
    const auto wide = [&](const at::Tensor &t, const char *name) {
        if (x.type != FP4Q_OUT_BF16 || t.scalar_type() != at::kBFloat16 || t.dim() != 2 || t.size(0) != M ||
            t.size(1) < 2 * F || t.device() != x.t.device())
            throw Refused(std::string("dh must be bf16 and ") + name + " a bf16 [" + std::to_string(M) + " x >= " +
                          std::to_string(2 * F) + "] tensor on its device");
        return rows_of(t, name);
    };
    Matrix mc;
    Packed c8{};
    if constexpr (kPack8)
        c8 = packed(a[C], a[SCALES], kCodes, M, 2 * F, x.t);
    else
        mc = wide(tensor(a[C], "c"), "c");
    at::Tensor dc, h;
    if (const at::Tensor *g = tensor_or_null(a[DC], "dc"))
        dc = *g;
    else
        dc = on.empty({M, 2 * F}, x.t.options());
    const Matrix mo = wide(dc, "dc"), mh = x.output(on, a[H], "h", truth(a[WANT_H]), h);
    void *st = stream_of(x.t);
    if constexpr (kPack8)
        done("fp4_swiglu_grad_pack8", lib.swiglu_grad_pack8(mi.p, mi.ld, c8.codes, c8.scales, M, F, integer(a[PAIR]),
                                                            mo.p, mo.ld, mh.p, mh.ld, st));
    else
        done("fp4_swiglu_grad_bf16", lib.swiglu_grad(mi.p, mi.ld, mc.p, M, F, mc.ld, integer(a[PAIR]), mo.p, mo.ld, mh.p,
                                                     mh.ld, st));
    on.done();
    return results({&dc, &h});
}

PyObject *rotary(PyObject *const *a)
{
    enum { X, POSITIONS, FREQ, STYLE, SCALE, INVERSE, Y, STREAM };
    const at::Tensor &x = tensor(a[X], "x");
    const int type = type_of(x);
    if (type < 0 || x.dim() != 3) throw Refused("x must be a [tokens, heads, dim] fp32 or bf16 tensor");
    OnStream on(a[STREAM], x);
    const int64_t n = x.size(0), heads = x.size(1), dim = x.size(2);
    struct Strides {
        int64_t token, head;
    };
    const auto strides = [&](const at::Tensor &t, const char *name) {
        if (t.stride(2) != 1 && dim > 1) throw Refused(std::string(name) + " must have unit stride along dim");
        const int64_t head = heads > 1 ? t.stride(1) : dim;
        return Strides{n > 1 ? t.stride(0) : (heads > 1 ? heads : 1) * head, head};
    };
    const Strides sx = strides(x, "x");
    at::Tensor y;
    if (const at::Tensor *g = tensor_or_null(a[Y], "y")) {
        if (g->sizes() != x.sizes() || g->scalar_type() != x.scalar_type() || g->device() != x.device())
            throw Refused("y must be a tensor of x's shape, type and device");
        y = *g;
    } else {
        y = on.empty(x.sizes(), x.options());
    }
    const Strides sy = strides(y, "y");
    const at::Tensor &pos = tensor(a[POSITIONS], "positions"), &freq = tensor(a[FREQ], "inv_freq");
    const bool wide = pos.scalar_type() == at::kLong;
    if ((!wide && pos.scalar_type() != at::kInt) || pos.numel() != n || pos.device() != x.device() || !pos.is_contiguous())
        throw Refused("positions must be one contiguous int32 or int64 per token on the same device");
    if (freq.scalar_type() != at::kFloat || freq.device() != x.device() || !freq.is_contiguous())
        throw Refused("inv_freq must be contiguous fp32 on the same device");
    void *st = stream_of(x);
    done("fp4_rotary",
         lib.rotary(x.data_ptr(), n, heads, dim, sx.token, sx.head, type, pos.data_ptr(), wide ? 64 : 32,
                    static_cast<const float *>(freq.data_ptr()), 2 * freq.numel(), (int)integer(a[STYLE]),
                    truth(a[INVERSE]) ? 1 : 0, (float)real(a[SCALE]), y.data_ptr(), sy.token, sy.head, st));
    on.done();
    return result(y);
}

PyObject *pack8(PyObject *const *a)
{
    enum { X, CODES, SCALES, STREAM };
    const Like x(a[X], "x");
    OnStream on(a[STREAM], x.t);
    const Matrix mx = x.matrix(x.t, "x");
    at::Tensor keep[2];
    const Packed p = packed(a[CODES], a[SCALES], kCodes, x.rows, x.cols, x.t, &on, keep);
    void *st = stream_of(x.t);
    done("fp4_pack8", lib.pack8(mx.p, x.rows, x.cols, mx.ld, x.type, p.codes, p.scales, st));
    on.done();
    return results({&keep[0], &keep[1]});
}

PyObject *unpack8(PyObject *const *a)
{
    enum { CODES, SCALES, TYPE, Y, STREAM };
    const at::Tensor &codes = tensor(a[CODES], "codes");
    if (codes.dim() != 2) throw Refused("codes must be a 2-D tensor");
    OnStream on(a[STREAM], codes);
    const int64_t rows = codes.size(0), cols = codes.size(1);
    const Packed p = packed(a[CODES], a[SCALES], kCodes, rows, cols, codes);
    at::Tensor y;
    if (const at::Tensor *g = tensor_or_null(a[Y], "y")) {
        if (g->dim() != 2 || g->sizes() != codes.sizes() || type_of(*g) < 0 || g->device() != codes.device())
            throw Refused("y must be an fp32 or bf16 tensor of the codes' shape and device");
        y = *g;
    } else {
        y = on.empty({rows, cols}, codes.options().dtype(integer(a[TYPE]) == FP4Q_OUT_BF16 ? at::kBFloat16 : at::kFloat));
    }
    const Matrix my = rows_of(y, "y");
    void *st = stream_of(codes);
    done("fp4_unpack8", lib.unpack8(p.codes, p.scales, rows, cols, my.p, my.ld, type_of(y), st));
    on.done();
    return result(y);
}

// Products of few rows with FP4 weights.  X: bf16 rows, or where X_SCALES is
// given the codes of 8-bit rows; TENSOR_SCALE is given where the weights are
// NVFP4.  N None: as many as the codes have rows.
PyObject *matvec(PyObject *const *a)
{
    enum { X, X_SCALES, CODES, SCALES, TENSOR_SCALE, DOMAIN, ALPHA, TYPE, LAYOUT, N, Y, STREAM };
    const at::Tensor &x = tensor(a[X], "x"), &codes = tensor(a[CODES], "w_codes"), &scales = tensor(a[SCALES], "w_scales");
    const at::Tensor *ts = tensor_or_null(a[TENSOR_SCALE], "w_tensor_scale");
    const bool packs = a[X_SCALES] != Py_None;
    if (x.dim() != 2 || codes.dim() != 2) throw Refused("x and w_codes must be 2-D tensors");
    if (!packs && x.scalar_type() != at::kBFloat16) throw Refused("x must be bf16");
    OnStream on(a[STREAM], x);
    const int64_t m = x.size(0), k = x.size(1), n = a[N] == Py_None ? codes.size(0) : integer(a[N]);
    if (n < 0 || n > INT32_MAX) throw Refused("n must be the operand's rows");
    const int layout = (int)integer(a[LAYOUT]), domain = (int)integer(a[DOMAIN]);
    const int64_t rows = layout == FP4Q_LAYOUT_TILED ? (n + 31) / 32 * 32 : n;  // of the operand
    dense(codes, "w_codes", at::kByte, {rows, k / 2}, x);
    if (ts) {
        dense(scales, "w_scales", at::kByte, {rows, k / 16}, x);
        const int64_t need = domain == FP4Q_NV_GLOBAL ? 1 : (n + 127) / 128 * (k / 128);
        if (ts->scalar_type() != at::kFloat || ts->numel() != need || ts->device() != x.device() || !ts->is_contiguous())
            throw Refused("w_tensor_scale must be " + std::to_string(need) + " contiguous Float elements on the same device");
    } else if (layout == FP4Q_LAYOUT_TILED) {
        dense(scales, "w_scales", at::kByte, {k / 128, rows, 4}, x);
    } else {
        dense(scales, "w_scales", at::kByte, {rows, k / 32}, x);
    }
    Matrix mx{};
    Packed p{};
    static const char *names[2] = {"x_codes", "x_scales"};
    if (packs)
        p = packed(a[X], a[X_SCALES], names, m, k, x);
    else
        mx = rows_of(x, "x");
    at::Tensor y;
    if (const at::Tensor *g = tensor_or_null(a[Y], "y")) {
        if (g->dim() != 2 || g->size(0) != m || g->size(1) != n || type_of(*g) < 0 || g->device() != x.device())
            throw Refused("y must be an fp32 or bf16 [" + std::to_string(m) + " x " + std::to_string(n) +
                          "] tensor on the same device");
        y = *g;
    } else {
        y = on.empty({m, n}, x.options().dtype(integer(a[TYPE]) == FP4Q_OUT_BF16 ? at::kBFloat16 : at::kFloat));
    }
    const Matrix my = rows_of(y, "y");
    const float alpha = (float)real(a[ALPHA]);
    void *st = stream_of(x);
    if (ts)
        done("fp4_matvec_nv", lib.matvec_nv(mx.p, m, k, mx.ld, codes.data_ptr(), scales.data_ptr(),
                                            static_cast<const float *>(ts->data_ptr()), domain, n, alpha, layout, my.p,
                                            type_of(y), my.ld, st));
    else if (packs)
        done("fp4_matvec_mx_pack8", lib.matvec_mx_pack8(p.codes, p.scales, m, k, codes.data_ptr(), scales.data_ptr(), n,
                                                        alpha, layout, my.p, type_of(y), my.ld, st));
    else
        done("fp4_matvec_mx", lib.matvec_mx(mx.p, m, k, mx.ld, codes.data_ptr(), scales.data_ptr(), n, alpha, layout, my.p,
                                            type_of(y), my.ld, st));
    on.done();
    return result(y);
}

// ---- the module

template <PyObject *(*kCall)(PyObject *const *), Py_ssize_t kArgs>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != kArgs || !lib.norm) {
        PyErr_SetString(PyExc_TypeError, lib.norm ? "wrong number of arguments" : "bind() has not been called");
        return nullptr;
    }
    try {
        return kCall(args);
    } catch (const PythonError &) {
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (...) {  // torch's own, such as memory that its allocator refuses, as torch raises them
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

PyObject *bind(PyObject *, PyObject *args)
{
    unsigned long long f[14];
    PyObject *error, *current, *raw, *external;
    if (!PyArg_ParseTuple(args, "(KKKKKKKKKKKKKK)OOOO", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &f[7], &f[8],
                          &f[9], &f[10], &f[11], &f[12], &f[13], &error, &current, &raw, &external))
        return nullptr;
    Py_INCREF(error);
    Py_INCREF(current);
    Py_INCREF(raw);
    Py_INCREF(external);
    lib.dropout = reinterpret_cast<decltype(lib.dropout)>(f[0]);
    lib.norm = reinterpret_cast<decltype(lib.norm)>(f[1]);
    lib.norm_grad_workspace = reinterpret_cast<decltype(lib.norm_grad_workspace)>(f[2]);
    lib.norm_grad = reinterpret_cast<decltype(lib.norm_grad)>(f[3]);
    lib.swiglu_grad = reinterpret_cast<decltype(lib.swiglu_grad)>(f[4]);
    lib.rotary = reinterpret_cast<decltype(lib.rotary)>(f[5]);
    lib.pack8 = reinterpret_cast<decltype(lib.pack8)>(f[6]);
    lib.unpack8 = reinterpret_cast<decltype(lib.unpack8)>(f[7]);
    lib.norm_pack8 = reinterpret_cast<decltype(lib.norm_pack8)>(f[8]);
    lib.norm_grad_pack8 = reinterpret_cast<decltype(lib.norm_grad_pack8)>(f[9]);
    lib.swiglu_grad_pack8 = reinterpret_cast<decltype(lib.swiglu_grad_pack8)>(f[10]);
    lib.matvec_mx = reinterpret_cast<decltype(lib.matvec_mx)>(f[11]);
    lib.matvec_mx_pack8 = reinterpret_cast<decltype(lib.matvec_mx_pack8)>(f[12]);
    lib.matvec_nv = reinterpret_cast<decltype(lib.matvec_nv)>(f[13]);
    lib.error = error;
    lib.current = current;
    lib.raw = raw;
    lib.external = external;
    Py_RETURN_NONE;
}

template <typename F> PyCFunction method(F *f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, "the library's entry points, Fp4qError, torch's current device and stream, ExternalStream"},
                         {"dropout", method(entry<dropout, 7>), METH_FASTCALL, nullptr},
                         {"norm", method(entry<norm<false>, 19>), METH_FASTCALL, nullptr},
                         {"norm_grad", method(entry<norm_grad<false>, 17>), METH_FASTCALL, nullptr},
                         {"swiglu_grad", method(entry<swiglu_grad<false>, 7>), METH_FASTCALL, nullptr},
                         {"rotary", method(entry<rotary, 8>), METH_FASTCALL, nullptr},
                         {"pack8", method(entry<pack8, 4>), METH_FASTCALL, nullptr},
                         {"unpack8", method(entry<unpack8, 5>), METH_FASTCALL, nullptr},
                         {"norm_pack8", method(entry<norm<true>, 21>), METH_FASTCALL, nullptr},
                         {"norm_grad_pack8", method(entry<norm_grad<true>, 18>), METH_FASTCALL, nullptr},
                         {"swiglu_grad_pack8", method(entry<swiglu_grad<true>, 8>), METH_FASTCALL, nullptr},
                         {"matvec", method(entry<matvec, 12>), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_row_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__row_calls() { return PyModule_Create(&module); }
