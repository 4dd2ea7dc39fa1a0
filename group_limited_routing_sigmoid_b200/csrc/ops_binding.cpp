// Python binding of the handle-free operators: what ops.py's functions do on
// every call -- the checks of tensors, the outputs, the current stream -- beside
// kernels of a few microseconds (in Python these took 5 to 10 us a call,
// here about 1).  The operators themselves are the C functions of beam_ops.h,
// whose addresses ops.py hands over once (bind).
//
// Every function runs on the device and the current stream of its first
// tensor's device.  Types and shapes that do not fit raise TypeError, values
// and devices ValueError, refusals of the library BeamMoEError.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "beam_ops.h"

namespace {

struct Library {
    decltype(&beam_rms_norm) rms_norm;
    decltype(&beam_mx_tensor_scale) tensor_scale;
    decltype(&beam_mx_quantize) quantize;
    decltype(&beam_mx_quantize_nvfp4) quantize_nvfp4;
    decltype(&beam_mx_dequantize) dequantize;
    decltype(&beam_mx_tile_scales) tile_scales;
    decltype(&beam_mx_matmul) matmul;
    decltype(&beam_route_scores) route;
    decltype(&beam_ops_error) error;
} lib;

// BeamMoEError, NormResult and MxTensor (named tuples)
PyObject *beam_error = nullptr;
PyTypeObject *norm_result = nullptr, *mx_tensor = nullptr;

// A Python exception is set.
struct Raised {};

[[noreturn]] void raise_type(const char *fmt, const std::string &a, const std::string &b)
{
    PyErr_Format(PyExc_TypeError, fmt, a.c_str(), b.c_str());
    throw Raised{};
}

[[noreturn]] void raise_beam(int code, const char *text)
{
    PyObject *e = PyObject_CallFunction(beam_error, "is", code, text);
    if (e) {
        PyErr_SetObject(beam_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

void check(int rc)
{
    if (rc != BEAM_OK) raise_beam(rc, lib.error());
}

long long integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}

int small_integer(PyObject *o)
{
    const long long v = integer(o);
    if (v < INT_MIN || v > INT_MAX) {
        PyErr_SetString(PyExc_ValueError, "an integer argument is out of range");
        throw Raised{};
    }
    return (int)v;
}

float real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return (float)v;
}

std::string shape_of(const at::Tensor &t)
{
    const auto list = [](at::IntArrayRef v) {
        std::string s = "[";
        for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
        return s + "]";
    };
    return std::string(toString(t.scalar_type())) + " " + list(t.sizes()) + ", strides " + list(t.strides());
}

// A CUDA tensor, on `device` unless that is null.
const at::Tensor &tensor(PyObject *o, const char *name, const at::Tensor *first)
{
    if (!THPVariable_Check(o)) raise_type("%s: expected a CUDA tensor, got %s", name, Py_TYPE(o)->tp_name);
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) raise_type("%s: expected a CUDA tensor, got one on %s", name, t.device().str());
    if (first && t.device() != first->device()) {
        PyErr_Format(PyExc_ValueError, "%s: on %s, the others on %s", name, t.device().str().c_str(),
                     first->device().str().c_str());
        throw Raised{};
    }
    return t;
}

int dtype_code(at::ScalarType t)
{
    return t == at::kBFloat16 ? BEAM_BF16 : t == at::kHalf ? BEAM_F16 : t == at::kFloat ? BEAM_F32 : -1;
}

at::ScalarType scalar_type(int code) { return code == BEAM_BF16 ? at::kBFloat16 : code == BEAM_F16 ? at::kHalf : at::kFloat; }

// A matrix of a supported type whose rows are contiguous.
struct Rows {
    void *p = nullptr;
    long long rows = 0, cols = 0, ld = 0;
    int code = -1;
    Rows() = default;
    Rows(const at::Tensor &t, const char *name)
    {
        code = dtype_code(t.scalar_type());
        if (code < 0) raise_type("%s: expected torch.bfloat16, torch.float16 or torch.float32, got %s", name, shape_of(t));
        if (t.dim() != 2 || t.layout() != at::kStrided || (t.size(1) > 1 && t.stride(1) != 1))
            raise_type("%s: expected a matrix with contiguous rows, got %s", name, shape_of(t));
        rows = t.size(0), cols = t.size(1);
        ld = rows <= 1 ? cols : t.stride(0);
        if (ld < cols) raise_type("%s: rows overlap, got %s", name, shape_of(t));
        p = t.data_ptr();
    }
    int columns(const char *name) const
    {
        if (cols > INT_MAX) raise_type("%s: %s", name, "too many columns");
        return (int)cols;
    }
    int height(const char *name) const
    {
        if (rows > INT_MAX) raise_type("%s: %s", name, "too many rows");
        return (int)rows;
    }
};

// A new tensor on first's device: the CUDA allocation itself, half the time of
// the dispatched at::empty.
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor &first)
{
    return at::Tensor(at::detail::empty_cuda(sizes, type, first.device(), c10::nullopt));
}

// An output matrix: the caller's (checked) or a new one.
at::Tensor output(PyObject *given, const char *name, long long rows, long long cols, int code, const at::Tensor &first,
                  Rows &r)
{
    if (given == Py_None) {
        at::Tensor t = fresh({rows, cols}, scalar_type(code), first);
        r.p = t.data_ptr(), r.rows = rows, r.cols = cols, r.ld = cols, r.code = code;
        return t;
    }
    const at::Tensor &t = tensor(given, name, &first);
    r = Rows(t, name);
    if (r.rows != rows || r.cols != cols || r.code != code)
        raise_type("%s: got %s", name,
                   shape_of(t) + " where " + toString(scalar_type(code)) + " [" + std::to_string(rows) + ", " +
                       std::to_string(cols) + "] is expected");
    return t;
}

// A contiguous tensor of n elements of a type.
template <typename T>
T *flat(PyObject *o, const char *name, at::ScalarType type, long long n, const at::Tensor *first)
{
    const at::Tensor &t = tensor(o, name, first);
    if (t.scalar_type() != type || t.numel() != n || !t.is_contiguous())
        raise_type("%s: got %s", name,
                   shape_of(t) + " where " + std::to_string(n) + " contiguous elements of " + toString(type) + " are expected");
    return static_cast<T *>(t.data_ptr());
}

template <typename T>
T *flat_or_null(PyObject *o, const char *name, at::ScalarType type, long long n, const at::Tensor *first)
{
    return o == Py_None ? nullptr : flat<T>(o, name, type, n, first);
}

// The current device set to the tensors', and its current stream.
struct On {
    c10::cuda::OptionalCUDAGuard guard;
    void *stream;
    explicit On(const at::Tensor &t)
    {
        if (t.get_device() != c10::cuda::current_device()) guard.set_device(t.device());
        stream = c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
    }
};

long long block(int format) { return format == BEAM_NVFP4 ? 16 : 32; }

long long scale_count(int format, long long rows, long long K, int layout)
{
    if (rows < 0 || K <= 0 || K % block(format) || rows > (1ll << 60) / K) {
        char text[160];
        snprintf(text, sizeof(text), "K must be a positive multiple of %lld, rows >= 0 and both fit memory, got %lld x %lld",
                 block(format), rows, K);
        raise_beam(BEAM_ERR_INVALID_ARG, text);
    }
    const long long n = K / block(format);
    return layout == BEAM_SCALES_ROWS ? rows * n : (rows + 127) / 128 * ((n + 3) / 4) * 512;
}

long long code_bytes(int format, long long rows, long long K) { return format == BEAM_MXFP8 ? rows * K : rows * (K / 2); }

struct Operand {
    at::Tensor codes, scales;
    uint8_t *c = nullptr, *s = nullptr;
};

// Codes and scales to write: the caller's (checked) or new ones.
Operand new_operand(PyObject *codes, PyObject *scales, int format, int layout, long long rows, long long K,
                    const at::Tensor &first)
{
    Operand o;
    const long long n = scale_count(format, rows, K, layout);
    if (codes == Py_None) {
        o.codes = fresh({rows, format == BEAM_MXFP8 ? K : K / 2}, at::kByte, first);
        o.scales = layout == BEAM_SCALES_ROWS ? fresh({rows, K / block(format)}, at::kByte, first) : fresh({n}, at::kByte, first);
        o.c = static_cast<uint8_t *>(o.codes.data_ptr());
        o.s = static_cast<uint8_t *>(o.scales.data_ptr());
    } else {
        o.c = flat<uint8_t>(codes, "codes", at::kByte, code_bytes(format, rows, K), &first);
        o.s = flat<uint8_t>(scales, "scales", at::kByte, n, &first);
        o.codes = THPVariable_Unpack(codes), o.scales = THPVariable_Unpack(scales);
    }
    return o;
}

// The fields of an MxTensor, format and layout as the library's codes.
struct Fields {
    PyObject *codes, *scales, *tensor_scale;
    int format, layout;
    long long rows, K;
};

int choice(PyObject *o, const char *name, std::initializer_list<const char *> names)
{
    int i = 0;
    if (PyUnicode_Check(o))
        for (const char *n : names) {
            if (PyUnicode_CompareWithASCIIString(o, n) == 0) return i;
            ++i;
        }
    std::string all;
    for (const char *n : names) all += std::string(all.empty() ? "" : ", ") + n;
    PyErr_Format(PyExc_ValueError, "%s: expected one of %s, got %R", name, all.c_str(), o);
    throw Raised{};
}

Fields fields(PyObject *o, const char *name)
{
    if (!PyObject_TypeCheck(o, mx_tensor) || PyTuple_GET_SIZE(o) != 7)
        raise_type("%s: expected an MxTensor, got %s", name, Py_TYPE(o)->tp_name);
    PyObject **f = &PyTuple_GET_ITEM(o, 0);
    return {f[0], f[1], f[6], choice(f[2], name, {"nvfp4", "mxfp4", "mxfp8"}), choice(f[3], name, {"rows", "tiled"}),
            integer(f[4]), integer(f[5])};
}

int fits(long long v, const char *name)
{
    if (v < INT_MIN || v > INT_MAX) {
        PyErr_Format(PyExc_ValueError, "%s: a size is out of range", name);
        throw Raised{};
    }
    return (int)v;
}

PyObject *wrap_or_none(const at::Tensor &t)
{
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject *none()
{
    Py_INCREF(Py_None);
    return Py_None;
}

PyObject *same(PyObject *o)
{
    Py_INCREF(o);
    return o;
}

// A tuple, or one of the named ones.  Steals the references of `items`.
PyObject *pack(std::initializer_list<PyObject *> items, PyTypeObject *type = nullptr)
{
    PyObject *t = type ? type->tp_alloc(type, (Py_ssize_t)items.size()) : PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject *o : items) {
        if (!o || !t) {
            for (; i < (Py_ssize_t)items.size(); ++i) Py_XDECREF(items.begin()[i]);
            Py_XDECREF(t);
            throw Raised{};
        }
        PyTuple_SET_ITEM(t, i++, o);
    }
    return t;
}

void need(Py_ssize_t got, Py_ssize_t want)
{
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
        throw Raised{};
    }
}

// No exception of C++ leaves an entry point.
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        return F(a, n);
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// The MxTensor of an operand; format and layout are given as the strings it holds.
PyObject *pack_operand(const Operand &q, PyObject *format, PyObject *layout, long long rows, long long K, const at::Tensor &scale)
{
    return pack({THPVariable_Wrap(q.codes), THPVariable_Wrap(q.scales), same(format), same(layout), PyLong_FromLongLong(rows),
                 PyLong_FromLongLong(K), wrap_or_none(scale)},
                mx_tensor);
}

// x, gamma, residual, alpha, beta, eps, dtype, quantize (None or the format's name), layout, its name, out,
// residual_out, want_out, codes, scales -> NormResult
PyObject *rms_norm(PyObject *const *a, Py_ssize_t n)
{
    need(n, 15);
    const at::Tensor &x = tensor(a[0], "x", nullptr);
    const Rows xr(x, "x");
    const int T = xr.height("x"), H = xr.columns("x"), dtype = small_integer(a[6]), layout = small_integer(a[8]);
    const bool quantize = a[7] != Py_None, want_out = a[12] == Py_True;
    Rows r, ro, o;
    at::Tensor residual_out, out;
    const On on(x);
    const float *gamma = flat<float>(a[1], "gamma", at::kFloat, H, &x);
    if (a[2] != Py_None) {
        const at::Tensor &t = tensor(a[2], "residual", &x);
        r = Rows(t, "residual");
        if (r.rows != T || r.cols != H || (r.code != BEAM_F32 && r.code != xr.code))
            raise_type("%s: expected x's shape in fp32 or x's type, got %s", "residual", shape_of(t));
        residual_out = output(a[11], "residual_out", T, H, r.code, x, ro);
    }
    if (want_out) out = output(a[10], "out", T, H, dtype, x, o);
    Operand q;
    if (quantize) q = new_operand(a[13], a[14], BEAM_MXFP8, layout, T, H, x);
    check(lib.rms_norm(on.stream, xr.p, xr.code, xr.ld, r.p, r.code, r.ld, ro.p, ro.ld, real(a[3]), real(a[4]), gamma,
                       real(a[5]), T, H, o.p, dtype, o.ld, q.c, q.s, layout));
    PyObject *operand = quantize ? pack_operand(q, a[7], a[9], T, H, at::Tensor()) : none();
    return pack({wrap_or_none(out), wrap_or_none(residual_out), operand}, norm_result);
}

// x, out -> out
PyObject *tensor_scale(PyObject *const *a, Py_ssize_t n)
{
    need(n, 2);
    const at::Tensor &x = tensor(a[0], "x", nullptr);
    const Rows r(x, "x");
    const On on(x);
    at::Tensor out;
    if (a[1] == Py_None) {
        out = fresh({1}, at::kFloat, x);
    } else {
        flat<float>(a[1], "out", at::kFloat, 1, &x);
        out = THPVariable_Unpack(a[1]);
    }
    check(lib.tensor_scale(on.stream, r.p, r.code, r.rows, r.columns("x"), r.ld, static_cast<float *>(out.data_ptr())));
    return THPVariable_Wrap(out);
}

// x, format, layout, tensor_scale, codes, scales, the format's and the layout's names -> MxTensor
PyObject *quantize(PyObject *const *a, Py_ssize_t n)
{
    need(n, 8);
    const at::Tensor &x = tensor(a[0], "x", nullptr);
    const Rows r(x, "x");
    const int format = small_integer(a[1]), layout = small_integer(a[2]);
    const On on(x);
    Operand q = new_operand(a[4], a[5], format, layout, r.rows, r.cols, x);
    const int K = r.columns("x");
    at::Tensor scale;
    if (format == BEAM_NVFP4 && a[3] == Py_None) {
        scale = fresh({1}, at::kFloat, x);
        check(lib.quantize_nvfp4(on.stream, r.p, r.code, r.rows, K, r.ld, layout, static_cast<float *>(scale.data_ptr()), q.c, q.s));
    } else {
        const float *g = format == BEAM_NVFP4 ? flat<float>(a[3], "tensor_scale", at::kFloat, 1, &x) : nullptr;
        if (g) scale = THPVariable_Unpack(a[3]);
        check(lib.quantize(on.stream, r.p, r.code, r.rows, K, r.ld, format, layout, g, q.c, q.s));
    }
    return pack_operand(q, a[6], a[7], r.rows, r.cols, scale);
}

// MxTensor, dtype, out -> out
PyObject *dequantize(PyObject *const *a, Py_ssize_t n)
{
    need(n, 3);
    const Fields q = fields(a[0], "q");
    const int K = fits(q.K, "q"), dtype = small_integer(a[1]);
    const at::Tensor &codes = tensor(q.codes, "codes", nullptr);
    const long long ns = scale_count(q.format, q.rows, K, q.layout);
    const uint8_t *c = flat<uint8_t>(q.codes, "codes", at::kByte, code_bytes(q.format, q.rows, K), nullptr);
    const uint8_t *s = flat<uint8_t>(q.scales, "scales", at::kByte, ns, &codes);
    const float *g = flat_or_null<float>(q.tensor_scale, "tensor_scale", at::kFloat, 1, &codes);
    const On on(codes);
    Rows o;
    at::Tensor out = output(a[2], "out", q.rows, K, dtype, codes, o);
    check(lib.dequantize(on.stream, c, s, g, q.format, q.layout, q.rows, K, o.p, dtype, o.ld));
    return THPVariable_Wrap(out);
}

// scales, format, rows, K -> tiled scales
PyObject *tile_scales(PyObject *const *a, Py_ssize_t n)
{
    need(n, 4);
    const int format = small_integer(a[1]);
    const long long rows = integer(a[2]);
    const int K = small_integer(a[3]);
    const at::Tensor &scales = tensor(a[0], "scales", nullptr);
    const uint8_t *s = flat<uint8_t>(a[0], "scales", at::kByte, scale_count(format, rows, K, BEAM_SCALES_ROWS), nullptr);
    const On on(scales);
    at::Tensor out = fresh({scale_count(format, rows, K, BEAM_SCALES_TILED)}, at::kByte, scales);
    check(lib.tile_scales(on.stream, format, s, rows, K, static_cast<uint8_t *>(out.data_ptr())));
    return THPVariable_Wrap(out);
}

// MxTensor a, MxTensor w, dtype, out -> out
PyObject *matmul(PyObject *const *a, Py_ssize_t n)
{
    need(n, 4);
    const Fields x = fields(a[0], "a"), w = fields(a[1], "w");
    if (x.layout != BEAM_SCALES_TILED || w.layout != BEAM_SCALES_TILED) {
        PyErr_SetString(PyExc_ValueError, "mx_matmul takes scales in the tiled layout (mx_tile_scales)");
        throw Raised{};
    }
    if (x.K != w.K) {
        PyErr_Format(PyExc_ValueError, "a has %lld columns, w %lld", x.K, w.K);
        throw Raised{};
    }
    const int T = fits(x.rows, "a"), N = fits(w.rows, "w"), K = fits(x.K, "a"), dtype = small_integer(a[2]);
    const at::Tensor &first = tensor(x.codes, "a.codes", nullptr);
    const long long x_scales = scale_count(x.format, T, K, BEAM_SCALES_TILED), w_scales = scale_count(w.format, N, K, BEAM_SCALES_TILED);
    const uint8_t *xc = flat<uint8_t>(x.codes, "a.codes", at::kByte, code_bytes(x.format, T, K), nullptr);
    const uint8_t *xs = flat<uint8_t>(x.scales, "a.scales", at::kByte, x_scales, &first);
    const float *xg = flat_or_null<float>(x.tensor_scale, "a.tensor_scale", at::kFloat, 1, &first);
    const uint8_t *wc = flat<uint8_t>(w.codes, "w.codes", at::kByte, code_bytes(w.format, N, K), &first);
    const uint8_t *ws = flat<uint8_t>(w.scales, "w.scales", at::kByte, w_scales, &first);
    const float *wg = flat_or_null<float>(w.tensor_scale, "w.tensor_scale", at::kFloat, 1, &first);
    const On on(first);
    Rows o;
    at::Tensor out = output(a[3], "out", T, N, dtype, first, o);
    check(lib.matmul(on.stream, x.format, xc, xs, xg, w.format, wc, ws, wg, T, N, K, o.p, dtype, o.ld));
    return THPVariable_Wrap(out);
}

// logits, top_k, score, bias, n_group, topk_group, group_top, renormalize, scale, idx, w -> idx, w
PyObject *route_scores(PyObject *const *a, Py_ssize_t n)
{
    need(n, 11);
    const at::Tensor &l = tensor(a[0], "logits", nullptr);
    const Rows r(l, "logits");
    if (r.code != BEAM_F32) raise_type("%s: expected torch.float32, got %s", "logits", shape_of(l));
    const int T = r.height("logits"), E = r.columns("logits"), top_k = small_integer(a[1]);
    const bool refused = top_k < 1 || top_k > 32;   // by the library, before any output is made
    const long long k = refused ? 0 : top_k;
    const On on(l);
    const float *bias = flat_or_null<float>(a[3], "bias", at::kFloat, E, &l);
    at::Tensor idx, w;
    if (refused || a[9] == Py_None) {
        idx = fresh({T, k}, at::kInt, l);
    } else {
        flat<int32_t>(a[9], "idx", at::kInt, T * k, &l);
        idx = THPVariable_Unpack(a[9]);
    }
    if (refused || a[10] == Py_None) {
        w = fresh({T, k}, at::kFloat, l);
    } else {
        flat<float>(a[10], "w", at::kFloat, T * k, &l);
        w = THPVariable_Unpack(a[10]);
    }
    const int renormalize = PyObject_IsTrue(a[7]);
    if (renormalize < 0) throw Raised{};
    check(lib.route(on.stream, static_cast<const float *>(r.p), T, E, r.ld, small_integer(a[2]), bias, small_integer(a[4]),
                    small_integer(a[5]), small_integer(a[6]), top_k, renormalize, real(a[8]),
                    static_cast<int32_t *>(idx.data_ptr()), static_cast<float *>(w.data_ptr())));
    return pack({THPVariable_Wrap(idx), THPVariable_Wrap(w)});
}

// BeamMoEError, NormResult, MxTensor, then the addresses of the library's functions in Library's order
PyObject *bind(PyObject *const *a, Py_ssize_t n)
{
    constexpr Py_ssize_t types = 3, functions = sizeof(Library) / sizeof(void *);
    need(n, types + functions);
    for (Py_ssize_t i = 1; i < types; ++i)
        if (!PyType_Check(a[i]) || !PyType_IsSubtype(reinterpret_cast<PyTypeObject *>(a[i]), &PyTuple_Type))
            raise_type("%s: %s", "bind", "expected types of tuples");
    void *p[functions];
    for (Py_ssize_t i = 0; i < functions; ++i) p[i] = reinterpret_cast<void *>(integer(a[types + i]));
    memcpy(&lib, p, sizeof(lib));
    for (Py_ssize_t i = 0; i < types; ++i) Py_INCREF(a[i]);   // for good
    beam_error = a[0];
    norm_result = reinterpret_cast<PyTypeObject *>(a[1]);
    mx_tensor = reinterpret_cast<PyTypeObject *>(a[2]);
    Py_RETURN_NONE;
}

#define BEAM_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {BEAM_METHOD(bind),       BEAM_METHOD(rms_norm),    BEAM_METHOD(tensor_scale),
                         BEAM_METHOD(quantize),   BEAM_METHOD(dequantize),  BEAM_METHOD(tile_scales),
                         BEAM_METHOD(matmul),     BEAM_METHOD(route_scores), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyMODINIT_FUNC PyInit__ops_binding(void) { return PyModule_Create(&module); }
