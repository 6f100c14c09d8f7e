// Native binding of the quantised-row producers and the MXFP4 product
// (include/w4a4.h): argument checks, output allocation and the call, for
// _lib.py.  A decoder step makes dozens of these calls on a few rows, where
// the kernels take 3 to 6 us each.  Checks and marshalling take 0.3 to 0.4 us a
// call, new outputs 0.7 to 1.0 more, the launch 2.5 to 2.7; checks and allocations
// written in Python took 12 to 14 with it.
//
// Every function takes positional arguments (None for those left out), raises
// the exception type given to init() and lets no C++ exception out.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "w4a4.h"

namespace {

PyObject *g_error = nullptr;  // W4A4Error

struct Refused {
    std::string what;
};
struct PythonError {};  // already set

[[noreturn]] void refuse(const std::string &what) { throw Refused{what}; }

std::string str(int64_t v) { return std::to_string(v); }

// ------------------------------------------------------------- arguments

// A tensor argument (undefined for None).
const at::Tensor &tensor(PyObject *o, const char *name) {
    static const at::Tensor none;
    if (o == Py_None) return none;
    if (!THPVariable_Check(o)) refuse(std::string(name) + ": expected a tensor");
    return THPVariable_Unpack(o);
}
const at::Tensor &required(PyObject *o, const char *name) {
    const at::Tensor &t = tensor(o, name);
    if (!t.defined()) refuse(std::string(name) + " is required");
    return t;
}
const at::Tensor &matrix(PyObject *o, const char *name) {
    const at::Tensor &t = tensor(o, name);
    if (!t.defined() || t.dim() != 2) refuse(std::string(name) + " must be a 2-D matrix");
    return t;
}
int64_t integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}
// The library's own bounds, here so that the sizes computed from k and n fit 64 bits.
int64_t width(int64_t k, const char *more = "") {
    if (k < 0 || k % 32) refuse(more + ("k = " + str(k) + " is not a multiple of 32"));
    if (k > int64_t{1} << 24) refuse("k = " + str(k) + ", at most 2^24");
    return k;
}
int64_t columns(int64_t n) {
    if (n < 0) refuse("n = " + str(n) + " is negative");
    if (n > int64_t{1} << 26) refuse("n = " + str(n) + ", at most 2^26");
    return n;
}
// The k of an optional argument, x's width by default.
int64_t width_of(PyObject *k, const at::Tensor &x) { return width(k == Py_None ? x.size(1) : integer(k)); }

w4a4_dtype row_type(at::ScalarType t, const char *name) {
    if (t == at::kFloat) return W4A4_DTYPE_F32;
    if (t == at::kHalf) return W4A4_DTYPE_F16;
    if (t == at::kBFloat16) return W4A4_DTYPE_BF16;
    refuse(std::string(name) + ": dtype " + c10::toString(t) + ", expected float32, float16 or bfloat16");
}

// t (when defined) has the type, is contiguous and holds at least nbytes.
void need(const at::Tensor &t, const char *name, at::ScalarType type, int64_t nbytes) {
    if (!t.defined()) return;
    if (t.scalar_type() != type)
        refuse(std::string(name) + ": dtype " + c10::toString(t.scalar_type()) + ", expected " + c10::toString(type));
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    const int64_t has = t.numel() * (int64_t)t.element_size();
    if (has < nbytes) refuse(std::string(name) + ": " + str(has) + " bytes, at least " + str(nbytes) + " needed");
}

// t is at least rows x cols of a row type with unit column stride and rows
// that do not overlap; returns its row stride.
int64_t need_rows(const at::Tensor &t, const char *name, int64_t rows, int64_t cols) {
    row_type(t.scalar_type(), name);
    if (t.dim() != 2 || t.size(0) < rows || t.size(1) < cols)
        refuse(std::string(name) + ": shape, expected at least (" + str(rows) + ", " + str(cols) + ")");
    if ((rows > 0 && cols > 1 && t.stride(1) != 1) || (rows > 1 && t.stride(0) < cols))
        refuse(std::string(name) + ": strides (" + str(t.stride(0)) + ", " + str(t.stride(1)) +
               "), expected unit column stride and row stride >= " + str(cols));
    return std::max(t.stride(0), cols);
}

void *ptr(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
size_t bytes(const at::Tensor &t) { return t.defined() ? (size_t)t.numel() * t.element_size() : 0; }

// -------------------------------------------------------- device and call

// The one GPU that every tensor given lives on.
c10::Device one_device(std::initializer_list<const at::Tensor *> ts) {
    const at::Tensor *first = nullptr;
    for (const at::Tensor *t : ts) {
        if (!t->defined()) continue;
        if (!t->is_cuda()) refuse("tensors must live on the GPU");
        if (!first) first = t;
        else if (t->device() != first->device())
            refuse("tensors on " + first->device().str() + " and " + t->device().str() + ", expected one device");
    }
    return first->device();
}

// Makes a device current for its own lifetime, also where that ends by an exception.
class Current {
  public:
    explicit Current(c10::Device device) : before(c10::hip::current_device()), other(before != device.index()) {
        if (other) c10::hip::set_device(device.index());
    }
    ~Current() {
        if (other) (void)c10::hip::MaybeSetDevice(before);  // it was current: no failure to report
    }
    Current(const Current &) = delete;
    Current &operator=(const Current &) = delete;

  private:
    const c10::DeviceIndex before;
    const bool other;
};

// Calls f(stream) with the device current, on its current stream.
template <class F>
void call(const char *name, c10::Device device, F f) {
    const Current current(device);
    const w4a4_status st = f((void *)c10::hip::getCurrentHIPStream(device.index()).stream());
    if (st == W4A4_OK) return;
    const std::string detail = st == W4A4_ERR_HIP ? w4a4_last_hip_error() : "";
    refuse(std::string(name) + ": " + w4a4_status_string(st) + (detail.empty() ? "" : " (" + detail + ")"));
}

// A new tensor from PyTorch's caching allocator (directly: the dispatcher
// would add a third to an allocation's time).
at::Tensor make(c10::IntArrayRef sizes, at::ScalarType type, c10::Device device) {
    return at::Tensor(at::detail::empty_cuda(sizes, type, device, c10::nullopt));
}

// What a call returns for an output: the caller's own object, or the new tensor.
PyObject *give(PyObject *given, const at::Tensor &t) {
    if (given != Py_None) {
        Py_INCREF(given);
        return given;
    }
    return THPVariable_Wrap(t);
}
PyObject *none() {
    Py_INCREF(Py_None);
    return Py_None;
}
PyObject *pack(std::initializer_list<PyObject *> items) {
    PyObject *t = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject *o : items) {
        if (!t || !o) {
            Py_XDECREF(o);
            continue;
        }
        PyTuple_SET_ITEM(t, i++, o);
    }
    if (!t || i < (Py_ssize_t)items.size()) {
        Py_XDECREF(t);
        throw PythonError{};
    }
    return t;
}

// ---------------------------------------------------------------- formats

struct Format {
    w4a4_act_format fmt;
    int64_t m, k;
    at::ScalarType code_type, scale_type;
    int64_t code_cols, scale_cols;
    bool mx4() const { return fmt == W4A4_ACT_MX4 || fmt == W4A4_ACT_MX4_H32; }
};
Format format(int64_t f, int64_t m, int64_t k) {
    switch (f) {
    case W4A4_ACT_INT4:
    case W4A4_ACT_INT4_SMALL: return {(w4a4_act_format)f, m, k, at::kByte, at::kFloat, k / 2, k / 32};
    case W4A4_ACT_INT8: return {W4A4_ACT_INT8, m, k, at::kChar, at::kFloat, k, k / 32};
    case W4A4_ACT_MX4:
    case W4A4_ACT_MX4_H32:
        return {(w4a4_act_format)f, m, k, at::kByte, at::kByte, k / 2, (int64_t)w4a4_mx4_scale_stride(k)};
    }
    refuse("unknown format " + str(f));
}
// A buffer given as a matrix has the format's width: its rows are the format's rows.
void need_width(const at::Tensor &t, const char *name, int64_t cols) {
    if (t.defined() && t.dim() == 2 && t.size(1) != cols)
        refuse(std::string(name) + ": rows of " + str(t.size(1)) + ", expected " + str(cols));
}
void need_codes(const Format &f, const at::Tensor &codes, const at::Tensor &scales) {
    need(codes, "codes", f.code_type, f.m * f.code_cols);
    need(scales, "scales", f.scale_type, f.m * f.scale_cols * (f.scale_type == at::kFloat ? 4 : 1));
    need_width(codes, "codes", f.code_cols);
    need_width(scales, "scales", f.scale_cols);
}
void check_outputs(const Format &f, const at::Tensor &codes, const at::Tensor &scales, const at::Tensor &operand) {
    if (f.fmt == W4A4_ACT_INT4_SMALL && f.m > 16) refuse("ACT_INT4_SMALL: " + str(f.m) + " rows (at most 16)");
    need_codes(f, codes, scales);
    if (!operand.defined()) return;
    if (f.mx4()) refuse("operand: MXFP4 rows have none");
    need(operand, "operand", at::kByte, (int64_t)w4a4_act_format_operand_bytes(f.fmt, f.m, f.k));
}
void make_outputs(const Format &f, at::Tensor &codes, at::Tensor &scales, at::Tensor *operand, c10::Device device) {
    if (!codes.defined()) codes = make({f.m, f.code_cols}, f.code_type, device);
    if (!scales.defined()) scales = make({f.m, f.scale_cols}, f.scale_type, device);
    if (operand && !operand->defined() && f.fmt == W4A4_ACT_INT4_SMALL)
        *operand = make({(int64_t)w4a4_act_format_operand_bytes(f.fmt, f.m, f.k)}, at::kByte, device);
}

// -------------------------------------------------------------- the calls

// x, rotate, k, codes, scales -> (codes, scales)
PyObject *quantize_mx4(PyObject *const *a) {
    const at::Tensor &x = matrix(a[0], "x");
    const int rotate = PyObject_IsTrue(a[1]);
    if (rotate < 0) throw PythonError{};
    const w4a4_dtype dt = row_type(x.scalar_type(), "x");
    const int64_t m = x.size(0), k = width_of(a[2], x), ldx = need_rows(x, "x", m, k);
    at::Tensor codes = tensor(a[3], "codes"), scales = tensor(a[4], "scales");
    const Format f = format(rotate ? W4A4_ACT_MX4_H32 : W4A4_ACT_MX4, m, k);
    need_codes(f, codes, scales);
    const c10::Device device = one_device({&x, &codes, &scales});
    make_outputs(f, codes, scales, nullptr, device);
    call("w4a4_quantize_mx4", device, [&](void *s) {
        return w4a4_quantize_mx4(ptr(x), dt, m, k, ldx, rotate, (uint8_t *)ptr(codes), (uint8_t *)ptr(scales), s);
    });
    return pack({give(a[3], codes), give(a[4], scales)});
}

// codes, scales, k, fmt, out, dtype -> out
PyObject *dequantize_act(PyObject *const *a) {
    const at::Tensor &codes = matrix(a[0], "codes"), &scales = required(a[1], "scales");
    const int64_t m = codes.size(0), k = width(integer(a[2]));
    const Format f = format(integer(a[3]), m, k);
    need_codes(f, codes, scales);
    at::Tensor out = tensor(a[4], "out");
    at::ScalarType type;
    if (out.defined()) {
        type = out.scalar_type();
        need_rows(out, "out", m, k);
    } else {
        if (!THPDtype_Check(a[5])) refuse("dtype: expected a torch.dtype");
        type = reinterpret_cast<THPDtype *>(a[5])->scalar_type;
    }
    const w4a4_dtype dt = row_type(type, "dtype");
    const c10::Device device = one_device({&codes, &scales, &out});
    if (!out.defined()) out = make({m, k}, type, device);
    const int64_t ld = std::max(out.stride(0), k);
    call("w4a4_dequantize_act", device,
         [&](void *s) { return w4a4_dequantize_act(f.fmt, ptr(codes), ptr(scales), m, k, ptr(out), dt, ld, s); });
    return give(a[4], out);
}

// x, weight, eps, fmt, residual, h, codes, scales, operand -> (codes, scales, h or None)
PyObject *rms_norm_quantize(PyObject *const *a) {
    const at::Tensor &x = matrix(a[0], "x"), &weight = tensor(a[1], "weight"), &residual = tensor(a[4], "residual");
    const double eps = PyFloat_AsDouble(a[2]);
    if (eps == -1.0 && PyErr_Occurred()) throw PythonError{};
    const int64_t m = x.size(0), k = width(x.size(1));
    const Format f = format(integer(a[3]), m, k);
    at::Tensor h = tensor(a[5], "h"), codes = tensor(a[6], "codes"), scales = tensor(a[7], "scales"),
               operand = tensor(a[8], "operand");
    const w4a4_dtype xdt = row_type(x.scalar_type(), "x");
    const int64_t ldx = need_rows(x, "x", m, k);
    const at::Tensor &held = residual.defined() ? residual : h.defined() ? h : x;
    const w4a4_dtype rdt = row_type(held.scalar_type(), residual.defined() ? "residual" : "h");
    const int64_t ldr = residual.defined() ? need_rows(residual, "residual", m, k) : 0;
    int64_t ldh = h.defined() ? need_rows(h, "h", m, k) : k;
    if (h.defined() && h.scalar_type() != held.scalar_type())
        refuse(std::string("h: dtype ") + c10::toString(h.scalar_type()) + ", expected the residual's " +
               c10::toString(held.scalar_type()));
    need(weight, "weight", at::kFloat, 4 * k);
    if (!(eps > 0.0) || !std::isfinite(eps)) refuse("eps = " + std::to_string(eps) + ", expected a positive number");
    check_outputs(f, codes, scales, operand);
    const c10::Device device = one_device({&x, &weight, &residual, &h, &codes, &scales, &operand});
    make_outputs(f, codes, scales, &operand, device);
    if (!h.defined() && residual.defined()) h = make({m, k}, held.scalar_type(), device);
    call("w4a4_rms_norm_quantize", device, [&](void *s) {
        return w4a4_rms_norm_quantize(ptr(x), xdt, ldx, ptr(residual), rdt, ldr, (const float *)ptr(weight), eps, m, k,
                                      ptr(h), ldh, f.fmt, ptr(codes), ptr(scales), ptr(operand), bytes(operand), s);
    });
    return pack({give(a[6], codes), give(a[7], scales), h.defined() ? give(a[5], h) : none()});
}

// gate, up, fmt, act, k, codes, scales, operand -> (codes, scales)
PyObject *glu_quantize(PyObject *const *a) {
    const at::Tensor &gate = matrix(a[0], "gate"), &up = matrix(a[1], "up");
    const int64_t act = integer(a[3]);
    if (act != W4A4_GLU_SILU && act != W4A4_GLU_GELU_TANH) refuse("unknown activation " + str(act));
    const int64_t m = gate.size(0), k = width_of(a[4], gate);
    const Format f = format(integer(a[2]), m, k);
    at::Tensor codes = tensor(a[5], "codes"), scales = tensor(a[6], "scales"), operand = tensor(a[7], "operand");
    const w4a4_dtype dt = row_type(gate.scalar_type(), "gate");
    const int64_t ldg = need_rows(gate, "gate", m, k), ldu = need_rows(up, "up", m, k);
    if (up.scalar_type() != gate.scalar_type())
        refuse(std::string("up: dtype ") + c10::toString(up.scalar_type()) + ", expected the gate's " +
               c10::toString(gate.scalar_type()));
    check_outputs(f, codes, scales, operand);
    const c10::Device device = one_device({&gate, &up, &codes, &scales, &operand});
    make_outputs(f, codes, scales, &operand, device);
    call("w4a4_glu_quantize", device, [&](void *s) {
        return w4a4_glu_quantize(ptr(gate), ptr(up), dt, m, k, ldg, ldu, (w4a4_glu_act)act, f.fmt, ptr(codes), ptr(scales),
                                 ptr(operand), bytes(operand), s);
    });
    return pack({give(a[5], codes), give(a[6], scales)});
}

// codes, scales, n, k, out -> out
PyObject *repack_mx4(PyObject *const *a) {
    const at::Tensor &codes = required(a[0], "codes"), &scales = required(a[1], "scales");
    const int64_t n = columns(integer(a[2])), k = width(integer(a[3]));
    need_codes(format(W4A4_ACT_MX4, n, k), codes, scales);
    at::Tensor out = tensor(a[4], "out");
    const int64_t size = (int64_t)w4a4_mx4_packed_bytes(n, k);
    need(out, "out", at::kByte, size);
    const c10::Device device = one_device({&codes, &scales, &out});
    if (!out.defined()) out = make({size}, at::kByte, device);
    call("w4a4_repack_mx4", device, [&](void *s) {
        return w4a4_repack_mx4((const uint8_t *)ptr(codes), (const uint8_t *)ptr(scales), n, k, ptr(out), s);
    });
    return give(a[4], out);
}

// packed, codes, scales, n, k, y, workspace, dtype -> y
PyObject *gemm_mx4(PyObject *const *a) {
    const at::Tensor &packed = required(a[0], "packed"), &codes = matrix(a[1], "codes"), &scales = required(a[2], "scales");
    const int64_t m = codes.size(0), k = width(integer(a[4]), "codes must be rows of whole blocks: "), n = columns(integer(a[3]));
    need(packed, "packed", at::kByte, m && n ? (int64_t)w4a4_mx4_packed_bytes(n, k) : 0);
    need_codes(format(W4A4_ACT_MX4, m, k), codes, scales);
    at::Tensor y = tensor(a[5], "y"), workspace = tensor(a[6], "workspace");
    at::ScalarType type;
    if (y.defined()) {
        type = y.scalar_type();
        need_rows(y, "y", m, n);
    } else {
        if (!THPDtype_Check(a[7])) refuse("dtype: expected a torch.dtype");
        type = reinterpret_cast<THPDtype *>(a[7])->scalar_type;
    }
    const w4a4_dtype dt = row_type(type, "y");
    const int64_t size = (int64_t)w4a4_gemm_mx4_workspace_bytes(m, n, k);
    need(workspace, "workspace", at::kByte, size);
    const c10::Device device = one_device({&packed, &codes, &scales, &y, &workspace});
    if (!y.defined()) y = make({m, n}, type, device);
    if (!workspace.defined() && size) workspace = make({size}, at::kByte, device);
    const int64_t ldy = std::max(y.stride(0), n);
    call("w4a4_gemm_mx4", device, [&](void *s) {
        return w4a4_gemm_mx4(ptr(packed), (const uint8_t *)ptr(codes), (const uint8_t *)ptr(scales), ptr(y), dt, m, n, k, ldy,
                             ptr(workspace), bytes(workspace), s);
    });
    return give(a[5], y);
}

// ----------------------------------------------------------------- module

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused &r) {
        PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, r.what.c_str());
    } catch (const PythonError &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

PyObject *init(PyObject *, PyObject *error) {
    Py_INCREF(error);
    Py_XDECREF(g_error);
    g_error = error;
    return none();
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
constexpr PyMethodDef method(const char *name) {
    return {name, (PyCFunction)(void *)entry<F, N>, METH_FASTCALL, nullptr};
}
PyMethodDef kMethods[] = {method<quantize_mx4, 5>("quantize_mx4"),
                          method<dequantize_act, 6>("dequantize_act"),
                          method<rms_norm_quantize, 9>("rms_norm_quantize"),
                          method<glu_quantize, 8>("glu_quantize"),
                          method<repack_mx4, 5>("repack_mx4"),
                          method<gemm_mx4, 8>("gemm_mx4"),
                          {"init", init, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&kModule); }
