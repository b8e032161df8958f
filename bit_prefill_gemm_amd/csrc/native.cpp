// native.cpp -- the Python entry points of the operators between the products
// (rmsnorm_quantize_act, dequantize_act, w4a4_gemm_epilogue, moe_route_topk),
// of the 8-bit floating-point route (quantize_fp8, fp8_gemm, fp8_gemm_gated,
// fp8_gemm_gated_quantize) and of token_logprobs, compiled: their tensor checks,
// output allocation and the call of the C ABI
// (include/bpg.h).  Host code only; every step of the operators runs in
// libbpg.so's kernels.
//
// Why compiled: these calls come between the products of one token, where a
// kernel takes 2 to 7 us.  The same checks and allocations in Python, and the
// call through ctypes with its 18 arguments, took 11 to 13 us of host time a
// call (MI355X host).
//
// The C ABI sees only pointers and sizes, so a tensor of the wrong shape would
// become an out-of-bounds device access: every tensor is checked here first,
// shapes, types, layouts and overlaps before devices, so that every such error
// is reported the same way with or without a GPU.
#include <torch/csrc/python_headers.h>

#include <ATen/hip/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdarg>
#include <string>

#include "bpg.h"

namespace {

PyObject *g_error; // BpgError

// an argument that the call refuses (ValueError)
struct Refusal {
    std::string text;
};

[[noreturn]] void fail(const char *where, const char *format, ...)
{
    char text[400];
    va_list args;
    va_start(args, format);
    vsnprintf(text, sizeof text, format, args);
    va_end(args);
    throw Refusal{std::string(where) + ": " + text};
}

// a Python error is already set
struct Raised {};

template <class F>
PyObject *guarded(F &&body)
{
    HANDLE_TH_ERRORS
    try {
        return body();
    } catch (const Refusal &r) {
        PyErr_SetString(PyExc_ValueError, r.text.c_str());
        return nullptr;
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// f() without the interpreter's lock: an allocation may wait for the device
// and a launch for room in its queue, and what is before it there may be a
// host callback that needs the lock.  f touches no Python object.
template <class F> auto unlocked(F &&f)
{
    struct Unlocked {
        PyThreadState *state = PyEval_SaveThread();
        ~Unlocked() { PyEval_RestoreThread(state); }
    } guard;
    return f();
}

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Raised{};
    return v;
}

double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Raised{};
    return v;
}

std::string text_of(PyObject *o)
{
    const char *s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
    PyErr_Clear();
    return s ? s : "";
}

std::string shape_text(at::IntArrayRef s)
{
    std::string t = "(";
    for (size_t i = 0; i < s.size(); i++)
        t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

std::string type_text(at::ScalarType t)
{
    switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kDouble: return "torch.float64";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    case at::kLong: return "torch.int64";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
    }
}

// a tensor argument, or an undefined one for None
at::Tensor optional_tensor(const char *where, const char *name, PyObject *o)
{
    if (o == Py_None)
        return at::Tensor();
    if (!THPVariable_Check(o))
        fail(where, "%s must be a torch tensor", name);
    return THPVariable_Unpack(o);
}

at::Tensor matrix(const char *where, const char *name, PyObject *o)
{
    if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != 2)
        fail(where, "%s must be a 2-D tensor", name);
    return THPVariable_Unpack(o);
}

bpg_x_dtype float_code(const char *where, const char *name, at::ScalarType t)
{
    if (t == at::kBFloat16)
        return BPG_X_BF16;
    if (t != at::kFloat)
        fail(where, "%s has dtype %s, expected torch.float32 or torch.bfloat16", name,
             type_text(t).c_str());
    return BPG_X_F32;
}

void check_type(const char *where, const char *name, const at::Tensor &t, at::ScalarType want)
{
    if (t.scalar_type() != want)
        fail(where, "%s has dtype %s, expected %s", name, type_text(t.scalar_type()).c_str(),
             type_text(want).c_str());
}

void check_shape(const char *where, const char *name, const at::Tensor &t, at::IntArrayRef want)
{
    if (t.sizes() != want)
        fail(where, "%s has shape %s, expected %s", name, shape_text(t.sizes()).c_str(),
             shape_text(want).c_str());
}

void check_contiguous(const char *where, const char *name, const at::Tensor &t)
{
    if (!t.is_contiguous())
        fail(where, "%s must be contiguous", name);
}

// a matrix of rows with unit column stride that do not overlap
void check_rows(const char *where, const char *name, const at::Tensor &t)
{
    const int64_t rows = t.size(0), cols = t.size(1);
    if (rows > 0 && cols > 0 && (t.stride(1) != 1 || (rows > 1 && t.stride(0) < cols)))
        fail(where, "%s must have unit column stride and row stride >= %lld", name,
             (long long)cols);
}

// the leading dimension: that of a single row is free, so the smallest
// multiple of `unit` that holds it
int64_t row_stride(const at::Tensor &t, int64_t unit)
{
    return t.size(0) > 1 ? t.stride(0) : (t.size(1) + unit - 1) / unit * unit;
}

// The bytes of a tensor: rows of `width` bytes that begin `stride` apart.
struct Bytes {
    int64_t at, rows, width, stride;
};

Bytes bytes_of(const at::Tensor &t)
{
    const int64_t size = (int64_t)t.element_size();
    const int64_t at = (int64_t)reinterpret_cast<uintptr_t>(t.data_ptr());
    if (t.numel() == 0 || at == 0)
        return {0, 0, 0, 0};
    if (t.is_contiguous() || t.dim() != 2)
        return {at, 1, t.numel() * size, 0};
    return {at, t.size(0), t.size(1) * size, t.stride(0) * size};
}

int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); } // b > 0

// whether two tensors share a byte
bool share(Bytes a, Bytes b)
{
    if (a.rows == 0 || b.rows == 0 || a.at + (a.rows - 1) * a.stride + a.width <= b.at ||
        b.at + (b.rows - 1) * b.stride + b.width <= a.at)
        return false;
    if (a.rows == 1 && b.rows == 1)
        return true;
    if (a.rows == 1 || b.rows == 1 || a.stride == b.stride) {
        // row i of a and row i + t of b do where -b.width < d + t stride < a.width
        const int64_t stride = a.rows == 1 ? b.stride : a.stride, d = b.at - a.at;
        const int64_t first = floor_div(-b.width - d, stride) + 1;
        const int64_t last = -floor_div(d - a.width, stride) - 1;
        return std::max(first, 1 - a.rows) <= std::min(last, b.rows - 1);
    }
    if (a.rows > b.rows)
        std::swap(a, b);
    for (int64_t i = 0; i < a.rows; i++)
        if (share({a.at + i * a.stride, 1, a.width, 0}, b))
            return true;
    return false;
}

// Rows of two matrices of one shape and type in the same place.
bool same_rows(const at::Tensor &a, const at::Tensor &b)
{
    return a.data_ptr() == b.data_ptr() && a.scalar_type() == b.scalar_type() &&
           (a.size(0) <= 1 || a.stride(0) == b.stride(0));
}

struct Named {
    const char *name;
    const at::Tensor &tensor;
};

// An output given by the caller shares no memory with what the kernel reads or
// writes beside it: one workgroup's store could come before another's load.
void check_apart(const char *where, const char *name, const at::Tensor &out,
                 std::initializer_list<Named> others)
{
    const Bytes bytes = bytes_of(out);
    for (const Named &o : others)
        if (o.tensor.defined() && share(bytes, bytes_of(o.tensor)))
            fail(where, "%s overlaps %s", name, o.name);
}

void check_bits(const char *where, int64_t bits)
{
    if (bits != 4 && bits != 8)
        fail(where, "act_bits must be 4 or 8, got %lld", (long long)bits);
}

void check_rotation(const char *where, int64_t rotation)
{
    if (rotation != 0 && rotation != 32 && rotation != 64 && rotation != 128)
        fail(where, "rotation must be 0, 32, 64 or 128, got %lld", (long long)rotation);
}

void check_span(const char *where, int64_t rotation, int64_t k)
{
    check_rotation(where, rotation);
    const int64_t unit = rotation ? rotation : 32;
    if (k <= 0 || k % unit != 0)
        fail(where, "K = %lld is not a positive multiple of %lld", (long long)k, (long long)unit);
}

// codes [rows][k/2] (4-bit) or [rows][k] (8-bit) bytes, scales [rows][k/32] fp32
void check_codes(const char *where, const at::Tensor &codes, const at::Tensor &scales, int64_t bits,
                 int64_t rows, int64_t k)
{
    if (codes.scalar_type() != at::kByte && codes.scalar_type() != at::kChar)
        fail(where, "codes has dtype %s, expected torch.uint8 or torch.int8",
             type_text(codes.scalar_type()).c_str());
    check_shape(where, "codes", codes, {rows, bits == 4 ? k / 2 : k});
    check_contiguous(where, "codes", codes);
    check_type(where, "scales", scales, at::kFloat);
    check_shape(where, "scales", scales, {rows, k / 32});
    check_contiguous(where, "scales", scales);
}

// every defined tensor on one cuda device
c10::Device one_device(const char *where, std::initializer_list<const at::Tensor *> tensors)
{
    c10::Device first(c10::DeviceType::CPU);
    bool any = false;
    for (const at::Tensor *t : tensors) {
        if (!t->defined())
            continue;
        if (!t->is_cuda())
            fail(where, "every tensor must be on a cuda device (got %s)", t->device().str().c_str());
        if (any && t->device() != first)
            fail(where, "tensors are on different devices: %s, %s", first.str().c_str(),
                 t->device().str().c_str());
        first = t->device();
        any = true;
    }
    return first;
}

// a new tensor beside `like`; for a cuda one without at::empty's dispatch
at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Tensor &like)
{
    if (like.is_cuda())
        return unlocked([&] {
            return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
        });
    return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}

// the current stream of the tensors' device, as the C ABI takes it
void *stream_of(const c10::Device &device)
{
    return c10::hip::getCurrentHIPStream(device.index()).stream();
}

void check_status(const char *where, bpg_status s)
{
    if (s == BPG_OK)
        return;
    PyObject *e = PyObject_CallFunction(g_error, "is", (int)s, where);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

template <class T = void> T *address(const at::Tensor &t)
{
    return t.defined() ? static_cast<T *>(t.data_ptr()) : nullptr;
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }

PyObject *tuple_of(std::initializer_list<PyObject *> items)
{
    PyObject *t = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject *o : items) {
        if (!o || !t) { // out of memory: a leak is the lesser harm
            throw Raised{};
        }
        PyTuple_SET_ITEM(t, i++, o);
    }
    return t;
}

// (x, residual, weight, eps, act_bits, rotation, h, codes, scales)
PyObject *rmsnorm_quantize_act(PyObject *, PyObject *const *a, Py_ssize_t)
{
    return guarded([&]() -> PyObject * {
        const char *where = "rmsnorm_quantize_act";
        at::AutoDispatchBelowADInplaceOrView below;
        const at::Tensor x = matrix(where, "x", a[0]);
        const bpg_x_dtype x_dt = float_code(where, "x", x.scalar_type());
        check_rows(where, "x", x);
        const int64_t bits = integer(a[4]), rotation = integer(a[5]);
        const float eps = (float)number(a[3]);
        check_bits(where, bits);
        const int64_t m = x.size(0), k = x.size(1);
        check_span(where, rotation, k);
        at::Tensor residual = optional_tensor(where, "residual", a[1]);
        at::Tensor weight = optional_tensor(where, "weight", a[2]);
        at::Tensor h = optional_tensor(where, "h", a[6]);
        at::Tensor codes = optional_tensor(where, "codes", a[7]);
        at::Tensor scales = optional_tensor(where, "scales", a[8]);
        bpg_x_dtype r_dt = BPG_X_F32, w_dt = BPG_X_F32;
        const bool new_h = !h.defined();
        if (residual.defined()) {
            r_dt = float_code(where, "residual", residual.scalar_type());
            check_shape(where, "residual", residual, {m, k});
            check_rows(where, "residual", residual);
            if (new_h) {
                h = make({m, k}, residual.scalar_type(), x);
            } else {
                if (h.scalar_type() != residual.scalar_type())
                    fail(where, "h has dtype %s, the residual %s", type_text(h.scalar_type()).c_str(),
                         type_text(residual.scalar_type()).c_str());
                check_shape(where, "h", h, {m, k});
                check_rows(where, "h", h);
            }
        } else if (h.defined()) {
            fail(where, "h needs a residual (without one the stream is x)");
        }
        if (weight.defined()) {
            w_dt = float_code(where, "weight", weight.scalar_type());
            check_shape(where, "weight", weight, {k});
            check_contiguous(where, "weight", weight);
        }
        const bool new_codes = !codes.defined(), new_scales = !scales.defined();
        if (new_codes)
            codes = make({m, bits == 4 ? k / 2 : k}, at::kByte, x);
        if (new_scales)
            scales = make({m, k / 32}, at::kFloat, x);
        check_codes(where, codes, scales, bits, m, k);
        if (h.defined() && !new_h) {
            check_apart(where, "h", h, {{"x", x}, {"the weight", weight}});
            if (!same_rows(h, residual))
                check_apart(where, "h", h, {{"the residual", residual}});
        }
        if (!new_codes)
            check_apart(where, "codes", codes,
                        {{"x", x}, {"the residual", residual}, {"h", h}, {"the weight", weight}});
        if (!new_scales)
            check_apart(where, "scales", scales,
                        {{"x", x}, {"the residual", residual}, {"h", h}, {"the weight", weight},
                         {"codes", codes}});
        const c10::Device device = one_device(where, {&x, &residual, &h, &weight, &codes, &scales});
        const c10::DeviceGuard guard(device);
        check_status(where, unlocked([&] {
                         return ::rmsnorm_quantize_act(
                             address(x), x_dt, row_stride(x, 4), address(residual), r_dt,
                             residual.defined() ? row_stride(residual, 4) : 0, address(h),
                             h.defined() ? row_stride(h, 4) : 0, address(weight), w_dt, eps, m, k,
                             (int)bits, (int)rotation, address(codes), address<float>(scales),
                             stream_of(device));
                     }));
        auto given = [](PyObject *o) { return Py_INCREF(o), o; };
        return tuple_of({!residual.defined() ? given(a[0]) : new_h ? wrap(h) : given(a[6]),
                         new_codes ? wrap(codes) : given(a[7]),
                         new_scales ? wrap(scales) : given(a[8])});
    });
}

// (codes, scales, act_bits, rotation, y, dtype)
PyObject *dequantize_act(PyObject *, PyObject *const *a, Py_ssize_t)
{
    return guarded([&]() -> PyObject * {
        const char *where = "dequantize_act";
        at::AutoDispatchBelowADInplaceOrView below;
        const at::Tensor scales = matrix(where, "scales", a[1]);
        const at::Tensor codes = matrix(where, "codes", a[0]);
        const int64_t bits = integer(a[2]), rotation = integer(a[3]);
        check_bits(where, bits);
        const int64_t m = scales.size(0), k = scales.size(1) * 32;
        check_codes(where, codes, scales, bits, m, k);
        check_span(where, rotation, k);
        at::Tensor y = optional_tensor(where, "y", a[4]);
        if (a[5] != Py_None && !THPDtype_Check(a[5]))
            fail(where, "dtype must be a torch.dtype");
        at::ScalarType type = a[5] == Py_None ? (y.defined() ? y.scalar_type() : at::kFloat)
                                              : reinterpret_cast<THPDtype *>(a[5])->scalar_type;
        const bpg_x_dtype y_dt = float_code(where, "y", type);
        const bool made = !y.defined();
        if (made)
            y = make({m, k}, type, codes);
        check_type(where, "y", y, type);
        check_shape(where, "y", y, {m, k});
        check_rows(where, "y", y);
        if (!made)
            check_apart(where, "y", y, {{"codes", codes}, {"scales", scales}});
        const c10::Device device = one_device(where, {&codes, &scales, &y});
        const c10::DeviceGuard guard(device);
        check_status(where, unlocked([&] {
                         return ::dequantize_act(address(codes), address<float>(scales), (int)bits,
                                                 (int)rotation, m, k, address(y), y_dt,
                                                 row_stride(y, 4), stream_of(device));
                     }));
        return made ? wrap(y) : (Py_INCREF(a[4]), a[4]);
    });
}

// (codes, scales, act_bits, address of the stamp, image, bias, activation, residual, y, dtype,
//  rotation)
PyObject *w4a4_gemm_epilogue(PyObject *, PyObject *const *a, Py_ssize_t)
{
    return guarded([&]() -> PyObject * {
        const char *where = "w4a4_gemm_epilogue";
        at::AutoDispatchBelowADInplaceOrView below;
        at::Tensor y = optional_tensor(where, "y", a[8]);
        if (a[9] != Py_None && !THPDtype_Check(a[9]))
            fail(where, "dtype must be a torch.dtype");
        const at::ScalarType type = a[9] == Py_None
                                        ? (y.defined() ? y.scalar_type() : at::kFloat)
                                        : reinterpret_cast<THPDtype *>(a[9])->scalar_type;
        const bpg_x_dtype y_dt = float_code(where, "y", type);
        static const char *const names[] = {"none", "relu", "silu", "gelu", "gelu_tanh"};
        const std::string activation = text_of(a[6]);
        int act = 0;
        while (act < 5 && activation != names[act])
            act++;
        if (act == 5)
            fail(where, "activation must be one of none, relu, silu, gelu, gelu_tanh, got %s",
                 activation.c_str());
        const at::Tensor codes = matrix(where, "codes", a[0]);
        const at::Tensor scales = matrix(where, "scales", a[1]);
        const int64_t bits = integer(a[2]), rotation = integer(a[10]);
        const bpg_weights_desc *w =
            reinterpret_cast<const bpg_weights_desc *>(static_cast<uintptr_t>(integer(a[3])));
        check_bits(where, bits);
        check_rotation(where, rotation);
        const int64_t m = codes.size(0), n = w->n;
        check_codes(where, codes, scales, bits, m, w->k);
        if (!THPVariable_Check(a[4]))
            fail(where, "the weight image is on the host: call .to(device) first");
        const at::Tensor image = THPVariable_Unpack(a[4]);
        if (image.scalar_type() != at::kByte || image.dim() != 1 || !image.is_contiguous())
            fail(where, "the weight image must be a contiguous 1-D uint8 tensor");
        if ((uint64_t)image.numel() < w->bytes)
            fail(where, "the weight image has %lld bytes, its stamp names %llu",
                 (long long)image.numel(), (unsigned long long)w->bytes);
        const bool made = !y.defined();
        if (n <= 0)
            check_status(where, BPG_ERR_STAMP);
        if (made)
            y = make({m, n}, type, codes);
        check_type(where, "y", y, type);
        check_shape(where, "y", y, {m, n});
        check_rows(where, "y", y);
        bpg_epilogue ep{};
        ep.act = (bpg_activation)act;
        const at::Tensor bias = optional_tensor(where, "bias", a[5]);
        if (bias.defined()) {
            ep.bias_dt = float_code(where, "bias", bias.scalar_type());
            check_shape(where, "bias", bias, {n});
            check_contiguous(where, "bias", bias);
            ep.bias = address(bias);
        }
        at::Tensor residual;
        if (a[7] != Py_None) {
            residual = matrix(where, "residual", a[7]);
            ep.residual_dt = float_code(where, "residual", residual.scalar_type());
            check_shape(where, "residual", residual, {m, n});
            check_rows(where, "residual", residual);
            ep.residual = address(residual);
            ep.ldr = row_stride(residual, 1);
        }
        if (!made) {
            check_apart(where, "y", y,
                        {{"codes", codes}, {"scales", scales}, {"the weight image", image},
                         {"the bias", bias}});
            if (residual.defined() && !same_rows(y, residual))
                check_apart(where, "y", y, {{"the residual", residual}});
        }
        const c10::Device device = one_device(where, {&codes, &scales, &image, &y, &bias, &residual});
        const c10::DeviceGuard guard(device);
        check_status(where, unlocked([&] {
                         return ::w4a4_gemm_epilogue(address(codes), address<float>(scales),
                                                     (int)bits, (int)rotation, m, w, address(image),
                                                     &ep, address(y), y_dt, row_stride(y, 8),
                                                     stream_of(device));
                     }));
        return made ? wrap(y) : (Py_INCREF(a[8]), a[8]);
    });
}

// (logits, topk, score, bias, groups, topk_groups, group_score, renormalize, scale, expert_of,
//  weights)
PyObject *moe_route_topk(PyObject *, PyObject *const *a, Py_ssize_t)
{
    return guarded([&]() -> PyObject * {
        const char *where = "moe_route_topk";
        at::AutoDispatchBelowADInplaceOrView below;
        const at::Tensor logits = matrix(where, "logits", a[0]);
        const bpg_x_dtype dt = float_code(where, "logits", logits.scalar_type());
        check_rows(where, "logits", logits);
        const int64_t tokens = logits.size(0), experts = logits.size(1), topk = integer(a[1]);
        const std::string score = text_of(a[2]), group_score = text_of(a[6]);
        if (score != "softmax" && score != "sigmoid")
            fail(where, "score must be softmax or sigmoid, got %s", score.c_str());
        if (group_score != "max" && group_score != "top2")
            fail(where, "group_score must be max or top2, got %s", group_score.c_str());
        if (topk < 1 || topk > 64)
            fail(where, "topk must be positive and at most 64, got %lld", (long long)topk);
        const at::Tensor bias = optional_tensor(where, "bias", a[3]);
        if (bias.defined()) {
            check_type(where, "bias", bias, at::kFloat);
            check_shape(where, "bias", bias, {experts});
            check_contiguous(where, "bias", bias);
        }
        const int64_t n = tokens * topk;
        at::Tensor ids = optional_tensor(where, "expert_of", a[9]);
        at::Tensor weights = optional_tensor(where, "weights", a[10]);
        const bool new_ids = !ids.defined(), new_weights = !weights.defined();
        if (new_ids)
            ids = make({n}, at::kInt, logits);
        if (new_weights)
            weights = make({n}, at::kFloat, logits);
        check_type(where, "expert_of", ids, at::kInt);
        check_shape(where, "expert_of", ids, {n});
        check_contiguous(where, "expert_of", ids);
        check_type(where, "weights", weights, at::kFloat);
        check_shape(where, "weights", weights, {n});
        check_contiguous(where, "weights", weights);
        const int renormalize = PyObject_IsTrue(a[7]);
        if (renormalize < 0)
            throw Raised{};
        const int64_t groups = integer(a[4]), topk_groups = integer(a[5]);
        const float scale = (float)number(a[8]);
        if (!new_ids)
            check_apart(where, "expert_of", ids, {{"logits", logits}, {"the bias", bias}});
        if (!new_weights)
            check_apart(where, "weights", weights,
                        {{"logits", logits}, {"the bias", bias}, {"expert_of", ids}});
        const c10::Device device = one_device(where, {&logits, &bias, &ids, &weights});
        const c10::DeviceGuard guard(device);
        check_status(where, unlocked([&] {
                         return ::moe_route_topk(
                             address(logits), dt, tokens, experts, row_stride(logits, 1),
                             score == "softmax" ? BPG_SCORE_SOFTMAX : BPG_SCORE_SIGMOID,
                             address<float>(bias), groups, topk_groups,
                             group_score == "max" ? BPG_GROUP_MAX : BPG_GROUP_TOP2, topk,
                             renormalize, scale, address<int32_t>(ids), address<float>(weights),
                             stream_of(device));
                     }));
        return tuple_of({new_ids ? wrap(ids) : (Py_INCREF(a[9]), a[9]),
                         new_weights ? wrap(weights) : (Py_INCREF(a[10]), a[10])});
    });
}

// The type of an output: `dtype`, else that of a given y, else `otherwise`.
at::ScalarType output_type(const char *where, PyObject *dtype, const at::Tensor &y,
                           at::ScalarType otherwise)
{
    if (dtype != Py_None && !THPDtype_Check(dtype))
        fail(where, "dtype must be a torch.dtype");
    if (dtype == Py_None)
        return y.defined() ? y.scalar_type() : otherwise;
    return reinterpret_cast<THPDtype *>(dtype)->scalar_type;
}

// blocks of 128 values
int64_t blocks_of(int64_t k) { return (k + 127) / 128; }

// e4m3 codes [rows][k], k a positive multiple of 32, under fp32 scales
// [scale_rows][ceil(k / 128)]
void check_fp8_codes(const char *where, const char *name, const at::Tensor &codes,
                     const char *scales_name, const at::Tensor &scales, int64_t rows, int64_t k,
                     int64_t scale_rows)
{
    check_type(where, name, codes, at::kFloat8_e4m3fn);
    if (k <= 0 || k % 32 != 0)
        fail(where, "K = %lld is not a positive multiple of 32", (long long)k);
    check_shape(where, name, codes, {rows, k});
    check_contiguous(where, name, codes);
    check_type(where, scales_name, scales, at::kFloat);
    check_shape(where, scales_name, scales, {scale_rows, blocks_of(k)});
    check_contiguous(where, scales_name, scales);
}

// (x, block_rows, codes, scales)
PyObject *quantize_fp8(PyObject *, PyObject *const *a, Py_ssize_t)
{
    return guarded([&]() -> PyObject * {
        const char *where = "quantize_fp8";
        at::AutoDispatchBelowADInplaceOrView below;
        const at::Tensor x = matrix(where, "x", a[0]);
        const bpg_x_dtype dt = float_code(where, "x", x.scalar_type());
        check_rows(where, "x", x);
        const int64_t m = x.size(0), k = x.size(1), block_rows = integer(a[1]);
        if (block_rows != 1 && block_rows != 128)
            fail(where, "block_rows must be 1 or 128, got %lld", (long long)block_rows);
        if (k <= 0 || k % 32 != 0)
            fail(where, "K = %lld is not a positive multiple of 32", (long long)k);
        at::Tensor codes = optional_tensor(where, "codes", a[2]);
        at::Tensor scales = optional_tensor(where, "scales", a[3]);
        const bool new_codes = !codes.defined(), new_scales = !scales.defined();
        const int64_t lines = block_rows == 1 ? m : blocks_of(m);
        if (new_codes)
            codes = make({m, k}, at::kFloat8_e4m3fn, x);
        if (new_scales)
            scales = make({lines, blocks_of(k)}, at::kFloat, x);
        check_fp8_codes(where, "codes", codes, "scales", scales, m, k, lines);
        if (!new_codes)
            check_apart(where, "codes", codes, {{"x", x}});
        if (!new_scales)
            check_apart(where, "scales", scales, {{"x", x}, {"codes", codes}});
        const c10::Device device = one_device(where, {&x, &codes, &scales});
        const c10::DeviceGuard guard(device);
        check_status(where, unlocked([&] {
                         return ::quantize_fp8(address(x), dt, m, k, row_stride(x, 4), block_rows,
                                               address(codes), address<float>(scales),
                                               stream_of(device));
                     }));
        return tuple_of({new_codes ? wrap(codes) : (Py_INCREF(a[2]), a[2]),
                         new_scales ? wrap(scales) : (Py_INCREF(a[3]), a[3])});
    });
}

// Activations and one or two weight matrices of the products below.
struct Fp8Operands {
    at::Tensor codes, scales, w, w_scales, up, up_scales;
    int64_t m, n, k;
};

Fp8Operands fp8_operands(const char *where, PyObject *const *a, bool gated)
{
    Fp8Operands o;
    o.codes = matrix(where, "codes", a[0]);
    o.scales = matrix(where, "scales", a[1]);
    const char *name = gated ? "the gate's codes" : "the weights' codes";
    const char *scales_name = gated ? "the gate's scales" : "the weights' scales";
    o.w = matrix(where, name, a[2]);
    o.w_scales = matrix(where, scales_name, a[3]);
    o.m = o.codes.size(0);
    o.n = o.w.size(0);
    o.k = o.w.size(1);
    if (o.n < 1)
        fail(where, "the weights have no rows");
    check_fp8_codes(where, name, o.w, scales_name, o.w_scales, o.n, o.k, blocks_of(o.n));
    check_fp8_codes(where, "codes", o.codes, "scales", o.scales, o.m, o.k, o.m);
    if (gated) {
        o.up = matrix(where, "the up projection's codes", a[4]);
        o.up_scales = matrix(where, "the up projection's scales", a[5]);
        check_fp8_codes(where, "the up projection's codes", o.up, "the up projection's scales",
                        o.up_scales, o.n, o.k, blocks_of(o.n));
    }
    return o;
}

void check_apart(const char *where, const char *name, const at::Tensor &out, const Fp8Operands &o)
{
    check_apart(where, name, out,
                {{"codes", o.codes}, {"scales", o.scales}, {"the weights", o.w},
                 {"the weights' scales", o.w_scales}, {"the up projection", o.up},
                 {"the up projection's scales", o.up_scales}});
}

bpg_activation activation_of(const char *where, PyObject *o)
{
    static const char *const names[] = {"none", "relu", "silu", "gelu", "gelu_tanh"};
    const std::string activation = text_of(o);
    for (int act = 0; act < 5; act++)
        if (activation == names[act])
            return (bpg_activation)act;
    fail(where, "activation must be one of none, relu, silu, gelu, gelu_tanh, got %s",
         activation.c_str());
}

// (codes, scales, w, w_scales, y, dtype), or
// (codes, scales, gate, gate_scales, up, up_scales, activation, y, dtype)
PyObject *fp8_product(const char *where, PyObject *const *a, bool gated)
{
    return guarded([&]() -> PyObject * {
        at::AutoDispatchBelowADInplaceOrView below;
        PyObject *given = a[gated ? 7 : 4];
        const bpg_activation act = gated ? activation_of(where, a[6]) : BPG_ACT_NONE;
        at::Tensor y = optional_tensor(where, "y", given);
        const at::ScalarType type = output_type(where, a[gated ? 8 : 5], y, at::kFloat);
        const bpg_x_dtype y_dt = float_code(where, "y", type);
        const Fp8Operands o = fp8_operands(where, a, gated);
        const bool made = !y.defined();
        if (made)
            y = make({o.m, o.n}, type, o.codes);
        check_type(where, "y", y, type);
        check_shape(where, "y", y, {o.m, o.n});
        check_rows(where, "y", y);
        if (!made)
            check_apart(where, "y", y, o);
        const c10::Device device =
            one_device(where, {&o.codes, &o.scales, &o.w, &o.w_scales, &o.up, &o.up_scales, &y});
        const c10::DeviceGuard guard(device);
        // on the current stream, like the call: free for the next one behind it
        const int64_t bytes = gated ? 0 : (int64_t)::fp8_gemm_bytes(o.m, o.n, o.k, y_dt);
        const at::Tensor workspace = bytes ? make({bytes}, at::kByte, o.codes) : at::Tensor();
        check_status(where, unlocked([&] {
                         const int64_t ldy = row_stride(y, 1);
                         if (gated)
                             return ::fp8_gemm_gated(
                                 address(o.codes), address<float>(o.scales), o.m, address(o.w),
                                 address<float>(o.w_scales), address(o.up),
                                 address<float>(o.up_scales), o.n, o.k, act, address(y), y_dt, ldy,
                                 stream_of(device));
                         return ::fp8_gemm(address(o.codes), address<float>(o.scales), o.m,
                                           address(o.w), address<float>(o.w_scales), o.n, o.k,
                                           address(y), y_dt, ldy, address(workspace), (size_t)bytes,
                                           stream_of(device));
                     }));
        return made ? wrap(y) : (Py_INCREF(given), given);
    });
}

PyObject *fp8_gemm(PyObject *, PyObject *const *a, Py_ssize_t)
{
    return fp8_product("fp8_gemm", a, false);
}

PyObject *fp8_gemm_gated(PyObject *, PyObject *const *a, Py_ssize_t)
{
    return fp8_product("fp8_gemm_gated", a, true);
}

// (codes, scales, gate, gate_scales, up, up_scales, activation, out_codes, out_scales, exact)
PyObject *fp8_gemm_gated_quantize(PyObject *, PyObject *const *a, Py_ssize_t)
{
    return guarded([&]() -> PyObject * {
        const char *where = "fp8_gemm_gated_quantize";
        at::AutoDispatchBelowADInplaceOrView below;
        const bpg_activation act = activation_of(where, a[6]);
        const int truth = PyObject_IsTrue(a[9]);
        if (truth < 0)
            throw Raised{};
        const bool exact = truth > 0;
        const Fp8Operands o = fp8_operands(where, a, true);
        if (o.n % 32 != 0)
            fail(where, "F = %lld is not a multiple of 32", (long long)o.n);
        at::Tensor codes = optional_tensor(where, "out_codes", a[7]);
        at::Tensor scales = optional_tensor(where, "out_scales", a[8]);
        const bool new_codes = !codes.defined(), new_scales = !scales.defined();
        if (new_codes)
            codes = make({o.m, o.n}, at::kFloat8_e4m3fn, o.codes);
        if (new_scales)
            scales = make({o.m, blocks_of(o.n)}, at::kFloat, o.codes);
        check_fp8_codes(where, "out_codes", codes, "out_scales", scales, o.m, o.n, o.m);
        if (!new_codes)
            check_apart(where, "out_codes", codes, o);
        if (!new_scales) {
            check_apart(where, "out_scales", scales, o);
            check_apart(where, "out_scales", scales, {{"out_codes", codes}});
        }
        const c10::Device device = one_device(
            where, {&o.codes, &o.scales, &o.w, &o.w_scales, &o.up, &o.up_scales, &codes, &scales});
        const c10::DeviceGuard guard(device);
        // on the current stream, like the call: free for the next one behind it
        const int64_t bytes = exact ? 4 * o.m * o.n
                                    : (int64_t)::fp8_gemm_gated_quantize_bytes(o.m, o.n, o.k);
        const at::Tensor workspace = bytes ? make({bytes}, at::kByte, o.codes) : at::Tensor();
        check_status(where, unlocked([&] {
                         if (exact) { // fp32 values, and their codes
                             const bpg_status s = ::fp8_gemm_gated(
                                 address(o.codes), address<float>(o.scales), o.m, address(o.w),
                                 address<float>(o.w_scales), address(o.up),
                                 address<float>(o.up_scales), o.n, o.k, act, address(workspace),
                                 BPG_X_F32, o.n, stream_of(device));
                             if (s != BPG_OK)
                                 return s;
                             return ::quantize_fp8(address(workspace), BPG_X_F32, o.m, o.n, o.n, 1,
                                                   address(codes), address<float>(scales),
                                                   stream_of(device));
                         }
                         return ::fp8_gemm_gated_quantize(
                             address(o.codes), address<float>(o.scales), o.m, address(o.w),
                             address<float>(o.w_scales), address(o.up), address<float>(o.up_scales),
                             o.n, o.k, act, address(codes), address<float>(scales),
                             address(workspace), (size_t)bytes, stream_of(device));
                     }));
        return tuple_of({new_codes ? wrap(codes) : (Py_INCREF(a[7]), a[7]),
                         new_scales ? wrap(scales) : (Py_INCREF(a[8]), a[8])});
    });
}

// (logits, tokens, topk, logprobs, entropy, ids, top)
PyObject *token_logprobs(PyObject *, PyObject *const *a, Py_ssize_t)
{
    return guarded([&]() -> PyObject * {
        const char *where = "token_logprobs";
        at::AutoDispatchBelowADInplaceOrView below;
        const at::Tensor logits = matrix(where, "logits", a[0]);
        const bpg_x_dtype dt = float_code(where, "logits", logits.scalar_type());
        check_rows(where, "logits", logits);
        const int64_t rows = logits.size(0), vocab = logits.size(1), topk = integer(a[2]);
        if (vocab < 1)
            fail(where, "the logits have no columns");
        if (topk < 0 || topk > 64 || topk > vocab)
            fail(where, "topk must be between 0 and the smaller of 64 and the %lld logits, got %lld",
                 (long long)vocab, (long long)topk);
        const at::Tensor tokens = optional_tensor(where, "tokens", a[1]);
        at::Tensor logprobs = optional_tensor(where, "logprobs", a[3]);
        at::Tensor entropy = optional_tensor(where, "entropy", a[4]);
        at::Tensor ids = optional_tensor(where, "ids", a[5]);
        at::Tensor top = optional_tensor(where, "top", a[6]);
        if (tokens.defined()) {
            if (tokens.scalar_type() != at::kInt && tokens.scalar_type() != at::kLong)
                fail(where, "tokens has dtype %s, expected torch.int32 or torch.int64",
                     type_text(tokens.scalar_type()).c_str());
            check_shape(where, "tokens", tokens, {rows});
            check_contiguous(where, "tokens", tokens);
        } else if (logprobs.defined()) {
            fail(where, "logprobs needs tokens");
        }
        auto output = [&](const char *name, at::Tensor &t, at::ScalarType type,
                          at::IntArrayRef shape) {
            if (!t.defined()) {
                t = make(shape, type, logits);
                return true;
            }
            check_type(where, name, t, type);
            check_shape(where, name, t, shape);
            check_contiguous(where, name, t);
            check_apart(where, name, t, {{"logits", logits}, {"tokens", tokens}});
            return false;
        };
        const bool new_logprobs =
            tokens.defined() && output("logprobs", logprobs, at::kFloat, {rows});
        const bool new_entropy = output("entropy", entropy, at::kFloat, {rows});
        const bool new_ids = output("ids", ids, at::kInt, {rows, topk});
        const bool new_top = output("top", top, at::kFloat, {rows, topk});
        if (!new_entropy)
            check_apart(where, "entropy", entropy, {{"logprobs", logprobs}});
        if (!new_ids)
            check_apart(where, "ids", ids, {{"logprobs", logprobs}, {"entropy", entropy}});
        if (!new_top)
            check_apart(where, "top", top,
                        {{"logprobs", logprobs}, {"entropy", entropy}, {"ids", ids}});
        const c10::Device device =
            one_device(where, {&logits, &tokens, &logprobs, &entropy, &ids, &top});
        const c10::DeviceGuard guard(device);
        const int64_t bytes = (int64_t)::token_logprobs_bytes(rows, vocab, topk);
        const at::Tensor workspace = bytes ? make({bytes}, at::kByte, logits) : at::Tensor();
        const bool wide = tokens.defined() && tokens.scalar_type() == at::kLong;
        check_status(where, unlocked([&] {
                         return ::token_logprobs(
                             address(logits), dt, rows, vocab, row_stride(logits, 1),
                             address(tokens), wide ? BPG_I64 : BPG_I32, topk,
                             address<float>(logprobs), address<float>(entropy),
                             address<int32_t>(ids), address<float>(top), address(workspace),
                             (size_t)bytes, stream_of(device));
                     }));
        auto given = [](PyObject *o) { return Py_INCREF(o), o; };
        return tuple_of({new_logprobs ? wrap(logprobs) : given(a[3]),
                         new_entropy ? wrap(entropy) : given(a[4]), new_ids ? wrap(ids) : given(a[5]),
                         new_top ? wrap(top) : given(a[6])});
    });
}

// (BpgError): the class of the library's own errors
PyObject *set_error(PyObject *, PyObject *cls)
{
    Py_INCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

// a method of exactly N positional arguments
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t), int N>
PyObject *exactly(PyObject *self, PyObject *const *args, Py_ssize_t count)
{
    if (count != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, count);
        return nullptr;
    }
    return F(self, args, count);
}

#define BPG_METHOD(name, count)                                                                    \
    {                                                                                              \
        #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(exactly<name, count>)),  \
            METH_FASTCALL, nullptr                                                                 \
    }

PyMethodDef methods[] = {
    BPG_METHOD(rmsnorm_quantize_act, 9),
    BPG_METHOD(dequantize_act, 6),
    BPG_METHOD(w4a4_gemm_epilogue, 11),
    BPG_METHOD(moe_route_topk, 11),
    BPG_METHOD(quantize_fp8, 4),
    BPG_METHOD(fp8_gemm, 6),
    BPG_METHOD(fp8_gemm_gated, 9),
    BPG_METHOD(fp8_gemm_gated_quantize, 10),
    BPG_METHOD(token_logprobs, 7),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods};

} // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
