// Python module of the calls whose kernels take a few microseconds
// (add_rms_norm, token_weights, kv_evict, value_gate_lora, norm_rope,
// query_absorb, index_scores, index_select): argument checks,
// output allocation and the call into the C ABI, without the Python
// interpreter in between.  On the Grace host a call takes 2.3 us of it with
// its outputs given and 1.3 more for each that it allocates (2.0 through
// at::empty, by way of the dispatcher); the same in Python through ctypes took
// 11 to 21.
//
// Every function takes its arguments by position (the public functions in
// __init__.py name and document them) and returns its outputs, or the
// library's non-zero status as an int.  Bad arguments raise ValueError.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <sstream>
#include <stdexcept>
#include <string>
#include <tuple>
#include <utility>
#include <vector>

#include "../../include/mla_decode.h"

namespace {

using at::ScalarType;
constexpr auto kE4m3 = at::kFloat8_e4m3fn;

[[noreturn]] void refuse(const std::string &msg) { throw std::invalid_argument(msg); }

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject *o, const char *name, int64_t lo, int64_t hi) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(name) + " must be an integer");
    }
    if (v < lo || v > hi) refuse(std::string(name) + " out of range");
    return v;
}

int int32(PyObject *o, const char *name) { return (int)integer(o, name, INT32_MIN, INT32_MAX); }

float real(PyObject *o, const char *name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(name) + " must be a number");
    }
    return (float)v;
}

std::string shape_of(at::IntArrayRef s) {
    std::ostringstream o;
    o << s;
    return o.str();
}

// A contiguous tensor of this type and shape on the first argument's device.
const at::Tensor &dense(const at::Tensor &t, const char *name, ScalarType type, at::IntArrayRef shape, int64_t dev) {
    if (t.scalar_type() != type || t.sizes() != shape || t.layout() != at::kStrided || !t.is_contiguous() ||
        t.get_device() != dev)
        refuse(std::string(name) + " must be a contiguous " + at::toString(type) + " tensor of shape " +
               shape_of(shape) + " on the first argument's device");
    return t;
}

// Row stride of a 2-D tensor of this type and shape with contiguous rows.
int64_t rows_of(const at::Tensor &t, const char *name, ScalarType type, at::IntArrayRef shape, int64_t dev) {
    if (t.scalar_type() != type || t.sizes() != shape || t.layout() != at::kStrided || t.stride(1) != 1 ||
        t.get_device() != dev)
        refuse(std::string(name) + " must be a " + at::toString(type) + " tensor of shape " + shape_of(shape) +
               " with contiguous rows on the first argument's device");
    return shape[0] > 1 ? t.stride(0) : shape[1];
}

// Where a call runs: the device of its tensors, made current, and the given
// stream (None: that device's current one).  Outputs of a call on a stream
// of its own are allocated there, so that their memory is not still in use
// by work of the current stream.
struct Place {
    c10::cuda::OptionalCUDAGuard guard;
    c10::Device device{c10::kCUDA};
    cudaStream_t stream = nullptr;
    bool own = false;

    Place(int64_t dev, PyObject *s) {
        if (dev < 0) refuse("tensors must be CUDA tensors");
        device = c10::Device(c10::kCUDA, (c10::DeviceIndex)dev);
        guard.set_index((c10::DeviceIndex)dev);
        if (s == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
            return;
        }
        PyObject *attr = PyObject_GetAttrString(s, "cuda_stream");
        if (!attr) PyErr_Clear();
        const unsigned long long h = PyLong_AsUnsignedLongLong(attr ? attr : s);
        Py_XDECREF(attr);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            refuse("stream must be a stream or its handle");
        }
        stream = reinterpret_cast<cudaStream_t>(h);
        own = true;
    }
    at::Tensor empty(at::IntArrayRef shape, ScalarType type) const {
        const auto options = at::TensorOptions().dtype(type).device(device);
        if (!own) return at::Tensor(at::detail::empty_cuda(shape, options));
        c10::cuda::CUDAStreamGuard on(c10::cuda::getStreamFromExternal(stream, device.index()));
        return at::Tensor(at::detail::empty_cuda(shape, options));
    }
    // Two tensors in one allocation (0.4 us less than two), the second 256-byte aligned in it.
    std::pair<at::Tensor, at::Tensor> empty(at::IntArrayRef shape, ScalarType type, at::IntArrayRef shape2,
                                            ScalarType type2) const {
        const int64_t bytes = (c10::multiply_integers(shape) * (int64_t)c10::elementSize(type) + 255) / 256 * 256;
        const int64_t bytes2 = c10::multiply_integers(shape2) * (int64_t)c10::elementSize(type2);
        const at::Tensor whole = empty({bytes + bytes2}, at::kByte);
        const auto part = [&](at::IntArrayRef s, ScalarType t, int64_t offset) {
            at::Tensor x = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(),
                                                                    c10::scalarTypeToTypeMeta(t));
            x.unsafeGetTensorImpl()->set_sizes_contiguous(s);
            x.unsafeGetTensorImpl()->set_storage_offset(offset / (int64_t)c10::elementSize(t));
            return x;
        };
        return {part(shape, type, 0), part(shape2, type2, bytes)};
    }
};

void *ptr(const at::Tensor &t) { return t.data_ptr(); }
template <class T>
T *ptr(const at::Tensor &t) {
    return static_cast<T *>(t.data_ptr());
}

// A caller's output or, for None, a new one.
template <class Check>
at::Tensor output(PyObject *o, const char *name, const Place &at, at::IntArrayRef shape, ScalarType type, Check check) {
    if (o == Py_None) return at.empty(shape, type);
    const at::Tensor &t = tensor(o, name);
    check(t);
    return t;
}

at::Tensor dense_output(PyObject *o, const char *name, const Place &at, at::IntArrayRef shape, ScalarType type) {
    return output(o, name, at, shape, type,
                  [&](const at::Tensor &t) { dense(t, name, type, shape, at.device.index()); });
}

// The caller's workspace, or one of `need` bytes (none for 0).
at::Tensor workspace(PyObject *o, const Place &at, int64_t need) {
    if (o == Py_None) return need > 0 ? at.empty({need}, at::kByte) : at::Tensor();
    const at::Tensor &t = tensor(o, "workspace");
    return dense(t, "workspace", at::kByte, {t.numel()}, at.device.index());
}

PyObject *wrap(const at::Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject *pack(std::initializer_list<at::Tensor> ts) {
    PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
    Py_ssize_t i = 0;
    for (const auto &t : ts) {
        PyObject *o = r ? wrap(t) : nullptr;
        if (!o) {
            Py_XDECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// Runs f with C++ exceptions turned into Python's.
template <class F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (const std::invalid_argument &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError &e) {
        PyObject *torch = PyImport_ImportModule("torch");
        PyObject *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        PyErr_Clear();
        PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

int norm_type(ScalarType t) { return t == at::kBFloat16 ? MLA_TYPE_BF16 : t == at::kHalf ? MLA_TYPE_F16 : MLA_TYPE_F32; }

// (x, weight, eps, residual, quant, scale, out, out_scales, residual_out, stream)
PyObject *add_rms_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject * {
        const at::Tensor &x = tensor(a[0], "x");
        const ScalarType type = x.scalar_type();
        if (x.dim() != 2 || (type != at::kBFloat16 && type != at::kHalf)) refuse("x must be bf16 or fp16 [T, D]");
        const int64_t dev = x.get_device(), T = x.size(0), D = x.size(1);
        const at::IntArrayRef shape = x.sizes();
        const int64_t xs = rows_of(x, "x", type, shape, dev);
        const at::Tensor &w = dense(tensor(a[1], "weight"), "weight", type, {D}, dev);
        const float eps = real(a[2], "eps");
        const int quant = int32(a[4], "quant");
        const bool scales = quant == MLA_QUANT_ROW || quant == MLA_QUANT_GROUP;
        if ((a[5] != Py_None) != (quant == MLA_QUANT_STATIC)) refuse("scale goes with quant='static'");
        const float scale = a[5] == Py_None ? 0.f : real(a[5], "scale");
        at::Tensor residual;
        int64_t rs = 0;
        if (a[3] != Py_None) {
            residual = tensor(a[3], "residual");
            if (residual.scalar_type() != type && residual.scalar_type() != at::kFloat)
                refuse("residual must be x's type or float32");
            rs = rows_of(residual, "residual", residual.scalar_type(), shape, dev);
        } else if (a[8] != Py_None) {
            refuse("residual_out needs a residual");
        }
        if (!scales && a[7] != Py_None) refuse("out_scales goes with quant='row' or 'group'");
        const Place at(dev, a[9]);
        int64_t os = D, ros = 0;
        ScalarType otype = quant == MLA_QUANT_NONE ? type : kE4m3;
        if (quant != MLA_QUANT_NONE && a[6] != Py_None && tensor(a[6], "out").scalar_type() == at::kByte) otype = at::kByte;
        const at::Tensor out = output(a[6], "out", at, shape, otype,
                                      [&](const at::Tensor &t) { os = rows_of(t, "out", otype, shape, dev); });
        at::Tensor residual_out, out_scales;
        if (residual.defined()) {
            ros = D;
            residual_out = output(a[8], "residual_out", at, shape, residual.scalar_type(), [&](const at::Tensor &t) {
                ros = rows_of(t, "residual_out", residual.scalar_type(), shape, dev);
            });
        }
        if (quant == MLA_QUANT_ROW) out_scales = dense_output(a[7], "out_scales", at, {T}, at::kFloat);
        if (quant == MLA_QUANT_GROUP) out_scales = dense_output(a[7], "out_scales", at, {T, (D + 127) / 128}, at::kFloat);
        const mla_status st = D > INT32_MAX
                                  ? MLA_ERR_INVALID
                                  : mla_add_rms_norm(ptr(x), xs, norm_type(type), residual.defined() ? ptr(residual) : nullptr,
                                                     rs, residual.defined() ? norm_type(residual.scalar_type()) : 0, ptr(w),
                                                     eps, T, (int)D, quant, scale, ptr(out), os,
                                                     scales ? ptr<float>(out_scales) : nullptr,
                                                     residual_out.defined() ? ptr(residual_out) : nullptr, ros, at.stream);
        if (st != MLA_OK) return PyLong_FromLong(st);
        return pack({out, out_scales, residual_out});
    });
}

// Strides of a [rows, heads, width] tensor of this type with contiguous
// heads, or of [rows, width] as one head (rows, heads of one: dense; a lone
// row has no stride to exceed the limit, however far apart its heads lie).
struct HeadRows {
    int64_t rows, heads, width, row, head;
};
HeadRows heads_of(const at::Tensor &t, const char *name, int64_t dev) {
    const int64_t n = t.dim();
    if ((n != 2 && n != 3) || t.layout() != at::kStrided || t.get_device() != dev ||
        (t.size(n - 1) > 1 && t.stride(n - 1) != 1))
        refuse(std::string(name) + " must be [T, H, D] or [T, D] with contiguous heads on the first argument's device");
    HeadRows h = {t.size(0), n == 3 ? t.size(1) : 1, t.size(n - 1), 0, 0};
    h.head = h.heads > 1 ? t.stride(1) : h.width;
    h.row = h.rows > 1 ? t.stride(0) : h.width;
    return h;
}

// (x, weight, eps, positions, cos_sin, rope_start, pairs, quant, scale, slots, out, out_scales, stream)
PyObject *norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject * {
        const at::Tensor &x = tensor(a[0], "x");
        const ScalarType type = x.scalar_type();
        if (type != at::kBFloat16 && type != at::kHalf) refuse("x must be bf16 or fp16");
        const int64_t dev = x.get_device();
        const HeadRows hx = heads_of(x, "x", dev);
        const int64_t T = hx.rows;
        if (hx.width > INT32_MAX || hx.heads > INT32_MAX) refuse("x too wide");
        const void *weight = nullptr;
        int64_t norm_dim = 0;
        if (a[1] != Py_None) {
            const at::Tensor &w = tensor(a[1], "weight");
            norm_dim = w.numel();
            weight = ptr(dense(w, "weight", type, {norm_dim}, dev));
            if (norm_dim > hx.width || norm_dim == 0) refuse("weight must have 8 to D elements");
        }
        const float eps = real(a[2], "eps");
        if ((a[3] != Py_None) != (a[4] != Py_None)) refuse("positions and cos_sin go together");
        const int64_t *positions = nullptr, *slots = nullptr;
        const float *table = nullptr;
        int64_t table_rows = 0, rope_dim = 0;
        if (a[3] != Py_None) {
            positions = ptr<int64_t>(dense(tensor(a[3], "positions"), "positions", at::kLong, {T}, dev));
            const at::Tensor &cs = tensor(a[4], "cos_sin");
            if (cs.dim() != 2 || cs.size(1) > INT32_MAX) refuse("cos_sin must be float32 [positions, rope_dim]");
            table_rows = cs.size(0), rope_dim = cs.size(1);
            table = ptr<float>(dense(cs, "cos_sin", at::kFloat, {table_rows, rope_dim}, dev));
        }
        const int rope_start = int32(a[5], "rope_start");
        const int pairs = PyObject_IsTrue(a[6]);
        if (pairs < 0) return nullptr;
        const int quant = int32(a[7], "quant");
        if ((a[8] != Py_None) != (quant == MLA_QUANT_STATIC)) refuse("scale goes with quant='static'");
        const float scale = a[8] == Py_None ? 0.f : real(a[8], "scale");
        const bool scales = quant == MLA_QUANT_ROW;
        if (!scales && a[11] != Py_None) refuse("out_scales goes with quant='head'");
        if (a[9] != Py_None) {
            slots = ptr<int64_t>(dense(tensor(a[9], "slots"), "slots", at::kLong, {T}, dev));
            if (a[10] == Py_None || (scales && a[11] == Py_None)) refuse("slots need the cache as out (and out_scales)");
        }
        const Place at(dev, a[12]);
        ScalarType otype = quant == MLA_QUANT_NONE ? type : kE4m3;
        if (quant != MLA_QUANT_NONE && a[10] != Py_None && tensor(a[10], "out").scalar_type() == at::kByte) otype = at::kByte;
        HeadRows ho = {T, hx.heads, hx.width, hx.heads * hx.width, hx.width};
        at::Tensor out, out_scales;
        std::vector<int64_t> scales_shape;
        if (scales && a[10] == Py_None && a[11] == Py_None) {
            scales_shape = x.sizes().vec();
            scales_shape.pop_back();
            std::tie(out, out_scales) = at.empty(x.sizes(), otype, scales_shape, at::kFloat);
        } else {
            out = output(a[10], "out", at, x.sizes(), otype, [&](const at::Tensor &t) {
                ho = heads_of(t, "out", dev);
                if (t.scalar_type() != otype || t.dim() != x.dim() || ho.heads != hx.heads || ho.width != hx.width ||
                    (a[9] == Py_None && ho.rows != T))
                    refuse(std::string("out must be ") + at::toString(otype) + (a[9] == Py_None ? "" : " rows") +
                           " of x's shape");
            });
            if (scales) {
                scales_shape = {ho.rows};
                if (x.dim() == 3) scales_shape.push_back(ho.heads);
                out_scales = dense_output(a[11], "out_scales", at, scales_shape, at::kFloat);
            }
        }
        const mla_status st = mla_norm_rope(
            ptr(x), hx.row, hx.head, norm_type(type), weight, (int)norm_dim, eps, positions, table, table_rows, rope_start,
            (int)rope_dim, pairs ? MLA_ROPE_PAIRS : 0u, T, (int)hx.heads, (int)hx.width, quant, scale, slots, ho.rows,
            ptr(out), ho.row, ho.head, scales ? ptr<float>(out_scales) : nullptr, at.stream);
        if (st != MLA_OK) return PyLong_FromLong(st);
        return pack({out, out_scales});
    });
}

// (q, w_uk, positions, cos_sin, pairs, q_scale, out, stream)
PyObject *query_absorb(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject * {
        constexpr int64_t kWidth = MLA_D_NOPE + MLA_D_ROPE;
        const at::Tensor &q = tensor(a[0], "q");
        const int64_t dev = q.get_device();
        if (q.scalar_type() != at::kBFloat16 || q.dim() != 3 || q.size(2) != kWidth) refuse("q must be bf16 [S, H, 192]");
        const HeadRows hq = heads_of(q, "q", dev);
        const int64_t S = hq.rows, H = hq.heads;
        if (H > MLA_MAX_HEADS) refuse("q must have at most 128 heads");
        const at::Tensor &w = dense(tensor(a[1], "w_uk"), "w_uk", at::kBFloat16, {H, MLA_D_NOPE, MLA_D_LATENT}, dev);
        if ((a[2] != Py_None) != (a[3] != Py_None)) refuse("positions and cos_sin go together");
        const int64_t *positions = nullptr;
        const float *table = nullptr;
        int64_t table_rows = 0;
        if (a[2] != Py_None) {
            positions = ptr<int64_t>(dense(tensor(a[2], "positions"), "positions", at::kLong, {S}, dev));
            const at::Tensor &cs = tensor(a[3], "cos_sin");
            table_rows = cs.dim() == 2 ? cs.size(0) : -1;
            table = ptr<float>(dense(cs, "cos_sin", at::kFloat, {table_rows, MLA_D_ROPE}, dev));
        }
        const int pairs = PyObject_IsTrue(a[4]);
        if (pairs < 0) return nullptr;
        const bool fp8 = a[5] != Py_None;
        const float q_scale = fp8 ? real(a[5], "q_scale") : 1.f;
        const Place at(dev, a[7]);
        ScalarType otype = fp8 ? kE4m3 : at::kBFloat16;
        if (fp8 && a[6] != Py_None && tensor(a[6], "out").scalar_type() == at::kByte) otype = at::kByte;
        int64_t out_row = H * MLA_D_QK;
        const at::Tensor out = output(a[6], "out", at, {S, H, MLA_D_QK}, otype, [&](const at::Tensor &t) {
            const HeadRows ho = heads_of(t, "out", dev);
            if (t.scalar_type() != otype || t.dim() != 3 || ho.rows != S || ho.heads < H || ho.width != MLA_D_QK ||
                ho.head != MLA_D_QK)
                refuse(std::string("out must be ") + at::toString(otype) + " [S, H or more, 576] with contiguous rows of heads");
            if (ho.rows > 1) out_row = ho.row;
        });
        const mla_status st = mla_query_absorb(ptr(q), hq.row, hq.head, ptr(w), positions, table, table_rows,
                                               (pairs ? MLA_ABSORB_PAIRS : 0u) | (fp8 ? MLA_ABSORB_OUT_FP8 : 0u), S, (int)H,
                                               q_scale, ptr(out), out_row, at.stream);
        if (st != MLA_OK) return PyLong_FromLong(st);
        return wrap(out);
    });
}

// (q, kv, pages, indptr, scale, kv_scale, lse, heads, qlen, weights, decay, causal, q_scale, out, workspace, stream)
PyObject *token_weights(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 16, [&]() -> PyObject * {
        const at::Tensor &q = tensor(a[0], "q");
        const bool q8 = q.scalar_type() == kE4m3 || q.scalar_type() == at::kByte;
        if (!(q8 || q.scalar_type() == at::kBFloat16) || q.dim() != 3 || q.size(2) != MLA_D_QK)
            refuse("q must be bf16 or fp8 e4m3 [S, H, 576]");
        const int64_t dev = q.get_device(), S = q.size(0), hpad = q.size(1);
        const at::Tensor &kv = tensor(a[1], "kv"), &pages = tensor(a[2], "pages"), &indptr = tensor(a[3], "indptr");
        const float scale = real(a[4], "scale"), kv_scale = real(a[5], "kv_scale"), q_scale = real(a[12], "q_scale");
        const int64_t heads = a[7] == Py_None ? hpad : integer(a[7], "heads", 0, INT32_MAX);
        const int qlen = int32(a[8], "qlen");
        const int64_t R = indptr.numel() - 1, pages_n = pages.numel();
        if (q.stride(2) != 1 || (hpad > 1 && q.stride(1) != MLA_D_QK)) refuse("q rows must have contiguous [H, 576] heads");
        if (R < 0 || R > INT32_MAX || S != R * qlen || heads > hpad)
            refuse("q shape does not match indptr / qlen / heads");
        if (kv.scalar_type() != at::kByte && kv.scalar_type() != kE4m3) refuse("kv must be uint8 codes or float8_e4m3fn");
        const int64_t pool = kv.dim() == 2 ? kv.size(0) : -1;
        dense(kv, "kv", kv.scalar_type(), {pool, MLA_D_QK}, dev);
        dense(pages, "pages", at::kInt, {pages_n}, dev);
        dense(indptr, "indptr", at::kInt, {R + 1}, dev);
        const at::Tensor &lse = dense(tensor(a[6], "lse"), "lse", at::kFloat, {S, heads}, dev);
        const float *weights = nullptr;
        if (a[9] != Py_None) weights = ptr<float>(dense(tensor(a[9], "weights"), "weights", at::kFloat, {pages_n}, dev));
        const float decay = weights ? real(a[10], "decay") : 0.f;
        const int causal = PyObject_IsTrue(a[11]);
        if (causal < 0) return nullptr;
        const Place at(dev, a[15]);
        const at::Tensor out = dense_output(a[13], "out", at, {pages_n}, at::kFloat);
        const unsigned flags = (causal ? MLA_ATTEND_CAUSAL : 0u) | (q8 ? MLA_ATTEND_Q_FP8 : 0u);
        int64_t need = 0;
        if (a[14] == Py_None && (need = mla_token_weights_workspace(qlen, (int)heads, pages_n, flags)) < 0)
            return PyLong_FromLongLong(need);
        const at::Tensor ws = workspace(a[14], at, need);
        const mla_status st = mla_token_weights(
            ptr(q), S > 1 ? q.stride(0) : heads * MLA_D_QK, ptr(kv), pool, ptr<int32_t>(pages), pages_n,
            ptr<int32_t>(indptr), (int)R, qlen, (int)heads, scale, kv_scale, q_scale, ptr<float>(lse), decay, weights,
            ptr<float>(out), flags, ws.defined() ? ptr(ws) : nullptr, ws.defined() ? ws.numel() : 0, at.stream);
        if (st != MLA_OK) return PyLong_FromLong(st);
        return wrap(out);
    });
}

// (q, weights, k, pages, indptr, q_scales, scale, qlen, causal, out, stream)
PyObject *index_scores(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject * {
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[2], "k"), &pages = tensor(a[3], "pages"),
                         &indptr = tensor(a[4], "indptr");
        const int64_t dev = q.get_device();
        if ((q.scalar_type() != kE4m3 && q.scalar_type() != at::kByte) || q.dim() != 3) refuse("q must be e4m3 codes [S, H, 128]");
        const int64_t S = q.size(0), H = q.size(1), R = indptr.numel() - 1, pages_n = pages.numel();
        dense(q, "q", q.scalar_type(), {S, H, MLA_D_INDEX}, dev);
        const at::Tensor &w = dense(tensor(a[1], "weights"), "weights", at::kFloat, {S, H}, dev);
        if (k.scalar_type() != kE4m3 && k.scalar_type() != at::kByte) refuse("k must be e4m3 codes [pool, 128]");
        const int64_t pool = k.dim() == 2 ? k.size(0) : -1;
        dense(k, "k", k.scalar_type(), {pool, MLA_D_INDEX}, dev);
        dense(pages, "pages", at::kInt, {pages_n}, dev);
        const float *q_scales = nullptr;
        if (a[5] != Py_None) q_scales = ptr<float>(dense(tensor(a[5], "q_scales"), "q_scales", at::kFloat, {S, H}, dev));
        const float scale = real(a[6], "scale");
        const int qlen = int32(a[7], "qlen");
        if (R < 0 || R > INT32_MAX || S != R * qlen || H > INT32_MAX) refuse("q's rows do not match indptr / qlen");
        dense(indptr, "indptr", at::kInt, {R + 1}, dev);
        const int causal = PyObject_IsTrue(a[8]);
        if (causal < 0) return nullptr;
        const Place at(dev, a[10]);
        const at::Tensor out = dense_output(a[9], "out", at, {qlen < 0 ? 0 : qlen, pages_n}, at::kFloat);
        const mla_status st = mla_index_scores(ptr(q), ptr<float>(w), q_scales, ptr(k), pool, ptr<int32_t>(pages), pages_n,
                                               ptr<int32_t>(indptr), (int)R, qlen, (int)H, scale, ptr<float>(out),
                                               causal ? MLA_ATTEND_CAUSAL : 0u, at.stream);
        if (st != MLA_OK) return PyLong_FromLong(st);
        return wrap(out);
    });
}

// (scores, pages, indptr, topk, block, recent, sinks, causal, pages_out, indptr_out, stream)
PyObject *index_select(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject * {
        const at::Tensor &scores = tensor(a[0], "scores"), &pages = tensor(a[1], "pages"), &indptr = tensor(a[2], "indptr");
        const int64_t dev = scores.get_device(), pages_n = pages.numel(), R = indptr.numel() - 1;
        if (scores.dim() != 2 || scores.size(0) > MLA_MAX_QLEN) refuse("scores must be float32 [qlen, pages], qlen up to 16");
        const int qlen = (int)scores.size(0);
        if (R < 0 || R > INT32_MAX) refuse("indptr must have R + 1 entries");
        dense(scores, "scores", at::kFloat, {qlen, pages_n}, dev);
        dense(pages, "pages", at::kInt, {pages_n}, dev);
        dense(indptr, "indptr", at::kInt, {R + 1}, dev);
        const int topk = int32(a[3], "topk"), block = int32(a[4], "block"), recent = int32(a[5], "recent"),
                  sinks = int32(a[6], "sinks");
        const int causal = PyObject_IsTrue(a[7]);
        if (causal < 0) return nullptr;
        const Place at(dev, a[10]);
        const int64_t need = mla_index_select_capacity((int)R, qlen, pages_n, topk, block);
        if (need < 0) return PyLong_FromLongLong(need);
        at::Tensor po, io;
        if (a[8] == Py_None && a[9] == Py_None) {
            std::tie(po, io) = at.empty({need}, at::kInt, {R * qlen + 1}, at::kInt);
        } else {
            po = output(a[8], "pages_out", at, {need}, at::kInt, [&](const at::Tensor &t) {
                dense(t, "pages_out", at::kInt, {t.numel()}, dev);
            });
            io = dense_output(a[9], "indptr_out", at, {R * qlen + 1}, at::kInt);
        }
        const mla_status st = mla_index_select(ptr<float>(scores), ptr<int32_t>(pages), pages_n, ptr<int32_t>(indptr), (int)R,
                                               qlen, topk, block, recent, sinks, causal ? MLA_ATTEND_CAUSAL : 0u,
                                               ptr<int32_t>(po), po.numel(), ptr<int32_t>(io), at.stream);
        if (st != MLA_OK) return PyLong_FromLong(st);
        return pack({po, io});
    });
}

// (pages, indptr, weights, budget, recent, sinks, pages_out, indptr_out, weights_out, stream)
PyObject *kv_evict(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject * {
        const at::Tensor &pages = tensor(a[0], "pages"), &indptr = tensor(a[1], "indptr");
        const int64_t dev = pages.get_device(), pages_n = pages.numel(), R = indptr.numel() - 1;
        if (R < 0 || R > INT32_MAX) refuse("indptr must have R + 1 entries");
        dense(pages, "pages", at::kInt, {pages_n}, dev);
        dense(indptr, "indptr", at::kInt, {R + 1}, dev);
        const at::Tensor &w = dense(tensor(a[2], "weights"), "weights", at::kFloat, {pages_n}, dev);
        const int32_t *budgets = nullptr;
        int budget = 0;
        if (THPVariable_Check(a[3])) budgets = ptr<int32_t>(dense(tensor(a[3], "budget"), "budget", at::kInt, {R}, dev));
        else budget = int32(a[3], "budget");
        const int recent = int32(a[4], "recent"), sinks = int32(a[5], "sinks");
        const Place at(dev, a[9]);
        const at::Tensor po = dense_output(a[6], "pages_out", at, {pages_n}, at::kInt);
        const at::Tensor io = dense_output(a[7], "indptr_out", at, {R + 1}, at::kInt);
        const at::Tensor wo = dense_output(a[8], "weights_out", at, {pages_n}, at::kFloat);
        const mla_status st = mla_kv_evict(ptr<int32_t>(pages), pages_n, ptr<int32_t>(indptr), (int)R, ptr<float>(w),
                                           budgets, budget, recent, sinks, ptr<int32_t>(po), ptr<int32_t>(io),
                                           ptr<float>(wo), at.stream);
        if (st != MLA_OK) return PyLong_FromLong(st);
        return pack({po, io, wo});
    });
}

// (latent, w_uv, gate, lengths, lora_a, lora_b, adapters, lora_scale, qlen, out, workspace, stream)
PyObject *value_gate_lora(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject * {
        const at::Tensor &latent = tensor(a[0], "latent"), &lora_a = tensor(a[4], "lora_a"),
                         &lengths = tensor(a[3], "lengths");
        if (latent.dim() != 3 || lora_a.dim() != 3) refuse("latent must be [S, heads, 512], lora_a [n, rank, 512]");
        const int64_t dev = latent.get_device(), S = latent.size(0), H = latent.size(1);
        const int64_t adapters_n = lora_a.size(0), rank = lora_a.size(1), R = lengths.numel();
        const int qlen = int32(a[8], "qlen");
        if (R > INT32_MAX || H > INT32_MAX || adapters_n > INT32_MAX || rank > INT32_MAX || R * qlen != S)
            refuse("lengths must be [S / qlen]");
        dense(latent, "latent", at::kBFloat16, {S, H, MLA_D_LATENT}, dev);
        const at::Tensor &w = dense(tensor(a[1], "w_uv"), "w_uv", at::kBFloat16, {H, MLA_D_V, MLA_D_LATENT}, dev);
        const at::Tensor &gate = dense(tensor(a[2], "gate"), "gate", at::kBFloat16, {S, H * MLA_D_V}, dev);
        dense(lengths, "lengths", at::kInt, {R}, dev);
        dense(lora_a, "lora_a", at::kBFloat16, {adapters_n, rank, MLA_D_LATENT}, dev);
        const at::Tensor &lora_b = dense(tensor(a[5], "lora_b"), "lora_b", at::kBFloat16, {adapters_n, H * MLA_D_V, rank}, dev);
        const at::Tensor &adapters = dense(tensor(a[6], "adapters"), "adapters", at::kInt, {R}, dev);
        const at::Tensor &scale = dense(tensor(a[7], "lora_scale"), "lora_scale", at::kFloat, {adapters_n}, dev);
        const Place at(dev, a[11]);
        const at::Tensor out = dense_output(a[9], "out", at, {S, H * MLA_D_V}, at::kBFloat16);
        int64_t need = 0;
        if (a[10] == Py_None && (need = mla_value_gate_lora_workspace((int)R, qlen, (int)H, (int)rank)) < 0)
            return PyLong_FromLongLong(need);
        const at::Tensor ws = workspace(a[10], at, need);
        const mla_status st = mla_value_gate_lora(
            ptr(latent), ptr(w), ptr(gate), ptr<int32_t>(lengths), ptr(lora_a), ptr(lora_b), ptr<int32_t>(adapters),
            ptr<float>(scale), (int)adapters_n, (int)rank, (int)R, qlen, (int)H, ptr(out), ws.defined() ? ptr(ws) : nullptr,
            ws.defined() ? ws.numel() : 0, at.stream);
        if (st != MLA_OK) return PyLong_FromLong(st);
        return wrap(out);
    });
}

#define MLA_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MLA_METHOD(add_rms_norm), MLA_METHOD(token_weights), MLA_METHOD(kv_evict),
                         MLA_METHOD(value_gate_lora), MLA_METHOD(norm_rope),
                         MLA_METHOD(query_absorb), MLA_METHOD(index_scores),
                         MLA_METHOD(index_select), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "mla_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_mla_ops() { return PyModule_Create(&module); }
