// torch_ops.cpp -- torch tensors in, libmoe calls out, for the operators around the experts
// (include/moe.h): the module behind ops.py.
//
// Argument marshalling only, like the ctypes binding of the layer, in C++ because these calls are small:
// for one decoded token the kernel runs 2 to 4 us, and checking the tensors, allocating the outputs and
// passing a dozen arguments from Python took 8 to 12 us more.  Functions take their arguments by
// position (None for an absent tensor), run on the tensors' device and its current stream, and return
// the outputs; a tensor the library cannot take raises ValueError, a refusal by the library MoeError.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <initializer_list>
#include <limits>
#include <sstream>
#include <stdexcept>
#include <string>

#include "../../include/moe.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

PyObject* g_moe_error = nullptr;   // the exception class for the library's codes

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct Failed {
    int code;
};

void check(int code) {
    if (code != MOE_OK) throw Failed{code};
}

// Runs f, which returns a new reference, and turns what it throws into Python exceptions.
template <typename F> PyObject* guarded(F f) {
    try {
        return f();
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const Failed& e) {
        PyObject* err = PyObject_CallFunction(g_moe_error, "is", e.code, moe_last_error());
        if (err) {
            PyErr_SetObject(g_moe_error, err);
            Py_DECREF(err);
        }
    } catch (const std::exception&) {   // torch's own: memory that ran out raises the class that programs catch for it
        if (!PyErr_Occurred()) torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// The interpreter's lock given up from here to end(), as in torch's own operators: allocations and launches may wait for
// the device (a full launch queue, memory to be freed), and what the device waits for may be up to another thread.
class Unlocked {
    PyThreadState* held_ = PyEval_SaveThread();

public:
    void end() {
        if (held_) PyEval_RestoreThread(held_);
        held_ = nullptr;
    }
    ~Unlocked() { end(); }
};

void expect_args(Py_ssize_t have, Py_ssize_t want, const char* name) {
    if (have != want) throw Refused(std::string(name) + ": " + std::to_string(want) + " arguments are needed");
}

const Tensor* optional_tensor(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + ": a tensor is needed");
    return &THPVariable_Unpack(o);
}
const Tensor& tensor(PyObject* o, const char* name) {
    const Tensor* t = optional_tensor(o, name);
    if (!t) throw Refused(std::string(name) + ": a tensor is needed");
    return *t;
}

[[noreturn]] void wrong(const Tensor& t, const char* name, ScalarType st, IntArrayRef shape, int dev) {
    std::ostringstream s;
    s << name << ": a contiguous " << st << " tensor of shape " << shape << " on cuda:" << dev << " is needed, got "
      << t.scalar_type() << " " << t.sizes() << " on " << t.device() << (t.is_contiguous() ? "" : ", not contiguous");
    throw Refused(s.str());
}

// The device all tensors of a call must share: that of `t`.
int device_of(const Tensor& t, const char* name) {
    if (!t.is_cuda()) throw Refused(std::string(name) + ": CUDA tensors are needed");
    return t.get_device();
}

// t's address, checked (NULL for an absent tensor).
void* at_of(const Tensor* t, const char* name, ScalarType st, IntArrayRef shape, int dev) {
    if (!t) return nullptr;
    if (!t->is_cuda() || t->get_device() != dev || t->scalar_type() != st || t->sizes() != shape || !t->is_contiguous())
        wrong(*t, name, st, shape, dev);
    return t->data_ptr();
}
template <typename T> T* at_of(const Tensor* t, const char* name, ScalarType st, IntArrayRef shape, int dev) {
    return static_cast<T*>(at_of(t, name, st, shape, dev));
}

int rows_dtype(ScalarType st, const char* name) {
    switch (st) {
        case at::kBFloat16: return MOE_DTYPE_BF16;
        case at::kHalf: return MOE_DTYPE_FP16;
        case at::kFloat: return MOE_DTYPE_FP32;
        default: break;
    }
    std::ostringstream s;
    s << name << ": bf16, fp16 or fp32 is needed, got " << st;
    throw Refused(s.str());
}
ScalarType scalar_type(int dtype) {
    switch (dtype) {
        case MOE_DTYPE_BF16: return at::kBFloat16;
        case MOE_DTYPE_FP16: return at::kHalf;
        case MOE_DTYPE_FP32: return at::kFloat;
    }
    throw Refused("dtype: bf16, fp16 or fp32 is needed");
}

int32_t small(int64_t n, const char* name) {
    if (n > std::numeric_limits<int32_t>::max() || n < std::numeric_limits<int32_t>::min())
        throw Refused(std::string(name) + ": does not fit 32 bits");
    return (int32_t)n;
}
// Sizes of a matrix.
std::pair<int32_t, int32_t> matrix(const Tensor& t, const char* name) {
    if (t.dim() != 2) {
        std::ostringstream s;
        s << name << ": a matrix is needed, got shape " << t.sizes();
        throw Refused(s.str());
    }
    return {small(t.size(0), name), small(t.size(1), name)};
}
int32_t integer(PyObject* o, const char* name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused(std::string(name) + ": an integer is needed");
    }
    return small(v, name);
}
float real(PyObject* o, const char* name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused(std::string(name) + ": a number is needed");
    }
    return (float)v;
}

bool truth(PyObject* o, const char* name) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) {
        PyErr_Clear();
        throw Refused(std::string(name) + ": a truth value is needed");
    }
    return v > 0;
}

Tensor empty(IntArrayRef shape, ScalarType st, int dev) {
    return at::detail::empty_cuda(shape, st, c10::Device(c10::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
}
void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

// Moves on the version of the tensors that the caller gave to be written: automatic differentiation finds out that
// way that values it saved are gone.  (A tensor made in inference mode has no version.)
void written(std::initializer_list<const Tensor*> given) {
    for (const Tensor* t : given)
        if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

PyObject* wrap(const Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
template <typename... Ts> PyObject* pack(const Ts&... ts) {
    PyObject* tuple = PyTuple_New(sizeof...(Ts));
    Py_ssize_t i = 0;
    ((void)(tuple && (PyTuple_SET_ITEM(tuple, i, wrap(ts)), ++i)), ...);
    return tuple;
}

// ---- rows by expert --------------------------------------------------------------------------------
// dispatch_rows(x, idx, E, rows) -> (rows, offsets, perm, pos)
PyObject* dispatch_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect_args(n, 4, "dispatch_rows");
        const Tensor& idx = tensor(a[1], "idx");
        const Tensor *x = optional_tensor(a[0], "x"), *into = optional_tensor(a[3], "rows");
        const int32_t E = integer(a[2], "E");
        Unlocked unlocked;
        const int dev = device_of(idx, "idx");
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const auto [T, k] = matrix(idx, "idx");
        if (E < 1) throw Refused("E must be positive");
        const int64_t pairs = (int64_t)T * k;
        const auto* ip = at_of<int32_t>(&idx, "idx", at::kInt, {T, k}, dev);
        int32_t H = 8, dt = 0;
        void *xp = nullptr, *rp = nullptr;
        Tensor rows;
        if (x) {
            H = matrix(*x, "x").second;
            dt = rows_dtype(x->scalar_type(), "x");
            xp = at_of(x, "x", x->scalar_type(), {T, H}, dev);
            rows = into ? *into : empty({pairs, H}, x->scalar_type(), dev);
            rp = at_of(&rows, "rows", x->scalar_type(), {pairs, H}, dev);
        } else if (into) {
            throw Refused("rows needs x");
        }
        Tensor offsets = empty({(int64_t)E + 1}, at::kInt, dev), perm = empty({pairs}, at::kInt, dev), pos = empty({T, k}, at::kInt, dev);
        const size_t need = moe_dispatch_workspace(T, k, E);
        Tensor ws;
        if (need) ws = empty({(int64_t)need}, at::kByte, dev);
        check(moe_dispatch_rows(xp, dt, T, H, ip, k, E, rp, offsets.data_ptr<int32_t>(), perm.data_ptr<int32_t>(),
                                pos.data_ptr<int32_t>(), need ? ws.data_ptr() : nullptr, need, stream_of(dev)));
        written({into});
        unlocked.end();
        return pack(rows, offsets, perm, pos);
    });
}

// dispatch_rows_backward(drows, pos, out) -> dx
PyObject* dispatch_rows_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect_args(n, 3, "dispatch_rows_backward");
        const Tensor &drows = tensor(a[0], "drows"), &pos = tensor(a[1], "pos");
        const Tensor* into = optional_tensor(a[2], "out");
        Unlocked unlocked;
        const int dev = device_of(drows, "drows");
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const auto [R, H] = matrix(drows, "drows");
        const auto [T, k] = matrix(pos, "pos");
        const ScalarType st = drows.scalar_type();
        const int dt = rows_dtype(st, "drows");
        void* dp = at_of(&drows, "drows", st, {R, H}, dev);
        const auto* pp = at_of<int32_t>(&pos, "pos", at::kInt, {T, k}, dev);
        Tensor out = into ? *into : empty({T, H}, st, dev);
        void* op = at_of(&out, "out", st, {T, H}, dev);
        check(moe_dispatch_rows_backward(dp, dt, R, pp, T, k, H, op, stream_of(dev)));
        written({into});
        unlocked.end();
        return wrap(out);
    });
}

// combine_weighted(rows, pos, gates, base, out) -> out
PyObject* combine_weighted(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect_args(n, 5, "combine_weighted");
        const Tensor &rows = tensor(a[0], "rows"), &pos = tensor(a[1], "pos"), &gates = tensor(a[2], "gates");
        const Tensor *base = optional_tensor(a[3], "base"), *into = optional_tensor(a[4], "out");
        Unlocked unlocked;
        const int dev = device_of(rows, "rows");
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const auto [R, H] = matrix(rows, "rows");
        const auto [T, k] = matrix(pos, "pos");
        const ScalarType st = rows.scalar_type();
        const int dt = rows_dtype(st, "rows");
        void* rp = at_of(&rows, "rows", st, {R, H}, dev);
        const auto* pp = at_of<int32_t>(&pos, "pos", at::kInt, {T, k}, dev);
        const auto* gp = at_of<float>(&gates, "gates", at::kFloat, {T, k}, dev);
        void* bp = at_of(base, "base", st, {T, H}, dev);
        Tensor out = into ? *into : empty({T, H}, st, dev);
        void* op = at_of(&out, "out", st, {T, H}, dev);
        check(moe_combine_weighted(rp, dt, R, pp, gp, T, k, H, bp, op, stream_of(dev)));
        written({into});
        unlocked.end();
        return wrap(out);
    });
}

// combine_weighted_backward(dout, rows, pos, gates, drows) -> (drows, dgates)
PyObject* combine_weighted_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect_args(n, 5, "combine_weighted_backward");
        const Tensor &dout = tensor(a[0], "dout"), &rows = tensor(a[1], "rows"), &pos = tensor(a[2], "pos"),
                     &gates = tensor(a[3], "gates");
        const Tensor* into = optional_tensor(a[4], "drows");
        Unlocked unlocked;
        const int dev = device_of(rows, "rows");
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const auto [R, H] = matrix(rows, "rows");
        const auto [T, k] = matrix(pos, "pos");
        const ScalarType st = rows.scalar_type();
        const int dt = rows_dtype(st, "rows");
        void* op = at_of(&dout, "dout", st, {T, H}, dev);
        void* rp = at_of(&rows, "rows", st, {R, H}, dev);
        const auto* pp = at_of<int32_t>(&pos, "pos", at::kInt, {T, k}, dev);
        const auto* gp = at_of<float>(&gates, "gates", at::kFloat, {T, k}, dev);
        Tensor drows = into ? *into : empty({R, H}, st, dev), dgates = empty({T, k}, at::kFloat, dev);
        void* dp = at_of(&drows, "drows", st, {R, H}, dev);
        check(moe_combine_weighted_backward(op, dt, rp, R, pp, gp, T, k, H, dp, dgates.data_ptr<float>(), stream_of(dev)));
        written({into});
        unlocked.end();
        return pack(drows, dgates);
    });
}

// ---- block norms -----------------------------------------------------------------------------------
// block_norm(h, y, w_pre, w_post, gate, scale, eps, norm_post, n_dtype, h_out, n_out, pre)
//   -> (h, n, r_post, r_pre); n_dtype: MOE_DTYPE_* of n without y, -1 for h's
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect_args(n, 12, "block_norm");
        const Tensor& h = tensor(a[0], "h");
        const Tensor *y = optional_tensor(a[1], "y"), *w_pre = optional_tensor(a[2], "w_pre"),
                     *w_post = optional_tensor(a[3], "w_post"), *gate = optional_tensor(a[4], "gate"),
                     *h_into = optional_tensor(a[9], "h_out"), *n_into = optional_tensor(a[10], "n_out");
        const float scale = real(a[5], "scale"), eps = real(a[6], "eps");
        const bool norm_post = truth(a[7], "norm_post"), pre = truth(a[11], "pre");
        const int given = integer(a[8], "n_dtype");
        Unlocked unlocked;
        const int dev = device_of(h, "h");
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const auto [T, H] = matrix(h, "h");
        const ScalarType ht = h.scalar_type(), yt = y ? y->scalar_type() : given >= 0 ? scalar_type(given) : ht;
        const int hd = rows_dtype(ht, "h"), yd = rows_dtype(yt, "y");
        if (given >= 0 && given != yd) throw Refused("n has y's type");
        void *hp = at_of(&h, "h", ht, {T, H}, dev), *yp = at_of(y, "y", yt, {T, H}, dev);
        const auto *wp = at_of<float>(w_pre, "w_pre", at::kFloat, {H}, dev), *wq = at_of<float>(w_post, "w_post", at::kFloat, {H}, dev),
                   *gp = at_of<float>(gate, "gate", at::kFloat, {T}, dev);
        Tensor h_out, n_out, r_post, r_pre;
        if (h_into) h_out = *h_into;
        else if (y) h_out = empty({T, H}, ht, dev);
        if (n_into) n_out = *n_into;
        else if (pre) n_out = empty({T, H}, yt, dev);
        if (norm_post) r_post = empty({T}, at::kFloat, dev);
        if (pre) r_pre = empty({T}, at::kFloat, dev);
        void *op = h_out.defined() ? at_of(&h_out, "h_out", ht, {T, H}, dev) : nullptr;
        void *np = n_out.defined() ? at_of(&n_out, "n_out", yt, {T, H}, dev) : nullptr;
        check(moe_block_norm(hp, hd, yp, yd, T, H, wq, norm_post, gp, scale, wp, eps, op, np,
                             norm_post ? r_post.data_ptr<float>() : nullptr, pre ? r_pre.data_ptr<float>() : nullptr,
                             stream_of(dev)));
        written({h_into, n_into});
        unlocked.end();
        return pack(h_out, n_out, r_post, r_pre);
    });
}

// block_norm_backward(dn, dh_out, h_out, y, r_pre, r_post, w_pre, w_post, gate, scale)
//   -> (dh, dy, dw_pre, dw_post, dgate)
PyObject* block_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect_args(n, 10, "block_norm_backward");
        const Tensor& h = tensor(a[2], "h_out");
        const Tensor *dn = optional_tensor(a[0], "dn"), *dh_in = optional_tensor(a[1], "dh_out"), *y = optional_tensor(a[3], "y"),
                     *r_pre = optional_tensor(a[4], "r_pre"), *r_post = optional_tensor(a[5], "r_post"),
                     *w_pre = optional_tensor(a[6], "w_pre"), *w_post = optional_tensor(a[7], "w_post"),
                     *gate = optional_tensor(a[8], "gate");
        const float scale = real(a[9], "scale");
        Unlocked unlocked;
        const int dev = device_of(h, "h_out");
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const auto [T, H] = matrix(h, "h_out");
        const ScalarType ht = h.scalar_type(), yt = y ? y->scalar_type() : dn ? dn->scalar_type() : ht;
        const int hd = rows_dtype(ht, "h_out"), yd = rows_dtype(yt, "y");
        void *np = at_of(dn, "dn", yt, {T, H}, dev), *ip = at_of(dh_in, "dh_out", ht, {T, H}, dev),
             *hp = at_of(&h, "h_out", ht, {T, H}, dev), *yp = at_of(y, "y", yt, {T, H}, dev);
        const auto *rp = at_of<float>(r_pre, "r_pre", at::kFloat, {T}, dev), *rq = at_of<float>(r_post, "r_post", at::kFloat, {T}, dev),
                   *wp = at_of<float>(w_pre, "w_pre", at::kFloat, {H}, dev), *wq = at_of<float>(w_post, "w_post", at::kFloat, {H}, dev),
                   *gp = at_of<float>(gate, "gate", at::kFloat, {T}, dev);
        Tensor dh = empty({T, H}, ht, dev), dy, dw_pre, dw_post, dgate, ws;
        if (y) dy = empty({T, H}, yt, dev);
        if (w_pre) dw_pre = empty({H}, at::kFloat, dev);
        if (w_post) dw_post = empty({H}, at::kFloat, dev);
        if (gate) dgate = empty({T}, at::kFloat, dev);
        const size_t need = w_pre || w_post ? moe_block_norm_backward_workspace(T, H) : 0;
        if (need) ws = empty({(int64_t)need}, at::kByte, dev);
        auto ptr = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
        check(moe_block_norm_backward(np, ip, hp, hd, yp, yd, T, H, rp, rq, wp, wq, r_post != nullptr, gp, scale, ptr(dh), ptr(dy),
                                      static_cast<float*>(ptr(dw_pre)), static_cast<float*>(ptr(dw_post)),
                                      static_cast<float*>(ptr(dgate)), ptr(ws), need, stream_of(dev)));
        unlocked.end();
        return pack(dh, dy, dw_pre, dw_post, dgate);
    });
}

// ---- microscaled 4-bit floating point --------------------------------------------------------------
// mx4_quantize(x, pos, act, codes, scales) -> (codes, scales)
PyObject* mx4_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect_args(n, 5, "mx4_quantize");
        const Tensor& x = tensor(a[0], "x");
        const Tensor *pos = optional_tensor(a[1], "pos"), *c_into = optional_tensor(a[3], "codes"), *s_into = optional_tensor(a[4], "scales");
        const int act = integer(a[2], "act");
        Unlocked unlocked;
        const int dev = device_of(x, "x");
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const auto [T, W] = matrix(x, "x");
        if (act == MOE_ACT_SWIGLU && W % 2) throw Refused("x: swiglu needs rows of an even width");
        const int32_t K = act == MOE_ACT_SWIGLU ? W / 2 : W;
        const int dt = rows_dtype(x.scalar_type(), "x");
        void* xp = at_of(&x, "x", x.scalar_type(), {T, W}, dev);
        const int32_t k = pos ? matrix(*pos, "pos").second : 1;
        if (k < 1) throw Refused("pos: at least one place per token is needed");   // (its address would be NULL)
        const auto* pp = at_of<int32_t>(pos, "pos", at::kInt, {T, k}, dev);
        const int32_t rows = c_into ? matrix(*c_into, "codes").first : small((int64_t)T * k, "pos");
        Tensor codes = c_into ? *c_into : empty({rows, K / 2}, at::kByte, dev);
        Tensor scales = s_into ? *s_into : empty({rows, K / 32}, at::kByte, dev);
        auto* cp = at_of<uint8_t>(&codes, "codes", at::kByte, {rows, K / 2}, dev);
        auto* sp = at_of<uint8_t>(&scales, "scales", at::kByte, {rows, K / 32}, dev);
        check(moe_mx4_quantize(xp, dt, T, K, act, pp, k, rows, cp, sp, stream_of(dev)));
        written({c_into, s_into});
        unlocked.end();
        return pack(codes, scales);
    });
}

// mx4_dequantize(codes, scales, dtype) -> values
PyObject* mx4_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect_args(n, 3, "mx4_dequantize");
        const Tensor &codes = tensor(a[0], "codes"), &scales = tensor(a[1], "scales");
        const int dt = integer(a[2], "dtype");
        Unlocked unlocked;
        const int dev = device_of(codes, "codes");
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        if (codes.dim() < 1) throw Refused("codes: a tensor of rows is needed");
        std::vector<int64_t> shape = codes.sizes().vec();
        const auto* cp = at_of<uint8_t>(&codes, "codes", at::kByte, shape, dev);
        const int32_t K = small(2 * shape.back(), "codes");
        shape.back() = K / 32;
        const auto* sp = at_of<uint8_t>(&scales, "scales", at::kByte, shape, dev);
        shape.back() = K;
        Tensor out = empty(shape, scalar_type(dt), dev);
        check(moe_mx4_dequantize(cp, sp, K ? out.numel() / K : 0, K, out.data_ptr(), dt, stream_of(dev)));
        unlocked.end();
        return wrap(out);
    });
}

// mx4_matmul(codes, scales, w_codes, w_scales, offsets, out, dtype) -> y
PyObject* mx4_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect_args(n, 7, "mx4_matmul");
        const Tensor &codes = tensor(a[0], "codes"), &scales = tensor(a[1], "scales"), &w_codes = tensor(a[2], "w_codes"),
                     &w_scales = tensor(a[3], "w_scales"), &offsets = tensor(a[4], "offsets");
        const Tensor* into = optional_tensor(a[5], "out");
        const int dt = integer(a[6], "dtype");
        Unlocked unlocked;
        const int dev = device_of(codes, "codes");
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const auto [R, Kh] = matrix(codes, "codes");
        if (w_codes.dim() != 3) throw Refused("w_codes: [E, N, K/2] is needed");
        const int32_t E = small(w_codes.size(0), "w_codes"), N = small(w_codes.size(1), "w_codes"), K = small(2 * (int64_t)Kh, "codes");
        const auto* cp = at_of<uint8_t>(&codes, "codes", at::kByte, {R, Kh}, dev);
        const auto* sp = at_of<uint8_t>(&scales, "scales", at::kByte, {R, Kh / 16}, dev);
        const auto* wp = at_of<uint8_t>(&w_codes, "w_codes", at::kByte, {E, N, Kh}, dev);
        const auto* wq = at_of<uint8_t>(&w_scales, "w_scales", at::kByte, {E, N, Kh / 16}, dev);
        const auto* fp = at_of<int32_t>(&offsets, "offsets", at::kInt, {(int64_t)E + 1}, dev);
        Tensor out = into ? *into : empty({R, N}, scalar_type(dt), dev);
        void* op = at_of(&out, "out", out.scalar_type(), {R, N}, dev);
        check(moe_mx4_matmul(cp, sp, R, K, wp, wq, E, N, fp, op, rows_dtype(out.scalar_type(), "out"), stream_of(dev)));
        written({into});
        unlocked.end();
        return wrap(out);
    });
}

PyObject* set_error(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XSETREF(g_moe_error, cls);
    Py_RETURN_NONE;
}

#define OPS_FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {OPS_FAST(dispatch_rows),
                          OPS_FAST(dispatch_rows_backward),
                          OPS_FAST(combine_weighted),
                          OPS_FAST(combine_weighted_backward),
                          OPS_FAST(block_norm),
                          OPS_FAST(block_norm_backward),
                          OPS_FAST(mx4_quantize),
                          OPS_FAST(mx4_dequantize),
                          OPS_FAST(mx4_matmul),
                          {"set_error", set_error, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_ops", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_ops() {
    PyObject* m = PyModule_Create(&kModule);
    if (m && PyModule_AddStringConstant(m, "built_for", MOE_BUILT_FOR) < 0) Py_CLEAR(m);
    return m;
}
