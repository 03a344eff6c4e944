// The binding of the calls around the layer and of the 4-bit experts: checks of the arguments,
// outputs from torch's allocator, the C ABI's call on torch's current stream. It is native
// because these calls are small: a norm of one token takes the GPU 3 us, and from Python its
// checks, two allocations and the foreign call took 12 (6 here). moe.py documents the functions
// and passes every argument by position; what is refused raises the exception class given to
// init() (MoeError).
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "moe.h"

namespace {

PyObject* g_error = nullptr;  // MoeError

struct Refused {
    std::string what;
};
struct PyRaised {};  // a Python exception is set

std::string shape_of(at::IntArrayRef s)
{
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

const char* type_name(at::ScalarType t)
{
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kHalf: return "torch.float16";
        case at::kFloat: return "torch.float32";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kByte: return "torch.uint8";
        default: return c10::toString(t);
    }
}

// a tensor argument, NULL for None
const at::Tensor* tensor(PyObject* o, const char* name)
{
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw Refused{std::string(name) + ": a tensor is expected"};
    return &THPVariable_Unpack(o);
}

void need(const at::Tensor* t, const char* name, at::ScalarType dtype, at::IntArrayRef shape,
          const at::Device& dev)
{
    if (t == nullptr) throw Refused{std::string(name) + " is required"};
    if (t->scalar_type() != dtype)
        throw Refused{std::string(name) + ": dtype " + type_name(t->scalar_type()) + ", expected " +
                      type_name(dtype)};
    if (t->sizes() != shape)
        throw Refused{std::string(name) + ": shape " + shape_of(t->sizes()) + ", expected " +
                      shape_of(shape)};
    if (t->device() != dev)
        throw Refused{std::string(name) + ": on " + t->device().str() + ", expected " + dev.str()};
    if (!t->is_contiguous()) throw Refused{std::string(name) + " must be contiguous"};
}

void need_opt(const at::Tensor* t, const char* name, at::ScalarType dtype, at::IntArrayRef shape,
              const at::Device& dev)
{
    if (t != nullptr) need(t, name, dtype, shape, dev);
}

// a workspace that the caller keeps: `bytes` consecutive bytes of the device, of any type
void need_ws(const at::Tensor& t, size_t bytes, const at::Device& dev)
{
    if (t.device() != dev)
        throw Refused{"workspace on " + t.device().str() + ", expected " + dev.str()};
    if (!t.is_contiguous()) throw Refused{"the workspace must be contiguous"};
    if (t.nbytes() < bytes)
        throw Refused{"workspace of " + std::to_string(t.nbytes()) + " bytes < " +
                      std::to_string(bytes)};
}

// MOE_BF16 .. of a type, -1 of others
int code_of(at::ScalarType t)
{
    return t == at::kBFloat16 ? MOE_BF16 : t == at::kHalf ? MOE_F16 : t == at::kFloat ? MOE_F32 : -1;
}

// a contiguous 2-D bf16, fp16 or fp32 tensor
const at::Tensor& activation(PyObject* o, const char* name)
{
    const at::Tensor* t = tensor(o, name);
    if (t == nullptr) throw Refused{std::string(name) + " is required"};
    if (code_of(t->scalar_type()) < 0 || t->dim() != 2)
        throw Refused{std::string(name) + ": a 2-D bf16, fp16 or fp32 tensor is expected, got " +
                      type_name(t->scalar_type()) + " " + shape_of(t->sizes())};
    if (!t->is_contiguous()) throw Refused{std::string(name) + " must be contiguous"};
    return *t;
}

void need_cuda(const at::Device& dev)
{
    if (!dev.is_cuda()) throw Refused{"tensors on " + dev.str() + ", expected a CUDA device"};
}

const void* ptr(const at::Tensor* t) { return t == nullptr ? nullptr : t->const_data_ptr(); }
void* out_ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

double number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PyRaised{};
    return v;
}

int64_t integer(PyObject* o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PyRaised{};
    return v;
}

int truth(PyObject* o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PyRaised{};
    return v;
}

int64_t attribute(PyObject* o, const char* name)
{
    PyObject* v = PyObject_GetAttrString(o, name);
    if (v == nullptr) throw PyRaised{};
    const long long r = PyLong_AsLongLong(v);
    Py_DECREF(v);
    if (r == -1 && PyErr_Occurred()) throw PyRaised{};
    return r;
}

int32_t int32_of(int64_t v)  // out of range: a value that every size check refuses
{
    return v == (int32_t)v ? (int32_t)v : -1;
}

moe_cfg config(PyObject* o)
{
    moe_cfg c{};
    c.T = int32_of(attribute(o, "T"));
    c.H = int32_of(attribute(o, "H"));
    c.E = int32_of(attribute(o, "E"));
    c.K = int32_of(attribute(o, "K"));
    c.I = int32_of(attribute(o, "I"));
    c.I_shared = int32_of(attribute(o, "I_shared"));
    c.score_fn = int32_of(attribute(o, "score_fn"));
    c.n_group = int32_of(attribute(o, "n_group"));
    c.topk_group = int32_of(attribute(o, "topk_group"));
    PyObject* v = PyObject_GetAttrString(o, "renorm");
    if (v == nullptr) throw PyRaised{};
    c.renorm = PyObject_IsTrue(v) > 0;
    Py_DECREF(v);
    v = PyObject_GetAttrString(o, "route_scale");
    if (v == nullptr) throw PyRaised{};
    c.route_scale = (float)PyFloat_AsDouble(v);
    Py_DECREF(v);
    if (PyErr_Occurred()) throw PyRaised{};
    return c;
}

// f(stream) on dev's current stream, with dev the current device and the interpreter released
template <typename F>
void call(const at::Device& dev, const char* what, F f)
{
    need_cuda(dev);
    int rc;
    {
        const c10::cuda::OptionalCUDAGuard guard(dev);
        void* stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
        Py_BEGIN_ALLOW_THREADS
        rc = f(stream);
        Py_END_ALLOW_THREADS
    }
    if (rc != MOE_OK)
        throw Refused{std::string(what) + ": " + moe_status_string(rc) + " (" + std::to_string(rc) +
                      ")"};
}

PyObject* wrap(const at::Tensor& t)
{
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject* tuple2(PyObject* a, PyObject* b)
{
    PyObject* r = a != nullptr && b != nullptr ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return r;
}

// arguments of a call by position
void expect(Py_ssize_t got, Py_ssize_t want)
{
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", got, want);
        throw PyRaised{};
    }
}

// what residual_norm and its backward share, from args[0..]: w_post, gate, w_next, eps,
// residual_scale, branch_scale, p, rng, first_row, row_ids
struct Norm {
    moe_norm_cfg cfg{};
    const at::Tensor *y, *w_post, *gate, *w_next, *rng, *row_ids;
};

Norm norm_setup(const at::Tensor& x, const at::Tensor* y, PyObject* const* a)
{
    Norm n;
    const at::ScalarType dt = x.scalar_type();
    const at::Device dev = x.device();
    const int64_t T = x.size(0), H = x.size(1);
    n.y = y;
    n.w_post = tensor(a[0], "w_post");
    n.gate = tensor(a[1], "gate");
    n.w_next = tensor(a[2], "w_next");
    const double eps = number(a[3]), rs = number(a[4]), bs = number(a[5]), p = number(a[6]);
    n.rng = tensor(a[7], "rng");
    const int64_t first_row = integer(a[8]);
    n.row_ids = tensor(a[9], "row_ids");
    if (y != nullptr) {
        need(y, "y", dt, x.sizes(), dev);
    } else if (n.w_post != nullptr || n.gate != nullptr || p != 0.0 || n.w_next == nullptr ||
               rs != 1.0) {
        throw Refused{"without y there is only the norm: w_next is required, and w_post, gate, p "
                      "and residual_scale do not apply"};
    }
    int mode = MOE_GATE_NONE;
    if (n.gate != nullptr) {
        const at::IntArrayRef s = n.gate->sizes();
        if (s.size() == 1 && s[0] == H) mode = MOE_GATE_CHANNEL;
        else if (s.size() == 2 && s[0] == T && s[1] == 1) mode = MOE_GATE_TOKEN;
        else if (s == x.sizes()) mode = MOE_GATE_FULL;
        else
            throw Refused{"gate: shape " + shape_of(s) + ", expected " + shape_of({H}) + ", " +
                          shape_of({T, 1}) + " or " + shape_of({T, H})};
    }
    const at::Tensor* small = mode == MOE_GATE_FULL ? nullptr : n.gate;
    if (mode == MOE_GATE_FULL) need(n.gate, "gate", dt, x.sizes(), dev);
    const at::Tensor* first = n.w_post != nullptr ? n.w_post : n.w_next != nullptr ? n.w_next : small;
    const at::ScalarType pd = first == nullptr ? at::kFloat : first->scalar_type();
    if (pd != at::kFloat && pd != dt)
        throw Refused{std::string("parameters: dtype ") + type_name(pd) +
                      ", expected torch.float32 or " + type_name(dt)};
    need_opt(n.w_post, "w_post", pd, {H}, dev);
    need_opt(n.w_next, "w_next", pd, {H}, dev);
    if (small != nullptr) need(small, "gate", pd, small->sizes(), dev);
    if (p != 0.0) need(n.rng, "rng", at::kLong, {2}, dev);
    else n.rng = nullptr;
    need_opt(n.row_ids, "row_ids", at::kInt, {T}, dev);
    n.cfg.T = T;
    n.cfg.first_row = first_row;
    n.cfg.p = p;
    n.cfg.H = int32_of(H);
    n.cfg.dtype = code_of(dt);
    n.cfg.param_dtype = code_of(pd);
    n.cfg.gate = mode;
    n.cfg.eps = (float)eps;
    n.cfg.residual_scale = (float)rs;
    n.cfg.branch_scale = (float)bs;
    return n;
}

// an output argument: given (checked) or allocated like x
at::Tensor output(PyObject* o, const char* name, const at::Tensor& x)
{
    const at::Tensor* t = tensor(o, name);
    if (t == nullptr) return at::empty_like(x);
    need(t, name, x.scalar_type(), x.sizes(), x.device());
    return *t;
}

// x, y, w_post, gate, w_next, eps, residual_scale, branch_scale, p, rng, first_row, row_ids, r, n
PyObject* residual_norm(PyObject* const* a)
{
    const at::Tensor& x = activation(a[0], "x");
    const Norm s = norm_setup(x, tensor(a[1], "y"), a + 2);
    at::Tensor r, n;
    if (s.y != nullptr) r = output(a[12], "r", x);
    else if (a[12] != Py_None) throw Refused{"without y, r is x: no output to write"};
    if (s.w_next != nullptr) n = output(a[13], "n", x);
    else if (a[13] != Py_None) throw Refused{"n needs w_next"};
    call(x.device(), "moe_residual_norm", [&](void* stream) {
        return moe_residual_norm(&s.cfg, ptr(&x), ptr(s.y), ptr(s.w_post), ptr(s.gate),
                                 ptr(s.w_next), static_cast<const int64_t*>(ptr(s.rng)),
                                 static_cast<const int32_t*>(ptr(s.row_ids)), out_ptr(r),
                                 out_ptr(n), stream);
    });
    return tuple2(wrap(s.y != nullptr ? r : x), wrap(n));
}

// r, y, dr, dn, w_post, gate, w_next, eps, residual_scale, branch_scale, p, rng, first_row, row_ids
PyObject* residual_norm_backward(PyObject* const* a)
{
    const at::Tensor& r = activation(a[0], "r");
    const at::Tensor *dr = tensor(a[2], "dr"), *dn = tensor(a[3], "dn");
    const Norm s = norm_setup(r, tensor(a[1], "y"), a + 4);
    const at::Device dev = r.device();
    need_opt(dr, "dr", r.scalar_type(), r.sizes(), dev);
    need_opt(dn, "dn", r.scalar_type(), r.sizes(), dev);
    if ((dn == nullptr) != (s.w_next == nullptr)) throw Refused{"dn is given exactly with w_next"};
    if (dr == nullptr && dn == nullptr) throw Refused{"dr or dn is required"};
    need_cuda(dev);
    const auto f32 = at::TensorOptions().dtype(at::kFloat).device(dev);
    at::Tensor dx = at::empty_like(r), dy, dw_post, dgate, dw_next;
    if (s.y != nullptr) dy = at::empty_like(r);
    if (s.w_post != nullptr) dw_post = at::empty(s.w_post->sizes(), f32);
    if (s.gate != nullptr)
        dgate = s.cfg.gate == MOE_GATE_FULL ? at::empty_like(r) : at::empty(s.gate->sizes(), f32);
    if (s.w_next != nullptr) dw_next = at::empty(s.w_next->sizes(), f32);
    const size_t bytes = moe_residual_norm_workspace_bytes(&s.cfg);
    const at::Tensor ws = at::empty({(int64_t)(bytes > 16 ? bytes : 16)}, f32.dtype(at::kByte));
    call(dev, "moe_residual_norm_backward", [&](void* stream) {
        return moe_residual_norm_backward(
            &s.cfg, ptr(&r), ptr(s.y), ptr(s.w_post), ptr(s.gate), ptr(s.w_next),
            static_cast<const int64_t*>(ptr(s.rng)), static_cast<const int32_t*>(ptr(s.row_ids)),
            ptr(dr), ptr(dn), out_ptr(dx), out_ptr(dy), static_cast<float*>(out_ptr(dw_post)),
            out_ptr(dgate), static_cast<float*>(out_ptr(dw_next)), out_ptr(ws), bytes, stream);
    });
    PyObject* d = PyDict_New();
    if (d == nullptr) return nullptr;
    const std::pair<const char*, const at::Tensor*> g[] = {
        {"dx", &dx}, {"dy", &dy}, {"dw_post", &dw_post}, {"dgate", &dgate}, {"dw_next", &dw_next}};
    for (const auto& e : g) {
        if (!e.second->defined()) continue;
        PyObject* v = wrap(*e.second);
        if (v == nullptr || PyDict_SetItemString(d, e.first, v) < 0) {
            Py_XDECREF(v);
            Py_DECREF(d);
            return nullptr;
        }
        Py_DECREF(v);
    }
    return d;
}

// x, p, rng, first_row, row_ids, out
PyObject* dropout(PyObject* const* a)
{
    const at::Tensor& x = activation(a[0], "x");
    const double p = number(a[1]);
    const at::Tensor *rng = tensor(a[2], "rng"), *row_ids = tensor(a[4], "row_ids");
    const int64_t first_row = integer(a[3]);
    need(rng, "rng", at::kLong, {2}, x.device());
    need_opt(row_ids, "row_ids", at::kInt, {x.size(0)}, x.device());
    const at::Tensor out = output(a[5], "out", x);
    call(x.device(), "moe_dropout", [&](void* stream) {
        return moe_dropout(x.size(0), int32_of(x.size(1)), code_of(x.scalar_type()), p, ptr(&x),
                           static_cast<const int64_t*>(ptr(rng)), first_row,
                           static_cast<const int32_t*>(ptr(row_ids)), out_ptr(out), stream);
    });
    return wrap(out);
}

at::Tensor bytes_like(const at::Tensor& t, at::IntArrayRef shape)
{
    return at::empty(shape, at::TensorOptions().dtype(at::kByte).device(t.device()));
}

int64_t ceil128(int64_t v) { return (v + 127) / 128; }

// x, tiled
PyObject* mx_quantize(PyObject* const* a)
{
    const at::Tensor& x = activation(a[0], "x");
    const int tiled = truth(a[1]);
    const int64_t R = x.size(0), K = x.size(1);
    need_cuda(x.device());
    const at::Tensor codes = bytes_like(x, {R, K / 2});
    const at::Tensor scales = tiled ? bytes_like(x, {ceil128(R), ceil128(K), 512})
                                    : bytes_like(x, {R, K / 32});
    call(x.device(), "moe_mx_quantize", [&](void* stream) {
        return moe_mx_quantize(R, int32_of(K), code_of(x.scalar_type()), tiled, ptr(&x),
                               static_cast<uint8_t*>(out_ptr(codes)),
                               static_cast<uint8_t*>(out_ptr(scales)), stream);
    });
    return tuple2(wrap(codes), wrap(scales));
}

// codes, scales, dtype
PyObject* mx_dequantize(PyObject* const* a)
{
    const at::Tensor *codes = tensor(a[0], "codes"), *scales = tensor(a[1], "scales");
    const at::ScalarType dt =
        THPDtype_Check(a[2]) ? reinterpret_cast<THPDtype*>(a[2])->scalar_type : at::kByte;
    if (codes == nullptr || codes->dim() != 2 || code_of(dt) < 0 || codes->size(1) % 16 != 0)
        throw Refused{"codes " + (codes == nullptr ? std::string("None") : shape_of(codes->sizes())) +
                      " to " + type_name(dt) +
                      ": [R, K/2] with K a multiple of 32, and bf16, fp16 or fp32, are expected"};
    const int64_t R = codes->size(0), K = 2 * codes->size(1);
    const at::Device dev = codes->device();
    need(codes, "codes", at::kByte, {R, K / 2}, dev);
    const int tiled = scales != nullptr && scales->dim() == 3;
    if (tiled) need(scales, "scales", at::kByte, {ceil128(R), ceil128(K), 512}, dev);
    else need(scales, "scales", at::kByte, {R, K / 32}, dev);
    need_cuda(dev);
    const at::Tensor out = at::empty({R, K}, at::TensorOptions().dtype(dt).device(dev));
    call(dev, "moe_mx_dequantize", [&](void* stream) {
        return moe_mx_dequantize(R, int32_of(K), code_of(dt), tiled,
                                 static_cast<const uint8_t*>(ptr(codes)),
                                 static_cast<const uint8_t*>(ptr(scales)), out_ptr(out), stream);
    });
    return wrap(out);
}

// codes, scales, offsets, w_codes, w_scales, swiglu, out, status
PyObject* mx_grouped_gemm(PyObject* const* a)
{
    const at::Tensor *codes = tensor(a[0], "codes"), *scales = tensor(a[1], "scales");
    const at::Tensor *offsets = tensor(a[2], "offsets"), *wc = tensor(a[3], "w_codes");
    const at::Tensor *ws = tensor(a[4], "w_scales"), *given = tensor(a[6], "out");
    const at::Tensor* status = tensor(a[7], "status");
    const int swiglu = truth(a[5]);
    if (codes == nullptr || wc == nullptr || codes->dim() != 2 || wc->dim() != 3)
        throw Refused{"codes [R, K/2] and w_codes [E, N, K/2] are expected"};
    const int64_t R = codes->size(0), K = 2 * codes->size(1), E = wc->size(0), n = wc->size(1);
    const int64_t unit = swiglu ? 256 : 128;
    if (n % unit != 0 || K % 128 != 0)
        throw Refused{"N " + std::to_string(n) + " and K " + std::to_string(K) + ": multiples of " +
                      std::to_string(unit) + " and 128"};
    const at::Device dev = codes->device();
    need(codes, "codes", at::kByte, {R, K / 2}, dev);
    need(scales, "scales", at::kByte, {ceil128(R), K / 128, 512}, dev);
    need(offsets, "offsets", at::kInt, {E + 1}, dev);
    need(wc, "w codes", at::kByte, {E, n, K / 2}, dev);
    need(ws, "w scales", at::kByte, {E, n / 128, K / 128, 512}, dev);
    need_opt(status, "status", at::kInt, {MOE_STATUS_WORDS}, dev);
    need_cuda(dev);
    const int64_t cols = swiglu ? n / 2 : n;
    at::Tensor out;
    if (given != nullptr) {
        need(given, "out", at::kBFloat16, {R, cols}, dev);
        out = *given;
    } else {
        out = at::empty({R, cols}, at::TensorOptions().dtype(at::kBFloat16).device(dev));
    }
    call(dev, "moe_mx_grouped_gemm", [&](void* stream) {
        return moe_mx_grouped_gemm(
            R, int32_of(K), int32_of(n), int32_of(E), swiglu,
            static_cast<const uint8_t*>(ptr(codes)), static_cast<const uint8_t*>(ptr(scales)),
            static_cast<const int32_t*>(ptr(offsets)), static_cast<const uint8_t*>(ptr(wc)),
            static_cast<const uint8_t*>(ptr(ws)), static_cast<uint16_t*>(out_ptr(out)),
            static_cast<int32_t*>(status == nullptr ? nullptr : status->data_ptr()), stream);
    });
    return wrap(out);
}

// (codes, tiled scales) of matrices [n, k], `lead` of them (0: one, without the dimension), held:
// a sequence may make its members when asked, and then nothing else refers to them
struct MxWeight {
    at::Tensor codes, scales;
};

const uint8_t* bytes_of(const at::Tensor& t)  // NULL for none
{
    return t.defined() ? static_cast<const uint8_t*>(t.const_data_ptr()) : nullptr;
}

MxWeight mx_weight(PyObject* o, const char* name, int64_t lead, int64_t n, int64_t k,
                   const at::Device& dev)
{
    PyObject* s = PySequence_Check(o) && !THPVariable_Check(o) ? PySequence_Fast(o, "") : nullptr;
    if (s == nullptr || PySequence_Fast_GET_SIZE(s) != 2) {
        PyErr_Clear();
        Py_XDECREF(s);
        throw Refused{std::string(name) + ": (codes, scales) of mx_weight() are expected"};
    }
    struct Release {
        PyObject* o;
        ~Release() { Py_DECREF(o); }
    } const release{s};
    const std::string cn = std::string(name) + " codes", sn = std::string(name) + " scales";
    const at::Tensor *codes = tensor(PySequence_Fast_GET_ITEM(s, 0), cn.c_str());
    const at::Tensor *scales = tensor(PySequence_Fast_GET_ITEM(s, 1), sn.c_str());
    if (lead > 0) {
        need(codes, cn.c_str(), at::kByte, {lead, n, k / 2}, dev);
        need(scales, sn.c_str(), at::kByte, {lead, n / 128, k / 128, 512}, dev);
    } else {
        need(codes, cn.c_str(), at::kByte, {n, k / 2}, dev);
        need(scales, sn.c_str(), at::kByte, {n / 128, k / 128, 512}, dev);
    }
    return {*codes, *scales};
}

// cfg, x, dest_row, offsets, w13, w2, w13_s, w2_s, ws, status
PyObject* mx_grouped_ffn(PyObject* const* a)
{
    const moe_cfg c = config(a[0]);
    const at::Tensor *x = tensor(a[1], "x"), *dest = tensor(a[2], "dest_row");
    const at::Tensor *offsets = tensor(a[3], "offsets"), *given = tensor(a[8], "ws");
    const at::Tensor* status = tensor(a[9], "status");
    if (x == nullptr) throw Refused{"x is required"};
    const at::Device dev = x->device();
    need(x, "x", at::kBFloat16, {c.T, c.H}, dev);
    need(dest, "dest_row", at::kInt, {c.T, c.K}, dev);
    need(offsets, "offsets", at::kInt, {(int64_t)c.E + 1}, dev);
    const MxWeight w13 = mx_weight(a[4], "w13", c.E, 2 * (int64_t)c.I, c.H, dev);
    const MxWeight w2 = mx_weight(a[5], "w2", c.E, c.H, c.I, dev);
    MxWeight w13s, w2s;
    if (c.I_shared > 0) {
        w13s = mx_weight(a[6], "w13_s", 0, 2 * (int64_t)c.I_shared, c.H, dev);
        w2s = mx_weight(a[7], "w2_s", 0, c.H, c.I_shared, dev);
    }
    need_opt(status, "status", at::kInt, {MOE_STATUS_WORDS}, dev);
    const size_t bytes = moe_workspace_bytes(&c, MOE_STAGE_MX_FFN);
    if (given != nullptr) need_ws(*given, bytes, dev);
    need_cuda(dev);
    const auto bf16 = at::TensorOptions().dtype(at::kBFloat16).device(dev);
    const at::Tensor y = at::empty({(int64_t)c.T * c.K, c.H}, bf16);
    const at::Tensor ys = c.I_shared > 0 ? at::empty({c.T, c.H}, bf16) : at::Tensor();
    const at::Tensor ws =
        given != nullptr ? *given
                         : at::empty({(int64_t)(bytes > 16 ? bytes : 16)}, bf16.dtype(at::kByte));
    call(dev, "moe_mx_grouped_ffn", [&](void* stream) {
        return moe_mx_grouped_ffn(
            &c, static_cast<const uint16_t*>(ptr(x)), static_cast<const int32_t*>(ptr(dest)),
            static_cast<const int32_t*>(ptr(offsets)), bytes_of(w13.codes), bytes_of(w13.scales),
            bytes_of(w2.codes), bytes_of(w2.scales), bytes_of(w13s.codes), bytes_of(w13s.scales),
            bytes_of(w2s.codes), bytes_of(w2s.scales), static_cast<uint16_t*>(out_ptr(y)),
            static_cast<uint16_t*>(out_ptr(ys)),
            static_cast<int32_t*>(status == nullptr ? nullptr : status->data_ptr()), out_ptr(ws),
            bytes, stream);
    });
    return tuple2(wrap(y), wrap(ys));
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t nargs)
{
    HANDLE_TH_ERRORS
    try {
        expect(nargs, N);
        return F(args);
    } catch (const Refused& e) {
        PyErr_SetString(g_error, e.what.c_str());
        return nullptr;
    } catch (const PyRaised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject* init(PyObject*, PyObject* error)
{
    Py_INCREF(error);
    Py_XSETREF(g_error, error);
    Py_RETURN_NONE;
}

#define FAST(name, n)                                                              \
    {                                                                              \
        #name, reinterpret_cast<PyCFunction>(                                      \
                   reinterpret_cast<void (*)()>(&entry<&name, n>)), METH_FASTCALL, \
            nullptr                                                                \
    }

PyMethodDef kMethods[] = {{"init", init, METH_O, nullptr},
                          FAST(residual_norm, 14),
                          FAST(residual_norm_backward, 14),
                          FAST(dropout, 6),
                          FAST(mx_quantize, 2),
                          FAST(mx_dequantize, 3),
                          FAST(mx_grouped_gemm, 8),
                          FAST(mx_grouped_ffn, 10),
                          {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "moe_binding", nullptr, -1, kMethods,
                       nullptr,               nullptr,       nullptr, nullptr};

}  // namespace

// what this file was compiled against (a macro of the build), read from the built file before it is
// loaded: another torch's C++ interface is not this one's
extern "C" __attribute__((used, visibility("default"))) const char moe_binding_built_for[] =
    "moe_binding built for " MOE_BINDING_TARGET;

PyMODINIT_FUNC PyInit_moe_binding(void) { return PyModule_Create(&kModule); }
