// fa_binding.cpp -- host side of the Python calls of the operators around cached attention.
//
// Argument marshalling only, as in the ctypes binding beside it: every argument's type, shape,
// device and layout is checked, outputs that were not given are allocated, the current stream is
// looked up, and the C ABI of include/fa.h is called.  These operators are called once or twice a
// layer in a serving loop; through ctypes and Python checks a call took 12 to 25 us of host time on
// the GB300's Grace cores, several times the kernels'.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <array>
#include <cmath>
#include <initializer_list>
#include <string>

#include "../../include/fa.h"

namespace {

using at::Tensor;
constexpr auto kBf16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kI32 = at::kInt;

const char* type_name(at::ScalarType t)
{
    switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kHalf: return "torch.float16";
    case at::kDouble: return "torch.float64";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kByte: return "torch.uint8";
    case at::kBool: return "torch.bool";
    default: return c10::toString(t);
    }
}

// With the Python error set; the entry points hand it on.
[[noreturn]] void refuse(const std::string& why, PyObject* kind = PyExc_ValueError)
{
    PyErr_SetString(kind, why.c_str());
    throw python_error();
}

std::string shape_text(at::IntArrayRef s)
{
    std::string t = "[";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + "]";
}

// A tensor argument; `device` < 0: the call's first, on any CUDA device.
const Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a torch.Tensor", PyExc_TypeError);
    return THPVariable_Unpack(o);
}

void check(const Tensor& t, const char* name, at::ScalarType type, int device)
{
    if (t.scalar_type() != type) refuse(std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
    if (!t.is_cuda()) refuse(std::string(name) + " must be on a CUDA device");
    if (device >= 0 && t.get_device() != device)
        refuse(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", expected cuda:" + std::to_string(device));
}

void check_shape(const Tensor& t, const char* name, at::IntArrayRef shape)
{
    if (t.sizes() != shape) refuse(std::string(name) + " must be " + shape_text(shape) + ", got " + shape_text(t.sizes()));
}

// Data pointer of a contiguous tensor of this type and shape on this device.
void* arg(PyObject* o, const char* name, at::ScalarType type, int device, at::IntArrayRef shape)
{
    const Tensor& t = tensor(o, name);
    check(t, name, type, device);
    check_shape(t, name, shape);
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    return t.data_ptr();
}

void* optional_arg(PyObject* o, const char* name, at::ScalarType type, int device, at::IntArrayRef shape)
{
    return o == Py_None ? nullptr : arg(o, name, type, device, shape);
}

// Data pointer and token stride of [B, N, heads, head_dim] with its heads contiguous and its tokens
// evenly spaced: a whole tensor, or a slice of the heads of one.
struct Rows {
    void* ptr = nullptr;
    long long stride = 0;
};

Rows rows(PyObject* o, const char* name, at::ScalarType type, int device, at::IntArrayRef shape)
{
    const Tensor& t = tensor(o, name);
    check(t, name, type, device);
    check_shape(t, name, shape);
    const int64_t B = shape[0], N = shape[1], H = shape[2], d = shape[3];
    const at::IntArrayRef s = t.strides();
    const int64_t tok = N > 1 ? s[1] : B > 1 ? s[0] : H * d;
    if ((d > 1 && s[3] != 1) || (H > 1 && s[2] != d) || (B > 1 && s[0] != N * tok))
        refuse(std::string(name) + " must have its heads contiguous and its tokens evenly spaced");
    return Rows{t.data_ptr(), tok};
}

const Tensor& first(PyObject* o, const char* name, int64_t dims, const char* layout)
{
    const Tensor& t = tensor(o, name);
    check(t, name, kBf16, -1);
    if (t.dim() != dims) refuse(std::string(name) + " must be " + layout);
    return t;
}

int as_int(int64_t x)
{
    // the C ABI takes sizes as int; a larger one is refused there like any other bad size
    return x > 0x7fffffff ? -1 : static_cast<int>(x);
}

double number(PyObject* o)
{
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return x;
}

int flag(PyObject* o)
{
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw python_error();
    return x;
}

fa_dtype out_type(at::ScalarType t)
{
    if (t == kBf16) return FA_BF16;
    if (t == kF32) return FA_F32;
    refuse(std::string("output dtype must be bfloat16 or float32, not ") + type_name(t));
}

// The given output, or a new one (allocated directly: through the dispatcher it takes twice the time).
Tensor output(PyObject* o, const Tensor& like, at::ScalarType type, at::IntArrayRef shape)
{
    return o == Py_None ? Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt)) : Tensor();
}

// Owns nothing: the Python object to return for an output that was given or made here.
PyObject* result(PyObject* given, const Tensor& made)
{
    if (!made.defined()) {
        Py_INCREF(given);
        return given;
    }
    return THPVariable_Wrap(made);
}

PyObject* tuple(std::initializer_list<PyObject*> items)
{
    PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
    Py_ssize_t i = 0;
    bool ok = t != nullptr;
    for (PyObject* x : items) ok = ok && x != nullptr;
    for (PyObject* x : items) {
        if (ok) PyTuple_SET_ITEM(t, i++, x);
        else Py_XDECREF(x);
    }
    if (!ok) {
        Py_XDECREF(t);
        throw python_error();
    }
    return t;
}

void* pointer_of(PyObject* given, const Tensor& made, const char* name, at::ScalarType type, int device, at::IntArrayRef shape)
{
    return made.defined() ? made.data_ptr() : arg(given, name, type, device, shape);
}

void* stream(int device) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }

// A status other than FA_OK, with what to do about it left to the caller: returned as (status,).
PyObject* status_only(fa_status s) { return PyLong_FromLong(s); }

void expect(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want) refuse(std::to_string(n) + " arguments, " + std::to_string(want) + " expected", PyExc_TypeError);
}

// What the norm's forms share.
struct Rope {
    int device;
    int64_t B, N, Hq, Hkv, d;
    Rows q, k;
    void *wq, *wk, *cos, *sin;
    int64_t rot, max_pos;
    fa_dtype w_dtype;
    const Tensor* like;
    Rope(PyObject* q_, PyObject* k_, PyObject* wq_, PyObject* wk_, PyObject* cos_, PyObject* sin_)
    {
        const char* layout = "[B, N, heads, head_dim]";
        const Tensor& t = first(q_, "q", 4, layout);
        like = &t;
        device = static_cast<int>(t.get_device());
        B = t.size(0), N = t.size(1), Hq = t.size(2), d = t.size(3);
        const Tensor& u = tensor(k_, "k");
        if (u.dim() != 4) refuse(std::string("k must be ") + layout);
        Hkv = u.size(2);
        q = rows(q_, "q", kBf16, device, {B, N, Hq, d});
        k = rows(k_, "k", kBf16, device, {B, N, Hkv, d});
        const at::ScalarType wt = tensor(wq_, "q_weight").scalar_type();
        if (wt != kBf16 && wt != kF32) refuse("weights must be bfloat16 or float32");
        wq = arg(wq_, "q_weight", wt, device, {d});
        wk = arg(wk_, "k_weight", wt, device, {d});
        w_dtype = out_type(wt);
        const Tensor& c = tensor(cos_, "cos");
        if (c.dim() != 2) refuse("cos and sin must be [max_pos, rot / 2]");
        max_pos = c.size(0), rot = 2 * c.size(1);
        cos = arg(cos_, "cos", kF32, device, c.sizes());
        sin = arg(sin_, "sin", kF32, device, c.sizes());
    }
};

PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    // q k v q_weight k_weight cos sin positions eps interleaved expand q_out k_out v_out
    expect(n, 14);
    const Rope r(a[0], a[1], a[3], a[4], a[5], a[6]);
    const int expand = flag(a[10]);
    const std::array<int64_t, 4> qs{r.B, r.Hq, r.N, r.d}, kvs{r.B, expand ? r.Hq : r.Hkv, r.N, r.d};
    Rows v;
    Tensor vo;
    void* vp = nullptr;
    if (a[2] != Py_None) {
        v = rows(a[2], "v", kBf16, r.device, {r.B, r.N, r.Hkv, r.d});
        vo = output(a[13], *r.like, kBf16, kvs);
        vp = pointer_of(a[13], vo, "v_out", kBf16, r.device, kvs);
    } else if (a[13] != Py_None) {
        refuse("v_out without v");
    }
    void* pos = optional_arg(a[7], "positions", kI32, r.device, {r.B, r.N});
    const Tensor qo = output(a[11], *r.like, kBf16, qs), ko = output(a[12], *r.like, kBf16, kvs);
    void* qp = pointer_of(a[11], qo, "q_out", kBf16, r.device, qs);
    void* kp = pointer_of(a[12], ko, "k_out", kBf16, r.device, kvs);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(r.device));
    const fa_status s = fa_qk_norm_rope(
        r.q.ptr, r.k.ptr, v.ptr, r.wq, r.wk, static_cast<const float*>(r.cos), static_cast<const float*>(r.sin),
        static_cast<const int*>(pos), qp, kp, vp, r.q.stride, r.k.stride, v.stride, as_int(r.B), as_int(r.N), as_int(r.Hq),
        as_int(r.Hkv), as_int(r.d), as_int(r.rot), as_int(r.max_pos), flag(a[9]), expand, static_cast<float>(number(a[8])),
        r.w_dtype, stream(r.device));
    if (s != FA_OK) return status_only(s);
    return tuple({result(a[11], qo), result(a[12], ko), result(a[13], vo)});
    END_HANDLE_TH_ERRORS
}

PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    // dq dk dv q k q_weight k_weight cos sin positions eps interleaved expand out_f32 grad_q grad_k grad_v workspace
    expect(n, 18);
    const Rope r(a[3], a[4], a[5], a[6], a[7], a[8]);
    const int expand = flag(a[12]);
    const at::ScalarType ot = flag(a[13]) ? kF32 : kBf16;
    const std::array<int64_t, 4> dqs{r.B, r.Hq, r.N, r.d}, dkvs{r.B, expand ? r.Hq : r.Hkv, r.N, r.d};
    const std::array<int64_t, 4> qs{r.B, r.N, r.Hq, r.d}, kvs{r.B, r.N, r.Hkv, r.d};
    void* pos = optional_arg(a[9], "positions", kI32, r.device, {r.B, r.N});
    const at::ScalarType gt = tensor(a[0], "dq").scalar_type();
    const fa_dtype gd = out_type(gt);
    void* dq = arg(a[0], "dq", gt, r.device, dqs);
    void* dk = arg(a[1], "dk", gt, r.device, dkvs);
    void* dv = optional_arg(a[2], "dv", gt, r.device, dkvs);
    const bool values = dv != nullptr;
    const bool given = a[14] != Py_None;  // all of the gradients' buffers, or none
    if ((a[15] != Py_None) != given) refuse("grad_q goes with grad_k");
    if (a[16] != Py_None ? !given || !values : given && values) refuse("grad_v goes with dv and the other gradients");
    Tensor gq, gk, gv;
    Rows rq, rk, rv;
    if (given) {
        rq = rows(a[14], "grad_q", ot, r.device, qs);
        rk = rows(a[15], "grad_k", ot, r.device, kvs);
        if (values) rv = rows(a[16], "grad_v", ot, r.device, kvs);
    } else {
        gq = output(Py_None, *r.like, ot, qs);
        gk = output(Py_None, *r.like, ot, kvs);
        rq = Rows{gq.data_ptr(), r.Hq * r.d};
        rk = Rows{gk.data_ptr(), r.Hkv * r.d};
        if (values) {
            gv = output(Py_None, *r.like, ot, kvs);
            rv = Rows{gv.data_ptr(), r.Hkv * r.d};
        }
    }
    const Tensor wq = output(Py_None, *r.like, kF32, {r.d}), wk = output(Py_None, *r.like, kF32, {r.d});
    Tensor made;
    void* ws;
    int64_t ws_bytes;
    if (a[17] == Py_None) {
        ws_bytes = static_cast<int64_t>(fa_qk_norm_rope_bwd_workspace_size(as_int(r.d)));
        made = output(Py_None, *r.like, at::kByte, {ws_bytes});
        ws = made.data_ptr();
    } else {
        const Tensor& w = tensor(a[17], "workspace");
        ws = arg(a[17], "workspace", at::kByte, r.device, w.sizes());
        ws_bytes = w.numel();
    }
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(r.device));
    const fa_status s = fa_qk_norm_rope_bwd(
        dq, dk, dv, r.q.ptr, r.k.ptr, r.wq, r.wk, static_cast<const float*>(r.cos), static_cast<const float*>(r.sin),
        static_cast<const int*>(pos), rq.ptr, rk.ptr, rv.ptr, wq.data_ptr<float>(), wk.data_ptr<float>(), ws,
        static_cast<size_t>(ws_bytes), r.q.stride, r.k.stride, rq.stride, rk.stride, rv.stride, as_int(r.B), as_int(r.N),
        as_int(r.Hq), as_int(r.Hkv), as_int(r.d), as_int(r.rot), as_int(r.max_pos), flag(a[11]), expand,
        static_cast<float>(number(a[10])), r.w_dtype, gd, out_type(ot), stream(r.device));
    if (s != FA_OK) return status_only(s);
    return tuple({result(a[14], gq), result(a[15], gk), values ? result(a[16], gv) : result(Py_None, Tensor()),
                  THPVariable_Wrap(wq), THPVariable_Wrap(wk)});
    END_HANDLE_TH_ERRORS
}

PyObject* qk_norm_rope_append(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    // q k v q_weight k_weight cos sin k_cache v_cache seqlens parents n_nodes eps interleaved q_out
    expect(n, 15);
    const Rope r(a[0], a[1], a[3], a[4], a[5], a[6]);
    const Rows v = rows(a[2], "v", kBf16, r.device, {r.B, r.N, r.Hkv, r.d});
    const Tensor& c = tensor(a[7], "k_cache");
    if (c.dim() != 4) refuse("k_cache must be [B, Hkv, Nk_max, head_dim]");
    const std::array<int64_t, 4> cs{r.B, r.Hkv, c.size(2), r.d}, qs{r.B, r.Hq, r.N, r.d};
    void* kc = arg(a[7], "k_cache", kBf16, r.device, cs);
    void* vc = arg(a[8], "v_cache", kBf16, r.device, cs);
    void* lens = arg(a[9], "seqlens", kI32, r.device, {r.B});
    void* parents = optional_arg(a[10], "parents", kI32, r.device, {r.B, r.N});
    void* nodes = optional_arg(a[11], "n_nodes", kI32, r.device, {r.B});
    const Tensor qo = output(a[14], *r.like, kBf16, qs);
    void* qp = pointer_of(a[14], qo, "q_out", kBf16, r.device, qs);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(r.device));
    const fa_status s = fa_qk_norm_rope_append(
        r.q.ptr, r.k.ptr, v.ptr, r.wq, r.wk, static_cast<const float*>(r.cos), static_cast<const float*>(r.sin),
        static_cast<const int*>(lens), static_cast<const int*>(parents), static_cast<const int*>(nodes), qp, kc, vc, r.q.stride,
        r.k.stride, v.stride, as_int(r.B), as_int(r.N), as_int(r.Hq), as_int(r.Hkv), as_int(cs[2]), as_int(r.d), as_int(r.rot),
        as_int(r.max_pos), flag(a[13]), static_cast<float>(number(a[12])), r.w_dtype, stream(r.device));
    if (s != FA_OK) return status_only(s);
    return tuple({result(a[14], qo)});
    END_HANDLE_TH_ERRORS
}

PyObject* decode_tree(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    // q k_cache v_cache seqlens parents n_nodes scale out_f32 out lse return_lse workspace num_sms
    expect(n, 13);
    const char* layout = "[B, heads, rows, head_dim]";
    const Tensor& q = first(a[0], "q", 4, layout);
    const Tensor& k = first(a[1], "k_cache", 4, layout);
    const int device = static_cast<int>(q.get_device());
    const int64_t B = q.size(0), Hq = q.size(1), T = q.size(2), d = q.size(3), Hkv = k.size(1), Nk = k.size(2);
    const std::array<int64_t, 4> qs{B, Hq, T, d}, cs{B, Hkv, Nk, d};
    void* qp = arg(a[0], "q", kBf16, device, qs);
    void* kp = arg(a[1], "k_cache", kBf16, device, cs);
    void* vp = arg(a[2], "v_cache", kBf16, device, cs);
    void* lens = arg(a[3], "seqlens", kI32, device, {B});
    void* parents = optional_arg(a[4], "parents", kI32, device, {B, T});
    void* nodes = optional_arg(a[5], "n_nodes", kI32, device, {B});
    const double scale = a[6] == Py_None ? 1.0 / std::sqrt(static_cast<double>(d)) : number(a[6]);
    const at::ScalarType ot = a[8] != Py_None ? tensor(a[8], "out").scalar_type() : flag(a[7]) ? kF32 : kBf16;
    const fa_dtype od = out_type(ot);
    const Tensor out = output(a[8], q, ot, qs);
    void* op = pointer_of(a[8], out, "out", ot, device, qs);
    Tensor lse;
    void* lp = nullptr;
    const bool want = a[9] != Py_None || flag(a[10]);
    if (want) {
        lse = output(a[9], q, kF32, {B, Hq, T});
        lp = pointer_of(a[9], lse, "lse", kF32, device, {B, Hq, T});
    }
    Tensor made;
    void* ws;
    int64_t ws_bytes;
    if (a[11] == Py_None) {
        const long sms = PyLong_AsLong(a[12]);
        if (sms == -1 && PyErr_Occurred()) throw python_error();
        ws_bytes = static_cast<int64_t>(
            fa_decode_tree_workspace_size(as_int(Hq), as_int(Hkv), as_int(T), as_int(d), static_cast<int>(sms)));
        made = output(Py_None, q, at::kByte, {ws_bytes > 256 ? ws_bytes : 256});
        ws = made.data_ptr();
    } else {
        const Tensor& w = tensor(a[11], "workspace");
        ws = arg(a[11], "workspace", at::kByte, device, w.sizes());
        ws_bytes = w.numel();
    }
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
    const fa_status s =
        fa_decode_tree(qp, kp, vp, static_cast<const int*>(lens), static_cast<const int*>(parents), static_cast<const int*>(nodes),
                       op, static_cast<float*>(lp), ws, static_cast<size_t>(ws_bytes), as_int(B), as_int(Hq), as_int(Hkv),
                       as_int(T), as_int(Nk), as_int(d), as_int(d), static_cast<float>(scale), od, stream(device));
    if (s != FA_OK) return status_only(s);
    return tuple({result(a[8], out), want ? result(a[9], lse) : result(Py_None, Tensor())});
    END_HANDLE_TH_ERRORS
}

// Workspace: the given one, or `bytes` made here.
struct Space {
    Tensor made;
    void* ptr = nullptr;
    size_t bytes = 0;
    Space(PyObject* o, const Tensor& like, int device, size_t need)
    {
        if (o == Py_None) {
            if (need == 0) return;
            made = output(Py_None, like, at::kByte, {static_cast<int64_t>(need)});
            ptr = made.data_ptr();
            bytes = need;
        } else {
            const Tensor& w = tensor(o, "workspace");
            ptr = arg(o, "workspace", at::kByte, device, w.sizes());
            bytes = static_cast<size_t>(w.numel());
        }
    }
};

int sm_count(PyObject* o)
{
    const long sms = PyLong_AsLong(o);
    if (sms == -1 && PyErr_Occurred()) throw python_error();
    return static_cast<int>(sms);
}

// What forward and backward under score rules share: q k v and causal scale softcap slopes documents prefix_lens.
struct Rules {
    int device;
    int64_t B, Hq, Hkv, N, Nk, d;
    std::array<int64_t, 4> qs, kvs;
    void *q, *k, *v;
    int causal;
    float scale, softcap;
    const float* slopes;
    const int *documents, *prefix_lens;
    const Tensor* like;
    Rules(PyObject* const* a, PyObject* const* r)
    {
        const char* layout = "[B, heads, rows, head_dim]";
        const Tensor& t = first(a[0], "q", 4, layout);
        const Tensor& u = first(a[1], "k", 4, layout);
        like = &t;
        device = static_cast<int>(t.get_device());
        B = t.size(0), Hq = t.size(1), N = t.size(2), d = t.size(3), Hkv = u.size(1), Nk = u.size(2);
        qs = {B, Hq, N, d};
        kvs = {B, Hkv, Nk, d};
        q = arg(a[0], "q", kBf16, device, qs);
        k = arg(a[1], "k", kBf16, device, kvs);
        v = arg(a[2], "v", kBf16, device, kvs);
        causal = flag(r[0]);
        scale = static_cast<float>(r[1] == Py_None ? 1.0 / std::sqrt(static_cast<double>(d)) : number(r[1]));
        softcap = static_cast<float>(number(r[2]));
        slopes = static_cast<const float*>(optional_arg(r[3], "slopes", kF32, device, {Hq}));
        documents = static_cast<const int*>(optional_arg(r[4], "documents", kI32, device, {B, Nk}));
        prefix_lens = static_cast<const int*>(optional_arg(r[5], "prefix_lens", kI32, device, {B}));
    }
};

PyObject* fwd_rules(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    // q k v causal scale softcap slopes documents prefix_lens out_f32 out lse return_lse workspace
    expect(n, 14);
    const Rules r(a, a + 3);
    const at::ScalarType ot = a[10] != Py_None ? tensor(a[10], "out").scalar_type() : flag(a[9]) ? kF32 : kBf16;
    const fa_dtype od = out_type(ot);
    const Tensor out = output(a[10], *r.like, ot, r.qs);
    void* op = pointer_of(a[10], out, "out", ot, r.device, r.qs);
    Tensor lse;
    void* lp = nullptr;
    const bool want = a[11] != Py_None || flag(a[12]);
    if (want) {
        lse = output(a[11], *r.like, kF32, {r.B, r.Hq, r.N});
        lp = pointer_of(a[11], lse, "lse", kF32, r.device, {r.B, r.Hq, r.N});
    }
    const Space ws(a[13], *r.like, r.device, r.documents != nullptr ? fa_fwd_rules_workspace_size(as_int(r.B), as_int(r.N)) : 0);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(r.device));
    const fa_status s = fa_fwd_rules(r.q, r.k, r.v, r.slopes, r.documents, r.prefix_lens, op, static_cast<float*>(lp), ws.ptr,
                                     ws.bytes, as_int(r.B), as_int(r.Hq), as_int(r.Hkv), as_int(r.N), as_int(r.Nk), as_int(r.d),
                                     as_int(r.d), r.causal, r.scale, r.softcap, od, stream(r.device));
    if (s != FA_OK) return status_only(s);
    return tuple({result(a[10], out), want ? result(a[11], lse) : result(Py_None, Tensor())});
    END_HANDLE_TH_ERRORS
}

PyObject* bwd_rules(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    // q k v o lse do causal scale softcap slopes documents prefix_lens out_f32 dq dk dv workspace num_sms
    expect(n, 18);
    const Rules r(a, a + 6);
    const at::ScalarType it = tensor(a[3], "o").scalar_type();
    const fa_dtype id = out_type(it);
    void* o = arg(a[3], "o", it, r.device, r.qs);
    void* lse = arg(a[4], "lse", kF32, r.device, {r.B, r.Hq, r.N});
    void* g = arg(a[5], "do", kBf16, r.device, r.qs);
    const bool given = a[13] != Py_None;  // all of the gradients' buffers, or none
    if ((a[14] != Py_None) != given || (a[15] != Py_None) != given) refuse("grads must hold dq, dk and dv");
    const at::ScalarType ot = given ? tensor(a[13], "dq").scalar_type() : flag(a[12]) ? kF32 : kBf16;
    const fa_dtype od = out_type(ot);
    const Tensor dq = output(a[13], *r.like, ot, r.qs), dk = output(a[14], *r.like, ot, r.kvs), dv = output(a[15], *r.like, ot, r.kvs);
    void* qp = pointer_of(a[13], dq, "dq", ot, r.device, r.qs);
    void* kp = pointer_of(a[14], dk, "dk", ot, r.device, r.kvs);
    void* vp = pointer_of(a[15], dv, "dv", ot, r.device, r.kvs);
    const size_t need = a[16] != Py_None ? 0
                                         : fa_bwd_rules_workspace_size(as_int(r.B), as_int(r.Hq), as_int(r.Hkv), as_int(r.N),
                                                                       as_int(r.Nk), as_int(r.d), sm_count(a[17]));
    const Space ws(a[16], *r.like, r.device, need > 256 ? need : 256);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(r.device));
    const fa_status s = fa_bwd_rules(r.q, r.k, r.v, o, static_cast<const float*>(lse), g, r.slopes, r.documents, r.prefix_lens, qp,
                                     kp, vp, ws.ptr, ws.bytes, as_int(r.B), as_int(r.Hq), as_int(r.Hkv), as_int(r.N),
                                     as_int(r.Nk), as_int(r.d), as_int(r.d), r.causal, r.scale, r.softcap, id, od,
                                     stream(r.device));
    if (s != FA_OK) return status_only(s);
    return tuple({result(a[13], dq), result(a[14], dk), result(a[15], dv)});
    END_HANDLE_TH_ERRORS
}

PyObject* decode_prefix(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    // q k_prefix v_prefix k_cache v_cache seqlens prefix_len scale softcap slopes out_f32 out lse return_lse workspace num_sms
    expect(n, 16);
    const Tensor& q = first(a[0], "q", 4, "[B, heads, 1, head_dim]");
    const Tensor& k = first(a[3], "k_cache", 4, "[B, Hkv, Nk_max, head_dim]");
    const int device = static_cast<int>(q.get_device());
    const int64_t B = q.size(0), Hq = q.size(1), d = q.size(3), Hkv = k.size(1), Nk = k.size(2);
    const std::array<int64_t, 4> qs{B, Hq, 1, d}, cs{B, Hkv, Nk, d};
    void* qp = arg(a[0], "q", kBf16, device, qs);
    void* kp = arg(a[3], "k_cache", kBf16, device, cs);
    void* vp = arg(a[4], "v_cache", kBf16, device, cs);
    void* lens = arg(a[5], "seqlens", kI32, device, {B});
    int64_t P = 0;
    void *kpre = nullptr, *vpre = nullptr, *plen = nullptr;
    if (a[1] != Py_None) {
        P = first(a[1], "k_prefix", 3, "[Hkv, prefix, head_dim]").size(1);
        const std::array<int64_t, 3> ps{Hkv, P, d};
        kpre = arg(a[1], "k_prefix", kBf16, device, ps);
        vpre = arg(a[2], "v_prefix", kBf16, device, ps);
        plen = optional_arg(a[6], "prefix_len", kI32, device, {1});
    } else if (a[2] != Py_None || a[6] != Py_None) {
        refuse("v_prefix and prefix_len go with k_prefix");
    }
    const double scale = a[7] == Py_None ? 1.0 / std::sqrt(static_cast<double>(d)) : number(a[7]);
    void* slopes = optional_arg(a[9], "slopes", kF32, device, {Hq});
    const at::ScalarType ot = a[11] != Py_None ? tensor(a[11], "out").scalar_type() : flag(a[10]) ? kF32 : kBf16;
    const fa_dtype od = out_type(ot);
    const Tensor out = output(a[11], q, ot, qs);
    void* op = pointer_of(a[11], out, "out", ot, device, qs);
    Tensor lse;
    void* lp = nullptr;
    const bool want = a[12] != Py_None || flag(a[13]);
    if (want) {
        lse = output(a[12], q, kF32, {B, Hq, 1});
        lp = pointer_of(a[12], lse, "lse", kF32, device, {B, Hq, 1});
    }
    const size_t need = a[14] != Py_None ? 0
                                         : fa_decode_prefix_workspace_size(as_int(B), as_int(Hq), as_int(Hkv), as_int(d), sm_count(a[15]));
    const Space ws(a[14], q, device, need > 256 ? need : 256);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
    const fa_status s = fa_decode_prefix(qp, kpre, vpre, static_cast<const int*>(plen), kp, vp, static_cast<const int*>(lens),
                                         static_cast<const float*>(slopes), op, static_cast<float*>(lp), ws.ptr, ws.bytes, as_int(B),
                                         as_int(Hq), as_int(Hkv), as_int(P), as_int(Nk), as_int(d), as_int(d),
                                         static_cast<float>(scale), static_cast<float>(number(a[8])), od, stream(device));
    if (s != FA_OK) return status_only(s);
    return tuple({result(a[11], out), want ? result(a[12], lse) : result(Py_None, Tensor())});
    END_HANDLE_TH_ERRORS
}

PyObject* cache_compact(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    // k_cache v_cache seqlens accepted n_accepted seqlens_out
    expect(n, 6);
    const Tensor& k = tensor(a[0], "k_cache");
    if (k.dim() != 4 && k.dim() != 5) refuse("caches must be [B, Hkv, Nk_max, head_dim], with or without layers before");
    check(k, "k_cache", kBf16, -1);
    const int device = static_cast<int>(k.get_device());
    const at::IntArrayRef cs = k.sizes();
    const int64_t o = k.dim() - 4, L = o ? cs[0] : 1, B = cs[o], Hkv = cs[o + 1], Nk = cs[o + 2], d = cs[o + 3];
    const Tensor& acc = tensor(a[3], "accepted");
    if (acc.dim() != 2) refuse("accepted must be [B, T]");
    const int64_t T = acc.size(1);
    void* kp = arg(a[0], "k_cache", kBf16, device, cs);
    void* vp = arg(a[1], "v_cache", kBf16, device, cs);
    void* lens = arg(a[2], "seqlens", kI32, device, {B});
    void* ap = arg(a[3], "accepted", kI32, device, {B, T});
    void* np = arg(a[4], "n_accepted", kI32, device, {B});
    const Tensor out = output(a[5], k, kI32, {B});
    void* op = pointer_of(a[5], out, "seqlens_out", kI32, device, {B});
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
    const fa_status s = fa_cache_compact(kp, vp, static_cast<const int*>(lens), static_cast<const int*>(ap),
                                         static_cast<const int*>(np), static_cast<int*>(op), as_int(L), as_int(B), as_int(Hkv),
                                         as_int(Nk), as_int(d), as_int(d), as_int(T), stream(device));
    if (s != FA_OK) return status_only(s);
    return tuple({result(a[5], out)});
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<qk_norm_rope>("qk_norm_rope"),
    method<qk_norm_rope_bwd>("qk_norm_rope_bwd"),
    method<qk_norm_rope_append>("qk_norm_rope_append"),
    method<decode_tree>("decode_tree"),
    method<cache_compact>("cache_compact"),
    method<fwd_rules>("fwd_rules"),
    method<bwd_rules>("bwd_rules"),
    method<decode_prefix>("decode_prefix"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fa_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_binding() { return PyModule_Create(&module); }
