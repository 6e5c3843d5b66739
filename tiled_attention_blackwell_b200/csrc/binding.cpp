// Native side of the Python calls that a step makes once per layer (head norms
// with rotation, the cache write, the decode, attention with first tokens that
// stay visible): checks of the tensors, allocation of outputs, and the call
// into the library.  In Python these cost two to four times as long as the
// launches themselves.
//
// Everything here is argument marshalling; the work is libattn.so's, whose
// functions attn.py hands over by address.  A wrong argument raises TypeError,
// an error of the library AttnError (through the function that attn.py hands
// over), torch's own errors what torch raises.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/attn.h"

namespace {

// Set once by bind().
decltype(&attn_qk_norm_rope) g_norm_rope;
decltype(&attn_qk_norm_rope_cache) g_norm_rope_cache;
decltype(&attn_qk_norm_rope_bwd) g_norm_rope_bwd;
decltype(&attn_qk_norm_rope_bwd_workspace_size) g_norm_rope_bwd_workspace;
decltype(&attn_decode_paged) g_decode;
decltype(&attn_decode_paged_workspace_size) g_decode_workspace;
decltype(&attn_fwd_sinks) g_fwd_sinks;
decltype(&attn_fwd_sinks_workspace_size) g_fwd_sinks_workspace;
decltype(&attn_bwd_sinks) g_bwd_sinks;
decltype(&attn_bwd_sinks_workspace_size) g_bwd_sinks_workspace;
PyObject *g_check = nullptr;  // (status, name): raises unless the status is ATTN_OK

constexpr auto kBF16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kF8 = at::kFloat8_e4m3fn;

// Thrown with a Python error set.
struct PythonError {};

template <class... Args>
[[noreturn]] void type_error(const char *fmt, Args... args) {
    PyErr_Format(PyExc_TypeError, fmt, args...);
    throw PythonError{};
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) type_error("%s must be a tensor", name);
    return THPVariable_Unpack(o);
}

void require(bool ok, const char *name, const char *what) {
    if (!ok) type_error("%s must be %s", name, what);
}

// All tensors of a call on one CUDA device.
class Device {
   public:
    void add(const at::Tensor &t, const char *name) {
        if (!t.is_cuda()) type_error("%s must be a CUDA tensor", name);
        if (index_ < 0) index_ = t.get_device();
        else if (t.get_device() != index_) type_error("%s is on another device", name);
    }
    int index() const { return index_; }

   private:
    int index_ = -1;
};

float number(PyObject *o) {
    const double d = PyFloat_AsDouble(o);
    if (d == -1.0 && PyErr_Occurred()) throw PythonError{};
    return (float)d;
}
int integer(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    if (v < INT_MIN || v > INT_MAX) type_error("integer argument out of range");
    return (int)v;
}

// A number of first keys: more than `most` are `most` (more than there are keys are
// all of them), a negative one is the library's to refuse.
int first_keys(PyObject *o, int most) {
    int overflow = 0;
    const long long n = PyLong_AsLongLongAndOverflow(o, &overflow);
    if (n == -1 && PyErr_Occurred()) throw PythonError{};
    return overflow > 0 || n > most ? most : overflow < 0 || n < 0 ? -1 : (int)n;
}

// Calls run on the device's current stream, whose pool the outputs come from.
void *current_stream(int device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }

void check(int status, const char *name) {
    if (status == ATTN_OK) return;
    PyObject *r = PyObject_CallFunction(g_check, "is", status, name);
    Py_XDECREF(r);
    throw PythonError{};
}

// Distance, in values, of consecutive tokens of a [..., H, D] tensor whose
// heads are contiguous and whose tokens are evenly spaced.
long long token_stride(const at::Tensor &t, const char *name) {
    const int n = (int)t.dim();
    const long long H = t.size(n - 2), D = t.size(n - 1);
    if (t.is_contiguous()) return H * D;
    if (t.stride(n - 1) != 1 || (H > 1 && t.stride(n - 2) != D))
        type_error("%s: the heads of a token must be contiguous", name);
    long long step = -1, upto = 0;
    for (int i = n - 3; i >= 0; --i) {
        if (t.size(i) == 1) continue;
        if (step < 0) step = upto = t.stride(i);
        else if (t.stride(i) != upto) type_error("%s: the tokens must be evenly spaced", name);
        upto *= t.size(i);
    }
    return step < 0 ? H * D : step;
}

// A given output, or one like `like`.
at::Tensor output(PyObject *o, const at::Tensor &like, const char *name) {
    if (o == Py_None) return at::empty_like(like);
    const at::Tensor &t = tensor(o, name);
    require(t.sizes() == like.sizes(), name, "of its input's shape");
    require(t.scalar_type() == kBF16, name, "a bf16 tensor");
    return t;
}

// q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved: what every
// form of the norm and rotation has, checked but for the device.
struct Norm {
    const at::Tensor &q, &k, &qw, &kw, &cos, &sin, &pos;
    float eps;
    int interleaved;
    long long tokens;
    int Hq, Hkv, D;

    explicit Norm(PyObject *const *a)
        : q(tensor(a[0], "q")), k(tensor(a[1], "k")), qw(tensor(a[2], "q_weight")),
          kw(tensor(a[3], "k_weight")), cos(tensor(a[4], "cos")), sin(tensor(a[5], "sin")),
          pos(tensor(a[6], "positions")), eps(number(a[7])), interleaved(PyObject_IsTrue(a[8])) {
        if (interleaved < 0) throw PythonError{};
        const int n = (int)q.dim();
        require(q.scalar_type() == kBF16 && n >= 3, "q", "a bf16 tensor [..., Hq, D]");
        require(k.scalar_type() == kBF16 && k.dim() == n && k.size(n - 1) == q.size(n - 1) &&
                    k.sizes().slice(0, n - 2) == q.sizes().slice(0, n - 2),
                "k", "a bf16 tensor [..., Hkv, D] of q's tokens");
        require(q.size(n - 2) <= INT_MAX && k.size(n - 2) <= INT_MAX && q.size(n - 1) <= INT_MAX, "q", "smaller");
        Hq = (int)q.size(n - 2), Hkv = (int)k.size(n - 2), D = (int)q.size(n - 1);
        const auto dtype = qw.scalar_type();
        require((dtype == kBF16 || dtype == kF32) && qw.dim() == 1 && qw.size(0) == D && qw.is_contiguous(),
                "q_weight", "a contiguous bf16 or fp32 tensor [D]");
        require(kw.scalar_type() == dtype && kw.dim() == 1 && kw.size(0) == D && kw.is_contiguous(),
                "k_weight", "a contiguous tensor [D] of q_weight's type");
        require(cos.scalar_type() == kF32 && cos.dim() == 2 && cos.is_contiguous() && cos.size(0) <= INT_MAX &&
                    cos.size(1) <= INT_MAX / 2,
                "cos", "a contiguous fp32 tensor [max_positions, rot / 2]");
        require(sin.scalar_type() == kF32 && sin.sizes() == cos.sizes() && sin.is_contiguous(), "sin",
                "a contiguous fp32 tensor of cos' shape");
        require(pos.scalar_type() == at::kInt && pos.sizes() == q.sizes().slice(0, n - 2) && pos.is_contiguous(),
                "positions", "a contiguous int32 tensor with an entry per token");
        tokens = pos.numel();
    }
    void on(Device &dev) const {
        dev.add(q, "q");
        dev.add(k, "k");
        dev.add(qw, "q_weight");
        dev.add(kw, "k_weight");
        dev.add(cos, "cos");
        dev.add(sin, "sin");
        dev.add(pos, "positions");
    }
    int w_fp32() const { return qw.scalar_type() == kF32; }
    const float *cos_ptr() const { return static_cast<const float *>(cos.data_ptr()); }
    const float *sin_ptr() const { return static_cast<const float *>(sin.data_ptr()); }
    const int *pos_ptr() const { return static_cast<const int *>(pos.data_ptr()); }
    int rot() const { return 2 * (int)cos.size(1); }
    int max_positions() const { return (int)cos.size(0); }
};

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }

// (q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, q_out, k_out)
PyObject *norm_rope(PyObject *const *a) {
    const Norm n(a);
    Device dev;
    n.on(dev);
    c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev.index());
    const at::Tensor q_out = output(a[9], n.q, "q_out"), k_out = output(a[10], n.k, "k_out");
    dev.add(q_out, "q_out");
    dev.add(k_out, "k_out");
    check(g_norm_rope(n.q.data_ptr(), n.k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(),
                      token_stride(n.q, "q"), token_stride(n.k, "k"), token_stride(q_out, "q_out"),
                      token_stride(k_out, "k_out"), n.qw.data_ptr(), n.kw.data_ptr(), n.w_fp32(),
                      n.cos_ptr(), n.sin_ptr(), n.pos_ptr(), n.tokens, n.Hq, n.Hkv, n.D, n.rot(),
                      n.max_positions(), n.eps, n.interleaved, current_stream(dev.index())),
          "attn_qk_norm_rope");
    return Py_BuildValue("(NN)", wrap(q_out), wrap(k_out));
}

// Both caches [num_pages, page_size, Hkv, D]; returns ATTN_KV_*.
int cache_type(const at::Tensor &k, const at::Tensor &v) {
    const auto dtype = k.scalar_type();
    require((dtype == kBF16 || dtype == kF8) && k.dim() == 4 && k.is_contiguous(), "k_cache",
            "a contiguous bf16 or float8_e4m3fn tensor [num_pages, page_size, Hkv, D]");
    require(v.scalar_type() == dtype && v.sizes() == k.sizes() && v.is_contiguous(), "v_cache",
            "a contiguous tensor of k_cache's type and shape");
    for (int i = 0; i < 4; ++i) require(k.size(i) <= INT_MAX, "k_cache", "smaller");
    return dtype == kBF16 ? ATTN_KV_BF16 : ATTN_KV_E4M3;
}

// (q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, v, slots, k_cache, v_cache,
//  k_descale, v_descale, q_out)
PyObject *norm_rope_cache(PyObject *const *a) {
    const Norm n(a);
    const at::Tensor &v = tensor(a[9], "v"), &slots = tensor(a[10], "slots");
    const at::Tensor &kc = tensor(a[11], "k_cache"), &vc = tensor(a[12], "v_cache");
    require(v.scalar_type() == kBF16 && v.sizes() == n.k.sizes(), "v", "a bf16 tensor of k's shape");
    require(slots.scalar_type() == at::kInt && slots.sizes() == n.pos.sizes() && slots.is_contiguous(), "slots",
            "a contiguous int32 tensor with an entry per token");
    const int kv = cache_type(kc, vc);
    require(kc.size(2) == n.Hkv && kc.size(3) == n.D, "k_cache", "of k's heads");
    const float kd = number(a[13]), vd = number(a[14]);
    Device dev;
    n.on(dev);
    dev.add(v, "v");
    dev.add(slots, "slots");
    dev.add(kc, "k_cache");
    dev.add(vc, "v_cache");
    c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev.index());
    const at::Tensor q_out = output(a[15], n.q, "q_out");
    dev.add(q_out, "q_out");
    check(g_norm_rope_cache(n.q.data_ptr(), n.k.data_ptr(), v.data_ptr(), q_out.data_ptr(),
                            token_stride(n.q, "q"), token_stride(n.k, "k"), token_stride(v, "v"),
                            token_stride(q_out, "q_out"), n.qw.data_ptr(), n.kw.data_ptr(), n.w_fp32(),
                            n.cos_ptr(), n.sin_ptr(), n.pos_ptr(), static_cast<const int *>(slots.data_ptr()),
                            kc.data_ptr(), vc.data_ptr(), kv, kd, vd, kc.size(0) * kc.size(1), n.tokens, n.Hq,
                            n.Hkv, n.D, n.rot(), n.max_positions(), n.eps, n.interleaved,
                            current_stream(dev.index())),
          "attn_qk_norm_rope_cache");
    return wrap(q_out);
}

at::Tensor workspace(size_t bytes, const at::Tensor &like) {
    return at::empty({(int64_t)bytes}, like.options().dtype(at::kByte));
}

// (q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, dq, dk, dq_in, dk_in)
PyObject *norm_rope_backward(PyObject *const *a) {
    const Norm n(a);
    const at::Tensor &dq = tensor(a[9], "dq"), &dk = tensor(a[10], "dk");
    for (auto [t, x, name] : {std::make_tuple(&dq, &n.q, "dq"), std::make_tuple(&dk, &n.k, "dk")})
        require((t->scalar_type() == kBF16 || t->scalar_type() == kF32) && t->sizes() == x->sizes(), name,
                "a bf16 or fp32 tensor of its output's shape");
    Device dev;
    n.on(dev);
    dev.add(dq, "dq");
    dev.add(dk, "dk");
    c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev.index());
    const at::Tensor dq_in = output(a[11], n.q, "dq_in"), dk_in = output(a[12], n.k, "dk_in");
    dev.add(dq_in, "dq_in");
    dev.add(dk_in, "dk_in");
    const at::Tensor dqw = at::empty_like(n.qw, n.qw.options().dtype(kF32));
    const at::Tensor dkw = at::empty_like(n.kw, n.kw.options().dtype(kF32));
    const at::Tensor ws = workspace(g_norm_rope_bwd_workspace(n.D), n.q);
    check(g_norm_rope_bwd(dq.data_ptr(), dk.data_ptr(), dq.scalar_type() == kF32, dk.scalar_type() == kF32,
                          n.q.data_ptr(), n.k.data_ptr(), dq_in.data_ptr(), dk_in.data_ptr(),
                          static_cast<float *>(dqw.data_ptr()), static_cast<float *>(dkw.data_ptr()),
                          token_stride(dq, "dq"), token_stride(dk, "dk"), token_stride(n.q, "q"),
                          token_stride(n.k, "k"), token_stride(dq_in, "dq_in"), token_stride(dk_in, "dk_in"),
                          n.qw.data_ptr(), n.kw.data_ptr(), n.w_fp32(), n.cos_ptr(), n.sin_ptr(), n.pos_ptr(),
                          n.tokens, n.Hq, n.Hkv, n.D, n.rot(), n.max_positions(), n.eps, n.interleaved,
                          ws.data_ptr(), (size_t)ws.numel(), current_stream(dev.index())),
          "attn_qk_norm_rope_bwd");
    return Py_BuildValue("(NNNN)", wrap(dq_in), wrap(dk_in), wrap(dqw), wrap(dkw));
}

// (q, k_cache, v_cache, page_table, seq_lens, scale, window_left, sinks, softcap, alibi_slopes,
//  k_descale, v_descale, o, lse, workspace)
PyObject *decode(PyObject *const *a) {
    const at::Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache");
    const at::Tensor &table = tensor(a[3], "page_table"), &lens = tensor(a[4], "seq_lens");
    require(q.scalar_type() == kBF16 && q.dim() == 3 && q.is_contiguous() && q.size(0) <= INT_MAX &&
                q.size(1) <= INT_MAX && q.size(2) <= INT_MAX,
            "q", "a contiguous bf16 tensor [B, Hq, D]");
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2);
    const int kv = cache_type(kc, vc);
    require(kc.size(3) == D, "k_cache", "of q's head dimension");
    require(table.scalar_type() == at::kInt && table.dim() == 2 && table.size(0) == B && table.is_contiguous() &&
                table.size(1) <= INT_MAX,
            "page_table", "a contiguous int32 tensor [B, max_pages]");
    require(lens.scalar_type() == at::kInt && lens.dim() == 1 && lens.size(0) == B && lens.is_contiguous(),
            "seq_lens", "a contiguous int32 tensor [B]");
    Device dev;
    dev.add(q, "q");
    dev.add(kc, "k_cache");
    dev.add(vc, "v_cache");
    dev.add(table, "page_table");
    dev.add(lens, "seq_lens");
    const float *slopes = nullptr;
    if (a[9] != Py_None) {
        const at::Tensor &t = tensor(a[9], "alibi_slopes");
        require(t.scalar_type() == kF32 && t.numel() == Hq && t.is_contiguous(), "alibi_slopes",
                "a contiguous fp32 tensor of Hq entries");
        dev.add(t, "alibi_slopes");
        slopes = static_cast<const float *>(t.data_ptr());
    }
    c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev.index());
    const at::Tensor o = output(a[12], q, "o");
    require(o.is_contiguous(), "o", "contiguous");
    const at::Tensor lse =
        a[13] == Py_None ? at::empty({B, Hq}, q.options().dtype(kF32)) : tensor(a[13], "lse");
    require(lse.scalar_type() == kF32 && lse.dim() == 2 && lse.size(0) == B && lse.size(1) == Hq &&
                lse.is_contiguous(),
            "lse", "a contiguous fp32 tensor [B, Hq]");
    const at::Tensor ws =
        a[14] == Py_None ? workspace(g_decode_workspace((int)D), q) : tensor(a[14], "workspace");
    require(ws.scalar_type() == at::kByte && ws.is_contiguous(), "workspace", "a contiguous uint8 tensor");
    dev.add(o, "o");
    dev.add(lse, "lse");
    dev.add(ws, "workspace");
    check(g_decode(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), kv, number(a[10]), number(a[11]),
                   static_cast<const int *>(table.data_ptr()), static_cast<const int *>(lens.data_ptr()),
                   o.data_ptr(), static_cast<float *>(lse.data_ptr()), (int)B, (int)Hq, (int)kc.size(2), (int)D,
                   (int)kc.size(0), (int)kc.size(1), (int)table.size(1), number(a[5]), integer(a[6]),
                   first_keys(a[7], INT_MAX), number(a[8]), slopes, ws.data_ptr(), (size_t)ws.numel(),
                   current_stream(dev.index())),
          "attn_decode_paged");
    return Py_BuildValue("(NN)", wrap(o), wrap(lse));
}

// q, k, v of an attention call [B, S, H, D] and its mask: q, k, v, scale,
// causal, window_left, window_right, sinks.
struct Masked {
    const at::Tensor &q, &k, &v;
    float scale;
    int causal, left, right, sinks;
    int B, Hq, Hkv, Sq, Sk, D;

    explicit Masked(PyObject *const *a)
        : q(tensor(a[0], "q")), k(tensor(a[1], "k")), v(tensor(a[2], "v")), scale(number(a[3])),
          causal(PyObject_IsTrue(a[4])), left(integer(a[5])), right(integer(a[6])) {
        if (causal < 0) throw PythonError{};
        require(q.scalar_type() == kBF16 && q.dim() == 4 && q.is_contiguous(), "q",
                "a contiguous bf16 tensor [B, Sq, Hq, D]");
        require(k.scalar_type() == kBF16 && k.dim() == 4 && k.is_contiguous() && k.size(0) == q.size(0) &&
                    k.size(3) == q.size(3),
                "k", "a contiguous bf16 tensor [B, Sk, Hkv, D] of q's batch and head dimension");
        require(v.scalar_type() == kBF16 && v.sizes() == k.sizes() && v.is_contiguous(), "v",
                "a contiguous bf16 tensor of k's shape");
        for (const at::Tensor *t : {&q, &k})
            for (int i = 0; i < 4; ++i) require(t->size(i) <= INT_MAX, "q or k", "smaller");
        B = (int)q.size(0), Sq = (int)q.size(1), Hq = (int)q.size(2), D = (int)q.size(3);
        Sk = (int)k.size(1), Hkv = (int)k.size(2);
        sinks = first_keys(a[7], Sk);
    }
    void on(Device &dev) const {
        dev.add(q, "q");
        dev.add(k, "k");
        dev.add(v, "v");
    }
};

// An option struct by address (None: the defaults).
template <class T>
const T *options(PyObject *o) {
    if (o == Py_None) return nullptr;
    const void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw PythonError{};
    return static_cast<const T *>(p);
}

// (q, k, v, scale, causal, window_left, window_right, sinks, options)
PyObject *fwd_sinks(PyObject *const *a) {
    const Masked m(a);
    Device dev;
    m.on(dev);
    c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev.index());
    const at::Tensor o = at::empty_like(m.q);
    const at::Tensor lse = at::empty({m.B, m.Hq, m.Sq}, m.q.options().dtype(kF32));
    const size_t size = g_fwd_sinks_workspace(m.B, m.Hq, m.Hkv, m.Sq, m.Sk, m.D, m.causal, m.left, m.right, m.sinks);
    at::Tensor ws;
    if (size) ws = workspace(size, m.q);
    check(g_fwd_sinks(m.q.data_ptr(), m.k.data_ptr(), m.v.data_ptr(), o.data_ptr(),
                      static_cast<float *>(lse.data_ptr()), m.B, m.Hq, m.Hkv, m.Sq, m.Sk, m.D, m.scale, m.causal,
                      m.left, m.right, m.sinks, size ? ws.data_ptr() : nullptr, size ? (size_t)ws.numel() : 0,
                      options<attn_fwd_options_t>(a[8]), current_stream(dev.index())),
          "attn_fwd_sinks");
    return Py_BuildValue("(NN)", wrap(o), wrap(lse));
}

// (q, k, v, scale, causal, window_left, window_right, sinks, o, lse, dout, options)
PyObject *bwd_sinks(PyObject *const *a) {
    const Masked m(a);
    const at::Tensor &o = tensor(a[8], "o"), &lse = tensor(a[9], "lse"), &dout = tensor(a[10], "dout");
    require(o.scalar_type() == kBF16 && o.sizes() == m.q.sizes() && o.is_contiguous(), "o",
            "a contiguous bf16 tensor of q's shape");
    require(dout.scalar_type() == kBF16 && dout.sizes() == m.q.sizes() && dout.is_contiguous(), "dout",
            "a contiguous bf16 tensor of q's shape");
    require(lse.scalar_type() == kF32 && lse.dim() == 3 && lse.size(0) == m.B && lse.size(1) == m.Hq &&
                lse.size(2) == m.Sq && lse.is_contiguous(),
            "lse", "a contiguous fp32 tensor [B, Hq, Sq]");
    Device dev;
    m.on(dev);
    dev.add(o, "o");
    dev.add(lse, "lse");
    dev.add(dout, "dout");
    c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev.index());
    const at::Tensor dq = at::empty_like(m.q, m.q.options().dtype(kF32));
    const at::Tensor dk = at::empty_like(m.k), dv = at::empty_like(m.v);
    const at::Tensor ws =
        workspace(g_bwd_sinks_workspace(m.B, m.Hq, m.Hkv, m.Sq, m.Sk, m.D, std::max(m.sinks, 0)), m.q);
    check(g_bwd_sinks(m.q.data_ptr(), m.k.data_ptr(), m.v.data_ptr(), o.data_ptr(),
                      static_cast<const float *>(lse.data_ptr()), dout.data_ptr(),
                      static_cast<float *>(dq.data_ptr()), dk.data_ptr(), dv.data_ptr(), m.B, m.Hq, m.Hkv, m.Sq,
                      m.Sk, m.D, m.scale, m.causal, m.left, m.right, m.sinks, ws.data_ptr(), (size_t)ws.numel(),
                      options<attn_bwd_options_t>(a[11]), current_stream(dev.index())),
          "attn_bwd_sinks");
    return Py_BuildValue("(NNN)", wrap(dq), wrap(dk), wrap(dv));
}

// bind(check, addresses...): the library's functions, in the order of the
// table in attn.py.
PyObject *bind(PyObject *const *a) {
    void **to[] = {reinterpret_cast<void **>(&g_norm_rope),      reinterpret_cast<void **>(&g_norm_rope_cache),
                   reinterpret_cast<void **>(&g_norm_rope_bwd),  reinterpret_cast<void **>(&g_norm_rope_bwd_workspace),
                   reinterpret_cast<void **>(&g_decode),         reinterpret_cast<void **>(&g_decode_workspace),
                   reinterpret_cast<void **>(&g_fwd_sinks),      reinterpret_cast<void **>(&g_fwd_sinks_workspace),
                   reinterpret_cast<void **>(&g_bwd_sinks),      reinterpret_cast<void **>(&g_bwd_sinks_workspace)};
    for (int i = 0; i < 10; ++i) {
        void *p = PyLong_AsVoidPtr(a[1 + i]);
        if (!p) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null function");
            throw PythonError{};
        }
        *to[i] = p;
    }
    Py_INCREF(a[0]);
    Py_XDECREF(g_check);
    g_check = a[0];
    Py_RETURN_NONE;
}

// One entry point: a fixed number of positional arguments; no C++ exception
// leaves it.
template <PyObject *(*F)(PyObject *const *), int N, bool BOUND = true>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected", N);
        return nullptr;
    }
    if (BOUND && !g_check) {
        PyErr_SetString(PyExc_RuntimeError, "the library is not bound");
        return nullptr;
    }
    try {
        return F(args);
    } catch (const PythonError &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef g_methods[] = {
    {"bind", FAST((&entry<bind, 11, false>))},
    {"norm_rope", FAST((&entry<norm_rope, 11>))},
    {"norm_rope_cache", FAST((&entry<norm_rope_cache, 16>))},
    {"norm_rope_backward", FAST((&entry<norm_rope_backward, 13>))},
    {"decode", FAST((&entry<decode, 15>))},
    {"fwd_sinks", FAST((&entry<fwd_sinks, 9>))},
    {"bwd_sinks", FAST((&entry<bwd_sinks, 12>))},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__binding() {
    return PyModule_Create(&g_module);
}
