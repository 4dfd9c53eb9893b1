// torch_calls.cpp -- the calls of the softmax-attention layers' operators (include/delta_rule.h) on
// torch tensors: checks, output allocation and the current stream, in C++.
//
// These calls are made for every layer of a decoding step, and their kernels take 3 to 15 us there;
// the same checks, allocations and foreign calls from Python take 16 to 22 us.  The module holds no
// computation and no reference to the library: binding.py hands it the C entry points' addresses.
// A function returns its tensors, or the entry point's error code (an int); a wrong element type,
// device, shape or layout is a ValueError.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/delta_rule.h"

namespace {

decltype(&delta_rule_pages) c_pages;
decltype(&delta_rule_qkrope) c_qkrope;
decltype(&delta_rule_qkrope_workspace_size) c_qkrope_ws;
decltype(&delta_rule_qkrope_bwd) c_qkrope_bwd;
decltype(&delta_rule_qkrope_cache) c_qkrope_cache;
decltype(&delta_rule_attn_decode_workspace_size) c_attn_ws;
decltype(&delta_rule_attn_decode) c_attn;

typedef PyObject *const *Args;

const at::Tensor &tensor(PyObject *o, const char *what) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), what, " must be a tensor, got ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

long long integer(PyObject *o) {
    PyObject *i = PyNumber_Index(o);
    if (!i) throw python_error();
    const long long v = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
int integer32(PyObject *o, const char *what) {
    const long long v = integer(o);
    TORCH_CHECK_VALUE(v >= INT_MIN && v <= INT_MAX, what, " = ", v, " is out of range");
    return (int)v;
}
int extent(int64_t n, const char *what) {
    TORCH_CHECK_VALUE(n <= INT_MAX, what, " has ", n, " entries along one dimension");
    return (int)n;
}
bool truth(PyObject *o) {
    const int t = PyObject_IsTrue(o);
    if (t < 0) throw python_error();
    return t != 0;
}

at::Device cuda_of(const at::Tensor &t, const char *what) {
    TORCH_CHECK_VALUE(t.is_cuda(), what, " must be a CUDA tensor");
    return t.device();
}
int dtype_of(const at::Tensor &t, const char *what) {
    TORCH_CHECK_VALUE(t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16, what,
                      ": expected torch.float32 or torch.bfloat16, got ", t.scalar_type());
    return t.scalar_type() == at::kBFloat16 ? DR_BF16 : DR_F32;
}
void check(const at::Tensor &t, const char *what, at::ScalarType type, at::Device dev) {
    TORCH_CHECK_VALUE(t.scalar_type() == type && t.device() == dev, what, ": expected ", type, " on ", dev, ", got ",
                      t.scalar_type(), " on ", t.device());
}
// address of a dense tensor of n elements (n < 0: of any number)
void *dense(const at::Tensor &t, const char *what, at::ScalarType type, at::Device dev, int64_t n) {
    check(t, what, type, dev);
    TORCH_CHECK_VALUE(n < 0 || t.numel() == n, what, ": expected ", n, " elements, got shape ", t.sizes());
    TORCH_CHECK_VALUE(t.is_contiguous(), what, " must be contiguous");
    return t.data_ptr();
}
void *dense_or_none(PyObject *o, const char *what, at::ScalarType type, at::Device dev, int64_t n) {
    return o == Py_None ? nullptr : dense(tensor(o, what), what, type, dev, n);
}
void same_shape(const at::Tensor &t, const char *what, at::IntArrayRef shape) {
    TORCH_CHECK_VALUE(t.sizes() == shape, what, ": expected shape ", shape, ", got ", t.sizes());
}

// Elements from a token to the next of a [B, T, H, d] or [N, H, d] tensor with dense heads.
long long token_stride(const at::Tensor &t, const char *what) {
    const int64_t n = t.dim();
    bool ok = n == 3 || n == 4;
    long long tok = 0;
    if (ok) {
        const auto shape = t.sizes(), st = t.strides();
        const int64_t H = shape[n - 2], d = shape[n - 1];
        ok = (st[n - 1] == 1 || d == 1) && (st[n - 2] == d || H == 1);
        tok = st[n - 3];
        if (n == 4 && shape[1] == 1) tok = st[0];
        else if (n == 4 && shape[0] > 1) ok = ok && st[0] == shape[1] * tok;
        if (shape[n - 3] <= 1 && (n == 3 || shape[0] <= 1)) tok = H * d;  // one token: its stride says nothing
        if (t.numel() == 0) ok = true, tok = H * d;
    }
    TORCH_CHECK_VALUE(ok, what, ": expected [B, T, H, d] or [N, H, d] with dense heads and evenly spaced tokens, got strides ",
                      t.strides(), " of shape ", t.sizes());
    return tok;
}

// Elements from a page, a token and a head to the next of a cache [pages, page, Hk, d] with dense
// channels (of a dimension of one entry: as if dense).
struct Strides {
    long long page, token, head;
};
Strides cache_strides(const at::Tensor &t, const char *what) {
    TORCH_CHECK_VALUE(t.dim() == 4, what, ": expected [pages, page, Hk, d], got shape ", t.sizes());
    const auto shape = t.sizes(), st = t.strides();
    const int64_t page = shape[1], H = shape[2], d = shape[3];
    TORCH_CHECK_VALUE(st[3] == 1 || d == 1, what, ": a head's channels must be dense, got strides ", st);
    return {shape[0] > 1 ? st[0] : page * H * d, page > 1 ? st[1] : H * d, H > 1 ? st[2] : d};
}

// The call's device and its current stream.
struct On {
    c10::cuda::CUDAGuard guard;
    void *stream;
    explicit On(at::Device dev) : guard(dev), stream(c10::cuda::getCurrentCUDAStream(dev.index()).stream()) {}
};

// a new dense tensor, straight from the allocator (at::empty's dispatch takes as long again)
at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
    return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}
at::Tensor like(const at::Tensor &t) { return empty(t.sizes(), t.scalar_type(), t.device()); }

// Several new dense tensors side by side in one allocation, each beginning at a multiple of its element
// size (an allocation takes half a microsecond).  All of it lives as long as any of them, so outputs
// beyond a megabyte get allocations of their own.
struct Together {
    at::Tensor all;
    int64_t at = 0;
    Together(int64_t bytes, at::Device dev) : all(empty({bytes}, at::kByte, dev)) {}
    at::Tensor next(at::ScalarType type, at::IntArrayRef shape) {
        const int64_t size = (int64_t)c10::elementSize(type);
        auto t = c10::make_intrusive<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), c10::scalarTypeToTypeMeta(type));
        t->set_storage_offset(at / size);
        t->set_sizes_contiguous(shape);
        at += t->numel() * size;
        return at::Tensor(std::move(t));
    }
};
constexpr int64_t SMALL = 1 << 20;
// two tensors like a and b
std::pair<at::Tensor, at::Tensor> like_both(const at::Tensor &a, const at::Tensor &b) {
    const int64_t bytes = (a.numel() + b.numel()) * a.element_size();
    if (bytes > SMALL || a.numel() * a.element_size() % 256) return {like(a), like(b)};
    Together t(bytes, a.device());
    at::Tensor x = t.next(a.scalar_type(), a.sizes());
    return {x, t.next(b.scalar_type(), b.sizes())};
}

PyObject *code(int rc) { return PyLong_FromLong(rc); }
template <typename... T> PyObject *give(const T &...t) {
    PyObject *r = PyTuple_New(sizeof...(t));
    if (!r) throw python_error();
    Py_ssize_t i = 0;
    auto put = [&](const at::Tensor &x) {
        PyObject *o = x.defined() ? THPVariable_Wrap(x) : Py_NewRef(Py_None);
        if (!o) {
            Py_DECREF(r);
            throw python_error();
        }
        PyTuple_SET_ITEM(r, i++, o);
    };
    (put(t), ...);
    return r;
}
void count(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

// (cached, fresh, free_pages, n_free, table, page, tokens)
PyObject *pages(PyObject *, Args a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 7);
    const at::Tensor &cached = tensor(a[0], "cached"), &fresh = tensor(a[1], "fresh"), &stack = tensor(a[2], "free_pages"),
                     &n_free = tensor(a[3], "n_free"), &table = tensor(a[4], "table");
    const int page = integer32(a[5], "page"), N = integer32(a[6], "tokens");
    const at::Device dev = cuda_of(cached, "cached");
    TORCH_CHECK_VALUE(cached.dim() == 1 && table.dim() == 2 && stack.dim() == 1 && table.size(0) == cached.size(0) && N >= 0,
                      "delta_rule_pages takes cached, fresh [R], free_pages [F], n_free [1], table [R, width] and tokens >= 0, "
                      "got cached ", cached.sizes(), ", free_pages ", stack.sizes(), ", table ", table.sizes(), ", tokens ", N);
    const int R = extent(cached.numel(), "cached");
    void *cp = dense(cached, "cached", at::kInt, dev, -1), *fp = dense(fresh, "fresh", at::kInt, dev, R),
         *sp = dense(stack, "free_pages", at::kInt, dev, -1), *np = dense(n_free, "n_free", at::kInt, dev, 1),
         *tp = dense(table, "table", at::kInt, dev, -1);
    if (R > 8192 || N > 1 << 30) return code(DR_ERR_UNSUPPORTED);  // before gigabytes are allocated for the refusal
    On on(dev);
    // lens and n_left are kept for the next step, the rows' outputs are not: those of many tokens stand alone
    const bool apart = 12ll * N > SMALL;
    at::Tensor slots, pos;
    if (apart) {
        slots = empty({N}, at::kLong, dev);
        pos = empty({N}, at::kInt, dev);
    }
    Together t((apart ? 0 : 12ll * N) + 8ll * R + 8, dev);  // the 8-byte elements first
    if (!apart) {
        slots = t.next(at::kLong, {N});
        pos = t.next(at::kInt, {N});
    }
    const at::Tensor lens = t.next(at::kInt, {R}), cu = t.next(at::kInt, {R + 1ll}), left = t.next(at::kInt, {1});
    const int rc = c_pages((int *)cp, (int *)fp, (int *)sp, (int *)np, (int *)tp, (int *)lens.data_ptr(), (int *)cu.data_ptr(),
                           (int *)pos.data_ptr(), (long long *)slots.data_ptr(), (int *)left.data_ptr(), R,
                           extent(stack.numel(), "free_pages"), extent(table.size(1), "table"), page, N, on.stream);
    return rc == DR_OK ? give(lens, cu, pos, slots, left) : code(rc);
    END_HANDLE_TH_ERRORS
}

// What the forms of the norm with rotation take alike: (q, k, wq, wk, inv_freq, positions).
struct QK {
    const at::Tensor &q, &k;
    at::Device dev;
    int dtype, B, T, Hq, Hk, d, rot;
    long long qs, ks;
    float *wq, *wk;
    double *f;
    int *pos;
    explicit QK(Args a)
        : q(tensor(a[0], "q")), k(tensor(a[1], "k")), dev(cuda_of(q, "q")), dtype(dtype_of(q, "q")) {
        check(k, "k", q.scalar_type(), dev);
        qs = token_stride(q, "q");
        ks = token_stride(k, "k");
        const int64_t n = q.dim();
        bool alike = k.dim() == n && k.size(n - 1) == q.size(n - 1);
        for (int64_t i = 0; alike && i < n - 2; ++i) alike = k.size(i) == q.size(i);
        TORCH_CHECK_VALUE(alike, "k: expected the tokens and channels of q ", q.sizes(), ", got ", k.sizes());
        B = n == 4 ? extent(q.size(0), "q") : 1;
        T = extent(q.size(n - 3), "q");
        Hq = extent(q.size(n - 2), "q");
        Hk = extent(k.size(n - 2), "k");
        d = extent(q.size(n - 1), "q");
        wq = (float *)dense_or_none(a[2], "wq", at::kFloat, dev, d);
        wk = (float *)dense_or_none(a[3], "wk", at::kFloat, dev, d);
        f = (double *)dense_or_none(a[4], "inv_freq", at::kDouble, dev, -1);
        rot = a[4] == Py_None ? 0 : 2 * extent(tensor(a[4], "inv_freq").numel(), "inv_freq");
        pos = (int *)dense_or_none(a[5], "positions", at::kInt, dev, (int64_t)B * T);
    }
};

// (..., interleaved)
PyObject *qkrope(PyObject *, Args a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 7);
    const QK x(a);
    const bool inter = truth(a[6]);
    On on(x.dev);
    const auto [qo, ko] = like_both(x.q, x.k);
    const int rc = c_qkrope(x.q.data_ptr(), x.k.data_ptr(), x.wq, x.wk, x.f, x.pos, qo.data_ptr(), ko.data_ptr(), x.B, x.T, x.Hq,
                            x.Hk, x.d, x.rot, inter, x.qs, x.ks, x.dtype, on.stream);
    return rc == DR_OK ? give(qo, ko) : code(rc);
    END_HANDLE_TH_ERRORS
}

// a tensor of t's shape, type and device: the one given, or a new one
at::Tensor out_like(PyObject *o, const char *what, const at::Tensor &t) {
    if (o == Py_None) return like(t);
    const at::Tensor &x = tensor(o, what);
    check(x, what, t.scalar_type(), t.device());
    same_shape(x, what, t.sizes());
    return x;
}

// (..., interleaved, dq_out, dk_out, dq, dk, want_dw)
PyObject *qkrope_bwd(PyObject *, Args a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 12);
    const QK x(a);
    const bool inter = truth(a[6]), want = truth(a[11]);
    const at::Tensor &gq = tensor(a[7], "dq_out"), &gk = tensor(a[8], "dk_out");
    same_shape(gq, "dq_out", x.q.sizes());
    same_shape(gk, "dk_out", x.k.sizes());
    void *gqp = dense(gq, "dq_out", x.q.scalar_type(), x.dev, -1), *gkp = dense(gk, "dk_out", x.q.scalar_type(), x.dev, -1);
    On on(x.dev);
    const bool ours = a[9] == Py_None && a[10] == Py_None;
    const auto [nq, nk] = ours ? like_both(x.q, x.k) : std::pair(out_like(a[9], "dq", x.q), out_like(a[10], "dk", x.k));
    const at::Tensor &dq = nq, &dk = nk;
    const long long dqs = token_stride(dq, "dq"), dks = token_stride(dk, "dk");
    at::Tensor dwq, dwk, ws;
    size_t need = 0;
    if (want) {
        need = c_qkrope_ws(x.d);
        if (need == (size_t)-1) return code(DR_ERR_UNSUPPORTED);
        Together t(8ll * x.d, x.dev);
        dwq = t.next(at::kFloat, {x.d});
        dwk = t.next(at::kFloat, {x.d});
        ws = empty({(int64_t)need}, at::kByte, x.dev);
    }
    const int rc = c_qkrope_bwd(x.q.data_ptr(), x.k.data_ptr(), x.wq, x.wk, x.f, x.pos, gqp, gkp, dq.data_ptr(), dk.data_ptr(),
                                want ? (float *)dwq.data_ptr() : nullptr, want ? (float *)dwk.data_ptr() : nullptr, x.B, x.T,
                                x.Hq, x.Hk, x.d, x.rot, inter, x.qs, x.ks, dqs, dks, x.dtype, want ? ws.data_ptr() : nullptr,
                                need, on.stream);
    return rc == DR_OK ? give(dq, dk, dwq, dwk) : code(rc);
    END_HANDLE_TH_ERRORS
}

// (..., interleaved, v, slots, k_cache, v_cache, q_out)
PyObject *qkrope_cache(PyObject *, Args a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 12);
    const QK x(a);
    const bool inter = truth(a[6]);
    const at::Tensor &v = tensor(a[7], "v"), &kc = tensor(a[9], "k_cache"), &vc = tensor(a[10], "v_cache");
    const auto type = x.q.scalar_type();
    check(v, "v", type, x.dev);
    same_shape(v, "v", x.k.sizes());
    check(kc, "k_cache", type, x.dev);
    check(vc, "v_cache", type, x.dev);
    const long long vs = token_stride(v, "v");
    const Strides ks = cache_strides(kc, "k_cache"), vst = cache_strides(vc, "v_cache");
    TORCH_CHECK_VALUE(kc.sizes() == vc.sizes() && kc.size(2) == x.Hk && kc.size(3) == x.d, "the caches must be [pages, page, ",
                      x.Hk, ", ", x.d, "], got ", kc.sizes(), " and ", vc.sizes());
    const int64_t tokens = (int64_t)x.B * x.T;
    TORCH_CHECK_VALUE(x.pos, "delta_rule_qkrope_cache takes a position for each token");
    void *slots = dense(tensor(a[8], "slots"), "slots", at::kLong, x.dev, tokens);
    On on(x.dev);
    const at::Tensor qo = out_like(a[11], "q_out", x.q);
    TORCH_CHECK_VALUE(qo.is_contiguous(), "q_out must be contiguous");
    const int rc = c_qkrope_cache(x.q.data_ptr(), x.k.data_ptr(), v.data_ptr(), x.wq, x.wk, x.f, x.pos, (long long *)slots,
                                  qo.data_ptr(), kc.data_ptr(), vc.data_ptr(), extent(tokens, "q"), x.Hq, x.Hk, x.d, x.rot, inter,
                                  x.qs, x.ks, vs, extent(kc.size(0), "k_cache"), extent(kc.size(1), "k_cache"), ks.page, ks.token, ks.head,
                                  vst.page, vst.token, vst.head, x.dtype, on.stream);
    return rc == DR_OK ? give(qo) : code(rc);
    END_HANDLE_TH_ERRORS
}

// (q, k_cache, v_cache, table, lens, scale or None, window, want_lse, out or None, workspace or None)
PyObject *attn_decode(PyObject *, Args a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 10);
    const at::Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache"),
                     &table = tensor(a[3], "table"), &lens = tensor(a[4], "lens");
    const at::Device dev = cuda_of(q, "q");
    const int dtype = dtype_of(q, "q");
    TORCH_CHECK_VALUE(q.dim() == 3 && table.dim() == 2 && table.size(0) == q.size(0),
                      "delta_rule_attn_decode takes q [R, Hq, d] and table [R, width], got ", q.sizes(), " and ", table.sizes());
    const int R = extent(q.size(0), "q"), Hq = extent(q.size(1), "q"), d = extent(q.size(2), "q");
    check(kc, "k_cache", q.scalar_type(), dev);
    check(vc, "v_cache", q.scalar_type(), dev);
    const Strides ks = cache_strides(kc, "k_cache"), vs = cache_strides(vc, "v_cache");
    TORCH_CHECK_VALUE(kc.sizes() == vc.sizes() && kc.size(3) == d, "the caches must be [pages, page, Hk, ", d, "], got ", kc.sizes(),
                      " and ", vc.sizes());
    const int Hk = extent(kc.size(2), "k_cache");
    void *qp = dense(q, "q", q.scalar_type(), dev, -1), *tp = dense(table, "table", at::kInt, dev, -1),
         *lp = dense(lens, "lens", at::kInt, dev, R);
    double scale = 0;
    if (a[5] == Py_None) {
        scale = 1.0 / std::sqrt((double)d);
    } else {
        scale = PyFloat_AsDouble(a[5]);
        if (scale == -1.0 && PyErr_Occurred()) throw python_error();
    }
    const int window = integer32(a[6], "window");
    const bool want = truth(a[7]);
    const size_t need = c_attn_ws(Hq, Hk, d, dtype);
    if (need == (size_t)-1) return code(Hq > 0 && Hk > 0 && Hq % Hk == 0 && d > 0 ? DR_ERR_UNSUPPORTED : DR_ERR_ARG);
    On on(dev);
    at::Tensor out, lse, ws;
    const int64_t bytes = q.numel() * q.element_size();
    if (want && a[8] == Py_None && bytes <= SMALL && bytes % 256 == 0) {
        Together t(bytes + 4ll * R * Hq, dev);
        out = t.next(q.scalar_type(), q.sizes());
        lse = t.next(at::kFloat, {R, Hq});
    } else {
        out = out_like(a[8], "out", q);
        TORCH_CHECK_VALUE(out.is_contiguous(), "out must be contiguous");
        if (want) lse = empty({R, Hq}, at::kFloat, dev);
    }
    if (a[9] != Py_None) {
        ws = tensor(a[9], "workspace");
        dense(ws, "workspace", at::kByte, dev, -1);
    }
    if (!ws.defined() || (size_t)ws.numel() < need) ws = empty({(int64_t)need}, at::kByte, dev);
    const int rc = c_attn(qp, kc.data_ptr(), vc.data_ptr(), (int *)tp, (int *)lp, out.data_ptr(),
                          want ? (float *)lse.data_ptr() : nullptr, R, Hq, Hk, d, extent(kc.size(0), "k_cache"),
                          extent(kc.size(1), "k_cache"), extent(table.size(1), "table"), ks.page, ks.token, ks.head, vs.page,
                          vs.token, vs.head, (float)scale, window, dtype,
                          ws.data_ptr(), need, on.stream);
    return rc == DR_OK ? give(out, lse) : code(rc);
    END_HANDLE_TH_ERRORS
}

// the layouts alone, for tests without a GPU
PyObject *stride_of_tokens(PyObject *, Args a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 1);
    return PyLong_FromLongLong(token_stride(tensor(a[0], "tensor"), "tensor"));
    END_HANDLE_TH_ERRORS
}
PyObject *strides_of_cache(PyObject *, Args a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 1);
    const Strides st = cache_strides(tensor(a[0], "tensor"), "tensor");
    return Py_BuildValue("LLL", st.page, st.token, st.head);
    END_HANDLE_TH_ERRORS
}

// the entry points' addresses, in the order of the declarations above
PyObject *bind(PyObject *, Args a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 7);
    void *p[7];
    for (int i = 0; i < 7; ++i) p[i] = (void *)(uintptr_t)integer(a[i]);
    c_pages = (decltype(c_pages))p[0];
    c_qkrope = (decltype(c_qkrope))p[1];
    c_qkrope_ws = (decltype(c_qkrope_ws))p[2];
    c_qkrope_bwd = (decltype(c_qkrope_bwd))p[3];
    c_qkrope_cache = (decltype(c_qkrope_cache))p[4];
    c_attn_ws = (decltype(c_attn_ws))p[5];
    c_attn = (decltype(c_attn))p[6];
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),        FAST(pages),       FAST(qkrope),           FAST(qkrope_bwd),     FAST(qkrope_cache),
                         FAST(attn_decode), FAST(stride_of_tokens), FAST(strides_of_cache), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

#ifndef CALLS_KEY
#define CALLS_KEY ""
#endif
// `built_from`: the key of the sources, the command, torch and Python that the module was built from
PyMODINIT_FUNC PyInit__torch_calls(void) {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_from", CALLS_KEY) != 0) Py_CLEAR(m);
    return m;
}
