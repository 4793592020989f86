// py_attn.cpp -- the Python side of the attention sublayer's entry points:
// argument checks and marshalling, as a CPython module (_attn_calls).
//
// These calls are made for every layer of a decoding step, where the host's
// time is the call's time.  The same checks in Python with a ctypes call take
// 17 to 28 us on the host of a GB300, most of it interpretation; here a tensor
// costs its attributes' getters.  The module knows nothing of torch but the
// names of those attributes; outputs come from the caller's allocator.
//
// Every function returns (status, outputs...) with the library's status, or
// raises TypeError / ValueError for what the library could not see.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <math.h>
#include <stdint.h>

#include "../../include/mhc.h"

namespace {

// Interned attribute names and the objects that `setup` is given.
struct Names {
    PyObject *dtype, *is_cuda, *shape, *stride, *data_ptr, *numel, *is_contiguous, *device, *get_device;
} N;
struct Kinds {
    PyObject *bf16, *f32, *i32, *i64, *u8, *raw_stream;
} K;

// One owned reference.
class Ref {
  public:
    explicit Ref(PyObject* p = nullptr) : p_(p) {}
    Ref(const Ref&) = delete;
    Ref& operator=(const Ref&) = delete;
    ~Ref() { Py_XDECREF(p_); }
    PyObject* get() const { return p_; }
    PyObject* release() {
        PyObject* p = p_;
        p_ = nullptr;
        return p;
    }
    void reset(PyObject* p) {
        Py_XDECREF(p_);
        p_ = p;
    }
    explicit operator bool() const { return p_ != nullptr; }

  private:
    PyObject* p_;
};

bool to_i64(PyObject* o, int64_t* out) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) return false;
    *out = v;
    return true;
}
bool to_int(PyObject* o, int* out) {
    int64_t v;
    if (!to_i64(o, &v)) return false;
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_SetString(PyExc_OverflowError, "the argument does not fit 32 bits");
        return false;
    }
    *out = static_cast<int>(v);
    return true;
}
bool to_float(PyObject* o, float* out) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) return false;
    *out = static_cast<float>(v);
    return true;
}

bool is_true(PyObject* t, PyObject* name) {
    Ref v(PyObject_GetAttr(t, name));
    return v && v.get() == Py_True;
}
bool call_i64(PyObject* t, PyObject* name, int64_t* out) {
    Ref v(PyObject_CallMethodNoArgs(t, name));
    return v && to_i64(v.get(), out);
}

// A tuple attribute or method result of exactly n integers.
bool ints_of(PyObject* tuple, Py_ssize_t n, int64_t* out, const char* name) {
    if (!PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) != n) {
        PyErr_Format(PyExc_ValueError, "%s must have %zd dimensions", name, n);
        return false;
    }
    for (Py_ssize_t i = 0; i < n; ++i)
        if (!to_i64(PyTuple_GET_ITEM(tuple, i), out + i)) return false;
    return true;
}
bool shape_of(PyObject* t, Py_ssize_t n, int64_t* out, const char* name) {
    Ref s(PyObject_GetAttr(t, N.shape));
    return s && ints_of(s.get(), n, out, name);
}
bool stride_of(PyObject* t, Py_ssize_t n, int64_t* out, const char* name) {
    Ref s(PyObject_CallMethodNoArgs(t, N.stride));
    return s && ints_of(s.get(), n, out, name);
}

bool check_dtype(PyObject* t, PyObject* want, const char* name) {
    Ref d(PyObject_GetAttr(t, N.dtype));
    if (!d) return false;
    if (d.get() == want) return true;
    PyErr_Format(PyExc_TypeError, "%s must be %S, got %S", name, want, d.get());
    return false;
}
bool check_cuda(PyObject* t) {
    if (is_true(t, N.is_cuda)) return true;
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "the mHC library takes CUDA tensors only");
    return false;
}
bool pointer_of(PyObject* t, void** out) {
    int64_t v;
    if (!call_i64(t, N.data_ptr, &v)) return false;
    *out = reinterpret_cast<void*>(static_cast<uintptr_t>(v));
    return true;
}

// The activations' type (a borrowed reference) and its code.
bool activations(PyObject* t, PyObject** dtype, mhc_dtype* code) {
    Ref d(PyObject_GetAttr(t, N.dtype));
    if (!d) return false;
    if (d.get() == K.bf16) *code = MHC_BF16;
    else if (d.get() == K.f32) *code = MHC_F32;
    else {
        PyErr_Format(PyExc_TypeError, "activations must be bfloat16 or float32, got %S", d.get());
        return false;
    }
    *dtype = *code == MHC_BF16 ? K.bf16 : K.f32;
    return true;
}

// A tensor of heads [T, H, Dh]: address and distance of its tokens, which may
// be apart (a part of a packed projection); a token's heads are not.
struct Heads {
    void* p;
    int64_t stride;
};
bool heads_of(PyObject* t, const char* name, PyObject* dtype, const int64_t (&shape)[3], Heads* out) {
    int64_t st[3];
    if (!check_dtype(t, dtype, name) || !check_cuda(t) || !stride_of(t, 3, st, name)) return false;
    if ((st[2] != 1 && shape[2] > 1) || (st[1] != shape[2] && shape[1] > 1)) {
        PyErr_Format(PyExc_ValueError, "%s: the heads of a token must lie one after the other", name);
        return false;
    }
    out->stride = shape[0] > 1 ? st[0] : shape[1] * shape[2];
    return pointer_of(t, &out->p);
}

// A dense tensor of n entries.
bool flat_of(PyObject* t, const char* name, PyObject* dtype, int64_t n, void** out) {
    int64_t have;
    if (!check_dtype(t, dtype, name) || !call_i64(t, N.numel, &have)) return false;
    if (have != n) {
        PyErr_Format(PyExc_ValueError, "%s must have %lld entries, got %lld", name, static_cast<long long>(n),
                     static_cast<long long>(have));
        return false;
    }
    if (!check_cuda(t)) return false;
    Ref c(PyObject_CallMethodNoArgs(t, N.is_contiguous));
    if (!c) return false;
    if (c.get() != Py_True) {
        PyErr_SetString(PyExc_ValueError, "the mHC library takes contiguous tensors only");
        return false;
    }
    return pointer_of(t, out);
}

// A cache [pages, page_size, Hk, Dh] in any memory order that keeps a head's
// values together.
struct Cache {
    void* p;
    int64_t page, slot, head;
};
bool cache_of(PyObject* t, const char* name, PyObject* dtype, const int64_t (&shape)[4], Cache* out) {
    int64_t have[4], st[4];
    if (!check_dtype(t, dtype, name) || !check_cuda(t) || !shape_of(t, 4, have, name) || !stride_of(t, 4, st, name))
        return false;
    for (int i = 0; i < 4; ++i)
        if (have[i] != shape[i]) {
            PyErr_Format(PyExc_ValueError, "%s must be [%lld, %lld, %lld, %lld]", name,
                         static_cast<long long>(shape[0]), static_cast<long long>(shape[1]),
                         static_cast<long long>(shape[2]), static_cast<long long>(shape[3]));
            return false;
        }
    if (st[3] != 1 && shape[3] > 1) {
        PyErr_Format(PyExc_ValueError, "%s: the values of a head must lie one after the other", name);
        return false;
    }
    out->page = shape[0] > 1 ? st[0] : shape[1] * shape[2] * shape[3];
    out->slot = shape[1] > 1 ? st[1] : shape[2] * shape[3];
    out->head = shape[2] > 1 ? st[2] : shape[3];
    return pointer_of(t, &out->p);
}

// Positions and angles; both may be None.
struct Rope {
    void *positions = nullptr, *cos_sin = nullptr;
    int64_t max_pos = 0;
    int rot = 0;
};
bool rope_of(PyObject* positions, PyObject* cos_sin, int64_t T, Rope* out) {
    if (cos_sin == Py_None) return true;
    int64_t s[2];
    if (!shape_of(cos_sin, 2, s, "cos_sin")) return false;
    out->max_pos = s[0];
    out->rot = s[1] > INT32_MAX ? INT32_MAX : static_cast<int>(s[1]);
    return flat_of(positions, "positions", K.i32, T, &out->positions) &&
           flat_of(cos_sin, "cos_sin", K.f32, s[0] * s[1], &out->cos_sin);
}

// q [T, Hq, Dh] and k [T, Hk, Dh].
bool same_tokens(PyObject* q, PyObject* k, int64_t (&sq)[3], int64_t (&sk)[3]) {
    if (!shape_of(q, 3, sq, "q") || !shape_of(k, 3, sk, "k")) return false;
    if (sq[0] == sk[0] && sq[2] == sk[2]) return true;
    PyErr_SetString(PyExc_ValueError, "q and k must have the same tokens and head size");
    return false;
}
bool same_shape(PyObject* t, const int64_t (&want)[3], const char* message) {
    int64_t s[3];
    if (!shape_of(t, 3, s, "a tensor of heads")) return false;
    if (s[0] == want[0] && s[1] == want[1] && s[2] == want[2]) return true;
    PyErr_SetString(PyExc_ValueError, message);
    return false;
}

bool stream_of(PyObject* t, cudaStream_t* out) {
    Ref dev(PyObject_CallMethodNoArgs(t, N.get_device));
    if (!dev) return false;
    Ref s(PyObject_CallOneArg(K.raw_stream, dev.get()));
    int64_t v;
    if (!s || !to_i64(s.get(), &v)) return false;
    *out = reinterpret_cast<cudaStream_t>(static_cast<uintptr_t>(v));
    return true;
}

// empty(shape, dtype, device) and the new tensor's address.
PyObject* make(PyObject* empty, PyObject* dtype, PyObject* device, int n, const int64_t* shape, void** p) {
    Ref dims(PyTuple_New(n));
    if (!dims) return nullptr;
    for (int i = 0; i < n; ++i) {
        PyObject* v = PyLong_FromLongLong(shape[i]);
        if (v == nullptr) return nullptr;
        PyTuple_SET_ITEM(dims.get(), i, v);
    }
    PyObject* args[3] = {dims.get(), dtype, device};
    Ref t(PyObject_Vectorcall(empty, args, 3, nullptr));
    if (!t || !pointer_of(t.get(), p)) return nullptr;
    return t.release();
}
PyObject* make_bytes(PyObject* empty, PyObject* device, size_t bytes, void** p) {
    const int64_t n = bytes > 0 ? static_cast<int64_t>(bytes) : 16;
    return make(empty, K.u8, device, 1, &n, p);
}

bool arguments(Py_ssize_t have, Py_ssize_t want) {
    if (have == want && K.bf16 != nullptr) return true;
    PyErr_SetString(PyExc_TypeError, K.bf16 == nullptr ? "setup() has not been called" : "wrong number of arguments");
    return false;
}
int clip(int64_t v) { return v > INT32_MAX ? INT32_MAX : static_cast<int>(v); }

// --------------------------------------------------------------- functions ---

// (empty, q, k, w_q, w_k, positions, cos_sin, eps, flags) -> (status, q_out, k_out)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arguments(n, 9)) return nullptr;
    int64_t sq[3], sk[3];
    PyObject* dt;
    mhc_dtype code;
    void *wq, *wk, *qo, *ko;
    Heads q, k;
    Rope rope;
    float eps;
    int flags;
    cudaStream_t stream;
    if (!same_tokens(a[1], a[2], sq, sk) || !activations(a[1], &dt, &code) ||
        !flat_of(a[3], "w_q", K.f32, sq[2], &wq) || !flat_of(a[4], "w_k", K.f32, sq[2], &wk) ||
        !heads_of(a[1], "q", dt, sq, &q) || !heads_of(a[2], "k", dt, sk, &k) ||
        !rope_of(a[5], a[6], sq[0], &rope) || !to_float(a[7], &eps) || !to_int(a[8], &flags) ||
        !stream_of(a[1], &stream))
        return nullptr;
    Ref dev(PyObject_GetAttr(a[1], N.device));
    if (!dev) return nullptr;
    Ref to(make(a[0], dt, dev.get(), 3, sq, &qo));
    if (!to) return nullptr;
    Ref tk(make(a[0], dt, dev.get(), 3, sk, &ko));
    if (!tk) return nullptr;
    const int st = mhc_qk_norm_rope(code, q.p, q.stride, k.p, k.stride, static_cast<float*>(wq), static_cast<float*>(wk),
                                    static_cast<int32_t*>(rope.positions), static_cast<float*>(rope.cos_sin),
                                    rope.max_pos, sq[0], clip(sq[1]), clip(sk[1]), clip(sq[2]), rope.rot, flags, eps, qo,
                                    sq[1] * sq[2], ko, sk[1] * sk[2], stream);
    return Py_BuildValue("iOO", st, to.get(), tk.get());
}

// (empty, g_q, g_k, q, k, w_q, w_k, positions, cos_sin, eps, flags, dq | None, dk | None)
//   -> (status, dq, dk, dw_q, dw_k)
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arguments(n, 13)) return nullptr;
    int64_t sq[3], sk[3];
    PyObject* dt;
    mhc_dtype code;
    void *wq, *wk, *dwq, *dwk, *ws;
    Heads gq, gk, q, k, dq, dk;
    Rope rope;
    float eps;
    int flags;
    cudaStream_t stream;
    if (!same_tokens(a[3], a[4], sq, sk) || !activations(a[3], &dt, &code) ||
        !same_shape(a[1], sq, "q, k and their gradients must have the same shapes") ||
        !same_shape(a[2], sk, "q, k and their gradients must have the same shapes") ||
        !flat_of(a[5], "w_q", K.f32, sq[2], &wq) || !flat_of(a[6], "w_k", K.f32, sq[2], &wk) ||
        !heads_of(a[1], "g_q", dt, sq, &gq) || !heads_of(a[2], "g_k", dt, sk, &gk) ||
        !heads_of(a[3], "q", dt, sq, &q) || !heads_of(a[4], "k", dt, sk, &k) ||
        !rope_of(a[7], a[8], sq[0], &rope) || !to_float(a[9], &eps) || !to_int(a[10], &flags) ||
        !stream_of(a[3], &stream))
        return nullptr;
    Ref dev(PyObject_GetAttr(a[3], N.device));
    if (!dev) return nullptr;
    Ref tq, tk;
    if (a[11] == Py_None) {
        tq.reset(make(a[0], dt, dev.get(), 3, sq, &dq.p));
        if (!tq) return nullptr;
        dq.stride = sq[1] * sq[2];
    } else {
        if (!same_shape(a[11], sq, "dq and dk must have the shapes of q and k") || !heads_of(a[11], "dq", dt, sq, &dq))
            return nullptr;
        tq.reset(Py_NewRef(a[11]));
    }
    if (a[12] == Py_None) {
        tk.reset(make(a[0], dt, dev.get(), 3, sk, &dk.p));
        if (!tk) return nullptr;
        dk.stride = sk[1] * sk[2];
    } else {
        if (!same_shape(a[12], sk, "dq and dk must have the shapes of q and k") || !heads_of(a[12], "dk", dt, sk, &dk))
            return nullptr;
        tk.reset(Py_NewRef(a[12]));
    }
    Ref twq(make(a[0], K.f32, dev.get(), 1, sq + 2, &dwq));
    if (!twq) return nullptr;
    Ref twk(make(a[0], K.f32, dev.get(), 1, sq + 2, &dwk));
    if (!twk) return nullptr;
    const size_t need = mhc_qk_norm_rope_bwd_workspace_bytes(sq[0], clip(sq[2]));
    Ref tws(make_bytes(a[0], dev.get(), need, &ws));
    if (!tws) return nullptr;
    const int st = mhc_qk_norm_rope_bwd(
        code, gq.p, gq.stride, gk.p, gk.stride, q.p, q.stride, k.p, k.stride, static_cast<float*>(wq),
        static_cast<float*>(wk), static_cast<int32_t*>(rope.positions), static_cast<float*>(rope.cos_sin), rope.max_pos,
        sq[0], clip(sq[1]), clip(sk[1]), clip(sq[2]), rope.rot, flags, eps, dq.p, dq.stride, dk.p, dk.stride,
        static_cast<float*>(dwq), static_cast<float*>(dwk), ws, need, stream);
    return Py_BuildValue("iOOOO", st, tq.get(), tk.get(), twq.get(), twk.get());
}

// (empty, q, k, v, w_q, w_k, k_cache, v_cache, slots, positions, cos_sin, eps, flags) -> (status, q_out)
PyObject* qk_norm_rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arguments(n, 13)) return nullptr;
    int64_t sq[3], sk[3], sc[4];
    PyObject* dt;
    mhc_dtype code;
    void *wq, *wk, *slots, *qo;
    Heads q, k, v;
    Cache kc, vc;
    Rope rope;
    float eps;
    int flags;
    cudaStream_t stream;
    if (!same_tokens(a[1], a[2], sq, sk) || !activations(a[1], &dt, &code) ||
        !same_shape(a[3], sk, "k and v must have the same shape") || !shape_of(a[6], 4, sc, "k_cache"))
        return nullptr;
    if (sc[2] != sk[1] || sc[3] != sk[2]) {
        PyErr_Format(PyExc_ValueError, "k_cache must be [pages, page_size, %lld, %lld]", static_cast<long long>(sk[1]),
                     static_cast<long long>(sk[2]));
        return nullptr;
    }
    if (!flat_of(a[4], "w_q", K.f32, sq[2], &wq) || !flat_of(a[5], "w_k", K.f32, sq[2], &wk) ||
        !heads_of(a[1], "q", dt, sq, &q) || !heads_of(a[2], "k", dt, sk, &k) || !heads_of(a[3], "v", dt, sk, &v) ||
        !cache_of(a[6], "k_cache", dt, sc, &kc) || !cache_of(a[7], "v_cache", dt, sc, &vc) ||
        !flat_of(a[8], "slots", K.i64, sq[0], &slots) || !rope_of(a[9], a[10], sq[0], &rope) ||
        !to_float(a[11], &eps) || !to_int(a[12], &flags) || !stream_of(a[1], &stream))
        return nullptr;
    Ref dev(PyObject_GetAttr(a[1], N.device));
    if (!dev) return nullptr;
    Ref to(make(a[0], dt, dev.get(), 3, sq, &qo));
    if (!to) return nullptr;
    const int st = mhc_qk_norm_rope_append(
        code, q.p, q.stride, k.p, k.stride, v.p, v.stride, static_cast<float*>(wq), static_cast<float*>(wk),
        static_cast<int32_t*>(rope.positions), static_cast<float*>(rope.cos_sin), rope.max_pos,
        static_cast<int64_t*>(slots), sq[0], clip(sq[1]), clip(sk[1]), clip(sq[2]), rope.rot, flags, eps, qo,
        sq[1] * sq[2], kc.p, kc.page, kc.slot, kc.head, vc.p, vc.page, vc.slot, vc.head, sc[0], clip(sc[1]), stream);
    return Py_BuildValue("iO", st, to.get());
}

// (empty, q, k_cache, v_cache, page_table, cu_q, kv_lens, max_q, max_kv, scale, window, softcap, workspace, out)
//   -> (status, o, lse); None: the lengths where there is a planned workspace, bounds and scale from the shapes, a
//   new workspace, a new output
PyObject* paged_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arguments(n, 14)) return nullptr;
    int64_t sq[3], sc[4], stab[2], tab[2], max_q, max_kv;
    PyObject* dt;
    mhc_dtype code;
    void *table, *cu = nullptr, *kv = nullptr, *o, *lse, *ws;
    Heads q;
    Cache kc, vc;
    float scale, softcap;
    int window;
    cudaStream_t stream;
    if (!shape_of(a[1], 3, sq, "q") || !activations(a[1], &dt, &code) || !shape_of(a[2], 4, sc, "k_cache") ||
        !shape_of(a[4], 2, stab, "page_table") ||
        !to_int(a[10], &window) || !to_float(a[11], &softcap))
        return nullptr;
    if (sc[3] != sq[2]) {
        PyErr_Format(PyExc_ValueError, "k_cache must be [pages, page_size, heads, %lld]", static_cast<long long>(sq[2]));
        return nullptr;
    }
    const int64_t T = sq[0], B = stab[0], width = stab[1], page = sc[1];
    if (a[7] == Py_None) max_q = T;
    else if (!to_i64(a[7], &max_q)) return nullptr;
    if (a[8] == Py_None) max_kv = width * page;
    else if (!to_i64(a[8], &max_kv)) return nullptr;
    if (a[9] == Py_None) scale = 1.0f / sqrtf(static_cast<float>(sq[2]));
    else if (!to_float(a[9], &scale)) return nullptr;
    if (!check_dtype(a[4], K.i32, "page_table") || !check_cuda(a[4]) || !stride_of(a[4], 2, tab, "page_table"))
        return nullptr;
    if (width * page < max_kv) {
        PyErr_Format(PyExc_ValueError, "page_table holds %lld tokens a sequence, max_kv is %lld",
                     static_cast<long long>(width * page), static_cast<long long>(max_kv));
        return nullptr;
    }
    if (tab[1] != 1 && width > 1) {
        PyErr_SetString(PyExc_ValueError, "page_table: the pages of a sequence must lie one after the other");
        return nullptr;
    }
    if (a[12] == Py_None && (!flat_of(a[5], "cu_q", K.i32, B + 1, &cu) || !flat_of(a[6], "kv_lens", K.i32, B, &kv)))
        return nullptr;
    if (!pointer_of(a[4], &table) || !heads_of(a[1], "q", dt, sq, &q) || !cache_of(a[2], "k_cache", dt, sc, &kc) ||
        !cache_of(a[3], "v_cache", dt, sc, &vc) || !stream_of(a[1], &stream))
        return nullptr;
    Ref dev(PyObject_GetAttr(a[1], N.device));
    if (!dev) return nullptr;
    Ref tw;
    int64_t ws_bytes;
    if (a[12] == Py_None) {
        ws_bytes = static_cast<int64_t>(mhc_paged_attn_workspace_bytes(code, T, clip(B), clip(sq[1]), clip(sc[2]),
                                                                       clip(sq[2]), clip(page), max_q));
        tw.reset(make_bytes(a[0], dev.get(), static_cast<size_t>(ws_bytes), &ws));
        if (!tw) return nullptr;
    } else if (!call_i64(a[12], N.numel, &ws_bytes) || !pointer_of(a[12], &ws)) {
        return nullptr;
    }
    Ref to;
    if (a[13] == Py_None) {
        to.reset(make(a[0], dt, dev.get(), 3, sq, &o));
        if (!to) return nullptr;
    } else {
        if (!same_shape(a[13], sq, "out must have the shape of q") ||
            !flat_of(a[13], "out", dt, sq[0] * sq[1] * sq[2], &o))
            return nullptr;
        to.reset(Py_NewRef(a[13]));
    }
    Ref tl(make(a[0], K.f32, dev.get(), 2, sq, &lse));
    if (!tl) return nullptr;
    const int st = mhc_paged_attn(code, q.p, q.stride, kc.p, kc.page, kc.slot, kc.head, vc.p, vc.page, vc.slot, vc.head,
                                  sc[0], clip(page), static_cast<int32_t*>(table), B > 1 ? tab[0] : width,
                                  static_cast<int32_t*>(cu), static_cast<int32_t*>(kv), T, clip(B), clip(sq[1]),
                                  clip(sc[2]), clip(sq[2]), max_q, max_kv, window, scale, softcap, o,
                                  static_cast<float*>(lse), ws, static_cast<size_t>(ws_bytes), stream);
    return Py_BuildValue("iOO", st, to.get(), tl.get());
}

// (bfloat16, float32, int32, int64, uint8, raw_stream): torch's types, and its
// function from a device's index to the current stream's handle.
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "setup takes six arguments");
        return nullptr;
    }
    PyObject** to[6] = {&K.bf16, &K.f32, &K.i32, &K.i64, &K.u8, &K.raw_stream};
    for (int i = 0; i < 6; ++i) {
        PyObject* old = *to[i];
        *to[i] = Py_NewRef(a[i]);
        Py_XDECREF(old);
    }
    Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(setup),      FAST(qk_norm_rope), FAST(qk_norm_rope_bwd), FAST(qk_norm_rope_append),
                         FAST(paged_attn), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_calls", "Marshalling of the attention sublayer's calls.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_calls() {
    struct { PyObject** to; const char* name; } names[] = {
        {&N.dtype, "dtype"}, {&N.is_cuda, "is_cuda"}, {&N.shape, "shape"}, {&N.stride, "stride"},
        {&N.data_ptr, "data_ptr"}, {&N.numel, "numel"}, {&N.is_contiguous, "is_contiguous"}, {&N.device, "device"},
        {&N.get_device, "get_device"}};
    for (auto& e : names)
        if ((*e.to = PyUnicode_InternFromString(e.name)) == nullptr) return nullptr;
    return PyModule_Create(&module);
}
