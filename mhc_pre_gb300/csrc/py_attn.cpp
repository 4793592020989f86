// py_attn.cpp -- the Python side of the attention sublayer's entry points:
// argument checks and marshalling, as a CPython module (_attn_calls).
//
// These calls are made for every layer of a decoding step, where the host's
// time is the call's time.  On the host of a GB300 qk_norm_rope takes 6.5 us
// here, about 4 of them the launch and 2 its two outputs, and its backward
// (two launches, five buffers) 12.7 us.  Reading the tensors through their
// Python attributes instead of torch's C++ classes costs 3 to 8 us more, the
// same checks in Python with a ctypes call 17 to 28 us.
//
// Every function returns (status, outputs...) with the library's status, or
// raises TypeError / ValueError for what the library could not see.  Its first
// argument allocates the outputs (None: torch's empty).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <math.h>
#include <stdint.h>
#include <string.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mhc.h"

namespace {

using at::ScalarType;

// The library's entry points, handed over by bind().  The module is not linked
// to the library: whichever one the package has loaded is the one that both its
// ctypes calls and these calls run, wherever the package lies.
struct Library {
    decltype(&mhc_qk_norm_rope) qk_norm_rope;
    decltype(&mhc_qk_norm_rope_bwd) qk_norm_rope_bwd;
    decltype(&mhc_qk_norm_rope_bwd_workspace_bytes) qk_norm_rope_bwd_workspace_bytes;
    decltype(&mhc_qk_norm_rope_append) qk_norm_rope_append;
    decltype(&mhc_paged_attn) paged_attn;
    decltype(&mhc_paged_attn_workspace_bytes) paged_attn_workspace_bytes;
};
Library lib = {};
constexpr int ENTRIES = sizeof(Library) / sizeof(void*);

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

const char* type_name(ScalarType t) {
    switch (t) {
        case ScalarType::BFloat16: return "torch.bfloat16";
        case ScalarType::Float: return "torch.float32";
        case ScalarType::Int: return "torch.int32";
        case ScalarType::Long: return "torch.int64";
        case ScalarType::Byte: return "torch.uint8";
        default: return "another type";
    }
}

// A borrowed tensor; raises TypeError for anything else.
bool tensor_of(PyObject* o, const char* name, const at::Tensor** out) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor, got %R", name, reinterpret_cast<PyObject*>(Py_TYPE(o)));
        return false;
    }
    *out = &THPVariable_Unpack(o);
    return true;
}
bool shape_of(PyObject* o, int64_t n, int64_t* out, const char* name) {
    const at::Tensor* t;
    if (!tensor_of(o, name, &t)) return false;
    if (t->dim() != n) {
        PyErr_Format(PyExc_ValueError, "%s must have %lld dimensions", name, static_cast<long long>(n));
        return false;
    }
    for (int64_t i = 0; i < n; ++i) out[i] = t->size(i);
    return true;
}

bool check_dtype(PyObject* o, const at::Tensor& t, ScalarType want, const char* name) {
    if (t.scalar_type() == want) return true;
    Ref have(PyObject_GetAttrString(o, "dtype"));
    if (have) PyErr_Format(PyExc_TypeError, "%s must be %s, got %S", name, type_name(want), have.get());
    return false;
}
bool check_cuda(const at::Tensor& t) {
    if (t.is_cuda()) return true;
    PyErr_SetString(PyExc_ValueError, "the mHC library takes CUDA tensors only");
    return false;
}

// The activations' type and its code.
bool activations(PyObject* o, ScalarType* dtype, mhc_dtype* code) {
    const at::Tensor* t;
    if (!tensor_of(o, "the activations", &t)) return false;
    *dtype = t->scalar_type();
    if (*dtype == ScalarType::BFloat16) *code = MHC_BF16;
    else if (*dtype == ScalarType::Float) *code = MHC_F32;
    else {
        Ref have(PyObject_GetAttrString(o, "dtype"));
        if (have) PyErr_Format(PyExc_TypeError, "activations must be bfloat16 or float32, got %S", have.get());
        return false;
    }
    return true;
}

// A tensor of heads [T, H, Dh]: address and distance of its tokens, which may
// be apart (a part of a packed projection); a token's heads are not.
struct Heads {
    void* p;
    int64_t stride;
};
bool heads_of(PyObject* o, const char* name, ScalarType dtype, const int64_t (&shape)[3], Heads* out) {
    const at::Tensor* t;
    if (!tensor_of(o, name, &t) || !check_dtype(o, *t, dtype, name) || !check_cuda(*t)) return false;
    if ((t->stride(2) != 1 && shape[2] > 1) || (t->stride(1) != shape[2] && shape[1] > 1)) {
        PyErr_Format(PyExc_ValueError, "%s: the heads of a token must lie one after the other", name);
        return false;
    }
    out->stride = shape[0] > 1 ? t->stride(0) : shape[1] * shape[2];
    out->p = t->data_ptr();
    return true;
}

// A dense tensor of n entries.
bool flat_of(PyObject* o, const char* name, ScalarType dtype, int64_t n, void** out) {
    const at::Tensor* t;
    if (!tensor_of(o, name, &t) || !check_dtype(o, *t, dtype, name)) return false;
    if (t->numel() != n) {
        PyErr_Format(PyExc_ValueError, "%s must have %lld entries, got %lld", name, static_cast<long long>(n),
                     static_cast<long long>(t->numel()));
        return false;
    }
    if (!check_cuda(*t)) return false;
    if (!t->is_contiguous()) {
        PyErr_SetString(PyExc_ValueError, "the mHC library takes contiguous tensors only");
        return false;
    }
    *out = t->data_ptr();
    return true;
}

// A cache [pages, page_size, Hk, Dh] in any memory order that keeps a head's
// values together.
struct Cache {
    void* p;
    int64_t page, slot, head;
};
bool cache_of(PyObject* o, const char* name, ScalarType dtype, const int64_t (&shape)[4], Cache* out) {
    const at::Tensor* t;
    int64_t have[4];
    if (!tensor_of(o, name, &t) || !check_dtype(o, *t, dtype, name) || !check_cuda(*t) || !shape_of(o, 4, have, name))
        return false;
    for (int i = 0; i < 4; ++i)
        if (have[i] != shape[i]) {
            PyErr_Format(PyExc_ValueError, "%s must be [%lld, %lld, %lld, %lld]", name,
                         static_cast<long long>(shape[0]), static_cast<long long>(shape[1]),
                         static_cast<long long>(shape[2]), static_cast<long long>(shape[3]));
            return false;
        }
    if (t->stride(3) != 1 && shape[3] > 1) {
        PyErr_Format(PyExc_ValueError, "%s: the values of a head must lie one after the other", name);
        return false;
    }
    out->page = shape[0] > 1 ? t->stride(0) : shape[1] * shape[2] * shape[3];
    out->slot = shape[1] > 1 ? t->stride(1) : shape[2] * shape[3];
    out->head = shape[2] > 1 ? t->stride(2) : shape[3];
    out->p = t->data_ptr();
    return true;
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
    return flat_of(positions, "positions", ScalarType::Int, T, &out->positions) &&
           flat_of(cos_sin, "cos_sin", ScalarType::Float, s[0] * s[1], &out->cos_sin);
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

cudaStream_t stream_of(PyObject* o) { return c10::cuda::getCurrentCUDAStream(THPVariable_Unpack(o).get_device()).stream(); }

// A new tensor on the device of `like`, and its address.  `empty`: a callable
// of (shape, dtype, device), or None.
PyObject* make(PyObject* empty, ScalarType dtype, PyObject* like, int n, const int64_t* shape, void** p) {
    const at::Tensor& l = THPVariable_Unpack(like);
    if (empty == Py_None) {
        const at::Tensor t = at::empty(c10::IntArrayRef(shape, n), l.options().dtype(dtype));
        *p = t.data_ptr();
        return THPVariable_Wrap(t);
    }
    Ref dims(PyTuple_New(n)), torch(PyImport_ImportModule("torch")), device(PyObject_GetAttrString(like, "device"));
    if (!dims || !torch || !device) return nullptr;
    for (int i = 0; i < n; ++i) {
        PyObject* v = PyLong_FromLongLong(shape[i]);
        if (v == nullptr) return nullptr;
        PyTuple_SET_ITEM(dims.get(), i, v);
    }
    Ref kind(PyObject_GetAttrString(torch.get(), type_name(dtype) + 6));   // past "torch."
    if (!kind) return nullptr;
    PyObject* args[3] = {dims.get(), kind.get(), device.get()};
    Ref t(PyObject_Vectorcall(empty, args, 3, nullptr));
    const at::Tensor* made;
    if (!t || !tensor_of(t.get(), "a new tensor", &made)) return nullptr;
    *p = made->data_ptr();
    return t.release();
}
PyObject* make_bytes(PyObject* empty, PyObject* like, size_t bytes, void** p) {
    const int64_t n = bytes > 0 ? static_cast<int64_t>(bytes) : 16;
    return make(empty, ScalarType::Byte, like, 1, &n, p);
}

bool arguments(Py_ssize_t have, Py_ssize_t want) {
    if (lib.qk_norm_rope == nullptr) {
        PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
        return false;
    }
    if (have == want) return true;
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return false;
}
int clip(int64_t v) { return v > INT32_MAX ? INT32_MAX : static_cast<int>(v); }

// --------------------------------------------------------------- functions ---

// (addresses of the entry points, in the order of Library) -> None
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != ENTRIES) {
        PyErr_SetString(PyExc_TypeError, "wrong number of entry points");
        return nullptr;
    }
    void* at[ENTRIES];
    for (int i = 0; i < ENTRIES; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i]);
        if (at[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point is missing");
            return nullptr;
        }
    }
    memcpy(&lib, at, sizeof(lib));
    Py_RETURN_NONE;
}

// (empty, q, k, w_q, w_k, positions, cos_sin, eps, flags) -> (status, q_out, k_out)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 9)) return nullptr;
    int64_t sq[3], sk[3];
    ScalarType dt;
    mhc_dtype code;
    void *wq, *wk, *qo, *ko;
    Heads q, k;
    Rope rope;
    float eps;
    int flags;
    if (!same_tokens(a[1], a[2], sq, sk) || !activations(a[1], &dt, &code) ||
        !flat_of(a[3], "w_q", ScalarType::Float, sq[2], &wq) || !flat_of(a[4], "w_k", ScalarType::Float, sq[2], &wk) ||
        !heads_of(a[1], "q", dt, sq, &q) || !heads_of(a[2], "k", dt, sk, &k) ||
        !rope_of(a[5], a[6], sq[0], &rope) || !to_float(a[7], &eps) || !to_int(a[8], &flags))
        return nullptr;
    Ref to(make(a[0], dt, a[1], 3, sq, &qo));
    if (!to) return nullptr;
    Ref tk(make(a[0], dt, a[1], 3, sk, &ko));
    if (!tk) return nullptr;
    const int st = lib.qk_norm_rope(code, q.p, q.stride, k.p, k.stride, static_cast<float*>(wq), static_cast<float*>(wk),
                                    static_cast<int32_t*>(rope.positions), static_cast<float*>(rope.cos_sin),
                                    rope.max_pos, sq[0], clip(sq[1]), clip(sk[1]), clip(sq[2]), rope.rot, flags, eps, qo,
                                    sq[1] * sq[2], ko, sk[1] * sk[2], stream_of(a[1]));
    return Py_BuildValue("iOO", st, to.get(), tk.get());
    END_HANDLE_TH_ERRORS
}

// (empty, g_q, g_k, q, k, w_q, w_k, positions, cos_sin, eps, flags, dq | None, dk | None)
//   -> (status, dq, dk, dw_q, dw_k)
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 13)) return nullptr;
    int64_t sq[3], sk[3];
    ScalarType dt;
    mhc_dtype code;
    void *wq, *wk, *dwq, *dwk, *ws;
    Heads gq, gk, q, k, dq, dk;
    Rope rope;
    float eps;
    int flags;
    if (!same_tokens(a[3], a[4], sq, sk) || !activations(a[3], &dt, &code) ||
        !same_shape(a[1], sq, "q, k and their gradients must have the same shapes") ||
        !same_shape(a[2], sk, "q, k and their gradients must have the same shapes") ||
        !flat_of(a[5], "w_q", ScalarType::Float, sq[2], &wq) || !flat_of(a[6], "w_k", ScalarType::Float, sq[2], &wk) ||
        !heads_of(a[1], "g_q", dt, sq, &gq) || !heads_of(a[2], "g_k", dt, sk, &gk) ||
        !heads_of(a[3], "q", dt, sq, &q) || !heads_of(a[4], "k", dt, sk, &k) ||
        !rope_of(a[7], a[8], sq[0], &rope) || !to_float(a[9], &eps) || !to_int(a[10], &flags))
        return nullptr;
    Ref tq, tk;
    if (a[11] == Py_None) {
        tq.reset(make(a[0], dt, a[3], 3, sq, &dq.p));
        if (!tq) return nullptr;
        dq.stride = sq[1] * sq[2];
    } else {
        if (!same_shape(a[11], sq, "dq and dk must have the shapes of q and k") || !heads_of(a[11], "dq", dt, sq, &dq))
            return nullptr;
        tq.reset(Py_NewRef(a[11]));
    }
    if (a[12] == Py_None) {
        tk.reset(make(a[0], dt, a[3], 3, sk, &dk.p));
        if (!tk) return nullptr;
        dk.stride = sk[1] * sk[2];
    } else {
        if (!same_shape(a[12], sk, "dq and dk must have the shapes of q and k") || !heads_of(a[12], "dk", dt, sk, &dk))
            return nullptr;
        tk.reset(Py_NewRef(a[12]));
    }
    Ref twq(make(a[0], ScalarType::Float, a[3], 1, sq + 2, &dwq));
    if (!twq) return nullptr;
    Ref twk(make(a[0], ScalarType::Float, a[3], 1, sq + 2, &dwk));
    if (!twk) return nullptr;
    const size_t need = lib.qk_norm_rope_bwd_workspace_bytes(sq[0], clip(sq[2]));
    Ref tws(make_bytes(a[0], a[3], need, &ws));
    if (!tws) return nullptr;
    const int st = lib.qk_norm_rope_bwd(
        code, gq.p, gq.stride, gk.p, gk.stride, q.p, q.stride, k.p, k.stride, static_cast<float*>(wq),
        static_cast<float*>(wk), static_cast<int32_t*>(rope.positions), static_cast<float*>(rope.cos_sin), rope.max_pos,
        sq[0], clip(sq[1]), clip(sk[1]), clip(sq[2]), rope.rot, flags, eps, dq.p, dq.stride, dk.p, dk.stride,
        static_cast<float*>(dwq), static_cast<float*>(dwk), ws, need, stream_of(a[3]));
    return Py_BuildValue("iOOOO", st, tq.get(), tk.get(), twq.get(), twk.get());
    END_HANDLE_TH_ERRORS
}

// (empty, q, k, v, w_q, w_k, k_cache, v_cache, slots, positions, cos_sin, eps, flags) -> (status, q_out)
PyObject* qk_norm_rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 13)) return nullptr;
    int64_t sq[3], sk[3], sc[4];
    ScalarType dt;
    mhc_dtype code;
    void *wq, *wk, *slots, *qo;
    Heads q, k, v;
    Cache kc, vc;
    Rope rope;
    float eps;
    int flags;
    if (!same_tokens(a[1], a[2], sq, sk) || !activations(a[1], &dt, &code) ||
        !same_shape(a[3], sk, "k and v must have the same shape") || !shape_of(a[6], 4, sc, "k_cache"))
        return nullptr;
    if (sc[2] != sk[1] || sc[3] != sk[2]) {
        PyErr_Format(PyExc_ValueError, "k_cache must be [pages, page_size, %lld, %lld]", static_cast<long long>(sk[1]),
                     static_cast<long long>(sk[2]));
        return nullptr;
    }
    if (!flat_of(a[4], "w_q", ScalarType::Float, sq[2], &wq) || !flat_of(a[5], "w_k", ScalarType::Float, sq[2], &wk) ||
        !heads_of(a[1], "q", dt, sq, &q) || !heads_of(a[2], "k", dt, sk, &k) || !heads_of(a[3], "v", dt, sk, &v) ||
        !cache_of(a[6], "k_cache", dt, sc, &kc) || !cache_of(a[7], "v_cache", dt, sc, &vc) ||
        !flat_of(a[8], "slots", ScalarType::Long, sq[0], &slots) || !rope_of(a[9], a[10], sq[0], &rope) ||
        !to_float(a[11], &eps) || !to_int(a[12], &flags))
        return nullptr;
    Ref to(make(a[0], dt, a[1], 3, sq, &qo));
    if (!to) return nullptr;
    const int st = lib.qk_norm_rope_append(
        code, q.p, q.stride, k.p, k.stride, v.p, v.stride, static_cast<float*>(wq), static_cast<float*>(wk),
        static_cast<int32_t*>(rope.positions), static_cast<float*>(rope.cos_sin), rope.max_pos,
        static_cast<int64_t*>(slots), sq[0], clip(sq[1]), clip(sk[1]), clip(sq[2]), rope.rot, flags, eps, qo,
        sq[1] * sq[2], kc.p, kc.page, kc.slot, kc.head, vc.p, vc.page, vc.slot, vc.head, sc[0], clip(sc[1]), stream_of(a[1]));
    return Py_BuildValue("iO", st, to.get());
    END_HANDLE_TH_ERRORS
}

// (empty, q, k_cache, v_cache, page_table, cu_q, kv_lens, max_q, max_kv, scale, window, softcap, workspace, out)
//   -> (status, o, lse); None: the lengths where there is a planned workspace, bounds and scale from the shapes, a
//   new workspace, a new output
PyObject* paged_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 14)) return nullptr;
    int64_t sq[3], sc[4], stab[2], max_q, max_kv;
    const at::Tensor* t;
    ScalarType dt;
    mhc_dtype code;
    void *table, *cu = nullptr, *kv = nullptr, *o, *lse, *ws;
    Heads q;
    Cache kc, vc;
    float scale, softcap;
    int window;
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
    if (!tensor_of(a[4], "page_table", &t) || !check_dtype(a[4], *t, ScalarType::Int, "page_table") || !check_cuda(*t))
        return nullptr;
    if (width * page < max_kv) {
        PyErr_Format(PyExc_ValueError, "page_table holds %lld tokens a sequence, max_kv is %lld",
                     static_cast<long long>(width * page), static_cast<long long>(max_kv));
        return nullptr;
    }
    if (t->stride(1) != 1 && width > 1) {
        PyErr_SetString(PyExc_ValueError, "page_table: the pages of a sequence must lie one after the other");
        return nullptr;
    }
    if (a[12] == Py_None && (!flat_of(a[5], "cu_q", ScalarType::Int, B + 1, &cu) || !flat_of(a[6], "kv_lens", ScalarType::Int, B, &kv)))
        return nullptr;
    table = t->data_ptr();
    if (!heads_of(a[1], "q", dt, sq, &q) || !cache_of(a[2], "k_cache", dt, sc, &kc) ||
        !cache_of(a[3], "v_cache", dt, sc, &vc))
        return nullptr;
    Ref tw;
    int64_t ws_bytes;
    if (a[12] == Py_None) {
        ws_bytes = static_cast<int64_t>(lib.paged_attn_workspace_bytes(code, T, clip(B), clip(sq[1]), clip(sc[2]),
                                                                       clip(sq[2]), clip(page), max_q));
        tw.reset(make_bytes(a[0], a[1], static_cast<size_t>(ws_bytes), &ws));
        if (!tw) return nullptr;
    } else {
        const at::Tensor* w;
        if (!tensor_of(a[12], "the plan", &w)) return nullptr;
        ws_bytes = static_cast<int64_t>(w->nbytes());
        ws = w->data_ptr();
    }
    Ref to;
    if (a[13] == Py_None) {
        to.reset(make(a[0], dt, a[1], 3, sq, &o));
        if (!to) return nullptr;
    } else {
        if (!same_shape(a[13], sq, "out must have the shape of q") ||
            !flat_of(a[13], "out", dt, sq[0] * sq[1] * sq[2], &o))
            return nullptr;
        to.reset(Py_NewRef(a[13]));
    }
    Ref tl(make(a[0], ScalarType::Float, a[1], 2, sq, &lse));
    if (!tl) return nullptr;
    const int st = lib.paged_attn(code, q.p, q.stride, kc.p, kc.page, kc.slot, kc.head, vc.p, vc.page, vc.slot, vc.head,
                                  sc[0], clip(page), static_cast<int32_t*>(table), B > 1 ? t->stride(0) : width,
                                  static_cast<int32_t*>(cu), static_cast<int32_t*>(kv), T, clip(B), clip(sq[1]),
                                  clip(sc[2]), clip(sq[2]), max_q, max_kv, window, scale, softcap, o,
                                  static_cast<float*>(lse), ws, static_cast<size_t>(ws_bytes), stream_of(a[1]));
    return Py_BuildValue("iOO", st, to.get(), tl.get());
    END_HANDLE_TH_ERRORS
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(qk_norm_rope), FAST(qk_norm_rope_bwd), FAST(qk_norm_rope_append), FAST(paged_attn),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_calls", "Marshalling of the attention sublayer's calls.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_calls() {
    Ref m(PyModule_Create(&module));
    // the torch and Python that this was compiled for
    if (!m || PyModule_AddStringConstant(m.get(), "made_for", MHC_CALLS_MADE_FOR) < 0) return nullptr;
    return m.release();
}
