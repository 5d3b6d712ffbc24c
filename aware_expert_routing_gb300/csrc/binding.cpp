// binding.cpp -- the Python calls that are made several times a token
// (moe_kv_append and moe_tree_attention with their other forms, moe_kv_read_q8,
// moe_route_scores) as one C function each:
// a small call runs for 4 to 8 us on the GPU, and checking and passing its
// tensors one attribute at a time from Python takes longer than that.
//
// Each function checks the tensors (ValueError), fills the C ABI's structs and
// returns the call's moe_status; the package raises MoeError for it.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <string>

#include "../../include/moe.h"

namespace {

struct Bad {};   // a Python exception has been set

[[noreturn]] void refuse(const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    PyErr_SetString(PyExc_ValueError, buf);
    throw Bad{};
}

const char* type_name(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        default: return "its type";
    }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
    return THPVariable_Unpack(o);
}

// The current device, of which a call's tensors have to be: the library launches there.
// (A default stream does not say which device is meant.)  -1: not looked up in this call.
thread_local int g_device = -1;

void check_device(int device, const char* name) {
    if (g_device < 0) g_device = c10::cuda::current_device();
    if (device != g_device) refuse("%s is on cuda:%d, the current device is cuda:%d", name, device, g_device);
}

// A contiguous CUDA tensor of a type; null for None where that is allowed.
const at::Tensor* dense(PyObject* o, at::ScalarType type, const char* name, bool none_ok = false) {
    if (o == Py_None) {
        if (none_ok) return nullptr;
        refuse("%s is required", name);
    }
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda() || t.scalar_type() != type || !t.is_contiguous())
        refuse("%s must be a contiguous CUDA tensor of %s", name, type_name(type));
    check_device(t.device().index(), name);
    return &t;
}

// A CUDA tensor [T][heads][D] whose heads are dense inside.
const at::Tensor& rows(PyObject* o, at::ScalarType type, int64_t T, int64_t heads, int64_t D, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda() || t.scalar_type() != type || t.dim() != 3 || t.size(0) != T || t.size(1) != heads || t.size(2) != D)
        refuse("%s must be a CUDA tensor (%lld, %lld, %lld) of %s", name, (long long)T, (long long)heads, (long long)D,
               type_name(type));
    if (t.stride(2) != 1) refuse("%s: the components of a head must be adjacent", name);
    check_device(t.device().index(), name);
    return t;
}

// The distance along a dimension; one of size 1 has none (its stride may be any number).
int64_t distance(const at::Tensor& t, int64_t dim) { return t.size(dim) > 1 ? t.stride(dim) : 0; }

const void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

// None: the tensor's device's current stream; else a torch.cuda.Stream.
moe_stream_t stream_of(PyObject* o, const at::Tensor& on) {
    if (o == Py_None) return reinterpret_cast<moe_stream_t>(c10::cuda::getCurrentCUDAStream(on.device().index()).stream());
    PyObject* s = PyObject_GetAttrString(o, "cuda_stream");
    if (!s) throw Bad{};
    void* p = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    if (PyErr_Occurred()) throw Bad{};
    return static_cast<moe_stream_t>(p);
}

int32_t narrow(int64_t x, const char* name) {
    if (x < INT32_MIN || x > INT32_MAX) refuse("%s=%lld does not fit 32 bits", name, (long long)x);
    return (int32_t)x;
}

int32_t int_field(PyObject* o, PyObject* name) {
    PyObject* v = PyObject_GetAttr(o, name);
    if (!v) throw Bad{};
    const long long x = PyLong_AsLongLong(v);   // bools are integers too
    Py_DECREF(v);
    if (x == -1 && PyErr_Occurred()) throw Bad{};
    return narrow(x, "a parameter");
}

float float_field(PyObject* o, PyObject* name) {
    PyObject* v = PyObject_GetAttr(o, name);
    if (!v) throw Bad{};
    const double x = PyFloat_AsDouble(v);
    Py_DECREF(v);
    if (x == -1.0 && PyErr_Occurred()) throw Bad{};
    return (float)x;
}

template <typename F>
PyObject* guarded(PyObject* const* args, Py_ssize_t n, Py_ssize_t want, F&& f) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        return nullptr;
    }
    g_device = -1;
    try {
        return PyLong_FromLong((long)f(args));
    } catch (const Bad&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// A KvCache's or KvCacheQ8's struct: what the C ABI reads, and the tensors' device.
template <typename T> struct OnDevice {
    T cache;
    int32_t device;
};

// What the calls read of a cache, in its type or in 8 bits.
struct Cache {
    const moe_kv_cache* plain = nullptr;
    const moe_kv_cache_q8* q8 = nullptr;
    int32_t kv_heads, head_dim, n_requests, device;
    at::ScalarType type;   // of the tensors that are not in the cache
};

Cache cache_of(PyObject* o, bool q8) {
    const void* p = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw Bad{};
    Cache c;
    auto fill = [&](const auto* on) {
        const auto* x = &on->cache;
        c.kv_heads = x->kv_heads;
        c.head_dim = x->head_dim;
        c.n_requests = x->n_requests;
        c.device = on->device;
        c.type = x->dtype == MOE_DTYPE_BF16 ? at::kBFloat16 : at::kFloat;
        return x;
    };
    if (q8) c.q8 = fill(static_cast<const OnDevice<moe_kv_cache_q8>*>(p));
    else c.plain = fill(static_cast<const OnDevice<moe_kv_cache>*>(p));
    return c;
}

// A HeadNorm's struct: what the C ABI reads, and the shapes that it was made for.
struct Norm {
    moe_head_norm norm;
    int32_t head_dim, dtype;
    int32_t q_heads, k_heads;   // with per_head; 0: no weights
    int32_t device;
};

enum AppendKind { kAppend, kAppendNorm, kAppendQ8 };

// q, k, v, rope, positions, slots, [norm,] cache, q_out, workspace, interleaved, stream
template <AppendKind kKind>
PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t n) {
    constexpr int kShift = kKind == kAppend ? 0 : 1;
    return guarded(args, n, 11 + kShift, [](PyObject* const* x) {
        PyObject* const* a = x + kShift;   // from the cache on
        const Cache c = cache_of(a[6], kKind == kAppendQ8);
        const at::ScalarType dt = c.type;
        const int64_t D = c.head_dim, K = c.kv_heads;
        const at::Tensor& k0 = tensor(x[1], "k");
        const int64_t T = k0.dim() == 3 ? k0.size(0) : -1;
        const at::Tensor &k = rows(x[1], dt, T, K, D, "k"), &v = rows(x[2], dt, T, K, D, "v");
        moe_append_params p{};
        const at::Tensor *q = nullptr, *out = nullptr;
        if ((x[0] == Py_None) != (a[7] == Py_None)) refuse("q and q_out must both be given, or neither");
        if (x[0] != Py_None) {
            const at::Tensor& q0 = tensor(x[0], "q");
            const int64_t heads = q0.dim() == 3 ? q0.size(1) : -1;
            q = &rows(x[0], dt, T, heads, D, "q");
            out = &rows(a[7], dt, T, heads, D, "q_out");
            p.heads = narrow(heads, "heads");
            p.q_tok = distance(*q, 0);
            p.q_head = distance(*q, 1);
            p.out_tok = distance(*out, 0);
            p.out_head = distance(*out, 1);
        }
        const at::Tensor *rope = dense(x[3], at::kFloat, "rope", true), *pos = nullptr;
        if (rope) {
            if (rope->dim() != 2) refuse("rope must be [n_pos][rot]");
            p.n_pos = narrow(rope->size(0), "n_pos");
            p.rot = narrow(rope->size(1), "rot");
            pos = dense(x[4], at::kInt, "positions");
            if (pos->numel() != T) refuse("positions must hold %lld values", (long long)T);
        }
        const at::Tensor* slots = dense(x[5], at::kLong, "slots");
        if (slots->numel() != T) refuse("slots must hold %lld values", (long long)T);
        const at::Tensor* ws = dense(a[8], at::kByte, "workspace");
        check_device(c.device, "cache");
        p.T = narrow(T, "T");
        const int inter = PyObject_IsTrue(a[9]);
        if (inter < 0) throw Bad{};
        p.interleaved = inter;
        p.k_tok = distance(k, 0);
        p.k_head = distance(k, 1);
        p.v_tok = distance(v, 0);
        p.v_head = distance(v, 1);
        const moe_head_norm* norm = nullptr;
        if (kKind == kAppendNorm && x[6] == Py_None) refuse("norm is required");
        if (kKind != kAppend && x[6] != Py_None) {
            const void* at = PyLong_AsVoidPtr(x[6]);
            if (PyErr_Occurred()) throw Bad{};
            const Norm* w = static_cast<const Norm*>(at);
            if (w->norm.q_weight || w->norm.k_weight) {
                check_device(w->device, "norm");
                if (w->head_dim != D || w->dtype != (dt == at::kBFloat16 ? MOE_DTYPE_BF16 : MOE_DTYPE_F32))
                    refuse("the norm's weights must hold %lld values of %s a head", (long long)D, type_name(dt));
                if (w->norm.per_head && ((w->norm.q_weight && q && w->q_heads != p.heads) || (w->norm.k_weight && w->k_heads != K)))
                    refuse("the norm's weights are for %d and %d heads", w->q_heads, w->k_heads);
            }
            norm = &w->norm;
        }
        const void *qp = ptr(q), *kp = k.data_ptr(), *vp = v.data_ptr();
        const float* rp = static_cast<const float*>(ptr(rope));
        const int32_t* pp = static_cast<const int32_t*>(ptr(pos));
        const int64_t* sp = static_cast<const int64_t*>(ptr(slots));
        void* op = const_cast<void*>(ptr(out));
        const moe_stream_t stream = stream_of(a[10], k);
        const size_t bytes = (size_t)ws->numel();
        if constexpr (kKind == kAppend) return moe_kv_append(qp, kp, vp, rp, pp, sp, &p, c.plain, op, ws->data_ptr(), bytes, stream);
        else if constexpr (kKind == kAppendNorm)
            return moe_kv_append_norm(qp, kp, vp, rp, pp, sp, &p, norm, c.plain, op, ws->data_ptr(), bytes, stream);
        else return moe_kv_append_q8(qp, kp, vp, rp, pp, sp, &p, norm, c.q8, op, ws->data_ptr(), bytes, stream);
    });
}

// slots, cache, k_out, v_out, workspace, stream
PyObject* kv_read_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(a, n, 6, [](PyObject* const* a) {
        const Cache c = cache_of(a[1], true);
        const at::Tensor* slots = dense(a[0], at::kLong, "slots");
        const int64_t T = slots->numel();
        moe_read_params p{};
        p.T = narrow(T, "T");
        const at::Tensor *k = nullptr, *v = nullptr;
        if (a[2] == Py_None && a[3] == Py_None) refuse("k_out or v_out is required");
        if (a[2] != Py_None) {
            k = &rows(a[2], c.type, T, c.kv_heads, c.head_dim, "k_out");
            p.k_tok = distance(*k, 0);
            p.k_head = distance(*k, 1);
        }
        if (a[3] != Py_None) {
            v = &rows(a[3], c.type, T, c.kv_heads, c.head_dim, "v_out");
            p.v_tok = distance(*v, 0);
            p.v_head = distance(*v, 1);
        }
        const at::Tensor* ws = dense(a[4], at::kByte, "workspace");
        check_device(c.device, "cache");
        return moe_kv_read_q8(static_cast<const int64_t*>(ptr(slots)), &p, c.q8, const_cast<void*>(ptr(k)),
                              const_cast<void*>(ptr(v)), ws->data_ptr(), (size_t)ws->numel(), stream_of(a[5], *slots));
    });
}

// q, q_offsets, ctx_len, mask, cache, out, lse, workspace, scale, stream
template <bool kQ8>
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(a, n, 10, [](PyObject* const* a) {
        const Cache c = cache_of(a[4], kQ8);
        const at::ScalarType dt = c.type;
        const at::Tensor& q0 = tensor(a[0], "q");
        if (q0.dim() != 3) refuse("q must be [T][heads][head_dim]");
        const int64_t T = q0.size(0), H = q0.size(1), R = c.n_requests;
        const at::Tensor& q = rows(a[0], dt, T, H, c.head_dim, "q");
        const at::Tensor* out = dense(a[5], dt, "out");
        if (out->sizes() != q.sizes()) refuse("out must have q's shape");
        const at::Tensor* lse = dense(a[6], at::kFloat, "lse", true);
        if (lse && (lse->dim() != 2 || lse->size(0) != T || lse->size(1) != H))
            refuse("lse must be [%lld][%lld]", (long long)T, (long long)H);
        const at::Tensor *off = dense(a[1], at::kInt, "q_offsets"), *ctx = dense(a[2], at::kInt, "ctx_len");
        if (off->numel() != R + 1 || ctx->numel() != R)
            refuse("q_offsets must hold %lld values and ctx_len %lld", (long long)R + 1, (long long)R);
        moe_attention_params p{};
        const at::Tensor* mask = dense(a[3], at::kInt, "mask", true);
        if (mask) {
            // (an empty tensor's pointer is null, which the C ABI takes for no mask)
            if (mask->dim() != 2 || mask->size(0) != T || (T > 0 && mask->size(1) < 1))
                refuse("mask must be [%lld][words], of one word at least", (long long)T);
            p.mask_words = narrow(mask->size(1), "mask_words");
        }
        const at::Tensor* ws = dense(a[7], at::kByte, "workspace");
        check_device(c.device, "cache");
        p.T = narrow(T, "T");
        p.heads = narrow(H, "heads");
        if (a[8] == Py_None) {
            p.scale = (float)(1.0 / std::sqrt((double)c.head_dim));
        } else {
            p.scale = (float)PyFloat_AsDouble(a[8]);
            if (PyErr_Occurred()) throw Bad{};
        }
        p.q_tok = distance(q, 0);
        p.q_head = distance(q, 1);
        const int32_t *po = static_cast<const int32_t*>(ptr(off)), *pc = static_cast<const int32_t*>(ptr(ctx));
        const uint32_t* pm = static_cast<const uint32_t*>(ptr(mask));
        float* pl = static_cast<float*>(const_cast<void*>(ptr(lse)));
        const moe_stream_t stream = stream_of(a[9], q);
        const size_t bytes = (size_t)ws->numel();
        if constexpr (kQ8) return moe_tree_attention_q8(q.data_ptr(), po, pc, pm, &p, c.q8, out->data_ptr(), pl, ws->data_ptr(), bytes, stream);
        else return moe_tree_attention(q.data_ptr(), po, pc, pm, &p, c.plain, out->data_ptr(), pl, ws->data_ptr(), bytes, stream);
    });
}

PyObject* g_names[32];
enum Name { kB, kBValid, kD, kN, kK, kMode, kK0, kP, kMaxP, kKmax, kDtype, kScore, kNGroup, kTopkGroup, kGroupTop,
            kRenormalise, kScale, kExpertIdx, kWeights, kT, kActive, kCounts, kOffsets, kPerm, kNBase, kNames };
const char* const kText[kNames] = {"B", "B_valid", "d", "N", "k", "mode", "k0", "p", "maxP", "kmax", "dtype", "score", "n_group",
                                   "topk_group", "group_top", "renormalise", "scale", "expert_idx", "weights", "T", "active",
                                   "counts", "offsets", "perm", "n_base"};

// scores, select_bias, params, select, routing, workspace, stream
PyObject* route_scores(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(a, n, 7, [](PyObject* const* a) {
        moe_route_params p{};
        PyObject* P = a[2];
        p.B = int_field(P, g_names[kB]);
        p.B_valid = int_field(P, g_names[kBValid]);
        p.d = int_field(P, g_names[kD]);
        p.N = int_field(P, g_names[kN]);
        p.k = int_field(P, g_names[kK]);
        p.mode = int_field(P, g_names[kMode]);
        p.k0 = int_field(P, g_names[kK0]);
        p.p = float_field(P, g_names[kP]);
        p.maxP = int_field(P, g_names[kMaxP]);
        p.kmax = int_field(P, g_names[kKmax]);
        p.dtype = int_field(P, g_names[kDtype]);
        if (p.mode != MOE_MODE_OEA) p.k0 = p.k;
        moe_select_params s{};
        s.score = int_field(a[3], g_names[kScore]);
        s.n_group = int_field(a[3], g_names[kNGroup]);
        s.topk_group = int_field(a[3], g_names[kTopkGroup]);
        s.group_top = int_field(a[3], g_names[kGroupTop]);
        s.renormalise = int_field(a[3], g_names[kRenormalise]);
        s.scale = float_field(a[3], g_names[kScale]);
        const at::Tensor* x = dense(a[0], at::kFloat, "scores");
        if (x->dim() != 2 || x->size(0) != p.B || x->size(1) != p.N) refuse("scores must be [%d][%d]", p.B, p.N);
        const at::Tensor* bias = dense(a[1], at::kFloat, "select_bias", true);
        if (bias && bias->numel() != p.N) refuse("select_bias must hold %d values", p.N);
        const at::Tensor* ws = dense(a[5], at::kByte, "workspace");
        // The routing's buffers are its own; it holds them while this call runs.
        // One made for a smaller batch or fewer experts is refused.
        auto buffer = [&](Name name, at::ScalarType type, int64_t least) -> void* {
            PyObject* o = PyObject_GetAttr(a[4], g_names[name]);
            if (!o) throw Bad{};
            struct Held {
                PyObject* o;
                ~Held() { Py_DECREF(o); }
            } held{o};
            const at::Tensor* t = dense(o, type, kText[name], name == kNBase);
            if (t && t->numel() < least) refuse("the routing's %s must hold %lld values", kText[name], (long long)least);
            return t ? t->data_ptr() : nullptr;
        };
        const int64_t pairs = (int64_t)p.B * p.k, N = p.N;   // (top-k mode: k slots a token)
        moe_routing r{};
        r.expert_idx = static_cast<int32_t*>(buffer(kExpertIdx, at::kInt, pairs));
        r.weights = static_cast<float*>(buffer(kWeights, at::kFloat, pairs));
        r.T = static_cast<int32_t*>(buffer(kT, at::kInt, 1));
        r.active = static_cast<int32_t*>(buffer(kActive, at::kInt, N));
        r.counts = static_cast<int32_t*>(buffer(kCounts, at::kInt, N));
        r.offsets = static_cast<int32_t*>(buffer(kOffsets, at::kInt, N + 1));
        r.perm = static_cast<int32_t*>(buffer(kPerm, at::kInt, pairs));
        r.n_base = static_cast<int32_t*>(buffer(kNBase, at::kInt, p.B));
        return moe_route_scores(static_cast<const float*>(ptr(x)), static_cast<const float*>(ptr(bias)), &p, &s, &r,
                                ws->data_ptr(), (size_t)ws->numel(), stream_of(a[6], *x));
    });
}

#define MOE_METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {
    MOE_METHOD("kv_append", append<kAppend>),
    MOE_METHOD("kv_append_norm", append<kAppendNorm>),
    MOE_METHOD("kv_append_q8", append<kAppendQ8>),
    MOE_METHOD("kv_read_q8", kv_read_q8),
    MOE_METHOD("tree_attention", tree_attention<false>),
    MOE_METHOD("tree_attention_q8", tree_attention<true>),
    MOE_METHOD("route_scores", route_scores),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    for (int i = 0; i < kNames; ++i)
        if (!(g_names[i] = PyUnicode_InternFromString(kText[i]))) return nullptr;
    return PyModule_Create(&kModule);
}
