// Torch marshalling of the cache, attention and log-probability calls.
//
// These calls run on every layer of every step, and a small one takes the GPU
// two to ten microseconds: checking tensors and converting arguments in Python
// took longer than that (13 us for a cache append against 3.6 us for the C
// call itself).  This module checks the same things natively, allocates the
// outputs and calls the C ABI of libspecverify.so; it holds no arithmetic.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/core/Tensor.h>
#include <ATen/EmptyTensor.h>
#include <c10/core/Allocator.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <map>
#include <mutex>
#include <optional>
#include <sstream>
#include <string>
#include <tuple>

#include "spec_verify.h"

namespace {

// A Python exception of the given type; caught at the functions' ends.
struct PyFail {
    PyObject* type;
    std::string text;
};
struct StatusFail {
    spec_status_t status;
    const char* what;
};
struct PyPending {};          // a Python call has set the exception itself

std::string shape_text(c10::IntArrayRef s) {
    std::ostringstream o;
    o << "(";
    for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
    o << ")";
    return o.str();
}

const at::Tensor* tensor_of(PyObject* o, const char* name) {
    if (!THPVariable_Check(o))
        throw PyFail{PyExc_TypeError, std::string(name) + " must be a torch tensor, got " + Py_TYPE(o)->tp_name};
    return &THPVariable_Unpack(o);
}

void on_cuda(const at::Tensor& t, const char* name, int device) {
    if (!t.is_cuda()) throw PyFail{PyExc_ValueError, std::string(name) + " must be a CUDA tensor, got device " + t.device().str()};
    if (device >= 0 && t.get_device() != device)
        throw PyFail{PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", the other arguments on cuda:" + std::to_string(device)};
}

void of_type(const at::Tensor& t, const char* name, at::ScalarType want) {
    if (t.scalar_type() != want)
        throw PyFail{PyExc_TypeError, std::string(name) + " must have dtype " + c10::toString(want) + ", got " + c10::toString(t.scalar_type())};
}

void of_shape(const at::Tensor& t, const char* name, c10::IntArrayRef want) {
    if (t.sizes() != want)
        throw PyFail{PyExc_ValueError, std::string(name) + " must have shape " + shape_text(want) + ", got " + shape_text(t.sizes())};
}

void packed(const at::Tensor& t, const char* name) {
    if (!t.is_contiguous()) throw PyFail{PyExc_ValueError, std::string(name) + " must be contiguous"};
}

// A contiguous tensor of one type and shape; null for None where that is allowed.
template <typename T>
T* plain(PyObject* o, const char* name, at::ScalarType type, c10::IntArrayRef shape, int device, bool nullable = false) {
    if (nullable && o == Py_None) return nullptr;
    const at::Tensor& t = *tensor_of(o, name);
    on_cuda(t, name, device);
    of_type(t, name, type);
    of_shape(t, name, shape);
    packed(t, name);
    return static_cast<T*>(t.data_ptr());
}

int32_t* ints(PyObject* o, const char* name, c10::IntArrayRef shape, int device, bool nullable = false) {
    return plain<int32_t>(o, name, at::kInt, shape, device, nullable);
}

// A bfloat16 [B, N, heads, D] tensor with its heads side by side and its
// tokens one stride apart.
struct Rows {
    void* p = nullptr;
    int64_t B = 0, N = 0, H = 0, stride = 0;
};
Rows rows_of(PyObject* o, const char* name, int64_t D, int device) {
    const at::Tensor& t = *tensor_of(o, name);
    on_cuda(t, name, device);
    of_type(t, name, at::kBFloat16);
    if (t.dim() != 4 || t.size(3) != D)
        throw PyFail{PyExc_ValueError, std::string(name) + " must have shape (B, N, heads, " + std::to_string(D) + "), got " + shape_text(t.sizes())};
    Rows r;
    r.p = t.data_ptr();
    r.B = t.size(0);
    r.N = t.size(1);
    r.H = t.size(2);
    const auto s = t.strides();
    if (s[3] != 1 || (s[2] != D && r.H > 1) || (s[0] != r.N * s[1] && r.B > 1 && r.N > 1))
        throw PyFail{PyExc_ValueError, std::string(name) + ": heads must lie side by side and tokens one stride apart, got strides " + shape_text(s)};
    r.stride = r.N > 1 ? s[1] : r.B > 1 ? s[0] : r.H * D;      // (of one token any stride may stand there)
    return r;
}
void same_rows(const Rows& r, const char* name, int64_t B, int64_t N, int64_t H) {
    if (r.B != B || r.N != N || r.H != H)
        throw PyFail{PyExc_ValueError, std::string(name) + " must hold " + shape_text({B, N, H}) + " rows, got " + shape_text({r.B, r.N, r.H})};
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PyPending{};
    return v;
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PyPending{};
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PyPending{};
    return v != 0;
}

// The cache's structure and the sequences its block table has.
struct Cache {
    const spec_kv_cache_t* c;
    int64_t batch;
    int device;
};
Cache cache_of(PyObject* addr, PyObject* batch, PyObject* device) {
    return {reinterpret_cast<const spec_kv_cache_t*>(static_cast<uintptr_t>(integer(addr))), integer(batch), (int)integer(device)};
}
void fits(const Cache& c, int64_t B) {
    if (B > c.batch)
        throw PyFail{PyExc_ValueError, std::to_string(B) + " sequences, the cache's block table has " + std::to_string(c.batch)};
}

// The stream of a call.  Where one is given, outputs and workspaces are
// allocated under it, so that the allocator reuses their memory in its order.
struct OnStream {
    cudaStream_t h;
    // (in this order: the stream's guard, made second, has to be the first to go)
    std::optional<c10::cuda::CUDAGuard> other;               // the tensors are not the current device's
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    OnStream(PyObject* stream, int device) {
        if (c10::cuda::current_device() != device) other.emplace((c10::DeviceIndex)device);
        if (stream == Py_None) {
            h = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
            return;
        }
        PyObject* v = PyObject_GetAttrString(stream, "cuda_stream");
        if (!v) throw PyPending{};
        const void* p = PyLong_AsVoidPtr(v);
        Py_DECREF(v);
        if (PyErr_Occurred()) throw PyPending{};
        h = static_cast<cudaStream_t>(const_cast<void*>(p));
        guard.emplace(c10::cuda::getStreamFromExternal(h, (c10::DeviceIndex)device));
    }
};

// A new tensor on the current device, which OnStream has made the call's: straight
// from torch's allocator (at::empty's way there takes the host 0.4 us more).
at::Tensor empty(c10::IntArrayRef shape, at::ScalarType type) {
    static c10::Allocator* const from = c10::GetAllocator(c10::kCUDA);
    return at::detail::empty_generic(shape, from, c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt);
}

// A contiguous tensor over a stretch of another's storage, from element `at` of
// its own type on.
at::Tensor stretch(const at::Tensor& whole, c10::IntArrayRef shape, at::ScalarType type, int64_t at) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(),
                                                            c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    t.unsafeGetTensorImpl()->set_storage_offset(at);
    return t;
}

constexpr int64_t kSharedOutput = 1 << 20;     // elements of an output that may share its allocation

// The default workspace of one kind of call on one stream of one device: calls
// on different streams overlap and must not share one.  (Host threads may share a
// stream: a call keeps the interpreter's lock over its launches, so no other's
// come between an attention kernel and the join of its parts.)  Kept for later calls until
// one needs more, and never freed at exit (the CUDA context may be gone by then).
// A captured call gets one of its own, never the kept one: a graph would go on
// writing there after a larger call has given it back, or, replayed on another
// stream, beside a call on this one.  Its memory is the graph's (the allocator
// serves a capture from that graph's pool), its error word is not cleared,
// as nobody can read it.
constexpr size_t kHeadBytes = 256;       // what a call may want zeroed once (the error word)
at::Tensor scratch(int kind, int device, cudaStream_t h, size_t need) {
    using Key = std::tuple<int, int, cudaStream_t>;
    static std::mutex* lock = new std::mutex;
    static auto* kept = new std::map<Key, at::Tensor>;
    const Key key{kind, device, h};
    const size_t n = need < kHeadBytes ? kHeadBytes : need;
    if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None)
        return empty({(int64_t)n}, at::kByte);
    const std::lock_guard<std::mutex> hold(*lock);
    const auto it = kept->find(key);
    if (it != kept->end() && (size_t)it->second.nbytes() >= need) return it->second;
    at::Tensor t = empty({(int64_t)n}, at::kByte);
    const spec_status_t s = spec_verify_workspace_init(t.data_ptr(), kHeadBytes, h);
    if (s != SPEC_OK) throw StatusFail{s, "spec_verify_workspace_init"};
    (*kept)[key] = t;
    return t;
}
at::Tensor workspace_of(PyObject* given, int kind, int device, cudaStream_t h, size_t need) {
    if (given == Py_None) return scratch(kind, device, h, need);
    const at::Tensor& t = *tensor_of(given, "workspace");
    on_cuda(t, "workspace", device);
    of_type(t, "workspace", at::kByte);
    packed(t, "workspace");
    return t;
}

void done(spec_status_t s, const char* what) {
    if (s != SPEC_OK) throw StatusFail{s, what};
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
    PyObject* out = PyTuple_New((Py_ssize_t)ts.size());
    if (!out) throw PyPending{};
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) {
        PyObject* o;
        if (t.defined()) {
            o = wrap(t);
        } else {
            o = Py_None;
            Py_INCREF(o);
        }
        if (!o) {
            Py_DECREF(out);
            throw PyPending{};
        }
        PyTuple_SET_ITEM(out, i++, o);
    }
    return out;
}

void set_status(const StatusFail& f) {
    PyObject* m = PyImport_ImportModule("speculative_decoding_verification_59_gb300");
    PyObject* type = m ? PyObject_GetAttrString(m, "SpecVerifyError") : nullptr;
    PyObject* e = type ? PyObject_CallFunction(type, "is", (int)f.status, f.what) : nullptr;
    if (e) PyErr_SetObject(type, e);
    Py_XDECREF(e);
    Py_XDECREF(type);
    Py_XDECREF(m);
}

// Runs a call's body with every C++ exception turned into a Python one.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F body) {
    HANDLE_TH_ERRORS
    try {
        if (n != want) throw PyFail{PyExc_TypeError, "wrong number of arguments"};
        return body();
    } catch (const PyFail& f) {
        PyErr_SetString(f.type, f.text.c_str());
    } catch (const StatusFail& f) {
        set_status(f);
    } catch (const PyPending&) {
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

// (addr, batch, device, q, k, v, context_lens, rope, q_weight, k_weight, eps, interleaved, new_lens,
//  positions, out, stream)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 16, [&]() -> PyObject* {
        const Cache c = cache_of(a[0], a[1], a[2]);
        const int64_t D = c.c->head_dim, H = c.c->kv_heads;
        const Rows k = rows_of(a[4], "k", D, c.device), v = rows_of(a[5], "v", D, c.device);
        same_rows(k, "k", k.B, k.N, H);
        same_rows(v, "v", k.B, k.N, H);
        fits(c, k.B);
        Rows q;
        if (a[3] != Py_None) {
            q = rows_of(a[3], "q", D, c.device);
            same_rows(q, "q", k.B, k.N, q.H);
        }
        const int32_t* ctx = ints(a[6], "context_lens", {k.B}, c.device);
        const float* rope = nullptr;
        int64_t rope_rows = 0, rot = 0;
        if (a[7] != Py_None) {
            const at::Tensor& t = *tensor_of(a[7], "rope");
            on_cuda(t, "rope", c.device);
            of_type(t, "rope", at::kFloat);
            if (t.dim() != 2) throw PyFail{PyExc_ValueError, "rope must have shape (rows, rot_dim), got " + shape_text(t.sizes())};
            packed(t, "rope");
            rope_rows = t.size(0);
            rot = t.size(1);
            rope = static_cast<const float*>(t.data_ptr());
        }
        const void* qw = plain<void>(a[8], "q_weight", at::kBFloat16, {D}, c.device, true);
        const void* kw = plain<void>(a[9], "k_weight", at::kBFloat16, {D}, c.device, true);
        const int32_t* newl = ints(a[12], "new_lens", {k.B}, c.device, true);
        const int32_t* pos = ints(a[13], "positions", {k.B, k.N}, c.device, true);
        const OnStream on(a[15], c.device);
        at::Tensor out;
        void* op = nullptr;
        if (a[3] != Py_None) {
            if (a[14] == Py_None) {
                out = empty({k.B, k.N, q.H, D}, at::kBFloat16);
                op = out.data_ptr();
            } else {
                op = plain<void>(a[14], "out", at::kBFloat16, {k.B, k.N, q.H, D}, c.device);
                out = *tensor_of(a[14], "out");
            }
        }
        done(spec_kv_append(c.c, q.p, k.p, v.p, q.stride, k.stride, v.stride, qw, kw, (float)real(a[10]), rope,
                            (int)rope_rows, (int)rot, truth(a[11]), ctx, newl, pos, (int)k.B, (int)k.N, (int)q.H, op, on.h),
             "spec_kv_append");
        if (!out.defined()) Py_RETURN_NONE;
        return wrap(out);
    });
}

// (addr, batch, device, T, starts, counts, float32, stream)
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject* {
        const Cache c = cache_of(a[0], a[1], a[2]);
        const int64_t T = integer(a[3]);
        int64_t B = c.batch;
        for (int i : {5, 4})
            if (a[i] != Py_None) {
                const at::Tensor& t = *tensor_of(a[i], i == 4 ? "starts" : "counts");
                B = t.numel();
            }
        fits(c, B);
        const int32_t* starts = ints(a[4], "starts", {B}, c.device, true);
        const int32_t* counts = ints(a[5], "counts", {B}, c.device, true);
        if (T < 0 || T > INT32_MAX) throw PyFail{PyExc_ValueError, "T must be in 0 .. 2^31 - 1, got " + std::to_string(T)};
        const bool f32 = truth(a[6]);
        const OnStream on(a[7], c.device);
        const int64_t shape[4] = {B, T, c.c->kv_heads, c.c->head_dim};
        // a small call's two outputs in one allocation (1 us of the host's time each); large
        // ones apart, so that either can be given up without the other
        const at::ScalarType type = f32 ? at::kFloat : at::kBFloat16;
        const int64_t n = B * T * shape[2] * shape[3];
        at::Tensor k, v;
        if (n > 0 && n <= kSharedOutput) {
            const at::Tensor both = empty({2 * n}, type);
            k = stretch(both, shape, type, 0);
            v = stretch(both, shape, type, n);
        } else {
            k = empty(shape, type);
            v = empty(shape, type);
        }
        done(spec_kv_read(c.c, starts, counts, (int)B, (int)T, f32 ? SPEC_DTYPE_F32 : SPEC_DTYPE_BF16, k.data_ptr(),
                          v.data_ptr(), on.h),
             "spec_kv_read");
        return tuple_of({k, v});
    });
}

// (addr, batch, device, context_lens, path_nodes, num_accepted, stream)
PyObject* kv_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        const Cache c = cache_of(a[0], a[1], a[2]);
        const at::Tensor& path = *tensor_of(a[4], "path_nodes");
        if (path.dim() != 2) throw PyFail{PyExc_ValueError, "path_nodes must have shape (B, N), got " + shape_text(path.sizes())};
        const int64_t B = path.size(0), N = path.size(1);
        fits(c, B);
        const int32_t* pn = ints(a[4], "path_nodes", {B, N}, c.device);
        const int32_t* ctx = ints(a[3], "context_lens", {B}, c.device);
        const int32_t* acc = ints(a[5], "num_accepted", {B}, c.device);
        const OnStream on(a[6], c.device);
        done(spec_kv_compact(c.c, ctx, pn, acc, (int)B, (int)N, on.h), "spec_kv_compact");
        Py_RETURN_NONE;
    });
}

// (addr, batch, device, q, context_lens, parents, new_lens, scale, lse, out, workspace, stream)
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const Cache c = cache_of(a[0], a[1], a[2]);
        const int64_t D = c.c->head_dim;
        const Rows q = rows_of(a[3], "q", D, c.device);
        fits(c, q.B);
        const int32_t* ctx = ints(a[4], "context_lens", {q.B}, c.device);
        const int32_t* par = ints(a[5], "parents", {q.B, q.N}, c.device, true);
        const int32_t* newl = ints(a[6], "new_lens", {q.B}, c.device, true);
        const float scale = (float)real(a[7]);
        const size_t need = spec_attention_workspace_size((int)q.B, (int)q.N, (int)q.H, c.c->kv_heads, (int)D);
        if (need == 0)
            throw PyFail{PyExc_ValueError, "paged_attention: unsupported sizes N=" + std::to_string(q.N) + " q_heads=" +
                                               std::to_string(q.H) + " kv_heads=" + std::to_string(c.c->kv_heads)};
        const OnStream on(a[11], c.device);
        at::Tensor out, lse;
        void* op;
        if (a[9] == Py_None) {
            out = empty({q.B, q.N, q.H, D}, at::kBFloat16);
            op = out.data_ptr();
        } else {
            op = plain<void>(a[9], "out", at::kBFloat16, {q.B, q.N, q.H, D}, c.device);
            out = *tensor_of(a[9], "out");
        }
        const bool want = truth(a[8]);
        if (want) lse = empty({q.B, q.N, q.H}, at::kFloat);
        const at::Tensor ws = workspace_of(a[10], 0, c.device, on.h, need);
        done(spec_paged_attention(c.c, q.p, q.stride, ctx, newl, par, scale, (int)q.B, (int)q.N, (int)q.H, op,
                                  want ? static_cast<float*>(lse.data_ptr()) : nullptr, ws.data_ptr(), ws.nbytes(), on.h),
             "spec_paged_attention");
        return want ? tuple_of({out, lse}) : wrap(out);
    });
}

// (logits, tokens, K, temperature, workspace, stream)
PyObject* token_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject* {
        const at::Tensor& z = *tensor_of(a[0], "logits");
        on_cuda(z, "logits", -1);
        const int device = z.get_device();
        const bool bf16 = z.scalar_type() == at::kBFloat16;
        if (!bf16) of_type(z, "logits", at::kFloat);
        if (z.dim() < 1) throw PyFail{PyExc_ValueError, "logits must have shape (..., V), got ()"};
        packed(z, "logits");
        const c10::IntArrayRef lead = z.sizes().slice(0, z.dim() - 1);
        const int64_t V = z.size(-1), K = integer(a[2]);
        int64_t rows = 1;
        for (int64_t d : lead) rows *= d;
        const int32_t* tok = ints(a[1], "tokens", lead, device);
        const size_t need = rows <= INT32_MAX && V <= INT32_MAX && K >= 0 && K <= 8
                                ? spec_logprobs_workspace_size((int)rows, (int)V, (int)K) : 0;
        if (need == 0)
            throw PyFail{PyExc_ValueError, "token_logprobs: unsupported sizes rows=" + std::to_string(rows) + " V=" +
                                               std::to_string(V) + " K=" + std::to_string(K)};
        const OnStream on(a[5], device);
        // one allocation for the four outputs, 4 bytes an element: an allocation takes
        // the host 1.2 us, and a call on a few short rows the GPU 3.7
        const at::Tensor all = empty({rows * (2 + 2 * K)}, at::kFloat);
        const at::Tensor lp = stretch(all, lead, at::kFloat, 0), ent = stretch(all, lead, at::kFloat, rows);
        at::Tensor ti, tl;
        if (K > 0) {
            c10::SmallVector<int64_t, 5> s(lead.begin(), lead.end());
            s.push_back(K);
            ti = stretch(all, s, at::kInt, 2 * rows);
            tl = stretch(all, s, at::kFloat, (2 + K) * rows);
        }
        const at::Tensor ws = workspace_of(a[4], 1, device, on.h, need);
        done(spec_token_logprobs(z.data_ptr(), bf16 ? SPEC_DTYPE_BF16 : SPEC_DTYPE_F32, tok, (float)real(a[3]), (int)rows,
                                 (int)V, (int)K, static_cast<float*>(lp.data_ptr()), static_cast<float*>(ent.data_ptr()),
                                 K > 0 ? static_cast<int32_t*>(ti.data_ptr()) : nullptr,
                                 K > 0 ? static_cast<float*>(tl.data_ptr()) : nullptr, ws.data_ptr(), ws.nbytes(), on.h),
             "spec_token_logprobs");
        return tuple_of({lp, ent, ti, tl});
    });
}

#define SV_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {SV_METHOD(kv_append), SV_METHOD(kv_read), SV_METHOD(kv_compact), SV_METHOD(paged_attention),
                          SV_METHOD(token_logprobs), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
