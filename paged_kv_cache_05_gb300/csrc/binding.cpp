// Python binding of the grouped-head entry points: tensor checks and the call,
// without the computation.
//
// A decode step's calls take a few microseconds on the GPU; checking a dozen
// tensors from Python and converting two dozen arguments through ctypes takes
// 10 (GB300 host), so these three calls read the tensors here.  Everything else
// is the C ABI's: the functions return its status, and raise ValueError or
// TypeError for tensors that cannot be described to it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <string>

#include "pagedkv.h"

namespace {

struct Refusal {
    PyObject* type;
    std::string what;
};

[[noreturn]] void refuse(const std::string& what) { throw Refusal{PyExc_ValueError, what}; }

// The arguments of one call, in order.
struct Reader {
    PyObject* const* at;
    PyObject* const* end;

    PyObject* next() {
        if (at == end) throw Refusal{PyExc_TypeError, "too few arguments"};
        return *at++;
    }
    const at::Tensor& tensor(const char* name) {
        PyObject* o = next();
        if (!THPVariable_Check(o))
            throw Refusal{PyExc_TypeError, std::string(name) + " must be a tensor"};
        return THPVariable_Unpack(o);
    }
    const at::Tensor* optional(const char* name) {
        if (at != end && *at == Py_None) {
            ++at;
            return nullptr;
        }
        return &tensor(name);
    }
    float number(const char* name) {
        const double v = PyFloat_AsDouble(next());
        if (v == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            throw Refusal{PyExc_TypeError, std::string(name) + " must be a number"};
        }
        return (float)v;
    }
    int truth(const char* name) {
        const int v = PyObject_IsTrue(next());
        if (v < 0) {
            PyErr_Clear();
            throw Refusal{PyExc_TypeError, std::string(name) + " must be a truth value"};
        }
        return v;
    }
    int integer(const char* name) {
        int overflow = 0;
        const long long v = PyLong_AsLongLongAndOverflow(next(), &overflow);
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            throw Refusal{PyExc_TypeError, std::string(name) + " must be an integer"};
        }
        if (overflow || v < INT_MIN || v > INT_MAX) refuse(std::string(name) + " is out of range");
        return (int)v;
    }
};

int size(int64_t n, const char* name) {
    if (n > INT_MAX) refuse(std::string(name) + " is out of range");
    return (int)n;
}

// What the call's tensors have in common: those of the queries.
struct Common {
    int dev;
    at::ScalarType type;
    pkv_dtype code;

    explicit Common(const at::Tensor& q) {
        if (!q.is_cuda()) refuse("q must be a CUDA tensor");
        dev = q.get_device();
        type = q.scalar_type();
        if (type != at::kHalf && type != at::kBFloat16)
            throw Refusal{PyExc_TypeError, "fp16 or bf16 storage expected"};
        code = type == at::kHalf ? PKV_F16 : PKV_BF16;
    }
    void on_device(const at::Tensor& t, const char* name, at::ScalarType want) const {
        if (!t.is_cuda() || t.get_device() != dev)
            refuse(std::string(name) + " must be a CUDA tensor on the device of q");
        if (t.scalar_type() != want)
            throw Refusal{PyExc_TypeError, std::string(name) + " must be " + c10::toString(want) +
                                               ", got " + c10::toString(t.scalar_type())};
    }
    void* whole(const at::Tensor& t, const char* name, at::ScalarType want) const {
        on_device(t, name, want);
        if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
        return t.data_ptr();
    }
    void* whole(const at::Tensor& t, const char* name) const { return whole(t, name, type); }
    const float* floats(const at::Tensor* t, int64_t n, const char* name) const {
        if (!t) return nullptr;
        if (t->dim() != 1 || t->size(0) != n)
            refuse(std::string(name) + " must have " + std::to_string(n) + " elements");
        return static_cast<const float*>(whole(*t, name, at::kFloat));
    }
    // rows of heads that lie side by side, tokens any stride apart
    const void* rows(const at::Tensor& t, const char* name, int64_t* stride) const {
        on_device(t, name, type);
        const int64_t T = t.size(0), H = t.size(1), D = t.size(2);
        if ((D > 1 && t.stride(2) != 1) || (H > 1 && t.stride(1) != D))
            refuse(std::string(name) + " must have its heads side by side in each token's row");
        // one token has no next one: any stride will do
        *stride = T > 1 ? t.stride(0) : H * D;
        return t.data_ptr();
    }
};

bool is(const at::Tensor& t, std::initializer_list<int64_t> shape) {
    return t.sizes().equals(at::IntArrayRef(shape));
}

cudaStream_t stream_of(Reader& r, int dev) {
    PyObject* o = r.next();
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refusal{PyExc_TypeError, "stream must be a CUDA stream"};
    }
    return static_cast<cudaStream_t>(p);
}

// Runs `call` on the device, the interpreter's lock released.
template <typename F>
pkv_status launch(int dev, F call) {
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    pkv_status st;
    Py_BEGIN_ALLOW_THREADS
    st = call();
    Py_END_ALLOW_THREADS
    return st;
}

pkv_status norm_rope_and_cache(Reader& r) {
    const at::Tensor& q_out = r.tensor("q_out");
    const at::Tensor& q = r.tensor("q");
    const at::Tensor& k = r.tensor("k");
    const at::Tensor& v = r.tensor("v");
    const at::Tensor& kc = r.tensor("k_cache");
    const at::Tensor& vc = r.tensor("v_cache");
    const at::Tensor& slots = r.tensor("slot_mapping");
    const at::Tensor& positions = r.tensor("positions");
    const at::Tensor* phases = r.optional("phases");
    const at::Tensor* qw = r.optional("q_weight");
    const at::Tensor* kw = r.optional("k_weight");
    const float eps = r.number("eps"), scale = r.number("rope_scale");
    const int interleaved = r.truth("interleaved");
    const Common c(q);
    if (q.dim() != 3 || kc.dim() != 4)
        refuse("q must be [num_tokens, num_heads, head_dim], k_cache [blocks, heads, B, head_dim]");
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
    const int64_t nb = kc.size(0), HK = kc.size(1), B = kc.size(2);
    if (kc.size(3) != D || !vc.sizes().equals(kc.sizes()) || !is(k, {T, HK, D}) ||
        !is(v, {T, HK, D}) || !q_out.sizes().equals(q.sizes()))
        refuse("q_out/q/k/v/cache shape mismatch");
    if (!is(slots, {T}) || !is(positions, {T}))
        refuse("slot_mapping and positions must be [num_tokens]");
    if (phases && phases->dim() != 1) refuse("phases must be [rot_dim / 2]");
    int64_t qs, ks, vs;
    const void* qp = c.rows(q, "q", &qs);
    const void* kp = c.rows(k, "k", &ks);
    const void* vp = c.rows(v, "v", &vs);
    void* op = c.whole(q_out, "q_out");
    void* kcp = c.whole(kc, "k_cache");
    void* vcp = c.whole(vc, "v_cache");
    const auto* sp = static_cast<const int64_t*>(c.whole(slots, "slot_mapping", at::kLong));
    const auto* pp = static_cast<const int32_t*>(c.whole(positions, "positions", at::kInt));
    const auto* ph =
        phases ? static_cast<const uint64_t*>(c.whole(*phases, "phases", at::kLong)) : nullptr;
    const int rot = phases ? size(2 * phases->size(0), "phases") : 0;
    const float* qwp = c.floats(qw, D, "q_weight");
    const float* kwp = c.floats(kw, D, "k_weight");
    const int t = size(T, "num_tokens"), h = size(H, "num_heads"), hk = size(HK, "num_kv_heads"),
              d = size(D, "head_dim"), b = size(B, "block_size");
    const cudaStream_t stream = stream_of(r, c.dev);
    return launch(c.dev, [&] {
        return pkv_norm_rope_and_cache(op, qp, kp, vp, qs, ks, vs, kcp, vcp, sp, pp, ph, rot,
                                       interleaved, scale, qwp, kwp, eps, t, h, hk, d, b, nb,
                                       c.code, stream);
    });
}

pkv_status decode_grouped(Reader& r) {
    const at::Tensor& out = r.tensor("out");
    const at::Tensor& q = r.tensor("q");
    const at::Tensor& kc = r.tensor("k_cache");
    const at::Tensor& vc = r.tensor("v_cache");
    const at::Tensor& tables = r.tensor("block_tables");
    const at::Tensor& lens = r.tensor("context_lens");
    const float scale = r.number("scale"), cap = r.number("softcap");
    const int window = r.integer("window");
    const at::Tensor* slopes = r.optional("slopes");
    const at::Tensor& ws = r.tensor("workspace");
    const Common c(q);
    if (q.dim() != 3 || kc.dim() != 4)
        refuse("q must be [num_seqs, num_heads, head_dim], k_cache [blocks, heads, B, head_dim]");
    const int64_t S = q.size(0), H = q.size(1), D = q.size(2);
    if (kc.size(3) != D || !vc.sizes().equals(kc.sizes()) || !out.sizes().equals(q.sizes()))
        refuse("out/q/cache shape mismatch");
    if (tables.dim() != 2 || tables.size(0) != S || !is(lens, {S}))
        refuse("block_tables must be [num_seqs, max_blocks], context_lens [num_seqs]");
    void* op = c.whole(out, "out");
    const void* qp = c.whole(q, "q");
    const void* kp = c.whole(kc, "k_cache");
    const void* vp = c.whole(vc, "v_cache");
    const auto* bt = static_cast<const int32_t*>(c.whole(tables, "block_tables", at::kInt));
    const auto* cl = static_cast<const int32_t*>(c.whole(lens, "context_lens", at::kInt));
    const float* sl = c.floats(slopes, H, "slopes");
    void* wp = c.whole(ws, "workspace", at::kByte);
    const int s = size(S, "num_seqs"), h = size(H, "num_heads"),
              hk = size(kc.size(1), "num_kv_heads"), d = size(D, "head_dim"),
              b = size(kc.size(2), "block_size"), width = size(tables.size(1), "max_blocks");
    const cudaStream_t stream = stream_of(r, c.dev);
    return launch(c.dev, [&] {
        return pkv_paged_attention_decode_grouped(op, qp, kp, vp, bt, cl, sl, scale, cap, window, s,
                                                  h, hk, d, b, width, kc.size(0), c.code, wp,
                                                  (size_t)ws.numel(), stream);
    });
}

pkv_status prefill_grouped(Reader& r) {
    const at::Tensor& out = r.tensor("out");
    const at::Tensor& q = r.tensor("q");
    const at::Tensor& kc = r.tensor("k_cache");
    const at::Tensor& vc = r.tensor("v_cache");
    const at::Tensor& tables = r.tensor("block_tables");
    const at::Tensor& lens = r.tensor("context_lens");
    const at::Tensor& starts = r.tensor("query_start");
    const float scale = r.number("scale");
    const int most = r.integer("max_query_len");
    const float cap = r.number("softcap");
    const int window = r.integer("window");
    const at::Tensor* slopes = r.optional("slopes");
    const at::Tensor* ws = r.optional("workspace");
    const Common c(q);
    if (q.dim() != 3 || kc.dim() != 4 || lens.dim() != 1)
        refuse("q must be [num_query_tokens, num_heads, head_dim], k_cache [blocks, heads, B, "
               "head_dim], context_lens [num_seqs]");
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2), S = lens.size(0);
    if (kc.size(3) != D || !vc.sizes().equals(kc.sizes()) || !out.sizes().equals(q.sizes()))
        refuse("out/q/cache shape mismatch");
    if (tables.dim() != 2 || tables.size(0) != S || !is(starts, {S + 1}))
        refuse("block_tables [S, max_blocks], query_start [S+1] expected");
    void* op = c.whole(out, "out");
    const void* qp = c.whole(q, "q");
    const void* kp = c.whole(kc, "k_cache");
    const void* vp = c.whole(vc, "v_cache");
    const auto* bt = static_cast<const int32_t*>(c.whole(tables, "block_tables", at::kInt));
    const auto* cl = static_cast<const int32_t*>(c.whole(lens, "context_lens", at::kInt));
    const auto* qs = static_cast<const int32_t*>(c.whole(starts, "query_start", at::kInt));
    const float* sl = c.floats(slopes, H, "slopes");
    const int s = size(S, "num_seqs"), h = size(H, "num_heads"),
              hk = size(kc.size(1), "num_kv_heads"), d = size(D, "head_dim"),
              b = size(kc.size(2), "block_size"), width = size(tables.size(1), "max_blocks"),
              t = size(T, "num_query_tokens");
    const cudaStream_t stream = stream_of(r, c.dev);
    // a workspace of the call's own, where one is of use: taken from the allocator
    // as its stream's memory (another stream's may have work pending on it) and
    // given back when the call returns, for work queued after it on that stream
    at::Tensor own;
    size_t bytes = 0;
    if (!ws && pkv_prefill_grouped_workspace_size(s, h, hk, d, b, width, most, &bytes) == PKV_OK &&
        bytes > 0) {
        const auto dev = (c10::DeviceIndex)c.dev;
        c10::cuda::OptionalCUDAStreamGuard on;
        if (stream != c10::cuda::getCurrentCUDAStream(dev).stream())
            on.reset_stream(c10::cuda::getStreamFromExternal(stream, dev));
        own = at::empty({(int64_t)bytes}, q.options().dtype(at::kByte));
        ws = &own;
    }
    void* wp = ws ? c.whole(*ws, "workspace", at::kByte) : nullptr;
    return launch(c.dev, [&] {
        return pkv_paged_attention_prefill_grouped(op, qp, kp, vp, bt, cl, qs, sl, scale, cap,
                                                   window, s, h, hk, d, b, width, kc.size(0), most,
                                                   t, c.code, wp, ws ? (size_t)ws->numel() : 0,
                                                   stream);
    });
}

// No C++ exception leaves a call.
template <pkv_status (*F)(Reader&)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    try {
        Reader r{args, args + n};
        return PyLong_FromLong(F(r));
    } catch (const Refusal& e) {
        PyErr_SetString(e.type, e.what.c_str());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

template <pkv_status (*F)(Reader&)>
PyCFunction function() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F>));
}

PyMethodDef g_methods[] = {
    {"norm_rope_and_cache", function<norm_rope_and_cache>(), METH_FASTCALL, nullptr},
    {"paged_attention_decode_grouped", function<decode_grouped>(), METH_FASTCALL, nullptr},
    {"paged_attention_prefill_grouped", function<prefill_grouped>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_pkvbind", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pkvbind(void) { return PyModule_Create(&g_module); }
