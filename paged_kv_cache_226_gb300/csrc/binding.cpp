// Python binding of the bounded-cache operators and of those of speculative
// decoding (CPython and torch C++ API).
//
// A layer makes three of these calls per step and the small ones are a launch
// or two of 2 to 6 us, so what a call costs on the host is what it costs.
// Here the checks of a call read the tensors' fields directly and its arrays
// are allocated in place.  Measured per call from Python (us; in brackets the
// same checks written in Python over ctypes): rotary write of 64 tokens 5.4
// (20.0), decode weights of 4 short sequences, two launches, 9.1 (27.2),
// eviction of 64 sequences by a block 13.4, the kernel's own time (22.8).
//
// Every function takes its arguments by position, checks them in the order
// given, raises TypeError or ValueError, and enqueues on the current stream of
// the cache's device.  It returns what the Python function returns, or the
// entry point's status as an int if that refused.  The interpreter lock is
// released around allocation and launch, which may wait for the GPU.  The
// entry points are those of the library that bind() was given last.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <dlfcn.h>

#include <algorithm>
#include <cstdint>
#include <limits>
#include <string>
#include <vector>

#include "pa.h"

namespace {

using at::Tensor;

[[noreturn]] void refuse(PyObject* type, const std::string& what) {
    PyErr_SetString(type, what.c_str());
    throw python_error();
}

// The library's entry points.  A set is made per bind() and kept, so that calls
// under way in other threads end on the one they began with.
struct Entries {
    decltype(&pa_rope_and_cache) rope_and_cache;
    decltype(&pa_rope_and_cache_fp8) rope_and_cache_fp8;
    decltype(&pa_decode_weights_workspace_size) decode_weights_workspace_size;
    decltype(&pa_decode_weights) decode_weights;
    decltype(&pa_decode_weights_fp8) decode_weights_fp8;
    decltype(&pa_prefill_weights_workspace_size) prefill_weights_workspace_size;
    decltype(&pa_prefill_weights) prefill_weights;
    decltype(&pa_evict_workspace_size) evict_workspace_size;
    decltype(&pa_evict) evict;
    decltype(&pa_evict_fp8) evict_fp8;
    decltype(&pa_norm_rope_and_cache) norm_rope_and_cache;
    decltype(&pa_norm_rope_and_cache_fp8) norm_rope_and_cache_fp8;
    decltype(&pa_tree_attention_workspace_size) tree_attention_workspace_size;
    decltype(&pa_tree_attention) tree_attention;
    decltype(&pa_tree_attention_fp8) tree_attention_fp8;
    decltype(&pa_accept_tree) accept_tree;
    decltype(&pa_commit_path) commit_path;
    decltype(&pa_commit_path_fp8) commit_path_fp8;
};

const Entries* g_entries = nullptr;

const Entries& entries() {
    if (!g_entries) refuse(PyExc_RuntimeError, "no library is bound");
    return *g_entries;
}

template <typename F>
void find(void* handle, const char* name, F& f) {
    f = reinterpret_cast<F>(dlsym(handle, name));
    if (!f) refuse(PyExc_ImportError, std::string("the library has no ") + name);
}

// (handle): the dlopen handle of the library to call, which must stay open.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 1) refuse(PyExc_TypeError, "expected 1 argument");
    void* handle = PyLong_AsVoidPtr(a[0]);
    if (!handle) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no library handle");
        throw python_error();
    }
    Entries e;
    find(handle, "pa_rope_and_cache", e.rope_and_cache);
    find(handle, "pa_rope_and_cache_fp8", e.rope_and_cache_fp8);
    find(handle, "pa_decode_weights_workspace_size", e.decode_weights_workspace_size);
    find(handle, "pa_decode_weights", e.decode_weights);
    find(handle, "pa_decode_weights_fp8", e.decode_weights_fp8);
    find(handle, "pa_prefill_weights_workspace_size", e.prefill_weights_workspace_size);
    find(handle, "pa_prefill_weights", e.prefill_weights);
    find(handle, "pa_evict_workspace_size", e.evict_workspace_size);
    find(handle, "pa_evict", e.evict);
    find(handle, "pa_evict_fp8", e.evict_fp8);
    find(handle, "pa_norm_rope_and_cache", e.norm_rope_and_cache);
    find(handle, "pa_norm_rope_and_cache_fp8", e.norm_rope_and_cache_fp8);
    find(handle, "pa_tree_attention_workspace_size", e.tree_attention_workspace_size);
    find(handle, "pa_tree_attention", e.tree_attention);
    find(handle, "pa_tree_attention_fp8", e.tree_attention_fp8);
    find(handle, "pa_accept_tree", e.accept_tree);
    find(handle, "pa_commit_path", e.commit_path);
    find(handle, "pa_commit_path_fp8", e.commit_path_fp8);
    g_entries = new Entries(e);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

std::string dtype_name(at::ScalarType t) {
    switch (t) {
        case at::kHalf: return "torch.float16";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kDouble: return "torch.float64";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kByte: return "torch.uint8";
        default: return std::string("torch.") + c10::toString(t);
    }
}

bool is_16bit(at::ScalarType t) { return t == at::kHalf || t == at::kBFloat16; }

int32_t dtype_code(at::ScalarType t) { return t == at::kHalf ? PA_FP16 : PA_BF16; }

// ---- arguments ---------------------------------------------------------------

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

constexpr int64_t kMaxInt32 = std::numeric_limits<int32_t>::max();

int32_t int32(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    if (v > kMaxInt32 || v < -kMaxInt32 - 1)
        refuse(PyExc_ValueError, std::string(name) + " does not fit in 32 bits");
    return (int32_t)v;
}

float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return (float)v;
}

void on_device(const Tensor& t, const char* name, int index) {
    if (t.get_device() != index)
        refuse(PyExc_ValueError, std::string(name) + " is on " + t.device().str() +
                                     ", expected cuda:" + std::to_string(index));
}

const Tensor& dense(PyObject* o, const char* name) {
    const Tensor& t = tensor(o, name);
    if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
    if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
    return t;
}

const Tensor& dense(PyObject* o, const char* name, at::ScalarType dtype, int index) {
    const Tensor& t = dense(o, name);
    if (t.scalar_type() != dtype)
        refuse(PyExc_TypeError, std::string(name) + " must be " + dtype_name(dtype) + ", got " +
                                    dtype_name(t.scalar_type()));
    on_device(t, name, index);
    return t;
}

// An int32 array of one entry per sequence.
const Tensor& per_sequence(PyObject* o, const char* name, int64_t n, int index) {
    const Tensor& t = dense(o, name, at::kInt, index);
    if (t.dim() != 1 || t.size(0) != n)
        refuse(PyExc_ValueError, std::string(name) + " must be an int32 [" + std::to_string(n) + "]");
    return t;
}

// An array of one entry per token.
const void* per_token(PyObject* o, const char* name, at::ScalarType dtype, int64_t n, int index) {
    const Tensor& t = dense(o, name, dtype, index);
    if (t.dim() != 1 || t.size(0) != n)
        refuse(PyExc_ValueError, std::string(name) + " must be [" + std::to_string(n) + "]");
    return t.data_ptr();
}

// [T][heads][dim], the heads of a token contiguous.
struct Rows {
    const void* data;
    int64_t tokens, stride;
};

Rows rows(PyObject* o, const char* name, int64_t heads, int64_t dim, at::ScalarType dtype, int index) {
    const Tensor& t = tensor(o, name);
    if (t.scalar_type() != dtype)
        refuse(PyExc_TypeError, std::string(name) + " must be " + dtype_name(dtype) + ", got " +
                                    dtype_name(t.scalar_type()));
    on_device(t, name, index);
    if (t.dim() != 3 || t.size(1) != heads || t.size(2) != dim)
        refuse(PyExc_ValueError, std::string(name) + " must be [num_tokens][" + std::to_string(heads) +
                                     "][" + std::to_string(dim) + "]");
    if ((t.stride(2) != 1 && dim > 1) || (t.stride(1) != dim && heads > 1))
        refuse(PyExc_ValueError, std::string(name) + ": the heads of a token must be contiguous");
    return {t.data_ptr(), t.size(0), t.size(0) > 1 ? t.stride(0) : heads * dim};
}

struct Pools {
    void *k, *v;
    int index;
    int64_t blocks, block_size, heads, dim;
    at::ScalarType dtype;
    bool fp8;

    Pools(PyObject* ko, PyObject* vo) {
        const Tensor& kt = dense(ko, "k_cache");
        const Tensor& vt = ko == vo ? kt : dense(vo, "v_cache", kt.scalar_type(), kt.get_device());
        if (kt.dim() != 4 || vt.sizes() != kt.sizes())
            refuse(PyExc_ValueError,
                   "caches must be [num_blocks][block_size][num_kv_heads][head_dim]");
        dtype = kt.scalar_type();
        fp8 = dtype == at::kByte;
        if (!fp8 && !is_16bit(dtype))
            refuse(PyExc_TypeError, "cache dtype must be float16, bfloat16 or uint8 (E4M3), got " +
                                        dtype_name(dtype));
        index = (int)kt.get_device();
        blocks = kt.size(0), block_size = kt.size(1), heads = kt.size(2), dim = kt.size(3);
        k = kt.data_ptr(), v = vt.data_ptr();
    }

    pa_shape shape(int64_t num_seqs, int64_t q_heads, int64_t max_blocks, at::ScalarType t) const {
        for (int64_t n : {num_seqs, q_heads, max_blocks, block_size, heads, dim})
            if (n > kMaxInt32)
                refuse(PyExc_ValueError, "a dimension does not fit in 32 bits");
        pa_shape s{};
        s.num_seqs = (int32_t)num_seqs;
        s.num_q_heads = (int32_t)q_heads;
        s.num_kv_heads = (int32_t)heads;
        s.head_dim = (int32_t)dim;
        s.block_size = (int32_t)block_size;
        s.max_blocks_per_seq = (int32_t)max_blocks;
        s.num_blocks = blocks;
        s.dtype = dtype_code(t);
        return s;
    }

    at::TensorOptions options(at::ScalarType t) const {
        return at::TensorOptions().dtype(t).device(at::kCUDA, (c10::DeviceIndex)index);
    }
};

// The scales go with an E4M3 cache or not at all.
struct Scales {
    float k = 0.f, v = 0.f;
    Scales(bool fp8, PyObject* ko, PyObject* vo) {
        if (fp8 && (ko == Py_None || vo == Py_None))
            refuse(PyExc_ValueError, "an FP8 cache needs k_scale and v_scale");
        if (!fp8 && (ko != Py_None || vo != Py_None))
            refuse(PyExc_ValueError, "k_scale and v_scale belong to an FP8 cache");
        if (fp8) k = real(ko), v = real(vo);
    }
};

struct Batch {
    const int32_t *tables, *lens;
    int64_t seqs, blocks;
    Batch(PyObject* bo, PyObject* lo, int index) {
        const Tensor& b = dense(bo, "block_tables", at::kInt, index);
        const Tensor& l = dense(lo, "context_lens", at::kInt, index);
        if (b.dim() != 2 || l.dim() != 1 || l.size(0) != b.size(0))
            refuse(PyExc_ValueError,
                   "block_tables must be [num_seqs][blocks], context_lens [num_seqs]");
        tables = (const int32_t*)b.data_ptr(), lens = (const int32_t*)l.data_ptr();
        seqs = b.size(0), blocks = b.size(1);
    }
};

// A [B][Hkv][>= W] state tensor.
const Tensor& state(PyObject* o, const char* name, const Batch& b, const Pools& p, at::ScalarType dtype) {
    const Tensor& t = dense(o, name, dtype, p.index);
    if (t.dim() != 3 || t.size(0) != b.seqs || t.size(1) != p.heads || t.size(2) < b.blocks * p.block_size)
        refuse(PyExc_ValueError, std::string(name) + " must be [" + std::to_string(b.seqs) + "][" +
                                     std::to_string(p.heads) + "][>= " +
                                     std::to_string(b.blocks * p.block_size) + "]");
    return t;
}

// ---- calls -------------------------------------------------------------------

struct Unlocked {
    PyThreadState* s = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(s); }
};

// The caller's workspace, or one that the allocator takes back on the current
// stream when the call has been enqueued.
struct Workspace {
    void* data = nullptr;
    size_t bytes = 0;
    c10::DataPtr own;

    Workspace(PyObject* o, int index) {
        if (o == Py_None) return;
        const Tensor& t = dense(o, "workspace");
        on_device(t, "workspace", index);
        data = t.data_ptr(), bytes = t.nbytes();
        given = true;
    }
    // false: nbytes is 0, the entry point's word for arguments it refuses
    bool need(size_t nbytes) {
        if (nbytes == 0) return false;
        if (!given) {
            own = c10::cuda::CUDACachingAllocator::get()->allocate(nbytes);
            data = own.get(), bytes = nbytes;
        }
        return true;
    }

  private:
    bool given = false;
};

PyObject* refused(int status) { return PyLong_FromLong(status); }

PyObject* same_or_new(PyObject* given, Tensor& made) {
    return given == Py_None ? THPVariable_Wrap(std::move(made)) : Py_NewRef(given);
}

PyObject* pair(PyObject* a, PyObject* b) {
    PyObject* t = a && b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return t;
}

void expect(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) refuse(PyExc_TypeError, "expected " + std::to_string(want) + " arguments");
}

// The arguments that rotary writes share, checked: rows of q, k and v, slots
// and frequencies, and where the turned q goes.
struct RopeCall {
    const Pools& p;
    at::ScalarType dt;
    Rows k, v, q{nullptr, 0, 0}, out{nullptr, 0, 0};
    const int64_t* slots;
    const float* inv_freq;
    int64_t T, half, hq = 0;
    int interleaved;
    float factor;
    bool given, make;
    Tensor made;

    RopeCall(const Pools& pools, PyObject* qo, PyObject* ko, PyObject* vo, PyObject* so, PyObject* fo,
             PyObject* oo, PyObject* io, PyObject* mo)
        : p(pools), dt(tensor(ko, "k").scalar_type()) {
        if (!is_16bit(dt) || !(p.fp8 || dt == p.dtype))
            refuse(PyExc_TypeError, "k must have the cache's 16-bit dtype, got " + dtype_name(dt));
        k = rows(ko, "k", p.heads, p.dim, dt, p.index);
        v = rows(vo, "v", p.heads, p.dim, dt, p.index);
        const Tensor& slot = dense(so, "slot_mapping", at::kLong, p.index);
        const Tensor& inv = dense(fo, "inv_freq", at::kFloat, p.index);
        T = q.tokens = out.tokens = k.tokens;
        if (v.tokens != T || slot.dim() != 1 || slot.size(0) != T || inv.dim() != 1)
            refuse(PyExc_ValueError, "v, positions and slot_mapping must have a row per token of k, "
                                     "inv_freq one dimension");
        slots = (const int64_t*)slot.data_ptr(), inv_freq = (const float*)inv.data_ptr();
        half = inv.size(0);
        given = qo != Py_None, make = given && oo == Py_None;
        if (given) {
            const Tensor& qt = tensor(qo, "q");
            hq = qt.dim() == 3 ? qt.size(1) : 0;
            q = rows(qo, "q", hq, p.dim, dt, p.index);
            if (make)
                out.stride = hq * p.dim;
            else
                out = rows(oo, "q_out", hq, p.dim, dt, p.index);
            if (q.tokens != T || out.tokens != T)
                refuse(PyExc_ValueError, "q and q_out must have a row per token of k");
        } else if (oo != Py_None) {
            refuse(PyExc_ValueError, "q_out needs q");
        }
        interleaved = PyObject_IsTrue(io);
        if (interleaved < 0) throw python_error();
        factor = real(mo);
    }
    int32_t rotary_dim() const { return (int32_t)std::min(2 * half, kMaxInt32); }
    // the current stream, with q_out allocated on it if the call makes one
    void* begin() {
        if (make) {
            made = at::empty({T, hq, p.dim}, p.options(dt));
            out.data = made.data_ptr();
        }
        return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)p.index).stream();
    }
    PyObject* result(int status, PyObject* oo) {
        if (status != PA_OK) return refused(status);
        if (!given) Py_RETURN_NONE;
        return same_or_new(oo, made);
    }
};

// (q, k, v, positions, slot_mapping, inv_freq, k_cache, v_cache, q_out,
//  interleaved, factor, k_scale, v_scale) -> q_out
PyObject* rope_and_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 13);
    const Entries& lib = entries();
    const Pools p(a[6], a[7]);
    const Scales s(p.fp8, a[11], a[12]);
    RopeCall c(p, a[0], a[1], a[2], a[4], a[5], a[8], a[9], a[10]);
    const Tensor& pos = dense(a[3], "positions", at::kLong, p.index);
    if (pos.dim() != 1 || pos.size(0) != c.T)
        refuse(PyExc_ValueError, "positions must have a row per token of k");
    const pa_shape shp = p.shape(0, c.hq, 1, c.dt);
    int status;
    {
        Unlocked u;
        c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.index);
        void* stream = c.begin();
        const int64_t* pp = (const int64_t*)pos.data_ptr();
        status = p.fp8 ? lib.rope_and_cache_fp8(c.q.data, c.q.stride, c.k.data, c.k.stride, c.v.data,
                                                c.v.stride, pp, c.slots, c.inv_freq, c.rotary_dim(),
                                                c.interleaved, c.factor, (void*)c.out.data, c.out.stride,
                                                p.k, p.v, c.T, s.k, s.v, &shp, stream)
                       : lib.rope_and_cache(c.q.data, c.q.stride, c.k.data, c.k.stride, c.v.data,
                                            c.v.stride, pp, c.slots, c.inv_freq, c.rotary_dim(),
                                            c.interleaved, c.factor, (void*)c.out.data, c.out.stride,
                                            p.k, p.v, c.T, &shp, stream);
    }
    return c.result(status, a[8]);
    END_HANDLE_TH_ERRORS
}

// A norm's weights, or null.
const void* norm_weight(PyObject* o, const char* name, const RopeCall& c) {
    if (o == Py_None) return nullptr;
    const Tensor& t = dense(o, name, c.dt, c.p.index);
    if (t.dim() != 1 || t.size(0) != c.p.dim)
        refuse(PyExc_ValueError, std::string(name) + " must be [" + std::to_string(c.p.dim) + "]");
    return t.data_ptr();
}

// (q, k, v, positions, slot_mapping, inv_freq, k_cache, v_cache, q_weight,
//  k_weight, eps, axes, q_out, interleaved, factor, k_scale, v_scale) -> q_out
PyObject* norm_rope_and_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 17);
    const Entries& lib = entries();
    const Pools p(a[6], a[7]);
    const Scales s(p.fp8, a[15], a[16]);
    RopeCall c(p, a[0], a[1], a[2], a[4], a[5], a[12], a[13], a[14]);
    const void* qw = norm_weight(a[8], "q_weight", c);
    const void* kw = norm_weight(a[9], "k_weight", c);
    const float eps = real(a[10]);
    const Tensor& pos = dense(a[3], "positions", at::kLong, p.index);
    const bool several = pos.dim() == 2;
    if ((pos.dim() != 1 && !several) || pos.size(several) != c.T || (several && pos.size(0) > kMaxInt32))
        refuse(PyExc_ValueError, "positions must be [num_tokens] or [axes][num_tokens]");
    if (several != (a[11] != Py_None))
        refuse(PyExc_ValueError, "axes belong to positions of several axes");
    const int32_t* axes = nullptr;
    if (several) {
        const Tensor& t = dense(a[11], "axes", at::kInt, p.index);
        if (t.dim() != 1 || t.size(0) != c.half)
            refuse(PyExc_ValueError, "axes must have an entry per entry of inv_freq");
        axes = (const int32_t*)t.data_ptr();
    }
    const pa_shape shp = p.shape(0, c.hq, 1, c.dt);
    int status;
    {
        Unlocked u;
        c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.index);
        void* stream = c.begin();
        const int64_t* pp = (const int64_t*)pos.data_ptr();
        const int32_t num_axes = several ? (int32_t)pos.size(0) : 1;
        status = p.fp8 ? lib.norm_rope_and_cache_fp8(c.q.data, c.q.stride, c.k.data, c.k.stride, c.v.data,
                                                     c.v.stride, qw, kw, eps, pp, num_axes, axes, c.slots,
                                                     c.inv_freq, c.rotary_dim(), c.interleaved, c.factor,
                                                     (void*)c.out.data, c.out.stride, p.k, p.v, c.T, s.k,
                                                     s.v, &shp, stream)
                       : lib.norm_rope_and_cache(c.q.data, c.q.stride, c.k.data, c.k.stride, c.v.data,
                                                 c.v.stride, qw, kw, eps, pp, num_axes, axes, c.slots,
                                                 c.inv_freq, c.rotary_dim(), c.interleaved, c.factor,
                                                 (void*)c.out.data, c.out.stride, p.k, p.v, c.T, &shp,
                                                 stream);
    }
    return c.result(status, a[12]);
    END_HANDLE_TH_ERRORS
}

// weights_out, by default weights themselves or fresh zeros; both checked.
struct Weights {
    const float* in = nullptr;
    float* out = nullptr;
    int64_t stride = 0;
    PyObject* given;                    // what the call returns, None: `made`
    Tensor made;

    Weights(PyObject* w, PyObject* wo, const Batch& b, const Pools& p) {
        given = wo != Py_None ? wo : w;
        if (given != Py_None) {
            const Tensor& t = state(given, wo != Py_None ? "weights_out" : "weights", b, p, at::kFloat);
            out = (float*)t.data_ptr();
            stride = t.size(2);
        }
        if (w != Py_None) {
            const Tensor& t = w == given ? THPVariable_Unpack(w) : state(w, "weights", b, p, at::kFloat);
            if (t.size(2) != stride)
                refuse(PyExc_ValueError, "weights and weights_out must have the same shape");
            in = (const float*)t.data_ptr();
        }
    }
    void make(const Batch& b, const Pools& p) {
        if (given != Py_None) return;
        stride = b.blocks * p.block_size;
        made = at::zeros({b.seqs, p.heads, stride}, p.options(at::kFloat));
        out = (float*)made.data_ptr();
    }
};

// (q, k_cache, v_cache, block_tables, context_lens, scale, max_context_len,
//  weights, weights_out, out, partition_size, workspace, k_scale, v_scale)
// -> (out, weights_out).  partition_size may be the function that chooses it.
PyObject* decode_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 14);
    const Entries& lib = entries();
    const Pools p(a[1], a[2]);
    const Scales s(p.fp8, a[12], a[13]);
    const Batch b(a[3], a[4], p.index);
    const at::ScalarType dt = tensor(a[0], "q").scalar_type();
    if (!is_16bit(dt) || !(p.fp8 || dt == p.dtype))
        refuse(PyExc_TypeError, "q must have the cache's 16-bit dtype, got " + dtype_name(dt));
    const Tensor& q = dense(a[0], "q", dt, p.index);
    if (q.dim() != 3 || q.size(0) != b.seqs || q.size(2) != p.dim)
        refuse(PyExc_ValueError, "q must be [num_seqs][num_q_heads][head_dim]");
    Weights w(a[7], a[8], b, p);
    void* out = nullptr;
    if (a[9] != Py_None) {
        const Tensor& t = dense(a[9], "out", dt, p.index);
        if (t.sizes() != q.sizes()) refuse(PyExc_ValueError, "out must have q's shape");
        out = t.data_ptr();
    }
    const float scale = real(a[5]);
    const int32_t longest = int32(a[6], "max_context_len");
    int32_t partition;
    if (PyCallable_Check(a[10])) {
        PyObject* v = PyObject_CallFunction(a[10], "LLiOi", (long long)b.seqs, (long long)p.heads,
                                            longest, p.fp8 ? Py_True : Py_False, p.index);
        if (!v) throw python_error();
        partition = (int32_t)PyLong_AsLong(v);
        Py_DECREF(v);
    } else {
        partition = int32(a[10], "partition_size");
    }
    Workspace ws(a[11], p.index);
    const pa_shape shp = p.shape(b.seqs, q.size(1), b.blocks, dt);
    Tensor made;
    int status;
    {
        Unlocked u;
        c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.index);
        if (!ws.need(b.seqs ? lib.decode_weights_workspace_size(&shp, longest, partition) : 1)) {
            status = PA_ERR_INVALID_ARG;
        } else {
            w.make(b, p);
            if (!out) {
                made = at::empty(q.sizes(), p.options(dt));
                out = made.data_ptr();
            }
            void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)p.index).stream();
            status = p.fp8 ? lib.decode_weights_fp8(q.data_ptr(), p.k, p.v, b.tables, b.lens, scale, s.k,
                                                    s.v, longest, partition, w.in, w.out, w.stride,
                                                    ws.data, ws.bytes, out, &shp, stream)
                           : lib.decode_weights(q.data_ptr(), p.k, p.v, b.tables, b.lens, scale, longest,
                                                partition, w.in, w.out, w.stride, ws.data, ws.bytes,
                                                out, &shp, stream);
        }
        ws.own.clear();
    }
    if (status != PA_OK) return refused(status);
    return pair(same_or_new(a[9], made), same_or_new(w.given, w.made));
    END_HANDLE_TH_ERRORS
}

// (q, k_cache, block_tables, context_lens, query_start, scale, max_query_len,
//  max_context_len, window, weights, weights_out, workspace) -> weights_out
PyObject* prefill_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 12);
    const Entries& lib = entries();
    const Pools p(a[1], a[1]);
    if (p.fp8) refuse(PyExc_TypeError, "prefill_weights reads a float16 or bfloat16 cache");
    const Batch b(a[2], a[3], p.index);
    const Tensor& q = dense(a[0], "q", p.dtype, p.index);
    const Tensor& start = dense(a[4], "query_start", at::kInt, p.index);
    if (q.dim() != 3 || q.size(2) != p.dim || start.dim() != 1 || start.size(0) != b.seqs + 1)
        refuse(PyExc_ValueError, "q must be [total_tokens][Hq][D], query_start [num_seqs + 1]");
    Weights w(a[9], a[10], b, p);
    const float scale = real(a[5]);
    const int32_t longest_chunk = int32(a[6], "max_query_len");
    const int32_t longest = int32(a[7], "max_context_len");
    const int32_t window = int32(a[8], "window");
    Workspace ws(a[11], p.index);
    const pa_shape shp = p.shape(b.seqs, q.size(1), b.blocks, p.dtype);
    int status;
    {
        Unlocked u;
        c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.index);
        if (!ws.need(lib.prefill_weights_workspace_size(&shp, longest_chunk, longest, window))) {
            status = PA_ERR_INVALID_ARG;
        } else {
            w.make(b, p);
            void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)p.index).stream();
            status = lib.prefill_weights(q.data_ptr(), p.k, b.tables, b.lens,
                                         (const int32_t*)start.data_ptr(), scale, q.size(0),
                                         longest_chunk, longest, window, w.in, w.out, w.stride, ws.data,
                                         ws.bytes, &shp, stream);
        }
        ws.own.clear();
    }
    if (status != PA_OK) return refused(status);
    return same_or_new(w.given, w.made);
    END_HANDLE_TH_ERRORS
}

// (k_cache, v_cache, block_tables, context_lens, seen_lens, budget, weights,
//  positions, known_lens, trigger, sinks, recent, weights_out, positions_out,
//  new_lens, workspace) -> new_lens
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 16);
    const Entries& lib = entries();
    const Pools p(a[0], a[1]);
    const Batch b(a[2], a[3], p.index);
    const Tensor& w = state(a[6], "weights", b, p, at::kFloat);
    const Tensor& pos = state(a[7], "positions", b, p, at::kInt);
    const Tensor& wo = a[12] == Py_None ? w : state(a[12], "weights_out", b, p, at::kFloat);
    const Tensor& po = a[13] == Py_None ? pos : state(a[13], "positions_out", b, p, at::kInt);
    const int64_t width = w.size(2);
    if (pos.size(2) != width || wo.size(2) != width || po.size(2) != width)
        refuse(PyExc_ValueError, "weights, positions and their outputs must have the same shape");
    const Tensor& seen = per_sequence(a[4], "seen_lens", b.seqs, p.index);
    int32_t* fresh = nullptr;
    if (a[14] != Py_None) fresh = (int32_t*)per_sequence(a[14], "new_lens", b.seqs, p.index).data_ptr();
    const int32_t* known = nullptr;
    if (a[8] != Py_None)
        known = (const int32_t*)per_sequence(a[8], "known_lens", b.seqs, p.index).data_ptr();
    const int32_t budget = int32(a[5], "budget");
    const int32_t trigger = a[9] == Py_None ? budget : int32(a[9], "trigger");
    const int32_t sinks = int32(a[10], "sinks"), recent = int32(a[11], "recent");
    Workspace ws(a[15], p.index);
    const pa_shape shp = p.shape(b.seqs, p.heads, b.blocks, p.fp8 ? at::kHalf : p.dtype);
    Tensor made;
    int status;
    {
        Unlocked u;
        c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.index);
        if (!ws.need(b.seqs ? lib.evict_workspace_size(&shp, budget) : 1)) {
            status = PA_ERR_INVALID_ARG;
        } else {
            if (a[14] == Py_None) {
                made = at::empty({b.seqs}, p.options(at::kInt));
                fresh = (int32_t*)made.data_ptr();
            }
            void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)p.index).stream();
            status = (p.fp8 ? lib.evict_fp8 : lib.evict)(
                p.k, p.v, b.tables, b.lens, (const int32_t*)seen.data_ptr(), known,
                (const float*)w.data_ptr(), (const int32_t*)pos.data_ptr(), width, budget, trigger,
                sinks, recent, (float*)wo.data_ptr(), (int32_t*)po.data_ptr(), fresh, ws.data, ws.bytes,
                &shp, stream);
        }
        ws.own.clear();
    }
    if (status != PA_OK) return refused(status);
    return same_or_new(a[14], made);
    END_HANDLE_TH_ERRORS
}

// The batch's int32 [num_seqs + 1] starts.
const int32_t* starts(PyObject* o, int64_t seqs, int index) {
    const Tensor& t = dense(o, "query_start", at::kInt, index);
    if (t.dim() != 1 || t.size(0) != seqs + 1)
        refuse(PyExc_ValueError, "query_start must be [num_seqs + 1]");
    return (const int32_t*)t.data_ptr();
}

// (q, k_cache, v_cache, block_tables, context_lens, query_start, parents,
//  scale, max_query_len, max_context_len, out, workspace, k_scale, v_scale)
// -> out
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 14);
    const Entries& lib = entries();
    const Pools p(a[1], a[2]);
    const Scales s(p.fp8, a[12], a[13]);
    const Batch b(a[3], a[4], p.index);
    const at::ScalarType dt = tensor(a[0], "q").scalar_type();
    if (!is_16bit(dt) || !(p.fp8 || dt == p.dtype))
        refuse(PyExc_TypeError, "q must have the cache's 16-bit dtype, got " + dtype_name(dt));
    const Tensor& q = dense(a[0], "q", dt, p.index);
    if (q.dim() != 3 || q.size(2) != p.dim)
        refuse(PyExc_ValueError, "q must be [num_tokens][num_q_heads][head_dim]");
    const int32_t* start = starts(a[5], b.seqs, p.index);
    const int32_t* parents = nullptr;
    if (a[6] != Py_None) parents = (const int32_t*)per_token(a[6], "parents", at::kInt, q.size(0), p.index);
    const float scale = real(a[7]);
    const int32_t largest = int32(a[8], "max_query_len"), longest = int32(a[9], "max_context_len");
    void* out = nullptr;
    if (a[10] != Py_None) {
        const Tensor& t = dense(a[10], "out", dt, p.index);
        if (t.sizes() != q.sizes()) refuse(PyExc_ValueError, "out must have q's shape");
        out = t.data_ptr();
    }
    Workspace ws(a[11], p.index);
    const pa_shape shp = p.shape(b.seqs, q.size(1), b.blocks, dt);
    Tensor made;
    int status;
    {
        Unlocked u;
        c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.index);
        // 0 bytes: the entry point says what it refuses
        ws.need(lib.tree_attention_workspace_size(&shp, largest, longest));
        if (a[10] == Py_None) {
            made = at::empty(q.sizes(), p.options(dt));
            out = made.data_ptr();
        }
        void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)p.index).stream();
        status = p.fp8 ? lib.tree_attention_fp8(q.data_ptr(), p.k, p.v, b.tables, b.lens, start, parents, scale,
                                                s.k, s.v, q.size(0), largest, longest, ws.data, ws.bytes, out,
                                                &shp, stream)
                       : lib.tree_attention(q.data_ptr(), p.k, p.v, b.tables, b.lens, start, parents, scale,
                                            q.size(0), largest, longest, ws.data, ws.bytes, out, &shp, stream);
        ws.own.clear();
    }
    if (status != PA_OK) return refused(status);
    return same_or_new(a[10], made);
    END_HANDLE_TH_ERRORS
}

// A contiguous CUDA tensor from element `at` of a storage on.
Tensor part_of(const c10::Storage& room, at::ScalarType dtype, int64_t at, at::IntArrayRef sizes) {
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(room), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                        c10::scalarTypeToTypeMeta(dtype));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
    t.unsafeGetTensorImpl()->set_storage_offset(at);
    return t;
}

// (draft_tokens, target_tokens, parents, query_start, max_query_len)
// -> (path, path_lens, next_tokens)
PyObject* accept_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 5);
    const Entries& lib = entries();
    const Tensor& draft = dense(a[0], "draft_tokens");
    if (draft.scalar_type() != at::kLong || draft.dim() != 1)
        refuse(PyExc_TypeError, "draft_tokens must be an int64 [num_tokens]");
    const int index = (int)draft.get_device();
    const int64_t T = draft.size(0);
    const int64_t* target = (const int64_t*)per_token(a[1], "target_tokens", at::kLong, T, index);
    const int32_t* parents = nullptr;
    if (a[2] != Py_None) parents = (const int32_t*)per_token(a[2], "parents", at::kInt, T, index);
    const Tensor& start = dense(a[3], "query_start", at::kInt, index);
    if (start.dim() != 1 || start.size(0) < 1 || start.size(0) - 1 > kMaxInt32)
        refuse(PyExc_ValueError, "query_start must be [num_seqs + 1]");
    const int64_t seqs = start.size(0) - 1;
    const int32_t largest = int32(a[4], "max_query_len");
    Tensor path, lens, next;
    int status;
    {
        Unlocked u;
        c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
        if (largest >= 1 && largest <= PA_TREE_NODES) {
            // one allocation for the three (each by itself: 1.5 us a call more apiece)
            const size_t bytes = 8 * (size_t)seqs + 4 * (size_t)seqs * (largest + 1);
            c10::Allocator* const a = c10::cuda::CUDACachingAllocator::get();
            const c10::Storage room(c10::make_intrusive<c10::StorageImpl>(c10::StorageImpl::use_byte_size_t(), bytes,
                                                                         a->allocate(bytes), a, false));
            next = part_of(room, at::kLong, 0, {seqs});
            path = part_of(room, at::kInt, 2 * seqs, {seqs, largest});
            lens = part_of(room, at::kInt, 2 * seqs + seqs * largest, {seqs});
        }
        void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
        status = lib.accept_tree((const int64_t*)draft.data_ptr(), target, parents, (const int32_t*)start.data_ptr(),
                                 (int32_t)seqs, T, largest, path.defined() ? (int32_t*)path.data_ptr() : nullptr,
                                 path.defined() ? (int32_t*)lens.data_ptr() : nullptr,
                                 path.defined() ? (int64_t*)next.data_ptr() : nullptr, stream);
    }
    if (status != PA_OK) return refused(status);
    PyObject* first = pair(THPVariable_Wrap(std::move(path)), THPVariable_Wrap(std::move(lens)));
    PyObject* last = THPVariable_Wrap(std::move(next));
    PyObject* t = first && last ? PyTuple_Pack(3, PyTuple_GET_ITEM(first, 0), PyTuple_GET_ITEM(first, 1), last) : nullptr;
    Py_XDECREF(first);
    Py_XDECREF(last);
    return t;
    END_HANDLE_TH_ERRORS
}

// (k_caches, v_caches, block_tables, context_lens, query_start, path,
//  path_lens, new_lens) -> new_lens.  k_caches, v_caches: tuples, or a cache each.
PyObject* commit_path(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 8);
    const Entries& lib = entries();
    PyObject* const* ks = a;
    PyObject* const* vs = a + 1;
    Py_ssize_t layers = 1;
    if (PyTuple_Check(a[0]) || PyTuple_Check(a[1])) {
        if (!PyTuple_Check(a[0]) || !PyTuple_Check(a[1]) || PyTuple_GET_SIZE(a[0]) != PyTuple_GET_SIZE(a[1]))
            refuse(PyExc_ValueError, "k_caches and v_caches must have a cache for every layer");
        layers = PyTuple_GET_SIZE(a[0]);
        if (layers == 0) refuse(PyExc_ValueError, "k_caches must not be empty");
        ks = &PyTuple_GET_ITEM(a[0], 0), vs = &PyTuple_GET_ITEM(a[1], 0);
    }
    const Pools p(ks[0], vs[0]);
    std::vector<void*> k(layers, p.k), v(layers, p.v);
    const at::IntArrayRef sizes = THPVariable_Unpack(ks[0]).sizes();
    for (Py_ssize_t i = 1; i < layers; ++i) {
        const Tensor& kt = dense(ks[i], "k_cache", THPVariable_Unpack(ks[0]).scalar_type(), p.index);
        const Tensor& vt = dense(vs[i], "v_cache", THPVariable_Unpack(ks[0]).scalar_type(), p.index);
        if (kt.sizes() != sizes || vt.sizes() != sizes)
            refuse(PyExc_ValueError, "the caches of all layers must have the same shape");
        k[i] = kt.data_ptr(), v[i] = vt.data_ptr();
    }
    const Batch b(a[2], a[3], p.index);
    const int32_t* start = starts(a[4], b.seqs, p.index);
    const Tensor& path = dense(a[5], "path", at::kInt, p.index);
    if (path.dim() != 2 || path.size(0) != b.seqs || path.size(1) > kMaxInt32)
        refuse(PyExc_ValueError, "path must be [num_seqs][nodes]");
    const int32_t* lens = (const int32_t*)per_sequence(a[6], "path_lens", b.seqs, p.index).data_ptr();
    int32_t* fresh = nullptr;
    if (a[7] != Py_None) fresh = (int32_t*)per_sequence(a[7], "new_lens", b.seqs, p.index).data_ptr();
    const pa_shape shp = p.shape(b.seqs, p.heads, b.blocks, p.fp8 ? at::kHalf : p.dtype);
    Tensor made;
    int status;
    {
        Unlocked u;
        c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.index);
        if (a[7] == Py_None) {
            made = at::empty({b.seqs}, p.options(at::kInt));
            fresh = (int32_t*)made.data_ptr();
        }
        void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)p.index).stream();
        status = (p.fp8 ? lib.commit_path_fp8 : lib.commit_path)(
            k.data(), v.data(), (int32_t)std::min<Py_ssize_t>(layers, kMaxInt32), b.tables, b.lens, start,
            (const int32_t*)path.data_ptr(), (int32_t)path.size(1), lens, fresh, &shp, stream);
    }
    if (status != PA_OK) return refused(status);
    return same_or_new(a[7], made);
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
constexpr PyMethodDef method(const char* name) {
    return {name, (PyCFunction)(void (*)())F, METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<rope_and_cache>("rope_and_cache"), method<decode_weights>("decode_weights"),
                         method<prefill_weights>("prefill_weights"), method<evict>("evict"), method<bind>("bind"),
                         method<norm_rope_and_cache>("norm_rope_and_cache"), method<tree_attention>("tree_attention"),
                         method<accept_tree>("accept_tree"), method<commit_path>("commit_path"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_native", "Binding of the bounded-cache and speculative-decoding operators.", -1,
                          methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module_def); }
