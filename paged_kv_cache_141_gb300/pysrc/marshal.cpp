// marshal.cpp -- the binding's argument marshalling for the calls of every
// decode step (rope_and_cache, key_bounds, sparse_decode; extend_tables, trim_tables,
// scaled_append, scaled_attention, verify_drafts), as a Python module
// against PyTorch's C++ headers. The checks and conversions are those a Python
// function would make; read from the tensors directly they take a fraction of a
// microsecond where attribute by attribute they took eight, several times the
// launch. The calls themselves are the C ABI's (include/pagedkv.h), handed over
// by address in bind(); this module links neither the library nor CUDA.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "pagedkv.h"

namespace {

struct TypeProblem : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct PythonProblem {};                           // the Python error is set

decltype(&pa_rope_and_cache) rope_fn = nullptr;
decltype(&pa_key_bounds) bounds_fn = nullptr;
decltype(&pa_sparse_decode) sparse_fn = nullptr;
decltype(&pa_extend_tables) extend_fn = nullptr;
decltype(&pa_trim_tables) trim_fn = nullptr;
decltype(&pa_scaled_append) append_fn = nullptr;
decltype(&pa_scaled_attention) attention_fn = nullptr;
decltype(&pa_verify_drafts) verify_fn = nullptr;
PyObject *stream_of = nullptr, *current_device = nullptr, *exchange_device = nullptr;

[[noreturn]] void bad(const std::string& what) { throw std::invalid_argument(what); }

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw TypeProblem(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

pa_dtype code_of(const at::Tensor& t) {
    switch (t.scalar_type()) {
    case at::kFloat: return PA_F32;
    case at::kHalf: return PA_F16;
    case at::kBFloat16: return PA_BF16;
    case at::kByte:
    case at::kFloat8_e4m3fn: return PA_FP8_E4M3;
    default: throw TypeProblem(std::string("unsupported tensor dtype ") + c10::toString(t.scalar_type()));
    }
}

int index_of(const at::Tensor& t) {
    if (!t.is_cuda()) bad("tensor must live on a CUDA device");
    return (int)t.get_device();
}

// A contiguous tensor's data on device `dev`; null for None where allowed.
void* data(PyObject* o, int dev, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda() || t.get_device() != dev) bad("all tensors must live on one CUDA device");
    if (!t.is_contiguous()) bad("tensor must be contiguous");
    return t.data_ptr();
}
void* data_or_null(PyObject* o, int dev, const char* name) { return o == Py_None ? nullptr : data(o, dev, name); }

// [T, heads, head_size] rows whose last two dimensions are contiguous (a view
// of a wider projection output is fine): pointer, and elements between tokens.
const void* token_rows(const at::Tensor& t, int dev, int64_t T, int64_t heads, int64_t D, const char* name,
                       int64_t& stride) {
    if (!t.is_cuda() || t.get_device() != dev) bad("all tensors must live on one CUDA device");
    if (t.dim() != 3 || t.size(0) != T || t.size(1) != heads || t.size(2) != D)
        bad(std::string(name) + " must be [" + std::to_string(T) + ", " + std::to_string(heads) + ", " +
            std::to_string(D) + "]");
    if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != D))
        bad(std::string(name) + ": each token's [heads, head_size] rows must be contiguous");
    stride = T > 1 ? t.stride(0) : heads * D;
    return t.data_ptr();
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonProblem();
    return v;
}
// An argument the ABI takes as int.
int small(PyObject* o) {
    const int64_t v = integer(o);
    if (v != (int)v) bad("argument does not fit 32 bits");
    return (int)v;
}
int small_size(int64_t v) {
    if (v != (int)v) bad("a tensor's dimension does not fit 32 bits");
    return (int)v;
}
float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonProblem();
    return (float)v;
}

int device_call(PyObject* fn, int dev) {
    PyObject* a = PyLong_FromLong(dev);
    if (!a) throw PythonProblem();
    PyObject* r = PyObject_CallOneArg(fn, a);
    Py_DECREF(a);
    if (!r) throw PythonProblem();
    const long v = PyLong_AsLong(r);
    Py_DECREF(r);
    return (int)v;
}

// The given stream (an integer, or an object with cuda_stream), or the
// device's current one.
void* stream_handle(PyObject* o, int dev) {
    PyObject* h;
    if (o == Py_None) {
        PyObject* a = PyLong_FromLong(dev);
        if (!a) throw PythonProblem();
        h = PyObject_CallOneArg(stream_of, a);
        Py_DECREF(a);
    } else if (PyLong_Check(o)) {
        h = Py_NewRef(o);
    } else {
        h = PyObject_GetAttrString(o, "cuda_stream");
    }
    if (!h) throw PythonProblem();
    void* s = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!s && PyErr_Occurred()) throw PythonProblem();
    return s;
}

// f() with device `dev` current.
template <typename F>
PyObject* run(int dev, F f) {
    PyObject* now = PyObject_CallNoArgs(current_device);
    if (!now) throw PythonProblem();
    const int was = (int)PyLong_AsLong(now);
    Py_DECREF(now);
    if (was != dev) device_call(exchange_device, dev);
    pa_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    if (was != dev) device_call(exchange_device, was);
    return PyLong_FromLong(st);
}

template <typename F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const PythonProblem&) {
    } catch (const TypeProblem& e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    }
    return nullptr;
}

bool wrong_count(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return false;
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", want, n);
    return true;
}

struct Pool {                                      // [num_blocks, Hkv, B, D]
    int64_t blocks;
    int heads, block, head;
};

Pool pool_of(const at::Tensor& k) {
    if (k.dim() != 4) bad("k_cache must be [num_blocks, num_kv_heads, block_size, head_size]");
    return {k.size(0), small_size(k.size(1)), small_size(k.size(2)), small_size(k.size(3))};
}

// query_out, query, key, value, k_cache, v_cache, cos_sin, positions, slot_mapping, q_weight, k_weight,
// eps, freq_axes, adjacent_pairs, k_scale, v_scale, dev_status, stream
PyObject* rope_and_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (wrong_count(n, 18)) return nullptr;
    return guarded([&] {
        const at::Tensor &qo = tensor(a[0], "query_out"), &q = tensor(a[1], "query"), &k = tensor(a[2], "key"),
                         &v = tensor(a[3], "value"), &kc = tensor(a[4], "k_cache"), &vc = tensor(a[5], "v_cache"),
                         &cs = tensor(a[6], "cos_sin"), &pos = tensor(a[7], "positions"),
                         &slots = tensor(a[8], "slot_mapping");
        const int dev = index_of(q);
        if (q.dim() != 3) bad("query must be [num_tokens, num_q_heads, head_size]");
        const int64_t T = q.size(0);
        const int Hq = small_size(q.size(1)), D = small_size(q.size(2));
        const Pool p = pool_of(kc);
        if (!vc.sizes().equals(kc.sizes()) || p.head != D) bad("inconsistent query/cache shapes");
        const at::ScalarType dt = q.scalar_type();
        if (k.scalar_type() != dt || v.scalar_type() != dt || qo.scalar_type() != dt)
            bad("query, key, value and query_out must share one dtype");
        if (vc.scalar_type() != kc.scalar_type()) bad("k_cache and v_cache must share one dtype");
        if (!qo.sizes().equals(q.sizes())) bad("query_out must have the query's shape");
        if (cs.scalar_type() != at::kFloat || cs.dim() != 2) bad("cos_sin must be float32 [max_position, rotary_dim]");
        const int rotary = small_size(cs.size(1));
        if (pos.scalar_type() != at::kLong || pos.dim() < 1 || pos.dim() > 2 || pos.size(-1) != T ||
            (pos.dim() == 2 && pos.size(0) < 1))
            bad("positions must be int64 [num_tokens] or [axes, num_tokens]");
        const int axes = pos.dim() == 1 ? 1 : small_size(pos.size(0));
        if (slots.scalar_type() != at::kLong || slots.numel() != T) bad("slot_mapping must be int64 [num_tokens]");
        for (int i = 9; i <= 10; ++i)
            if (a[i] != Py_None) {
                const at::Tensor& w = tensor(a[i], "norm weight");
                if (w.scalar_type() != at::kFloat || w.numel() != D) bad("norm weights must be float32 [head_size]");
            }
        struct Bytes {                             // the axes, for the call
            PyObject* o = nullptr;
            ~Bytes() { Py_XDECREF(o); }
        } fa;
        if (axes > 1) {
            if (a[12] != Py_None) {
                fa.o = PyBytes_FromObject(a[12]);
                if (!fa.o) throw PythonProblem();
            }
            if (!fa.o || PyBytes_GET_SIZE(fa.o) != rotary / 2)
                bad("several axes need freq_axes, one axis for each of rotary_dim / 2 frequencies");
        }
        const int adjacent = PyObject_IsTrue(a[13]);
        if (adjacent < 0) throw PythonProblem();
        int64_t qs, ks, vs;
        const void* qp = token_rows(q, dev, T, Hq, D, "query", qs);
        const void* kp = token_rows(k, dev, T, p.heads, D, "key", ks);
        const void* vp = token_rows(v, dev, T, p.heads, D, "value", vs);
        void *out = data(a[0], dev, "query_out"), *kcp = data(a[4], dev, "k_cache"), *vcp = data(a[5], dev, "v_cache");
        const float* csp = static_cast<const float*>(data(a[6], dev, "cos_sin"));
        const int64_t* pp = static_cast<const int64_t*>(data(a[7], dev, "positions"));
        const int64_t* sp = static_cast<const int64_t*>(data(a[8], dev, "slot_mapping"));
        const float* qw = static_cast<const float*>(data_or_null(a[9], dev, "q_weight"));
        const float* kw = static_cast<const float*>(data_or_null(a[10], dev, "k_weight"));
        const float eps = number(a[11]), k_scale = number(a[14]), v_scale = number(a[15]);
        uint32_t* status = static_cast<uint32_t*>(data_or_null(a[16], dev, "dev_status"));
        const pa_dtype in = code_of(q), cache = code_of(kc);
        const int64_t max_position = cs.size(0);
        const uint8_t* axes_of = fa.o ? reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(fa.o)) : nullptr;
        void* stream = stream_handle(a[17], dev);
        return run(dev, [&] {
            return rope_fn(out, qp, qs, kp, ks, vp, vs, kcp, vcp, csp, max_position, rotary, pp, axes, axes_of,
                           adjacent, qw, kw, eps, sp, T, Hq, p.heads, D, p.block, p.blocks, in, cache, k_scale,
                           v_scale, status, stream);
        });
    });
}

// block_tables [S, max_blocks] and context_lens [S], int32
int check_tables(const at::Tensor& bt, const at::Tensor& cl, int64_t S) {
    if (bt.scalar_type() != at::kInt || cl.scalar_type() != at::kInt) bad("block_tables and context_lens must be int32");
    if (bt.dim() != 2 || bt.size(0) != S || cl.numel() != S)
        bad("block_tables must be [num_seqs, max_blocks], context_lens [num_seqs]");
    return small_size(bt.size(1));
}

void check_bounds(const at::Tensor& kb, const Pool& p) {
    if (kb.dim() != 4 || kb.size(0) != p.blocks || kb.size(1) != p.heads || kb.size(2) != 2 || kb.size(3) != p.head)
        bad("k_bounds must be [num_blocks, num_kv_heads, 2, head_size]");
}

// k_bounds, k_cache, block_tables, context_lens, max_context_len, new_tokens, max_new_tokens, dev_status, stream
PyObject* key_bounds(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (wrong_count(n, 9)) return nullptr;
    return guarded([&] {
        const at::Tensor &kb = tensor(a[0], "k_bounds"), &kc = tensor(a[1], "k_cache"),
                         &bt = tensor(a[2], "block_tables"), &cl = tensor(a[3], "context_lens");
        const int dev = index_of(kc);
        const Pool p = pool_of(kc);
        check_bounds(kb, p);
        const int S = small_size(cl.numel()), mb = check_tables(bt, cl, S);
        if (a[5] != Py_None) {
            const at::Tensor& nt = tensor(a[5], "new_tokens");
            if (nt.scalar_type() != at::kInt || nt.numel() != S) bad("new_tokens must be int32 [num_seqs]");
        }
        void *kbp = data(a[0], dev, "k_bounds"), *kcp = data(a[1], dev, "k_cache");
        const int32_t* btp = static_cast<const int32_t*>(data(a[2], dev, "block_tables"));
        const int32_t* clp = static_cast<const int32_t*>(data(a[3], dev, "context_lens"));
        const int max_len = small(a[4]), max_new = small(a[6]);
        const int32_t* ntp = static_cast<const int32_t*>(data_or_null(a[5], dev, "new_tokens"));
        uint32_t* status = static_cast<uint32_t*>(data_or_null(a[7], dev, "dev_status"));
        const pa_dtype cache = code_of(kc), bounds = code_of(kb);
        void* stream = stream_handle(a[8], dev);
        return run(dev, [&] {
            return bounds_fn(kbp, kcp, btp, mb, clp, ntp, max_new, S, p.heads, p.head, p.block, p.blocks, max_len,
                             cache, bounds, status, stream);
        });
    });
}

// out, query, k_cache, v_cache, k_bounds, block_tables, context_lens, max_context_len, scale, num_select,
// workspace, first_blocks, recent_blocks, selected, k_scale, v_scale, dev_status, stream
PyObject* sparse_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (wrong_count(n, 18)) return nullptr;
    return guarded([&] {
        const at::Tensor &out = tensor(a[0], "out"), &q = tensor(a[1], "query"), &kc = tensor(a[2], "k_cache"),
                         &vc = tensor(a[3], "v_cache"), &kb = tensor(a[4], "k_bounds"),
                         &bt = tensor(a[5], "block_tables"), &cl = tensor(a[6], "context_lens"),
                         &ws = tensor(a[10], "workspace");
        const int dev = index_of(q);
        if (q.dim() != 3) bad("query must be [num_seqs, num_q_heads, head_size]");
        const int S = small_size(q.size(0)), Hq = small_size(q.size(1)), D = small_size(q.size(2));
        const Pool p = pool_of(kc);
        if (p.head != D) bad("query and cache head sizes differ");
        const int mb = check_tables(bt, cl, S);
        if (!out.sizes().equals(q.sizes()) || out.scalar_type() != q.scalar_type())
            bad("out must have the query's shape and dtype");
        if (!vc.sizes().equals(kc.sizes()) || vc.scalar_type() != kc.scalar_type())
            bad("k_cache and v_cache must have one shape and dtype");
        check_bounds(kb, p);
        if (kb.scalar_type() != q.scalar_type()) bad("k_bounds must have the query's dtype");
        const int max_len = small(a[7]), select = small(a[9]), first = small(a[11]), recent = small(a[12]);
        if (a[13] != Py_None) {
            const at::Tensor& sel = tensor(a[13], "selected");
            if (sel.scalar_type() != at::kInt || sel.dim() != 3 || sel.size(0) != S || sel.size(1) != p.heads ||
                sel.size(2) != select)
                bad("selected must be int32 [num_seqs, num_kv_heads, num_select]");
        }
        void* op = data(a[0], dev, "out");
        const void *qp = data(a[1], dev, "query"), *kcp = data(a[2], dev, "k_cache"), *vcp = data(a[3], dev, "v_cache"),
                   *kbp = data(a[4], dev, "k_bounds");
        const int32_t* btp = static_cast<const int32_t*>(data(a[5], dev, "block_tables"));
        const int32_t* clp = static_cast<const int32_t*>(data(a[6], dev, "context_lens"));
        void* wsp = data(a[10], dev, "workspace");
        const size_t ws_bytes = ws.nbytes();
        const float scale = number(a[8]), k_scale = number(a[14]), v_scale = number(a[15]);
        int32_t* selp = static_cast<int32_t*>(data_or_null(a[13], dev, "selected"));
        uint32_t* status = static_cast<uint32_t*>(data_or_null(a[16], dev, "dev_status"));
        const pa_dtype qt = code_of(q), cache = code_of(kc);
        void* stream = stream_handle(a[17], dev);
        return run(dev, [&] {
            return sparse_fn(op, qp, kcp, vcp, kbp, btp, mb, clp, S, Hq, p.heads, D, p.block, p.blocks, max_len, scale,
                             select, first, recent, selp, qt, cache, k_scale, v_scale, wsp, ws_bytes, status, stream);
        });
    });
}

// ---- a step that does not wait for the host

const at::Tensor& ints(PyObject* o, const char* name, int64_t n) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != at::kInt || t.numel() != n) bad(std::string(name) + " must be int32 [" + std::to_string(n) + "]");
    return t;
}
int32_t* int_data(PyObject* o, int dev, const char* name, int64_t n) {
    ints(o, name, n);
    return static_cast<int32_t*>(data(o, dev, name));
}
int32_t* int_data_or_null(PyObject* o, int dev, const char* name, int64_t n) {
    return o == Py_None ? nullptr : int_data(o, dev, name, n);
}
int32_t* table_data(PyObject* o, int dev, int64_t S, int& max_blocks) {
    const at::Tensor& t = tensor(o, "block_tables");
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != S) bad("block_tables must be int32 [num_seqs, max_blocks]");
    max_blocks = small_size(t.size(1));
    return static_cast<int32_t*>(data(o, dev, "block_tables"));
}
int64_t* long_data(PyObject* o, int dev, const char* name) {
    if (tensor(o, name).scalar_type() != at::kLong) bad(std::string(name) + " must be int64");
    return static_cast<int64_t*>(data(o, dev, name));
}

// block_tables, context_lens, new_tokens, free_blocks, num_free, slot_mapping, query_start, block_size,
// positions, new_lens, new_num_free, dev_status, stream
PyObject* extend_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (wrong_count(n, 13)) return nullptr;
    return guarded([&] {
        const at::Tensor &cl = tensor(a[1], "context_lens"), &stack = tensor(a[3], "free_blocks"),
                         &slots = tensor(a[5], "slot_mapping");
        const int dev = index_of(cl);
        const int S = small_size(cl.numel());
        int mb;
        int32_t* bt = table_data(a[0], dev, S, mb);
        int32_t *len = int_data(a[1], dev, "context_lens", S), *more = int_data(a[2], dev, "new_tokens", S);
        int32_t *sp = int_data(a[3], dev, "free_blocks", stack.numel()), *nf = int_data(a[4], dev, "num_free", 1);
        int64_t* slp = long_data(a[5], dev, "slot_mapping");
        int32_t* qs = int_data(a[6], dev, "query_start", (int64_t)S + 1);
        int64_t* pos = a[8] == Py_None ? nullptr : long_data(a[8], dev, "positions");
        const int64_t cap = stack.numel(), T = slots.numel();
        if (pos && tensor(a[8], "positions").numel() != T) bad("positions must have slot_mapping's size");
        int32_t *nl = a[9] == Py_None ? len : int_data(a[9], dev, "new_lens", S),
                *nn = a[10] == Py_None ? nf : int_data(a[10], dev, "new_num_free", 1);
        const int B = small(a[7]);
        uint32_t* status = static_cast<uint32_t*>(data_or_null(a[11], dev, "dev_status"));
        void* stream = stream_handle(a[12], dev);
        return run(dev, [&] {
            return extend_fn(bt, mb, len, more, S, sp, nf, cap, B, slp, pos, T, qs, nl, nn, status, stream);
        });
    });
}

// block_tables, context_lens, drop_tokens, free_blocks, num_free, block_size, shared_blocks, new_lens,
// new_num_free, dev_status, stream
PyObject* trim_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (wrong_count(n, 11)) return nullptr;
    return guarded([&] {
        const at::Tensor &cl = tensor(a[1], "context_lens"), &stack = tensor(a[3], "free_blocks");
        const int dev = index_of(cl);
        const int S = small_size(cl.numel());
        int mb;
        const int32_t* bt = table_data(a[0], dev, S, mb);
        int32_t *len = int_data(a[1], dev, "context_lens", S), *drop = int_data(a[2], dev, "drop_tokens", S);
        int32_t *sp = int_data(a[3], dev, "free_blocks", stack.numel()), *nf = int_data(a[4], dev, "num_free", 1);
        const int32_t* shared = int_data_or_null(a[6], dev, "shared_blocks", S);
        const int64_t cap = stack.numel();
        int32_t *nl = a[7] == Py_None ? len : int_data(a[7], dev, "new_lens", S),
                *nn = a[8] == Py_None ? nf : int_data(a[8], dev, "new_num_free", 1);
        const int B = small(a[5]);
        uint32_t* status = static_cast<uint32_t*>(data_or_null(a[9], dev, "dev_status"));
        void* stream = stream_handle(a[10], dev);
        return run(dev, [&] { return trim_fn(bt, mb, len, drop, S, sp, nf, cap, B, shared, nl, nn, status, stream); });
    });
}

pa_dtype scaled_code(const at::Tensor& t) { return t.scalar_type() == at::kChar ? PA_INT8 : code_of(t); }

// Caches of codes and their scales, as they lie.
struct ScaledPool : Pool {
    void *k, *v;
    float *k_scales, *v_scales;
    pa_dtype type;
};
ScaledPool scaled_pool(PyObject* const* a, int dev) {              // k_cache, v_cache, k_scales, v_scales
    const at::Tensor &kc = tensor(a[0], "k_cache"), &vc = tensor(a[1], "v_cache"), &ks = tensor(a[2], "k_scales"),
                     &vs = tensor(a[3], "v_scales");
    ScaledPool p;
    static_cast<Pool&>(p) = pool_of(kc);
    if (!vc.sizes().equals(kc.sizes()) || vc.scalar_type() != kc.scalar_type())
        bad("k_cache and v_cache must have one shape and dtype");
    for (const at::Tensor* t : {&ks, &vs})
        if (t->scalar_type() != at::kFloat || t->dim() != 2 || t->size(0) != p.blocks || t->size(1) != p.heads)
            bad("k_scales and v_scales must be float32 [num_blocks, num_kv_heads]");
    p.k = data(a[0], dev, "k_cache");
    p.v = data(a[1], dev, "v_cache");
    p.k_scales = static_cast<float*>(data(a[2], dev, "k_scales"));
    p.v_scales = static_cast<float*>(data(a[3], dev, "v_scales"));
    p.type = scaled_code(kc);
    return p;
}

// key, value, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, max_new_tokens, query_start,
// dev_status, stream
PyObject* scaled_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (wrong_count(n, 12)) return nullptr;
    return guarded([&] {
        const at::Tensor &k = tensor(a[0], "key"), &v = tensor(a[1], "value"), &cl = tensor(a[7], "context_lens");
        const int dev = index_of(k);
        const ScaledPool p = scaled_pool(a + 2, dev);
        if (k.dim() != 3) bad("key must be [num_tokens, num_kv_heads, head_size]");
        if (v.scalar_type() != k.scalar_type()) bad("key and value must share one dtype");
        const int64_t T = k.size(0);
        int64_t kst, vst;
        const void *kp = token_rows(k, dev, T, p.heads, p.head, "key", kst),
                   *vp = token_rows(v, dev, T, p.heads, p.head, "value", vst);
        const int S = small_size(cl.numel());
        int mb;
        const int32_t* bt = table_data(a[6], dev, S, mb);
        const int32_t* len = int_data(a[7], dev, "context_lens", S);
        const int32_t* qs = int_data_or_null(a[9], dev, "query_start", (int64_t)S + 1);
        const int most = small(a[8]);
        uint32_t* status = static_cast<uint32_t*>(data_or_null(a[10], dev, "dev_status"));
        const pa_dtype in = code_of(k);
        void* stream = stream_handle(a[11], dev);
        return run(dev, [&] {
            return append_fn(kp, kst, vp, vst, p.k, p.v, p.k_scales, p.v_scales, bt, mb, len, qs, T, most, S, p.heads,
                             p.head, p.block, p.blocks, in, p.type, status, stream);
        });
    });
}

// out, query, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, max_context_len, scale,
// workspace, query_start, max_queries_per_seq, dev_status, stream
PyObject* scaled_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (wrong_count(n, 15)) return nullptr;
    return guarded([&] {
        const at::Tensor &out = tensor(a[0], "out"), &q = tensor(a[1], "query"), &cl = tensor(a[7], "context_lens");
        const int dev = index_of(q);
        const ScaledPool p = scaled_pool(a + 2, dev);
        if (q.dim() != 3 || q.size(2) != p.head) bad("query must be [num_queries, num_q_heads, head_size] of the cache's head size");
        if (!out.sizes().equals(q.sizes()) || out.scalar_type() != q.scalar_type())
            bad("out must have the query's shape and dtype");
        const int T = small_size(q.size(0)), Hq = small_size(q.size(1)), S = small_size(cl.numel());
        void* op = data(a[0], dev, "out");
        const void* qp = data(a[1], dev, "query");
        int mb;
        const int32_t* bt = table_data(a[6], dev, S, mb);
        const int32_t* len = int_data(a[7], dev, "context_lens", S);
        const int32_t* qs = int_data_or_null(a[11], dev, "query_start", (int64_t)S + 1);
        void* wsp = data_or_null(a[10], dev, "workspace");
        const size_t ws_bytes = wsp ? tensor(a[10], "workspace").nbytes() : 0;
        const int max_len = small(a[8]), most = small(a[12]);
        const float scale = number(a[9]);
        uint32_t* status = static_cast<uint32_t*>(data_or_null(a[13], dev, "dev_status"));
        const pa_dtype qt = code_of(q);
        void* stream = stream_handle(a[14], dev);
        return run(dev, [&] {
            return attention_fn(op, qp, p.k, p.v, p.k_scales, p.v_scales, bt, mb, len, qs, T, most, S, Hq, p.heads, p.head,
                                p.block, p.blocks, max_len, scale, qt, p.type, wsp, ws_bytes, status, stream);
        });
    });
}

// Rows of a vocabulary, the last dimension contiguous and the others evenly spaced.
const float* prob_rows(PyObject* o, int dev, const char* name, int64_t& rows, int64_t& vocab, int64_t& stride) {
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda() || t.get_device() != dev) bad("all tensors must live on one CUDA device");
    if (t.scalar_type() != at::kFloat || t.dim() < 2) bad(std::string(name) + " must be float32 rows of the vocabulary");
    const int64_t d = t.dim();
    vocab = t.size(d - 1);
    rows = t.numel() == 0 ? 0 : t.numel() / vocab;
    if (rows == 0 && d <= 3) {                     // a step without drafts: nothing is spaced
        stride = vocab;
        return t.const_data_ptr<float>();
    }
    stride = t.size(d - 2) > 1 ? t.stride(d - 2) : (d == 3 && t.size(0) > 1 ? t.stride(0) : vocab);
    if ((vocab > 1 && t.stride(d - 1) != 1) || (d == 3 && t.size(0) > 1 && t.stride(0) != t.size(1) * stride) || d > 3)
        bad(std::string(name) + ": rows must be contiguous and evenly spaced");
    return t.const_data_ptr<float>();
}

// out_tokens, accepted, target_probs, draft_tokens, uniforms, query_start, draft_probs, rejected, dev_status, stream
PyObject* verify_drafts(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (wrong_count(n, 10)) return nullptr;
    return guarded([&] {
        const at::Tensor &ot = tensor(a[0], "out_tokens"), &dt = tensor(a[3], "draft_tokens"), &u = tensor(a[4], "uniforms");
        const int dev = index_of(tensor(a[2], "target_probs"));
        if (dt.dim() != 2) bad("draft_tokens must be int64 [num_seqs, max_drafts]");
        const int S = small_size(dt.size(0)), K = small_size(dt.size(1));
        if (ot.dim() != 2 || ot.size(0) != S || ot.size(1) != (int64_t)K + 1) bad("out_tokens must be int64 [num_seqs, max_drafts + 1]");
        if (u.scalar_type() != at::kFloat || u.dim() != 2 || u.size(0) != S || u.size(1) != (int64_t)K + 1)
            bad("uniforms must be float32 [num_seqs, max_drafts + 1]");
        int64_t rows, V, stride, drows, dV, dstride = 0;
        const float* tp = prob_rows(a[2], dev, "target_probs", rows, V, stride);
        const float* dp = nullptr;
        if (a[6] != Py_None) {
            dp = prob_rows(a[6], dev, "draft_probs", drows, dV, dstride);
            if (dV != V || drows != (int64_t)S * K) bad("draft_probs must be [num_seqs, max_drafts] rows of the target's vocabulary");
            if (drows <= 1) dstride = V;
        }
        if (rows <= 1) stride = V;
        int64_t *otp = long_data(a[0], dev, "out_tokens"), *dtp = long_data(a[3], dev, "draft_tokens");
        const float* up = static_cast<const float*>(data(a[4], dev, "uniforms"));
        int32_t* acc = int_data(a[1], dev, "accepted", S);
        const int32_t* qs = int_data(a[5], dev, "query_start", (int64_t)S + 1);
        int32_t* rej = int_data_or_null(a[7], dev, "rejected", S);
        const int vocab = small_size(V);
        uint32_t* status = static_cast<uint32_t*>(data_or_null(a[8], dev, "dev_status"));
        void* stream = stream_handle(a[9], dev);
        return run(dev, [&] {
            return verify_fn(otp, acc, rej, tp, stride, rows, dp, dstride, dtp, up, qs, S, K, vocab, status, stream);
        });
    });
}

// The addresses of the five entry points above.
PyObject* bind_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (wrong_count(n, 5)) return nullptr;
    extend_fn = reinterpret_cast<decltype(extend_fn)>(PyLong_AsVoidPtr(a[0]));
    trim_fn = reinterpret_cast<decltype(trim_fn)>(PyLong_AsVoidPtr(a[1]));
    append_fn = reinterpret_cast<decltype(append_fn)>(PyLong_AsVoidPtr(a[2]));
    attention_fn = reinterpret_cast<decltype(attention_fn)>(PyLong_AsVoidPtr(a[3]));
    verify_fn = reinterpret_cast<decltype(verify_fn)>(PyLong_AsVoidPtr(a[4]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

// The addresses of the first three entry points, and PyTorch's raw getters: the
// current stream of a device, the current device, and its exchange.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (wrong_count(n, 6)) return nullptr;
    rope_fn = reinterpret_cast<decltype(rope_fn)>(PyLong_AsVoidPtr(a[0]));
    bounds_fn = reinterpret_cast<decltype(bounds_fn)>(PyLong_AsVoidPtr(a[1]));
    sparse_fn = reinterpret_cast<decltype(sparse_fn)>(PyLong_AsVoidPtr(a[2]));
    if (PyErr_Occurred()) return nullptr;
    Py_XSETREF(stream_of, Py_NewRef(a[3]));
    Py_XSETREF(current_device, Py_NewRef(a[4]));
    Py_XSETREF(exchange_device, Py_NewRef(a[5]));
    Py_RETURN_NONE;
}

#define PA_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PA_METHOD(bind), PA_METHOD(rope_and_cache), PA_METHOD(key_bounds),
                         PA_METHOD(sparse_decode), PA_METHOD(extend_tables), PA_METHOD(trim_tables),
                         PA_METHOD(scaled_append), PA_METHOD(scaled_attention), PA_METHOD(verify_drafts),
                         PA_METHOD(bind_step), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
