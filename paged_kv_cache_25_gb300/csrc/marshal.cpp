// Argument marshalling of the serving calls for Python: tensors become pointers, sizes
// and strides, and what the library would read wrongly through bare pointers (another
// type, order or device) raises.  Nothing is computed here.
//
// In C++ because a decode step makes these calls at microsecond rates: the same forty
// attribute reads and checks took 6 of a call's 11 microseconds in Python, the foreign
// call through ctypes another 1.7.
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "../../include/pa.h"

namespace {

// The library's calls, as the loaded libpa.so has them (bind()).
decltype(&pa_rope_axes_and_cache) lib_rope;
decltype(&pa_decode_shared) lib_decode_shared;
decltype(&pa_decode_scored) lib_decode_scored;
decltype(&pa_prefill_scored) lib_prefill_scored;
decltype(&pa_decode_verify) lib_decode;
decltype(&pa_prefill_chunk) lib_prefill;
decltype(&pa_gather_cache) lib_gather;

struct Raised {};   // a Python exception is set

[[noreturn]] void raise(PyObject* type, const char* what)
{
    PyErr_SetString(type, what);
    throw Raised{};
}

const at::Tensor& tensor(PyObject* o)
{
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "tensors expected");
    return THPVariable_Unpack(o);
}

pa_dtype pa_type(at::ScalarType t)
{
    switch (t) {
        case at::kFloat: return PA_F32;
        case at::kHalf: return PA_F16;
        case at::kBFloat16: return PA_BF16;
        case at::kFloat8_e4m3fn: return PA_FP8_E4M3;
        case at::kByte: return PA_FP4_E2M1;    // (pools of bytes)
        default: raise(PyExc_TypeError, "unsupported dtype");
    }
}

int to_int(int64_t x)
{
    if (x < INT_MIN || x > INT_MAX) raise(PyExc_ValueError, "a size does not fit 32 bits");
    return static_cast<int>(x);
}

int as_int(PyObject* o)
{
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Raised{};
    return to_int(x);
}

double as_double(PyObject* o)
{
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Raised{};
    return x;
}

// a scale of an FP8 or FP4 pool; missing ones reach the library as 0 and are refused there
float scale_or_zero(PyObject* o) { return o == Py_None ? 0.f : static_cast<float>(as_double(o)); }

// Other Python threads run while the library works, as they do in a foreign call.
struct Released {
    PyThreadState* const state = PyEval_SaveThread();
    Released() = default;
    ~Released() { PyEval_RestoreThread(state); }
    Released(const Released&) = delete;
};

// stream: a handle, or None for the current stream
void* stream_of(PyObject* o)
{
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Raised{};
    return reinterpret_cast<void*>(static_cast<intptr_t>(x));
}

template <typename... T>
void on_current_device(const T&... t)
{
    bool ok = (t.is_cuda() && ...);
    if (ok) {
        const int dev = c10::cuda::current_device();
        ok = ((t.get_device() == dev) && ...);
    }
    if (!ok) raise(PyExc_ValueError, "the tensors must be on the current CUDA device");
}

template <typename... T>
bool all_contiguous(const T&... t)
{
    return (t.is_contiguous() && ...);
}

pa_cache_desc descriptor(const at::Tensor& k_cache, at::ScalarType act, PyObject* k_scale, PyObject* v_scale)
{
    pa_cache_desc c{};
    c.num_blocks = to_int(k_cache.size(0));
    c.n_kv_heads = to_int(k_cache.size(1));
    c.block_size = to_int(k_cache.size(2));
    c.head_dim = to_int(k_cache.size(3));
    c.dtype = pa_type(k_cache.scalar_type());
    if (c.dtype == PA_FP4_E2M1) {   // rows of 9 bytes for 16 elements
        if (c.head_dim % 9) raise(PyExc_ValueError, "FP4 pools [blocks][n_kv][block_size][9 * head_dim / 16] expected");
        c.head_dim = c.head_dim / 9 * 16;
    }
    if (c.dtype == PA_FP8_E4M3 || c.dtype == PA_FP4_E2M1) {
        c.k_scale = scale_or_zero(k_scale);
        c.v_scale = scale_or_zero(v_scale);
        c.act_dtype = pa_type(act);
    } else {
        c.k_scale = c.v_scale = 1.f;
        c.act_dtype = c.dtype;
    }
    return c;
}

// elements of a pool's rows
int64_t head_dim(const at::Tensor& pool)
{
    return pool.scalar_type() == at::kByte ? pool.size(3) / 9 * 16 : pool.size(3);
}

template <typename T>
const T* data(const at::Tensor& t)
{
    return static_cast<const T*>(t.data_ptr());
}

// What the attention calls have in common: out and q of one shape [..][n_q][d], pools,
// tables and lengths of at least `seqs` sequences.
struct Attention {
    const at::Tensor &out, &q, &kc, &vc, &tables, &lens;
    pa_cache_desc cache;
    pa_dtype out_dtype;
    int width;
};

Attention attention(PyObject* const* a, int64_t seqs, PyObject* k_scale, PyObject* v_scale)
{
    Attention x{tensor(a[0]), tensor(a[1]), tensor(a[2]), tensor(a[3]), tensor(a[4]), tensor(a[5]), {}, PA_F32, 0};
    if (!all_contiguous(x.out, x.q, x.kc, x.vc, x.tables, x.lens))
        raise(PyExc_ValueError, "contiguous tensors expected");
    if (x.q.dim() < 3 || x.out.sizes() != x.q.sizes() || x.kc.dim() != 4 || x.q.size(-1) != head_dim(x.kc) ||
        x.vc.numel() != x.kc.numel())
        raise(PyExc_ValueError, "out and q [..][n_q][d] and pools of that head_dim expected");
    if (x.tables.dim() != 2 || x.tables.size(0) < seqs || x.lens.numel() < seqs)
        raise(PyExc_ValueError, "a block table and a context length for every sequence expected");
    if (x.tables.scalar_type() != at::kInt || x.lens.scalar_type() != at::kInt)
        raise(PyExc_TypeError, "block_tables and context_lens: int32 expected");
    const auto kv = x.kc.scalar_type();
    if (x.vc.scalar_type() != kv || (x.q.scalar_type() != kv && kv != at::kFloat8_e4m3fn && kv != at::kByte))
        raise(PyExc_TypeError, "q and the pools must have one dtype (FP8 and FP4 pools: bf16 or fp16 q)");
    on_current_device(x.q, x.out, x.kc, x.vc, x.tables, x.lens);
    x.cache = descriptor(x.kc, x.q.scalar_type(), k_scale, v_scale);
    x.out_dtype = pa_type(x.out.scalar_type());
    x.width = to_int(x.tables.size(1));
    return x;
}

// workspace: a tensor or None
void* workspace(PyObject* o, size_t* bytes)
{
    *bytes = 0;
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o);
    on_current_device(t);
    if (!t.is_contiguous()) raise(PyExc_ValueError, "contiguous workspace expected");
    *bytes = t.nbytes();
    return t.data_ptr();
}

PyObject *s_softcap, *s_slopes, *s_window, *s_first, *s_prefix;   // attribute names of ScoreMod

struct Attr {   // an attribute, released at the end
    PyObject* o;
    Attr(PyObject* from, PyObject* name) : o(PyObject_GetAttr(from, name))
    {
        if (!o) throw Raised{};
    }
    ~Attr() { Py_DECREF(o); }
    Attr(const Attr&) = delete;
};

const void* mod_array(PyObject* o, at::ScalarType type, int64_t n, const char* what)
{
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o);
    if (t.scalar_type() != type) raise(PyExc_TypeError, what);
    if (t.numel() != n || !t.is_contiguous()) raise(PyExc_ValueError, what);
    on_current_device(t);
    return t.data_ptr();
}

// The tensors behind the pointers stay alive: the ScoreMod holds them during the call.
pa_score_mod score_mod(PyObject* m, int64_t n_q, int64_t rows, int64_t reqs)
{
    const Attr cap(m, s_softcap), slopes(m, s_slopes), window(m, s_window), first(m, s_first), prefix(m, s_prefix);
    pa_score_mod s{};
    s.softcap = static_cast<float>(as_double(cap.o));
    s.alibi_slopes = static_cast<const float*>(
        mod_array(slopes.o, at::kFloat, n_q, "alibi_slopes: float32 [n_q], contiguous, expected"));
    s.window = as_int(window.o);
    s.first_key = static_cast<const int32_t*>(
        mod_array(first.o, at::kInt, rows, "first_key: int32, one per query row, contiguous, expected"));
    s.prefix_lens = static_cast<const int32_t*>(
        mod_array(prefix.o, at::kInt, reqs, "prefix_lens: int32 [requests], contiguous, expected"));
    return s;
}

// Elements from token to token of t [T][heads][d]; a token's heads are contiguous.
int64_t token_stride(const at::Tensor& t)
{
    if (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != t.size(2)))
        raise(PyExc_ValueError, "[tokens][heads][head_dim] with contiguous heads expected");
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
}

// ---------------------------------------------------------------- the calls
struct Bytes {   // a contiguous buffer of bytes (bytes, a NumPy array), released at the end
    Py_buffer b;
    explicit Bytes(PyObject* o)
    {
        if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE)) throw Raised{};
    }
    ~Bytes() { PyBuffer_Release(&b); }
    Bytes(const Bytes&) = delete;
};

// (q_out, q, k, v, positions, cos_sin, k_cache, v_cache, slot_mapping, interleaved, stream,
//  k_scale, v_scale, axis_of_pair or None)
int rope(PyObject* const* a)
{
    const at::Tensor &q_out = tensor(a[0]), &q = tensor(a[1]), &k = tensor(a[2]), &v = tensor(a[3]),
                     &pos = tensor(a[4]), &cs = tensor(a[5]), &kc = tensor(a[6]), &vc = tensor(a[7]),
                     &slots = tensor(a[8]);
    if (q.dim() != 3 || kc.dim() != 4 || q_out.sizes() != q.sizes() || k.sizes() != v.sizes() || k.dim() != 3 ||
        k.size(0) != q.size(0) || k.size(1) != kc.size(1) || k.size(2) != q.size(2) || q.size(2) != head_dim(kc))
        raise(PyExc_ValueError, "q_out, q [T][n_q][d] and k, v [T][n_kv][d] expected");
    const auto t = q.scalar_type();
    if (q_out.scalar_type() != t || k.scalar_type() != t || v.scalar_type() != t)
        raise(PyExc_TypeError, "q_out, q, k and v must have one dtype");
    if (pos.scalar_type() != at::kInt || slots.scalar_type() != at::kLong || cs.scalar_type() != at::kFloat)
        raise(PyExc_TypeError, "positions int32, slot_mapping int64 and cos_sin float32 expected");
    const int64_t T = q.size(0);
    // several axes: positions [axes][T], rows at least T apart
    const bool many = a[13] != Py_None;
    const int64_t axes = many ? (pos.dim() == 2 ? pos.size(0) : 0) : 1;
    if (many && (axes < 1 || pos.size(1) != T || (T > 1 && pos.stride(1) != 1)))
        raise(PyExc_ValueError, "positions [axes][T] expected");
    if ((!many && (pos.numel() != T || !pos.is_contiguous())) || slots.numel() != T || cs.dim() != 2 ||
        !all_contiguous(slots, cs))
        raise(PyExc_ValueError, "positions [T], slot_mapping [T] and cos_sin [max_position][rot_dim], "
                                "contiguous, expected");
    if (!all_contiguous(kc, vc) || vc.scalar_type() != kc.scalar_type() || vc.numel() != kc.numel())
        raise(PyExc_ValueError, "contiguous pools of one dtype and size expected");
    const int64_t so = token_stride(q_out), sq = token_stride(q), sk = token_stride(k), sv = token_stride(v);
    const pa_dtype in = pa_type(t);
    on_current_device(q, q_out, k, v, pos, cs, kc, vc, slots);
    const pa_cache_desc c = descriptor(kc, t, a[11], a[12]);
    const int interleaved = PyObject_IsTrue(a[9]);
    if (interleaved < 0) throw Raised{};
    void* const stream = stream_of(a[10]);
    const int max_position = to_int(cs.size(0)), rot_dim = to_int(cs.size(1)), tokens = to_int(T);
    const int n_q = to_int(q.size(1)), n_axes = to_int(axes);
    auto call = [&](const uint8_t* axis_of_pair, int64_t axis_stride) {
        const Released released;
        return lib_rope(q_out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), in, so, sq, sk, sv,
                        data<int32_t>(pos), axis_stride, n_axes, axis_of_pair, data<float>(cs), max_position, rot_dim,
                        interleaved, kc.data_ptr(), vc.data_ptr(), data<int64_t>(slots), tokens, n_q, &c, stream);
    };
    if (!many) {
        static const uint8_t one_axis[PA_MAX_ROPE_PAIRS] = {};
        return call(one_axis, 0);
    }
    const Bytes map(a[13]);
    if (map.b.itemsize != 1 || map.b.len != rot_dim / 2)
        raise(PyExc_ValueError, "axis_of_pair: uint8 [rot_dim / 2] expected");
    // (rows that overlap or run backwards: refused; a single axis has no stride)
    const int64_t stride = axes > 1 ? pos.stride(0) : T;
    if (stride < T) raise(PyExc_ValueError, "positions: rows of at least T elements expected");
    return call(static_cast<const uint8_t*>(map.b.buf), stride);
}

// (k_out, v_out, k_cache, v_cache, slot_mapping, stream, k_scale, v_scale)
int gather(PyObject* const* a)
{
    const at::Tensor &ko = tensor(a[0]), &vo = tensor(a[1]), &kc = tensor(a[2]), &vc = tensor(a[3]), &slots = tensor(a[4]);
    if (kc.dim() != 4 || ko.dim() != 3 || ko.sizes() != vo.sizes() || ko.size(1) != kc.size(1) ||
        ko.size(2) != head_dim(kc) || slots.numel() != ko.size(0))
        raise(PyExc_ValueError, "k_out, v_out [T][n_kv][d] and slot_mapping [T] expected");
    if (ko.scalar_type() != vo.scalar_type() || slots.scalar_type() != at::kLong)
        raise(PyExc_TypeError, "k_out and v_out of one dtype and slot_mapping int64 expected");
    if (!all_contiguous(ko, vo, kc, vc, slots) || vc.scalar_type() != kc.scalar_type() || vc.numel() != kc.numel())
        raise(PyExc_ValueError, "contiguous tensors and pools of one dtype and size expected");
    on_current_device(ko, vo, kc, vc, slots);
    const pa_dtype out = pa_type(ko.scalar_type());
    const pa_cache_desc c = descriptor(kc, at::kBFloat16, a[6], a[7]);
    const int tokens = to_int(slots.numel());
    void* const stream = stream_of(a[5]);
    const Released released;
    return lib_gather(ko.data_ptr(), vo.data_ptr(), out, kc.data_ptr(), vc.data_ptr(), data<int64_t>(slots), tokens, &c,
                      stream);
}

// (out, q, k_cache, v_cache, block_tables, context_lens, scale, block_size, workspace, stream,
//  k_scale, v_scale): one row a sequence, or q_per_seq
int decode(PyObject* const* a)
{
    const at::Tensor& q = tensor(a[1]);
    if (q.dim() != 3 && q.dim() != 4) raise(PyExc_ValueError, "q [B][n_q][d] or [B][q_per_seq][n_q][d] expected");
    const int64_t B = q.size(0), nq = q.dim() == 4 ? q.size(1) : 1;
    const Attention x = attention(a, B, a[10], a[11]);
    size_t bytes;
    void* ws = workspace(a[8], &bytes);
    const float scale = static_cast<float>(as_double(a[6]));
    const int block_size = as_int(a[7]), seqs = to_int(B), per_seq = to_int(nq), heads = to_int(q.size(-2));
    void* const stream = stream_of(a[9]);
    const Released released;
    return lib_decode(x.out.data_ptr(), x.out_dtype, x.q.data_ptr(), x.kc.data_ptr(), x.vc.data_ptr(), &x.cache,
                      data<int32_t>(x.tables), x.width, data<int32_t>(x.lens), seqs, per_seq, heads, scale, block_size,
                      ws, bytes, stream);
}

// (out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc, max_query_len, scale,
//  block_size, stream, k_scale, v_scale)
int prefill(PyObject* const* a)
{
    const at::Tensor &q = tensor(a[1]), &start = tensor(a[6]);
    const int64_t R = tensor(a[5]).numel();
    if (q.dim() != 3) raise(PyExc_ValueError, "q [total][n_q][d] expected");
    if (start.scalar_type() != at::kInt || start.numel() != R + 1 || !start.is_contiguous())
        raise(PyExc_ValueError, "query_start_loc int32 [R + 1], contiguous, expected");
    const Attention x = attention(a, R, a[11], a[12]);
    on_current_device(start);
    const float scale = static_cast<float>(as_double(a[8]));
    const int block_size = as_int(a[9]), max_q = as_int(a[7]), reqs = to_int(R), n_q = to_int(q.size(1));
    void* const stream = stream_of(a[10]);
    const Released released;
    return lib_prefill(x.out.data_ptr(), x.out_dtype, x.q.data_ptr(), x.kc.data_ptr(), x.vc.data_ptr(), &x.cache,
                       data<int32_t>(x.tables), x.width, data<int32_t>(start), data<int32_t>(x.lens), reqs, max_q, n_q,
                       scale, block_size, nullptr, 0, stream);
}

// (out, q, k_cache, v_cache, block_tables, context_lens, group_of_seq, prefix_lens, scale,
//  block_size, workspace, stream, k_scale, v_scale)
int decode_shared(PyObject* const* a)
{
    const at::Tensor &group = tensor(a[6]), &prefix = tensor(a[7]);
    const int64_t B = tensor(a[1]).dim() == 3 ? tensor(a[1]).size(0) : -1;
    if (B < 0) raise(PyExc_ValueError, "q [B][n_q][d] expected");
    if (group.scalar_type() != at::kInt || prefix.scalar_type() != at::kInt)
        raise(PyExc_TypeError, "group_of_seq and prefix_lens: int32 expected");
    if (group.numel() != B || !all_contiguous(group, prefix))
        raise(PyExc_ValueError, "group_of_seq [B] and prefix_lens [groups], contiguous, expected");
    const Attention x = attention(a, B, a[12], a[13]);
    on_current_device(group, prefix);
    size_t bytes;
    void* ws = workspace(a[10], &bytes);
    const float scale = static_cast<float>(as_double(a[8]));
    const int block_size = as_int(a[9]), seqs = to_int(B), n_q = to_int(x.q.size(1));
    const int groups = to_int(prefix.numel());
    void* const stream = stream_of(a[11]);
    const Released released;
    return lib_decode_shared(x.out.data_ptr(), x.out_dtype, x.q.data_ptr(), x.kc.data_ptr(), x.vc.data_ptr(),
                             &x.cache, data<int32_t>(x.tables), x.width, data<int32_t>(x.lens), seqs, n_q,
                             scale, block_size, data<int32_t>(group), data<int32_t>(prefix), groups, ws, bytes,
                             stream);
}

// (out, q, k_cache, v_cache, block_tables, context_lens, mod, scale, block_size, workspace,
//  stream, k_scale, v_scale)
int decode_scored(PyObject* const* a)
{
    const at::Tensor& q = tensor(a[1]);
    if (q.dim() != 3 && q.dim() != 4) raise(PyExc_ValueError, "q [B][n_q][d] or [B][q_per_seq][n_q][d] expected");
    const int64_t B = q.size(0), nq = q.dim() == 4 ? q.size(1) : 1, n_q = q.size(-2);
    const Attention x = attention(a, B, a[11], a[12]);
    const pa_score_mod m = score_mod(a[6], n_q, B * nq, B);
    size_t bytes;
    void* ws = workspace(a[9], &bytes);
    const float scale = static_cast<float>(as_double(a[7]));
    const int block_size = as_int(a[8]), seqs = to_int(B), per_seq = to_int(nq), heads = to_int(n_q);
    void* const stream = stream_of(a[10]);
    const Released released;
    return lib_decode_scored(x.out.data_ptr(), x.out_dtype, x.q.data_ptr(), x.kc.data_ptr(), x.vc.data_ptr(),
                             &x.cache, data<int32_t>(x.tables), x.width, data<int32_t>(x.lens), seqs, per_seq,
                             heads, scale, block_size, &m, ws, bytes, stream);
}

// (out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc, max_query_len, mod,
//  scale, block_size, stream, k_scale, v_scale)
int prefill_scored(PyObject* const* a)
{
    const at::Tensor &q = tensor(a[1]), &start = tensor(a[6]);
    const int64_t R = tensor(a[5]).numel();
    if (q.dim() != 3) raise(PyExc_ValueError, "q [total][n_q][d] expected");
    if (start.scalar_type() != at::kInt || start.numel() != R + 1 || !start.is_contiguous())
        raise(PyExc_ValueError, "query_start_loc int32 [R + 1], contiguous, expected");
    const Attention x = attention(a, R, a[12], a[13]);
    on_current_device(start);
    const pa_score_mod m = score_mod(a[8], q.size(1), q.size(0), R);
    const float scale = static_cast<float>(as_double(a[9]));
    const int block_size = as_int(a[10]), max_q = as_int(a[7]), reqs = to_int(R), n_q = to_int(q.size(1));
    void* const stream = stream_of(a[11]);
    const Released released;
    return lib_prefill_scored(x.out.data_ptr(), x.out_dtype, x.q.data_ptr(), x.kc.data_ptr(), x.vc.data_ptr(),
                              &x.cache, data<int32_t>(x.tables), x.width, data<int32_t>(start),
                              data<int32_t>(x.lens), reqs, max_q, n_q, scale, block_size, &m, stream);
}

// (addresses of pa_rope_axes_and_cache, pa_decode_shared, pa_decode_scored, pa_prefill_scored,
//  pa_decode_verify, pa_prefill_chunk, pa_gather_cache)
int bind(PyObject* const* a)
{
    uintptr_t p[7];
    for (int i = 0; i < 7; i++) {
        p[i] = static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(a[i]));
        if (PyErr_Occurred()) throw Raised{};
    }
    lib_rope = reinterpret_cast<decltype(lib_rope)>(p[0]);
    lib_decode_shared = reinterpret_cast<decltype(lib_decode_shared)>(p[1]);
    lib_decode_scored = reinterpret_cast<decltype(lib_decode_scored)>(p[2]);
    lib_prefill_scored = reinterpret_cast<decltype(lib_prefill_scored)>(p[3]);
    lib_decode = reinterpret_cast<decltype(lib_decode)>(p[4]);
    lib_prefill = reinterpret_cast<decltype(lib_prefill)>(p[5]);
    lib_gather = reinterpret_cast<decltype(lib_gather)>(p[6]);
    return 0;
}

// Every call: positional arguments in, the library's status out; no C++ exception leaves.
template <int (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    try {
        if (n != N) raise(PyExc_TypeError, "wrong number of arguments");
        return PyLong_FromLong(F(a));
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

template <int (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<bind, 7>("bind"),
                         method<rope, 14>("rope"),
                         method<gather, 8>("gather"),
                         method<decode, 12>("decode"),
                         method<prefill, 13>("prefill"),
                         method<decode_shared, 14>("decode_shared"),
                         method<decode_scored, 13>("decode_scored"),
                         method<prefill_scored, 14>("prefill_scored"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pa_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_marshal()
{
    s_softcap = PyUnicode_InternFromString("softcap");
    s_slopes = PyUnicode_InternFromString("alibi_slopes");
    s_window = PyUnicode_InternFromString("window");
    s_first = PyUnicode_InternFromString("first_key");
    s_prefix = PyUnicode_InternFromString("prefix_lens");
    if (!s_softcap || !s_slopes || !s_window || !s_first || !s_prefix) return nullptr;
    return PyModule_Create(&module);
}
