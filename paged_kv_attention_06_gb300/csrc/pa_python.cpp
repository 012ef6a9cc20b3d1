// The Python side of the calls that take a model's step from the projection to
// the evicted cache (pa_qk_norm_rope_append, the window and weight calls,
// pa_kv_evict), of the 4-bit pools' calls and of the decode behind shared prefixes:
// argument checks, the tensors that a call makes where none are given (outputs, a
// workspace of this call alone, both made on the device of the call and for its
// stream), and the call of the C ABI on that device and stream. An append of one token
// takes 2.1 us on the GPU; a call of it 3.4 us, 10.7 with these checks written in
// Python.
//
// Module _pagedattn_calls; binding.py declares the signatures and documents them.
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include <cmath>
#include <limits>
#include <optional>
#include <string>

#include "../../include/pagedattn.h"

namespace {

PyObject* g_error = nullptr;   // PagedAttentionError

// The C call without the interpreter lock: a launch may wait for room in its stream's
// queue, and what would make room may need the lock. Nothing in it touches Python. (The
// tensors stay alive: the caller's frame holds them.)
template <typename F>
pa_status unlocked(F call)
{
    PyThreadState* const state = PyEval_SaveThread();
    const pa_status st = call();
    PyEval_RestoreThread(state);
    return st;
}

// Thrown with a Python error set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& what)
{
    PyErr_SetString(type, what.c_str());
    throw Raised();
}
[[noreturn]] void value_error(const std::string& what) { raise(PyExc_ValueError, what); }

// A call's body: what it raises, and what torch throws, as Python errors.
template <typename F>
PyObject* guarded(F body)
{
    HANDLE_TH_ERRORS
    try {
        return body();
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

const at::Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o))
        raise(PyExc_TypeError, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

int32_t integer(PyObject* o, const char* name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Raised();
    if (v < std::numeric_limits<int32_t>::min() || v > std::numeric_limits<int32_t>::max())
        value_error(std::string(name) + " does not fit 32 bits");
    return int32_t(v);
}

// A size of a tensor as the C ABI takes it.
int32_t size32(int64_t n, const char* what)
{
    if (n > std::numeric_limits<int32_t>::max())
        value_error(std::string(what) + " does not fit 32 bits");
    return int32_t(n);
}

double number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Raised();
    return v;
}

bool truth(PyObject* o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw Raised();
    return v != 0;
}

// The call's device, from its first tensor; its stream; and the checks of the
// others against them.
struct Call {
    c10::DeviceIndex device;
    std::optional<c10::cuda::CUDAGuard> guard;
    c10::cuda::CUDAStream current;
    cudaStream_t stream;
    bool other_stream = false;

    Call(const at::Tensor& first, const char* name, PyObject* stream_arg)
        : device(first.is_cuda() ? first.get_device() : -1),
          current(c10::cuda::CUDAStream::UNCHECKED, c10::Stream(c10::Stream::DEFAULT, c10::Device(c10::kCUDA, 0)))
    {
        if (device < 0)
            value_error(std::string(name) + " must be a CUDA tensor");
        guard.emplace(device);
        current = c10::cuda::getCurrentCUDAStream(device);
        stream = current.stream();
        if (stream_arg != Py_None) {
            const unsigned long long raw = PyLong_AsUnsignedLongLong(stream_arg);
            if (raw == ~0ull && PyErr_Occurred())
                throw Raised();
            other_stream = reinterpret_cast<cudaStream_t>(raw) != stream;
            stream = reinterpret_cast<cudaStream_t>(raw);
        }
    }

    void* check(const at::Tensor& t, at::ScalarType type, const char* name, bool contiguous = true) const
    {
        if (!t.is_cuda())
            value_error(std::string(name) + " must be a CUDA tensor");
        if (t.get_device() != device)
            value_error(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) +
                        ", expected cuda:" + std::to_string(device));
        if (t.scalar_type() != type)
            raise(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type) + ", got " +
                                       c10::toString(t.scalar_type()));
        if (contiguous && !t.is_contiguous())
            value_error(std::string(name) + " must be contiguous");
        return t.data_ptr();
    }
    void* check_or_null(PyObject* o, at::ScalarType type, const char* name) const
    {
        return o == Py_None ? nullptr : check(tensor(o, name), type, name);
    }

    // Memory for the call, of its stream's own: what was freed on the current one
    // may still be in use there. The caller reads it on the current stream.
    at::Tensor make(at::IntArrayRef sizes, at::ScalarType type) const
    {
        const auto options = at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, device));
        if (!other_stream)
            return at::empty(sizes, options);
        const c10::cuda::CUDAStreamGuard on(c10::cuda::getStreamFromExternal(stream, device));
        const at::Tensor t = at::empty(sizes, options);
        t.record_stream(current.unwrap());
        return t;
    }
    // The caller's workspace, or one of this call: the allocator orders its reuse
    // (a capture's lives in the graph's pool).
    at::Tensor workspace(PyObject* o, size_t need) const
    {
        if (o == Py_None)
            return make({int64_t(need < 16 ? 16 : need)}, at::kByte);
        const at::Tensor& t = tensor(o, "workspace");
        if (!t.is_cuda() || t.get_device() != device)
            value_error("workspace must be on the query's device");
        if (!t.is_contiguous())
            value_error("workspace must be contiguous");
        return t;
    }
};

bool raised(pa_status st, const char* what)
{
    if (st == PA_OK)
        return false;
    PyObject* e = PyObject_CallFunction(g_error, "is", int(st), what);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return true;
}

bool shape_is(const at::Tensor& t, at::IntArrayRef want) { return t.sizes() == want; }

void check_args(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want)
        raise(PyExc_TypeError, "expected " + std::to_string(want) + " arguments, got " + std::to_string(n));
}

// qkv, q_weight, k_weight, cos_sin, positions, key_pages, value_pages, slot_mapping,
// page_size, k_scale, v_scale (None: bf16 pools), eps, interleaved, query, stream
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        check_args(n, 15);
        const at::Tensor& qkv = tensor(a[0], "qkv");
        const at::Tensor &kp = tensor(a[5], "key_pages"), &vp = tensor(a[6], "value_pages");
        const at::Tensor& slots = tensor(a[7], "slot_mapping");
        const int32_t ps = integer(a[8], "page_size");
        const bool fp8 = a[9] != Py_None;
        const char* what = fp8 ? "pa_qk_norm_rope_append_fp8" : "pa_qk_norm_rope_append";
        if (qkv.dim() != 3)
            value_error("qkv must be [B, L, (H_q + 2 H_kv) * D]");
        const int64_t B = qkv.size(0), L = qkv.size(1), width = qkv.size(2);
        if (kp.dim() != 4 || kp.size(2) != ps || vp.sizes() != kp.sizes())
            value_error("page pool shape does not match page_size");
        const int64_t P = kp.size(0), H_kv = kp.size(1), D = kp.size(3);
        const int64_t H_q = D > 0 ? width / D - 2 * H_kv : 0;
        if (H_q <= 0 || (H_q + 2 * H_kv) * D != width)
            value_error("qkv's rows are not (H_q + 2 H_kv) heads of the pools' head_dim");
        if (!shape_is(slots, {B, L}))
            value_error("slot_mapping must be [B, L]");
        Call call(qkv, "qkv", a[14]);
        call.check(qkv, at::kBFloat16, "qkv", false);
        if (qkv.stride(2) != 1)
            value_error("qkv's rows must be contiguous");
        for (int i = 1; i < 3; ++i)
            if (a[i] != Py_None && !shape_is(tensor(a[i], "the weights"), {D}))
                value_error(i == 1 ? "q_weight must be [D]" : "k_weight must be [D]");
        int64_t table = 0, R = 0;
        const bool turns = a[3] != Py_None;
        if (turns) {
            const at::Tensor& cs = tensor(a[3], "cos_sin");
            if (a[4] == Py_None || !shape_is(tensor(a[4], "positions"), {B, L}))
                value_error("positions must be [B, L]");
            if (cs.dim() != 2 || cs.size(0) > std::numeric_limits<int32_t>::max())
                value_error("cos_sin must be [table_len, rotary_dim]");
            table = cs.size(0);
            R = size32(cs.size(1), "rotary_dim");
        }
        at::Tensor query;
        if (a[13] == Py_None) {
            query = call.make({B, H_q, L, D}, at::kBFloat16);
        } else {
            query = tensor(a[13], "query");
            if (!shape_is(query, {B, H_q, L, D}))
                value_error("query must be [B, H_q, L, D]");
        }
        const at::ScalarType pool = fp8 ? at::kByte : at::kBFloat16;
        void* q_ptr = call.check(query, at::kBFloat16, "query");
        void *k_ptr = call.check(kp, pool, "key_pages"), *v_ptr = call.check(vp, pool, "value_pages");
        void* qw = call.check_or_null(a[1], at::kBFloat16, "q_weight");
        void* kw = call.check_or_null(a[2], at::kBFloat16, "k_weight");
        void* cs = call.check_or_null(a[3], at::kFloat, "cos_sin");
        void* pos = turns ? call.check(tensor(a[4], "positions"), at::kInt, "positions") : nullptr;
        void* slot = call.check(slots, at::kInt, "slot_mapping");
        if (B > 0 && L > 0) {
            // the strides of an axis of one element say nothing
            const int64_t bs = B > 1 ? qkv.stride(0) : L * width, ts = L > 1 ? qkv.stride(1) : width;
            const pa_shape shape{size32(B, "B"), size32(H_q, "H_q"), size32(H_kv, "H_kv"), size32(D, "D"),
                                 size32(L, "L"), size32(P, "the number of pages"), 0};
            const float eps = float(number(a[11]));
            const int inter = truth(a[12]);
            const float ks = fp8 ? float(number(a[9])) : 1.f, vs = fp8 ? float(number(a[10])) : 1.f;
            const void* rows = qkv.data_ptr();
            const pa_status st = unlocked([&] {
                return fp8 ? pa_qk_norm_rope_append_fp8(rows, bs, ts, qw, kw, eps, static_cast<float*>(cs), int32_t(R),
                                                        int32_t(table), inter, static_cast<int32_t*>(pos), q_ptr, k_ptr,
                                                        v_ptr, static_cast<int32_t*>(slot), ps, ks, vs, shape,
                                                        call.stream)
                           : pa_qk_norm_rope_append(rows, bs, ts, qw, kw, eps, static_cast<float*>(cs), int32_t(R),
                                                    int32_t(table), inter, static_cast<int32_t*>(pos), q_ptr, k_ptr,
                                                    v_ptr, static_cast<int32_t*>(slot), ps, shape, call.stream);
            });
            if (raised(st, what))
                return nullptr;
        }
        return THPVariable_Wrap(query);
    });
}

// Bytes of a 4-bit pool's row, and the elements that it holds.
constexpr int64_t kQ4Row = 80, kQ4Elements = 128;

enum class Pool { kBf16, kE4m3, kQ4 };

// What the attention calls share: query, pools, tables, page size, scale, out.
struct Paged {
    Call call;
    void *q, *k, *v, *bt, *cl;
    pa_shape shape;
    int32_t ps;
    float scale;
    at::Tensor out;

    Paged(PyObject* const* a, PyObject* bt_arg, PyObject* cl_arg, PyObject* ps_arg, bool fp8, PyObject* scale_arg,
          PyObject* out_arg, PyObject* stream_arg)
        : Paged(a, bt_arg, cl_arg, ps_arg, fp8 ? Pool::kE4m3 : Pool::kBf16, scale_arg, out_arg, stream_arg)
    {
    }
    Paged(PyObject* const* a, PyObject* bt_arg, PyObject* cl_arg, PyObject* ps_arg, Pool kind, PyObject* scale_arg,
          PyObject* out_arg, PyObject* stream_arg)
        : call(tensor(a[0], "query"), "query", stream_arg)
    {
        const at::Tensor& query = tensor(a[0], "query");
        const at::Tensor &kp = tensor(a[1], "key_pages"), &vp = tensor(a[2], "value_pages");
        const at::Tensor &table = tensor(bt_arg, "block_table"), &lens = tensor(cl_arg, "context_lens");
        ps = integer(ps_arg, "page_size");
        if (query.dim() != 4)
            value_error("query must be [B, H_q, L, D]");
        if (kp.dim() != 4 || vp.sizes() != kp.sizes())
            value_error("page pools must be [P, H_kv, page_size, D]");
        if (kp.size(2) != ps)
            value_error("page pool shape does not match page_size");
        if (kind == Pool::kQ4 ? kp.size(3) != kQ4Row || query.size(3) != kQ4Elements : kp.size(3) != query.size(3))
            value_error(kind == Pool::kQ4 ? "4-bit pools hold rows of 80 bytes for a head_dim of 128"
                                          : "query and pages disagree on head_dim");
        if (table.dim() != 2 || table.size(0) != query.size(0) || !shape_is(lens, {query.size(0)}))
            value_error("block_table must be [B, max_pages] and context_lens [B]");
        const at::ScalarType pool = kind == Pool::kBf16 ? at::kBFloat16 : at::kByte;
        q = call.check(query, at::kBFloat16, "query");
        k = call.check(kp, pool, "key_pages");
        v = call.check(vp, pool, "value_pages");
        bt = call.check(table, at::kInt, "block_table");
        cl = call.check(lens, at::kInt, "context_lens");
        scale = scale_arg == Py_None ? float(1.0 / std::sqrt(double(query.size(3)))) : float(number(scale_arg));
        if (out_arg == Py_None) {
            out = call.make(query.sizes(), at::kBFloat16);
        } else {
            out = tensor(out_arg, "out");
            if (out.sizes() != query.sizes())
                value_error("out must have the query's shape");
            call.check(out, at::kBFloat16, "out");
        }
        shape = pa_shape{size32(query.size(0), "B"), size32(query.size(1), "H_q"), size32(kp.size(1), "H_kv"),
                         size32(query.size(3), "D"), size32(query.size(2), "L"),
                         size32(kp.size(0), "the number of pages"), size32(table.size(1), "max_pages")};
    }
    const int32_t* table() const { return static_cast<const int32_t*>(bt); }
    const int32_t* lens() const { return static_cast<const int32_t*>(cl); }
};

// which (0 decode, 1 prefill, 2 dispatch), query, key_pages, value_pages, block_table,
// context_lens, page_size, k_scale, v_scale (None: bf16 pools), window, sinks, scale, out,
// max_context_len, workspace, stream
PyObject* window(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        check_args(n, 16);
        const int32_t which = integer(a[0], "which");
        const bool fp8 = a[7] != Py_None;
        Paged p(a + 1, a[4], a[5], a[6], fp8, a[11], a[12], a[15]);
        const int32_t win = integer(a[9], "window"), sinks = integer(a[10], "sinks"),
                      longest = integer(a[13], "max_context_len");
        const float ks = fp8 ? float(number(a[7])) : 1.f, vs = fp8 ? float(number(a[8])) : 1.f;
        void* out = p.out.data_ptr();
        pa_status st;
        const char* what;
        if (which == 1) {
            what = "pa_prefill_window";
            st = unlocked([&] {
                return pa_prefill_window(p.q, p.k, p.v, p.table(), p.lens(), p.ps, p.scale, win, sinks, out, p.shape,
                                         p.call.stream);
            });
        } else {
            size_t need = 0;
            if (a[14] == Py_None)
                need = which == 0 ? pa_decode_window_workspace_bytes(p.shape)
                       : fp8      ? pa_attention_window_fp8_workspace_bytes(p.shape, p.ps, longest, win, sinks)
                                  : pa_attention_window_workspace_bytes(p.shape, p.ps, longest, win, sinks);
            const at::Tensor workspace = p.call.workspace(a[14], need);
            const size_t bytes = workspace.nbytes();
            void* ws = workspace.data_ptr();
            if (fp8) {
                what = which == 0 ? "pa_decode_window_fp8" : "pa_attention_window_fp8";
                const auto f = which == 0 ? pa_decode_window_fp8 : pa_attention_window_fp8;
                st = unlocked([&] {
                    return f(p.q, p.k, p.v, p.table(), p.lens(), p.ps, p.scale, ks, vs, win, sinks, out, p.shape,
                             longest, ws, bytes, p.call.stream);
                });
            } else {
                what = which == 0 ? "pa_decode_window" : "pa_attention_window";
                const auto f = which == 0 ? pa_decode_window : pa_attention_window;
                st = unlocked([&] {
                    return f(p.q, p.k, p.v, p.table(), p.lens(), p.ps, p.scale, win, sinks, out, p.shape, longest, ws,
                             bytes, p.call.stream);
                });
            }
        }
        if (raised(st, what))
            return nullptr;
        return THPVariable_Wrap(p.out);
    });
}

// The pools of a 4-bit call, [P, H_kv, page_size, 80].
pa_shape q4_pools(const at::Tensor& kp, const at::Tensor& vp, int32_t ps)
{
    if (kp.dim() != 4 || kp.size(2) != ps || kp.size(3) != kQ4Row || vp.sizes() != kp.sizes())
        value_error("4-bit page pools must be [P, H_kv, page_size, 80]");
    const int32_t heads = size32(kp.size(1), "H_kv");
    return pa_shape{0, heads, heads, int32_t(kQ4Elements), 0, size32(kp.size(0), "the number of pages"), 0};
}

// key, value, key_pages, value_pages, slot_mapping, page_size, stream
PyObject* append_q4(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        check_args(n, 7);
        const at::Tensor &key = tensor(a[0], "key"), &value = tensor(a[1], "value");
        const at::Tensor &kp = tensor(a[2], "key_pages"), &vp = tensor(a[3], "value_pages");
        const at::Tensor& slots = tensor(a[4], "slot_mapping");
        const int32_t ps = integer(a[5], "page_size");
        pa_shape shape = q4_pools(kp, vp, ps);
        if (key.dim() != 4 || key.size(1) != kp.size(1) || key.size(3) != kQ4Elements || value.sizes() != key.sizes())
            value_error("key and value must be [B, H_kv, L_new, 128], with the pools' H_kv");
        if (!shape_is(slots, {key.size(0), key.size(2)}))
            value_error("slot_mapping must be [B, L_new]");
        Call call(key, "key", a[6]);
        void *k = call.check(key, at::kBFloat16, "key"), *v = call.check(value, at::kBFloat16, "value");
        void *kpp = call.check(kp, at::kByte, "key_pages"), *vpp = call.check(vp, at::kByte, "value_pages");
        const int32_t* slot = static_cast<int32_t*>(call.check(slots, at::kInt, "slot_mapping"));
        shape.batch = size32(key.size(0), "B");
        shape.q_len = size32(key.size(2), "L_new");
        if (shape.batch > 0 && shape.q_len > 0) {
            const pa_status st = unlocked([&] { return pa_append_kv_q4(k, v, kpp, vpp, slot, ps, shape, call.stream); });
            if (raised(st, "pa_append_kv_q4"))
                return nullptr;
        }
        Py_RETURN_NONE;
    });
}

// key_pages, value_pages, block_table, context_lens, page_size, dense_len, key_dense, value_dense, stream
PyObject* gather_q4(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        check_args(n, 9);
        const at::Tensor &kp = tensor(a[0], "key_pages"), &vp = tensor(a[1], "value_pages");
        const at::Tensor &table = tensor(a[2], "block_table"), &lens = tensor(a[3], "context_lens");
        const int32_t ps = integer(a[4], "page_size"), len = integer(a[5], "dense_len");
        pa_shape shape = q4_pools(kp, vp, ps);
        const int64_t B = table.dim() == 2 ? table.size(0) : -1, H = kp.size(1);
        if (B < 0 || !shape_is(lens, {B}))
            value_error("block_table must be [B, max_pages] and context_lens [B]");
        if (len < 0)
            value_error("dense_len must not be negative");
        Call call(kp, "key_pages", a[8]);
        void *k = call.check(kp, at::kByte, "key_pages"), *v = call.check(vp, at::kByte, "value_pages");
        const int32_t* bt = static_cast<int32_t*>(call.check(table, at::kInt, "block_table"));
        const int32_t* cl = static_cast<int32_t*>(call.check(lens, at::kInt, "context_lens"));
        const at::Tensor kd = a[6] == Py_None ? call.make({B, H, len, kQ4Elements}, at::kBFloat16) : tensor(a[6], "key_dense");
        const at::Tensor vd = a[7] == Py_None ? call.make({B, H, len, kQ4Elements}, at::kBFloat16) : tensor(a[7], "value_dense");
        if (!shape_is(kd, {B, H, len, kQ4Elements}) || !shape_is(vd, {B, H, len, kQ4Elements}))
            value_error("dense buffers must be [B, H_kv, dense_len, 128]");
        void *ko = call.check(kd, at::kBFloat16, "key_dense"), *vo = call.check(vd, at::kBFloat16, "value_dense");
        shape.batch = size32(B, "B");
        shape.max_pages = size32(table.size(1), "max_pages");
        if (B > 0 && len > 0) {
            const pa_status st =
                unlocked([&] { return pa_gather_kv_q4(k, v, bt, cl, ps, shape, len, ko, vo, call.stream); });
            if (raised(st, "pa_gather_kv_q4"))
                return nullptr;
        }
        PyObject* x = THPVariable_Wrap(kd);
        PyObject* y = x ? THPVariable_Wrap(vd) : nullptr;
        PyObject* both = y ? PyTuple_Pack(2, x, y) : nullptr;
        Py_XDECREF(x);
        Py_XDECREF(y);
        return both;
    });
}

// which (0 decode, 1 prefill, 2 dispatch), query, key_pages, value_pages, block_table, context_lens,
// page_size, scale, causal, out, max_context_len, workspace, stream
PyObject* attention_q4(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        check_args(n, 13);
        const int32_t which = integer(a[0], "which");
        Paged p(a + 1, a[4], a[5], a[6], Pool::kQ4, a[7], a[9], a[12]);
        const int causal = truth(a[8]);
        const int32_t longest = integer(a[10], "max_context_len");
        size_t need = 0;
        if (a[11] == Py_None)
            need = which == 0   ? pa_decode_q4_workspace_bytes(p.shape)
                   : which == 1 ? pa_prefill_q4_workspace_bytes(p.shape, longest)
                                : pa_attention_q4_workspace_bytes(p.shape, longest);
        const at::Tensor workspace = p.call.workspace(a[11], need);
        const size_t bytes = workspace.nbytes();
        void *out = p.out.data_ptr(), *ws = workspace.data_ptr();
        const auto f = which == 0 ? pa_decode_q4 : which == 1 ? pa_prefill_q4 : pa_attention_q4;
        const pa_status st = unlocked([&] {
            return f(p.q, p.k, p.v, p.table(), p.lens(), p.ps, p.scale, causal, out, p.shape, longest, ws, bytes,
                     p.call.stream);
        });
        if (raised(st, which == 0 ? "pa_decode_q4" : which == 1 ? "pa_prefill_q4" : "pa_attention_q4"))
            return nullptr;
        return THPVariable_Wrap(p.out);
    });
}

// kind (0 bf16, 1 e4m3, 2 4-bit pools), query, key_pages, value_pages, block_table, context_lens,
// page_size, k_scale, v_scale, prefix_table, prefix_lens, prefix_starts, max_prefix_len (None: the
// table's width), scale, out, max_context_len, workspace, stream
PyObject* prefix(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        check_args(n, 18);
        const int32_t which = integer(a[0], "kind");
        const Pool kind = which == 0 ? Pool::kBf16 : which == 1 ? Pool::kE4m3 : Pool::kQ4;
        Paged p(a + 1, a[4], a[5], a[6], kind, a[13], a[14], a[17]);
        const at::Tensor &table = tensor(a[9], "prefix_table"), &lens = tensor(a[10], "prefix_lens"),
                         &starts = tensor(a[11], "prefix_starts");
        if (table.dim() != 2 || !shape_is(lens, {table.size(0)}) || !shape_is(starts, {table.size(0) + 1}))
            value_error("prefix_table must be [num_prefixes, prefix_pages], prefix_lens [num_prefixes] and "
                        "prefix_starts [num_prefixes + 1]");
        const int32_t* pt = static_cast<int32_t*>(p.call.check(table, at::kInt, "prefix_table"));
        const int32_t* pl = static_cast<int32_t*>(p.call.check(lens, at::kInt, "prefix_lens"));
        const int32_t* pst = static_cast<int32_t*>(p.call.check(starts, at::kInt, "prefix_starts"));
        const int32_t count = size32(table.size(0), "num_prefixes"), pages = size32(table.size(1), "prefix_pages");
        const int32_t most = a[12] == Py_None ? size32(int64_t(pages) * p.ps, "max_prefix_len")
                                              : integer(a[12], "max_prefix_len");
        const int32_t longest = integer(a[15], "max_context_len");
        const float ks = which == 1 ? float(number(a[7])) : 1.f, vs = which == 1 ? float(number(a[8])) : 1.f;
        size_t need = 0;
        if (a[16] == Py_None)
            need = (which == 0   ? pa_decode_prefix_workspace_bytes
                    : which == 1 ? pa_decode_prefix_fp8_workspace_bytes
                                 : pa_decode_prefix_q4_workspace_bytes)(p.shape, p.ps, count, most);
        const at::Tensor workspace = p.call.workspace(a[16], need);
        const size_t bytes = workspace.nbytes();
        void *out = p.out.data_ptr(), *ws = workspace.data_ptr();
        const pa_status st = unlocked([&] {
            return which == 1 ? pa_decode_prefix_fp8(p.q, p.k, p.v, p.table(), p.lens(), p.ps, p.scale, ks, vs, pt, pl,
                                                     pst, count, pages, most, out, p.shape, longest, ws, bytes,
                                                     p.call.stream)
                              : (which == 0 ? pa_decode_prefix : pa_decode_prefix_q4)(
                                    p.q, p.k, p.v, p.table(), p.lens(), p.ps, p.scale, pt, pl, pst, count, pages, most,
                                    out, p.shape, longest, ws, bytes, p.call.stream);
        });
        if (raised(st, which == 0 ? "pa_decode_prefix" : which == 1 ? "pa_decode_prefix_fp8" : "pa_decode_prefix_q4"))
            return nullptr;
        return THPVariable_Wrap(p.out);
    });
}

// query, key_pages, value_pages, weight_pages, block_table, context_lens, page_size, k_scale,
// v_scale (None: bf16 pools), max_context_len, decay, scale, causal, out, workspace, stream
PyObject* weights(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        check_args(n, 16);
        const bool fp8 = a[7] != Py_None;
        const at::Tensor &kp = tensor(a[1], "key_pages"), &wp = tensor(a[3], "weight_pages");
        if (kp.dim() != 4 || !shape_is(wp, kp.sizes().slice(0, 3)))
            value_error("weight_pages must be [P, H_kv, page_size]");
        Paged p(a, a[4], a[5], a[6], fp8, a[11], a[13], a[15]);
        float* w = static_cast<float*>(p.call.check(wp, at::kFloat, "weight_pages"));
        const int32_t longest = integer(a[9], "max_context_len");
        const float decay = float(number(a[10]));
        const int causal = truth(a[12]);
        const float ks = fp8 ? float(number(a[7])) : 1.f, vs = fp8 ? float(number(a[8])) : 1.f;
        const at::Tensor workspace = p.call.workspace(
            a[14], a[14] == Py_None ? pa_decode_weights_workspace_bytes(p.shape, longest) : 0);
        void *out = p.out.data_ptr(), *ws = workspace.data_ptr();
        const size_t bytes = workspace.nbytes();
        const pa_status st = unlocked([&] {
            return fp8 ? pa_decode_weights_fp8(p.q, p.k, p.v, w, p.table(), p.lens(), p.ps, p.scale, ks, vs, causal,
                                               decay, out, p.shape, longest, ws, bytes, p.call.stream)
                       : pa_decode_weights(p.q, p.k, p.v, w, p.table(), p.lens(), p.ps, p.scale, causal, decay, out,
                                           p.shape, longest, ws, bytes, p.call.stream);
        });
        if (raised(st, fp8 ? "pa_decode_weights_fp8" : "pa_decode_weights"))
            return nullptr;
        return THPVariable_Wrap(p.out);
    });
}

// key_pages, value_pages, weight_pages, block_table, context_lens, page_size, keep, sinks, recent,
// dst_block_table, kept, new_lens, fp8, stream
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        check_args(n, 14);
        const bool fp8 = truth(a[12]);
        const char* what = fp8 ? "pa_kv_evict_fp8" : "pa_kv_evict";
        const at::Tensor &kp = tensor(a[0], "key_pages"), &vp = tensor(a[1], "value_pages"),
                         &wp = tensor(a[2], "weight_pages"), &table = tensor(a[3], "block_table"),
                         &lens = tensor(a[4], "context_lens");
        const int32_t ps = integer(a[5], "page_size"), keep = integer(a[6], "keep"), sinks = integer(a[7], "sinks"),
                      recent = integer(a[8], "recent");
        if (kp.dim() != 4 || kp.size(2) != ps || vp.sizes() != kp.sizes())
            value_error("page pool shape does not match page_size");
        if (!shape_is(wp, kp.sizes().slice(0, 3)))
            value_error("weight_pages must be [P, H_kv, page_size]");
        const int64_t B = table.dim() == 2 ? table.size(0) : -1, H = kp.size(1);
        if (B < 0 || !shape_is(lens, {B}))
            value_error("block_table must be [B, max_pages] and context_lens [B]");
        const at::Tensor& dst = a[9] == Py_None ? table : tensor(a[9], "dst_block_table");
        if (dst.dim() != 2 || dst.size(0) != B)
            value_error("dst_block_table must be [B, dst_max_pages]");
        Call call(kp, "key_pages", a[13]);
        const at::ScalarType pool = fp8 ? at::kByte : at::kBFloat16;
        void *k = call.check(kp, pool, "key_pages"), *v = call.check(vp, pool, "value_pages");
        float* w = static_cast<float*>(call.check(wp, at::kFloat, "weight_pages"));
        const int32_t* bt = static_cast<int32_t*>(call.check(table, at::kInt, "block_table"));
        const int32_t* cl = static_cast<int32_t*>(call.check(lens, at::kInt, "context_lens"));
        const int32_t* dt = static_cast<int32_t*>(call.check(dst, at::kInt, "dst_block_table"));
        at::Tensor kept = a[10] == Py_None ? call.make({B, H, keep > 0 ? keep : 0}, at::kInt) : tensor(a[10], "kept");
        at::Tensor fresh = a[11] == Py_None ? call.make({B}, at::kInt) : tensor(a[11], "new_lens");
        if (a[10] != Py_None && !shape_is(kept, {B, H, keep}))
            value_error("kept must be [B, H_kv, keep]");
        if (!shape_is(fresh, {B}))
            value_error("new_lens must be [B]");
        int32_t* kept_ptr = static_cast<int32_t*>(call.check(kept, at::kInt, "kept"));
        int32_t* fresh_ptr = static_cast<int32_t*>(call.check(fresh, at::kInt, "new_lens"));
        if (B > 0) {
            const int32_t heads = size32(H, "H_kv");
            const pa_shape shape{size32(B, "B"), heads, heads, size32(kp.size(3), "D"), 1,
                                 size32(kp.size(0), "the number of pages"), size32(table.size(1), "max_pages")};
            const int32_t dst_pages = size32(dst.size(1), "dst_max_pages");
            const pa_status st = unlocked([&] {
                return (fp8 ? pa_kv_evict_fp8 : pa_kv_evict)(k, v, w, bt, cl, ps, keep, sinks, recent, dt, dst_pages,
                                                             kept_ptr, fresh_ptr, shape, call.stream);
            });
            if (raised(st, what))
                return nullptr;
        }
        PyObject* x = THPVariable_Wrap(kept);
        PyObject* y = x ? THPVariable_Wrap(fresh) : nullptr;
        PyObject* both = y ? PyTuple_Pack(2, x, y) : nullptr;
        Py_XDECREF(x);
        Py_XDECREF(y);
        return both;
    });
}

PyObject* set_error(PyObject*, PyObject* cls)
{
    Py_INCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F* f)
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef g_methods[] = {
    {"append", fast(append), METH_FASTCALL, "pa_qk_norm_rope_append and its e4m3 form"},
    {"window", fast(window), METH_FASTCALL, "the sliding-window calls"},
    {"weights", fast(weights), METH_FASTCALL, "pa_decode_weights and its e4m3 form"},
    {"evict", fast(evict), METH_FASTCALL, "pa_kv_evict and its e4m3 form"},
    {"append_q4", fast(append_q4), METH_FASTCALL, "pa_append_kv_q4"},
    {"gather_q4", fast(gather_q4), METH_FASTCALL, "pa_gather_kv_q4"},
    {"attention_q4", fast(attention_q4), METH_FASTCALL, "the attention calls over 4-bit pools"},
    {"prefix", fast(prefix), METH_FASTCALL, "pa_decode_prefix and its e4m3 and 4-bit forms"},
    {"set_error", set_error, METH_O, "the class raised for a pa_status"},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_pagedattn_calls", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pagedattn_calls() { return PyModule_Create(&g_module); }
