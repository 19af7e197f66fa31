// binding.cpp - the Python binding of the paged cache's writers, of the
// block-scaled cache's readers, of the norms with rotation and of the attention
// over contiguous keys, as a CPython module over the C ABI.
//
// It checks tensors, takes their pointers and sizes and the current CUDA
// stream, allocates the outputs that are not given, and calls the C ABI.  A
// call has some ten tensors and thirty arguments, and its kernels run for a few
// microseconds on small batches: marshalled in Python with ctypes the same
// checks took 17-35 us a call on the GPU's host, here about 3 us with the launch.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <initializer_list>
#include <stdexcept>
#include <string>
#include <utility>

#include "../../include/attn.h"

namespace {

struct Refused : std::invalid_argument {   // becomes a ValueError
    using std::invalid_argument::invalid_argument;
};

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

// The arguments of a call; an index past the last one reads as None.
struct Args {
    PyObject* const* a;
    Py_ssize_t n;
    bool none(int i) const { return i >= n || a[i] == Py_None; }
    const at::Tensor& tensor(const char* name, int i) const {
        if (none(i) || !THPVariable_Check(a[i])) throw Refused(std::string(name) + " must be a tensor");
        return THPVariable_Unpack(a[i]);
    }
    bool truth(int i) const {
        const int t = none(i) ? 0 : PyObject_IsTrue(a[i]);
        if (t < 0) throw Refused("a truth value was expected");
        return t != 0;
    }
};

// The device of the call's tensors, which has to be the current one.
at::Device call_device(const at::Tensor& t) {
    if (!t.is_cuda() || t.get_device() != c10::cuda::current_device())
        throw Refused("tensors must be on the current CUDA device");
    return t.device();
}

// Forward calls record nothing for torch's differentiation: where it would expect
// them to (an input wants a gradient, gradients are on), they are refused, so that
// no weight goes without its gradient unnoticed.
void expect_unrecorded(const Args& args, std::initializer_list<std::pair<const char*, int>> inputs, const char* advice) {
    if (!c10::GradMode::is_enabled()) return;
    for (const auto& [name, i] : inputs)
        if (!args.none(i) && THPVariable_Check(args.a[i]) && THPVariable_Unpack(args.a[i]).requires_grad())
            throw Refused(std::string(name) + " requires a gradient, which this call does not record: call it under torch.no_grad()" + advice);
}

// An output that is read or written as something else of the same call, too.  (Parts of
// one buffer whose rows lie between each other's are fine.)
void expect_apart(const char* name, const void* out, std::initializer_list<std::pair<const char*, const void*>> others) {
    for (const auto& [other, at] : others)
        if (out != nullptr && out == at) throw Refused(std::string(name) + " must not be the same memory as " + other);
}

// A dense tensor's pointer, after checks of its device, type and shape (-1: any size).
void* expect(const char* name, const at::Tensor& t, at::Device device, std::initializer_list<int64_t> shape,
             at::ScalarType type, at::ScalarType other = at::ScalarType::Undefined) {
    if (t.device() != device || !t.is_contiguous())
        throw Refused(std::string(name) + " must be a contiguous tensor on " + device.str());
    if (t.scalar_type() != type && t.scalar_type() != other)
        throw Refused(std::string(name) + " must be " + at::toString(type) +
                      (other == at::ScalarType::Undefined ? "" : std::string(" or ") + at::toString(other)) + ", not " +
                      at::toString(t.scalar_type()));
    bool same = static_cast<size_t>(t.dim()) == shape.size();
    size_t i = 0;
    for (const int64_t want : shape) {
        same = same && (want == -1 || t.size(static_cast<int64_t>(i)) == want);
        ++i;
    }
    if (!same)
        throw Refused(std::string(name) + " must have the shape " +
                      shape_text(at::IntArrayRef(shape.begin(), shape.size())) + " (-1: any), not " +
                      shape_text(t.sizes()));
    return t.data_ptr();
}

at::Tensor make_empty(at::IntArrayRef shape, at::ScalarType type, at::Device device) {
    return at::Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
}

int small(const char* name, int64_t n) {
    if (n > 0x7FFFFFFF) throw Refused(std::string(name) + " is too large");
    return static_cast<int>(n);
}

// A cache of block-scaled e4m3 codes: arguments i .. i + 3.
struct BlockCache {
    void *k, *v;
    float *k_scale, *v_scale;
    int pages, page_size, hkv, d, block;
};

BlockCache block_cache(const Args& args, int i, at::Device device) {
    constexpr auto u8 = at::ScalarType::Byte, e4m3 = at::ScalarType::Float8_e4m3fn;
    const at::Tensor &k = args.tensor("k_cache", i), &v = args.tensor("v_cache", i + 1);
    const at::Tensor &ks = args.tensor("k_scale", i + 2), &vs = args.tensor("v_scale", i + 3);
    BlockCache c;
    c.k = expect("k_cache", k, device, {-1, -1, -1, -1}, u8, e4m3);
    const int64_t pages = k.size(0), page = k.size(1), hkv = k.size(2), d = k.size(3);
    c.v = expect("v_cache", v, device, {pages, page, hkv, d}, u8, e4m3);
    c.k_scale = static_cast<float*>(expect("k_scale", ks, device, {pages, -1, hkv}, at::ScalarType::Float));
    const int64_t blocks = ks.size(1);
    if (blocks == 0 || page % blocks != 0)
        throw Refused("k_scale has " + std::to_string(blocks) + " blocks for pages of " + std::to_string(page) + " tokens");
    c.v_scale = static_cast<float*>(expect("v_scale", vs, device, {pages, blocks, hkv}, at::ScalarType::Float));
    c.pages = small("k_cache", pages);
    c.page_size = small("k_cache", page);
    c.hkv = small("k_cache", hkv);
    c.d = small("k_cache", d);
    c.block = small("k_cache", page / blocks);
    return c;
}

// Lengths and page lists of the sequences: arguments seq_lens, block_table, kv_indptr.
struct Sequences {
    const int32_t *lens, *table, *indptr;
    int count, width;
};

Sequences sequences(const Args& args, int lens_at, int table_at, int indptr_at, int64_t count, at::Device device) {
    const at::Tensor &lens = args.tensor("seq_lens", lens_at), &table = args.tensor("block_table", table_at);
    constexpr auto i32 = at::ScalarType::Int;
    if (count < 0) count = lens.numel();
    Sequences s{};
    s.count = small("seq_lens", count);
    s.lens = static_cast<const int32_t*>(expect("seq_lens", lens, device, {count}, i32));
    if (args.none(indptr_at)) {
        s.table = static_cast<const int32_t*>(expect("block_table", table, device, {count, -1}, i32));
        s.width = small("block_table", table.size(1));
    } else {
        s.table = static_cast<const int32_t*>(expect("block_table (with kv_indptr)", table, device, {-1}, i32));
        s.indptr = static_cast<const int32_t*>(
            expect("kv_indptr", args.tensor("kv_indptr", indptr_at), device, {count + 1}, i32));
    }
    return s;
}

int32_t* optional_int(const Args& args, const char* name, int i, int64_t count, at::Device device) {
    if (args.none(i)) return nullptr;
    return static_cast<int32_t*>(expect(name, args.tensor(name, i), device, {count}, at::ScalarType::Int));
}

// The device's status word: any int32 tensor's first element.
int32_t* status_word(const Args& args, int i, at::Device device) {
    if (args.none(i)) return nullptr;
    const at::Tensor& t = args.tensor("dev_status", i);
    if (t.device() != device || t.scalar_type() != at::ScalarType::Int || t.numel() < 1 || !t.is_contiguous())
        throw Refused("dev_status must be a contiguous int32 tensor on " + device.str());
    return static_cast<int32_t*>(t.data_ptr());
}

// Rows of bf16 heads: dense within a token, any distance from token to token.
void* token_rows(const char* name, const at::Tensor& x, at::Device device, long long& stride) {
    if (x.device() != device || x.scalar_type() != at::ScalarType::BFloat16 || x.dim() != 3)
        throw Refused(std::string(name) + " must be a bfloat16 tensor [tokens, heads, D] on " + device.str());
    if ((x.size(2) > 1 && x.stride(2) != 1) || (x.size(1) > 1 && x.stride(1) != x.size(2)))
        throw Refused(std::string(name) + ": the heads of a token must be dense");
    stride = x.size(0) > 1 ? x.stride(0) : x.size(1) * x.size(2);
    return x.data_ptr();
}

void* stream_of(at::Device device) { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }

void check(const char* fn, attn_status_t status) {
    if (status == ATTN_OK) return;
    // AttnError of the package, which carries the status
    PyObject* module = PyImport_ImportModule("causal_gqa_flashattention_attn_gb300");
    PyObject* type = module != nullptr ? PyObject_GetAttrString(module, "AttnError") : nullptr;
    PyObject* error = type != nullptr ? PyObject_CallFunction(type, "si", fn, static_cast<int>(status)) : nullptr;
    if (error != nullptr) PyErr_SetObject(type, error);
    Py_XDECREF(error);
    Py_XDECREF(type);
    Py_XDECREF(module);
    throw 0;   // the Python error is set
}

// Runs `body`; C++ exceptions become Python's, torch's their own (an allocation
// that fails is an OutOfMemoryError here as anywhere).
template <typename Body>
PyObject* guarded(Body body) {
    try {
        return body();
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception&) {
        torch::translate_exception_to_python(std::current_exception());
    } catch (int) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "call failed");
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

PyObject* wrap_or(const Args& args, int i, const at::Tensor& t) {
    if (!args.none(i)) {   // the caller's own object back
        Py_INCREF(args.a[i]);
        return args.a[i];
    }
    return THPVariable_Wrap(t);
}

// kv_append(q, k, v, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
// cos_sin, qo_indptr, kv_indptr, positions, interleaved, q_out, dev_status);
// k_scale None: a bf16 cache.
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        const Args args{a, n};
        const at::Tensor &k = args.tensor("k", 1), &v = args.tensor("v", 2);
        const at::Device device = call_device(k);
        long long qs = 0, ks = 0, vs = 0;
        void* kp = token_rows("k", k, device, ks);
        void* vp = token_rows("v", v, device, vs);
        if (v.sizes() != k.sizes()) throw Refused("k and v must have the same shape");
        const int64_t total = k.size(0), hkv = k.size(1), d = k.size(2);
        int64_t hq = hkv;
        void *qp = nullptr, *qop = nullptr;
        at::Tensor made;
        if (!args.none(0)) {
            const at::Tensor& q = args.tensor("q", 0);
            qp = token_rows("q", q, device, qs);
            hq = q.size(1);
            if (q.size(0) != total || q.size(2) != d)
                throw Refused("q, k and v must have the same tokens and head dimension");
            if (args.none(14)) made = make_empty({total, hq, d}, at::ScalarType::BFloat16, device);
            qop = expect("q_out", args.none(14) ? made : args.tensor("q_out", 14), device, {total, hq, d},
                         at::ScalarType::BFloat16);
        } else if (!args.none(14)) {
            throw Refused("q_out without q");
        }
        const Sequences s = sequences(args, 8, 7, 11, -1, device);
        const float* cs = nullptr;
        int64_t max_pos = 0, rot = 0;
        if (!args.none(9)) {
            const at::Tensor& t = args.tensor("cos_sin", 9);
            cs = static_cast<const float*>(expect("cos_sin", t, device, {-1, -1}, at::ScalarType::Float));
            max_pos = t.size(0);
            rot = t.size(1);
        }
        const int32_t* qo = optional_int(args, "qo_indptr", 10, s.count + 1, device);
        const int32_t* pos = optional_int(args, "positions", 12, total, device);
        int32_t* status = status_word(args, 15, device);
        const int t = small("k", total), h = small("q", hq), hk = small("k", hkv), dd = small("k", d);
        const int mp = small("cos_sin", max_pos), r = small("cos_sin", rot);
        if (args.none(5)) {
            constexpr auto bf16 = at::ScalarType::BFloat16;
            const at::Tensor &kc = args.tensor("k_cache", 3), &vc = args.tensor("v_cache", 4);
            void* kcp = expect("k_cache", kc, device, {-1, -1, hkv, d}, bf16);
            void* vcp = expect("v_cache", vc, device, {kc.size(0), kc.size(1), hkv, d}, bf16);
            check("attn_kv_append",
                  attn_kv_append(qp, kp, vp, qs, ks, vs, cs, mp, r, args.truth(13), pos, qo, s.lens, s.table, s.indptr,
                                 s.width, qop, kcp, vcp, s.count, t, h, hk, dd, small("k_cache", kc.size(0)),
                                 small("k_cache", kc.size(1)), status, stream_of(device)));
        } else {
            const BlockCache c = block_cache(args, 3, device);
            if (c.hkv != hkv || c.d != d) throw Refused("the cache's heads must be those of k and v");
            check("attn_kv_append_fp8_block",
                  attn_kv_append_fp8_block(qp, kp, vp, qs, ks, vs, cs, mp, r, args.truth(13), pos, qo, s.lens, s.table,
                                           s.indptr, s.width, qop, c.k, c.v, c.k_scale, c.v_scale, s.count, t, h, hk, dd,
                                           c.pages, c.page_size, c.block, status, stream_of(device)));
        }
        if (args.none(0)) Py_RETURN_NONE;
        return wrap_or(args, 14, made);
    });
}

// scale or 1 / sqrt(d)
float scale_or_default(const Args& args, int i, int d) {
    if (args.none(i)) return static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
    const double x = PyFloat_AsDouble(args.a[i]);
    if (x == -1.0 && PyErr_Occurred()) throw 0;
    return static_cast<float>(x);
}

PyObject* three(PyObject* a, PyObject* b, PyObject* c) {
    PyObject* t = a != nullptr && b != nullptr && c != nullptr ? PyTuple_New(3) : nullptr;
    if (t == nullptr) {
        Py_XDECREF(a);
        Py_XDECREF(b);
        Py_XDECREF(c);
        return nullptr;
    }
    PyTuple_SET_ITEM(t, 0, a);
    PyTuple_SET_ITEM(t, 1, b);
    PyTuple_SET_ITEM(t, 2, c);
    return t;
}

// decode(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, kv_indptr,
// scale, workspace, o, lse, dev_status) -> (o, lse, workspace)
PyObject* decode_fp8_block(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        const Args args{a, n};
        const at::Tensor& q = args.tensor("q", 0);
        const at::Device device = call_device(q);
        constexpr auto bf16 = at::ScalarType::BFloat16;
        const bool single = q.dim() == 3;
        if (!single && q.dim() != 4) throw Refused("q must be [B, Hq, D] or [B, q_len, Hq, D], not " + shape_text(q.sizes()));
        const int64_t bsz = q.size(0), nq = single ? 1 : q.size(1), hq = q.size(-2), d = q.size(-1);
        void* qp = single ? expect("q", q, device, {-1, -1, -1}, bf16) : expect("q", q, device, {-1, -1, -1, -1}, bf16);
        const BlockCache c = block_cache(args, 1, device);
        if (c.d != d) throw Refused("q and the cache must have the same head dimension");
        const Sequences s = sequences(args, 6, 5, 7, bsz, device);
        const int b = small("q", bsz), i = small("q", nq), h = small("q", hq);
        at::Tensor ws, o, lse;
        if (args.none(9)) {
            const size_t need = attn_decode_fp8_block_workspace_bytes(b, i, h, c.hkv, c.d);
            ws = make_empty({static_cast<int64_t>(std::max<size_t>(need, 16))}, at::ScalarType::Byte, device);
        }
        if (args.none(10)) o = make_empty(q.sizes(), bf16, device);
        if (args.none(11)) lse = make_empty(q.sizes().slice(0, q.dim() - 1), at::ScalarType::Float, device);
        const at::Tensor& wt = args.none(9) ? ws : args.tensor("workspace", 9);
        const at::Tensor& ot = args.none(10) ? o : args.tensor("o", 10);
        const at::Tensor& lt = args.none(11) ? lse : args.tensor("lse", 11);
        void* wp = expect("workspace", wt, device, {-1}, at::ScalarType::Byte);
        void* op = single ? expect("o", ot, device, {bsz, hq, d}, bf16) : expect("o", ot, device, {bsz, nq, hq, d}, bf16);
        float* lp = static_cast<float*>(single ? expect("lse", lt, device, {bsz, hq}, at::ScalarType::Float)
                                               : expect("lse", lt, device, {bsz, nq, hq}, at::ScalarType::Float));
        check("attn_decode_paged_fp8_block",
              attn_decode_paged_fp8_block(qp, c.k, c.v, c.k_scale, c.v_scale, s.table, s.indptr, s.width, s.lens, b, i, h,
                                          c.hkv, c.d, c.pages, c.page_size, c.block, scale_or_default(args, 8, c.d), wp,
                                          static_cast<size_t>(wt.numel()), op, lp,
                                          status_word(args, 12, device), stream_of(device)));
        return three(wrap_or(args, 10, o), wrap_or(args, 11, lse), wrap_or(args, 9, ws));
    });
}

// prefill(q, k_cache, v_cache, k_scale, v_scale, qo_indptr, block_table, seq_lens,
// kv_indptr, max_kv_rows, scale, workspace, o, lse, dev_status) -> (o, lse, workspace)
PyObject* prefill_fp8_block(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        const Args args{a, n};
        const at::Tensor& q = args.tensor("q", 0);
        const at::Device device = call_device(q);
        constexpr auto bf16 = at::ScalarType::BFloat16;
        void* qp = expect("q", q, device, {-1, -1, -1}, bf16);
        const int64_t total = q.size(0), hq = q.size(1), d = q.size(2);
        const BlockCache c = block_cache(args, 1, device);
        if (c.d != d) throw Refused("q and the cache must have the same head dimension");
        const Sequences s = sequences(args, 7, 6, 8, -1, device);
        const at::Tensor& qo = args.tensor("qo_indptr", 5);
        const int32_t* qop = static_cast<const int32_t*>(
            expect("qo_indptr", qo, device, {static_cast<int64_t>(s.count) + 1}, at::ScalarType::Int));
        // by default all that the page lists hold: sequences that share pages may have more rows than the pool
        long long rows = (s.indptr != nullptr ? args.tensor("block_table", 6).numel()
                                              : static_cast<long long>(s.count) * s.width) * c.page_size;
        if (!args.none(9)) {
            rows = PyLong_AsLongLong(args.a[9]);
            if (rows == -1 && PyErr_Occurred()) throw 0;
        } else if (rows > 0x7FFFFFFF || (rows > 0 && s.count > 0 && c.hkv > 0 && c.d == 128 &&
                                         attn_prefill_fp8_block_workspace_bytes(s.count, static_cast<int>(rows), c.hkv, c.d) == 0)) {
            throw Refused("the page lists hold " + std::to_string(rows) +
                          " tokens, more than a workspace may: max_kv_rows has to be given");
        }
        const int max_rows = small("max_kv_rows", std::max(rows, -1LL));
        at::Tensor ws, o, lse;
        if (args.none(11)) {
            const size_t need = attn_prefill_fp8_block_workspace_bytes(s.count, max_rows, c.hkv, c.d);
            ws = make_empty({static_cast<int64_t>(std::max<size_t>(need, 16))}, at::ScalarType::Byte, device);
        }
        if (args.none(12)) o = make_empty(q.sizes(), bf16, device);
        if (args.none(13)) lse = make_empty({total, hq}, at::ScalarType::Float, device);
        const at::Tensor& wt = args.none(11) ? ws : args.tensor("workspace", 11);
        void* wp = expect("workspace", wt, device, {-1}, at::ScalarType::Byte);
        void* op = expect("o", args.none(12) ? o : args.tensor("o", 12), device, {total, hq, d}, bf16);
        float* lp = static_cast<float*>(expect("lse", args.none(13) ? lse : args.tensor("lse", 13), device, {total, hq},
                                               at::ScalarType::Float));
        check("attn_prefill_paged_fp8_block",
              attn_prefill_paged_fp8_block(qp, c.k, c.v, c.k_scale, c.v_scale, qop, s.table, s.indptr, s.width, s.lens,
                                           s.count, small("q", total), small("q", hq), c.hkv, c.d, c.pages, c.page_size,
                                           c.block, max_rows, scale_or_default(args, 10, c.d), wp,
                                           static_cast<size_t>(wt.numel()), op, lp,
                                           status_word(args, 14, device), stream_of(device)));
        return three(wrap_or(args, 12, o), wrap_or(args, 13, lse), wrap_or(args, 11, ws));
    });
}

// float argument or a default
float number_or(const Args& args, int i, double otherwise) {
    if (args.none(i)) return static_cast<float>(otherwise);
    const double x = PyFloat_AsDouble(args.a[i]);
    if (x == -1.0 && PyErr_Occurred()) throw 0;
    return static_cast<float>(x);
}

PyObject* tuple_of(std::initializer_list<PyObject*> items) {
    bool good = true;
    for (PyObject* x : items) good = good && x != nullptr;
    PyObject* t = good ? PyTuple_New(static_cast<Py_ssize_t>(items.size())) : nullptr;
    Py_ssize_t i = 0;
    for (PyObject* x : items) {
        if (t != nullptr) PyTuple_SET_ITEM(t, i++, x);
        else Py_XDECREF(x);
    }
    return t;
}

// An output: the caller's tensor at argument i, or a new one; None where `there` is not.
PyObject* wrap_where(bool there, const Args& args, int i, const at::Tensor& t) {
    if (!there) Py_RETURN_NONE;
    return wrap_or(args, i, t);
}

// One side, queries (0) or keys (1), of a norm with rotation.
struct NormSide {
    void *x = nullptr, *dy = nullptr, *out = nullptr, *weight = nullptr;
    float* d_weight = nullptr;
    long long x_stride = 0, dy_stride = 0, out_stride = 0;
    int64_t tokens = 0, heads = 0, d = 0;
    bool there = false;
    attn_dtype_t type = ATTN_F32;
    at::Tensor made, d_made;
};

// Arguments: x, dy (or -1), weight, output, the weight's gradient (or -1).
NormSide norm_side(const Args& args, const char* name, const char* dy_name, const char* w_name, const char* out_name,
                   const char* dw_name, int x_at, int dy_at, int w_at, int out_at, int dw_at, at::Device device) {
    NormSide s;
    if (args.none(x_at)) {
        for (const int i : {dy_at, w_at, out_at, dw_at})
            if (i >= 0 && !args.none(i)) throw Refused(std::string(name) + " is absent, but not all that belongs to it");
        return s;
    }
    s.there = true;
    const at::Tensor& x = args.tensor(name, x_at);
    s.x = token_rows(name, x, device, s.x_stride);
    s.tokens = x.size(0), s.heads = x.size(1), s.d = x.size(2);
    if (dy_at >= 0) {
        const at::Tensor& dy = args.tensor(dy_name, dy_at);
        s.dy = token_rows(dy_name, dy, device, s.dy_stride);
        if (dy.sizes() != x.sizes()) throw Refused(std::string(dy_name) + " must have the shape of " + name);
    }
    if (args.none(out_at)) {
        s.made = make_empty(x.sizes(), at::ScalarType::BFloat16, device);
        s.out = token_rows(out_name, s.made, device, s.out_stride);
    } else {
        const at::Tensor& out = args.tensor(out_name, out_at);
        s.out = token_rows(out_name, out, device, s.out_stride);
        if (out.sizes() != x.sizes()) throw Refused(std::string(out_name) + " must have the shape of " + name);
    }
    if (!args.none(w_at)) {
        const at::Tensor& w = args.tensor(w_name, w_at);
        s.weight = expect(w_name, w, device, {s.d}, at::ScalarType::Float, at::ScalarType::BFloat16);
        s.type = w.scalar_type() == at::ScalarType::Float ? ATTN_F32 : ATTN_BF16;
        if (dw_at >= 0) {
            if (args.none(dw_at)) s.d_made = make_empty({s.d}, at::ScalarType::Float, device);
            s.d_weight = static_cast<float*>(expect(dw_name, args.none(dw_at) ? s.d_made : args.tensor(dw_name, dw_at), device,
                                                    {s.d}, at::ScalarType::Float));
        }
    } else if (dw_at >= 0 && !args.none(dw_at)) {
        throw Refused(std::string(dw_name) + " without " + w_name);
    }
    return s;
}

// What both calls share: sizes, the weights' type, the rotation's table.
struct NormCall {
    const float* cos_sin = nullptr;
    const int32_t* positions = nullptr;
    int max_pos = 0, rot = 0, total = 0, hq = 0, hkv = 0, d = 0;
    attn_dtype_t type = ATTN_F32;
};

NormCall norm_call(const Args& args, const NormSide& q, const NormSide& k, int table_at, int positions_at, at::Device device) {
    const NormSide& one = q.there ? q : k;
    if (q.there && k.there && (q.tokens != k.tokens || q.d != k.d))
        throw Refused("q and k must have the same tokens and head dimension");
    if (q.weight != nullptr && k.weight != nullptr && q.type != k.type) throw Refused("q_weight and k_weight must have one type");
    NormCall c;
    c.total = small("q", one.tokens);
    c.hq = small("q", q.heads);
    c.hkv = small("k", k.heads);
    c.d = small("q", one.d);
    c.type = q.weight != nullptr ? q.type : k.type;
    if (!args.none(table_at)) {
        const at::Tensor& t = args.tensor("cos_sin", table_at);
        c.cos_sin = static_cast<const float*>(expect("cos_sin", t, device, {-1, -1}, at::ScalarType::Float));
        c.max_pos = small("cos_sin", t.size(0));
        c.rot = small("cos_sin", t.size(1));
    }
    c.positions = optional_int(args, "positions", positions_at, one.tokens, device);
    return c;
}

// qk_norm_rope(q, k, q_weight, k_weight, eps, cos_sin, positions, interleaved, q_out,
// k_out, dev_status) -> (q_out, k_out)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        const Args args{a, n};
        expect_unrecorded(args, {{"q", 0}, {"k", 1}, {"q_weight", 2}, {"k_weight", 3}},
                          " or in a torch.autograd.Function, with attn_qk_norm_rope_bwd for the gradient");
        const at::Device device = call_device(args.tensor("q or k", args.none(0) ? 1 : 0));
        const NormSide q = norm_side(args, "q", "", "q_weight", "q_out", "", 0, -1, 2, 8, -1, device);
        const NormSide k = norm_side(args, "k", "", "k_weight", "k_out", "", 1, -1, 3, 9, -1, device);
        expect_apart("q_out", q.out, {{"k", k.x}, {"k_out", k.out}});
        expect_apart("k_out", k.out, {{"q", q.x}});
        const NormCall c = norm_call(args, q, k, 5, 6, device);
        check("attn_qk_norm_rope",
              attn_qk_norm_rope(q.x, k.x, q.x_stride, k.x_stride, q.weight, k.weight, c.type, number_or(args, 4, 1e-6),
                                c.cos_sin, c.max_pos, c.rot, args.truth(7), c.positions, q.out, k.out, q.out_stride,
                                k.out_stride, c.total, c.hq, c.hkv, c.d, status_word(args, 10, device), stream_of(device)));
        return tuple_of({wrap_where(q.there, args, 8, q.made), wrap_where(k.there, args, 9, k.made)});
    });
}

// qk_norm_rope_bwd(d_q_out, d_k_out, q, k, q_weight, k_weight, eps, cos_sin, positions,
// interleaved, workspace, d_q, d_k, d_q_weight, d_k_weight, dev_status)
// -> (d_q, d_k, d_q_weight, d_k_weight, workspace)
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        const Args args{a, n};
        const at::Device device = call_device(args.tensor("q or k", args.none(2) ? 3 : 2));
        const NormSide q = norm_side(args, "q", "d_q_out", "q_weight", "d_q", "d_q_weight", 2, 0, 4, 11, 13, device);
        const NormSide k = norm_side(args, "k", "d_k_out", "k_weight", "d_k", "d_k_weight", 3, 1, 5, 12, 14, device);
        expect_apart("d_q", q.out, {{"k", k.x}, {"d_k_out", k.dy}, {"d_k", k.out}});
        expect_apart("d_k", k.out, {{"q", q.x}, {"d_q_out", q.dy}});
        const NormCall c = norm_call(args, q, k, 7, 8, device);
        at::Tensor ws;
        if (args.none(10)) {
            const size_t need = attn_qk_norm_rope_bwd_workspace_bytes(c.total, c.hq, c.hkv, c.d);
            ws = make_empty({static_cast<int64_t>(std::max<size_t>(need, 16))}, at::ScalarType::Byte, device);
        }
        const at::Tensor& wt = args.none(10) ? ws : args.tensor("workspace", 10);
        void* wp = expect("workspace", wt, device, {-1}, at::ScalarType::Byte);
        check("attn_qk_norm_rope_bwd",
              attn_qk_norm_rope_bwd(q.dy, k.dy, q.dy_stride, k.dy_stride, q.x, k.x, q.x_stride, k.x_stride, q.weight, k.weight,
                                    c.type, number_or(args, 6, 1e-6), c.cos_sin, c.max_pos, c.rot, args.truth(9), c.positions,
                                    q.out, k.out, q.out_stride, k.out_stride, q.d_weight, k.d_weight, c.total, c.hq, c.hkv,
                                    c.d, wp, static_cast<size_t>(wt.numel()), status_word(args, 15, device),
                                    stream_of(device)));
        return tuple_of({wrap_where(q.there, args, 11, q.made), wrap_where(k.there, args, 12, k.made),
                         wrap_where(q.d_weight != nullptr, args, 13, q.d_made),
                         wrap_where(k.d_weight != nullptr, args, 14, k.d_made), wrap_or(args, 10, ws)});
    });
}

// Queries, keys and values of a ragged batch over contiguous keys, arguments i, i + 1, i + 2;
// its offsets and lengths, arguments at, at + 1, at + 2.
struct Ragged {
    void *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    const int32_t *qo, *kv, *lens;
    int count, total_q, total_kv, hq, hkv, d;
    at::IntArrayRef q_shape, k_shape;
};

Ragged ragged(const Args& args, int i, int at, at::Device device) {
    Ragged r{};
    const at::Tensor &q = args.tensor("q", i), &k = args.tensor("k", i + 1), &v = args.tensor("v", i + 2);
    r.q = token_rows("q", q, device, r.q_stride);
    r.k = token_rows("k", k, device, r.k_stride);
    r.v = token_rows("v", v, device, r.v_stride);
    if (v.sizes() != k.sizes()) throw Refused("k and v must have the same shape");
    if (q.size(2) != k.size(2)) throw Refused("q and k must have the same head dimension");
    r.q_shape = q.sizes(), r.k_shape = k.sizes();
    const at::Tensor& qo = args.tensor("qo_indptr", at);
    const int64_t count = qo.numel() - 1;
    r.qo = static_cast<const int32_t*>(expect("qo_indptr", qo, device, {-1}, at::ScalarType::Int));
    if (count < 1) throw Refused("qo_indptr must hold at least one sequence");
    r.kv = static_cast<const int32_t*>(expect("kv_indptr", args.tensor("kv_indptr", at + 1), device, {count + 1}, at::ScalarType::Int));
    r.lens = optional_int(args, "kv_lens", at + 2, count, device);
    r.count = small("qo_indptr", count);
    r.total_q = small("q", q.size(0));
    r.total_kv = small("k", k.size(0));
    r.hq = small("q", q.size(1));
    r.hkv = small("k", k.size(1));
    r.d = small("q", q.size(2));
    return r;
}

// varlen_fwd(q, k, v, qo_indptr, kv_indptr, kv_lens, causal, scale, workspace, o, lse,
// dev_status) -> (o, lse, workspace)
PyObject* varlen_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        const Args args{a, n};
        expect_unrecorded(args, {{"q", 0}, {"k", 1}, {"v", 2}},
                          " or in a torch.autograd.Function, with attn_varlen_bwd for the gradient");
        const at::Device device = call_device(args.tensor("q", 0));
        const Ragged r = ragged(args, 0, 3, device);
        at::Tensor ws, o, lse;
        if (args.none(8)) {
            const size_t need = attn_varlen_fwd_workspace_bytes(r.count, r.total_q, r.total_kv, r.hq, r.hkv, r.d);
            ws = make_empty({static_cast<int64_t>(std::max<size_t>(need, 16))}, at::ScalarType::Byte, device);
        }
        if (args.none(9)) o = make_empty(r.q_shape, at::ScalarType::BFloat16, device);
        if (args.none(10)) lse = make_empty({r.total_q, r.hq}, at::ScalarType::Float, device);
        const at::Tensor& wt = args.none(8) ? ws : args.tensor("workspace", 8);
        void* wp = expect("workspace", wt, device, {-1}, at::ScalarType::Byte);
        void* op = expect("o", args.none(9) ? o : args.tensor("o", 9), device, {r.total_q, r.hq, r.d}, at::ScalarType::BFloat16);
        float* lp = static_cast<float*>(expect("lse", args.none(10) ? lse : args.tensor("lse", 10), device, {r.total_q, r.hq},
                                               at::ScalarType::Float));
        expect_apart("o", op, {{"q", r.q}, {"k", r.k}, {"v", r.v}});
        check("attn_varlen_fwd",
              attn_varlen_fwd(r.q, r.k, r.v, r.q_stride, r.k_stride, r.v_stride, r.qo, r.kv, r.lens, args.truth(6), r.count,
                              r.total_q, r.total_kv, r.hq, r.hkv, r.d, scale_or_default(args, 7, r.d), wp,
                              static_cast<size_t>(wt.numel()), op, lp, status_word(args, 11, device), stream_of(device)));
        return tuple_of({wrap_or(args, 9, o), wrap_or(args, 10, lse), wrap_or(args, 8, ws)});
    });
}

// A gradient: the caller's rows (argument i) or new ones, of the shape of what it belongs to.
struct GradRows {
    void* at;
    long long stride;
    at::Tensor made;
};
GradRows grad_rows(const Args& args, const char* name, int i, at::IntArrayRef shape, at::Device device) {
    GradRows g;
    if (args.none(i)) g.made = make_empty(shape, at::ScalarType::BFloat16, device);
    const at::Tensor& t = args.none(i) ? g.made : args.tensor(name, i);
    g.at = token_rows(name, t, device, g.stride);
    if (t.sizes() != shape) throw Refused(std::string(name) + " must have the shape " + shape_text(shape) + ", not " + shape_text(t.sizes()));
    return g;
}

// varlen_bwd(d_o, q, k, v, o, lse, qo_indptr, kv_indptr, kv_lens, causal, scale, d_lse,
// workspace, d_q, d_k, d_v, dev_status) -> (d_q, d_k, d_v, workspace)
PyObject* varlen_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        const Args args{a, n};
        const at::Device device = call_device(args.tensor("q", 1));
        const Ragged r = ragged(args, 1, 6, device);
        long long do_stride = 0, o_stride = 0;
        const at::Tensor &d_o = args.tensor("d_o", 0), &o = args.tensor("o", 4);
        void* dop = token_rows("d_o", d_o, device, do_stride);
        void* op = token_rows("o", o, device, o_stride);
        if (d_o.sizes() != r.q_shape || o.sizes() != r.q_shape) throw Refused("d_o and o must have the shape of q");
        const float* lse = static_cast<const float*>(expect("lse", args.tensor("lse", 5), device, {r.total_q, r.hq}, at::ScalarType::Float));
        const float* d_lse = args.none(11) ? nullptr
                                           : static_cast<const float*>(expect("d_lse", args.tensor("d_lse", 11), device,
                                                                              {r.total_q, r.hq}, at::ScalarType::Float));
        at::Tensor ws;
        if (args.none(12)) {
            const size_t need = attn_varlen_bwd_workspace_bytes(r.count, r.total_q, r.total_kv, r.hq, r.hkv, r.d);
            ws = make_empty({static_cast<int64_t>(std::max<size_t>(need, 16))}, at::ScalarType::Byte, device);
        }
        const at::Tensor& wt = args.none(12) ? ws : args.tensor("workspace", 12);
        void* wp = expect("workspace", wt, device, {-1}, at::ScalarType::Byte);
        const GradRows dq = grad_rows(args, "d_q", 13, r.q_shape, device);
        const GradRows dk = grad_rows(args, "d_k", 14, r.k_shape, device);
        const GradRows dv = grad_rows(args, "d_v", 15, r.k_shape, device);
        expect_apart("d_q", dq.at, {{"d_o", dop}, {"q", r.q}, {"k", r.k}, {"v", r.v}, {"o", op}, {"d_k", dk.at}, {"d_v", dv.at}});
        expect_apart("d_k", dk.at, {{"d_o", dop}, {"q", r.q}, {"k", r.k}, {"v", r.v}, {"o", op}, {"d_v", dv.at}});
        expect_apart("d_v", dv.at, {{"d_o", dop}, {"q", r.q}, {"k", r.k}, {"v", r.v}, {"o", op}});
        check("attn_varlen_bwd",
              attn_varlen_bwd(dop, r.q, r.k, r.v, op, do_stride, r.q_stride, r.k_stride, r.v_stride, o_stride, lse, d_lse, r.qo,
                              r.kv, r.lens, args.truth(9), r.count, r.total_q, r.total_kv, r.hq, r.hkv, r.d,
                              scale_or_default(args, 10, r.d), wp, static_cast<size_t>(wt.numel()), dq.at, dk.at, dv.at,
                              dq.stride, dk.stride, dv.stride, status_word(args, 16, device), stream_of(device)));
        return tuple_of({wrap_or(args, 13, dq.made), wrap_or(args, 14, dk.made), wrap_or(args, 15, dv.made), wrap_or(args, 12, ws)});
    });
}

// cross_decode(q, k, v, kv_indptr, kv_lens, scale, workspace, o, lse, dev_status)
// -> (o, lse, workspace)
PyObject* cross_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        const Args args{a, n};
        expect_unrecorded(args, {{"q", 0}, {"k", 1}, {"v", 2}}, "");
        const at::Tensor& q = args.tensor("q", 0);
        const at::Device device = call_device(q);
        constexpr auto bf16 = at::ScalarType::BFloat16;
        const bool single = q.dim() == 3;
        if (!single && q.dim() != 4) throw Refused("q must be [B, Hq, D] or [B, q_len, Hq, D], not " + shape_text(q.sizes()));
        const int64_t bsz = q.size(0), nq = single ? 1 : q.size(1), hq = q.size(-2), d = q.size(-1);
        void* qp = single ? expect("q", q, device, {-1, -1, -1}, bf16) : expect("q", q, device, {-1, -1, -1, -1}, bf16);
        const at::Tensor &k = args.tensor("k", 1), &v = args.tensor("v", 2);
        long long ks = 0, vs = 0;
        void* kp = token_rows("k", k, device, ks);
        void* vp = token_rows("v", v, device, vs);
        if (v.sizes() != k.sizes()) throw Refused("k and v must have the same shape");
        if (k.size(2) != d) throw Refused("q and k must have the same head dimension");
        const int32_t* kv = static_cast<const int32_t*>(expect("kv_indptr", args.tensor("kv_indptr", 3), device, {bsz + 1}, at::ScalarType::Int));
        const int32_t* lens = optional_int(args, "kv_lens", 4, bsz, device);
        const int b = small("q", bsz), i = small("q", nq), h = small("q", hq), hkv = small("k", k.size(1)), dd = small("q", d);
        at::Tensor ws, o, lse;
        if (args.none(6)) {
            const size_t need = attn_cross_decode_workspace_bytes(b, i, h, hkv, dd);
            ws = make_empty({static_cast<int64_t>(std::max<size_t>(need, 16))}, at::ScalarType::Byte, device);
        }
        if (args.none(7)) o = make_empty(q.sizes(), bf16, device);
        if (args.none(8)) lse = make_empty(q.sizes().slice(0, q.dim() - 1), at::ScalarType::Float, device);
        const at::Tensor& wt = args.none(6) ? ws : args.tensor("workspace", 6);
        const at::Tensor& ot = args.none(7) ? o : args.tensor("o", 7);
        const at::Tensor& lt = args.none(8) ? lse : args.tensor("lse", 8);
        void* wp = expect("workspace", wt, device, {-1}, at::ScalarType::Byte);
        void* op = single ? expect("o", ot, device, {bsz, hq, d}, bf16) : expect("o", ot, device, {bsz, nq, hq, d}, bf16);
        float* lp = static_cast<float*>(single ? expect("lse", lt, device, {bsz, hq}, at::ScalarType::Float)
                                               : expect("lse", lt, device, {bsz, nq, hq}, at::ScalarType::Float));
        expect_apart("o", op, {{"q", qp}, {"k", kp}, {"v", vp}});
        check("attn_cross_decode",
              attn_cross_decode(qp, kp, vp, ks, vs, kv, lens, b, i, small("k", k.size(0)), h, hkv, dd,
                                scale_or_default(args, 5, dd), wp, static_cast<size_t>(wt.numel()), op, lp,
                                status_word(args, 9, device), stream_of(device)));
        return tuple_of({wrap_or(args, 7, o), wrap_or(args, 8, lse), wrap_or(args, 6, ws)});
    });
}

PyMethodDef methods[] = {
    {"cross_decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(cross_decode)), METH_FASTCALL, nullptr},
    {"varlen_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(varlen_bwd)), METH_FASTCALL, nullptr},
    {"varlen_fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(varlen_fwd)), METH_FASTCALL, nullptr},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(qk_norm_rope)), METH_FASTCALL, nullptr},
    {"qk_norm_rope_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(qk_norm_rope_bwd)), METH_FASTCALL, nullptr},
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(kv_append)), METH_FASTCALL, nullptr},
    {"decode_fp8_block", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(decode_fp8_block)), METH_FASTCALL, nullptr},
    {"prefill_fp8_block", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(prefill_fp8_block)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// The package compares torch_version with the torch that it runs with.
extern "C" PyMODINIT_FUNC PyInit__binding(void) {
    PyObject* m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
