// binding.cpp - the Python binding of the paged cache's writers and of the
// block-scaled cache's readers, as a CPython module over the C ABI.
//
// It checks tensors, takes their pointers and sizes and the current CUDA
// stream, allocates the outputs that are not given, and calls the C ABI.  A
// call has some ten tensors and thirty arguments, and its kernels run for a few
// microseconds on small batches: marshalled in Python with ctypes the same
// checks took 17-35 us a call on the GPU's host, here about 3 us with the launch.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
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

PyMethodDef methods[] = {
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
