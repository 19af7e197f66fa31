// prefill_fp8_block.cu - ragged causal prefill over an e4m3 KV cache with one
// scale per block of tokens and KV head.
//
// The cached rows are first written as bf16 values, code * scale, into one
// contiguous copy, every sequence from a 128-row border on with zeros up to the
// next one, and the tensor-core prefill reads that copy by TMA as a cache of
// 128-token pages in list order: no tile of a sequence holds another's rows, so
// a NaN stays in its own sequence.  With a power-of-two scale the value is a bf16 number, so the copy
// rounds nothing; another scale's values are rounded once to bf16, as the
// tensor cores' operands must be.  The copy costs 1 byte read and 2 written
// per element once, against one read of the cache per query block otherwise.
#include "paged.cuh"

namespace gb300 {
namespace {

constexpr int kD = 128;
constexpr int kPage = 128;      // rows of a page of the copy: the prefill's KV tile
constexpr int kThreads = 256;

struct Params {
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const float* k_scale;
    const float* v_scale;
    PageList list;
    const int32_t* seq_lens;
    int B, Hkv, block, max_rows;
    int32_t* start;   // [B + 1], first pages of the copy
    int32_t* last;    // [B], rows in each sequence's last page
    uint4* k_copy;    // [copy rows, Hkv, D] bf16
    uint4* v_copy;
    int32_t* status;
};

// Each sequence's first page of the copy and the rows in its last page; one
// CTA.  Sequences past max_rows tokens in all are cut there.
__global__ void __launch_bounds__(1024) fp8_block_starts_kernel(const Params p) {
    __shared__ long long warp_rows[32];
    __shared__ int warp_pages[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long rows_before = 0;   // tokens and pages of the sequences of earlier rounds
    int pages_before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 1024) {
        const int b = b0 + threadIdx.x;
        int len = 0;
        if (b < p.B) {
            len = p.seq_lens[b];
            const long long cap = static_cast<long long>(page_count(p.list, b)) * p.list.page_size;
            if (len < 0 || len > cap) {
                flag_status(p.status, ATTN_DEV_SEQ_TOO_LONG);
                len = len < 0 ? 0 : static_cast<int>(cap);
            }
        }
        long long rows = len;   // inclusive sums over the warp, then over the CTA
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, rows, off);
            if (lane >= off) rows += v;
        }
        if (lane == 31) warp_rows[warp] = rows;
        __syncthreads();
        long long first = rows_before + rows - len;
        for (int w = 0; w < warp; ++w) first += warp_rows[w];
        if (first + len > p.max_rows) {
            flag_status(p.status, ATTN_DEV_SEQ_TOO_LONG);
            len = first < p.max_rows ? static_cast<int>(p.max_rows - first) : 0;
        }
        const int n = (len + kPage - 1) / kPage;
        int pages = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, pages, off);
            if (lane >= off) pages += v;
        }
        if (lane == 31) warp_pages[warp] = pages;
        __syncthreads();
        int start = pages_before + pages - n;
        for (int w = 0; w < warp; ++w) start += warp_pages[w];
        if (b < p.B) {
            p.start[b] = start;
            p.last[b] = n > 0 ? len - (n - 1) * kPage : 0;
        }
        for (int w = 0; w < 32; ++w) {
            rows_before += warp_rows[w];
            pages_before += warp_pages[w];
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) p.start[p.B] = pages_before;
}

// Sixteen codes times a scale as bf16.
__device__ __forceinline__ void widen(uint4 w, float scale, uint4& lo, uint4& hi) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t f = e4m3x2_to_f16x2(u[i >> 1] >> (16 * (i & 1)));
        const __half2 h = *reinterpret_cast<const __half2*>(&f);
        const __nv_bfloat162 b = __floats2bfloat162_rn(__low2float(h) * scale, __high2float(h) * scale);
        r[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    lo = make_uint4(r[0], r[1], r[2], r[3]);
    hi = make_uint4(r[4], r[5], r[6], r[7]);
}

// One warp per row of the copy; rows past a sequence's end or on a missing
// page are zeros.
__global__ void __launch_bounds__(kThreads) fp8_block_copy_kernel(const Params p) {
    const int lane = threadIdx.x & 31;
    const int vecs = p.Hkv * (kD / 16);
    const long long n_warps = static_cast<long long>(gridDim.x) * (kThreads / 32);
    const long long end = static_cast<long long>(p.start[p.B]) * kPage;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    for (long long r = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < end; r += n_warps) {
        const int page_row = static_cast<int>(r / kPage);
        const int b = warp_rank(p.B, page_row, lane, [&](int i) { return p.start[i]; });
        const int t = static_cast<int>(r - static_cast<long long>(p.start[b]) * kPage);
        const int len = (p.start[b + 1] - p.start[b] - 1) * kPage + p.last[b];
        long long slot = -1;
        if (t < len) {
            const int page = page_at(p.list, b, t / p.list.page_size, page_count(p.list, b),
                                     lane == 0 ? p.status : nullptr);
            if (page >= 0) slot = static_cast<long long>(page) * p.list.page_size + t % p.list.page_size;
        }
        for (int v = lane; v < vecs; v += 32) {
            const size_t dst = (static_cast<size_t>(r) * vecs + v) * 2;
            uint4 k0 = zero, k1 = zero, v0 = zero, v1 = zero;
            if (slot >= 0) {
                const size_t src = static_cast<size_t>(slot) * vecs + v;
                const size_t at = static_cast<size_t>(slot / p.block) * p.Hkv + v / (kD / 16);
                widen(__ldg(reinterpret_cast<const uint4*>(p.k_cache) + src), __ldg(p.k_scale + at), k0, k1);
                widen(__ldg(reinterpret_cast<const uint4*>(p.v_cache) + src), __ldg(p.v_scale + at), v0, v1);
            }
            p.k_copy[dst] = k0;
            p.k_copy[dst + 1] = k1;
            p.v_copy[dst] = v0;
            p.v_copy[dst + 1] = v1;
        }
    }
}

// Rows of the copy: every sequence may leave kPage - 1 of them empty.
size_t copy_rows(int B, int max_kv_rows) {
    return (static_cast<size_t>(max_kv_rows) + static_cast<size_t>(B) * (kPage - 1) + kPage - 1) / kPage * kPage;
}

size_t copy_bytes(int B, int max_kv_rows, int Hkv) { return copy_rows(B, max_kv_rows) * Hkv * kD * 2; }

}  // namespace

// K copy, V copy, then the sequences' first pages and the rows in their last.
size_t prefill_fp8_block_workspace(int B, int max_kv_rows, int Hkv) {
    return 2 * copy_bytes(B, max_kv_rows, Hkv) + ((2 * static_cast<size_t>(B) + 1) * sizeof(int32_t) + 15) / 16 * 16;
}

cudaError_t launch_prefill_fp8_block(const PrefillBlockArgs& a, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    uint8_t* w = static_cast<uint8_t*>(a.workspace);
    Params p;
    p.k_cache = static_cast<const uint8_t*>(a.k_cache);
    p.v_cache = static_cast<const uint8_t*>(a.v_cache);
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.list = PageList{a.block_table, a.kv_indptr, a.max_pages, a.num_pages, a.page_size};
    p.seq_lens = a.seq_lens;
    p.B = a.B;
    p.Hkv = a.Hkv;
    p.block = a.block_tokens;
    p.max_rows = a.max_kv_rows;
    p.k_copy = reinterpret_cast<uint4*>(w);
    const size_t bytes = copy_bytes(a.B, a.max_kv_rows, a.Hkv);
    p.v_copy = reinterpret_cast<uint4*>(w + bytes);
    p.start = reinterpret_cast<int32_t*>(w + 2 * bytes);
    p.last = p.start + a.B + 1;
    p.status = a.dev_status;
    fp8_block_starts_kernel<<<1, 1024, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    fp8_block_copy_kernel<<<sms * 8, kThreads, 0, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // the copy as a cache of kPage-token pages in list order
    const size_t rows = copy_rows(a.B, a.max_kv_rows);
    VarlenArgs v{};
    v.q = a.q;
    v.k_cache = p.k_copy;
    v.v_cache = p.v_copy;
    v.qo_indptr = a.qo_indptr;
    v.kv_indptr = p.start;
    v.kv_indices = p.start;   // not read: the copy is in list order
    v.kv_last_page_len = p.last;
    v.o = a.o;
    v.lse = a.lse;
    v.B = a.B;
    v.Hq = a.Hq;
    v.Hkv = a.Hkv;
    v.D = kD;
    v.total_q = a.total_q;
    v.num_pages = static_cast<int>(rows / kPage);
    v.page_size = kPage;
    v.scale = a.scale;
    v.dev_status = a.dev_status;
    v.kv_ws = a.workspace;
    v.max_kv_rows = static_cast<int>(rows);
    v.copied = true;
    return launch_prefill_varlen_tc(v, stream);
}

}  // namespace gb300
