// prefill_fp8_block.cu - ragged causal prefill over an e4m3 KV cache with one
// scale per block of tokens and KV head.
//
// The cached rows are first written as bf16 values, code * scale, into one
// contiguous copy, every sequence from a 128-row border on with zeros up to the
// next one, and the tensor-core prefill reads that copy by TMA as a cache of
// 128-token pages in list order: no tile of a sequence holds another's rows, so
// a NaN stays in its own sequence.  With a power-of-two scale the value is a
// bf16 number, so the copy rounds nothing; another scale's values are rounded
// once to bf16, as the tensor cores' operands must be; so are the softmax weights
// in the prefill (2^-8 of each: O is 0.0022 of its size off where it is rounded
// to bf16 alone, 0.0017).  The copy costs 1 byte read and 2 written per element
// once, against one read of the cache per query block otherwise.  That is dear
// where few queries follow many tokens: 8 sequences of 32768 cached tokens and 8
// KV heads, 64 new ones each, take 692 us and 1.1 GB of workspace (147.6 us of
// operations at the GEMM rate, 80 us of bytes).
//
// Bound: the tensor cores.  8 sequences, 9.7k queries of 32 heads over 23.8k
// tokens of 4 KV heads (360 GFLOP): 311.5 us, 1155 TFLOP/s, about 15 us of it
// the copy before the prefill's first tile.  Three short prompts: 17.5 us, the
// latency of two launches and of five KV tiles one after another.
#include <algorithm>

#include "paged.cuh"
#include "ptx.cuh"

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
    const int32_t* qo_indptr;
    Divisor page_div, block_div;
    int B, Hkv, max_rows, page_blocks;
    int q_block;      // query positions of a work item of the prefill
    int max_pairs, pair_bits;
    uint32_t* order;  // [max_pairs], work items' (sequence, query block) pairs, longest first
    int32_t* start;   // [B + 1], first pages of the copy
    int32_t* last;    // [B], rows in each sequence's last page
    int32_t* pairs;   // how many pairs there are
    uint4* k_copy;    // [copy rows, Hkv, D] bf16
    uint4* v_copy;
    int32_t* status;
};

// Eight codes times a scale as bf16.
__device__ __forceinline__ uint4 widen(uint2 w, float scale) {
    const uint32_t u[2] = {w.x, w.y};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t f = (i & 1) != 0 ? e4m3x2_hi_to_f16x2(u[i >> 1]) : e4m3x2_to_f16x2(u[i >> 1]);
        const __half2 h = *reinterpret_cast<const __half2*>(&f);
        const __nv_bfloat162 b = __floats2bfloat162_rn(__low2float(h) * scale, __high2float(h) * scale);
        r[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

constexpr int kWarps = kThreads / 32;
constexpr int kKeys = 512;     // KV tiles of a work item's pair; 511 and more together
constexpr int kMaxSeqs = 2048;
constexpr int kCopyRows = 4;   // rows of the copy that a warp takes: they lie in one block of one page

// The sum of `x` over the CTA's threads before this one, and over all of them.
template <typename T>
__device__ __forceinline__ T scan_cta(T x, T* warp_sums, T& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T incl = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const T v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    __syncthreads();   // the last scan's sums have been read
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    T before = incl - x;
    all = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    return before;
}

// A warp's rows on their way: kCopyRows of 32 vectors, keys and values.
constexpr int kWarpBytes = 2 * kCopyRows * 32 * 16;

struct Shared {
    uint8_t rows[kWarps * kWarpBytes];
    int count[kKeys];
    long long row_sums[kWarps];
    int sums[kWarps];
    // behind it: int start[B + 1], first pages of the copy, and rows[B] of each sequence, cut at max_rows in all
    __device__ __forceinline__ int* start() { return reinterpret_cast<int*>(this + 1); }
};

size_t shared_bytes(int B) { return sizeof(Shared) + (2 * static_cast<size_t>(B) + 1) * sizeof(int); }

// The sequences' places in the copy, by the whole CTA.
__device__ __forceinline__ void place_sequences(const Params& p, Shared& sh, bool flag) {
    int* start_of = sh.start();
    int* len_of = start_of + p.B + 1;
    long long rows_before = 0;
    int pages_before = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        int len = 0;
        if (b < p.B) {
            len = p.seq_lens[b];
            const long long cap = static_cast<long long>(page_count(p.list, b)) * p.list.page_size;
            if (len < 0 || len > cap) {
                if (flag) flag_status(p.status, ATTN_DEV_SEQ_TOO_LONG);
                len = len < 0 ? 0 : static_cast<int>(cap);
            }
        }
        long long all_rows;
        const long long first = rows_before + scan_cta<long long>(len, sh.row_sums, all_rows);
        rows_before += all_rows;
        if (first + len > p.max_rows) {
            if (flag) flag_status(p.status, ATTN_DEV_SEQ_TOO_LONG);
            len = first < p.max_rows ? static_cast<int>(p.max_rows - first) : 0;
        }
        int all_pages;
        const int start = pages_before + scan_cta<int>((len + kPage - 1) / kPage, sh.sums, all_pages);
        pages_before += all_pages;
        if (b < p.B) {
            start_of[b] = start;
            len_of[b] = len;
        }
    }
    if (threadIdx.x == 0) start_of[p.B] = pages_before;
    __syncthreads();
}

// One CTA, for the prefill: the places, and its work items longest first by a
// counting sort over their KV tiles; items of one length come in any order, each
// gives the same result wherever it runs.  (In the prefill's own CTAs, one warp
// each, the same sort takes 15 us for 300 pairs.)
__device__ __forceinline__ void sort_items(const Params& p, Shared& sh) {
    const int* start_of = sh.start();
    const int* len_of = start_of + p.B + 1;
    for (int k = threadIdx.x; k < kKeys; k += kThreads) sh.count[k] = 0;
    int pairs = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        int blocks = 0;
        if (b < p.B) {
            p.start[b] = start_of[b];
            p.last[b] = len_of[b] > 0 ? len_of[b] - (len_of[b] - 1) / kPage * kPage : 0;
            blocks = (p.qo_indptr[b + 1] - p.qo_indptr[b] + p.q_block - 1) / p.q_block;   // as the prefill counts
        }
        int all;
        scan_cta<int>(blocks, sh.sums, all);
        pairs += all;
    }
    if (threadIdx.x == 0) {
        p.start[p.B] = start_of[p.B];
        *p.pairs = pairs;
    }
    if (pairs > p.max_pairs) return;   // too many to sort: taken in sequence order
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // every pair and its key, one warp a sequence, lanes its query blocks
    auto each_pair = [&](auto use) {
        for (int b = warp; b < p.B; b += kWarps) {
            const int q_len = p.qo_indptr[b + 1] - p.qo_indptr[b], kv_len = len_of[b];
            for (int qb = lane; qb * p.q_block < q_len; qb += 32) {
                const int end = min(kv_len, min((qb + 1) * p.q_block, q_len) + kv_len - q_len);   // keys the block sees
                use(min(end > 0 ? (end + kPage - 1) / kPage : 0, kKeys - 1), b, qb);
            }
        }
    };
    each_pair([&](int key, int, int) { atomicAdd(&sh.count[key], 1); });
    __syncthreads();
    // first place of each key, from the longest down: two keys a thread
    const int key = kKeys - 1 - 2 * static_cast<int>(threadIdx.x);
    const int longer = sh.count[key], shorter = sh.count[key - 1];
    int all;
    const int at = scan_cta<int>(longer + shorter, sh.sums, all);
    sh.count[key] = at;
    sh.count[key - 1] = at + longer;
    __syncthreads();
    each_pair([&](int k, int b, int qb) {
        const int to = atomicAdd(&sh.count[k], 1);
        if (to < p.max_pairs) p.order[to] = (static_cast<uint32_t>(b) << p.pair_bits) | static_cast<uint32_t>(qb);
    });
}
static_assert(kKeys == 2 * kThreads, "two keys a thread");

// CTA (0, 0) sorts the prefill's work items; the others copy.  A warp takes
// kCopyRows rows and 32 of their 16-byte vectors of codes, both caches' all in
// flight at once (24k rows of 4 heads: 6 us sooner done than with one row ahead
// in registers), and writes 16 bytes a lane side by side.  Rows past a
// sequence's end or on a missing page are zeros.  The loop over rows stays
// rolled: with eight rows unrolled the kernel took 23 us instead of 7 on a short
// batch, most of it for fetching instructions that run once.
__global__ void __launch_bounds__(kThreads) fp8_block_copy_kernel(const Params p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    const bool sorts = blockIdx.x == 0;
    if (sorts && blockIdx.y != 0) return;
    place_sequences(p, sh, sorts);
    if (sorts) {
        sort_items(p, sh);
        return;
    }
    const int* start_of = sh.start();
    const int* len_of = start_of + p.B + 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint8_t* buf = sh.rows + warp * kWarpBytes;
    const int vecs = p.Hkv * (kD / 16);
    const uint32_t chunks = (vecs + 31) / 32;
    const uint32_t parts = static_cast<uint32_t>(start_of[p.B]) * (kPage / kCopyRows);   // fewer than 2^31 rows
    for (uint32_t part = (blockIdx.x - 1) * kWarps + warp; part < parts; part += (gridDim.x - 1) * kWarps) {
        const int copy_page = static_cast<int>(part / (kPage / kCopyRows));
        const int b = warp_rank(p.B, copy_page, lane, [&](int i) { return start_of[i]; });
        const int t0 = static_cast<int>(part - static_cast<uint32_t>(start_of[b]) * (kPage / kCopyRows)) * kCopyRows;
        const int len = len_of[b];
        const int entry = p.page_div.div(t0);
        const int page = t0 < len ? page_at(p.list, b, entry, page_count(p.list, b), lane == 0 ? p.status : nullptr) : -1;
        const int n = page >= 0 ? min(kCopyRows, len - t0) : 0;
        const int o = t0 - entry * p.list.page_size;
        const size_t slot = static_cast<size_t>(page >= 0 ? page : 0) * p.list.page_size + o;
        const size_t block = static_cast<size_t>(page >= 0 ? page : 0) * p.page_blocks + p.block_div.div(o);
        for (uint32_t c = blockIdx.y; c < chunks; c += gridDim.y) {
            const int v0 = static_cast<int>(c) * 32, m = min(32, vecs - v0);   // vectors [v0, v0 + m) of each row
            const uint4* k_in = reinterpret_cast<const uint4*>(p.k_cache) + slot * vecs + v0 + lane;
            const uint4* v_in = reinterpret_cast<const uint4*>(p.v_cache) + slot * vecs + v0 + lane;
            __syncwarp();   // the rows before these have been read
#pragma unroll
            for (int r = 0; r < kCopyRows; ++r) {
                const bool there = lane < m && r < n;
                uint8_t* at = buf + r * 512 + lane * 16;
                cp_async16(at, there ? static_cast<const void*>(k_in + static_cast<size_t>(r) * vecs) : p.k_cache, there ? 16 : 0);
                cp_async16(at + kCopyRows * 512, there ? static_cast<const void*>(v_in + static_cast<size_t>(r) * vecs) : p.v_cache, there ? 16 : 0);
            }
            // a lane writes vectors lane and lane + 32 of the 2 m of each row
            float ks[2] = {0.f, 0.f}, vs[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (n > 0 && lane + 32 * i < 2 * m) {
                    const size_t at = block * p.Hkv + (2 * v0 + lane + 32 * i) / (kD / 8);
                    ks[i] = __ldg(p.k_scale + at);
                    vs[i] = __ldg(p.v_scale + at);
                }
            uint4* k_out = p.k_copy + (static_cast<size_t>(part) * kCopyRows * vecs + v0) * 2 + lane;
            uint4* v_out = p.v_copy + (static_cast<size_t>(part) * kCopyRows * vecs + v0) * 2 + lane;
            cp_async_wait_all();
            __syncwarp();
#pragma unroll 1
            for (int r = 0; r < kCopyRows; ++r) {
                const uint2* kr = reinterpret_cast<const uint2*>(buf + r * 512) + lane;
                const uint2* vr = reinterpret_cast<const uint2*>(buf + (kCopyRows + r) * 512) + lane;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (lane + 32 * i < 2 * m) {
                        k_out[32 * i] = widen(kr[32 * i], ks[i]);
                        v_out[32 * i] = widen(vr[32 * i], vs[i]);
                    }
                k_out += 2 * vecs;
                v_out += 2 * vecs;
            }
        }
    }
}

// Rows of the copy: every sequence may leave kPage - 1 of them empty.
size_t copy_rows(int B, int max_kv_rows) {
    return (static_cast<size_t>(max_kv_rows) + static_cast<size_t>(B) * (kPage - 1) + kPage - 1) / kPage * kPage;
}

size_t copy_bytes(int B, int max_kv_rows, int Hkv) { return copy_rows(B, max_kv_rows) * Hkv * kD * 2; }

}  // namespace

// K copy, V copy, the work items' order, then the sequences' first pages, the
// rows in their last, and the number of pairs.
size_t prefill_fp8_block_workspace(int B, int max_kv_rows, int Hkv) {
    return 2 * copy_bytes(B, max_kv_rows, Hkv) + varlen_max_pairs() * sizeof(uint32_t) +
           ((2 * static_cast<size_t>(B) + 2) * sizeof(int32_t) + 15) / 16 * 16;
}

cudaError_t launch_prefill_fp8_block(const PrefillBlockArgs& a, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    if (a.B > kMaxSeqs) return cudaErrorInvalidValue;
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
    p.qo_indptr = a.qo_indptr;
    p.page_div = make_divisor(a.page_size);
    p.block_div = make_divisor(a.block_tokens);
    p.page_blocks = a.page_size / a.block_tokens;
    p.q_block = 2 * (128 / (a.Hq / a.Hkv));
    p.max_rows = a.max_kv_rows;
    p.k_copy = reinterpret_cast<uint4*>(w);
    const size_t bytes = copy_bytes(a.B, a.max_kv_rows, a.Hkv);
    p.v_copy = reinterpret_cast<uint4*>(w + bytes);
    p.order = reinterpret_cast<uint32_t*>(w + 2 * bytes);
    p.max_pairs = varlen_max_pairs();
    p.pair_bits = varlen_pair_bits();
    p.start = reinterpret_cast<int32_t*>(p.order + p.max_pairs);
    p.last = p.start + a.B + 1;
    p.pairs = p.last + a.B;
    p.status = a.dev_status;
    // gridDim.x: the sorting CTA and the copying ones, no more than the copy has parts for
    const size_t rows = copy_rows(a.B, a.max_kv_rows);
    const unsigned copying = static_cast<unsigned>(std::min<size_t>(static_cast<size_t>(sms) * 4, rows / (kCopyRows * kWarps)));
    static std::atomic<uint64_t> done{0};
    cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(fp8_block_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(shared_bytes(kMaxSeqs)));
    });
    if (e != cudaSuccess) return e;
    fp8_block_copy_kernel<<<dim3(1 + copying, std::min((a.Hkv * (kD / 16) + 31) / 32, 64)), kThreads, shared_bytes(a.B), stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // the copy as a cache of kPage-token pages in list order
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
    v.order = p.order;
    v.order_n = p.pairs;
    return launch_prefill_varlen_tc(v, stream);
}

}  // namespace gb300
