// kv_append.cu - writes new keys and values into a paged cache, bf16 or e4m3
// with a scale per block of tokens and KV head, rotating queries and keys by
// their positions on the way.
//
// Rotation: with (c, s) = row `position` of the table, a pair (a, b) becomes
// (a c - b s, a s + b c); the pairs are elements (i, i + R/2) or (2i, 2i + 1)
// of the first R, the rest passes through.  Eight lanes take a row of 128
// elements, 16 each: lane l < R/16 holds the pairs 8l .. 8l + 7 in either
// order of the pairs, the other lanes hold what is not rotated.
//
// Blocks: a block is `block` tokens of one sequence, aligned to its start, of
// one KV head.  Its scale is the smallest power of two 2^e >= 2^-126 with
// max |x| / 2^e <= 448 (0 for a block of zeros), never smaller than the scale
// that the tokens already in the block have; if it grows, their codes are
// divided by the growth.  Powers of two make every product and quotient with
// a scale exact, so code * scale is off from x by one e4m3 rounding alone, old
// codes change only where they fall into e4m3's subnormals, and code * scale
// is a bf16 number.
#include "paged.cuh"

namespace gb300 {
namespace {

constexpr int kD = 128;
constexpr int kThreads = 256;

struct Params {
    const __nv_bfloat16* q;   // may be NULL (no queries)
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    long long q_stride, k_stride, v_stride;   // elements from token to token
    const float* cos_sin;
    const int32_t* positions;   // may be NULL
    const int32_t* qo_indptr;   // may be NULL: one token per sequence
    const int32_t* seq_lens;
    PageList list;
    __nv_bfloat16* q_out;
    void* k_cache;
    void* v_cache;
    float* k_scale;   // NULL: bf16 cache
    float* v_scale;
    int max_pos, rot, interleaved, B, total_q, Hq, Hkv, block, n_units;
    int32_t* status;
};

// Sixteen elements of a row as eight pairs: a[i], b[i].
struct Pairs {
    float a[8], b[8];
};

// Where lane l of a row's eight finds its two 8-element chunks.  Lanes below
// R/16 hold pairs: chunks l and l + R/16 (halves), or 2l and 2l + 1
// (neighbours); the others hold the chunks from R/8 on, two each.
__device__ __forceinline__ void chunks_of(const Params& p, int l, int& c0, int& c1) {
    const int n = p.rot >> 4;
    if (l < n && !p.interleaved) {
        c0 = l;
        c1 = l + n;
    } else {   // for the pairs of neighbours, and for l >= R/16, where R/8 + 2 (l - R/16) = 2l
        c0 = 2 * l;
        c1 = 2 * l + 1;
    }
}

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// The chunks' 16 elements <-> pairs: chunk by chunk, or neighbour by neighbour.
__device__ __forceinline__ void split_pairs(const float (&x)[8], const float (&y)[8], bool neighbours, Pairs& z) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        z.a[i] = neighbours ? (i < 4 ? x[2 * i] : y[2 * i - 8]) : x[i];
        z.b[i] = neighbours ? (i < 4 ? x[2 * i + 1] : y[2 * i - 7]) : y[i];
    }
}
__device__ __forceinline__ void join_pairs(const Pairs& z, bool neighbours, float (&x)[8], float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = neighbours ? ((i & 1) ? z.b[i >> 1] : z.a[i >> 1]) : z.a[i];
        y[i] = neighbours ? ((i & 1) ? z.b[4 + (i >> 1)] : z.a[4 + (i >> 1)]) : z.b[i];
    }
}

// Table row `pos`, pairs 8l .. 8l + 7.
__device__ __forceinline__ void load_angles(const Params& p, int pos, int l, float (&c)[8], float (&s)[8]) {
    const float* row = p.cos_sin + static_cast<size_t>(pos) * p.rot + 8 * l;
    const float4 c0 = __ldg(reinterpret_cast<const float4*>(row)), c1 = __ldg(reinterpret_cast<const float4*>(row) + 1);
    const float* srow = row + (p.rot >> 1);
    const float4 s0 = __ldg(reinterpret_cast<const float4*>(srow)), s1 = __ldg(reinterpret_cast<const float4*>(srow) + 1);
    c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
    s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w, s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
}

// A new token's place: its sequence, its index t in it (negative: a padded
// entry's token, left alone) and the row of the table for it.
struct Token {
    int b, t, pos;
};

__device__ __forceinline__ bool position_ok(const Params& p, int i, int t, int& pos) {
    pos = p.positions != nullptr ? p.positions[i] : t;
    if (p.rot == 0 || (pos >= 0 && pos < p.max_pos)) return true;
    flag_status(p.status, ATTN_DEV_POSITION_OUT_OF_RANGE);
    return false;
}

// New token i of the batch, found by a whole warp; false if nothing of it is
// to be written.
__device__ __forceinline__ bool find_token(const Params& p, int i, int lane, Token& tk) {
    if (p.qo_indptr == nullptr) {
        tk.b = i;
        tk.t = p.seq_lens[i] - 1;
    } else {
        if (i < p.qo_indptr[0] || i >= p.qo_indptr[p.B]) return false;   // rows of no sequence
        tk.b = warp_rank(p.B, i, lane, [&](int b) { return p.qo_indptr[b]; });
        tk.t = p.seq_lens[tk.b] - (p.qo_indptr[tk.b + 1] - i);
    }
    return tk.t >= 0 && position_ok(p, i, tk.t, tk.pos);
}

// Rotates (or copies) one bf16 row into another (which may be the same one).
__device__ __forceinline__ void rotate_row(const Params& p, const __nv_bfloat16* src, __nv_bfloat16* dst, bool turn,
                                           const float (&c)[8], const float (&s)[8], int l) {
    int c0, c1;
    chunks_of(p, l, c0, c1);
    uint4 w0 = reinterpret_cast<const uint4*>(src)[c0], w1 = reinterpret_cast<const uint4*>(src)[c1];
    if (turn && l < (p.rot >> 4)) {
        float x[8], y[8];
        Pairs z;
        unpack8(w0, x);
        unpack8(w1, y);
        split_pairs(x, y, p.interleaved != 0, z);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = z.a[i], b = z.b[i];
            z.a[i] = fmaf(a, c[i], -(b * s[i]));
            z.b[i] = fmaf(a, s[i], b * c[i]);
        }
        join_pairs(z, p.interleaved != 0, x, y);
        w0 = pack8(x);
        w1 = pack8(y);
    }
    reinterpret_cast<uint4*>(dst)[c0] = w0;
    reinterpret_cast<uint4*>(dst)[c1] = w1;
}

// Rows [0, n_q) of new token i: queries; then (bf16 cache) its keys and values.
__device__ __forceinline__ void token_rows(const Params& p, int i, bool with_kv) {
    const int lane = threadIdx.x & 31, l = threadIdx.x & 7;
    Token tk;
    if (!find_token(p, i, lane, tk)) return;
    float c[8], s[8];
    if (l < (p.rot >> 4)) load_angles(p, tk.pos, l, c, s);
    long long slot = -1;
    if (with_kv) {
        const int e = tk.t / p.list.page_size;
        const int page = page_at(p.list, tk.b, e, page_count(p.list, tk.b), threadIdx.x == 0 ? p.status : nullptr);
        if (page >= 0) slot = static_cast<long long>(page) * p.list.page_size + tk.t % p.list.page_size;
    }
    const int n_q = p.q != nullptr ? p.Hq : 0;
    const int n = n_q + (slot >= 0 ? 2 * p.Hkv : 0);
    for (int r = threadIdx.x >> 3; r < n; r += kThreads / 8) {
        if (r < n_q) {
            rotate_row(p, p.q + i * p.q_stride + r * kD, p.q_out + (static_cast<size_t>(i) * p.Hq + r) * kD, true, c, s, l);
        } else {
            const int h = (r - n_q) % p.Hkv;
            const bool key = r - n_q < p.Hkv;
            const __nv_bfloat16* src = (key ? p.k + i * p.k_stride : p.v + i * p.v_stride) + h * kD;
            __nv_bfloat16* cache = static_cast<__nv_bfloat16*>(key ? p.k_cache : p.v_cache);
            rotate_row(p, src, cache + (static_cast<size_t>(slot) * p.Hkv + h) * kD, key, c, s, l);
        }
    }
}

__global__ void __launch_bounds__(kThreads) kv_append_kernel(const Params p) { token_rows(p, blockIdx.x, true); }

// ------------------------------------------------------------- 8-bit blocks

// 2^e as a float, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// The scale of values of size `top` (finite, >= 0): 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_of(float top) {
    if (top == 0.f) return 0.f;
    const uint32_t u = __float_as_uint(top);
    const int e = static_cast<int>(u >> 23) - 127 - ((u & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
    return pow2(e < -126 ? -126 : e);
}

// A stored scale as a power of two: itself if it is one, else the next above
// (0 for what is no finite positive number).
__device__ __forceinline__ float old_scale_of(float s) {
    if (!(s > 0.f) || s > 3.0e38f) return 0.f;
    const uint32_t u = __float_as_uint(s);
    const int e = static_cast<int>(u >> 23) - 127 + ((u & 0x7FFFFFu) != 0u ? 1 : 0);
    return pow2(e < -126 ? -126 : (e > 127 ? 127 : e));
}

// a c - b s within 1.5 units in the last place, also where the products cancel.
__device__ __forceinline__ float cross(float a, float c, float b, float s) {
    const float w = b * s;
    return fmaf(a, c, -w) - fmaf(b, s, -w);
}

__device__ __forceinline__ float finite_size(float x) {
    const float y = fabsf(x);
    return y <= 3.402823466e38f ? y : 0.f;   // NaN and infinities do not count
}

// Whether fp32's value v of a rotated element (2 units off at most, scaled by
// a power of two) may lie on the other side of a border between two e4m3
// codes: its 20 dropped bits are near one half, or it is among e4m3's
// subnormals, where other bits are dropped, or not finite.
__device__ __forceinline__ bool near_border(float v) {
    const uint32_t u = __float_as_uint(v);
    const int off = static_cast<int>(u & 0xFFFFFu) - 0x80000;
    const float size = fabsf(v);
    return (off >= -4 && off <= 4) || (size < 0.015625f && size > 0.f) || !(size < 1e30f);
}

// a c - b s in 64 bits, times a power of two, rounded towards zero to fp32 with
// the last bit set if anything was lost: the e4m3 rounding of it is that of the
// 64-bit value.
__device__ __noinline__ float cross_exact(float a, float c, float b, float s, float inv) {
    const double x = (static_cast<double>(a) * c - static_cast<double>(b) * s) * static_cast<double>(inv);
    const float f = __double2float_rz(x);
    return static_cast<double>(f) == x || !(fabsf(f) < 1e30f) ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// One block of one sequence, one head, keys or values: a warp, eight lanes a
// row, four rows at a time.  Rows [lo, hi) of the sequence are new (batch rows
// from i0 on), rows [j0, lo) were there.
__device__ __forceinline__ void append_block(const Params& p, bool key, int h, int i0, int j0, int lo, int hi, int page,
                                             int lane) {
    const int l = lane & 7, sub = lane >> 3;
    const int slot0 = j0 % p.list.page_size;
    const size_t row0 = static_cast<size_t>(page) * p.list.page_size + slot0;
    uint8_t* cells = static_cast<uint8_t*>(key ? p.k_cache : p.v_cache) + (row0 * p.Hkv + h) * kD;
    const size_t cell_stride = static_cast<size_t>(p.Hkv) * kD;
    float* scale = (key ? p.k_scale : p.v_scale) + (row0 / p.block) * p.Hkv + h;
    const __nv_bfloat16* x0 = (key ? p.k : p.v) + h * kD;
    const long long stride = key ? p.k_stride : p.v_stride;
    const bool turn = key && l < (p.rot >> 4);
    const bool neighbours = p.interleaved != 0;
    int c0, c1;
    chunks_of(p, l, c0, c1);

    // the pairs of row t, their angles, and whether the row is written at all
    auto load = [&](int t, Pairs& z, float (&c)[8], float (&s)[8]) -> bool {
        const int i = i0 + (t - lo);
        int pos;
        if (!position_ok(p, i, t, pos)) return false;
        const uint4* src = reinterpret_cast<const uint4*>(x0 + i * stride);
        float x[8], y[8];
        unpack8(src[c0], x);
        unpack8(src[c1], y);
        split_pairs(x, y, neighbours && turn, z);
        if (turn) load_angles(p, pos, l, c, s);
        return true;
    };

    float top = 0.f;
    for (int t = lo + sub; t < hi; t += 4) {
        Pairs z;
        float c[8], s[8];
        if (!load(t, z, c, s)) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = z.a[i], b = z.b[i];
            top = fmaxf(top, finite_size(turn ? cross(a, c[i], b, s[i]) : a));
            top = fmaxf(top, finite_size(turn ? cross(a, s[i], -b, c[i]) : b));
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    // a size within a few units of 1.75 * 2^e may be off to its other side: in 64 bits
    const int edge = static_cast<int>(__float_as_uint(top) & 0x7FFFFFu) - 0x600000;
    if (key && p.rot > 0 && edge >= -4 && edge <= 4) {
        float up = 0.f;
        for (int t = lo + sub; t < hi; t += 4) {
            Pairs z;
            float c[8], s[8];
            if (!load(t, z, c, s)) continue;
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                up = fmaxf(up, finite_size(turn ? cross_exact(z.a[i], c[i], z.b[i], s[i], 1.f) : z.a[i]));
                up = fmaxf(up, finite_size(turn ? cross_exact(z.a[i], s[i], -z.b[i], c[i], 1.f) : z.b[i]));
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, off));
        top = up;
    }
    float now = scale_of(top);
    if (lo > j0) {
        const float was = *scale, before = old_scale_of(was);
        now = fmaxf(now, before);
        if (now != was) {   // the codes that are there move to the new scale
            const float ratio = now > 0.f && before > 0.f ? was / now : 0.f;
            for (int t = j0 + sub; t < lo; t += 4) {
                uint4* cell = reinterpret_cast<uint4*>(cells + (t - j0) * cell_stride) + l;
                uint4 w = *cell;
                uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t out = 0;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t f = e4m3x2_to_f16x2(u[i] >> (16 * k));
                        const __half2 hh = *reinterpret_cast<const __half2*>(&f);
                        out |= to_e4m3x2(__low2float(hh) * ratio, __high2float(hh) * ratio) << (16 * k);
                    }
                    u[i] = out;
                }
                *cell = make_uint4(u[0], u[1], u[2], u[3]);
            }
        }
    }
    __syncwarp();   // every lane has read the old scale
    if (lane == 0) *scale = now;
    const float inv = now > 0.f ? 1.f / now : 0.f;   // exact: now is 2^-126 .. 2^120
    for (int t = lo + sub; t < hi; t += 4) {
        Pairs z;
        float c[8], s[8];
        if (!load(t, z, c, s)) continue;
        if (turn) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = z.a[i], b = z.b[i];
                float x = cross(a, c[i], b, s[i]) * inv, y = cross(a, s[i], -b, c[i]) * inv;
                if (near_border(x)) x = cross_exact(a, c[i], b, s[i], inv);
                if (near_border(y)) y = cross_exact(a, s[i], -b, c[i], inv);
                z.a[i] = x;
                z.b[i] = y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                z.a[i] *= inv;
                z.b[i] *= inv;
            }
        }
        float x[8], y[8];
        join_pairs(z, neighbours && turn, x, y);
        uint2* out = reinterpret_cast<uint2*>(cells + (t - j0) * cell_stride);
        out[c0] = make_uint2(to_e4m3x2(x[0], x[1]) | (to_e4m3x2(x[2], x[3]) << 16),
                             to_e4m3x2(x[4], x[5]) | (to_e4m3x2(x[6], x[7]) << 16));
        out[c1] = make_uint2(to_e4m3x2(y[0], y[1]) | (to_e4m3x2(y[2], y[3]) << 16),
                             to_e4m3x2(y[4], y[5]) | (to_e4m3x2(y[6], y[7]) << 16));
    }
}

// CTAs [0, n_units) take one block each (every head, keys and values, a warp
// apiece), the others one token's queries each.  Sequence b's blocks are the
// units from S_b = qo_indptr[b] / block + 2b on: n new tokens touch at most
// n / block + 2 blocks, and S_{b+1} - S_b is at least that, so no prefix sum
// is needed; the units left over do nothing.
__global__ void __launch_bounds__(kThreads) kv_append_fp8_block_kernel(const Params p) {
    const int u = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (u >= p.n_units) {
        token_rows(p, u - p.n_units, false);
        return;
    }
    int b, i0, n, j;
    if (p.qo_indptr == nullptr) {
        b = i0 = u;
        n = 1;
        j = 0;
    } else {
        b = warp_rank(p.B, u, lane, [&](int x) { return p.qo_indptr[x] / p.block + 2 * x; });
        i0 = p.qo_indptr[b];
        n = p.qo_indptr[b + 1] - i0;
        j = u - (i0 / p.block + 2 * b);
        if (i0 < 0 || n <= 0 || j < 0 || i0 + n > p.total_q) return;
    }
    const int len = p.seq_lens[b];
    const int first = len - n;                        // tokens below 0: left alone
    const int from = first > 0 ? first : 0;
    const int j0 = (from / p.block + j) * p.block;    // the block's first token
    const int lo = from > j0 ? from : j0;
    const int hi = len < j0 + p.block ? len : j0 + p.block;
    if (lo >= hi) return;
    const int page = page_at(p.list, b, j0 / p.list.page_size, page_count(p.list, b),
                             threadIdx.x == 0 ? p.status : nullptr);
    if (page < 0) return;
    for (int w = warp; w < 2 * p.Hkv; w += kThreads / 32)
        append_block(p, w < p.Hkv, w < p.Hkv ? w : w - p.Hkv, i0 + (lo - first), j0, lo, hi, page, lane);
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream) {
    Params p;
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.k = static_cast<const __nv_bfloat16*>(a.k);
    p.v = static_cast<const __nv_bfloat16*>(a.v);
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.cos_sin = a.cos_sin;
    p.positions = a.positions;
    p.qo_indptr = a.qo_indptr;
    p.seq_lens = a.seq_lens;
    p.list = PageList{a.block_table, a.kv_indptr, a.max_pages, a.num_pages, a.page_size};
    p.q_out = static_cast<__nv_bfloat16*>(a.q_out);
    p.k_cache = a.k_cache;
    p.v_cache = a.v_cache;
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.max_pos = a.max_pos;
    p.rot = a.rot_dim;
    p.interleaved = a.interleaved;
    p.B = a.B;
    p.total_q = a.total_q;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.block = a.block_tokens;
    p.status = a.dev_status;
    if (a.k_scale == nullptr) {
        p.n_units = 0;
        kv_append_kernel<<<a.total_q, kThreads, 0, stream>>>(p);
    } else {
        p.n_units = a.qo_indptr == nullptr ? a.B : a.total_q / a.block_tokens + 2 * a.B;
        kv_append_fp8_block_kernel<<<p.n_units + (a.q != nullptr ? a.total_q : 0), kThreads, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace gb300
