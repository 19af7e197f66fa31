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
// is a bf16 number.  A key's code is that of its 64-bit rotation: fp32 decides
// unless the value lies within a few units of a border, where it is computed
// again in 64 bits (about one value in 10^4).
#include "paged.cuh"

namespace gb300 {
namespace {

constexpr int kD = 128;
constexpr int kThreads = 256;   // of a CTA that takes tokens
constexpr int kBatch = 3;       // rows that a lane has in flight
constexpr int kHeld = 2;        // rows of a block that a lane holds in registers

struct Params {
    const __nv_bfloat16* q;   // NULL: no queries
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
    int max_pos, rot, B, total_q, Hq, Hkv, block;
    int n_units, slices;   // block kernel: units of tokens, CTAs per unit
    int32_t* status;
};

// Sixteen elements of a row as eight pairs.
struct Pairs {
    float a[8], b[8];
};

// Cosines and sines of a lane's eight pairs.
struct Angles {
    float c[8], s[8];
};

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Where lane l of a row's eight finds its two 8-element chunks: lanes below
// R/16 hold pairs, chunks l and l + R/16 (halves), or 2l and 2l + 1
// (neighbours); the others hold the chunks from R/8 on, two each, 2l and 2l + 1.
template <bool kInter>
__device__ __forceinline__ int first_chunk(const Params& p, int l) {
    return !kInter && l < (p.rot >> 4) ? l : 2 * l;
}
template <bool kInter>
__device__ __forceinline__ int second_chunk(const Params& p, int l) {
    return !kInter && l < (p.rot >> 4) ? l + (p.rot >> 4) : 2 * l + 1;
}

// Two chunks of eight bf16 <-> eight pairs: neighbour by neighbour, or chunk by chunk.
template <bool kInter>
__device__ __forceinline__ void unpack(uint4 x, uint4 y, Pairs& z) {
    const uint32_t u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (kInter) {
            z.a[i] = lo_bf16(u[i]);
            z.b[i] = hi_bf16(u[i]);
        } else {
            z.a[i] = (i & 1) ? hi_bf16(u[i >> 1]) : lo_bf16(u[i >> 1]);
            z.b[i] = (i & 1) ? hi_bf16(u[4 + (i >> 1)]) : lo_bf16(u[4 + (i >> 1)]);
        }
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool kInter>
__device__ __forceinline__ void pack(const Pairs& z, uint4& x, uint4& y) {
    if constexpr (kInter) {
        x = make_uint4(pack2(z.a[0], z.b[0]), pack2(z.a[1], z.b[1]), pack2(z.a[2], z.b[2]), pack2(z.a[3], z.b[3]));
        y = make_uint4(pack2(z.a[4], z.b[4]), pack2(z.a[5], z.b[5]), pack2(z.a[6], z.b[6]), pack2(z.a[7], z.b[7]));
    } else {
        x = make_uint4(pack2(z.a[0], z.a[1]), pack2(z.a[2], z.a[3]), pack2(z.a[4], z.a[5]), pack2(z.a[6], z.a[7]));
        y = make_uint4(pack2(z.b[0], z.b[1]), pack2(z.b[2], z.b[3]), pack2(z.b[4], z.b[5]), pack2(z.b[6], z.b[7]));
    }
}

// Table row `pos`, pairs 8l .. 8l + 7.
__device__ __forceinline__ void load_angles(const Params& p, int pos, int l, Angles& t) {
    const float4* row = reinterpret_cast<const float4*>(p.cos_sin + static_cast<size_t>(pos) * p.rot + 8 * l);
    const float4* srow = row + (p.rot >> 3);
    const float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(srow), s1 = __ldg(srow + 1);
    t.c[0] = c0.x, t.c[1] = c0.y, t.c[2] = c0.z, t.c[3] = c0.w, t.c[4] = c1.x, t.c[5] = c1.y, t.c[6] = c1.z, t.c[7] = c1.w;
    t.s[0] = s0.x, t.s[1] = s0.y, t.s[2] = s0.z, t.s[3] = s0.w, t.s[4] = s1.x, t.s[5] = s1.y, t.s[6] = s1.z, t.s[7] = s1.w;
}

__device__ __forceinline__ void rotate(Pairs& z, const Angles& t) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = z.a[i], b = z.b[i];
        z.a[i] = fmaf(a, t.c[i], -(b * t.s[i]));
        z.b[i] = fmaf(a, t.s[i], b * t.c[i]);
    }
}

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

__device__ __forceinline__ void rotate_closely(Pairs& z, const Angles& t) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = z.a[i], b = z.b[i];
        z.a[i] = cross(a, t.c[i], b, t.s[i]);
        z.b[i] = cross(a, t.s[i], -b, t.c[i]);
    }
}

// The largest size of a row's sixteen values; NaN does not count, an infinity does.
__device__ __forceinline__ float size_of(const Pairs& z) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(fmaxf(top, fabsf(z.a[i])), fabsf(z.b[i]));
    return top;
}

// Whether fp32's maximum does not settle a block's scale: it is within a few
// units of 1.75 * 2^e (and the values are rotated), or infinite.
__device__ __forceinline__ bool doubtful(float top, bool rotated) {
    const int edge = static_cast<int>(__float_as_uint(top) & 0x7FFFFFu) - 0x600000;
    return (rotated && edge >= -4 && edge <= 4) || !(top < 3.0e38f);
}

// Whether fp32's value v of a rotated element (2 units off at most, scaled by
// a power of two) may lie on the other side of a border between two e4m3
// codes: its 20 dropped bits are near one half, or it is among e4m3's
// subnormals (or 0), where other bits are dropped, or above 448 or NaN.
__device__ __forceinline__ bool near_border(float v) {
    const uint32_t u = __float_as_uint(v);
    return (u & 0xFFFFFu) - 0x7FFFCu <= 8u || (u & 0x7FFFFFFFu) - 0x3C800000u > 0x43E00000u - 0x3C800000u;
}

// a c - b s in 64 bits, times a power of two, rounded towards zero to fp32 with
// the last bit set if anything was lost: the e4m3 rounding of it is that of the
// 64-bit value.
__device__ __noinline__ float cross_exact(float a, float c, float b, float s, float inv) {
    const double x = (static_cast<double>(a) * c - static_cast<double>(b) * s) * static_cast<double>(inv);
    const float f = __double2float_rz(x);
    return static_cast<double>(f) == x || !(fabsf(f) < 1e30f) ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

__device__ __forceinline__ float finite_size(float x) {
    const float y = fabsf(x);
    return y <= 3.402823466e38f ? y : 0.f;   // NaN and infinities do not count
}

// One row's source: where its two chunks are and which table row turns it (-1: none).
struct Source {
    const uint4* x;
    int c0, c1, pos;
};

// The largest finite size of a row in 64 bits (rounded to fp32 so that its
// scale is that of the 64-bit value), from memory.
template <bool kInter>
__device__ __noinline__ float size_again(const Params& p, const Source r, int l) {
    Pairs z;
    unpack<kInter>(r.x[r.c0], r.x[r.c1], z);
    Angles t;
    if (r.pos >= 0) load_angles(p, r.pos, l, t);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = r.pos >= 0 ? cross_exact(z.a[i], t.c[i], z.b[i], t.s[i], 1.f) : z.a[i];
        const float y = r.pos >= 0 ? cross_exact(z.a[i], t.s[i], -z.b[i], t.c[i], 1.f) : z.b[i];
        top = fmaxf(top, fmaxf(finite_size(x), finite_size(y)));
    }
    return top;
}

// A lane's sixteen values over the scale to codes: z holds the values (fp32's
// of rotated ones), inv = 1 / scale.
template <bool kInter>
__device__ __forceinline__ void store_codes(const Params& p, Pairs& z, float inv, const Source& r, uint8_t* row, int l) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        z.a[i] *= inv;
        z.b[i] *= inv;
    }
    if (r.pos >= 0) {
        bool near = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) near |= near_border(z.a[i]) || near_border(z.b[i]);
        if (near) {
            Pairs w;
            unpack<kInter>(r.x[r.c0], r.x[r.c1], w);
            Angles t;
            load_angles(p, r.pos, l, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // 0 of finite factors is exact
                if (near_border(z.a[i]) && z.a[i] != 0.f) z.a[i] = cross_exact(w.a[i], t.c[i], w.b[i], t.s[i], inv);
                if (near_border(z.b[i]) && z.b[i] != 0.f) z.b[i] = cross_exact(w.a[i], t.s[i], -w.b[i], t.c[i], inv);
            }
        }
    }
    uint2 x, y;
    if constexpr (kInter) {
        x = make_uint2(to_e4m3x2(z.a[0], z.b[0]) | (to_e4m3x2(z.a[1], z.b[1]) << 16),
                       to_e4m3x2(z.a[2], z.b[2]) | (to_e4m3x2(z.a[3], z.b[3]) << 16));
        y = make_uint2(to_e4m3x2(z.a[4], z.b[4]) | (to_e4m3x2(z.a[5], z.b[5]) << 16),
                       to_e4m3x2(z.a[6], z.b[6]) | (to_e4m3x2(z.a[7], z.b[7]) << 16));
    } else {
        x = make_uint2(to_e4m3x2(z.a[0], z.a[1]) | (to_e4m3x2(z.a[2], z.a[3]) << 16),
                       to_e4m3x2(z.a[4], z.a[5]) | (to_e4m3x2(z.a[6], z.a[7]) << 16));
        y = make_uint2(to_e4m3x2(z.b[0], z.b[1]) | (to_e4m3x2(z.b[2], z.b[3]) << 16),
                       to_e4m3x2(z.b[4], z.b[5]) | (to_e4m3x2(z.b[6], z.b[7]) << 16));
    }
    reinterpret_cast<uint2*>(row)[r.c0] = x;
    reinterpret_cast<uint2*>(row)[r.c1] = y;
}

// The codes of a row that is there, times ratio.
__device__ __forceinline__ void rescale_row(uint8_t* row, float ratio, int l) {
    uint4* cell = reinterpret_cast<uint4*>(row) + l;
    const uint4 w = *cell;
    uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t out = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t f = e4m3x2_to_f16x2(u[i] >> (16 * k));
            const __half2 h = *reinterpret_cast<const __half2*>(&f);
            out |= to_e4m3x2(__low2float(h) * ratio, __high2float(h) * ratio) << (16 * k);
        }
        u[i] = out;
    }
    *cell = make_uint4(u[0], u[1], u[2], u[3]);
}

// The scale of a block whose new values need `need` and whose earlier tokens
// (if any) have `was`; ratio = what their codes are multiplied with (1: nothing).
__device__ __forceinline__ float join_scales(float need, bool joins, float was, float& ratio) {
    ratio = 1.f;
    if (!joins) return need;
    const float before = old_scale_of(was), now = fmaxf(need, before);
    if (now != was) ratio = now > 0.f && before > 0.f ? was / now : 0.f;
    return now;
}

// ------------------------------------------------------------------- tokens

__device__ __forceinline__ bool position_ok(const Params& p, int i, int t, int& pos) {
    pos = p.positions != nullptr ? p.positions[i] : t;
    if (p.rot == 0 || (pos >= 0 && pos < p.max_pos)) return true;
    flag_status(p.status, ATTN_DEV_POSITION_OUT_OF_RANGE);
    return false;
}

// New token i: its sequence b, its index t in it and its row of the table;
// found by a whole warp.  False if nothing of it is to be written: it belongs
// to no sequence, its index is negative (a padded entry), its position is bad.
__device__ __forceinline__ bool find_token(const Params& p, int i, int lane, int& b, int& t, int& pos) {
    if (p.qo_indptr == nullptr) {
        b = i;
        t = p.seq_lens[i] - 1;
    } else {
        if (i < p.qo_indptr[0] || i >= p.qo_indptr[p.B]) return false;
        b = warp_rank(p.B, i, lane, [&](int x) { return p.qo_indptr[x]; });
        t = p.seq_lens[b] - (p.qo_indptr[b + 1] - i);
    }
    return t >= 0 && position_ok(p, i, t, pos);
}

// The rows of new token i by `warps` warps, `warp` being one of them: queries,
// and with kKv its keys and values, into a bf16 cache or (kFp8) as the one new
// token of an 8-bit block.  The rows' loads are issued before the token's
// place, which takes three loads in a row, is known.
template <bool kInter, bool kKv, bool kFp8>
__device__ __forceinline__ void token_rows(const Params& p, int i, int warp, int warps) {
    const int lane = threadIdx.x & 31, l = lane & 7;
    const int n_q = p.q != nullptr ? p.Hq : 0;
    const int n = n_q + (kKv ? 2 * p.Hkv : 0);
    const int c0 = first_chunk<kInter>(p, l), c1 = second_chunk<kInter>(p, l);
    auto source = [&](int r) -> const uint4* {
        const __nv_bfloat16* x;
        if (!kKv || r < n_q)
            x = p.q + i * p.q_stride + r * kD;
        else if (r < n_q + p.Hkv)
            x = p.k + i * p.k_stride + (r - n_q) * kD;
        else
            x = p.v + i * p.v_stride + (r - n_q - p.Hkv) * kD;
        return reinterpret_cast<const uint4*>(x);
    };
    int b = 0, t = 0, pos = 0, slot_in_page = 0;
    long long slot = -1;
    Angles turn;
    for (int r0 = warp * 4 + (lane >> 3), step = 4 * warps, first = 1; first || r0 < n; r0 += kBatch * step, first = 0) {
        uint4 x[kBatch], y[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (r0 + k * step < n) {
                const uint4* src = source(r0 + k * step);
                x[k] = src[c0];
                y[k] = src[c1];
            }
        if (first) {
            if (!find_token(p, i, lane, b, t, pos)) return;
            if (l < (p.rot >> 4)) load_angles(p, pos, l, turn);
            if constexpr (kKv) {
                const int page = page_at(p.list, b, t / p.list.page_size, page_count(p.list, b),
                                         warp == 0 && lane == 0 ? p.status : nullptr);
                slot_in_page = t % p.list.page_size;
                if (page >= 0) slot = static_cast<long long>(page) * p.list.page_size + slot_in_page;
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int r = r0 + k * step;
            if (r >= n) break;
            const bool query = !kKv || r < n_q, key = kKv && !query && r < n_q + p.Hkv;
            const bool turns = (query || key) && l < (p.rot >> 4);
            Pairs z;
            if (query || !kFp8) {
                if (turns) {
                    unpack<kInter>(x[k], y[k], z);
                    rotate(z, turn);
                    pack<kInter>(z, x[k], y[k]);
                }
                uint4* dst;
                if (query) {
                    dst = reinterpret_cast<uint4*>(p.q_out + (static_cast<size_t>(i) * p.Hq + r) * kD);
                } else {
                    if (slot < 0) continue;
                    const int h = key ? r - n_q : r - n_q - p.Hkv;
                    dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(key ? p.k_cache : p.v_cache) +
                                                   (static_cast<size_t>(slot) * p.Hkv + h) * kD);
                }
                dst[c0] = x[k];
                dst[c1] = y[k];
            } else if (slot >= 0) {
                // one new row of a block: eight lanes settle its scale
                const unsigned eight = 0xFFu << (lane & 24);
                const int h = key ? r - n_q : r - n_q - p.Hkv;
                const int there = t % p.block;   // rows of the block before it
                float* scale = (key ? p.k_scale : p.v_scale) + static_cast<size_t>(slot / p.block) * p.Hkv + h;
                uint8_t* row = static_cast<uint8_t*>(key ? p.k_cache : p.v_cache) + (static_cast<size_t>(slot) * p.Hkv + h) * kD;
                const float was = there > 0 ? *scale : 0.f;
                const Source src{source(r), c0, c1, turns ? pos : -1};
                unpack<kInter>(x[k], y[k], z);
                if (turns) rotate_closely(z, turn);
                float top = size_of(z);
#pragma unroll
                for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(eight, top, off));
                if (doubtful(top, key && p.rot > 0)) {
                    top = size_again<kInter>(p, src, l);
#pragma unroll
                    for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(eight, top, off));
                }
                float ratio;
                const float now = join_scales(scale_of(top), there > 0, was, ratio);
                __syncwarp(eight);   // all eight have read the old scale
                if (l == 0 && !(there > 0 && now == was)) *scale = now;
                if (ratio != 1.f)
                    for (int j = 1; j <= there; ++j) rescale_row(row - static_cast<size_t>(j) * p.Hkv * kD, ratio, l);
                store_codes<kInter>(p, z, now > 0.f ? 1.f / now : 0.f, src, row, l);
            }
        }
    }
}

// CTAs of kThreads threads, warps_per_token of whose warps take a token.
template <bool kInter, bool kFp8>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ Params p, int warps_per_token) {
    const int warp = threadIdx.x >> 5;
    const int i = blockIdx.x * (kThreads / 32 / warps_per_token) + warp / warps_per_token;
    if (i < p.total_q) token_rows<kInter, true, kFp8>(p, i, warp % warps_per_token, warps_per_token);
}

// 8-bit blocks of ragged batches.  CTAs [0, n_units * slices): a unit is one
// block of tokens of one sequence; groups of 4 * block threads (at most 512)
// take one head's keys or values of it at a time, a lane holding kHeld rows'
// sixteenths in registers from the load over the block's maximum to the codes,
// and the next head's rows in flight meanwhile.  The other CTAs take queries, two
// warps a token.  Sequence b's blocks are the units from S_b = qo_indptr[b] /
// block + 2b on: n new tokens touch at most n / block + 2 blocks, and S_{b+1} -
// S_b is at least that, so no prefix sum is needed; the units left over do
// nothing.
template <bool kInter>
__global__ void __launch_bounds__(512) kv_append_blocks_kernel(const __grid_constant__ Params p, int group_threads) {
    __shared__ float tops[2][16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 7;
    if (static_cast<int>(blockIdx.x) >= p.n_units * p.slices) {
        const int tokens = blockDim.x >> 6;
        const int i = (blockIdx.x - p.n_units * p.slices) * tokens + (warp >> 1);
        if (warp < 2 * tokens && i < p.total_q) token_rows<kInter, false, false>(p, i, warp & 1, 2);
        return;
    }
    const int u = blockIdx.x / p.slices, slice = blockIdx.x % p.slices;
    const int b = warp_rank(p.B, u, lane, [&](int x) { return p.qo_indptr[x] / p.block + 2 * x; });
    const int i0 = p.qo_indptr[b], n = p.qo_indptr[b + 1] - i0;
    const int j = u - (i0 / p.block + 2 * b);
    if (i0 < 0 || n <= 0 || j < 0 || i0 + n > p.total_q) return;
    const int len = p.seq_lens[b];
    const int start = len - n;                         // tokens below 0: left alone
    const int from = start > 0 ? start : 0;
    const long long j0l = (static_cast<long long>(from / p.block) + j) * p.block;   // the block's first token
    if (j0l >= len) return;
    const int j0 = static_cast<int>(j0l);
    const int lo = from > j0 ? from : j0;
    const int hi = len - j0 < p.block ? len : j0 + p.block;
    const int page = page_at(p.list, b, j0 / p.list.page_size, page_count(p.list, b),
                             threadIdx.x == 0 && slice == 0 ? p.status : nullptr);
    if (page < 0) return;
    const size_t row0 = static_cast<size_t>(page) * p.list.page_size + j0 % p.list.page_size;
    const size_t row_bytes = static_cast<size_t>(p.Hkv) * kD;
    const int group = threadIdx.x / group_threads, groups = blockDim.x / group_threads;
    const int row_in_group = (threadIdx.x - group * group_threads) >> 3, rows = group_threads >> 3;
    const int warps_per_group = group_threads >> 5, warp0 = group * warps_per_group;
    const bool held = p.block <= kHeld * rows;
    const int c0 = first_chunk<kInter>(p, l), c1 = second_chunk<kInter>(p, l);
    const bool lane_turns = l < (p.rot >> 4);

    // row `t` of the sequence for keys or values of head h, if it is new (and its position is good)
    auto source = [&](int t, int pair, Source& s) -> bool {
        if (t < lo || t >= hi) return false;
        const int i = i0 + (t - start);
        int pos;
        if (!position_ok(p, i, t, pos)) return false;
        const bool key = pair < p.Hkv;
        const __nv_bfloat16* x = key ? p.k + i * p.k_stride + pair * kD : p.v + i * p.v_stride + (pair - p.Hkv) * kD;
        s = Source{reinterpret_cast<const uint4*>(x), c0, c1, key && lane_turns ? pos : -1};
        return true;
    };
    auto load = [&](int pair, uint4 (&x)[kHeld], uint4 (&y)[kHeld]) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            Source s;
            if (pair < 2 * p.Hkv && source(j0 + row_in_group + k * rows, pair, s)) {
                x[k] = s.x[c0];
                y[k] = s.x[c1];
            }
        }
    };
    auto value = [&](const Source& s, uint4 x, uint4 y, Pairs& z) {
        unpack<kInter>(x, y, z);
        if (s.pos >= 0) {
            Angles t;
            load_angles(p, s.pos, l, t);
            rotate_closely(z, t);
        }
    };
    // the largest of every lane of the group
    auto group_max = [&](float top, int buffer) -> float {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        if (lane == 0) tops[buffer][warp] = top;
        __syncthreads();
        for (int w = 0; w < warps_per_group; ++w) top = fmaxf(top, tops[buffer][warp0 + w]);
        return top;
    };

    const int per_round = p.slices * groups;
    int buffer = 0;
    uint4 x[kHeld], y[kHeld];
    int pair = slice * groups + group;
    if (held) load(pair, x, y);
    for (int round = 0; round * per_round < 2 * p.Hkv; ++round, pair += per_round) {
        const bool live = pair < 2 * p.Hkv, key = pair < p.Hkv;
        const int h = key ? pair : pair - p.Hkv;
        float* scale = nullptr;
        uint8_t* cells = nullptr;
        float was = 0.f, top = 0.f;
        if (live) {
            scale = (key ? p.k_scale : p.v_scale) + row0 / p.block * p.Hkv + h;
            cells = static_cast<uint8_t*>(key ? p.k_cache : p.v_cache) + (row0 * p.Hkv + h) * kD;
            if (lo > j0) was = *scale;
        }
        Pairs z[kHeld];
        if (held) {
#pragma unroll
            for (int k = 0; k < kHeld; ++k) {
                Source s;
                if (live && source(j0 + row_in_group + k * rows, pair, s)) {
                    value(s, x[k], y[k], z[k]);
                    top = fmaxf(top, size_of(z[k]));
                }
            }
            load(pair + per_round, x, y);
        } else {
            for (int t = j0 + row_in_group; live && t < hi; t += rows) {
                Source s;
                if (!source(t, pair, s)) continue;
                value(s, s.x[c0], s.x[c1], z[0]);
                top = fmaxf(top, size_of(z[0]));
            }
        }
        top = group_max(top, buffer);
        buffer ^= 1;
        // every group of the CTA decides together: the barrier is the CTA's
        if (__syncthreads_or(live && doubtful(top, key && p.rot > 0))) {
            float again = 0.f;
            for (int t = j0 + row_in_group; live && t < hi; t += rows) {
                Source s;
                if (source(t, pair, s)) again = fmaxf(again, size_again<kInter>(p, s, l));
            }
            top = group_max(again, buffer);
            buffer ^= 1;
        }
        if (!live) continue;
        float ratio;
        const float now = join_scales(scale_of(top), lo > j0, was, ratio);
        const float inv = now > 0.f ? 1.f / now : 0.f;
        // (every lane read the old scale before the barrier)
        if (threadIdx.x == group * group_threads && !(lo > j0 && now == was)) *scale = now;
        if (ratio != 1.f)
            for (int t = j0 + row_in_group; t < lo; t += rows) rescale_row(cells + (t - j0) * row_bytes, ratio, l);
        if (held) {
#pragma unroll
            for (int k = 0; k < kHeld; ++k) {
                Source s;
                const int t = j0 + row_in_group + k * rows;
                if (source(t, pair, s)) store_codes<kInter>(p, z[k], inv, s, cells + (t - j0) * row_bytes, l);
            }
        } else {
            for (int t = j0 + row_in_group; t < hi; t += rows) {
                Source s;
                if (!source(t, pair, s)) continue;
                value(s, s.x[c0], s.x[c1], z[0]);
                store_codes<kInter>(p, z[0], inv, s, cells + (t - j0) * row_bytes, l);
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
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
    p.B = a.B;
    p.total_q = a.total_q;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.block = a.block_tokens;
    p.n_units = p.slices = 0;
    p.status = a.dev_status;
    if (a.k_scale == nullptr || a.qo_indptr == nullptr) {
        // all eight warps on a token while there are fewer tokens than CTAs fit at once, else two each
        const int per = a.total_q <= 4 * sms ? 8 : 2;
        const int tokens = kThreads / 32 / per;
        const int grid = (a.total_q + tokens - 1) / tokens;
        auto kern = a.k_scale != nullptr ? (a.interleaved ? kv_append_kernel<true, true> : kv_append_kernel<false, true>)
                                         : (a.interleaved ? kv_append_kernel<true, false> : kv_append_kernel<false, false>);
        kern<<<grid, kThreads, 0, stream>>>(p, per);
        return cudaGetLastError();
    }
    p.n_units = a.total_q / a.block_tokens + 2 * a.B;
    const int group = a.block_tokens < 128 ? 4 * a.block_tokens : 512;
    const int groups = group < 256 ? 256 / group : 1;
    const int rounds = (2 * a.Hkv + groups - 1) / groups;   // of one CTA that does the whole unit
    // CTAs of four rounds each, where that still gives every SM eight of them
    p.slices = static_cast<long long>(p.n_units) * rounds >= 32LL * sms ? (rounds + 3) / 4 : rounds;
    const int tokens = group * groups / 64;
    const int q_ctas = a.q != nullptr ? (a.total_q + tokens - 1) / tokens : 0;
    if (static_cast<long long>(p.n_units) * p.slices + q_ctas >= (1LL << 31)) p.slices = 1;   // the caller has checked that this fits
    const long long grid = static_cast<long long>(p.n_units) * p.slices + q_ctas;
    auto kern = a.interleaved ? kv_append_blocks_kernel<true> : kv_append_blocks_kernel<false>;
    kern<<<static_cast<unsigned>(grid), group * groups, 0, stream>>>(p, group);
    return cudaGetLastError();
}

}  // namespace gb300
