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
// is a bf16 number.  A key's code is that of its exact rotation: fp32 decides
// unless the value lies within a few units of a border, where it is computed
// again in twice the precision.
//
// Bound: the bytes, on long batches: 9k tokens of 32 + 2 x 4 heads into a bf16
// cache (185 MB) take 31.5 us, 5.9 TB/s; into 8-bit blocks see below.  A decode
// step of 64 tokens of 32 + 2 x 8 heads takes 2.4 us (8-bit blocks 3.3-4.0 by GPU
// while no scale grows), the latency of a launch and of three loads that wait for
// one another.  Where scales grow, the rows that are there are rescaled one after
// another: see token_rows.
#include "paged.cuh"
#include "ptx.cuh"

namespace gb300 {
namespace {

constexpr int kD = 128;
constexpr int kThreads = 256;    // of a CTA that takes several tokens
constexpr int kMostThreads = 512;

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
    bool wide;   // every row starts on 32 bytes
    Divisor page_div, block_div;
    Divisor pair_div, part_div;   // 2 Hkv, and Hq over the heads of a query task
    int n_units;   // ragged batches into 8-bit blocks: blocks of tokens, and spare ones
    int32_t* status;
};

// Two fp32 numbers that one instruction works on.
struct Two {
    float x, y;
};

__device__ __forceinline__ uint64_t bits_of(Two v) {
    return static_cast<uint64_t>(__float_as_uint(v.x)) | (static_cast<uint64_t>(__float_as_uint(v.y)) << 32);
}
__device__ __forceinline__ Two two_of(uint64_t b) {
    return Two{__uint_as_float(static_cast<uint32_t>(b)), __uint_as_float(static_cast<uint32_t>(b >> 32))};
}
__device__ __forceinline__ Two mul(Two a, Two b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits_of(a)), "l"(bits_of(b)));
    return two_of(d);
}
__device__ __forceinline__ Two add(Two a, Two b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits_of(a)), "l"(bits_of(b)));
    return two_of(d);
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits_of(a)), "l"(bits_of(b)), "l"(bits_of(c)));
    return two_of(d);
}
__device__ __forceinline__ Two minus(Two a) { return Two{-a.x, -a.y}; }
// max(m, |v.x|, |v.y|); NaN does not count.
__device__ __forceinline__ float max_size(float m, Two v) {
    float d;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(v.x), "f"(v.y));
    return d;
}

// Sixteen elements of a row as eight pairs (a, b), two by two.
struct Pairs {
    Two a[4], b[4];
};

// Cosines and sines of a lane's eight pairs.
struct Angles {
    Two c[4], s[4];
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

// A lane's two chunks of a row.  Where they lie side by side (pairs of
// neighbours) and rows start on 32 bytes (p.wide), one access takes them: two
// would each touch half of every 32-byte sector.
template <bool kInter>
__device__ __forceinline__ void load_chunks(const Params& p, const uint4* row, int c0, int c1, uint4& x, uint4& y) {
    if (kInter && p.wide) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w), "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                     : "l"(row + c0));
    } else {
        x = row[c0];
        y = row[c1];
    }
}
template <bool kInter>
__device__ __forceinline__ void store_chunks(const Params& p, uint4* row, int c0, int c1, uint4 x, uint4 y) {
    if (kInter && p.wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row + c0), "r"(x.x), "r"(x.y),
                     "r"(x.z), "r"(x.w), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w)
                     : "memory");
    } else {
        row[c0] = x;
        row[c1] = y;
    }
}

// Two chunks of eight bf16 <-> eight pairs: neighbour by neighbour, or chunk by chunk.
template <bool kInter>
__device__ __forceinline__ void unpack(uint4 x, uint4 y, Pairs& z) {
    const uint32_t u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kInter) {
            z.a[i] = Two{lo_bf16(u[2 * i]), lo_bf16(u[2 * i + 1])};
            z.b[i] = Two{hi_bf16(u[2 * i]), hi_bf16(u[2 * i + 1])};
        } else {
            z.a[i] = Two{lo_bf16(u[i]), hi_bf16(u[i])};
            z.b[i] = Two{lo_bf16(u[4 + i]), hi_bf16(u[4 + i])};
        }
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Word i of the two chunks from its two elements, by `join`.
template <bool kInter, typename Join>
__device__ __forceinline__ void pack(const Pairs& z, uint4& x, uint4& y, Join join) {
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kInter) {
            u[2 * i] = join(z.a[i].x, z.b[i].x);
            u[2 * i + 1] = join(z.a[i].y, z.b[i].y);
        } else {
            u[i] = join(z.a[i].x, z.a[i].y);
            u[4 + i] = join(z.b[i].x, z.b[i].y);
        }
    }
    x = make_uint4(u[0], u[1], u[2], u[3]);
    y = make_uint4(u[4], u[5], u[6], u[7]);
}

// Table row `pos`, pairs 8l .. 8l + 7.
__device__ __forceinline__ void load_angles(const Params& p, int pos, int l, Angles& t) {
    const float4* row = reinterpret_cast<const float4*>(p.cos_sin + static_cast<size_t>(pos) * p.rot + 8 * l);
    const float4* srow = row + (p.rot >> 3);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 c = __ldg(row + i), s = __ldg(srow + i);
        t.c[2 * i] = Two{c.x, c.y};
        t.c[2 * i + 1] = Two{c.z, c.w};
        t.s[2 * i] = Two{s.x, s.y};
        t.s[2 * i + 1] = Two{s.z, s.w};
    }
}

__device__ __forceinline__ void rotate(Pairs& z, const Angles& t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const Two a = z.a[i], b = z.b[i];
        z.a[i] = fma(b, minus(t.s[i]), mul(a, t.c[i]));
        z.b[i] = fma(a, t.s[i], mul(b, t.c[i]));
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
    return pow2(e < -126 ? -126 : (e > 126 ? 126 : e));
}

// Values below this make fp32's products subnormal; a block whose largest one is
// there has its rotated codes computed from scaled inputs.
constexpr float kTiny = 7.8886090522101181e-31f;   // 2^-100
// From here on a rotation may pass fp32's range, and cross_exact no longer takes
// back what it rounds: such a block's rotated codes come from scaled inputs too.
constexpr float kHuge = 3.0e38f;

// 1 / s for s = 0 (0) or a power of two from 2^-126 to 2^126.
__device__ __forceinline__ float inverse_of(float s) {
    return s > 0.f ? __uint_as_float(0x7F000000u - __float_as_uint(s)) : 0.f;
}

// The rotation within 1.5 units in the last place, also where the products
// cancel: one product rounded, the sum with the other, and the rounding taken
// back, each sum in one operation.
__device__ __forceinline__ void rotate_closely(Pairs& z, const Angles& t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const Two a = z.a[i], b = z.b[i], c = t.c[i], s = t.s[i], ns = minus(s);
        z.a[i] = add(fma(a, c, mul(b, ns)), fma(b, ns, mul(b, s)));
        z.b[i] = add(fma(b, c, mul(a, s)), fma(a, s, mul(a, ns)));
    }
}

// The largest size of a row's sixteen values; NaN does not count, an infinity does.
__device__ __forceinline__ float size_of(const Pairs& z) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max_size(max_size(top, z.a[i]), z.b[i]);
    return top;
}

// Whether fp32's maximum does not settle a block's scale: it is within a few
// units of 1.75 * 2^e and comes from a rotated row, or infinite.  own: the
// lane's own maximum, of rotated values or not.
__device__ __forceinline__ bool doubtful(float top, float own, bool rotated) {
    const int edge = static_cast<int>(__float_as_uint(top) & 0x7FFFFFu) - 0x600000;
    const bool lanes = rotated && __float_as_uint(own) + 8u >= __float_as_uint(top);
    return (lanes && edge >= -4 && edge <= 4) || !(top < kHuge);
}

// Whether fp32's value v of a rotated element (2 units off at most, scaled by
// a power of two) may lie on the other side of a border between two e4m3
// codes: its 20 dropped bits are near one half (of a code that is normal).
__device__ __forceinline__ bool near_half(float v) {
    return __float_as_uint(v) * 4096u + (0x80000000u + 4u * 4096u) <= 8u * 4096u;   // the 20 bits moved to the top
}
// a c - b s in twice fp32's precision (each product and the difference with
// its error), rounded towards zero to fp32 with the last bit set if anything
// was lost: the e4m3 rounding of it is that of the exact value.  fp64 would do
// the same at a sixty-fourth of the rate.
__device__ __forceinline__ float cross_exact(float a, float c, float b, float s) {
    const float p = a * c, q = b * s;
    const float r = p - q, back = r - p;
    const float err = (p - (r - back)) - (q + back);             // of the difference
    const float low = (fmaf(a, c, -p) - fmaf(b, s, -q)) + err;   // with the products' own
    const float h = r + low;
    const float rest = low - (h - r);
    if (!(fabsf(h) < kHuge)) return p - q;                       // infinities and NaN as they come
    if (rest == 0.f) return h;
    const uint32_t u = __float_as_uint(h);
    // towards zero: one unit back where the rest points inwards
    return __uint_as_float((((h < 0.f) != (rest < 0.f)) && h != 0.f ? u - 1u : u) | 1u);
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

// The largest finite size of a row's sixteenth, rotated values in twice fp32's
// precision (past fp32's range: its largest number, which has the same scale).
template <bool kInter>
__device__ __noinline__ float size_again(const Params& p, const Source r, int l) {
    Pairs z;
    unpack<kInter>(r.x[r.c0], r.x[r.c1], z);
    if (r.pos >= 0) {
        Angles t;
        load_angles(p, r.pos, l, t);
        auto turned = [&](float a, float c, float b, float s) {
            const float x = cross_exact(a, c, b, s);
            return !(fabsf(x) < kHuge) && fabsf(a) <= 3.4e38f && fabsf(b) <= 3.4e38f ? 3.402823466e38f : x;
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Two a = z.a[i], b = z.b[i], c = t.c[i], s = t.s[i];
            z.a[i] = Two{turned(a.x, c.x, b.x, s.x), turned(a.y, c.y, b.y, s.y)};
            z.b[i] = Two{turned(a.x, s.x, -b.x, c.x), turned(a.y, s.y, -b.y, c.y)};
        }
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        top = fmaxf(fmaxf(fmaxf(top, finite_size(z.a[i].x)), finite_size(z.a[i].y)),
                    fmaxf(finite_size(z.b[i].x), finite_size(z.b[i].y)));
    return top;
}

// Sixteen values as codes, the first chunk's eight in the first two words.
template <bool kInter>
__device__ __forceinline__ uint4 to_codes(const Pairs& z) {
    uint4 x, y;   // two codes a word
    pack<kInter>(z, x, y, [](float lo, float hi) { return to_e4m3x2(lo, hi); });
    return make_uint4(x.x | (x.y << 16), x.z | (x.w << 16), y.x | (y.y << 16), y.z | (y.w << 16));
}

// The codes of a rotated row's sixteenth in twice fp32's precision, from memory.
template <bool kInter>
__device__ __noinline__ uint4 codes_again(const Params& p, const Source r, float inv, int l) {
    Pairs z;
    unpack<kInter>(r.x[r.c0], r.x[r.c1], z);
    Angles t;
    load_angles(p, r.pos, l, t);
    const Two inv2{inv, inv};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const Two a = mul(z.a[i], inv2), b = mul(z.b[i], inv2), c = t.c[i], s = t.s[i];
        z.a[i] = Two{cross_exact(a.x, c.x, b.x, s.x), cross_exact(a.y, c.y, b.y, s.y)};
        z.b[i] = Two{cross_exact(a.x, s.x, -b.x, c.x), cross_exact(a.y, s.y, -b.y, c.y)};
    }
    return to_codes<kInter>(z);
}

// A lane's sixteen values over the scale to codes: z holds the values (fp32's
// of rotated ones), inv = 1 / scale.
template <bool kInter>
__device__ __forceinline__ void store_codes(const Params& p, Pairs& z, float inv, bool tiny, const Source& r, uint8_t* row,
                                            int l) {
    const Two inv2{inv, inv};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        z.a[i] = mul(z.a[i], inv2);
        z.b[i] = mul(z.b[i], inv2);
    }
    uint4 codes = to_codes<kInter>(z);
    if (r.pos >= 0) {
        // the row's smallest size stands for the subnormals, 0 * value for NaN and infinities
        bool near = false;
        float least = 1.f;
        Two none{0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            near |= near_half(z.a[i].x) | near_half(z.a[i].y) | near_half(z.b[i].x) | near_half(z.b[i].y);
            least = fminf(fminf(fminf(least, fabsf(z.a[i].x)), fminf(fabsf(z.a[i].y), fabsf(z.b[i].x))), fabsf(z.b[i].y));
            none = fma(z.a[i], Two{0.f, 0.f}, fma(z.b[i], Two{0.f, 0.f}, none));
        }
        if (least < 0.015625f) {
            // subnormal codes have the borders that 2^-6 above them has
            auto low = [](float v) { return near_half(fabsf(v) < 0.015625f ? fabsf(v) + 0.015625f : v); };
#pragma unroll
            for (int i = 0; i < 4; ++i) near |= low(z.a[i].x) | low(z.a[i].y) | low(z.b[i].x) | low(z.b[i].y);
        }
        if (near || tiny || none.x != 0.f || none.y != 0.f) codes = codes_again<kInter>(p, r, inv, l);
    }
    reinterpret_cast<uint2*>(row)[r.c0] = make_uint2(codes.x, codes.y);
    reinterpret_cast<uint2*>(row)[r.c1] = make_uint2(codes.z, codes.w);
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
// keys and values, into a bf16 cache or (kFp8) as the one new token of an 8-bit
// block.  The rows' loads, kBatch a lane, are issued before the token's place,
// which takes three loads in a row, is known.
template <bool kInter, bool kFp8, int kBatch>
__device__ __forceinline__ void token_rows(const Params& p, int i, int warp, int warps) {
    const int lane = threadIdx.x & 31, l = lane & 7;
    const int n_q = p.q != nullptr ? p.Hq : 0;
    const int n = n_q + 2 * p.Hkv;
    const int c0 = first_chunk<kInter>(p, l), c1 = second_chunk<kInter>(p, l);
    auto source = [&](int r) -> const uint4* {
        const __nv_bfloat16* x;
        if (r < n_q)
            x = p.q + i * p.q_stride + r * kD;
        else if (r < n_q + p.Hkv)
            x = p.k + i * p.k_stride + (r - n_q) * kD;
        else
            x = p.v + i * p.v_stride + (r - n_q - p.Hkv) * kD;
        return reinterpret_cast<const uint4*>(x);
    };
    int b = 0, t = 0, pos = 0;
    long long slot = -1;
    Angles turn;
    for (int r0 = warp * 4 + (lane >> 3), step = 4 * warps, first = 1; first || r0 < n; r0 += kBatch * step, first = 0) {
        uint4 x[kBatch], y[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (r0 + k * step < n) {
                load_chunks<kInter>(p, source(r0 + k * step), c0, c1, x[k], y[k]);
            }
        if (first) {
            if (!find_token(p, i, lane, b, t, pos)) return;
            if (l < (p.rot >> 4)) load_angles(p, pos, l, turn);
            const int entry = p.page_div.div(t);
            const int page = page_at(p.list, b, entry, page_count(p.list, b), warp == 0 && lane == 0 ? p.status : nullptr);
            if (page >= 0) slot = static_cast<long long>(page) * p.list.page_size + (t - entry * p.list.page_size);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int r = r0 + k * step;
            if (r >= n) break;
            const bool query = r < n_q, key = !query && r < n_q + p.Hkv;
            const bool turns = (query || key) && l < (p.rot >> 4);
            Pairs z;
            if (query || !kFp8) {
                if (turns) {
                    unpack<kInter>(x[k], y[k], z);
                    rotate(z, turn);
                    pack<kInter>(z, x[k], y[k], pack2);
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
                store_chunks<kInter>(p, dst, c0, c1, x[k], y[k]);
            } else if (slot >= 0) {
                // one new row of a block: eight lanes settle its scale
                const unsigned eight = 0xFFu << (lane & 24);
                const int h = key ? r - n_q : r - n_q - p.Hkv;
                const int there = t - p.block_div.div(t) * p.block;   // rows of the block before it
                float* scale = (key ? p.k_scale : p.v_scale) + static_cast<size_t>(p.block_div.div(static_cast<int>(slot))) * p.Hkv + h;
                uint8_t* row = static_cast<uint8_t*>(key ? p.k_cache : p.v_cache) + (static_cast<size_t>(slot) * p.Hkv + h) * kD;
                const float was = there > 0 ? *scale : 0.f;
                const Source src{source(r), c0, c1, turns ? pos : -1};
                unpack<kInter>(x[k], y[k], z);
                if (turns) rotate_closely(z, turn);
                const float own = size_of(z);
                float top = own;
#pragma unroll
                for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(eight, top, off));
                if (__any_sync(eight, doubtful(top, own, turns))) {
                    top = size_again<kInter>(p, src, l);
#pragma unroll
                    for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(eight, top, off));
                }
                float ratio;
                const float now = join_scales(scale_of(top), there > 0, was, ratio);
                __syncwarp(eight);   // all eight have read the old scale
                if (l == 0 && !(there > 0 && now == was)) *scale = now;
                // one row after another, a load and a store each: 64 sequences of 8 heads, normal values,
                // over 64 steps 4.3 us a step without a growth; with those that come, 7.3 us for blocks
                // of 16 tokens, 17.8 of 64 and 9.7 of 256, the longest step of them 35 us
                if (ratio != 1.f)
                    for (int j = 1; j <= there; ++j) rescale_row(row - static_cast<size_t>(j) * p.Hkv * kD, ratio, l);
                store_codes<kInter>(p, z, inverse_of(now), top < kTiny, src, row, l);
            }
        }
    }
}

// warps_per_token of a CTA's warps take a token.  With kBatch = 1 the CTA is one
// token's, eight threads a row: each path's code is there once, and runs once
// (64 tokens into 8-bit blocks 3.3 us; 3.5-4.1 with three rows unrolled).
template <bool kInter, bool kFp8, int kBatch>
__global__ void __launch_bounds__(kMostThreads) kv_append_kernel(const __grid_constant__ Params p, int warps_per_token) {
    const int warp = threadIdx.x >> 5, tokens = (blockDim.x >> 5) / warps_per_token;
    const int i = blockIdx.x * tokens + warp / warps_per_token;
    if (i < p.total_q) token_rows<kInter, kFp8, kBatch>(p, i, warp % warps_per_token, warps_per_token);
}

template <bool kFp8>
cudaError_t launch_tokens(const Params& p, bool interleaved, int sms, cudaStream_t stream) {
    // a CTA per token while they are at most about 768 threads an SM, or two
    // CTAs, else two warps each.  32 + 2 x 8 heads, bf16 / 8 bits: 256 tokens 3.1
    // / 5.2 us against 3.8 / 6.2, 400 tokens 4.5 / 7.8 against 3.8 / 6.2.
    const int rows = (p.q != nullptr ? p.Hq : 0) + 2 * p.Hkv;
    const int threads = std::min(kMostThreads, (rows * 8 + 31) / 32 * 32);
    if (p.total_q <= sms * std::max(2, 768 / threads)) {
        auto kern = interleaved ? kv_append_kernel<true, kFp8, 1> : kv_append_kernel<false, kFp8, 1>;
        kern<<<p.total_q, threads, 0, stream>>>(p, threads / 32);
    } else {
        constexpr int kPer = 2, kTokens = kThreads / 32 / kPer;
        auto kern = interleaved ? kv_append_kernel<true, kFp8, 2> : kv_append_kernel<false, kFp8, 2>;
        kern<<<(p.total_q + kTokens - 1) / kTokens, kThreads, 0, stream>>>(p, kPer);
    }
    return cudaGetLastError();
}

// Ragged batches into 8-bit blocks.  Every warp copies up to kRows rows into shared
// memory, all of them in flight at once, and works on them there, eight lanes a
// row, four rows at a time.  17k tokens of 32 + 2 x 8 heads (378 MB): 70.5 us, 80 %
// of the copy rate; alone the queries take 47 us (their bytes 41) and the blocks
// 40 (their bytes 15), bound by what a warp waits for at four warps a scheduler.
// Tried: unrolled over rows in registers 120 us (a quarter of it waiting for
// instructions, 12 warps an SM), 5 CTAs an SM 70 us but 8.7 instead of 8.1 for 13
// short chunks, the first angles and the lengths loaded sooner 71.5, a CTA of 8
// lanes per row and a round per head 105-118 us (what a head costs a warp beside
// its four rows), 6 CTAs an SM 80 us (80 registers spill), queries by token
// instead of by 8 tokens x 4 heads 79 us, the two kinds mixed 70.
constexpr int kTaskWarps = 4;
constexpr int kRows = 32;
constexpr int kRowBytes = 2 * kD;
constexpr int kTaskCtas = 4;   // an SM holds at once

struct TaskMemory {
    uint4 rows[kTaskWarps][kRows * kRowBytes / 16];
    float top[2][kTaskWarps];
    int doubt[kTaskWarps];
};

// Copies rows t0 .. of `n` into the warp's buffer; `row` gives a row's source.
template <typename Row>
__device__ __forceinline__ void copy_rows(uint4* buf, int n, int lane, Row row) {
    const int l = lane & 7;
#pragma unroll
    for (int k = 0; k < kRows / 4; ++k) {
        const int r = 4 * k + (lane >> 3);
        if (r < n) {
            const uint4* src = row(r);
            cp_async16(buf + r * 16 + l, src + l, 16);
            cp_async16(buf + r * 16 + l + 8, src + l + 8, 16);
        }
    }
}

// A rotated sixteenth in 16 bits each: bf16 rounded to odd (towards zero, the
// last bit set if anything was lost).  Eight significant bits, two more than
// the four of a code and its rounding need, give the code of the exact value
// whatever the power of two it is divided by later.  fp32's bits decide unless
// the 16 dropped ones are within a few units of 0.  z: the lane's raw pairs.
template <bool kInter>
__device__ __forceinline__ void rotate_to_odd(const Angles& t, Pairs& z, float& own, uint4& x, uint4& y) {
    Pairs r = z;
    rotate_closely(r, t);
    own = fmaxf(own, size_of(r));
    auto near_zero = [](float v) { return __float_as_uint(v) * 65536u + 4u * 65536u <= 8u * 65536u; };
    bool near = false;
    Two none{0.f, 0.f};   // 0 * value: NaN for NaN and infinities
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        near |= near_zero(r.a[i].x) | near_zero(r.a[i].y) | near_zero(r.b[i].x) | near_zero(r.b[i].y);
        none = fma(r.a[i], Two{0.f, 0.f}, fma(r.b[i], Two{0.f, 0.f}, none));
    }
    uint32_t odd = 0x00010001u;
    if (near || none.x != 0.f || none.y != 0.f) {
        odd = 0;
        auto exactly = [](float a, float c, float b, float s) {
            const uint32_t u = __float_as_uint(cross_exact(a, c, b, s));
            return __uint_as_float((u & 0xFFFFu) != 0u ? u | 0x10000u : u);
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Two a = z.a[i], b = z.b[i], c = t.c[i], s = t.s[i];
            r.a[i] = Two{exactly(a.x, c.x, b.x, s.x), exactly(a.y, c.y, b.y, s.y)};
            r.b[i] = Two{exactly(a.x, s.x, -b.x, c.x), exactly(a.y, s.y, -b.y, c.y)};
        }
    }
    pack<kInter>(r, x, y, [&](float lo, float hi) {
        return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632) | odd;
    });
}

// The largest size among two chunks of bf16, infinite if one is not finite.
__device__ __forceinline__ float size_of(uint4 x, uint4 y) {
    const uint32_t u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, u[i] & 0x7FFF7FFFu);
    m = max(m & 0xFFFFu, m >> 16);
    return m > 0x7F7Fu ? INFINITY : __uint_as_float(m << 16);
}

// Eight bf16 times inv as codes.
__device__ __forceinline__ uint2 codes_of(uint4 w, float inv) {
    const Two inv2{inv, inv};
    const Two a = mul(Two{lo_bf16(w.x), hi_bf16(w.x)}, inv2), b = mul(Two{lo_bf16(w.y), hi_bf16(w.y)}, inv2);
    const Two c = mul(Two{lo_bf16(w.z), hi_bf16(w.z)}, inv2), d = mul(Two{lo_bf16(w.w), hi_bf16(w.w)}, inv2);
    return make_uint2(to_e4m3x2(a.x, a.y) | (to_e4m3x2(b.x, b.y) << 16), to_e4m3x2(c.x, c.y) | (to_e4m3x2(d.x, d.y) << 16));
}

// kPartHeads heads of kPartTokens consecutive new tokens: queries.  Eight lanes
// keep a token's angles for all of its heads; lane j finds token j's place while
// the rows are on their way.
constexpr int kPartTokens = 8;
constexpr int kPartHeads = kRows / kPartTokens;

template <bool kInter>
__device__ __forceinline__ void query_task(const Params& p, int tile, int h0, uint4* buf, int lane) {
    const int l = lane & 7, base = tile * kPartTokens;
    const int heads = min(kPartHeads, p.Hq - h0);
    // buffer row 4k + (lane / 8): token 4 (k & 1) + lane / 8, head k / 2
#pragma unroll
    for (int k = 0; k < kRows / 4; ++k) {
        const int i = base + 4 * (k & 1) + (lane >> 3), h = k >> 1;
        if (i < p.total_q && h < heads) {
            const uint4* src = reinterpret_cast<const uint4*>(p.q + i * p.q_stride + (h0 + h) * kD);
            uint4* dst = buf + (4 * k + (lane >> 3)) * 16;
            cp_async16(dst + l, src + l, 16);
            cp_async16(dst + l + 8, src + l + 8, 16);
        }
    }
    const int i = base + lane;
    int pos = -1;
    bool there = lane < kPartTokens && i < p.total_q && i >= p.qo_indptr[0] && i < p.qo_indptr[p.B];
    if (there) {
        int lo = 0, hi = p.B;   // last b with qo_indptr[b] <= i
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.qo_indptr[mid] <= i) lo = mid; else hi = mid;
        }
        const int t = p.seq_lens[lo] - (p.qo_indptr[lo + 1] - i);
        there = t >= 0 && position_ok(p, i, t, pos);
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, there);
    const int c0 = first_chunk<kInter>(p, l), c1 = second_chunk<kInter>(p, l);
    const bool turns = l < (p.rot >> 4);
    Angles t[kPartTokens / 4];
#pragma unroll
    for (int k = 0; k < kPartTokens / 4; ++k) {
        const int r = 4 * k + (lane >> 3);
        const int at = __shfl_sync(0xffffffffu, pos, r);
        if (turns && ((mask >> r) & 1u)) load_angles(p, at, l, t[k]);
    }
    cp_async_wait_all();
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kPartTokens / 4; ++k) {
        const int r = 4 * k + (lane >> 3);
        if (!((mask >> r) & 1u)) continue;
        uint4* dst = reinterpret_cast<uint4*>(p.q_out + (static_cast<size_t>(base + r) * p.Hq + h0) * kD);
        const uint4* src = buf + r * 16;
#pragma unroll 2
        for (int h = 0; h < heads; ++h, dst += 16, src += kPartTokens * 16) {
            uint4 x = src[c0], y = src[c1];
            if (turns) {
                Pairs z;
                unpack<kInter>(x, y, z);
                rotate(z, t[k]);
                pack<kInter>(z, x, y, pack2);
            }
            store_chunks<kInter>(p, dst, c0, c1, x, y);
        }
    }
}

// One head's keys or values of one block of one sequence, by a group of `warps`
// warps (this one is number `w` of them), n_rows rows each (at most kRows): up
// to n_rows * warps new rows stay in shared memory between the maximum and the
// codes, rotated ones in 16 bits rounded to odd; more are read and rotated again.
template <bool kInter>
__device__ __forceinline__ void block_task(const Params& p, int u, int pair, TaskMemory& mem, int w, int warps, int n_rows,
                                           int lane) {
    const int l = lane & 7, warp = threadIdx.x >> 5, group = (warp - w) >> (warps >> 1);   // warps: 1, 2 or 4
    uint4* buf = mem.rows[warp];
    const int b = warp_rank(p.B, u, lane, [&](int x) { return p.block_div.div(p.qo_indptr[x]) + 2 * x; });
    const int i0 = p.qo_indptr[b], n = p.qo_indptr[b + 1] - i0;
    const int j = u - (p.block_div.div(i0) + 2 * b);
    if (i0 < 0 || n <= 0 || j < 0 || i0 + n > p.total_q) return;
    const int len = p.seq_lens[b];
    const int start = len - n;                         // tokens below 0: left alone
    const int from = start > 0 ? start : 0;
    const long long j0l = (static_cast<long long>(p.block_div.div(from)) + j) * p.block;   // the block's first token
    if (j0l >= len) return;
    const int j0 = static_cast<int>(j0l);
    const int lo = from > j0 ? from : j0;              // rows [lo, hi) of the block are new, [j0, lo) were there
    const int hi = len - j0 < p.block ? len : j0 + p.block;
    const bool key = pair < p.Hkv;
    const int h = key ? pair : pair - p.Hkv;
    const __nv_bfloat16* x0 = (key ? p.k : p.v) + h * kD;
    const long long stride = key ? p.k_stride : p.v_stride;
    const int t_first = lo + w * n_rows, t_step = warps * n_rows;
    const bool held = hi - lo <= t_step;
    auto source = [&](int t) { return reinterpret_cast<const uint4*>(x0 + (i0 + (t - start)) * stride); };
    auto copy = [&](int t0) { copy_rows(buf, min(n_rows, hi - t0), lane, [&](int r) { return source(t0 + r); }); };
    copy(t_first);
    const int entry = p.page_div.div(j0);
    const int page = page_at(p.list, b, entry, page_count(p.list, b), lane == 0 && w == 0 && pair == 0 ? p.status : nullptr);
    if (page < 0) {
        cp_async_wait_all();
        return;
    }
    const size_t row0 = static_cast<size_t>(page) * p.list.page_size + (j0 - entry * p.list.page_size);
    const size_t row_bytes = static_cast<size_t>(p.Hkv) * kD;
    uint8_t* cells = static_cast<uint8_t*>(key ? p.k_cache : p.v_cache) + (row0 * p.Hkv + h) * kD;
    float* scale = (key ? p.k_scale : p.v_scale) + p.block_div.div(static_cast<int>(row0)) * static_cast<size_t>(p.Hkv) + h;
    const float was = lo > j0 ? *scale : 0.f;
    const int c0 = first_chunk<kInter>(p, l), c1 = second_chunk<kInter>(p, l);
    const bool turns = key && l < (p.rot >> 4);
    // whether row t is to be written, and its row of the table
    auto is_there = [&](int t, int& pos) { return t < hi && position_ok(p, i0 + (t - start), t, pos); };
    float own = 0.f;
    // rotates the rows in the buffer, from t0 on, where they are, and takes their maximum
    auto turn_rows = [&](int t0) {
        cp_async_wait_all();
        __syncwarp();
        const int m = min(n_rows, hi - t0);
        if (turns) {
            Angles next;
            int pos;
            bool ok = (lane >> 3) < m && is_there(t0 + (lane >> 3), pos);
            if (ok) load_angles(p, pos, l, next);
#pragma unroll 1
            for (int r = lane >> 3; r < m; r += 4) {
                const Angles t = next;
                const bool now_ok = ok;
                ok = r + 4 < m && is_there(t0 + r + 4, pos);
                if (ok) load_angles(p, pos, l, next);   // ahead of their use
                if (!now_ok) continue;
                Pairs z;
                unpack<kInter>(buf[r * 16 + c0], buf[r * 16 + c1], z);
                uint4 x, y;
                rotate_to_odd<kInter>(t, z, own, x, y);
                buf[r * 16 + c0] = x;
                buf[r * 16 + c1] = y;
            }
        } else {
#pragma unroll 2
            for (int r = lane >> 3; r < m; r += 4) {
                int pos;
                if (is_there(t0 + r, pos)) own = fmaxf(own, size_of(buf[r * 16 + c0], buf[r * 16 + c1]));
            }
        }
        __syncwarp();
    };
    // the group's warps meet (the barrier's number as a constant, so that the CTA takes few of them)
    auto meet = [&] {
        if (warps == 1) __syncwarp();
        else if (warps == 4) __syncthreads();
        else if (group == 0) named_barrier_sync(1, 64);
        else named_barrier_sync(2, 64);
    };
    // the largest of every lane of the group (non-negative: bits are ordered as numbers)
    auto group_max = [&](float x, int turn) {
        x = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
        if (lane == 0) mem.top[turn][warp] = x;
        meet();
        for (int i = 0; i < warps; ++i) x = fmaxf(x, mem.top[turn][group * warps + i]);
        return x;
    };
    for (int t0 = t_first; t0 < hi; t0 += t_step) {
        if (t0 > t_first) copy(t0);
        turn_rows(t0);
    }
    float top = group_max(own, 0);
    const bool doubt = __any_sync(0xffffffffu, doubtful(top, own, turns));
    if (lane == 0) mem.doubt[warp] = doubt;
    meet();   // (and every warp of the group has read the old scale)
    int any = 0;
    for (int i = 0; i < warps; ++i) any |= mem.doubt[group * warps + i];
    if (any != 0) {
        own = 0.f;
        for (int t0 = t_first; t0 < hi; t0 += t_step)
            for (int t = t0 + (lane >> 3); t < min(t0 + n_rows, hi); t += 4) {
                int pos;
                if (is_there(t, pos))
                    own = fmaxf(own, size_again<kInter>(p, Source{source(t), c0, c1, turns ? pos : -1}, l));
            }
        top = group_max(own, 1);
    }
    float ratio;
    const float now = join_scales(scale_of(top), lo > j0, was, ratio);
    const float inv = inverse_of(now);
    if (lane == 0 && w == 0 && !(lo > j0 && now == was)) *scale = now;
    if (ratio != 1.f)
        for (int t = j0 + 4 * w + (lane >> 3); t < lo; t += 4 * warps) rescale_row(cells + (t - j0) * row_bytes, ratio, l);
    for (int t0 = t_first; t0 < hi; t0 += t_step) {
        if (!held) {
            copy(t0);
            turn_rows(t0);
        }
        const int m = min(n_rows, hi - t0);
#pragma unroll 2
        for (int r = lane >> 3; r < m; r += 4) {
            int pos;
            if (!is_there(t0 + r, pos)) continue;
            uint2* row = reinterpret_cast<uint2*>(cells + (t0 + r - j0) * row_bytes);
            uint2 x = codes_of(buf[r * 16 + c0], inv), y = codes_of(buf[r * 16 + c1], inv);
            // 16 bits rounded to odd do not hold the last bits of tiny values, nor those past fp32's range
            if (turns && (top < kTiny || !(top < kHuge))) {
                const uint4 codes = codes_again<kInter>(p, Source{source(t0 + r), c0, c1, pos}, inv, l);
                x = make_uint2(codes.x, codes.y);
                y = make_uint2(codes.z, codes.w);
            }
            row[c0] = x;
            row[c1] = y;
        }
        __syncwarp();
    }
}

// The first block_ctas CTAs take blocks, group_warps warps one head's keys or
// values, neighbouring groups neighbouring heads; the others take queries.
// Sequence b's blocks are the units from S_b = qo_indptr[b] / block + 2b on: n
// new tokens touch at most n / block + 2 blocks, and S_{b+1} - S_b is at least
// that, so no prefix sum is needed; the units left over do nothing.
template <bool kInter>
__global__ void __launch_bounds__(32 * kTaskWarps, kTaskCtas) kv_append_blocks_kernel(const __grid_constant__ Params p,
                                                                             int group_shift, int warp_rows, int block_ctas) {
    extern __shared__ __align__(128) uint8_t smem[];
    TaskMemory& mem = *reinterpret_cast<TaskMemory*>(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // (the host has checked that tasks are counted in int)
    if (static_cast<int>(blockIdx.x) < block_ctas) {
        const int task = static_cast<int>(blockIdx.x) * (kTaskWarps >> group_shift) + (warp >> group_shift);
        const int unit = p.pair_div.div(task), group_warps = 1 << group_shift;
        if (unit < p.n_units)
            block_task<kInter>(p, unit, task - unit * static_cast<int>(p.pair_div.d), mem, warp & (group_warps - 1), group_warps,
                               warp_rows, lane);
    } else {
        const int task = (static_cast<int>(blockIdx.x) - block_ctas) * kTaskWarps + warp;
        const int tile = p.part_div.div(task);
        if (tile * kPartTokens < p.total_q)
            query_task<kInter>(p, tile, (task - tile * static_cast<int>(p.part_div.d)) * kPartHeads, mem.rows[warp], lane);
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
    const uintptr_t starts = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.q_out) |
                             reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                             reinterpret_cast<uintptr_t>(a.k_cache) | reinterpret_cast<uintptr_t>(a.v_cache);
    p.wide = ((starts | static_cast<uintptr_t>(2 * (a.q_stride | a.k_stride | a.v_stride))) & 31u) == 0;
    p.max_pos = a.max_pos;
    p.rot = a.rot_dim;
    p.B = a.B;
    p.total_q = a.total_q;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.block = a.block_tokens;
    p.page_div = make_divisor(a.page_size);
    p.block_div = make_divisor(a.block_tokens);
    p.n_units = 0;
    p.status = a.dev_status;
    const bool fp8 = a.k_scale != nullptr;
    if (!fp8) return launch_tokens<false>(p, a.interleaved != 0, sms, stream);
    if (a.qo_indptr == nullptr) return launch_tokens<true>(p, a.interleaved != 0, sms, stream);
    p.n_units = a.total_q / a.block_tokens + 2 * a.B;
    const long long tasks = static_cast<long long>(p.n_units) * 2 * a.Hkv;
    int shift = a.block_tokens <= kRows ? 0 : (a.block_tokens <= 2 * kRows ? 1 : 2);   // log2 of a group's warps
    // a block's rows over more warps while all of them run at once: 13 chunks, 1.7k
    // tokens of 3 heads 8.1 -> 7.1 us with two (8.2 with four, which do not fit), one
    // of 54 tokens 6.4 -> 4.5, 2 of 600 of 5 heads 10.1 -> 7.9
    while ((1 << shift) < kTaskWarps && tasks << (shift + 1) <= static_cast<long long>(sms) * kTaskCtas * kTaskWarps) ++shift;
    const int warp_rows = std::min(kRows, ((a.block_tokens >> shift) + 3) / 4 * 4);
    const long long block_ctas = ((tasks << shift) + kTaskWarps - 1) / kTaskWarps;
    const int parts = (a.Hq + kPartHeads - 1) / kPartHeads;
    const long long queries = a.q != nullptr ? static_cast<long long>((a.total_q + kPartTokens - 1) / kPartTokens) * parts : 0;
    p.pair_div = make_divisor(2 * a.Hkv);
    p.part_div = make_divisor(parts);
    const long long grid = block_ctas + (queries + kTaskWarps - 1) / kTaskWarps;
    if (grid * kTaskWarps >= (1LL << 31)) return cudaErrorInvalidConfiguration;
    auto kern = a.interleaved ? kv_append_blocks_kernel<true> : kv_append_blocks_kernel<false>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = once_per_device(done, [] {
        const cudaError_t r = cudaFuncSetAttribute(kv_append_blocks_kernel<true>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                                   cudaSharedmemCarveoutMaxShared);
        return r != cudaSuccess ? r
                                : cudaFuncSetAttribute(kv_append_blocks_kernel<false>,
                                                       cudaFuncAttributePreferredSharedMemoryCarveout,
                                                       cudaSharedmemCarveoutMaxShared);
    });
    if (e != cudaSuccess) return e;
    kern<<<static_cast<unsigned>(grid), 32 * kTaskWarps, sizeof(TaskMemory), stream>>>(p, shift, warp_rows, static_cast<int>(block_ctas));
    return cudaGetLastError();
}

}  // namespace gb300
