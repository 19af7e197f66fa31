// paged.cuh - page lists, ragged batches and e4m3 conversions shared by the
// kernels that write a paged KV cache and those that read its 8-bit form.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace gb300 {

// Pages of the sequences: row b of a block table (indptr NULL), or entries
// [indptr[b], indptr[b+1]) of a CSR list.
struct PageList {
    const int32_t* pages;
    const int32_t* indptr;
    int max_pages;   // entries per row of the block table
    int num_pages, page_size;
};

// Entries of sequence b's list (none where the CSR offsets fall).
__device__ __forceinline__ int page_count(const PageList& l, int b) {
    return l.indptr != nullptr ? max(l.indptr[b + 1] - l.indptr[b], 0) : l.max_pages;
}

// The pool page in entry e >= 0 of sequence b's list of n entries, or -1 (and
// the status bit) past the list's end or outside the pool.
__device__ __forceinline__ int page_at(const PageList& l, int b, int e, int n, int32_t* status) {
    if (e >= n) {
        flag_status(status, ATTN_DEV_SEQ_TOO_LONG);
        return -1;
    }
    const size_t base = l.indptr != nullptr ? static_cast<size_t>(l.indptr[b])
                                            : static_cast<size_t>(b) * static_cast<size_t>(l.max_pages);
    const int page = l.pages[base + e];
    if (page < 0 || page >= l.num_pages) {
        flag_status(status, ATTN_DEV_PAGE_OUT_OF_RANGE);
        return -1;
    }
    return page;
}

// n / d for 0 <= n < 2^31 and a divisor fixed on the host: with s the least
// power 2^s >= d and mul = ceil(2^(31+s) / d) < 2^32, mul d - 2^(31+s) < 2^s, so
// the product's error stays below 1/d.
struct Divisor {
    uint32_t d, mul;
    int shift;
    __device__ __forceinline__ int div(int n) const {
        return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul) >> shift);
    }
};

inline Divisor make_divisor(int d) {
    int s = 0;
    while ((1LL << s) < d) ++s;
    const uint64_t one = 1ULL << (31 + s);
    return Divisor{static_cast<uint32_t>(d), static_cast<uint32_t>((one + d - 1) / d), 31 + s};
}

// Last b in [0, B) with key(b) <= x, for key(0) <= x and key not decreasing; a
// whole warp counts together, 32 keys per round with independent loads.
template <typename Key>
__device__ __forceinline__ int warp_rank(int B, int x, int lane, Key key) {
    int n = 0;
#pragma unroll 4
    for (int b0 = 0; b0 < B; b0 += 32)
        n += __popc(__ballot_sync(0xffffffffu, b0 + lane < B && key(b0 + lane) <= x));
    return n > 0 ? n - 1 : 0;
}

// Two floats to two e4m3 bytes (lo in the low byte), round to nearest even;
// beyond +-448 (infinities too) becomes +-448, NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 bytes, the low or the high half of a word, to two halves (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

}  // namespace gb300
