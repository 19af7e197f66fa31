// shares.cuh - the even cut of a decode's tiles into shares, one for each of a
// column's workers, and 8x8 fragment helpers of the kernels that walk them.
#pragma once

#include <cstdint>

namespace gb300 {

// The cut of `total` tiles (and ends) into shares: the first `extra` shares take each + 1
// tiles, the others `each`.
struct Cut {
    int shares, each, extra;
    __device__ __forceinline__ Cut(int workers, int total) {
        shares = max(1, min(workers, total));
        each = total / shares;
        extra = total - each * shares;
    }
    __device__ __forceinline__ int start(int w) const { return w * each + min(w, extra); }
    __device__ __forceinline__ int share_of(int x) const {
        const int big = extra * (each + 1);
        return x < big ? x / (each + 1) : extra + (x - big) / each;
    }
};

// Transpose of an 8x8 matrix of 16-bit elements held in fragment layout.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

}  // namespace gb300
