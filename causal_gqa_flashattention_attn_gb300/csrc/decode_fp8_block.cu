// decode_fp8_block.cu - paged decode over an e4m3 KV cache with one scale per
// block of tokens and KV head, one to sixteen causal queries per sequence.
//
// Mathematics, per query row r of a KV head, with codes k_t, v_t and the
// scales a_t, b_t of their blocks:
//   s_t = scale a_t (q_r . k_t),  O_r = sum_t p_t b_t v_t / sum_t p_t,
//   p_t = 2^(log2e s_t - m),  over the visible tokens t <= len - q_len + i.
// The codes enter m16n8k16 fp16 MMAs exactly (every e4m3 number is a half); q
// is taken in fp16 after a power of two that brings its row's largest element
// to [1, 2), so any bf16 magnitude fits.  a_t multiplies the fp32 score.  b_t
// multiplies p_t before p_t b_t is rounded to fp16 for the value MMA, against
// a running power M with p_t b_t 2^(m - M) <= 2^8 of its own: blocks whose
// scales are far apart do not push each other's weights into fp16's
// subnormals.  Sums and running maxima are fp32.
//
// Work: a column is a KV head with a group of up to 8 or 16 (query, head)
// rows; every warp of the grid takes one column and an equal share of the
// 32-token tiles of all sequences, so a ragged batch is balanced whatever its
// lengths, which only the device knows (a batch of short ones goes by whole
// sequences).  A share that holds a whole sequence writes its output; the pieces
// of a sequence that is cut between shares go to the workspace, and a second
// kernel, which is launched along with the first and waits for it on the device,
// joins them.  (The join by whichever CTA comes last, inside the first kernel,
// was slower.)
//
// Bound: one read of the codes from HBM.  64 ragged sequences of 512 to 32768
// tokens, 32 heads over 8 (2.05 GB): 292 us, 7.0 TB/s; 16 of 16384 (537 MB): 87
// us, 6.2 TB/s, 3 us of it the merge.  With 16 rows a column the loop is bound
// by its own latency, 832 instructions a tile at two warps a scheduler (1.5 us
// a tile): 24 sequences of up to 9000 tokens with 4 queries of 16 heads over 2
// (57 MB) 32.5 us.  One sequence of 1000 tokens: 8.2 us for the two kernels,
// latency alone.  Tried, with an earlier merge: 12 warps with two stages each, 302 and 91 us for the
// first two and 53 for the third (16 rows spill at 168 registers); a CTA that
// widens a tile once into shared memory for its warps' groups of 16 rows, 43 us
// for 24 sequences of 4500 tokens and 32 rows where the warps alone took 32, 59
// for 57 at 64 rows and 85 for 98 only at 128.
#include <algorithm>

#include "paged.cuh"
#include "ptx.cuh"
#include "shares.cuh"

namespace gb300 {
namespace {

constexpr int kD = 128;
constexpr int kTile = 32;       // tokens per step of a warp
constexpr int kWarps = 8;       // per CTA
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxSeqs = 4096;  // tile counts before each sequence, and lengths, in shared memory
constexpr int kStages = 3;      // tiles in flight or in use per warp
constexpr int kCodes = kTile * kD;                    // 4 KB: a tile's K (or V) codes of one head
constexpr int kWarpBytes = kStages * 2 * kCodes;
static_assert(kWarps * kWarpBytes + (2 * kMaxSeqs + 1) * 4 + 1024 <= 227 * 1024, "the tables fit beside the rings");
// A sequence's end (a tile with a mask, the piece's rows, the next queries)
// costs a warp about as much as two tiles more: counted as such in the cut,
// 24 sequences of 4 queries take 35.7 us instead of 37.0.
constexpr int kEnd = 2;
// Where no sequence has more tiles, none is cut: up to three tiles one after
// another take no longer than the join of pieces (61 sequences of at most 45
// tokens 11.6 -> 8.6 us, 40 of 88 11.6 -> 10.3, 1 of 96 level, of 126 tokens, four
// tiles, 9.5 -> 11.1).
constexpr int kWholeTiles = 3;
constexpr int kMergeWarps = 8;
constexpr int kBatch = 8;       // pieces a merging warp has in flight

struct Params {
    const __nv_bfloat16* q;   // [B, q_len, Hq, D]
    const uint8_t* k_cache;   // [num_pages, page_size, Hkv, D]
    const uint8_t* v_cache;
    const float* k_scale;     // [num_pages, page_size / block, Hkv]
    const float* v_scale;
    PageList list;
    const int32_t* seq_lens;
    Divisor page_div, block_div, cols_div, heads_div, group_div;
    int page_blocks;     // blocks of a page
    bool tile_in_page;   // pages are multiples of a tile
    int B, Hq, Hkv, G, nq;
    int cols;       // KV heads x row groups
    int workers;    // shares per column
    float scale_log2;
    __nv_bfloat16* o;
    float* lse;     // may be NULL
    float* part_o;  // [2 workers][cols][rows][D]
    float* part_l;  // [2 workers][cols][rows], log2
    int32_t* status;
};

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// m16n8k16 fp16 MMA, fp32 accumulators; not volatile, so that independent ones
// may be interleaved.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Sequence b's cached tokens: its length within what its page list holds.
__device__ __forceinline__ int length_of(const Params& p, int b, bool flag) {
    const int len = p.seq_lens[b];
    const long long cap = static_cast<long long>(page_count(p.list, b)) * p.list.page_size;
    if (len < 0 || len > cap) {
        if (flag) flag_status(p.status, ATTN_DEV_SEQ_TOO_LONG);
        return len < 0 ? 0 : static_cast<int>(cap);
    }
    return len;
}

__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }
// What a sequence counts for in the cut: its tiles, and its end.
__device__ __forceinline__ int span_of(int len) { return len > 0 ? tiles_of(len) + kEnd : 0; }

// Whether a CSR list holds so many tokens that tiles do not count in int (the
// host has checked block tables).
__device__ __forceinline__ bool too_many_tiles(const Params& p) {
    if (p.list.indptr == nullptr) return false;
    return static_cast<long long>(p.list.indptr[p.B]) * p.list.page_size / kTile + (1 + kEnd) * p.B >= (1LL << 31);
}

// before[b] = spans of the sequences before b (before[B] = all) and lens[b] =
// their lengths, by the whole CTA: each thread takes a run of sequences.
// Returns whether one of them has more than kWholeTiles tiles.
__device__ __forceinline__ bool count_tiles(const Params& p, int* before, int* lens, int* warp_sum, bool flag) {
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = threadIdx.x * per, b1 = min(b0 + per, p.B);
    int sum = 0, most = 0;
    for (int b = b0; b < b1; ++b) {
        lens[b] = length_of(p, b, flag);
        sum += span_of(lens[b]);
        most = max(most, tiles_of(lens[b]));
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int base = incl - sum;
    for (int w = 0; w < warp; ++w) base += warp_sum[w];
    for (int b = b0; b < b1; ++b) {
        before[b] = base;
        base += span_of(lens[b]);
    }
    if (threadIdx.x == kThreads - 1) before[p.B] = base;   // the last run ends with the last sequence, or is empty
    return __syncthreads_or(most > kWholeTiles) != 0;
}

// Per-warp state of the online softmax and the O^T accumulators of NB x 8 rows
// (row 2t4 + j of block n): m for the sums, M for the values.
template <int NB>
struct State {
    float o[NB][8][4];   // m-tile mt: elements 16g + 2mt (c0, c1) and + 1 (c2, c3)
    float m[NB][2], M[NB][2], l[NB][2];
};

template <int NB>
__device__ __forceinline__ void reset(State<NB>& st) {
#pragma unroll
    for (int n = 0; n < NB; ++n) {
#pragma unroll
        for (int i = 0; i < 8; ++i) st.o[n][i][0] = st.o[n][i][1] = st.o[n][i][2] = st.o[n][i][3] = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            st.m[n][j] = st.M[n][j] = -INFINITY;
            st.l[n][j] = 0.f;
        }
    }
}

// The query rows of a column in fp16 as B fragments: column g of block n is
// row n * 8 + g, k pairs of k-step ks are elements 32t4 + 4ks + {0, 1}, {2, 3};
// mul = log2e * scale over the row's power of two; lim = last visible token.
template <int NB>
struct Queries {
    uint32_t f[NB][8][2];
    float mul[NB][2];
    int lim[NB][2];
};

// Their loads, four 16-byte chunks of a lane's row (zeros past the rows).
template <int NB>
__device__ __forceinline__ void fetch_queries(const Params& p, int b, int kvh, int row0, int n_rows, int lane,
                                              uint4 (&raw)[NB][4]) {
    const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        const int r = row0 + 8 * n + g;
        const int i = p.group_div.div(r), h = r - i * p.G;
        const __nv_bfloat16* src =
            p.q + ((static_cast<size_t>(b) * p.nq + i) * p.Hq + static_cast<size_t>(kvh) * p.G + h) * kD + 32 * t4;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            raw[n][c] = r < n_rows ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0u, 0u, 0u, 0u);
    }
}

template <int NB>
__device__ __forceinline__ void take_queries(const Params& p, const uint4 (&raw)[NB][4], int row0, int n_rows, int len,
                                             int lane, Queries<NB>& qs) {
    const int t4 = lane & 3;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        float x[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t u[4] = {raw[n][c].x, raw[n][c].y, raw[n][c].z, raw[n][c].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[8 * c + 2 * k] = __uint_as_float(u[k] << 16);
                x[8 * c + 2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
            }
        }
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) top = fmaxf(top, fabsf(x[k]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^-e of the row's largest element (clamped so that both factors stay normal)
        int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
        e = top == 0.f ? 0 : (e < -120 ? -120 : (e > 120 ? 120 : e));
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            qs.f[n][ks][0] = pack_f16x2(x[4 * ks] * down, x[4 * ks + 1] * down);
            qs.f[n][ks][1] = pack_f16x2(x[4 * ks + 2] * down, x[4 * ks + 3] * down);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int col = 2 * t4 + j, rr = row0 + 8 * n + col;
            qs.mul[n][j] = __shfl_sync(0xffffffffu, up, 4 * col) * p.scale_log2;
            qs.lim[n][j] = rr < n_rows ? len - p.nq + p.group_div.div(rr) : -1;
        }
    }
}

// A bit for each of the four e4m3 bytes of a word that is NaN (bit 7 of the byte).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Values that are NaN in a tile whose tokens some rows do not see: a weight of
// 0 times NaN is NaN, so the code leaves the value MMA (as 0) and its element of
// O becomes NaN in the rows that do see the token.  Lanes of a quad hold chunk g
// of different tokens and O^T of different rows.
template <int NB>
__device__ __forceinline__ void take_nans(State<NB>& st, const Queries<NB>& qs, uint4 (&vx)[2][4], int tok0, int lane) {
    const float nan = __int_as_float(0x7FFFFFFF);
#pragma unroll
    for (int sb = 0; sb < 2; ++sb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t* words = &vx[sb][i].x;
#pragma unroll 1
            for (int src = 0; src < 4; ++src) {
                const int t = tok0 + 16 * sb + 2 * src + (i & 1) + 8 * (i >> 1);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t bad = nan_bytes(__shfl_sync(0xffffffffu, words[w], (lane & 28) + src));
#pragma unroll
                    for (int e = 0; e < 4; ++e)   // element 16g + 4w + e: m-tile 2w + e / 2, row half e mod 2
                        if ((bad >> (8 * e)) & 0x80u) {
#pragma unroll
                            for (int n = 0; n < NB; ++n)
#pragma unroll
                                for (int j = 0; j < 2; ++j)
                                    if (t <= qs.lim[n][j]) st.o[n][2 * w + (e >> 1)][2 * (e & 1) + j] = nan;
                        }
                }
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) words[w] &= ~((nan_bytes(words[w]) >> 7) * 0xFFu);
        }
}

// One 32-token tile of a warp as two 16-token sub-tiles.  kPartial: some token
// is not there (its codes are zeros and its bit of `valid` is not set), or some
// row does not see it.  codes: K, then V; k_at, v_at: this lane's chunks of the
// first sub-tile, the second is 16 rows on; ka, vb: the scales of the sub-tiles.
template <int NB, bool kPartial>
__device__ __forceinline__ void tile_step(State<NB>& st, const Queries<NB>& qs, const uint8_t* codes,
                                          const int (&k_at)[2], const int (&v_at)[2], const float (&ka)[2],
                                          const float (&vb)[2], int tok0, uint32_t valid, int lane) {
    const int g = lane >> 2;
    // scores: the sub-tiles' MMA chains side by side
    uint32_t wg[2][8], w8[2][8];   // chunks 2t4, 2t4 + 1 of token g, and of token g + 8
#pragma unroll
    for (int sb = 0; sb < 2; ++sb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 c = *reinterpret_cast<const uint4*>(codes + (16 * sb + 8 * (i >> 1)) * kD + k_at[i & 1]);
            uint32_t* w = (i < 2 ? wg[sb] : w8[sb]) + 4 * (i & 1);
            w[0] = c.x, w[1] = c.y, w[2] = c.z, w[3] = c.w;
        }
    float s[NB][2][4];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) s[n][sb][0] = s[n][sb][1] = s[n][sb][2] = s[n][sb][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) {
            const uint32_t a0 = e4m3x2_to_f16x2(wg[sb][ks]), a1 = e4m3x2_to_f16x2(w8[sb][ks]);
            const uint32_t a2 = e4m3x2_hi_to_f16x2(wg[sb][ks]), a3 = e4m3x2_hi_to_f16x2(w8[sb][ks]);
#pragma unroll
            for (int n = 0; n < NB; ++n) mma16816(s[n][sb], a0, a1, a2, a3, qs.f[n][ks][0], qs.f[n][ks][1]);
        }
#pragma unroll
    for (int sb = 0; sb < 2; ++sb)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[n][sb][e] *= ka[sb] * qs.mul[n][e & 1];
                if constexpr (kPartial) {
                    const int t = 16 * sb + g + 8 * (e >> 1);
                    if (!((valid >> t) & 1u) || tok0 + t > qs.lim[n][e & 1]) s[n][sb][e] = -INFINITY;
                }
            }
    uint4 vx[2][4];   // chunk g of tokens 2t4, 2t4 + 1, 2t4 + 8, 2t4 + 9
#pragma unroll
    for (int sb = 0; sb < 2; ++sb)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            vx[sb][i] = *reinterpret_cast<const uint4*>(codes + (16 * sb + 8 * (i >> 1)) * kD + v_at[i & 1]);
    if constexpr (kPartial) {
        uint32_t bad = 0;
#pragma unroll
        for (int sb = 0; sb < 2; ++sb)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                bad |= nan_bytes(vx[sb][i].x) | nan_bytes(vx[sb][i].y) | nan_bytes(vx[sb][i].z) | nan_bytes(vx[sb][i].w);
        if (__any_sync(0xffffffffu, bad != 0u)) take_nans<NB>(st, qs, vx, tok0, lane);
    }
    const float lb[2] = {__log2f(vb[0]), __log2f(vb[1])};   // -inf for a scale of 0
    // running maxima, raised (and the sums rescaled) only when a score passes them by 2^8
    bool over = false;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int sb = 0; sb < 2; ++sb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float x = fmaxf(s[n][sb][j], s[n][sb][2 + j]);
                over |= x > st.m[n][j] + 8.f || x + lb[sb] > st.M[n][j] + 8.f;
            }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float x0 = fmaxf(s[n][0][j], s[n][0][2 + j]), x1 = fmaxf(s[n][1][j], s[n][1][2 + j]);
                float mx = fmaxf(x0, x1), Mx = fmaxf(x0 + lb[0], x1 + lb[1]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                    Mx = fmaxf(Mx, __shfl_xor_sync(0xffffffffu, Mx, off));
                }
                if (mx > st.m[n][j]) {
                    st.l[n][j] *= ex2(st.m[n][j] - mx);
                    st.m[n][j] = mx;
                }
                if (Mx > st.M[n][j]) {
                    const float alpha = ex2(st.M[n][j] - Mx);
                    st.M[n][j] = Mx;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        st.o[n][i][j] *= alpha;
                        st.o[n][i][2 + j] *= alpha;
                    }
                }
            }
    }
#pragma unroll
    for (int sb = 0; sb < 2; ++sb) {
        uint32_t w0[NB], w1[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            float w[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float m = st.m[n][j] == -INFINITY ? 0.f : st.m[n][j];
                const float M = st.M[n][j] == -INFINITY ? 0.f : st.M[n][j];
                st.l[n][j] += ex2(s[n][sb][j] - m) + ex2(s[n][sb][2 + j] - m);
                // an exponential of its own: 2^(s - m) may be 0 where this is not
                w[j] = ex2(s[n][sb][j] + (lb[sb] - M));
                w[2 + j] = ex2(s[n][sb][2 + j] + (lb[sb] - M));
            }
            w0[n] = movmatrix_trans(pack_f16x2(w[0], w[1]));
            w1[n] = movmatrix_trans(pack_f16x2(w[2], w[3]));
        }
        const uint32_t* xa = &vx[sb][0].x;
        const uint32_t* xb = &vx[sb][1].x;
        const uint32_t* xc = &vx[sb][2].x;
        const uint32_t* xd = &vx[sb][3].x;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
            const uint32_t sel = (mt & 1) ? 0x7362u : 0x5140u;   // the two tokens' bytes of two elements
            const uint32_t ab = __byte_perm(xa[mt >> 1], xb[mt >> 1], sel);
            const uint32_t cd = __byte_perm(xc[mt >> 1], xd[mt >> 1], sel);
            const uint32_t a0 = e4m3x2_to_f16x2(ab), a1 = e4m3x2_hi_to_f16x2(ab);
            const uint32_t a2 = e4m3x2_to_f16x2(cd), a3 = e4m3x2_hi_to_f16x2(cd);
#pragma unroll
            for (int n = 0; n < NB; ++n) mma16816(st.o[n][mt], a0, a1, a2, a3, w0[n], w1[n]);
        }
    }
}

// What a tile's copies bring besides its codes.
struct TileInfo {
    float k[2], v[2];   // scales of the two sub-tiles
    uint32_t valid;     // tokens that are there
    uint32_t pad[3];
};

// Byte offset of 16-byte chunk c of row r of a tile's codes: the chunk is
// XOR-ed with the row, so the eight lanes of a shared-memory phase, which read
// one chunk of two rows' four or chunk pairs, meet eight different ones.
__device__ __forceinline__ int chunk_off(int r, int c) { return r * kD + (((c ^ r) & 7) << 4); }

// The tiles of a warp's share, fetched ahead: `x` is the next one, in sequence
// b; the page of its token `lane` has been looked up one step before it is used.
struct Feed {
    int x, x_end, b, len;
    int page, tok;   // tok: the lane's token, or -1 past the sequence's end
};

__device__ __forceinline__ void feed_look(const Params& p, const int* before, Feed& f, int lane) {
    if (f.x >= before[f.b + 1] - kEnd) f.x = before[f.b + 1];   // past the end
    if (f.x >= f.x_end) return;
    if (before[f.b + 1] <= f.x) {
        do ++f.b;
        while (before[f.b + 1] <= f.x);
        f.len = before[p.B + 1 + f.b];   // the lengths follow the counts
    }
    const int tok = (f.x - before[f.b]) * kTile + lane;
    f.tok = tok < f.len ? tok : -1;
    f.page = -1;
    if (f.tok >= 0) {
        const size_t base = p.list.indptr != nullptr ? static_cast<size_t>(p.list.indptr[f.b])
                                                     : static_cast<size_t>(f.b) * static_cast<size_t>(p.list.max_pages);
        f.page = __ldg(p.list.pages + base + p.page_div.div(tok));
    }
}

// Issues the copies of tile f.x into a stage (zeros for tokens that are not
// there), as one group, and looks at the next one.
__device__ __forceinline__ void feed_tile(const Params& p, const int* before, Feed& f, uint8_t* stage, TileInfo* info,
                                          int kvh, int lane) {
    if (f.x < f.x_end) {
        const bool there = f.tok >= 0 && f.page >= 0 && f.page < p.list.num_pages;
        if (f.tok >= 0 && !there) flag_status(p.status, ATTN_DEV_PAGE_OUT_OF_RANGE);
        const uint32_t valid = __ballot_sync(0xffffffffu, there);
        const int o = there ? f.tok - p.page_div.div(f.tok) * p.list.page_size : 0;
        const int page = there ? f.page : 0;
        const size_t row_bytes = static_cast<size_t>(p.Hkv) * kD;
        const size_t off = (static_cast<size_t>(page) * p.list.page_size + o) * row_bytes + static_cast<size_t>(kvh) * kD;
        if ((lane & 15) == 0) {
            const size_t at = (static_cast<size_t>(page) * p.page_blocks + p.block_div.div(o)) * p.Hkv + kvh;
            cp_async4(&info->k[lane >> 4], p.k_scale + at, there ? 4 : 0);
            cp_async4(&info->v[lane >> 4], p.v_scale + at, there ? 4 : 0);
        }
        if (lane == 0) info->valid = valid;
        const int c = lane & 7, r0 = lane >> 3;
        if (p.tile_in_page && valid == 0xffffffffu) {
            // the rows are row_bytes apart: a third of the instructions of finding each one's place
            const size_t at = __shfl_sync(0xffffffffu, off, 0) + r0 * row_bytes + 16 * c;
            const uint8_t* k = p.k_cache + at;
            const uint8_t* v = p.v_cache + at;
            uint8_t* even = stage + chunk_off(r0, c);       // rows r0, r0 + 8, ...
            uint8_t* odd = stage + chunk_off(r0 + 4, c);    // rows r0 + 4, r0 + 12, ...
#pragma unroll
            for (int i = 0; i < kTile / 4; ++i, k += 4 * row_bytes, v += 4 * row_bytes) {
                uint8_t* dst = (i & 1 ? odd : even) + (i >> 1) * 8 * kD;
                cp_async16(dst, k, 16);
                cp_async16(dst + kCodes, v, 16);
            }
            ++f.x;
            feed_look(p, before, f, lane);
            cp_async_commit();
            return;
        }
#pragma unroll
        for (int i = 0; i < kTile / 4; ++i) {
            const int r = r0 + 4 * i;
            const size_t src = __shfl_sync(0xffffffffu, off, r) + 16 * c;
            const uint32_t n = (valid >> r) & 1u ? 16 : 0;
            cp_async16(stage + chunk_off(r, c), p.k_cache + src, n);
            cp_async16(stage + kCodes + chunk_off(r, c), p.v_cache + src, n);
        }
        ++f.x;
        feed_look(p, before, f, lane);
    }
    cp_async_commit();
}

// (192 registers leave room on the SM for a CTA of the merge kernel, which then
// has its place and counts ready when this grid ends.)
template <int NB>
__global__ void __maxnreg__(NB == 1 ? 192 : 255) decode_fp8_block_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(128) uint8_t smem[];
    // the merge kernel's CTAs may come in as soon as there is room: they wait for this grid's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ TileInfo infos[kWarps][kStages];
    __shared__ int warp_sum[kWarps];
    int* before = reinterpret_cast<int*>(smem + kWarps * kWarpBytes);
    int* lens = before + p.B + 1;
    const bool cuts = count_tiles(p, before, lens, warp_sum, blockIdx.x == 0);
    if (too_many_tiles(p)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) flag_status(p.status, ATTN_DEV_SEQ_TOO_LONG);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int total = before[p.B];
    const Cut cut(p.workers, total);
    const int whole_shares = min(p.workers, p.B);   // of whole sequences
    const int n_rows = p.G * p.nq;
    const int n_warps = gridDim.x * kWarps;
    uint8_t* ring = smem + warp * kWarpBytes;
    TileInfo* info = infos[warp];
    int k_at[2], v_at[2];   // K: chunks 2t4, 2t4 + 1 of row g; V: chunk g of rows 2t4, 2t4 + 1
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        k_at[i] = chunk_off(g, 2 * t4 + i);
        v_at[i] = kCodes + chunk_off(2 * t4 + i, g);
    }

    for (int unit = blockIdx.x * kWarps + warp; unit < p.workers * p.cols; unit += n_warps) {
        const int w = p.cols_div.div(unit), col = unit - w * p.cols;
        const int part_of_head = p.heads_div.div(col), kvh = col - part_of_head * p.Hkv, row0 = part_of_head * 8 * NB;
        const int rows = min(8 * NB, n_rows - row0);
        auto out_row = [&](int b, int r) -> size_t {   // row of [B, q_len, Hq]
            const int rr = row0 + r, i = p.group_div.div(rr);
            return (static_cast<size_t>(b) * p.nq + i) * p.Hq + static_cast<size_t>(kvh) * p.G + (rr - i * p.G);
        };
        // sequences without tokens: nothing is visible
        for (int b = w; b < p.B; b += p.workers) {
            if (before[b + 1] != before[b]) continue;
            for (int r = 0; r < rows; ++r) {
                const size_t row = out_row(b, r);
                reinterpret_cast<uint2*>(p.o + row * kD)[lane] = make_uint2(0u, 0u);
                if (p.lse != nullptr && lane == 0) p.lse[row] = -INFINITY;
            }
        }
        if (w >= (cuts ? cut.shares : whole_shares)) continue;
        int x = cuts ? cut.start(w) : before[w * p.B / whole_shares];
        const int x_end = cuts ? cut.start(w + 1) : before[(w + 1) * p.B / whole_shares];
        if (x >= x_end) continue;
        int b = warp_rank(p.B, x, lane, [&](int i) { return before[i]; });
        if (x >= before[b + 1] - kEnd) x = before[b + 1];   // only the end is left of it
        if (x >= x_end) continue;
        while (before[b + 1] <= x) ++b;
        Feed f;
        f.x = x;
        f.x_end = x_end;
        f.b = b;
        f.len = lens[b];
        feed_look(p, before, f, lane);
        // the queries' loads go ahead of the codes', the page's is on its way
        uint4 raw[NB][4];
        fetch_queries<NB>(p, b, kvh, row0, n_rows, lane, raw);
        Queries<NB> qs;
#pragma unroll 1
        for (int i = 0; i < kStages - 1; ++i) feed_tile(p, before, f, ring + i * 2 * kCodes, info + i, kvh, lane);
        int slot = 0;
        for (bool first = true; x < x_end; first = false) {
            while (before[b + 1] <= x) ++b;
            const int t_lo = x - before[b], n_tiles = before[b + 1] - before[b] - kEnd;
            const int t_hi = min(n_tiles, t_lo + (x_end - x));
            x = t_hi == n_tiles ? before[b + 1] : x_end;
            const int len = lens[b];
            if (!first) fetch_queries<NB>(p, b, kvh, row0, n_rows, lane, raw);
            take_queries<NB>(p, raw, row0, n_rows, len, lane, qs);
            State<NB> st;
            reset<NB>(st);
            const int lim_min = len - p.nq + p.group_div.div(row0);   // the first row's limit, the smallest
            for (int t = t_lo; t < t_hi; ++t) {
                cp_async_wait_group<kStages - 2>();
                __syncwarp();   // everyone's copies of this stage are there; the stage before it has been read
                const int next = slot == 0 ? kStages - 1 : slot - 1;
                feed_tile(p, before, f, ring + next * 2 * kCodes, info + next, kvh, lane);
                const uint8_t* codes = ring + slot * 2 * kCodes;
                const float ka[2] = {info[slot].k[0], info[slot].k[1]};
                const float vb[2] = {info[slot].v[0], info[slot].v[1]};
                const uint32_t valid = info[slot].valid;
                const int tok0 = t * kTile;
                if (valid == 0xffffffffu && tok0 + kTile - 1 <= lim_min)
                    tile_step<NB, false>(st, qs, codes, k_at, v_at, ka, vb, tok0, valid, lane);
                else
                    tile_step<NB, true>(st, qs, codes, k_at, v_at, ka, vb, tok0, valid, lane);
                slot = slot + 1 == kStages ? 0 : slot + 1;
            }
            // the piece's rows: normalised O and log2 of the sum
            const bool whole = t_lo == 0 && t_hi == n_tiles;
            const size_t part = (static_cast<size_t>(2 * w + (t_lo == 0 ? 1 : 0)) * p.cols + col) * (8 * NB);
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float l = st.l[n][j];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                    const int r = 8 * n + 2 * t4 + j;
                    if (r >= rows) continue;
                    // O = 2^(M - m) sum p b v / l; rows that saw nothing have l = 0
                    const float m = st.m[n][j], M = st.M[n][j];
                    const float f = l == 0.f || M == -INFINITY ? 0.f : ex2(M - m) / l;
                    const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
                    if (whole) {
                        const size_t row = out_row(b, r);
                        uint32_t u[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) u[i] = pack_bf16x2(st.o[n][i][j] * f, st.o[n][i][2 + j] * f);
                        uint4* dst = reinterpret_cast<uint4*>(p.o + row * kD + 16 * g);
                        dst[0] = make_uint4(u[0], u[1], u[2], u[3]);
                        dst[1] = make_uint4(u[4], u[5], u[6], u[7]);
                        if (p.lse != nullptr && g == 0) p.lse[row] = lse2 * kLn2;
                    } else {
                        float4* dst = reinterpret_cast<float4*>(p.part_o + (part + r) * kD + 16 * g);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            dst[i] = make_float4(st.o[n][2 * i][j] * f, st.o[n][2 * i][2 + j] * f,
                                                 st.o[n][2 * i + 1][j] * f, st.o[n][2 * i + 1][2 + j] * f);
                        if (g == 0) p.part_l[part + r] = lse2;
                    }
                }
        }
        __syncwarp();   // the ring may be filled for another unit
    }
}

// Joins the pieces of the sequences that were cut: 1 << per_shift warps (up to 8)
// per output row, four elements a lane.  O = sum_s 2^(L_s - L) O_s / sum_s
// 2^(L_s - L); each warp takes every per_row-th piece, kBatch at a time.  Each CTA
// counts the tiles of all sequences, also where its own was not cut: 32 heads over
// 8, 64 sequences of 300 tokens take 15.7 us in all (their bytes 6.0), 1024 take
// 123 (96), 4096 take 496 (386), and 4096 of 90 tokens 251 (123).
__global__ void __launch_bounds__(32 * kMergeWarps, 4) decode_fp8_block_merge_kernel(const __grid_constant__ Params p,
                                                                                  int rows_per_col, int per_shift) {
    __shared__ int sums[2][kMergeWarps];
    __shared__ float4 warp_acc[kMergeWarps][32];
    __shared__ float warp_top[kMergeWarps], warp_sum[kMergeWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = p.nq * p.Hq;
    const int per_row = 1 << per_shift, rows_per_cta = kMergeWarps >> per_shift;
    const int cta_per_seq = (rows + rows_per_cta - 1) / rows_per_cta;
    const int b = blockIdx.x / cta_per_seq, row = blockIdx.x % cta_per_seq * rows_per_cta + (warp >> per_shift);
    // spans before the sequence, and of all of them
    int pre = 0, all = 0;
    bool cuts = false;
    for (int i = threadIdx.x; i < p.B; i += 32 * kMergeWarps) {
        const int len = length_of(p, i, false), t = span_of(len);
        cuts |= tiles_of(len) > kWholeTiles;
        all += t;
        if (i < b) pre += t;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        pre += __shfl_xor_sync(0xffffffffu, pre, off);
        all += __shfl_xor_sync(0xffffffffu, all, off);
    }
    if (lane == 0) sums[0][warp] = pre, sums[1][warp] = all;
    cuts = __syncthreads_or(cuts) != 0;
    pre = all = 0;
#pragma unroll
    for (int i = 0; i < kMergeWarps; ++i) pre += sums[0][i], all += sums[1][i];
    const int n_tiles = tiles_of(length_of(p, b, false));
    const Cut cut(p.workers, all);
    int w0 = 0, w1 = 0;   // its first and last share
    if (n_tiles != 0 && cuts && !too_many_tiles(p)) w0 = cut.share_of(pre), w1 = cut.share_of(pre + n_tiles - 1);
    // the warp's pieces: n rows of the workspace from `base` on, `step` apart (the
    // piece that starts the sequence is its share's second slot, `first` rows on;
    // fewer than 2^31 elements: two slots for each of the grid's warps)
    const int r = (row / p.Hq) * p.G + row % p.G, skip = warp & (per_row - 1), slots = p.cols * rows_per_col;
    int n = row < rows && w0 + skip <= w1 ? ((w1 - w0 - skip) >> per_shift) + 1 : 0;
    int base = 2 * (w0 + skip) * slots + ((r / rows_per_col) * p.Hkv + row % p.Hq / p.G) * rows_per_col + r % rows_per_col;
    int step = (2 << per_shift) * slots, first = skip == 0 ? slots : 0;
    // the first kernel is done and its writes are here; CTAs without work wait
    // too, so that this grid never ends before that one.  What has been computed
    // is computed before.
    asm volatile("griddepcontrol.wait;" : "+r"(w0), "+r"(w1), "+r"(n), "+r"(base), "+r"(step), "+r"(first)::"memory");
    if (w0 == w1) return;   // one share held it all, or there is nothing
    float top = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (; n > 0; n -= kBatch, base += kBatch * step, first = 0) {
        const int m = min(kBatch, n);
        const float l = lane < m ? __ldcg(p.part_l + base + lane * step + (lane == 0 ? first : 0)) : -INFINITY;
        const float4* piece = reinterpret_cast<const float4*>(p.part_o) + base * (kD / 4) + lane;
        float4 v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (i < m) v[i] = __ldcg(piece + (i * step + (i == 0 ? first : 0)) * (kD / 4));
        float high = l;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, off));
        high = fmaxf(high, top);
        const float back = top == -INFINITY ? 0.f : ex2(top - high);
        top = high;
        sum *= back;
        acc.x *= back, acc.y *= back, acc.z *= back, acc.w *= back;
        const float f = l == -INFINITY ? 0.f : ex2(l - top);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const float fi = __shfl_sync(0xffffffffu, f, i);
            if (i < m && fi != 0.f) {
                sum += fi;
                acc.x = fmaf(fi, v[i].x, acc.x);
                acc.y = fmaf(fi, v[i].y, acc.y);
                acc.z = fmaf(fi, v[i].z, acc.z);
                acc.w = fmaf(fi, v[i].w, acc.w);
            }
        }
    }
    if (per_row > 1) {   // the row's warps, in order
        warp_acc[warp][lane] = acc;
        if (lane == 0) warp_top[warp] = top, warp_sum[warp] = sum;
        __syncthreads();
        if (skip != 0) return;
        for (int i = 0; i < per_row; ++i) top = fmaxf(top, warp_top[warp + i]);
        sum = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < per_row; ++i) {
            if (warp_sum[warp + i] == 0.f) continue;
            const float f = ex2(warp_top[warp + i] - top);
            const float4 a = warp_acc[warp + i][lane];
            sum = fmaf(f, warp_sum[warp + i], sum);
            acc.x = fmaf(f, a.x, acc.x);
            acc.y = fmaf(f, a.y, acc.y);
            acc.z = fmaf(f, a.z, acc.z);
            acc.w = fmaf(f, a.w, acc.w);
        }
    }
    if (row >= rows) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const size_t out = static_cast<size_t>(b) * rows + row;
    reinterpret_cast<uint2*>(p.o + out * kD)[lane] =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (p.lse != nullptr && lane == 0) p.lse[out] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// The grid's warps over columns of `per` rows.
void set_columns(Params& p, int per, int sms) {
    p.cols = p.Hkv * ((p.G * p.nq + per - 1) / per);
    p.workers = std::max(1, sms * kWarps / p.cols);
}

// Rows of the workspace.
size_t part_rows(const Params& p, int per) { return static_cast<size_t>(2) * p.workers * p.cols * per; }

// Rows of a column: 16 where a KV head has more than 8, but 8 while the tokens
// that the pool holds, or that a block table of its width can name, make short
// shares of such columns.  A tile of 8 rows costs a warp 0.7 of one of 16, all
// that runs once for a share less than half, and its kernel leaves room for the
// merge's: 4 queries of 8 heads over 2, 2400 tokens (1 tile a share) 11.6 us
// against 16.5; 8 sequences of 1000 and 64 rows (4) 15.7 against 17.6; 29 ragged
// ones of 12 rows, 32k tokens (13) 29.2 against 30.2; 24 of 4500 and 32 rows (22)
// 38.4 against 31.9.  The host does not know the lengths: in a pool far larger
// than the batch a CSR list always takes 16, and a block table unless it is
// narrow (in a pool of 64k pages the first two take 14.4 and 16.4 us by CSR list,
// 10.1 and 15.7 by a table 32768 tokens wide, 10.3 and 15.0 in a pool of their
// own).  Lists that share pages may name more tokens than the pool holds; the
// rule is then off, the result is not.
constexpr int kNarrowTiles = 12;
int rows_per_column(Params& p, int sms) {
    set_columns(p, 8, sms);
    const long long listed = p.list.indptr != nullptr ? p.list.num_pages
                                                      : std::min<long long>(p.list.num_pages, static_cast<long long>(p.B) * p.list.max_pages);
    const long long tiles = listed * p.list.page_size / kTile + static_cast<long long>(kEnd) * p.B;
    if (p.G * p.nq <= 8 || tiles <= static_cast<long long>(kNarrowTiles) * p.workers) return 8;
    set_columns(p, 16, sms);
    return 16;
}

}  // namespace

int decode_fp8_block_max_seqs() { return kMaxSeqs; }

size_t decode_fp8_block_workspace(int q_len, int Hq, int Hkv, int sms) {
    Params p{};
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.nq = q_len;
    size_t rows = 0;   // enough for columns of either height
    for (int per : {8, 16}) {
        set_columns(p, per, sms);
        if (per == 8 || p.G * p.nq > 8) rows = std::max(rows, part_rows(p, per));
    }
    return rows * (kD + 1) * sizeof(float);
}

cudaError_t launch_decode_fp8_block(const DecodeBlockArgs& a, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    Params p;
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.k_cache = static_cast<const uint8_t*>(a.k_cache);
    p.v_cache = static_cast<const uint8_t*>(a.v_cache);
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.list = PageList{a.block_table, a.kv_indptr, a.max_pages, a.num_pages, a.page_size};
    p.seq_lens = a.seq_lens;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.nq = a.q_len;
    p.page_div = make_divisor(a.page_size);
    p.block_div = make_divisor(a.block_tokens);
    p.heads_div = make_divisor(a.Hkv);
    p.group_div = make_divisor(p.G);
    p.page_blocks = a.page_size / a.block_tokens;
    p.tile_in_page = a.page_size % kTile == 0;
    const int per = rows_per_column(p, sms);
    p.cols_div = make_divisor(p.cols);
    p.scale_log2 = a.scale * kLog2e;
    p.o = static_cast<__nv_bfloat16*>(a.o);
    p.lse = a.lse;
    p.part_o = static_cast<float*>(a.workspace);
    p.part_l = p.part_o + part_rows(p, per) * kD;
    p.status = a.dev_status;
    const size_t smem = kWarps * kWarpBytes + (2 * static_cast<size_t>(a.B) + 1) * sizeof(int);
    auto kern = per == 8 ? decode_fp8_block_kernel<1> : decode_fp8_block_kernel<2>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = once_per_device(done, [] {
        // both kernels with the same division of L1, so that neither waits for it to change
        cudaError_t r = cudaFuncSetAttribute(decode_fp8_block_merge_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                             cudaSharedmemCarveoutMaxShared);
        for (auto k : {decode_fp8_block_kernel<1>, decode_fp8_block_kernel<2>}) {
            if (r == cudaSuccess)
                r = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kWarps * kWarpBytes + (2 * kMaxSeqs + 1) * static_cast<int>(sizeof(int)));
            if (r == cudaSuccess)
                r = cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        }
        return r;
    });
    if (e != cudaSuccess) return e;
    kern<<<sms, kThreads, smem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.workers == 1) return e;   // one share per column: no sequence is cut
    // a sequence has about workers / B pieces, one that is longer than the others
    // more: as many warps to a row as there are kBatch pieces for, while the CTAs
    // (four fit on an SM) fit at once (one for every two pieces took 0.9 % longer
    // over 164 batches of all sizes)
    const long long all_rows = static_cast<long long>(a.B) * a.q_len * a.Hq;
    int per_shift = 0;
    while ((1 << per_shift) < kMergeWarps && p.workers > (static_cast<long long>(kBatch) << per_shift) * a.B &&
           all_rows << (per_shift + 1) <= 4LL * sms * kMergeWarps)
        ++per_shift;
    const int rows_per_cta = kMergeWarps >> per_shift;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B) * ((a.q_len * a.Hq + rows_per_cta - 1) / rows_per_cta));
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode_fp8_block_merge_kernel, p, per, per_shift);
}

}  // namespace gb300
