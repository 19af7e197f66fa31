// cross_decode.cu - single tokens' attention to an encoder's states: one to
// sixteen queries per sequence, all of which see every key.
//
// Mathematics, per query row r of a KV head:
//   s_t = scale (q_r . k_t),  O_r = sum_t p_t v_t / sum_t p_t,
//   p_t = 2^(log2e s_t - m),  over the sequence's keys.
// The products are m16n8k16 bf16 MMAs with the keys as the 16 rows, so that up
// to 8 (or 16) query rows cost no more than one; p_t is rounded to bf16 for the
// second (2^-8 of it at most).  Scores, maxima and sums are fp32.
//
// Work: a column is a KV head with a group of up to 8 or 16 (query, head) rows;
// every warp of the grid takes one column and an equal share of the 16-key tiles
// of all sequences, whatever their lengths, which only the device knows (a batch
// of short ones goes by whole sequences).  Tiles come by TMA, each warp into a
// ring of its own, so that warps wait for nothing but their own tiles.  A share
// that holds a whole sequence writes its output; the pieces of one that is cut
// go to the workspace, and a second kernel, which is launched along with the
// first and waits for it on the device, joins them in order.
//
// Bound: one read of the keys and values for every 16 rows of a KV head (more rows
// take columns of their own, which read them again: 16 sequences of 4096 keys, 16
// queries of 64 heads over 8, 180 us where one read takes 40).  64 sequences of 512
// to 6400 keys, four beams, 32 heads over 8 (819 MB): 138 us, 5.9 TB/s.  One sequence
// of 1500 keys: 8.6 us in a graph (launches, one tile, the join), 10.3 in a stream.
// Tried: shares of at least two to six tiles, more registers (no gain); the join's
// CTAs over several rows each (64 x 4 beams 1 % faster, one sequence a launch interval
// slower).
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "paged.cuh"
#include "ptx.cuh"
#include "shares.cuh"

namespace gb300 {
namespace {

constexpr int kTile = 16;       // keys per step of a warp
constexpr int kWarps = 8;       // per CTA
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxSeqs = 4096;  // tile counts before each sequence in shared memory
// A sequence's end (the piece's rows, the next queries) counts as so many tiles in
// the cut: 64 sequences of 500 to 6300 keys 136.0 us, with one 137.1, with four 136.4.
constexpr int kEnd = 2;
// Where no sequence has more tiles, none is cut: 16 sequences of 60 keys 7.6 us,
// cut 7.9; 32 of 200 keys whole 13.5 us, cut 8.5.
constexpr int kWholeTiles = 6;
// More spans than this (rising offsets have fewer than 2^26 + 3 kMaxSeqs) are not worked
// on: offsets that fall can name the same keys for every sequence.
constexpr int kMostSpans = 1 << 28;
constexpr int kMergeWarps = 8;
constexpr int kBatch = 8;       // pieces a merging warp has in flight

// Bytes of a tile's keys (or values), tiles in flight or in use per warp: 192 KB in all.
template <int kD>
constexpr int tile_bytes() { return kTile * kD * 2; }
template <int kD>
constexpr int stages() { return kD == 64 ? 6 : 3; }

struct Params {
    const __nv_bfloat16* q;   // [B, q_len, Hq, D]
    const int32_t* kv_indptr;
    const int32_t* kv_lens;   // may be NULL
    Divisor cols_div, heads_div, group_div;
    int B, total_kv, Hq, Hkv, G, nq;
    int cols;       // KV heads x row groups
    int workers;    // shares per column
    float scale_log2;
    __nv_bfloat16* o;
    float* lse;     // may be NULL
    float* part_o;  // [2 workers][cols][rows][D]
    float* part_l;  // [2 workers][cols][rows], log2
    int32_t* status;
};

// m16n8k16 bf16 MMA, fp32 accumulators; not volatile, so that independent ones
// may be interleaved.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// First key row of sequence b and how many it has, offsets outside the tensor cut to it.
__device__ __forceinline__ int start_of(const Params& p, int b) { return min(max(p.kv_indptr[b], 0), p.total_kv); }
__device__ __forceinline__ int length_of(const Params& p, int b) {
    const int start = start_of(p, b), room = min(max(p.kv_indptr[b + 1], start), p.total_kv) - start;
    return p.kv_lens != nullptr ? min(max(p.kv_lens[b], 0), room) : room;
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }
// What a sequence counts for in the cut: its tiles, and its end.
__device__ __forceinline__ int span_of(int len) { return len > 0 ? tiles_of(len) + kEnd : 0; }

// before[b] = spans of the sequences before b (before[B] = all), by the whole
// CTA: each thread takes a run of sequences.  Returns whether one of them has
// more than kWholeTiles tiles.
__device__ __forceinline__ bool count_tiles(const Params& p, int* before, int* lens, int* warp_sum) {
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(static_cast<int>(threadIdx.x) * per, p.B), b1 = min(b0 + per, p.B);
    int sum = 0, most = 0;
    for (int b = b0; b < b1; ++b) {
        lens[b] = length_of(p, b);
        sum += span_of(lens[b]);
        most = max(most, tiles_of(lens[b]));
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl = add_capped(incl, v);
    }
    int base = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane == 0) base = 0;
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    for (int w = 0; w < warp; ++w) base = add_capped(base, warp_sum[w]);
    for (int b = b0; b < b1; ++b) {
        before[b] = base;
        base = add_capped(base, span_of(lens[b]));
    }
    if (threadIdx.x == kThreads - 1) before[p.B] = base;   // the last run ends with the last sequence, or is empty
    return __syncthreads_or(most > kWholeTiles) != 0;
}

// The tiles of a warp's share, fetched ahead: `x` is the next one, in sequence b;
// `count` tiles have been asked for.
struct Feed {
    int x, x_end, b;
    uint32_t count;
};

template <int kD>
__device__ __forceinline__ void feed_tile(const Params& p, const CUtensorMap* k_map, const CUtensorMap* v_map,
                                          const int* before, Feed& f, uint8_t* ring, uint64_t* full, int kvh, int lane) {
    if (f.x >= before[f.b + 1] - kEnd) f.x = before[f.b + 1];   // past the sequence's end
    if (f.x >= f.x_end) return;
    while (before[f.b + 1] <= f.x) ++f.b;
    if (lane == 0) {
        const int s = static_cast<int>(f.count % stages<kD>()), row = start_of(p, f.b) + (f.x - before[f.b]) * kTile;
        uint8_t* dst = ring + s * 2 * tile_bytes<kD>();
        mbar_arrive_expect_tx(&full[s], 2 * tile_bytes<kD>());
#pragma unroll
        for (int h = 0; h < kD / 64; ++h) {
            tma_load_2d(dst + h * kTile * 128, k_map, &full[s], kvh * kD + 64 * h, row);
            tma_load_2d(dst + tile_bytes<kD>() + h * kTile * 128, v_map, &full[s], kvh * kD + 64 * h, row);
        }
    }
    ++f.x;
    ++f.count;
}

// (192 KB of rings: one CTA per SM, and the merge kernel's CTAs beside it.)
template <int kD, int NB>
__global__ void __launch_bounds__(kThreads, 1)
    cross_decode_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                        const __grid_constant__ Params p) {
    constexpr int kStages = stages<kD>(), kBytes = tile_bytes<kD>(), kSteps = kD / 16;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_1024(smem_raw);
    // the merge kernel's CTAs may come in as soon as there is room: they wait for this grid's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ __align__(8) uint64_t full_all[kWarps][kStages];
    __shared__ int warp_sum[kWarps];
    int* before = reinterpret_cast<int*>(smem + kWarps * kStages * 2 * kBytes);
    int* lens = before + p.B + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    if (threadIdx.x < kWarps * kStages) mbar_init(&full_all[0][0] + threadIdx.x, 1);
    fence_mbar_init();
    const bool cuts = count_tiles(p, before, lens, warp_sum);   // (ends with a barrier of the CTA)
    if (before[p.B] > kMostSpans) {
        if (threadIdx.x == 0) flag_status(p.status, ATTN_DEV_SEQ_TOO_LONG);
        return;
    }
    const Cut cut(p.workers, before[p.B]);
    const int whole_shares = min(p.workers, p.B);   // of whole sequences
    const int n_rows = p.G * p.nq;
    const int n_warps = gridDim.x * kWarps;
    uint8_t* ring = smem + warp * kStages * 2 * kBytes;
    uint64_t* full = full_all[warp];
    uint32_t used = 0;   // tiles this warp has gone through
    Feed f{0, 0, 0, 0};
    // ldmatrix addresses within a tile: keys (lane & 7) + 8 (i & 1) with the
    // chunks of i >> 1, values (lane & 7) + 8 (i >> 1) with those of i & 1 (i =
    // lane / 8); 128-byte swizzle, chunk XOR row
    const int mi = lane >> 3;
    const uint32_t k_row = (lane & 7) + 8 * (mi & 1), v_row = (lane & 7) + 8 * (mi >> 1), swz = lane & 7;

    for (int unit = blockIdx.x * kWarps + warp; unit < p.workers * p.cols; unit += n_warps) {
        const int w = p.cols_div.div(unit), col = unit - w * p.cols;
        const int part_of_head = p.heads_div.div(col), kvh = col - part_of_head * p.Hkv, row0 = part_of_head * 8 * NB;
        const int rows = min(8 * NB, n_rows - row0);
        auto out_row = [&](int b, int r) -> size_t {   // row of [B, q_len, Hq]
            const int rr = row0 + r, i = p.group_div.div(rr);
            return (static_cast<size_t>(b) * p.nq + i) * p.Hq + static_cast<size_t>(kvh) * p.G + (rr - i * p.G);
        };
        // sequences without keys: nothing is visible
        for (int b = w; b < p.B; b += p.workers) {
            if (before[b + 1] != before[b]) continue;
            for (int r = 0; r < rows; ++r) {
                const size_t row = out_row(b, r);
                for (int e = lane; e < kD / 2; e += 32) reinterpret_cast<uint32_t*>(p.o + row * kD)[e] = 0u;
                if (p.lse != nullptr && lane == 0) p.lse[row] = -INFINITY;
            }
        }
        if (w >= (cuts ? cut.shares : whole_shares)) continue;
        int x = cuts ? cut.start(w) : before[static_cast<long long>(w) * p.B / whole_shares];
        const int x_end = cuts ? cut.start(w + 1) : before[static_cast<long long>(w + 1) * p.B / whole_shares];
        if (x >= x_end) continue;
        int lo = 0, hi = p.B;   // the last sequence that starts at x or before
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before[mid] <= x) lo = mid; else hi = mid;
        }
        int b = lo;
        if (x >= before[b + 1] - kEnd) x = before[b + 1];   // only the end is left of it
        if (x >= x_end) continue;
        while (before[b + 1] <= x) ++b;
        f.x = x;
        f.x_end = x_end;
        f.b = b;
#pragma unroll 1
        for (int i = 0; i < kStages - 1; ++i) feed_tile<kD>(p, &k_map, &v_map, before, f, ring, full, kvh, lane);
        while (x < x_end) {
            while (before[b + 1] <= x) ++b;
            const int t_lo = x - before[b], n_tiles = before[b + 1] - before[b] - kEnd;
            const int t_hi = min(n_tiles, t_lo + (x_end - x));
            x = t_hi == n_tiles ? before[b + 1] : x_end;
            const int len = lens[b];
            // queries as B fragments: column g of block n is row n * 8 + g
            uint32_t qf[NB][kSteps][2];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const bool there = 8 * n + g < rows;
                const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + out_row(b, there ? 8 * n + g : 0) * kD) + t4;
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks) {
                    qf[n][ks][0] = there ? __ldg(src + 8 * ks) : 0u;
                    qf[n][ks][1] = there ? __ldg(src + 8 * ks + 4) : 0u;
                }
            }
            float o[NB][kSteps][4], m[NB][2], l[NB][2];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
#pragma unroll
                for (int i = 0; i < kSteps; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
                m[n][0] = m[n][1] = -INFINITY;
                l[n][0] = l[n][1] = 0.f;
            }
            for (int t = t_lo; t < t_hi; ++t, ++used) {
                const int s = static_cast<int>(used % kStages);
                if (!mbar_wait(&full[s], (used / kStages) & 1)) {
                    flag_status(p.status, ATTN_DEV_WAIT_TIMEOUT);
                    return;
                }
                __syncwarp();   // everyone has read the stage before, which is filled again
                feed_tile<kD>(p, &k_map, &v_map, before, f, ring, full, kvh, lane);
                uint8_t* kt = ring + s * 2 * kBytes;
                uint8_t* vt = kt + kBytes;
                const int there = len - t * kTile;
                if (there < kTile) {
                    // a weight of 0 times what lies behind the keys need not be 0
                    for (int i = there * 8 + lane; i < kTile * 8; i += 32)
#pragma unroll
                        for (int h = 0; h < kD / 64; ++h)
                            reinterpret_cast<uint4*>(vt + h * kTile * 128)[i] = make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();   // the stage is filled by TMA again
                    __syncwarp();
                }
                const uint32_t ka = smem_u32(kt) + k_row * 128, va = smem_u32(vt) + v_row * 128;
                float sc[NB][4];
#pragma unroll
                for (int n = 0; n < NB; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks) {
                    uint32_t a[4];
                    ldmatrix_x4(a[0], a[1], a[2], a[3],
                                ka + (ks >> 2) * kTile * 128 + (((2 * (ks & 3) + (mi >> 1)) ^ swz) << 4));
#pragma unroll
                    for (int n = 0; n < NB; ++n) mma16816(sc[n], a, qf[n][ks][0], qf[n][ks][1]);
                }
                bool over = false;
#pragma unroll
                for (int n = 0; n < NB; ++n) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sc[n][e] *= p.scale_log2;
                        if (g + 8 * (e >> 1) >= there) sc[n][e] = -INFINITY;
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) over |= fmaxf(sc[n][j], sc[n][2 + j]) > m[n][j] + 8.f;
                }
                // running maxima, raised (and the sums rescaled) only when a score passes them by 2^8
                if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float mx = fmaxf(sc[n][j], sc[n][2 + j]);
#pragma unroll
                            for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                            if (mx > m[n][j]) {
                                const float alpha = ex2(m[n][j] - mx);
                                m[n][j] = mx;
                                l[n][j] *= alpha;
#pragma unroll
                                for (int i = 0; i < kSteps; ++i) {
                                    o[n][i][j] *= alpha;
                                    o[n][i][2 + j] *= alpha;
                                }
                            }
                        }
                }
                uint32_t w0[NB], w1[NB];
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    float e[4];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float mm = m[n][j] == -INFINITY ? 0.f : m[n][j];
                        e[j] = ex2(sc[n][j] - mm);
                        e[2 + j] = ex2(sc[n][2 + j] - mm);
                        l[n][j] += e[j] + e[2 + j];
                    }
                    w0[n] = movmatrix_trans(pack_bf16x2(e[0], e[1]));
                    w1[n] = movmatrix_trans(pack_bf16x2(e[2], e[3]));
                }
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    uint32_t a[4];
                    ldmatrix_x4_trans(a[0], a[1], a[2], a[3],
                                      va + (i >> 2) * kTile * 128 + (((2 * (i & 3) + (mi & 1)) ^ swz) << 4));
#pragma unroll
                    for (int n = 0; n < NB; ++n) mma16816(o[n][i], a, w0[n], w1[n]);
                }
            }
            // the piece's rows: normalised O and log2 of the sum
            const bool whole = t_lo == 0 && t_hi == n_tiles;
            const size_t part = (static_cast<size_t>(2 * w + (t_lo == 0 ? 1 : 0)) * p.cols + col) * (8 * NB);
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                float inv[2], lse2[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], off);
                    inv[j] = l[n][j] == 0.f ? 0.f : 1.f / l[n][j];
                    lse2[j] = l[n][j] == 0.f ? -INFINITY : m[n][j] + log2f(l[n][j]);
                    const int r = 8 * n + 2 * t4 + j;
                    if (g == 0 && r < rows) {
                        if (!whole) p.part_l[part + r] = lse2[j];
                        else if (p.lse != nullptr) p.lse[out_row(b, r)] = lse2[j] * kLn2;
                    }
                }
                if (whole) {
                    // (row, element) pairs of an 8x8 block turned: lane g has row g, elements 2 t4, 2 t4 + 1
                    const bool there = 8 * n + g < rows;
                    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + out_row(b, there ? 8 * n + g : 0) * kD) + t4;
#pragma unroll
                    for (int i = 0; i < kSteps; ++i)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const uint32_t v = movmatrix_trans(pack_bf16x2(o[n][i][2 * c] * inv[0], o[n][i][2 * c + 1] * inv[1]));
                            if (there) dst[8 * i + 4 * c] = v;
                        }
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = 8 * n + 2 * t4 + j;
                        if (r >= rows) continue;
                        float* dst = p.part_o + (part + r) * kD + g;
#pragma unroll
                        for (int i = 0; i < kSteps; ++i) {
                            dst[16 * i] = o[n][i][j] * inv[j];
                            dst[16 * i + 8] = o[n][i][2 + j] * inv[j];
                        }
                    }
                }
            }
        }
        __syncwarp();   // the ring may be filled for another unit
    }
}

// Joins the pieces of the sequences that were cut: 1 << per_shift warps (up to 8)
// per output row.  O = sum_s 2^(L_s - L) O_s / sum_s 2^(L_s - L); each warp takes
// every per_row-th piece, kBatch at a time (of which only those that are there are
// loaded: 64 x 4 beams 140 -> 138 us), and the warps are joined in order.
template <int kD>
__global__ void __launch_bounds__(32 * kMergeWarps, 4) cross_decode_merge_kernel(const __grid_constant__ Params p,
                                                                                 int rows_per_col, int per_shift) {
    constexpr int kEach = kD / 32;
    __shared__ int sums[2][kMergeWarps];
    __shared__ float warp_acc[kMergeWarps][kD];
    __shared__ float warp_top[kMergeWarps], warp_all[kMergeWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = p.nq * p.Hq;
    const int per_row = 1 << per_shift, rows_per_cta = kMergeWarps >> per_shift;
    const int cta_per_seq = (rows + rows_per_cta - 1) / rows_per_cta;
    const int b = blockIdx.x / cta_per_seq, row = blockIdx.x % cta_per_seq * rows_per_cta + (warp >> per_shift);
    // spans before the sequence, and of all of them
    int pre = 0, all = 0;
    bool cuts = false;
    for (int i = threadIdx.x; i < p.B; i += 32 * kMergeWarps) {
        const int len = length_of(p, i), t = span_of(len);
        cuts |= tiles_of(len) > kWholeTiles;
        all = add_capped(all, t);
        if (i < b) pre = add_capped(pre, t);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        pre = add_capped(pre, __shfl_xor_sync(0xffffffffu, pre, off));
        all = add_capped(all, __shfl_xor_sync(0xffffffffu, all, off));
    }
    if (lane == 0) sums[0][warp] = pre, sums[1][warp] = all;
    cuts = __syncthreads_or(cuts) != 0;
    pre = all = 0;
#pragma unroll
    for (int i = 0; i < kMergeWarps; ++i) pre = add_capped(pre, sums[0][i]), all = add_capped(all, sums[1][i]);
    const int n_tiles = tiles_of(length_of(p, b));
    const Cut cut(p.workers, all);
    int w0 = 0, w1 = 0;   // its first and last share
    if (n_tiles != 0 && cuts && all <= kMostSpans) w0 = cut.share_of(pre), w1 = cut.share_of(pre + n_tiles - 1);
    // the first kernel is done and its writes are here; CTAs without work wait
    // too, so that this grid never ends before that one
    asm volatile("griddepcontrol.wait;" : "+r"(w0), "+r"(w1)::"memory");
    if (w0 == w1) return;   // one share held it all, or there is nothing
    const int skip = warp & (per_row - 1);
    const int i = row / p.Hq, head = row - i * p.Hq, kvh = head / p.G, r = i * p.G + head - kvh * p.G;
    const int col = (r / rows_per_col) * p.Hkv + kvh;
    auto slot = [&](int w) {   // the piece that starts the sequence is its share's second one
        return (static_cast<size_t>(2 * w + (w == w0 ? 1 : 0)) * p.cols + col) * rows_per_col + r % rows_per_col;
    };
    float top = -INFINITY, sum = 0.f, acc[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) acc[e] = 0.f;
    for (int w = w0 + skip; row < rows && w <= w1; w += kBatch << per_shift) {
        const int mine = w + (lane << per_shift);
        const float l = lane < kBatch && mine <= w1 ? __ldcg(p.part_l + slot(mine)) : -INFINITY;
        float v[kBatch][kEach];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int at = w + (k << per_shift);
            const float* src = p.part_o + slot(at) * kD + lane * kEach;
#pragma unroll
            for (int e = 0; e < kEach; e += 2) {
                const float2 u = at <= w1 ? __ldcg(reinterpret_cast<const float2*>(src + e)) : make_float2(0.f, 0.f);
                v[k][e] = u.x, v[k][e + 1] = u.y;
            }
        }
        float high = l;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, off));
        high = fmaxf(high, top);
        const float back = top == -INFINITY ? 0.f : ex2(top - high);
        top = high;
        sum *= back;
#pragma unroll
        for (int e = 0; e < kEach; ++e) acc[e] *= back;
        const float fl = l == -INFINITY ? 0.f : ex2(l - top);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const float fk = __shfl_sync(0xffffffffu, fl, k);
            if (fk == 0.f) continue;   // no such piece, or one that adds nothing
            sum += fk;
#pragma unroll
            for (int e = 0; e < kEach; ++e) acc[e] = fmaf(fk, v[k][e], acc[e]);
        }
    }
    if (per_row > 1) {   // the row's warps, in order
#pragma unroll
        for (int e = 0; e < kEach; ++e) warp_acc[warp][lane * kEach + e] = acc[e];
        if (lane == 0) warp_top[warp] = top, warp_all[warp] = sum;
        __syncthreads();
        if (skip != 0) return;
        for (int k = 0; k < per_row; ++k) top = fmaxf(top, warp_top[warp + k]);
        sum = 0.f;
#pragma unroll
        for (int e = 0; e < kEach; ++e) acc[e] = 0.f;
        for (int k = 0; k < per_row; ++k) {
            if (warp_all[warp + k] == 0.f) continue;
            const float fk = ex2(warp_top[warp + k] - top);
            sum = fmaf(fk, warp_all[warp + k], sum);
#pragma unroll
            for (int e = 0; e < kEach; ++e) acc[e] = fmaf(fk, warp_acc[warp + k][lane * kEach + e], acc[e]);
        }
    }
    if (row >= rows) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const size_t out = static_cast<size_t>(b) * rows + row;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + out * kD) + lane * (kEach / 2);
#pragma unroll
    for (int e = 0; e < kEach / 2; ++e) dst[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if (p.lse != nullptr && lane == 0) p.lse[out] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// The grid's warps over columns of 8 rows, or 16 where a KV head has more than 8.
int set_columns(Params& p, int sms) {
    const int per = p.G * p.nq <= 8 ? 8 : 16;
    p.cols = p.Hkv * ((p.G * p.nq + per - 1) / per);
    p.workers = std::max(1, sms * kWarps / p.cols);
    return per;
}

size_t part_rows(const Params& p, int per) { return static_cast<size_t>(2) * p.workers * p.cols * per; }

template <int kD>
cudaError_t launch(const CrossDecodeArgs& a, const Params& p, int per, int sms, const CUtensorMap& k, const CUtensorMap& v,
                   cudaStream_t stream) {
    constexpr size_t kRings = static_cast<size_t>(kWarps) * stages<kD>() * 2 * tile_bytes<kD>() + 1024;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = once_per_device(done, [] {
        // both kernels with the same division of L1, so that neither waits for it to change
        cudaError_t r = cudaFuncSetAttribute(cross_decode_merge_kernel<kD>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                             cudaSharedmemCarveoutMaxShared);
        for (auto kern : {cross_decode_kernel<kD, 1>, cross_decode_kernel<kD, 2>}) {
            if (r == cudaSuccess)
                r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kRings + (2 * kMaxSeqs + 1) * sizeof(int)));
            if (r == cudaSuccess)
                r = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        }
        return r;
    });
    if (e != cudaSuccess) return e;
    auto kern = per == 8 ? cross_decode_kernel<kD, 1> : cross_decode_kernel<kD, 2>;
    kern<<<sms, kThreads, kRings + (2 * static_cast<size_t>(a.B) + 1) * sizeof(int), stream>>>(k, v, p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.workers == 1) return e;   // one share per column: no sequence is cut
    // as many warps to a row as there are kBatch pieces for, while the CTAs (four fit on an SM) fit at once
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
    return cudaLaunchKernelEx(&cfg, cross_decode_merge_kernel<kD>, p, per, per_shift);
}

}  // namespace

int cross_decode_max_seqs() { return kMaxSeqs; }

size_t cross_decode_workspace(int q_len, int Hq, int Hkv, int D, int sms) {
    Params p{};
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.nq = q_len;
    const int per = set_columns(p, sms);
    return part_rows(p, per) * (D + 1) * sizeof(float);
}

cudaError_t launch_cross_decode(const CrossDecodeArgs& a, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    Params p{};
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.kv_indptr = a.kv_indptr;
    p.kv_lens = a.kv_lens;
    p.B = a.B;
    p.total_kv = a.total_kv;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.nq = a.q_len;
    const int per = set_columns(p, sms);
    p.cols_div = make_divisor(p.cols);
    p.heads_div = make_divisor(a.Hkv);
    p.group_div = make_divisor(p.G);
    p.scale_log2 = a.scale * kLog2e;
    p.o = static_cast<__nv_bfloat16*>(a.o);
    p.lse = a.lse;
    p.part_o = static_cast<float*>(a.workspace);
    p.part_l = p.part_o + part_rows(p, per) * a.D;
    p.status = a.dev_status;
    CUtensorMap k{}, v{};   // without keys neither is used
    if (a.total_kv > 0) {
        const uint64_t dims[2] = {static_cast<uint64_t>(a.Hkv) * a.D, static_cast<uint64_t>(a.total_kv)};
        const uint64_t ks[1] = {static_cast<uint64_t>(a.k_stride) * 2}, vs[1] = {static_cast<uint64_t>(a.v_stride) * 2};
        const uint32_t box[2] = {64, kTile};
        if (!encode_tiled_map(&k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.k, dims, ks, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_tiled_map(&v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.v, dims, vs, box, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    return a.D == 64 ? launch<64>(a, p, per, sms, k, v, stream) : launch<128>(a, p, per, sms, k, v, stream);
}

}  // namespace gb300
