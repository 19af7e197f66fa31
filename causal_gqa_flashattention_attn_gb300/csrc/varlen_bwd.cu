// varlen_bwd.cu - gradient of attention over contiguous keys, on the
// 5th-generation tensor cores.
//
// Mathematics, per sequence and head, with S = Q K^T and the forward pass's LSE:
//   P = exp(scale S - LSE),  delta = sum_d dO O - dLSE,
//   dV = P^T dO,  dP = dO V^T,  dS = P (dP - delta),
//   dQ = scale dS K,  dK = scale dS^T Q,
// dK and dV summed over the query heads of a KV head.  P is at most 1 and needs
// no running maximum.  P and dS are rounded to bf16 for their products (2^-8 of
// each at most); everything else is fp32.
//
// Two kernels, each its own pass over the tiles, so that every gradient is
// accumulated in one place and in one order: five products would do with dQ
// added up through global atomics, but then its rounding depends on timing.
//   dK, dV: a CTA owns 128 keys of a KV head; the tiles of its queries stream by.
//           S^T = K Q^T and dP^T = V dO^T are computed transposed, so that P^T
//           and dS^T go back to TMEM as the A operands of dV += P^T dO and
//           dK += dS^T Q and never touch shared memory;
//   dQ:     a CTA owns a tile of queries; the key tiles stream by:
//           S = Q K^T, dP = dO V^T, dQ += dS K.
// As in the forward kernel a tile of queries holds P = floor(128 / G) positions
// of all G heads of a KV head, position-major.
//
// Warp 0 loads by TMA, warp 1 issues the MMAs, warp 2 brings the queries' LSE and
// delta to the dK/dV kernel, warps 4-11 turn scores into P and dS (32 rows of the
// tile and half of its columns each).  The S and dP products of the
// next tile are issued while dS and P of this one are made: the tensor core
// waits for neither in turn.  TMEM: S 128 columns, dP 128, dV 128, dK 128 (in
// the dQ kernel a second S, or with D = 64 a second dP, and dQ).
//
// A first kernel computes delta and lists the blocks of all sequences, those of
// the longest first.  Few blocks are cut into parts along the streamed side,
// whose fp32 sums a last kernel adds up in order.
//
// Bound: the tensor cores.  Seven products, two more than atomics would need: 4
// sequences of 2048 queries of 32 heads to 4096 keys (1.37e12 FLOP of five, 1.92e12
// of seven) take 1138 us, 1245 in a long run (power), 1.7 PFLOP/s of the seven.  A
// step of dK/dV is about 2500 cycles, 78 an MMA, of dQ 2020, 84 an MMA; a CTA
// costs 9 and 5 us beside its steps (first loads, filling and draining, the rows
// out), more of the whole where blocks are short: 8 causal documents of 256 to
// 4096 tokens (1.04e12) 1105 us; 8 sequences of 20 queries to 1500 keys of 12
// heads, D = 64, 70 us, where the bytes need 11.
// Tried and slower: sixteen score warps (1570 -> 1641 us with an earlier MMA loop),
// all stages of a dQ step unrolled (9 %), first loads issued before the CTA has met
// (no change), a sequence's CTAs head by head (causal 4 %).
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "ptx.cuh"

namespace gb300 {
namespace {

constexpr int kBM = 128;        // rows and columns of a tile
constexpr int kThreads = 384;
constexpr int kProducerWarp = 0, kMmaWarp = 1, kStatWarp = 2;
constexpr int kScoreWarp = 4, kScoreThreads = 256;   // the first of eight
// Registers: launched at 168 per thread (384 x 168 = 64512); 2 x 128 x 208 + 128 x 88 = 64512.
constexpr uint32_t kRegsSoftmax = 208, kRegsControl = 88;
constexpr int kHalf = 128 * 128;   // bytes of one 64-column half of a 128-row tile
constexpr int kTile = 2 * kHalf;
constexpr int kStatSlots = 2;
// Stages of the streamed tiles: three of the first (Q, or K), two of the second
// (dO, or V).  A stage is free when a product issued after its last reader is
// done (MMAs complete in order), which is announced anyway:
//   dK, dV: Q after dK, by dP of the next tile; dO after dV, by S of the next tile;
//   dQ:     K after dQ, by dP of the next tile (D = 64: by dQ's own end); V after
//           its dP.
// The first is wanted half a step later than it would be free with two stages,
// less than a load takes: two stages of Q cost 550 to 1000 cycles a step of 3500.
constexpr int kStages1 = 3, kStages2 = 2;
// Shared memory, by addresses that are constants (the barriers and what the
// system reserves lie below kOffR1): two resident tiles, then the stages of the
// second streamed one and of the first, then (dK, dV) the queries' statistics.
// With them, and TMEM taken whole (its columns start at 0), every operand of
// every MMA but a stage is an immediate.
constexpr int kOffR1 = 2048, kOffR2 = kOffR1 + kTile;
constexpr int kOffY2 = kOffR2 + kTile;
constexpr int kOffY1 = kOffY2 + kStages2 * kTile;
constexpr int kOffStat = kOffY1 + kStages1 * kTile;
constexpr int kEnd = kOffStat + kStatSlots * 2 * kBM * 4;
// Barriers and words, where the dynamic part starts: behind the system's 1024
// bytes (there is no static part).
struct Control {
    uint64_t r_full, y1_full[kStages1], y2_full[kStages2];
    uint64_t s_full[2], dp_full[2];   // of even and odd tiles
    uint64_t p_ready, ds_ready, acc_full;   // (dQ with D = 64: p_ready is that S is read)
    uint64_t sum_done[2];                   // dQ with D = 64: of even and odd tiles
    uint64_t stat_full[kStatSlots], stat_empty[kStatSlots];
    uint32_t tmem_base;
    int abort;
};
constexpr int kSystem = 1024, kSmemBytes = kEnd - kSystem;
static_assert(kSystem + sizeof(Control) <= kOffR1 && kSmemBytes <= 227 * 1024, "all of an SM's shared memory");
// TMEM columns
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColDP = 128, kColAcc1 = 256, kColAcc2 = 384;   // dV, dK; or a second S or dP, dQ

struct Seq {
    int q_start, q_len, kv_start, kv_len, kv_room;
};
struct alignas(16) Block {   // block `at` of a sequence
    Seq s;
    int at, pad[2];
};

struct Params {
    const __nv_bfloat16* o;       // prepare
    const __nv_bfloat16* d_o;
    long long o_stride, do_stride;
    const float* lse;
    const float* d_lse;           // may be NULL
    const int32_t *qo_indptr, *kv_indptr, *kv_lens;
    int causal, B, total_q, total_kv, Hq, Hkv, G, P;
    float scale, scale_log2;
    float2* stats;                // [total_q * Hq] (-log2e LSE, -delta)
    int* counts;                  // blocks of keys, blocks of queries
    Block* kv_blocks;             // longest first
    Block* q_blocks;
    int max_kv_blocks, max_q_blocks, kv_pieces, q_pieces;
    __nv_bfloat16 *dq, *dk, *dv;
    long long dq_stride, dk_stride, dv_stride;
    float *dq_part, *dk_part, *dv_part;   // [pieces][rows][heads][D]
    int32_t* status;
};

// Offsets outside the tensors are cut to them.
__device__ __forceinline__ Seq seq_of(const Params& p, int b) {
    Seq s;
    s.q_start = min(max(p.qo_indptr[b], 0), p.total_q);
    s.q_len = min(max(p.qo_indptr[b + 1], s.q_start), p.total_q) - s.q_start;
    s.kv_start = min(max(p.kv_indptr[b], 0), p.total_kv);
    s.kv_room = min(max(p.kv_indptr[b + 1], s.kv_start), p.total_kv) - s.kv_start;
    s.kv_len = p.kv_lens != nullptr ? min(max(p.kv_lens[b], 0), s.kv_room) : s.kv_room;
    return s;
}
// The last key that position `pos` sees (-1 or less: none).
__device__ __forceinline__ int limit_of(const Params& p, const Seq& s, int pos) {
    return p.causal ? min(s.kv_len - 1, pos + s.kv_len - s.q_len) : s.kv_len - 1;
}

// --------------------------------------------------------------------- prepare

constexpr int kPrepThreads = 512;
constexpr int kMaxSeqs = 2048;

// The blocks of one side of all sequences, sequences in `order`; `flip`: each
// sequence's last block first.
__device__ void list_blocks(const int* order, const int* len, int B, int per, bool flip, int* before, int* warp_sum,
                            Block* out, int cap, int* count, const Params& p) {
    // blocks before each place of the order
    const int each = (B + kPrepThreads - 1) / kPrepThreads;
    const int i0 = min(static_cast<int>(threadIdx.x) * each, B), i1 = min(i0 + each, B);
    int sum = 0;
    for (int i = i0; i < i1; ++i) sum += (len[order[i]] + per - 1) / per;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;   // (below 2^31: 2^23 blocks a sequence at most, 128 sequences)
    __syncthreads();
    int base = incl - sum;
    for (int w = 0; w < warp; ++w) base = add_capped(base, warp_sum[w]);
    for (int i = i0; i < i1; ++i) {
        before[i] = base;
        base = add_capped(base, (len[order[i]] + per - 1) / per);
    }
    if (threadIdx.x == kPrepThreads - 1) before[B] = base;
    __syncthreads();
    const int total = min(before[B], cap);   // (offsets that overlap could name more)
    for (int x = threadIdx.x; x < total; x += kPrepThreads) {
        int lo = 0, hi = B;   // last place with before <= x
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before[mid] <= x) lo = mid; else hi = mid;
        }
        const int k = x - before[lo], n = (len[order[lo]] + per - 1) / per;
        out[x] = Block{seq_of(p, order[lo]), flip ? n - 1 - k : k, {0, 0}};
    }
    if (threadIdx.x == 0) *count = total;
    __syncthreads();
}

// CTA 0 lists the blocks; the others compute delta, D / 8 lanes a row.
template <int kD>
__global__ void __launch_bounds__(kPrepThreads) varlen_bwd_prepare_kernel(const __grid_constant__ Params p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0) {
        __shared__ int q_len[kMaxSeqs], kv_len[kMaxSeqs], order[kMaxSeqs], before[kMaxSeqs + 1], warp_sum[kPrepThreads / 32];
        for (int b = threadIdx.x; b < p.B; b += kPrepThreads) {
            const Seq s = seq_of(p, b);
            q_len[b] = s.q_len;
            kv_len[b] = s.kv_room;
        }
        __syncthreads();
        // keys' blocks cost their queries; with equal ones the lower sequence is first
        for (int side = 0; side < 2; ++side) {
            const int* cost = side == 0 ? q_len : kv_len;
            for (int b = threadIdx.x; b < p.B; b += kPrepThreads) {
                int rank = 0;
                for (int i = 0; i < p.B; ++i) rank += cost[i] > cost[b] || (cost[i] == cost[b] && i < b);
                order[rank] = b;
            }
            __syncthreads();
            if (side == 0)
                list_blocks(order, kv_len, p.B, kBM, false, before, warp_sum, p.kv_blocks, p.max_kv_blocks,
                            p.counts, p);
            else
                list_blocks(order, q_len, p.B, p.P, true, before, warp_sum, p.q_blocks, p.max_q_blocks,
                            p.counts + 1, p);
        }
        return;
    }
    constexpr int kLanes = kD / 8;
    const int l = threadIdx.x % kLanes;
    const long long rows = static_cast<long long>(p.total_q) * p.Hq;
    const long long row = static_cast<long long>(blockIdx.x - 1) * (kPrepThreads / kLanes) + threadIdx.x / kLanes;
    const bool live = row < rows;
    const long long token = live ? row / p.Hq : 0;
    const int head = live ? static_cast<int>(row - token * p.Hq) : 0;
    uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
    if (live) {
        a = *reinterpret_cast<const uint4*>(p.o + token * p.o_stride + head * kD + 8 * l);
        b = *reinterpret_cast<const uint4*>(p.d_o + token * p.do_stride + head * kD + 8 * l);
    }
    const uint32_t ua[4] = {a.x, a.y, a.z, a.w}, ub[4] = {b.x, b.y, b.z, b.w};
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sum = fmaf(__uint_as_float(ua[i] << 16), __uint_as_float(ub[i] << 16), sum);
        sum = fmaf(__uint_as_float(ua[i] & 0xFFFF0000u), __uint_as_float(ub[i] & 0xFFFF0000u), sum);
    }
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (live && l == 0) {
        const float lse = p.lse[row];
        // a row that saw nothing (LSE = -inf) has P = 0
        p.stats[row] = lse == -INFINITY ? make_float2(-INFINITY, 0.f)
                                        : make_float2(-lse * kLog2e, (p.d_lse != nullptr ? p.d_lse[row] : 0.f) - sum);
    }
}

// ---------------------------------------------------------------- the two passes

// kDq: the pass over keys for dQ; else the pass over queries for dK and dV.
// r1, r2: the resident tiles K, V (or Q, dO); y1, y2: the streamed ones Q, dO (or K, V).
template <bool kDq, bool kD64>
__global__ void __launch_bounds__(kThreads, 1)
    varlen_bwd_kernel(const __grid_constant__ CUtensorMap r1_map, const __grid_constant__ CUtensorMap r2_map,
                      const __grid_constant__ CUtensorMap y1_map, const __grid_constant__ CUtensorMap y2_map,
                      const __grid_constant__ Params p) {
    constexpr int kD = kD64 ? 64 : 128, kHalves = kD / 64;
    // dQ: two buffers of S, so that the next S goes ahead of this tile's sum; or (early) two of
    // dP, so that both go ahead and the score warps have a step's time for dS.  With D = 64
    // their work is what a step takes: 8 causal documents of 16 heads 533 to 560 us by device,
    // otherwise 552 to 572; with D = 128 the MMAs': 4 x 2048 queries to 4096 keys 1147, 1140.
    constexpr bool kEarly = kDq && kD64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw - kSystem;   // shared address 0
    Control& sh = *reinterpret_cast<Control*>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // The list of blocks and the statistics come from the first kernel, for which
    // dK/dV's CTAs wait.  Once the last of them is in, dQ's take the SMs that fall
    // free: what they read is there then, so they wait for nothing but, in the
    // grid's last CTA, for dK/dV's end, so that this grid does not end before.
    if (!kDq || p.total_kv == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (kDq && blockIdx.x + 1 == gridDim.x) asm volatile("griddepcontrol.wait;" ::: "memory");
    const int pieces = kDq ? p.q_pieces : p.kv_pieces;
    const int per_block = p.Hkv * pieces;
    const int entry = blockIdx.x / per_block;
    // (the list has room for the entry, whether or not it is there)
    const int4* listed = reinterpret_cast<const int4*>((kDq ? p.q_blocks : p.kv_blocks) + entry);
    const int4 lo = __ldcg(listed), hi = __ldcg(listed + 1);
    if (entry >= __ldcg(p.counts + (kDq ? 1 : 0))) return;
    const int kvh = (blockIdx.x % per_block) / pieces, piece = blockIdx.x % pieces;
    const Seq sq{lo.x, lo.y, lo.z, lo.w, hi.x};
    const int own = hi.y;
    const int delta = sq.kv_len - sq.q_len;
    const int kv0_own = own * kBM;   // dK, dV: the first key
    const int p0_own = own * p.P;    // dQ: the first position
    // streamed tiles that this block meets, and this part of them
    int first = 0, last = 0;
    if constexpr (kDq) {
        last = max(0, limit_of(p, sq, min(p0_own + p.P, sq.q_len) - 1) + kBM) / kBM;
    } else if (kv0_own < sq.kv_len) {
        last = (sq.q_len + p.P - 1) / p.P;
        if (p.causal) first = min(max(0, kv0_own - delta) / p.P, last);
    }
    const int j0 = first + static_cast<int>(static_cast<long long>(last - first) * piece / pieces);
    const int j1 = first + static_cast<int>(static_cast<long long>(last - first) * (piece + 1) / pieces);
    const int n = j1 - j0;

    if (threadIdx.x == 0) {
        mbar_init(&sh.r_full, 1);
        for (int s = 0; s < kStages1; ++s) mbar_init(&sh.y1_full[s], 1);
        for (int s = 0; s < kStages2; ++s) mbar_init(&sh.y2_full[s], 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.s_full[s], 1);
            mbar_init(&sh.dp_full[s], 1);
        }
        mbar_init(&sh.p_ready, 8);
        mbar_init(&sh.ds_ready, 8);
        mbar_init(&sh.acc_full, 1);
        for (int s = 0; s < 2; ++s) mbar_init(&sh.sum_done[s], 1);
        for (int s = 0; s < kStatSlots; ++s) {
            mbar_init(&sh.stat_full[s], 1);
            mbar_init(&sh.stat_empty[s], 8);
        }
        sh.abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&sh.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    const int rows_used = p.P * p.G;   // rows of a tile of queries
    if (!kDq && rows_used < kBM) {
        // the rows behind them are never loaded: zeros, which add nothing
        constexpr int kVecs = kHalf / 16;
        const int first_vec = rows_used * 8, per_half = kVecs - first_vec;
        for (int i = threadIdx.x; i < (kStages1 + kStages2) * kHalves * per_half; i += kThreads) {
            const int h = i / per_half;   // halves of the stages, in the order of their places
            const int at = kOffY2 + (h / kHalves) * kTile + (h % kHalves) * kHalf + (first_vec + i % per_half) * 16;
            *reinterpret_cast<uint4*>(smem + at) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();   // generic-proxy writes -> the tensor core's reads
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;
    // both hold by construction (the host has asked how much the system keeps);
    // without them nothing is done
    const bool placed = sh.tmem_base == tmem && smem_u32(smem_raw) == kSystem;
    if (!placed) flag_status(p.status, ATTN_DEV_WAIT_TIMEOUT);
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (mbar_wait(bar, parity, &sh.abort)) return true;
        flag_status(p.status, ATTN_DEV_WAIT_TIMEOUT);
        atomicExch(&sh.abort, 1);
        return false;
    };

    if (!placed) {
    } else if (warp >= kScoreWarp) {
        regs_inc<kRegsSoftmax>();
        const int r = threadIdx.x & 127, h = (warp - kScoreWarp) >> 2;   // row of the tile, half of its columns
        const int i_score = threadIdx.x - 32 * kScoreWarp;
        const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float sl2 = p.scale_log2;
        const float2 scl2 = make_float2(sl2, sl2);
        // Scores come in the layout of an MMA's accumulators: element 4 i + 2 k + e of half
        // u is row 16 u + 8 k + lane / 4 of the warp's 32, column 8 i + 2 (lane mod 4) + e
        // of its 64.  A thread meets 16 columns and 4 rows, so that a column's statistics
        // (dK, dV) are read by 8 lanes at once and not by each of 32.
        const int row0 = 32 * (warp & 3) + (lane >> 2), col0 = 64 * h + 2 * (lane & 3);
        int lim_first = -1;
        float2 stat[4];   // dQ: the rows' statistics
        if constexpr (kDq) {
            lim_first = limit_of(p, sq, p0_own);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int rr = row0 + 8 * k, at = rr / p.G, pp = p0_own + at;
                stat[k] = make_float2(-INFINITY, 0.f);
                if (rr < rows_used && pp < sq.q_len)
                    stat[k] = __ldcg(p.stats + (static_cast<size_t>(sq.q_start) + pp) * p.Hq + kvh * p.G + (rr - at * p.G));
            }
        }
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            const int y = j0 + j, st = j % kStages1, slot = j % kStatSlots;
            const float2* nlse = reinterpret_cast<const float2*>(smem + kOffStat + slot * 2 * kBM * 4) + (col0 >> 1);
            const float2* dlt = nlse + kBM / 2;
            bool masked = false;
            const uint32_t s_addr = tmem + lane_addr + ((kDq && !kEarly && (j & 1)) ? kColAcc1 : kColS) + 64 * h;
            const uint32_t dp_addr = tmem + lane_addr + ((kEarly && (j & 1)) ? kColAcc1 : kColDP) + 64 * h;
            // the statistics are there before the scores
            float2 nl[kDq ? 1 : 8];
            if constexpr (!kDq) {
                if (!(ok = wait(&sh.stat_full[slot], (j / kStatSlots) & 1))) break;
#pragma unroll
                for (int i = 0; i < 8; ++i) nl[i] = nlse[4 * i];
            }
            if (!(ok = wait(&sh.s_full[j & 1], (j >> 1) & 1))) break;
            tc_fence_after();
            uint32_t sr[2][32];
            tmem_ld_16x64(s_addr, sr[0]);
            tmem_ld_16x64(s_addr + (16u << 16), sr[1]);
            int there;   // rows (dQ: keys) of the streamed tile that are there
            if constexpr (kDq) {
                masked = y * kBM + kBM - 1 > lim_first;
                there = sq.kv_len - y * kBM;
                if (there < kBM) {
                    // dS is 0 there, but 0 times whatever lies behind the keys is not
                    for (int i = there * 8 + i_score; i < kHalf / 16; i += kScoreThreads) {
                        uint4* rows = reinterpret_cast<uint4*>(smem + kOffY1 + st * kTile);
                        rows[i] = make_uint4(0u, 0u, 0u, 0u);
                        if (!kD64) rows[kHalf / 16 + i] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
            } else {
                there = min(p.P, sq.q_len - y * p.P) * p.G;
                masked = there < rows_used || (p.causal && y * p.P + delta < kv0_own + kBM - 1);
                if (there < rows_used) {
                    if (!(ok = wait(&sh.y2_full[j % kStages2], (j / kStages2) & 1))) break;
                    for (int i = there * 8 + i_score; i < kHalf / 16; i += kScoreThreads) {
                        uint4* rows = reinterpret_cast<uint4*>(smem + kOffY1 + st * kTile);
                        uint4* rows2 = reinterpret_cast<uint4*>(smem + kOffY2 + (j % kStages2) * kTile);
                        rows[i] = rows2[i] = make_uint4(0u, 0u, 0u, 0u);
                        if (!kD64) rows[kHalf / 16 + i] = rows2[kHalf / 16 + i] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
            }
            // columns [lo, hi) of the tile count in row k of the thread
            auto range = [&](int k, int& lo, int& hi) {
                lo = 0;
                if constexpr (kDq) {
                    hi = limit_of(p, sq, p0_own + (row0 + 8 * k) / p.G) - y * kBM + 1;
                } else {
                    hi = there;
                    if (p.causal) {
                        const long long from = static_cast<long long>(kv0_own + row0 + 8 * k - delta - y * p.P) * p.G;
                        lo = static_cast<int>(min(max(from, 0LL), 128LL));
                    }
                }
            };
            float2 pr[2][16];
            tmem_ld_wait();
            if constexpr (kEarly) {   // the next tile's S may come
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_ready);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 16; ++e) {   // e = 2 i + k
                    const float2 l = kDq ? make_float2(stat[2 * u + (e & 1)].x, stat[2 * u + (e & 1)].x) : nl[kDq ? 0 : e >> 1];
                    const float2 x = __ffma2_rn(make_float2(__uint_as_float(sr[u][2 * e]), __uint_as_float(sr[u][2 * e + 1])), scl2, l);
                    pr[u][e] = make_float2(ex2(x.x), ex2(x.y));
                }
            if (masked) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    int lo, hi;
                    range(k, lo, hi);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int c = col0 + 8 * i;
                        float2& x = pr[k >> 1][2 * i + (k & 1)];
                        if (c < lo || c >= hi) x.x = 0.f;
                        if (c + 1 < lo || c + 1 >= hi) x.y = 0.f;
                    }
                }
            }
            uint32_t pk[2][16];
            if constexpr (!kDq) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 16; ++e) pk[u][e] = pack_bf16x2(pr[u][e].x, pr[u][e].y);
                tmem_st_16x32(s_addr, pk[0]);
                tmem_st_16x32(s_addr + (16u << 16), pk[1]);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_ready);
#pragma unroll
                for (int i = 0; i < 8; ++i) nl[i] = dlt[4 * i];
            }
            if (!(ok = wait(&sh.dp_full[j & 1], (j >> 1) & 1))) break;
            tc_fence_after();
            uint32_t dr[2][32];
            tmem_ld_16x64(dp_addr, dr[0]);
            tmem_ld_16x64(dp_addr + (16u << 16), dr[1]);
            tmem_ld_wait();
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 l = kDq ? make_float2(stat[2 * u + (e & 1)].y, stat[2 * u + (e & 1)].y) : nl[kDq ? 0 : e >> 1];
                    pr[u][e] = __fmul2_rn(__fadd2_rn(make_float2(__uint_as_float(dr[u][2 * e]), __uint_as_float(dr[u][2 * e + 1])), l), pr[u][e]);
                }
            if (masked) {   // again: what is not there may have a dP that is not finite
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    int lo, hi;
                    range(k, lo, hi);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int c = col0 + 8 * i;
                        float2& x = pr[k >> 1][2 * i + (k & 1)];
                        if (c < lo || c >= hi) x.x = 0.f;
                        if (c + 1 < lo || c + 1 >= hi) x.y = 0.f;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 16; ++e) pk[u][e] = pack_bf16x2(pr[u][e].x, pr[u][e].y);
            tmem_st_16x32(dp_addr, pk[0]);
            tmem_st_16x32(dp_addr + (16u << 16), pk[1]);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.ds_ready);
                if (!kDq) mbar_arrive(&sh.stat_empty[slot]);
            }
        }
        // -------------------------------------------------------------- epilogue
        if (ok && n > 0) ok = wait(&sh.acc_full, 0);
        if (ok) {
            tc_fence_after();
            // dQ: both halves of the threads share a row's columns; else the first four warps have dV, the others dK
            constexpr int kCols = kDq ? kD / 2 : kD;
            const uint32_t acc = tmem + lane_addr + (kDq ? kColAcc2 + kCols * h : (h == 0 ? kColAcc1 : kColAcc2));
            const int pos = p0_own + r / p.G, key = kv0_own + r;   // this thread's row now
            const bool row_real = r < rows_used && pos < sq.q_len;
            const bool store = kDq ? row_real : key < sq.kv_room;
            const bool real = n > 0 && (kDq || key < sq.kv_len);
            const float f = (kDq || h == 1) ? p.scale : 1.f;
            const size_t row = kDq ? static_cast<size_t>(sq.q_start) + pos : static_cast<size_t>(sq.kv_start) + key;
            const int head = kDq ? kvh * p.G + r % p.G : kvh;
            const int heads = kDq ? p.Hq : p.Hkv, rows = kDq ? p.total_q : p.total_kv;
            const int out0 = kDq ? kCols * h : 0;   // its first column
            __nv_bfloat16* out = kDq ? p.dq : (h == 0 ? p.dv : p.dk);
            const long long stride = kDq ? p.dq_stride : (h == 0 ? p.dv_stride : p.dk_stride);
            float* part = kDq ? p.dq_part : (h == 0 ? p.dv_part : p.dk_part);
            // bf16 rows leave through shared memory (the stages are done with), whole
            // rows side by side: 32 rows a warp, 16 bytes apart from a power of two
            constexpr int kPitch = kCols * 2 + 16, kLanes = kCols / 8;
            uint8_t* rows_sh = smem + kOffY2 + (warp - kScoreWarp) * 32 * kPitch;
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c) {
                uint32_t ar[32];
                tmem_ld32(acc + 32 * c, ar);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) ar[e] = real ? __float_as_uint(__uint_as_float(ar[e]) * f) : 0u;
                if (pieces > 1) {
                    if (!store) continue;
                    float4* dst = reinterpret_cast<float4*>(
                        part + ((static_cast<size_t>(piece) * rows + row) * heads + head) * kD + out0 + 32 * c);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[e] = make_float4(__uint_as_float(ar[4 * e]), __uint_as_float(ar[4 * e + 1]),
                                             __uint_as_float(ar[4 * e + 2]), __uint_as_float(ar[4 * e + 3]));
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(rows_sh + lane * kPitch + 64 * c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint4 v;
                        v.x = pack_bf16x2(__uint_as_float(ar[8 * e]), __uint_as_float(ar[8 * e + 1]));
                        v.y = pack_bf16x2(__uint_as_float(ar[8 * e + 2]), __uint_as_float(ar[8 * e + 3]));
                        v.z = pack_bf16x2(__uint_as_float(ar[8 * e + 4]), __uint_as_float(ar[8 * e + 5]));
                        v.w = pack_bf16x2(__uint_as_float(ar[8 * e + 6]), __uint_as_float(ar[8 * e + 7]));
                        dst[e] = v;
                    }
                }
            }
            if (pieces == 1) {
                const long long at = store ? static_cast<long long>(row) * stride + head * kD + out0 : -1;
                __syncwarp();
#pragma unroll
                for (int r0 = 0; r0 < 32; r0 += 32 / kLanes) {
                    const int rr = r0 + lane / kLanes, c = lane % kLanes;
                    const long long to = __shfl_sync(0xffffffffu, at, rr);
                    const uint4 v = *reinterpret_cast<const uint4*>(rows_sh + rr * kPitch + 16 * c);
                    if (to >= 0) *reinterpret_cast<uint4*>(out + to + 8 * c) = v;
                }
            }
        }
    } else {
        regs_dec<kRegsControl>();
        if (warp == kProducerWarp && n > 0) {
            if (lane == 0) {
                const uint32_t q_bytes = static_cast<uint32_t>(rows_used) * 128 * kHalves;
                constexpr uint32_t kKvBytes = kHalves * kHalf;
                auto load_q = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int tile) {
#pragma unroll
                    for (int hh = 0; hh < kHalves; ++hh)
                        tma_load_3d(dst + hh * kHalf, map, bar, 64 * hh, kvh * p.G, sq.q_start + tile * p.P);
                };
                auto load_kv = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int tile) {
#pragma unroll
                    for (int hh = 0; hh < kHalves; ++hh)
                        tma_load_2d(dst + hh * kHalf, map, bar, kvh * kD + 64 * hh, sq.kv_start + tile * kBM);
                };
                auto load = [&](bool queries, uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int tile) {
                    if (queries) load_q(dst, map, bar, tile);
                    else load_kv(dst, map, bar, tile);
                };
                mbar_arrive_expect_tx(&sh.r_full, 2 * (kDq ? q_bytes : kKvBytes));
                load(kDq, smem + kOffR1, &r1_map, &sh.r_full, own);
                load(kDq, smem + kOffR2, &r2_map, &sh.r_full, own);
                const uint32_t bytes = kDq ? kKvBytes : q_bytes;
                auto load1 = [&](int j) {
                    const int s = j % kStages1;
                    mbar_arrive_expect_tx(&sh.y1_full[s], bytes);
                    load(!kDq, smem + kOffY1 + s * kTile, &y1_map, &sh.y1_full[s], j0 + j);
                };
                auto load2 = [&](int j) {
                    const int s = j % kStages2;
                    mbar_arrive_expect_tx(&sh.y2_full[s], bytes);
                    load(!kDq, smem + kOffY2 + s * kTile, &y2_map, &sh.y2_full[s], j0 + j);
                };
                // (a barrier waited for here cannot run a round ahead: its next
                // phase is of a tile that is loaded only afterwards)
                for (int j = 0; j < n; ++j) {
                    if (kEarly && j >= 3 && !wait(&sh.sum_done[(j - 3) & 1], ((j - 3) >> 1) & 1)) break;   // dQ of tile j - 3
                    if (!kEarly && j >= 2 && !wait(&sh.dp_full[j & 1], ((j - 2) >> 1) & 1)) break;   // dP of tile j - 2
                    load1(j);
                    if (kEarly && j >= 2 && !wait(&sh.dp_full[j & 1], ((j - 2) >> 1) & 1)) break;
                    if (!kDq && j >= 2 && !wait(&sh.s_full[(j - 1) & 1], ((j - 1) >> 1) & 1)) break;   // S of tile j - 1
                    load2(j);
                }
            }
        } else if (warp == kStatWarp && !kDq) {
            bool ok = true;
            for (int j = 0; j < n; ++j) {
                const int slot = j % kStatSlots;
                const int p0 = (j0 + j) * p.P, there = min(p.P, sq.q_len - p0) * p.G;
                float2 v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = lane + 32 * e, at = c / p.G;
                    v[e] = make_float2(-INFINITY, 0.f);
                    if (c < there)
                        v[e] = __ldcg(p.stats + (static_cast<size_t>(sq.q_start) + p0 + at) * p.Hq + kvh * p.G + (c - at * p.G));
                }
                if (j >= kStatSlots) ok = wait(&sh.stat_empty[slot], ((j / kStatSlots) - 1) & 1);
                if (!__all_sync(0xffffffffu, ok)) break;
                float* dst = reinterpret_cast<float*>(smem + kOffStat) + slot * 2 * kBM;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dst[lane + 32 * e] = v[e].x;
                    dst[kBM + lane + 32 * e] = v[e].y;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.stat_full[slot]);
            }
        } else if (warp == kMmaWarp && n > 0) {
            const uint32_t lead = elect_one();
            {
                constexpr uint32_t idesc_s = idesc_bf16_f32(kBM, kBM, false);
                constexpr uint32_t idesc_acc = idesc_bf16_f32(kBM, kD, true);
                auto desc = [](int off, int lbo) constexpr -> uint32_t { return (off >> 4) | ((lbo >> 4) << 16); };
                auto scores = [&](uint32_t d, int a_off, int b_off) {   // D = A B^T over the head dimension
                    umma_ss_by<0>(lead, d, desc(a_off, 16), desc(b_off, 16), idesc_s);
#pragma unroll
                    for (int kk = 1; kk < kD / 16; ++kk) {
                        const int off = (kk >> 2) * kHalf + (kk & 3) * 32;
                        umma_ss_by<1>(lead, d, desc(a_off + off, 16), desc(b_off + off, 16), idesc_s);
                    }
                };
                // D (+)= A B over the 128 streamed rows; A in TMEM, two halves of 64 columns packed
                // to 32; `next`, what the product after it waits for, comes in the middle, where
                // the tensor core has MMAs to go on with
                auto gather = [&](uint32_t d, uint32_t a, int b_off, bool acc, auto next) -> bool {
                    umma_ts_by(lead, d, a, desc(b_off, kHalf), idesc_acc, acc ? 1u : 0u);
                    bool good = true;
#pragma unroll
                    for (int kk = 1; kk < kBM / 16; ++kk) {
                        if (kk == 5) good = next();
                        umma_ts_by(lead, d, a + (kk >> 2) * 64 + (kk & 3) * 8, desc(b_off + kk * 16 * 128, kHalf), idesc_acc, 1u);
                    }
                    return good;
                };
                // One tile's step, even or odd.  False: a wait ran out.  (The three stages of y1
                // are not unrolled: six copies of the step were 9 % slower.)
                int s1 = 0, n1 = 1;   // this tile's stage of y1, the next one's
                auto step = [&](int j, auto odd) -> bool {
                    constexpr int kOdd = decltype(odd)::value, n2 = !kOdd;
                    static_assert(kStages2 == 2, "even and odd tiles");
                    const int k = j + 1;
                    const bool more = k < n;
                    auto next1 = [&] { return !more || wait(&sh.y1_full[n1], (k / kStages1) & 1); };
                    auto next2 = [&] { return !more || wait(&sh.y2_full[n2], (k / kStages2) & 1); };
                    if constexpr (kEarly) {
                        if (more) {
                            if (!next1() || !wait(&sh.p_ready, j & 1)) return false;
                            tc_fence_after();
                            scores(tmem + kColS, kOffR1, kOffY1 + n1 * kTile);
                            umma_commit_by(lead, &sh.s_full[!kOdd]);
                            if (!next2()) return false;
                            tc_fence_after();
                            scores(tmem + (kOdd ? kColDP : kColAcc1), kOffR2, kOffY2 + n2 * kTile);
                            umma_commit_by(lead, &sh.dp_full[!kOdd]);
                        }
                        if (!wait(&sh.ds_ready, j & 1)) return false;
                        tc_fence_after();
                        if (!gather(tmem + kColAcc2, tmem + (kOdd ? kColAcc1 : kColDP), kOffY1 + s1 * kTile, j > 0, [] { return true; }))
                            return false;   // dQ += dS K
                        if (more) umma_commit_by(lead, &sh.sum_done[kOdd]);
                        s1 = n1;
                        n1 = n1 + 1 == kStages1 ? 0 : n1 + 1;
                        return true;
                    }
                    if constexpr (!kDq) {
                        if (!wait(&sh.p_ready, j & 1)) return false;
                        tc_fence_after();
                        if (!gather(tmem + kColAcc1, tmem + kColS, kOffY2 + kOdd * kTile, j > 0, next1)) return false;   // dV += P^T dO
                    } else if (!next1()) {
                        return false;
                    }
                    if (more) {   // (for dK, dV it overwrites P, which the product before it has read)
                        tc_fence_after();
                        scores(tmem + ((kDq && !kOdd) ? kColAcc1 : kColS), kOffR1, kOffY1 + n1 * kTile);
                        umma_commit_by(lead, &sh.s_full[!kOdd]);
                    }
                    if (!wait(&sh.ds_ready, j & 1)) return false;
                    tc_fence_after();
                    if (!gather(tmem + kColAcc2, tmem + kColDP, kOffY1 + s1 * kTile, j > 0, next2)) return false;   // dK += dS^T Q, or dQ += dS K
                    if (more) {   // overwrites dS
                        tc_fence_after();
                        scores(tmem + kColDP, kOffR2, kOffY2 + n2 * kTile);
                        umma_commit_by(lead, &sh.dp_full[!kOdd]);
                    }
                    s1 = n1;
                    n1 = n1 + 1 == kStages1 ? 0 : n1 + 1;
                    return true;
                };
                auto run = [&]() {
                    if (!wait(&sh.r_full, 0) || !wait(&sh.y1_full[0], 0)) return;
                    tc_fence_after();
                    scores(tmem + kColS, kOffR1, kOffY1);
                    umma_commit_by(lead, &sh.s_full[0]);
                    if (!wait(&sh.y2_full[0], 0)) return;
                    tc_fence_after();
                    scores(tmem + kColDP, kOffR2, kOffY2);
                    umma_commit_by(lead, &sh.dp_full[0]);
                    for (int j = 0; j < n;) {
                        bool good = step(j++, std::integral_constant<int, 0>{});
                        if (good && j < n) good = step(j++, std::integral_constant<int, 1>{});
                        if (!good) return;
                    }
                    umma_commit_by(lead, &sh.acc_full);
                };
                run();
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(sh.tmem_base, kTmemCols);
    }
}

// The parts of gradients added up, in order: [pieces][rows][row_elems] fp32 to bf16
// rows `stride` apart, of the rows that belong to a sequence; blockIdx.y is the gradient.
struct Sum {
    const float* part[2];
    __nv_bfloat16* out[2];
    long long stride[2];
    const int32_t* indptr;
    int pieces, rows, row_elems, B;
};
__global__ void __launch_bounds__(256) varlen_bwd_sum_kernel(const __grid_constant__ Sum a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int vecs = a.row_elems / 4;
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const long long row = i / vecs;
    if (row >= a.rows || row < a.indptr[0] || row >= a.indptr[a.B]) return;
    const float4* src = reinterpret_cast<const float4*>(blockIdx.y ? a.part[1] : a.part[0]) + i;
    float4 sum = __ldcg(src);
    for (int s = 1; s < a.pieces; ++s) {
        const float4 v = __ldcg(src + static_cast<long long>(s) * a.rows * vecs);
        sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
    }
    *reinterpret_cast<uint2*>((blockIdx.y ? a.out[1] : a.out[0]) + row * (blockIdx.y ? a.stride[1] : a.stride[0]) + (i - row * vecs) * 4) =
        make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
}

// ------------------------------------------------------------------- host side

// Parts of each block's streamed tiles, for the keys' and the queries' blocks:
// the host knows the totals, not the lengths.  With fewer blocks than half the
// SMs, as many parts as fill them, each of at least kPartTiles tiles of the mean
// sequence.  2048 queries of 16 heads to 100 keys 35 us, whole 175; 77 to 8192 keys
// 73 and 117.  Parts of two tiles in place of four: 5 sequences of up to 300
// queries 26.2 us against 23.9, 77 queries to 1500 keys 32.4 against 33.9.
constexpr int kMaxPieces = 16;
constexpr int kPartTiles = 4;
struct Plan {
    int kv_pieces, q_pieces;
    long long kv_blocks, q_blocks;   // most that there can be
};
Plan plan_of(int B, int total_q, int total_kv, int Hq, int Hkv, int sms) {
    const int P = kBM / (Hq / Hkv);
    Plan x;
    x.kv_blocks = total_kv / kBM + static_cast<long long>(B);
    x.q_blocks = total_q / P + static_cast<long long>(B);
    const long long kv_likely = std::max<long long>(B, (static_cast<long long>(total_kv) + kBM - 1) / kBM);
    const long long q_likely = std::max<long long>(B, (static_cast<long long>(total_q) + P - 1) / P);
    const long long q_tiles = std::max(1LL, q_likely / B), kv_tiles = std::max(1LL, kv_likely / B);
    auto pieces = [&](long long blocks, long long tiles) {
        return static_cast<int>(std::max<long long>(1, std::min<long long>({sms / (blocks * Hkv), tiles / kPartTiles, kMaxPieces})));
    };
    x.kv_pieces = pieces(kv_likely, q_tiles);
    x.q_pieces = pieces(q_likely, kv_tiles);
    return x;
}

size_t round16(size_t x) { return (x + 15) & ~static_cast<size_t>(15); }

struct Layout {
    size_t stats, counts, kv_blocks, q_blocks, dq, dk, dv, bytes;
};
Layout layout_of(const Plan& x, int total_q, int total_kv, int Hq, int Hkv, int D) {
    Layout l;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t from = at;
        at += round16(bytes);
        return from;
    };
    l.stats = take(static_cast<size_t>(total_q) * Hq * sizeof(float2));
    l.counts = take(2 * sizeof(int));
    l.kv_blocks = take(static_cast<size_t>(x.kv_blocks) * sizeof(Block));
    l.q_blocks = take(static_cast<size_t>(x.q_blocks) * sizeof(Block));
    const size_t q_part = static_cast<size_t>(total_q) * Hq * D * sizeof(float), kv_part = static_cast<size_t>(total_kv) * Hkv * D * sizeof(float);
    l.dq = take(x.q_pieces > 1 ? q_part * x.q_pieces : 0);
    l.dk = take(x.kv_pieces > 1 ? kv_part * x.kv_pieces : 0);
    l.dv = take(x.kv_pieces > 1 ? kv_part * x.kv_pieces : 0);
    l.bytes = at;
    return l;
}

// A launch whose CTAs may come in before the kernel before it has ended.
template <typename... Args>
cudaError_t launch_along(void (*kern)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                         const typename std::common_type<Args>::type&... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <bool kD64>
cudaError_t launch(const VarlenBwdArgs& a, const Params& p, const Plan& x, int sms, const CUtensorMap& q, const CUtensorMap& d_o,
                   const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
    constexpr int kD = kD64 ? 64 : 128;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = once_per_device(done, [] {
        // the addresses of shared memory are constants behind what the system keeps of it
        int dev = 0, kept = 0;
        cudaError_t r = cudaGetDevice(&dev);
        if (r == cudaSuccess) r = cudaDeviceGetAttribute(&kept, cudaDevAttrReservedSharedMemoryPerBlock, dev);
        if (r != cudaSuccess) return r;
        if (kept != kSystem) return cudaErrorNotSupported;
        r = cudaFuncSetAttribute(varlen_bwd_kernel<false, kD64>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        return r != cudaSuccess ? r
                                : cudaFuncSetAttribute(varlen_bwd_kernel<true, kD64>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    });
    if (e != cudaSuccess) return e;
    const long long rows = static_cast<long long>(a.total_q) * a.Hq;
    const long long per_cta = kPrepThreads / (kD / 8);
    const long long prepare_ctas = 1 + (rows + per_cta - 1) / per_cta;
    varlen_bwd_prepare_kernel<kD><<<static_cast<unsigned>(prepare_ctas), kPrepThreads, 0, stream>>>(p);
    e = cudaGetLastError();
    if (e == cudaSuccess && a.total_kv > 0) {
        // along only behind a first kernel of a CTA or two an SM: 5 sequences of up to 300
        // queries 33 -> 26 us, but coming in among many CTAs of it, causal batches take up
        // to a quarter longer (4 of 1000 tokens 130 -> 157)
        const long long grid = x.kv_blocks * a.Hkv * x.kv_pieces;
        if (grid <= sms && prepare_ctas <= 2LL * sms) {
            e = launch_along(varlen_bwd_kernel<false, kD64>, dim3(static_cast<unsigned>(grid)), kThreads, kSmemBytes, stream, k, v, q, d_o, p);
        } else {
            varlen_bwd_kernel<false, kD64><<<static_cast<unsigned>(grid), kThreads, kSmemBytes, stream>>>(k, v, q, d_o, p);
            e = cudaGetLastError();
        }
    }
    if (e == cudaSuccess && a.total_q > 0)
        e = launch_along(varlen_bwd_kernel<true, kD64>, dim3(static_cast<unsigned>(x.q_blocks * a.Hkv * x.q_pieces)), kThreads,
                         kSmemBytes, stream, q, d_o, k, v, p);
    auto sum = [&](const Sum& t, int gradients) {
        const long long vecs = static_cast<long long>(t.rows) * (t.row_elems / 4);
        return launch_along(varlen_bwd_sum_kernel, dim3(static_cast<unsigned>((vecs + 255) / 256), gradients), 256, 0, stream, t);
    };
    if (e == cudaSuccess && x.kv_pieces > 1 && a.total_kv > 0)
        e = sum(Sum{{p.dk_part, p.dv_part}, {p.dk, p.dv}, {p.dk_stride, p.dv_stride}, a.kv_indptr, x.kv_pieces, a.total_kv, a.Hkv * kD, a.B}, 2);
    if (e == cudaSuccess && x.q_pieces > 1 && a.total_q > 0)
        e = sum(Sum{{p.dq_part, nullptr}, {p.dq, nullptr}, {p.dq_stride, 0}, a.qo_indptr, x.q_pieces, a.total_q, a.Hq * kD, a.B}, 1);
    return e;
}

}  // namespace

size_t varlen_bwd_workspace(int B, int total_q, int total_kv, int Hq, int Hkv, int D, int sms) {
    return layout_of(plan_of(B, total_q, total_kv, Hq, Hkv, sms), total_q, total_kv, Hq, Hkv, D).bytes;
}

// Whether the grids of both passes count in int.
bool varlen_bwd_grid_ok(int B, int total_q, int total_kv, int Hq, int Hkv, int sms) {
    const Plan x = plan_of(B, total_q, total_kv, Hq, Hkv, sms);
    return x.kv_blocks * Hkv * x.kv_pieces < (1LL << 31) && x.q_blocks * Hkv * x.q_pieces < (1LL << 31);
}

cudaError_t launch_varlen_bwd(const VarlenBwdArgs& a, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const Plan x = plan_of(a.B, a.total_q, a.total_kv, a.Hq, a.Hkv, sms);
    const Layout l = layout_of(x, a.total_q, a.total_kv, a.Hq, a.Hkv, a.D);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    Params p{};
    p.o = static_cast<const __nv_bfloat16*>(a.o);
    p.d_o = static_cast<const __nv_bfloat16*>(a.d_o);
    p.o_stride = a.o_stride;
    p.do_stride = a.do_stride;
    p.lse = a.lse;
    p.d_lse = a.d_lse;
    p.qo_indptr = a.qo_indptr;
    p.kv_indptr = a.kv_indptr;
    p.kv_lens = a.kv_lens;
    p.causal = a.causal;
    p.B = a.B;
    p.total_q = a.total_q;
    p.total_kv = a.total_kv;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.P = kBM / p.G;
    p.scale = a.scale;
    p.scale_log2 = a.scale * kLog2e;
    p.stats = reinterpret_cast<float2*>(ws + l.stats);
    p.counts = reinterpret_cast<int*>(ws + l.counts);
    p.kv_blocks = reinterpret_cast<Block*>(ws + l.kv_blocks);
    p.q_blocks = reinterpret_cast<Block*>(ws + l.q_blocks);
    p.max_kv_blocks = static_cast<int>(x.kv_blocks);
    p.max_q_blocks = static_cast<int>(x.q_blocks);
    p.kv_pieces = x.kv_pieces;
    p.q_pieces = x.q_pieces;
    p.dq = static_cast<__nv_bfloat16*>(a.d_q);
    p.dk = static_cast<__nv_bfloat16*>(a.d_k);
    p.dv = static_cast<__nv_bfloat16*>(a.d_v);
    p.dq_stride = a.dq_stride;
    p.dk_stride = a.dk_stride;
    p.dv_stride = a.dv_stride;
    p.dq_part = reinterpret_cast<float*>(ws + l.dq);
    p.dk_part = reinterpret_cast<float*>(ws + l.dk);
    p.dv_part = reinterpret_cast<float*>(ws + l.dv);
    p.status = a.dev_status;
    const uint64_t D = static_cast<uint64_t>(a.D);
    CUtensorMap q, d_o, k, v;
    auto q_map = [&](CUtensorMap* m, const void* base, long long stride) {
        const uint64_t dims[3] = {D, static_cast<uint64_t>(a.Hq), static_cast<uint64_t>(a.total_q)};
        const uint64_t strides[2] = {D * 2, static_cast<uint64_t>(stride) * 2};
        const uint32_t box[3] = {64, static_cast<uint32_t>(p.G), static_cast<uint32_t>(p.P)};
        return encode_tiled_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    auto kv_map = [&](CUtensorMap* m, const void* base, long long stride) {
        const uint64_t dims[2] = {static_cast<uint64_t>(a.Hkv) * D, static_cast<uint64_t>(a.total_kv)};
        const uint64_t strides[1] = {static_cast<uint64_t>(stride) * 2};
        const uint32_t box[2] = {64, kBM};
        return encode_tiled_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    // a side without rows has no tiles, and its maps are not used
    bool good = true;
    if (a.total_q > 0) good = q_map(&q, a.q, a.q_stride) && q_map(&d_o, a.d_o, a.do_stride);
    if (good && a.total_kv > 0) good = kv_map(&k, a.k, a.k_stride) && kv_map(&v, a.v, a.v_stride);
    if (!good) return cudaErrorInvalidValue;
    if (a.total_q == 0) q = d_o = k;
    if (a.total_kv == 0) k = v = q;
    return a.D == 64 ? launch<true>(a, p, x, sms, q, d_o, k, v, stream) : launch<false>(a, p, x, sms, q, d_o, k, v, stream);
}

}  // namespace gb300
