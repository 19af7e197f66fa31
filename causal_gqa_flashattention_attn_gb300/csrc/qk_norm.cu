// qk_norm.cu - RMS norm of every query and key head with the rotation by its
// token's position in the same pass, and its gradient.
//
// Mathematics, per head vector x of D elements with weight w and the rotation
// R_t of its token:
//   r = (mean x^2 + eps)^(-1/2),  n = r x,  y = R_t (w n).
// Backward, with u = R_t^T dy:
//   dw = sum over rows of u n,  g = w u,  dx = r (g - n mean(g n)).
// r is computed again from x, which the pass reads anyway; nothing is kept by
// the forward pass.  Everything is fp32 and rounded once.
//
// Layout: D / 8 lanes own a row, two runs of four elements each, placed so that
// both elements of every rotated pair lie in one lane: (4l, rot/2 + 4l) for
// pairs half a head apart, eight neighbours otherwise.  A lane's angles are
// 4l .. 4l+3 either way, one 16-byte load each for cosines and sines, used for
// all the rows of a token that the lane takes.
//
// The gradient of a weight is a sum over all rows of all tokens: a CTA takes rows
// of one side, each lane keeps its eight columns in registers over the rows it
// takes, the CTA joins its lanes in order, and a second kernel the CTAs, in order:
// the result does not depend on timing.
//
// Bound: the bytes of x (and dy) in and y (or dx) out.  16384 tokens of 32 + 4
// heads of 128 (303 MB) 53.6 us, 5.65 TB/s; the gradient of 32 + 8 heads (505 MB)
// 90.9 us, 5.55 TB/s, 0.83 and 0.82 of a copy's rate; one token 4.6 to 5.1 us,
// host included.  Two thirds of the issue slots are taken, and how well the compiler
// interleaves four rows decides: two elements at a time throughout (72 / 137 us), two
// chunks in turn without moves (72 / 118) and the rows' sums side by side (spills,
// 73 / 131) were slower than this order, 60.5 / 90.9 for 16384 tokens of 32 + 8 heads.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace gb300 {
namespace {

constexpr int kThreads = 256;
constexpr int kReduceCols = 32, kReduceSlices = 32;

struct Params {
    const __nv_bfloat16* x[2];    // q, k
    const __nv_bfloat16* dy[2];   // backward only
    __nv_bfloat16* out[2];
    long long x_stride[2], dy_stride[2], out_stride[2];
    const void* w[2];             // NULL: not normalised
    int heads[2];                 // 0: absent
    int units[2];                 // chunks of kPer rows
    Divisor chunks[2];            // chunks per token
    int q_ctas;                   // CTAs of the queries, which come first
    bool w_bf16;
    float eps;
    const float* cos_sin;
    int max_pos, rot;
    const int32_t* positions;     // NULL: the token's index
    float* dw_part;               // [grid][D]
    int32_t* status;
};

__device__ __forceinline__ void unpack4(uint2 u, float* f) {
    f[0] = __uint_as_float(u.x << 16);
    f[1] = __uint_as_float(u.x & 0xFFFF0000u);
    f[2] = __uint_as_float(u.y << 16);
    f[3] = __uint_as_float(u.y & 0xFFFF0000u);
}

// Elements [i0, i0 + 4) and [i1, i1 + 4) of a row.
struct Place {
    int i0, i1;
    bool turns;   // the lane's elements are rotated
};
template <bool kHalves>
__device__ __forceinline__ Place place_of(int l, int rot) {
    Place a{8 * l, 8 * l + 4, 8 * l < rot};
    if (kHalves && a.turns) a.i0 = 4 * l, a.i1 = rot / 2 + 4 * l;
    return a;
}

// Loads that stay where they are written, ahead of the work that they overlap (of
// plain ones the compiler moves those of read-only data down to their use).
__device__ __forceinline__ int load_ahead(const int32_t* p) {
    int v;
    asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ void load_ahead(const float* p, float (&v)[4]) {
    asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "l"(p));
}

// What a lane reads of a row: one 16-byte load where its elements are neighbours.
template <bool kHalves>
__device__ __forceinline__ void load8(const __nv_bfloat16* row, const Place& a, uint2 (&u)[2]) {
    if constexpr (kHalves) {
        u[0] = *reinterpret_cast<const uint2*>(row + a.i0);
        u[1] = *reinterpret_cast<const uint2*>(row + a.i1);
    } else {
        const uint4 v = *reinterpret_cast<const uint4*>(row + a.i0);
        u[0] = make_uint2(v.x, v.y);
        u[1] = make_uint2(v.z, v.w);
    }
}
template <bool kHalves>
__device__ __forceinline__ void store8(__nv_bfloat16* row, const Place& a, const float (&y)[8]) {
    const uint2 lo = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    const uint2 hi = make_uint2(pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    if constexpr (kHalves) {
        *reinterpret_cast<uint2*>(row + a.i0) = lo;
        *reinterpret_cast<uint2*>(row + a.i1) = hi;
    } else {
        *reinterpret_cast<uint4*>(row + a.i0) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
}

__device__ __forceinline__ void load_weight(const Params& p, int which, const Place& a, float (&w)[8]) {
    const void* base = which == 0 ? p.w[0] : p.w[1];
    if (base == nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.f;
    } else if (p.w_bf16) {
        unpack4(*reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(base) + a.i0), w);
        unpack4(*reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(base) + a.i1), w + 4);
    } else {
        const float4 lo = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + a.i0);
        const float4 hi = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + a.i1);
        w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w;
        w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
    }
}

// (a, b) -> (a c - b s, a s + b c) for the lane's four pairs; sign -1 turns back.
template <bool kHalves>
__device__ __forceinline__ void turn(float (&y)[8], const float (&c)[4], const float (&s)[4], float sign) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float& a = kHalves ? y[i] : y[2 * i];
        float& b = kHalves ? y[4 + i] : y[2 * i + 1];
        const float sn = sign * s[i], a0 = a, b0 = b;
        a = fmaf(a0, c[i], -b0 * sn);
        b = fmaf(a0, sn, b0 * c[i]);
    }
}

template <int kLanes>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Rows [head, head + n) of a token, one chunk of a group of lanes; n = 0: nothing
// (a warp's groups go through their chunks together, their shuffles are by whole warps).
template <int kPer>
struct Chunk {
    int token, head, n;
    uint2 x[kPer][2], dy[kPer][2];
};

// One side (queries or keys) of the call, as a CTA sees it.
struct Side {
    const __nv_bfloat16 *x, *dy;
    __nv_bfloat16* out;
    long long x_stride, dy_stride, out_stride;
    int heads;
};

// kBwd: the gradient.  The grid's first p.q_ctas CTAs take the queries, the others
// the keys.  A group of D / 8 lanes takes chunks of kPer rows of one token, the next
// one's rows (and its angles, whose position came one chunk before) on their way
// while this one is worked on.  Neighbouring groups take neighbouring chunks: runs
// of several chunks of a token, which would read its angles once, were slower by
// half (a gradient of 16384 tokens of 40 heads 153 us against 94).
template <int kD, bool kHalves, int kPer, bool kBwd>
__global__ void __launch_bounds__(kThreads, (kBwd ? kQkNormBwdCtas : kQkNormCtas) + (kPer == 1)) qk_norm_kernel(const __grid_constant__ Params p) {
    constexpr int kLanes = kD / 8, kGroups = kThreads / kLanes, kInWarp = 32 / kLanes;
    if constexpr (kBwd) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int side = static_cast<int>(blockIdx.x) >= p.q_ctas;
    const int cta = blockIdx.x - (side ? p.q_ctas : 0), ctas = side ? gridDim.x - p.q_ctas : p.q_ctas;
    Side a;
    a.x = side ? p.x[1] : p.x[0];
    a.dy = side ? p.dy[1] : p.dy[0];
    a.out = side ? p.out[1] : p.out[0];
    a.x_stride = side ? p.x_stride[1] : p.x_stride[0];
    a.dy_stride = side ? p.dy_stride[1] : p.dy_stride[0];
    a.out_stride = side ? p.out_stride[1] : p.out_stride[0];
    a.heads = side ? p.heads[1] : p.heads[0];
    const Divisor chunks = side ? p.chunks[1] : p.chunks[0];
    const int n_units = side ? p.units[1] : p.units[0];
    const bool normed = (side ? p.w[1] : p.w[0]) != nullptr;
    const int l = threadIdx.x % kLanes, grp = threadIdx.x / kLanes, in_warp = grp % kInWarp;
    const Place at = place_of<kHalves>(l, p.rot);
    float w[8];
    load_weight(p, side, at, w);
    float dw[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] = 0.f;

    const int step = ctas * kGroups;
    int base = cta * kGroups + grp - in_warp;   // the chunk of the warp's first group
    auto position_of = [&](int u) -> int {
        if (p.rot == 0 || u >= n_units) return 0;
        return p.positions != nullptr ? load_ahead(p.positions + chunks.div(u)) : chunks.div(u);
    };
    auto fetch = [&](int u, Chunk<kPer>& c) {
        c.n = 0;
        if (u >= n_units) return;
        c.token = chunks.div(u);
        c.head = (u - c.token * static_cast<int>(chunks.d)) * kPer;
        c.n = min(kPer, a.heads - c.head);
        const long long in_row = static_cast<long long>(c.head) * kD;   // (heads are not bounded: it passes 32 bits)
        const __nv_bfloat16* xs = a.x + c.token * a.x_stride + in_row;
        const __nv_bfloat16* ds = kBwd ? a.dy + c.token * a.dy_stride + in_row : nullptr;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (i >= c.n) continue;
            load8<kHalves>(xs + i * kD, at, c.x[i]);
            if constexpr (kBwd) load8<kHalves>(ds + i * kD, at, c.dy[i]);
        }
    };
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    bool good = true;
    // the angles of position pos; false: it is not in the table
    auto angles = [&](int pos, bool flag, float (&c)[4], float (&s)[4]) -> bool {
        if (p.rot == 0) return true;
        if (pos < 0 || pos >= p.max_pos) {
            if (flag) flag_status(p.status, ATTN_DEV_POSITION_OUT_OF_RANGE);
            return false;
        }
        if (at.turns) {
            const float* row = p.cos_sin + static_cast<size_t>(pos) * p.rot + 4 * l;
            load_ahead(row, c);
            load_ahead(row + p.rot / 2, s);
        }
        return true;
    };
    Chunk<kPer> now, next;
    int pos_next = 0;
    if (base < n_units) {
        const int u = base + in_warp, pos = position_of(u);
        pos_next = position_of(u + step);
        fetch(u, now);
        good = angles(pos, l == 0 && u < n_units && now.head == 0, cs, sn);
    }
    while (base < n_units) {
        const int u_next = base + in_warp + step;
        const bool more = base + step < n_units;
        float cs_next[4] = {1.f, 1.f, 1.f, 1.f}, sn_next[4] = {0.f, 0.f, 0.f, 0.f};
        bool good_next = true;
        if (more) {
            fetch(u_next, next);
            good_next = angles(pos_next, l == 0 && u_next < n_units && next.head == 0, cs_next, sn_next);
            pos_next = position_of(u_next + step);
        }
        __nv_bfloat16* dst = a.out + now.token * a.out_stride + static_cast<long long>(now.head) * kD;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const bool live = i < now.n;
            float v[8], g[8];
            unpack4(now.x[i][0], v);
            unpack4(now.x[i][1], v + 4);
            if constexpr (kBwd) {
                unpack4(now.dy[i][0], g);
                unpack4(now.dy[i][1], g + 4);
                if (at.turns) turn<kHalves>(g, cs, sn, -1.f);
            }
            if (normed) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
                ss = group_sum<kLanes>(ss);
                const float r = rsqrtf(ss * (1.f / kD) + p.eps);
                if constexpr (kBwd) {
                    float along = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= r;   // n
                    if (live && good) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) dw[e] = fmaf(g[e], v[e], dw[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        g[e] *= w[e];
                        along = fmaf(g[e], v[e], along);
                    }
                    along = group_sum<kLanes>(along) * (1.f / kD);
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[e] = r * fmaf(-v[e], along, g[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= r * w[e];
                }
            }
            if constexpr (kBwd) {
                if (!good) {   // the forward pass left the token out
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[e] = 0.f;
                }
                if (live) store8<kHalves>(dst + i * kD, at, g);
            } else {
                if (at.turns) turn<kHalves>(v, cs, sn, 1.f);
                if (live && good) store8<kHalves>(dst + i * kD, at, v);
            }
        }
        if (!more) break;
        base += step;
        now = next;
        good = good_next;
#pragma unroll
        for (int e = 0; e < 4; ++e) cs[e] = cs_next[e], sn[e] = sn_next[e];
    }
    if constexpr (kBwd) {
        if (p.dw_part == nullptr) return;
        __shared__ float acc[kGroups][kD];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            acc[grp][at.i0 + e] = dw[e];
            acc[grp][at.i1 + e] = dw[4 + e];
        }
        __syncthreads();
        if (threadIdx.x < kD) {
            float sum = 0.f;
#pragma unroll 8
            for (int i = 0; i < kGroups; ++i) sum += acc[i][threadIdx.x];
            p.dw_part[static_cast<size_t>(blockIdx.x) * kD + threadIdx.x] = sum;
        }
    }
}

// The CTAs' sums, [q_ctas + k_ctas][d], joined for each side: 32 columns a CTA, 32
// slices of the sum each.
__global__ void __launch_bounds__(kReduceCols* kReduceSlices) qk_norm_reduce_kernel(const float* part, int q_ctas, int k_ctas,
                                                                                    int d, float* dwq, float* dwk) {
    __shared__ float acc[kReduceSlices][kReduceCols];
    const int lane = threadIdx.x % kReduceCols, slice = threadIdx.x / kReduceCols;
    const int per_side = d / kReduceCols, side = static_cast<int>(blockIdx.x) >= per_side;
    const int col = (blockIdx.x - side * per_side) * kReduceCols + lane;
    const int first = side ? q_ctas : 0, n = side ? k_ctas : q_ctas;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float sum = 0.f;
#pragma unroll 8
    for (int i = slice; i < n; i += kReduceSlices) sum += __ldcg(part + static_cast<size_t>(first + i) * d + col);
    acc[slice][lane] = sum;
    __syncthreads();
    if (slice != 0) return;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kReduceSlices; ++i) sum += acc[i][lane];
    float* out = side ? dwk : dwq;
    if (out != nullptr) out[col] = sum;
}

// Rows of one chunk: four have their loads in flight together; one where four
// would leave SMs without work.  16384 tokens of 32 + 8 heads, forward / gradient:
// four 60.1 / 92.5 us (90.9 since), two 61.5 / 96.1, one 93 / 140; one token: four 4.2 / 6.3,
// one 3.9 / 4.9.
constexpr int kMany = 4;
int rows_per_chunk(const QkNormArgs& a, int sms) {
    const long long lanes = static_cast<long long>(a.total) * (a.Hq + a.Hkv) * (a.D / 8);
    return lanes >= static_cast<long long>(kMany) * sms * kThreads ? kMany : 1;
}
// The call's parameters for chunks of `per` rows and up to most_ctas CTAs; the grid.
Params params_of(const QkNormArgs& a, int per, int most_ctas, int& grid) {
    Params p{};
    const int heads[2] = {a.Hq, a.Hkv}, groups = kThreads / (a.D / 8);
    int ctas[2];
    for (int i = 0; i < 2; ++i) {
        p.x[i] = static_cast<const __nv_bfloat16*>(a.x[i]);
        p.dy[i] = static_cast<const __nv_bfloat16*>(a.dy[i]);
        p.out[i] = static_cast<__nv_bfloat16*>(a.out[i]);
        p.x_stride[i] = a.x_stride[i];
        p.dy_stride[i] = a.dy_stride[i];
        p.out_stride[i] = a.out_stride[i];
        p.w[i] = a.weight[i];
        p.heads[i] = heads[i];
        const int chunks = (heads[i] + per - 1) / per;
        p.units[i] = a.total * chunks;
        p.chunks[i] = make_divisor(std::max(chunks, 1));
        const long long need = (static_cast<long long>(p.units[i]) + groups - 1) / groups;
        // a side's part of the CTAs goes by its rows
        const long long part = std::max<long long>(1, static_cast<long long>(most_ctas) * heads[i] / (a.Hq + a.Hkv));
        ctas[i] = heads[i] == 0 ? 0 : static_cast<int>(std::max<long long>(1, std::min(need, part)));
    }
    p.q_ctas = ctas[0];
    grid = ctas[0] + ctas[1];
    p.w_bf16 = a.weight_bf16;
    p.eps = a.eps;
    p.cos_sin = a.cos_sin;
    p.max_pos = a.max_pos;
    p.rot = a.rot_dim;
    p.positions = a.positions;
    p.status = a.dev_status;
    return p;
}

template <typename Call>
cudaError_t by_shape(const QkNormArgs& a, Call call) {
    const bool halves = a.rot_dim > 0 && !a.interleaved;
    if (a.D == 128)
        return halves ? call(std::integral_constant<int, 128>{}, std::true_type{})
                      : call(std::integral_constant<int, 128>{}, std::false_type{});
    return halves ? call(std::integral_constant<int, 64>{}, std::true_type{})
                  : call(std::integral_constant<int, 64>{}, std::false_type{});
}

template <int kPer>
cudaError_t forward(const QkNormArgs& a, int sms, cudaStream_t stream) {
    int grid;
    const Params p = params_of(a, kPer, sms * kQkNormCtas, grid);
    return by_shape(a, [&](auto d, auto halves) {
        qk_norm_kernel<decltype(d)::value, decltype(halves)::value, kPer, false><<<grid, kThreads, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

template <int kPer>
cudaError_t backward(const QkNormArgs& a, int sms, cudaStream_t stream) {
    int grid;
    Params p = params_of(a, kPer, sms * kQkNormBwdCtas, grid);
    const bool sums = a.d_weight[0] != nullptr || a.d_weight[1] != nullptr;
    if (sums) p.dw_part = static_cast<float*>(a.workspace);
    const cudaError_t e = by_shape(a, [&](auto d, auto halves) {
        qk_norm_kernel<decltype(d)::value, decltype(halves)::value, kPer, true><<<grid, kThreads, 0, stream>>>(p);
        return cudaGetLastError();
    });
    if (e != cudaSuccess || !sums) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * a.D / kReduceCols);
    cfg.blockDim = dim3(kReduceCols * kReduceSlices);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, qk_norm_reduce_kernel, static_cast<const float*>(p.dw_part), p.q_ctas, grid - p.q_ctas, a.D,
                              a.d_weight[0], a.d_weight[1]);
}

}  // namespace

size_t qk_norm_bwd_workspace(int D, int sms) { return (static_cast<size_t>(sms) * kQkNormBwdCtas + 1) * D * sizeof(float); }

cudaError_t launch_qk_norm(const QkNormArgs& a, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    return rows_per_chunk(a, sms) == 1 ? forward<1>(a, sms, stream) : forward<kMany>(a, sms, stream);
}

cudaError_t launch_qk_norm_bwd(const QkNormArgs& a, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    return rows_per_chunk(a, sms) == 1 ? backward<1>(a, sms, stream) : backward<kMany>(a, sms, stream);
}

}  // namespace gb300
