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
// The gradient of a weight is a sum over all rows of all tokens: each lane
// keeps its eight columns of both weights in registers over the rows it takes,
// a CTA joins its lanes in order, and a second kernel the CTAs, in order: the
// result does not depend on timing.
//
// Bound: the bytes of x (and dy) in and y (or dx) out.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
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
    int units[2];                 // units of kPer rows per token
    bool w_bf16;
    float eps;
    const float* cos_sin;
    int max_pos, rot;
    const int32_t* positions;     // NULL: the token's index
    int n_units;
    float* dw_part;               // [grid][2][D]
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

// The rows of unit `u`: up to kPer heads of one token's queries or keys.
struct Unit {
    int token, which, head, n;
};
template <int kPer>
__device__ __forceinline__ Unit unit_of(const Params& p, int u) {
    const int per_token = p.units[0] + p.units[1];
    Unit x;
    x.token = u / per_token;
    const int i = u - x.token * per_token;
    x.which = i >= p.units[0];
    x.head = (x.which ? i - p.units[0] : i) * kPer;
    x.n = min(kPer, (x.which ? p.heads[1] : p.heads[0]) - x.head);
    return x;
}
__device__ __forceinline__ const __nv_bfloat16* row_of(const __nv_bfloat16* const (&base)[2], const long long (&stride)[2],
                                                       const Unit& x, int d) {
    return (x.which ? base[1] : base[0]) + x.token * (x.which ? stride[1] : stride[0]) + x.head * d;
}

// Cosines and sines of the lane; false: the token's position is not in the table.
__device__ __forceinline__ bool angles(const Params& p, int token, int l, const Place& a, bool first, float (&c)[4],
                                       float (&s)[4]) {
    if (p.rot == 0) return true;
    const int pos = p.positions != nullptr ? p.positions[token] : token;
    const bool good = pos >= 0 && pos < p.max_pos;
    if (!good && first) flag_status(p.status, ATTN_DEV_POSITION_OUT_OF_RANGE);
    if (good && a.turns) {
        const float* row = p.cos_sin + static_cast<size_t>(pos) * p.rot + 4 * l;
        const float4 vc = *reinterpret_cast<const float4*>(row), vs = *reinterpret_cast<const float4*>(row + p.rot / 2);
        c[0] = vc.x, c[1] = vc.y, c[2] = vc.z, c[3] = vc.w;
        s[0] = vs.x, s[1] = vs.y, s[2] = vs.z, s[3] = vs.w;
    }
    return good;
}

template <int kD, bool kHalves, int kPer>
__global__ void __launch_bounds__(kThreads) qk_norm_kernel(const __grid_constant__ Params p) {
    constexpr int kLanes = kD / 8;
    const int l = threadIdx.x % kLanes;
    const int u = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    const bool live = u < p.n_units;
    const Place a = place_of<kHalves>(l, p.rot);
    const Unit x = unit_of<kPer>(p, live ? u : 0);
    const int n = live ? x.n : 0;
    const __nv_bfloat16* src = row_of(p.x, p.x_stride, x, kD);
    uint2 raw[kPer][2];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        raw[i][0] = raw[i][1] = make_uint2(0u, 0u);
        if (i < n) load8<kHalves>(src + i * kD, a, raw[i]);
    }
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f}, w[8];
    const bool good = angles(p, x.token, l, a, live && x.head == 0 && l == 0, c, s);
    load_weight(p, x.which, a, w);
    const bool normed = (x.which ? p.w[1] : p.w[0]) != nullptr;
    __nv_bfloat16* dst = (x.which ? p.out[1] : p.out[0]) + x.token * (x.which ? p.out_stride[1] : p.out_stride[0]) + x.head * kD;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        float y[8];
        unpack4(raw[i][0], y);
        unpack4(raw[i][1], y + 4);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
        ss = group_sum<kLanes>(ss);
        const float r = rsqrtf(ss * (1.f / kD) + p.eps);
        if (normed) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= r * w[e];
        }
        if (a.turns) turn<kHalves>(y, c, s, 1.f);
        if (i < n && good) store8<kHalves>(dst + i * kD, a, y);
    }
}

template <int kD, bool kHalves, int kPer>
__global__ void __launch_bounds__(kThreads) qk_norm_bwd_kernel(const __grid_constant__ Params p) {
    constexpr int kLanes = kD / 8, kGroups = kThreads / kLanes;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int l = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
    const Place a = place_of<kHalves>(l, p.rot);
    float dw[2][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.f;
    // (a warp's groups leave the loop together: its shuffles are by whole warps)
    const int warp_group = blockIdx.x * kGroups + (threadIdx.x & ~31) / kLanes, in_warp = grp - (threadIdx.x & ~31) / kLanes;
    for (long long u0 = warp_group; u0 < p.n_units; u0 += gridDim.x * kGroups) {
        const bool live = u0 + in_warp < p.n_units;
        const Unit x = unit_of<kPer>(p, live ? static_cast<int>(u0) + in_warp : 0);
        const int n = live ? x.n : 0;
        const __nv_bfloat16* xs = row_of(p.x, p.x_stride, x, kD);
        const __nv_bfloat16* ds = row_of(p.dy, p.dy_stride, x, kD);
        uint2 xr[kPer][2], dr[kPer][2];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            xr[i][0] = xr[i][1] = dr[i][0] = dr[i][1] = make_uint2(0u, 0u);
            if (i < n) {
                load8<kHalves>(xs + i * kD, a, xr[i]);
                load8<kHalves>(ds + i * kD, a, dr[i]);
            }
        }
        float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f}, w[8];
        const bool good = angles(p, x.token, l, a, live && x.head == 0 && l == 0, c, s);
        load_weight(p, x.which, a, w);
        const bool normed = (x.which ? p.w[1] : p.w[0]) != nullptr;
        __nv_bfloat16* dst = (x.which ? p.out[1] : p.out[0]) + x.token * (x.which ? p.out_stride[1] : p.out_stride[0]) + x.head * kD;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            float v[8], g[8];
            unpack4(xr[i][0], v);
            unpack4(xr[i][1], v + 4);
            unpack4(dr[i][0], g);
            unpack4(dr[i][1], g + 4);
            if (a.turns) turn<kHalves>(g, c, s, -1.f);
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
            ss = group_sum<kLanes>(ss);
            const float r = rsqrtf(ss * (1.f / kD) + p.eps);
            const bool counts = i < n && good;
            float along = 0.f, back[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] *= r;   // n
                const float t = counts ? g[e] * v[e] : 0.f;
                dw[0][e] += x.which ? 0.f : t;
                dw[1][e] += x.which ? t : 0.f;
                back[e] = g[e] * w[e];
                along = fmaf(back[e], v[e], along);
            }
            along = group_sum<kLanes>(along) * (1.f / kD);
            if (normed) {
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] = r * fmaf(-v[e], along, back[e]);
            }
            if (!good) {   // the forward pass left the token out
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] = 0.f;
            }
            if (i < n) store8<kHalves>(dst + i * kD, a, g);
        }
    }
    if (p.dw_part == nullptr) return;
    __shared__ float acc[kGroups][kD];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            acc[grp][a.i0 + e] = dw[which][e];
            acc[grp][a.i1 + e] = dw[which][4 + e];
        }
        __syncthreads();
        if (threadIdx.x < kD) {
            float sum = 0.f;
#pragma unroll 8
            for (int i = 0; i < kGroups; ++i) sum += acc[i][threadIdx.x];
            p.dw_part[(static_cast<size_t>(blockIdx.x) * 2 + which) * kD + threadIdx.x] = sum;
        }
    }
}

// The CTAs' sums, [n][2 d], joined: 32 columns a CTA, 32 slices of the sum each.
__global__ void __launch_bounds__(kReduceCols* kReduceSlices) qk_norm_reduce_kernel(const float* part, int n, int d,
                                                                                    float* dwq, float* dwk) {
    __shared__ float acc[kReduceSlices][kReduceCols];
    const int lane = threadIdx.x % kReduceCols, slice = threadIdx.x / kReduceCols;
    const int col = blockIdx.x * kReduceCols + lane;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float sum = 0.f;
#pragma unroll 8
    for (int i = slice; i < n; i += kReduceSlices) sum += __ldcg(part + static_cast<size_t>(i) * 2 * d + col);
    acc[slice][lane] = sum;
    __syncthreads();
    if (slice != 0) return;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kReduceSlices; ++i) sum += acc[i][lane];
    float* out = col < d ? dwq : dwk;   // (a CTA's columns belong to one of them)
    if (out != nullptr) out[col < d ? col : col - d] = sum;
}

// Heads of one unit: four rows share a token's angles and have their loads in
// flight together; one row where four would leave SMs without work.
constexpr int kMany = 4;
int rows_per_unit(const QkNormArgs& a, int sms) {
    const long long lanes = static_cast<long long>(a.total) * (a.Hq + a.Hkv) * (a.D / 8);
    return lanes >= static_cast<long long>(kMany) * sms * kThreads ? kMany : 1;
}

Params params_of(const QkNormArgs& a, int per) {
    Params p{};
    const int heads[2] = {a.Hq, a.Hkv};
    for (int i = 0; i < 2; ++i) {
        p.x[i] = static_cast<const __nv_bfloat16*>(a.x[i]);
        p.dy[i] = static_cast<const __nv_bfloat16*>(a.dy[i]);
        p.out[i] = static_cast<__nv_bfloat16*>(a.out[i]);
        p.x_stride[i] = a.x_stride[i];
        p.dy_stride[i] = a.dy_stride[i];
        p.out_stride[i] = a.out_stride[i];
        p.w[i] = a.weight[i];
        p.heads[i] = heads[i];
        p.units[i] = (heads[i] + per - 1) / per;
    }
    p.w_bf16 = a.weight_bf16;
    p.eps = a.eps;
    p.cos_sin = a.cos_sin;
    p.max_pos = a.max_pos;
    p.rot = a.rot_dim;
    p.positions = a.positions;
    p.n_units = a.total * (p.units[0] + p.units[1]);
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
cudaError_t forward(const QkNormArgs& a, cudaStream_t stream) {
    const Params p = params_of(a, kPer);
    const int groups = kThreads / (a.D / 8);
    const int grid = (p.n_units + groups - 1) / groups;
    return by_shape(a, [&](auto d, auto halves) {
        qk_norm_kernel<decltype(d)::value, decltype(halves)::value, kPer><<<grid, kThreads, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

template <int kPer>
cudaError_t backward(const QkNormArgs& a, int sms, cudaStream_t stream) {
    Params p = params_of(a, kPer);
    const int groups = kThreads / (a.D / 8);
    const int grid = std::max(1, std::min((p.n_units + groups - 1) / groups, sms * kQkNormCtas));
    const bool sums = a.d_weight[0] != nullptr || a.d_weight[1] != nullptr;
    if (sums) p.dw_part = static_cast<float*>(a.workspace);
    const cudaError_t e = by_shape(a, [&](auto d, auto halves) {
        qk_norm_bwd_kernel<decltype(d)::value, decltype(halves)::value, kPer><<<grid, kThreads, 0, stream>>>(p);
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
    return cudaLaunchKernelEx(&cfg, qk_norm_reduce_kernel, static_cast<const float*>(p.dw_part), grid, a.D, a.d_weight[0],
                              a.d_weight[1]);
}

}  // namespace

size_t qk_norm_bwd_workspace(int D, int sms) { return static_cast<size_t>(sms) * kQkNormCtas * 2 * D * sizeof(float); }

cudaError_t launch_qk_norm(const QkNormArgs& a, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    return rows_per_unit(a, sms) == 1 ? forward<1>(a, stream) : forward<kMany>(a, stream);
}

cudaError_t launch_qk_norm_bwd(const QkNormArgs& a, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    return rows_per_unit(a, sms) == 1 ? backward<1>(a, sms, stream) : backward<kMany>(a, sms, stream);
}

}  // namespace gb300
