// common.cuh - host/device declarations shared by the kernels and the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "../../include/attn.h"

namespace gb300 {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Records a device-side error bit (never traps).
__device__ __forceinline__ void flag_status(int32_t* status, int32_t bit) {
    if (status != nullptr) atomicOr(status, bit);
}

// a + b of counts that are not negative, at most INT_MAX: sums over sequences, whose
// rows overlap where offsets fall, so that no tensor's size bounds them.
__device__ __forceinline__ int add_capped(int a, int b) {
    return static_cast<int>(min(static_cast<unsigned>(a) + static_cast<unsigned>(b), 0x7FFFFFFFu));
}

__device__ __forceinline__ uint8_t* align_1024(uint8_t* p) {
    return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

__device__ __forceinline__ void named_barrier_sync(int id, int nthreads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// ---------------------------------------------------------------- host side

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link
// dependency on libcuda).  Returns false on failure.
bool encode_tiled_map(CUtensorMap* map, CUtensorMapDataType dtype, int rank, const void* base,
                      const uint64_t* dims, const uint64_t* strides_bytes, const uint32_t* box,
                      CUtensorMapSwizzle swizzle);

int device_sm_count();
// Whether the fused decodes may use cooperative launches (attn_decode_cooperative).
bool cooperative_launch_enabled();

// Launchers (return a cudaError_t from the launch).
struct DecodeArgs {
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_table;
    int max_pages;
    const int32_t* seq_lens;
    int kv_format;   // 0 bf16, 1 int4
    int n_groups;
    int B, Hq, Hkv, D, num_pages, page_size, split_tokens, max_kv_len, n_split;
    float scale;
    int q_len;   // queries per sequence (causal multi-query decode when > 1)
    float* o_part;
    float* lse_part;
    int32_t* dev_status;
    // fused mode (counters not NULL): the last split of each (sequence, KV head)
    // merges its partials into o_final / lse_final inside the launch
    int32_t* counters;   // [B * Hkv], zero when the launch starts
    void* o_final;       // bf16 [B, Hq, q_len, D]
    float* lse_final;    // [B, Hq, q_len] or NULL
};
// With `occ` set, a decode launcher launches nothing: it writes how many CTAs
// of the kernel it would launch fit on one SM at once.
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t stream, int* occ = nullptr);
cudaError_t launch_decode_int4(const DecodeArgs& a, cudaStream_t stream, int* occ = nullptr);
// int4 rows of four 32-element groups and at most 8 (query, head) rows per KV
// head: the fp16-subnormal code-space kernel of decode_int4_g32.cu.
bool decode_int4_g32_shape_ok(const DecodeArgs& a);   // shape only (no page or split size)
bool decode_int4_g32_supported(const DecodeArgs& a);
cudaError_t launch_decode_int4_g32(const DecodeArgs& a, cudaStream_t stream, int* occ = nullptr);
// fp8 rows, KV head counts that are multiples of 8 and at most 8 (query, head)
// rows per KV head: the persistent kernel of decode_fp8_g32.cu.
bool decode_fp8_g32_shape_ok(const DecodeArgs& a);   // shape only (no page or split size)
bool decode_fp8_g32_supported(const DecodeArgs& a);
cudaError_t launch_decode_fp8_g32(const DecodeArgs& a, const void* k_scale_shift, const void* v_scale_shift,
                                  cudaStream_t stream, int* occ = nullptr);
cudaError_t launch_decode_fp8(const DecodeArgs& a, const void* k_scale_shift, const void* v_scale_shift,
                              cudaStream_t stream, int* occ = nullptr);
int rows_per_cta(const DecodeArgs& a);

// CTAs of `kern` (with its shared-memory attributes set as for a launch)
// resident on one SM at once.
template <typename K>
cudaError_t ctas_per_sm(K kern, int threads, size_t smem, int* occ) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    return e == cudaSuccess ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(occ, kern, threads, smem) : e;
}

// Runs `set` (a kernel's attributes, which last) the first time it is asked on
// the current device.
template <typename Set>
cudaError_t once_per_device(std::atomic<uint64_t>& done, Set set) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
    e = set();
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

cudaError_t launch_wait_timeout_selftest(int32_t* status, uint64_t limit_ns, cudaStream_t stream);

cudaError_t launch_merge(const float* o_part, const float* lse_part, int N, int S, int D, void* o,
                         float* lse, int o_dtype, cudaStream_t stream);
cudaError_t launch_merge_bwd(const float* o_part, const float* lse_part, const float* d_o, const float* d_lse, int N,
                             int S, int D, float* d_o_part, float* d_lse_part, cudaStream_t stream);

struct PrefillArgs {
    const void* q;
    const void* k;
    const void* v;
    void* o;
    float* lse;
    int dtype;  // ATTN_F32 / ATTN_BF16
    int B, Hq, Hkv, q_len, kv_len, D;
    float scale;
    int32_t* dev_status;
    void* ws;          // split-schedule scratch (NULL: whole items only)
    size_t ws_bytes;
};
cudaError_t launch_prefill_simt(const PrefillArgs& a, cudaStream_t stream);
bool prefill_tc_supported(const PrefillArgs& a);
cudaError_t launch_prefill_tc(const PrefillArgs& a, cudaStream_t stream);
// Scratch of the split schedule on a device with `sms` SMs, and the leading
// part of it (the counters) that must be zero when a launch starts.
size_t prefill_tc_workspace_bytes(const PrefillArgs& a, int sms);
size_t prefill_tc_counter_bytes(const PrefillArgs& a);
// 1 if a launch with a workspace takes the split schedule, else 0; *grid = its CTAs.
int prefill_tc_plan(const PrefillArgs& a, int sms, int* grid);

struct VarlenArgs {
    const void* q;          // [total_q, Hq, D] bf16
    const void* k_cache;    // [num_pages, page_size, Hkv, D] bf16
    const void* v_cache;
    const int32_t* qo_indptr;
    const int32_t* kv_indptr;
    const int32_t* kv_indices;
    const int32_t* kv_last_page_len;   // may be NULL
    void* o;                // [total_q, Hq, D] bf16
    float* lse;             // [total_q, Hq]
    int B, Hq, Hkv, D, total_q, num_pages, page_size;
    float scale;
    int32_t* dev_status;
    void* kv_ws;            // NULL: gather rows inside the kernel; else contiguous K then V copy
    int max_kv_rows;        // rows the copy holds (>= kv_indptr[B] * page_size)
    bool copied;            // the caller has made the copy: no gather is launched
    // with `copied`, the (sequence, query block) pairs longest first,
    // varlen_max_pairs() words of sequence << varlen_pair_bits() | query block
    // (used if there are no more of them); NULL: every CTA sorts them itself
    const uint32_t* order;
    const int32_t* order_n;   // how many
};
// A paged cache's new tokens (kv_append.cu).
struct AppendArgs {
    const void* q;          // [total_q, Hq, D] bf16, rows q_stride elements apart; NULL: no queries
    const void* k;          // [total_q, Hkv, D] bf16
    const void* v;
    long long q_stride, k_stride, v_stride;
    const float* cos_sin;   // [max_pos, rot_dim]
    int max_pos, rot_dim, interleaved;
    const int32_t* positions;     // [total_q], may be NULL
    const int32_t* qo_indptr;     // [B + 1], may be NULL
    const int32_t* seq_lens;      // [B], after the append
    const int32_t* block_table;   // [B, max_pages], or with kv_indptr a CSR list
    const int32_t* kv_indptr;
    int max_pages;
    void* q_out;            // [total_q, Hq, D]
    void* k_cache;          // [num_pages, page_size, Hkv, D]
    void* v_cache;
    float* k_scale;         // NULL: bf16 cache; else [num_pages, page_size / block_tokens, Hkv]
    float* v_scale;
    int B, total_q, Hq, Hkv, num_pages, page_size, block_tokens;
    int32_t* dev_status;
};
cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream);

// The readers of the block-scaled e4m3 cache (decode_fp8_block.cu, prefill_fp8_block.cu).
struct DecodeBlockArgs {
    const void* q;          // [B, q_len, Hq, D] bf16
    const void* k_cache;    // [num_pages, page_size, Hkv, D] e4m3
    const void* v_cache;
    const float* k_scale;   // [num_pages, page_size / block_tokens, Hkv]
    const float* v_scale;
    const int32_t* block_table;
    const int32_t* kv_indptr;   // may be NULL
    int max_pages;
    const int32_t* seq_lens;
    int B, q_len, Hq, Hkv, num_pages, page_size, block_tokens;
    float scale;
    void* workspace;
    void* o;                // as q
    float* lse;             // [B, q_len, Hq] or NULL
    int32_t* dev_status;
};
int decode_fp8_block_max_seqs();
size_t decode_fp8_block_workspace(int q_len, int Hq, int Hkv, int sms);
cudaError_t launch_decode_fp8_block(const DecodeBlockArgs& a, cudaStream_t stream);

struct PrefillBlockArgs {
    const void* q;          // [total_q, Hq, D] bf16
    const void* k_cache;
    const void* v_cache;
    const float* k_scale;
    const float* v_scale;
    const int32_t* qo_indptr;   // [B + 1]
    const int32_t* block_table;
    const int32_t* kv_indptr;   // may be NULL
    int max_pages;
    const int32_t* seq_lens;
    int B, total_q, Hq, Hkv, num_pages, page_size, block_tokens, max_kv_rows;
    float scale;
    void* workspace;
    void* o;                // as q
    float* lse;             // [total_q, Hq] or NULL
    int32_t* dev_status;
};
size_t prefill_fp8_block_workspace(int B, int max_kv_rows, int Hkv);
cudaError_t launch_prefill_fp8_block(const PrefillBlockArgs& a, cudaStream_t stream);

// Norm and rotation of queries (0) and keys (1) by head (qk_norm.cu).
struct QkNormArgs {
    const void* x[2];       // [total, heads, D] bf16, rows x_stride elements apart
    const void* dy[2];      // backward: gradients of the outputs
    void* out[2];           // the outputs, or backward the gradients of x
    long long x_stride[2], dy_stride[2], out_stride[2];
    const void* weight[2];  // [D]; NULL: rotation alone
    bool weight_bf16;       // else float32
    float eps;
    const float* cos_sin;   // [max_pos, rot_dim]
    int max_pos, rot_dim, interleaved;
    const int32_t* positions;   // [total], may be NULL
    int total, Hq, Hkv, D;      // Hq or Hkv 0: absent
    float* d_weight[2];     // backward: [D] or NULL
    void* workspace;        // backward with a d_weight
    int32_t* dev_status;
};
constexpr int kQkNormCtas = 3, kQkNormBwdCtas = 2;   // CTAs per SM of the passes
size_t qk_norm_bwd_workspace(int D, int sms);
cudaError_t launch_qk_norm(const QkNormArgs& a, cudaStream_t stream);
cudaError_t launch_qk_norm_bwd(const QkNormArgs& a, cudaStream_t stream);

// Attention of a ragged batch over contiguous keys (prefill_tc.cu).
struct VarlenFwdArgs {
    const void* q;          // [total_q, Hq, D] bf16, rows q_stride elements apart
    const void* k;          // [total_kv, Hkv, D]
    const void* v;
    long long q_stride, k_stride, v_stride;
    const int32_t* qo_indptr;   // [B + 1]
    const int32_t* kv_indptr;   // [B + 1]
    const int32_t* kv_lens;     // [B], may be NULL
    int causal, B, total_q, total_kv, Hq, Hkv, D;
    float scale;
    void* workspace;
    void* o;                // [total_q, Hq, D], dense
    float* lse;             // [total_q, Hq] or NULL
    int32_t* dev_status;
};
size_t varlen_fwd_workspace(int B, int total_q, int total_kv, int Hq, int Hkv, int D, int sms);
cudaError_t launch_varlen_fwd(const VarlenFwdArgs& a, cudaStream_t stream);

// Its gradient (varlen_bwd.cu).
struct VarlenBwdArgs {
    const void* d_o;        // [total_q, Hq, D] bf16, as q, k, v and o: rows *_stride elements apart
    const void* q;
    const void* k;          // [total_kv, Hkv, D]
    const void* v;
    const void* o;
    long long do_stride, q_stride, k_stride, v_stride, o_stride;
    const float* lse;       // [total_q, Hq]
    const float* d_lse;     // [total_q, Hq] or NULL
    const int32_t* qo_indptr;
    const int32_t* kv_indptr;
    const int32_t* kv_lens;
    int causal, B, total_q, total_kv, Hq, Hkv, D;
    float scale;
    void* workspace;
    void* d_q;              // written, rows *_stride elements apart
    void* d_k;
    void* d_v;
    long long dq_stride, dk_stride, dv_stride;
    int32_t* dev_status;
};
size_t varlen_bwd_workspace(int B, int total_q, int total_kv, int Hq, int Hkv, int D, int sms);
bool varlen_bwd_grid_ok(int B, int total_q, int total_kv, int Hq, int Hkv, int sms);
cudaError_t launch_varlen_bwd(const VarlenBwdArgs& a, cudaStream_t stream);

// Single tokens' attention to contiguous keys (cross_decode.cu).
struct CrossDecodeArgs {
    const void* q;          // [B, q_len, Hq, D] bf16
    const void* k;          // [total_kv, Hkv, D], rows k_stride elements apart
    const void* v;
    long long k_stride, v_stride;
    const int32_t* kv_indptr;   // [B + 1]
    const int32_t* kv_lens;     // [B], may be NULL
    int B, q_len, total_kv, Hq, Hkv, D;
    float scale;
    void* workspace;
    void* o;                // as q
    float* lse;             // [B, q_len, Hq] or NULL
    int32_t* dev_status;
};
int cross_decode_max_seqs();
size_t cross_decode_workspace(int q_len, int Hq, int Hkv, int D, int sms);
cudaError_t launch_cross_decode(const CrossDecodeArgs& a, cudaStream_t stream);

int varlen_max_seqs();
int varlen_max_pairs();
int varlen_pair_bits();
cudaError_t launch_prefill_varlen_tc(const VarlenArgs& a, cudaStream_t stream);

}  // namespace gb300
