// pgd_prefill.h -- parameters of the prompt attention kernels, shared by the
// C ABI and the kernel unit.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pgd {

struct PrefillParams {
    const uint16_t *q;            // bf16 bits, token rows of Hq * D at q_stride
    const void *k, *v;            // packed bf16 rows, or the paged caches
    const int32_t *cu;            // [num_seqs + 1] first packed row of each sequence
    const int32_t *context_lens;  // [num_seqs] keys per sequence; null: packed K/V
    const int32_t *block_table;   // [num_seqs][max_blocks_per_seq]; null: packed K/V
    const float *k_scale, *v_scale;   // [Hkv] (FP8 only)
    uint16_t *out;                // bf16 bits [num_tokens][Hq][D]
    float *lse_out;               // [num_tokens][Hq] natural log, may be null
    float *o_part;                // [splits][num_tokens][Hq][D], splits > 1 only
    float *lse_part;              // [splits][num_tokens][Hq], natural log
    uint32_t *flags;
    int64_t q_stride, k_stride, v_stride;   // elements between packed tokens
    uint64_t wait_ns;
    int32_t num_seqs, num_tokens;
    int32_t num_q_heads, num_kv_heads, group, head_dim;
    int32_t max_blocks_per_seq, block_size, num_blocks;
    int32_t window, splits, fp8;
    float scale;
};

struct PrefillLaunch {
    PrefillParams p;
    int sms;
    cudaStream_t stream;
};

cudaError_t launch_prefill(const PrefillLaunch &a);

// Packed rows of K/V quantisation and of reading a cache back (pgd_rows.cu).
cudaError_t launch_kv_quant_scales(const void *k_new, const void *v_new, int32_t num_tokens,
                                   int32_t hkv, int32_t head_dim, bool accumulate, float *k_scale,
                                   float *v_scale, int sms, cudaStream_t stream);
cudaError_t launch_kv_gather(const void *k_cache, const void *v_cache, const int64_t *slots,
                             int32_t num_tokens, void *k_out, void *v_out, int32_t hkv,
                             int32_t head_dim, int32_t block_size, int64_t pool_slots, bool fp8,
                             const float *k_scale, const float *v_scale, uint32_t *flags,
                             cudaStream_t stream);

}  // namespace pgd
