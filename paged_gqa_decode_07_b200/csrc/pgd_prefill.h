// pgd_prefill.h -- parameters of the prompt attention kernels, shared by the
// C ABI and the kernel unit.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pgd {

// Shares of the work that a call may ask for.
constexpr int kMaxPrefillCtas = 1024;

// What the merge of cut units needs to know of each CTA's start.
struct alignas(16) PartRecord {
    long long unit;               // axis position of the unit it starts in
    int32_t cut, tiles;           // key tile of that unit it starts at (0: not inside), of how many
    int32_t row0, ntok, h, pad;
};

struct PrefillParams {
    const uint16_t *q;            // bf16 bits, token rows of Hq * D at q_stride
    const void *k, *v;            // packed bf16 rows, or the paged caches
    const int32_t *cu;            // [num_seqs + 1] first packed row of each sequence
    const int32_t *context_lens;  // [num_seqs] keys per sequence; null: packed K/V
    const int32_t *block_table;   // [num_seqs][max_blocks_per_seq]; null: packed K/V
    const float *k_scale, *v_scale;   // [Hkv] (FP8 only)
    uint16_t *out;                // bf16 bits [num_tokens][Hq][D]
    float *lse_out;               // [num_tokens][Hq] natural log, may be null
    PartRecord *parts;            // [grid]; null: units are not cut
    float *o_part;                // [2 * grid][256 or 128 rows][D]
    float *lse_part;              // [2 * grid][256 or 128 rows], natural log
    uint32_t *flags;
    int64_t q_stride, k_stride, v_stride;   // elements between packed tokens
    uint64_t wait_ns;
    int32_t num_seqs, num_tokens;
    int32_t num_q_heads, num_kv_heads, group, head_dim;
    int32_t max_blocks_per_seq, block_size, num_blocks;
    int32_t window, fp8, out32;   // out32: out starts on 32 bytes
    float scale;
};

// Query rows of a unit: two tiles of 128 at head_dim 128, one at 256.
inline int unit_rows(int head_dim) { return head_dim == 128 ? 256 : 128; }

// Workspace of a grid whose units may be cut: the records, then the partial
// outputs and log-sum-exps of two pieces per CTA.
inline size_t parts_bytes(int grid) {
    return (static_cast<size_t>(grid) * sizeof(PartRecord) + 127) / 128 * 128;
}
inline size_t prefill_workspace(int grid, int head_dim) {
    const size_t rows = static_cast<size_t>(2) * grid * unit_rows(head_dim);
    return parts_bytes(grid) + rows * head_dim * 4 + rows * 4;
}

struct PrefillLaunch {
    PrefillParams p;
    CUtensorMap map_q, map_k, map_v;
    int grid, sms;
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
                             int sms, cudaStream_t stream);

}  // namespace pgd
