// pgd_prefill_api.cu -- the C ABI of the prompt-stage operators (declared in
// include/pgd.h): argument checks and launches.  Nothing here synchronises
// with the host or allocates.
#include <climits>
#include <cmath>

#include "pgd_host.h"
#include "pgd_prefill.h"

namespace {

using namespace pgd;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool supported_block(int bs) { return bs == 16 || bs == 32 || bs == 64; }

// A token stride in elements: rows of `width` elements that do not overlap,
// each starting on a 16-byte boundary, with byte offsets far below 2^40.
bool good_stride(int64_t stride, int64_t width) {
    return stride >= width && stride % 8 == 0 && stride < (int64_t(1) << 36);
}

// Checks shared by the two attention entry points; PGD_OK with *empty = true
// means that there is nothing to do.
pgd_status check_common(int32_t num_seqs, int32_t num_tokens, int32_t max_q_len, int32_t window,
                        int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, float scale,
                        const void *workspace, size_t workspace_bytes, int32_t num_splits,
                        bool *empty) {
    *empty = false;
    if (num_seqs < 0 || num_tokens < 0 || max_q_len < 0 || window < 0 || num_q_heads <= 0 ||
        num_kv_heads <= 0 || num_splits < 0 || num_splits > 64)
        return PGD_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads) return PGD_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return PGD_ERR_INVALID_ARG;
    if (num_q_heads / num_kv_heads > 16) return PGD_ERR_UNSUPPORTED;
    if (head_dim != 128 && head_dim != 256) return PGD_ERR_UNSUPPORTED;
    if (!workspace && workspace_bytes) return PGD_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, 16)) return PGD_ERR_INVALID_ARG;
    *empty = num_seqs == 0 || num_tokens == 0;
    return PGD_OK;
}

pgd_status run(PrefillLaunch &a, void *stream) {
    const pgd_status st = device_info(&a.sms, &a.p.flags);
    if (st != PGD_OK) return st;
    a.p.wait_ns = wait_limit_ns();
    a.stream = static_cast<cudaStream_t>(stream);
    return launch_prefill(a) == cudaSuccess ? PGD_OK : PGD_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t pgd_prefill_workspace_bytes(int32_t num_seqs, int32_t num_tokens, int32_t max_q_len,
                                   int32_t max_context_len, int32_t num_q_heads,
                                   int32_t num_kv_heads, int32_t head_dim, int32_t num_splits) {
    (void)num_seqs; (void)num_tokens; (void)max_q_len; (void)max_context_len;
    (void)num_q_heads; (void)num_kv_heads; (void)head_dim; (void)num_splits;
    return 0;
}

pgd_status pgd_prefill_attention(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                 const void *v, int64_t v_stride, const int32_t *cu_seqlens,
                                 int32_t num_seqs, int32_t num_tokens, int32_t max_seq_len,
                                 int32_t window, int32_t num_q_heads, int32_t num_kv_heads,
                                 int32_t head_dim, float scale, void *out, float *lse_out,
                                 void *workspace, size_t workspace_bytes, int32_t num_splits,
                                 void *stream) {
    bool empty;
    pgd_status st = check_common(num_seqs, num_tokens, max_seq_len, window, num_q_heads,
                                 num_kv_heads, head_dim, scale, workspace, workspace_bytes,
                                 num_splits, &empty);
    if (st != PGD_OK || empty) return st;
    if (!q || !k || !v || !cu_seqlens || !out) return PGD_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
        !aligned(cu_seqlens, 4) || (lse_out && !aligned(lse_out, 4)))
        return PGD_ERR_INVALID_ARG;
    const int64_t qw = static_cast<int64_t>(num_q_heads) * head_dim;
    const int64_t kw = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (!good_stride(q_stride, qw) || !good_stride(k_stride, kw) || !good_stride(v_stride, kw))
        return PGD_ERR_INVALID_ARG;
    PrefillLaunch a = {};
    PrefillParams &p = a.p;
    p.q = static_cast<const uint16_t *>(q);
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.cu = cu_seqlens;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.head_dim = head_dim;
    p.window = window;
    p.splits = 1;
    p.scale = scale;
    p.out = static_cast<uint16_t *>(out);
    p.lse_out = lse_out;
    return run(a, stream);
}

pgd_status pgd_paged_prefill_attention(
    const void *q, int64_t q_stride, const void *k_cache, const void *v_cache,
    const int32_t *block_table, int32_t max_blocks_per_seq, const int32_t *context_lens,
    const int32_t *cu_seqlens, int32_t num_seqs, int32_t num_tokens, int32_t max_q_len,
    int32_t max_context_len, int32_t window, int32_t num_q_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t block_size, int32_t num_blocks, float scale, pgd_kv_dtype kv_dtype,
    const float *k_scale, const float *v_scale, void *out, float *lse_out, void *workspace,
    size_t workspace_bytes, int32_t num_splits, void *stream) {
    bool empty;
    pgd_status st = check_common(num_seqs, num_tokens, max_q_len, window, num_q_heads,
                                 num_kv_heads, head_dim, scale, workspace, workspace_bytes,
                                 num_splits, &empty);
    if (st != PGD_OK) return st;
    if (max_blocks_per_seq <= 0 || num_blocks <= 0 || max_context_len < 0)
        return PGD_ERR_INVALID_ARG;
    if (kv_dtype != PGD_KV_BF16 && kv_dtype != PGD_KV_FP8_E4M3) return PGD_ERR_INVALID_ARG;
    const bool fp8 = kv_dtype == PGD_KV_FP8_E4M3;
    if (!supported_block(block_size) || (fp8 && head_dim != 128)) return PGD_ERR_UNSUPPORTED;
    if (static_cast<long long>(num_blocks) * num_kv_heads >= INT_MAX ||
        static_cast<long long>(max_blocks_per_seq) * block_size >= INT_MAX)
        return PGD_ERR_UNSUPPORTED;
    if (empty) return PGD_OK;
    if (!q || !k_cache || !v_cache || !block_table || !context_lens || !cu_seqlens || !out)
        return PGD_ERR_INVALID_ARG;
    if (fp8 && (!k_scale || !v_scale)) return PGD_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(cu_seqlens, 4) ||
        (lse_out && !aligned(lse_out, 4)) || (k_scale && !aligned(k_scale, 4)) ||
        (v_scale && !aligned(v_scale, 4)))
        return PGD_ERR_INVALID_ARG;
    if (!good_stride(q_stride, static_cast<int64_t>(num_q_heads) * head_dim))
        return PGD_ERR_INVALID_ARG;
    PrefillLaunch a = {};
    PrefillParams &p = a.p;
    p.q = static_cast<const uint16_t *>(q);
    p.k = k_cache;
    p.v = v_cache;
    p.q_stride = q_stride;
    p.cu = cu_seqlens;
    p.context_lens = context_lens;
    p.block_table = block_table;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.fp8 = fp8;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.head_dim = head_dim;
    p.window = window;
    p.splits = 1;
    p.scale = scale;
    p.out = static_cast<uint16_t *>(out);
    p.lse_out = lse_out;
    return run(a, stream);
}

// The row kernels index a token's chunks with 32-bit integers.
constexpr int32_t kMaxRowHeads = 65536;

pgd_status pgd_kv_quant_scales(const void *k_new, const void *v_new, int32_t num_tokens,
                               int32_t num_kv_heads, int32_t head_dim, int32_t accumulate,
                               float *k_scale, float *v_scale, void *stream) {
    if (num_tokens < 0 || num_kv_heads <= 0 || (accumulate != 0 && accumulate != 1))
        return PGD_ERR_INVALID_ARG;
    if (head_dim != 128 && head_dim != 256) return PGD_ERR_UNSUPPORTED;
    if (num_kv_heads > kMaxRowHeads) return PGD_ERR_UNSUPPORTED;
    if (!k_scale || !v_scale || (num_tokens > 0 && (!k_new || !v_new)))
        return PGD_ERR_INVALID_ARG;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
        return PGD_ERR_INVALID_ARG;
    int sms = 0;
    uint32_t *flags = nullptr;
    const pgd_status st = device_info(&sms, &flags);
    if (st != PGD_OK) return st;
    return launch_kv_quant_scales(k_new, v_new, num_tokens, num_kv_heads, head_dim,
                                  accumulate != 0, k_scale, v_scale, sms,
                                  static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PGD_OK
               : PGD_ERR_CUDA;
}

pgd_status pgd_kv_gather(const void *k_cache, const void *v_cache, const int64_t *slot_mapping,
                         int32_t num_tokens, void *k_out, void *v_out, int32_t num_kv_heads,
                         int32_t head_dim, int32_t block_size, int32_t num_blocks,
                         pgd_kv_dtype kv_dtype, const float *k_scale, const float *v_scale,
                         void *stream) {
    if (num_tokens < 0 || num_kv_heads <= 0 || num_blocks <= 0) return PGD_ERR_INVALID_ARG;
    if (kv_dtype != PGD_KV_BF16 && kv_dtype != PGD_KV_FP8_E4M3) return PGD_ERR_INVALID_ARG;
    if (head_dim != 128 && head_dim != 256) return PGD_ERR_UNSUPPORTED;
    if (num_kv_heads > kMaxRowHeads || !supported_block(block_size)) return PGD_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PGD_OK;
    const bool fp8 = kv_dtype == PGD_KV_FP8_E4M3;
    if (!k_cache || !v_cache || !slot_mapping || !k_out || !v_out) return PGD_ERR_INVALID_ARG;
    if (fp8 && (!k_scale || !v_scale)) return PGD_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_out, 16) ||
        !aligned(v_out, 16) || !aligned(slot_mapping, 8) || (k_scale && !aligned(k_scale, 4)) ||
        (v_scale && !aligned(v_scale, 4)))
        return PGD_ERR_INVALID_ARG;
    int sms = 0;
    uint32_t *flags = nullptr;
    const pgd_status st = device_info(&sms, &flags);
    if (st != PGD_OK) return st;
    return launch_kv_gather(k_cache, v_cache, slot_mapping, num_tokens, k_out, v_out,
                            num_kv_heads, head_dim, block_size,
                            static_cast<int64_t>(num_blocks) * block_size, fp8, k_scale, v_scale,
                            flags, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PGD_OK
               : PGD_ERR_CUDA;
}

}  // extern "C"
