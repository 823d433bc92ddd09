// pgd_prefill_api.cu -- the C ABI of the prompt-stage operators (declared in
// include/pgd.h): argument checks and launches.  Nothing here synchronises
// with the host or allocates.
#include <algorithm>
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
                        const void *workspace, size_t workspace_bytes, int32_t num_ctas,
                        bool *empty) {
    *empty = false;
    if (num_seqs < 0 || num_tokens < 0 || max_q_len < 0 || window < 0 || num_q_heads <= 0 ||
        num_kv_heads <= 0 || num_ctas < 0 || num_ctas > kMaxPrefillCtas)
        return PGD_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads) return PGD_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return PGD_ERR_INVALID_ARG;
    if (num_q_heads / num_kv_heads > 16) return PGD_ERR_UNSUPPORTED;
    if (head_dim != 128 && head_dim != 256) return PGD_ERR_UNSUPPORTED;
    if (!workspace && workspace_bytes) return PGD_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, 32)) return PGD_ERR_INVALID_ARG;
    *empty = num_seqs == 0 || num_tokens == 0;
    return PGD_OK;
}

// Units are cut from this many keys on (the host's bound on what a unit's rows
// see).  Cutting evens out what the longest unit would take alone (about 1 us
// per 128 keys) and costs the merge, 9 - 14 us with caches flushed.  Whole /
// cut in us, caches flushed:
//   keys               1024         1280         1536         2048
//   32 heads over 8 of 128, bf16
//     one new token    26.7 / 25.6  30.8 / 27.7  34.8 / 27.8  41.1 / 33.8
//     a prompt         30.8 / 39.9  49.2 / 48.2  61.5 / 54.3  69.7 / 70.7
//     four prompts     65.6 / 76.8  90 / 101     115 / 126    174 / 185
//   32 heads over 8 of 128, E4M3
//     one new token    33.8 / 33.8  37.9 / 33.9  42.0 / 35.8  52.2 / 39.9
//     a prompt         42.0 / 52.2  67.6 / 64.5  76.7 / 64.5  84.0 / 80.9
//     four prompts     82.0 / 91.2  110 / 120    141 / 150    207 / 220
//   32 heads over 4 of 256, bf16
//     one new token    41.0 / 27.6  49.2 / 27.6  55.4 / 29.6  71.7 / 31.7
//     a prompt         43.1 / 52.3  57.4 / 62.3  71.7 / 72.7  111 / 99.3
//     four prompts     100 / 116    141 / 148    178 / 192    276 / 292
// Single tokens gain, equal prompts lose up to a tenth; the host's bounds do
// not tell them apart.
constexpr int64_t kCutKeys = 1280;

// Grid, and whether units are cut: one CTA per SM, one per unit where they
// stay whole.
struct PrefillPlan {
    int grid;
    bool cut;
};

PrefillPlan plan_prefill(int sms, int64_t num_seqs, int64_t num_tokens, int64_t max_keys,
                         int32_t window, int32_t num_q_heads, int32_t num_kv_heads,
                         int32_t head_dim, int32_t num_ctas) {
    if (num_ctas > 0) return {num_ctas, num_ctas > 1};
    const int tpu = unit_rows(head_dim) / 128 * (128 / (num_q_heads / num_kv_heads));
    const int64_t units = (num_tokens / tpu + num_seqs) * num_kv_heads;
    // a window bounds the keys of a unit's tpu rows
    int64_t keys = max_keys > 0 ? max_keys : INT_MAX;
    if (window > 0) keys = std::min<int64_t>(keys, static_cast<int64_t>(window) + tpu);
    if (keys >= kCutKeys) return {sms, true};
    return {static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(sms, units))), false};
}

pgd_status run(PrefillLaunch &a, int64_t max_keys, int32_t num_ctas, void *workspace,
               size_t workspace_bytes, int64_t packed_rows, void *stream) {
    PrefillParams &p = a.p;
    pgd_status st = device_info(&a.sms, &p.flags);
    if (st != PGD_OK) return st;
    PrefillPlan plan = plan_prefill(a.sms, p.num_seqs, p.num_tokens, max_keys, p.window,
                                    p.num_q_heads, p.num_kv_heads, p.head_dim, num_ctas);
    if (plan.cut && workspace_bytes < prefill_workspace(plan.grid, p.head_dim)) {
        if (num_ctas > 0) return PGD_ERR_WORKSPACE;
        plan.cut = false;
    }
    a.grid = plan.grid;
    p.out32 = aligned(p.out, 32);
    if (plan.cut) {
        uint8_t *w = static_cast<uint8_t *>(workspace);
        p.parts = reinterpret_cast<PartRecord *>(w);
        p.o_part = reinterpret_cast<float *>(w + parts_bytes(plan.grid));
        p.lse_part = p.o_part + static_cast<int64_t>(2) * plan.grid * unit_rows(p.head_dim) * p.head_dim;
    }
    p.wait_ns = wait_limit_ns();
    a.stream = static_cast<cudaStream_t>(stream);
    // Q: 64 elements of the group's heads of 128 / g tokens
    const uint64_t d = p.head_dim, hq = p.num_q_heads, hkv = p.num_kv_heads;
    {
        const uint64_t dims[3] = {d, hq, static_cast<uint64_t>(p.num_tokens)};
        const uint64_t strides[2] = {d * 2, static_cast<uint64_t>(p.q_stride) * 2};
        const uint32_t box[3] = {64, static_cast<uint32_t>(p.group),
                                 static_cast<uint32_t>(128 / p.group)};
        st = encode_tiled_map(&a.map_q, p.q, 2, 3, dims, strides, box);
        if (st != PGD_OK) return st;
    }
    for (int i = 0; i < 2; ++i) {
        CUtensorMap *m = i ? &a.map_v : &a.map_k;
        const void *base = i ? p.v : p.k;
        if (p.block_table) {
            // a block of one head: 128-byte lines of its rows
            const uint64_t bs = p.block_size, eb = p.fp8 ? 1 : 2, line = 128 / eb;
            const uint64_t dims[4] = {line, bs, d / line, static_cast<uint64_t>(p.num_blocks) * hkv};
            const uint64_t strides[3] = {d * eb, 128, bs * d * eb};
            const uint32_t box[4] = {static_cast<uint32_t>(line), static_cast<uint32_t>(bs), 1, 1};
            st = encode_tiled_map(m, base, static_cast<int>(eb), 4, dims, strides, box);
        } else {
            const int64_t stride = i ? p.v_stride : p.k_stride;
            const uint64_t dims[3] = {d, hkv, static_cast<uint64_t>(packed_rows)};
            const uint64_t strides[2] = {d * 2, static_cast<uint64_t>(stride) * 2};
            const uint32_t box[3] = {64, 1, 128};
            st = encode_tiled_map(m, base, 2, 3, dims, strides, box);
        }
        if (st != PGD_OK) return st;
    }
    return launch_prefill(a) == cudaSuccess ? PGD_OK : PGD_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t pgd_prefill_workspace_bytes(int32_t num_seqs, int32_t num_tokens, int32_t max_context_len,
                                   int32_t window, int32_t num_q_heads, int32_t num_kv_heads,
                                   int32_t head_dim, int32_t num_ctas) {
    bool empty;
    if (max_context_len < 0 ||
        check_common(num_seqs, num_tokens, 0, window, num_q_heads, num_kv_heads, head_dim, 1.f,
                     nullptr, 0, num_ctas, &empty) != PGD_OK || empty)
        return 0;
    int sms = 0;
    uint32_t *flags = nullptr;
    if (device_info(&sms, &flags) != PGD_OK) return 0;
    const PrefillPlan plan = plan_prefill(sms, num_seqs, num_tokens, max_context_len, window,
                                          num_q_heads, num_kv_heads, head_dim, num_ctas);
    return plan.cut ? prefill_workspace(plan.grid, head_dim) : 0;
}

pgd_status pgd_prefill_attention(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                 const void *v, int64_t v_stride, const int32_t *cu_seqlens,
                                 int32_t num_seqs, int32_t num_tokens, int32_t max_seq_len,
                                 int32_t window, int32_t num_q_heads, int32_t num_kv_heads,
                                 int32_t head_dim, float scale, void *out, float *lse_out,
                                 void *workspace, size_t workspace_bytes, int32_t num_ctas,
                                 void *stream) {
    bool empty;
    pgd_status st = check_common(num_seqs, num_tokens, max_seq_len, window, num_q_heads,
                                 num_kv_heads, head_dim, scale, workspace, workspace_bytes,
                                 num_ctas, &empty);
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
    p.scale = scale;
    p.out = static_cast<uint16_t *>(out);
    p.lse_out = lse_out;
    const int64_t keys = max_seq_len > 0 && max_seq_len < num_tokens ? max_seq_len : num_tokens;
    return run(a, keys, num_ctas, workspace, workspace_bytes, num_tokens, stream);
}

pgd_status pgd_paged_prefill_attention(
    const void *q, int64_t q_stride, const void *k_cache, const void *v_cache,
    const int32_t *block_table, int32_t max_blocks_per_seq, const int32_t *context_lens,
    const int32_t *cu_seqlens, int32_t num_seqs, int32_t num_tokens, int32_t max_q_len,
    int32_t max_context_len, int32_t window, int32_t num_q_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t block_size, int32_t num_blocks, float scale, pgd_kv_dtype kv_dtype,
    const float *k_scale, const float *v_scale, void *out, float *lse_out, void *workspace,
    size_t workspace_bytes, int32_t num_ctas, void *stream) {
    bool empty;
    pgd_status st = check_common(num_seqs, num_tokens, max_q_len, window, num_q_heads,
                                 num_kv_heads, head_dim, scale, workspace, workspace_bytes,
                                 num_ctas, &empty);
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
    p.scale = scale;
    p.out = static_cast<uint16_t *>(out);
    p.lse_out = lse_out;
    // the table's width bounds every context
    const int64_t cap = static_cast<int64_t>(max_blocks_per_seq) * block_size;
    const int64_t keys = max_context_len > 0 && max_context_len < cap ? max_context_len : cap;
    return run(a, keys, num_ctas, workspace, workspace_bytes, 0, stream);
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
                            flags, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PGD_OK
               : PGD_ERR_CUDA;
}

}  // extern "C"
