// pgd_prefill.cu -- prompt attention, one warp per query row.
#include "pgd_prefill.h"
#include "pgd_prefill_rows.cuh"

namespace pgd {

constexpr int kRowWarps = 8;

template <int D, bool FP8>
__global__ void __launch_bounds__(32 * kRowWarps) prefill_rows_kernel(const PrefillParams p) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
    if (row >= static_cast<int64_t>(p.num_tokens) * p.num_q_heads) return;
    const int32_t tok = static_cast<int32_t>(row / p.num_q_heads);
    const int32_t qh = static_cast<int32_t>(row % p.num_q_heads);
    int32_t a = 0, b = p.num_seqs;                 // the sequence with cu[a] <= tok < cu[a + 1]
    while (b - a > 1) {
        const int32_t mid = (a + b) / 2;
        if (__ldg(p.cu + mid) <= tok) a = mid; else b = mid;
    }
    const int32_t c0 = __ldg(p.cu + a), c1 = __ldg(p.cu + a + 1);
    if (c0 < 0 || c1 < c0 || c1 > p.num_tokens) raise_flag(p.flags, kFlagContextLen);
    if (tok < c0 || tok >= c1 || c0 < 0 || c1 > p.num_tokens) return;
    int32_t n = c1 - c0;
    const int h = qh / p.group;
    KvRows kv;
    kv.table = nullptr;
    kv.flags = p.flags;
    kv.head = h; kv.hkv = p.num_kv_heads; kv.bs = p.block_size; kv.num_blocks = p.num_blocks;
    kv.row_bytes = FP8 ? D : 2 * D;
    if (p.block_table) {
        n = __ldg(p.context_lens + a);
        const int32_t cap = p.max_blocks_per_seq * p.block_size;
        if (n < 0 || n > cap) {
            raise_flag(p.flags, kFlagContextLen);
            n = n < 0 ? 0 : cap;
        }
        kv.table = p.block_table + static_cast<int64_t>(a) * p.max_blocks_per_seq;
        kv.k = static_cast<const uint8_t *>(p.k);
        kv.v = static_cast<const uint8_t *>(p.v);
    } else {
        kv.k_stride = p.k_stride * 2;
        kv.v_stride = p.v_stride * 2;
        kv.k = static_cast<const uint8_t *>(p.k) + c0 * kv.k_stride + h * D * 2;
        kv.v = static_cast<const uint8_t *>(p.v) + c0 * kv.v_stride + h * D * 2;
    }
    const int32_t hi = n - (c1 - c0) + (tok - c0) + 1;
    const int32_t lo = p.window > 0 ? max(0, hi - p.window) : 0;
    const float sl2 = p.scale * 1.4426950408889634f * (FP8 ? __ldg(p.k_scale + h) : 1.f);
    float acc[E], m, l;
    attend_row<D, FP8>(p.q + tok * p.q_stride + qh * D, kv, lo, hi, sl2, acc, m, l);
    const float inv = l == 0.f ? 0.f : (FP8 ? __ldg(p.v_scale + h) : 1.f) / l;
    uint32_t *out = reinterpret_cast<uint32_t *>(p.out + row * D) + lane * (E / 2);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) out[i] = pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    if (p.lse_out && lane == 0)
        p.lse_out[row] = l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

cudaError_t launch_prefill(const PrefillLaunch &a) {
    const int64_t rows = static_cast<int64_t>(a.p.num_tokens) * a.p.num_q_heads;
    const unsigned grid = static_cast<unsigned>((rows + kRowWarps - 1) / kRowWarps);
    auto kernel = a.p.fp8 ? prefill_rows_kernel<128, true>
                          : a.p.head_dim == 128 ? prefill_rows_kernel<128, false>
                                                : prefill_rows_kernel<256, false>;
    kernel<<<grid, 32 * kRowWarps, 0, a.stream>>>(a.p);
    return cudaGetLastError();
}

}  // namespace pgd
