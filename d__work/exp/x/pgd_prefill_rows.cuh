// pgd_prefill_rows.cuh -- prompt attention of one query row by one warp, from
// the definition: the form that is right for every input.
#pragma once

#include "pgd_prefill.h"
#include "pgd_ptx.cuh"

namespace pgd {

// Where the K/V rows of one (sequence, KV head) are.
struct KvRows {
    const uint8_t *k, *v;         // packed: row 0 of the head; paged: the caches
    const int32_t *table;         // paged: the sequence's block ids
    int64_t k_stride, v_stride;   // packed: bytes between tokens
    int32_t head, hkv, bs, num_blocks, row_bytes;
    uint32_t *flags;

    __device__ __forceinline__ int64_t paged_row(int32_t t) const {
        int32_t b = __ldg(table + t / bs);
        if (b < 0 || b >= num_blocks) {
            raise_flag(flags, kFlagBlockId);
            b = 0;
        }
        return (static_cast<int64_t>(b) * hkv + head) * bs + t % bs;
    }
    __device__ __forceinline__ const uint8_t *k_row(int32_t t) const {
        return table ? k + paged_row(t) * row_bytes : k + t * k_stride;
    }
    __device__ __forceinline__ const uint8_t *v_row(int32_t t) const {
        return table ? v + paged_row(t) * row_bytes : v + t * v_stride;
    }
};

// E elements of a row, from element lane * E, as fp32.
template <int E, bool FP8>
__device__ __forceinline__ void load_elems(const uint8_t *row, int lane, float (&x)[E]) {
    if (FP8) {
        const uint32_t *s = reinterpret_cast<const uint32_t *>(row) + lane * (E / 4);
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            const uint32_t w = s[i];
            const float2 a = unpack_f16x2(e4m3x2_to_f16x2(w & 0xFFFFu));
            const float2 b = unpack_f16x2(e4m3x2_to_f16x2(w >> 16));
            x[4 * i] = a.x; x[4 * i + 1] = a.y; x[4 * i + 2] = b.x; x[4 * i + 3] = b.y;
        }
    } else {
        const uint2 *s = reinterpret_cast<const uint2 *>(row) + lane * (E / 4);
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            const uint2 w = s[i];
            const float2 a = unpack_bf16x2(w.x), b = unpack_bf16x2(w.y);
            x[4 * i] = a.x; x[4 * i + 1] = a.y; x[4 * i + 2] = b.x; x[4 * i + 3] = b.y;
        }
    }
}

// Online softmax of one row over keys [lo, hi) by one warp, in fp32; lane
// holds elements lane * D/32 ...  Leaves the unnormalised sum in acc, the
// weights' sum in l and the reference (log2 domain) in m.
template <int D, bool FP8>
__device__ void attend_row(const uint16_t *q_row, const KvRows &kv, int32_t lo, int32_t hi,
                           float scale_log2, float (&acc)[D / 32], float &m, float &l) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    float q[E];
    load_elems<E, false>(reinterpret_cast<const uint8_t *>(q_row), lane, q);
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.f;
    for (int32_t t = lo; t < hi; ++t) {
        float x[E];
        load_elems<E, FP8>(kv.k_row(t), lane, x);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) s += q[i] * x[i];
#pragma unroll
        for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= scale_log2;
        const float mn = fmaxf(m, s);
        // -inf - -inf: nothing weighs yet
        const float c = m == mn ? 1.f : ex2(m - mn);
        const float w = s == -INFINITY ? 0.f : ex2(s - mn);
        m = mn;
        l = l * c + w;
        load_elems<E, FP8>(kv.v_row(t), lane, x);
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = acc[i] * c + w * x[i];
    }
}

}  // namespace pgd
