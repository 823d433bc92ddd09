// pgd_prefill_rows.cuh -- single rows of V, read by one warp.
#pragma once

#include "pgd_prefill.h"
#include "pgd_ptx.cuh"

namespace pgd {

// The V rows of one (sequence, KV head), packed or in pages.
template <int D, bool FP8>
struct ValueRows {
    static constexpr int E = D / 32;          // elements of a lane
    const PrefillParams &p;
    const uint8_t *base;
    const int32_t *table;
    int h;

    __device__ ValueRows(const PrefillParams &p_, int seq, int h_, int kv0)
        : p(p_), base(static_cast<const uint8_t *>(p_.v)), table(nullptr), h(h_) {
        if (p.block_table) table = p.block_table + static_cast<int64_t>(seq) * p.max_blocks_per_seq;
        else base += (kv0 * p.v_stride + static_cast<int64_t>(h) * D) * 2;
    }

    // Elements lane * E ... of position t as fp32 (an FP8 cache's without its
    // scale); whether one of them is not finite.
    __device__ __forceinline__ bool load(int t, float (&x)[E]) const {
        const uint8_t *row;
        if (table) {
            int b = __ldg(table + t / p.block_size);
            if (b < 0 || b >= p.num_blocks) {
                raise_flag(p.flags, kFlagBlockId);
                b = 0;
            }
            const int64_t r = (static_cast<int64_t>(b) * p.num_kv_heads + h) * p.block_size +
                              t % p.block_size;
            row = base + r * (FP8 ? D : 2 * D);
        } else {
            row = base + t * p.v_stride * 2;
        }
        const int lane = threadIdx.x & 31;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            float2 a, b;
            if (FP8) {
                const uint32_t w = reinterpret_cast<const uint32_t *>(row)[lane * (E / 4) + i / 4];
                a = unpack_f16x2(e4m3x2_to_f16x2(w & 0xFFFFu));
                b = unpack_f16x2(e4m3x2_to_f16x2(w >> 16));
            } else {
                const uint2 w = reinterpret_cast<const uint2 *>(row)[lane * (E / 4) + i / 4];
                a = unpack_bf16x2(w.x);
                b = unpack_bf16x2(w.y);
            }
            x[i] = a.x; x[i + 1] = a.y; x[i + 2] = b.x; x[i + 3] = b.y;
#pragma unroll
            for (int k = i; k < i + 4; ++k) bad |= !(fabsf(x[k]) < INFINITY);
        }
        return bad;
    }
};

}  // namespace pgd
