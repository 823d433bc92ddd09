// pgd_prefill.cu -- launches of prompt attention, and the merge of cut units.
#include "pgd_prefill.cuh"

namespace pgd {

// Merge of the units that share boundaries cut.  Block (c - 1, y) looks at the
// boundary where CTA c starts: if it is the first one inside its unit, the
// unit's pieces are the second slot of CTA c - 1 and the first slots of CTAs
// c, c + 1, ... as long as their starts lie inside the same unit.  One warp
// per query row:
//   out = sum_j exp(lse_j - M) o_j / sum_j exp(lse_j - M),  M = max_j lse_j
constexpr int kMergeWarps = 8;
constexpr int kMergeSplit = 8;       // blocks per boundary

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) prefill_merge_kernel(const PrefillParams p,
                                                                         int grid) {
    constexpr int ROWS = D == 128 ? 256 : 128, E = D / 32;
    const int c = blockIdx.x + 1, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PartRecord r = p.parts[c];
    if (r.cut == 0) return;
    const PartRecord before = p.parts[c - 1];
    if (before.cut > 0 && before.unit == r.unit) return;
    const int tpq = 128 / p.group, n = r.ntok * p.group;
    for (int i = blockIdx.y * kMergeWarps + (threadIdx.x >> 5); i < n;
         i += kMergeSplit * kMergeWarps) {
        const int tok = i / p.group, hd = i - tok * p.group;
        const int row = tok / tpq * 128 + (tok % tpq) * p.group + hd;
        float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
        for (int k = 0; k < E; ++k) acc[k] = 0.f;
        int slot = 2 * (c - 1) + 1, cut = 0;
        for (int j = c;; ++j) {
            // the piece that ends where CTA j starts, or with the unit
            int next = r.tiles;
            bool last = true;
            if (j < grid) {
                const int4 x = *reinterpret_cast<const int4 *>(p.parts + j);
                const long long unit = static_cast<long long>(static_cast<uint32_t>(x.x)) |
                                       (static_cast<long long>(x.y) << 32);
                if (x.z > 0 && unit == r.unit) {
                    next = x.z;
                    last = false;
                }
            }
            if (next > cut) {
                const int64_t pr = static_cast<int64_t>(slot) * ROWS + row;
                const float lse = p.lse_part[pr];
                float o[E];
#pragma unroll
                for (int k = 0; k < E; k += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(
                        p.o_part + pr * D + k / 4 * 128 + lane * 4);
                    o[k] = x.x; o[k + 1] = x.y; o[k + 2] = x.z; o[k + 3] = x.w;
                }
                // NaN moves neither maximum nor branch, and stays in the sums
                if (lse != -INFINITY) {
                    const float mn = fmaxf(m, lse);
                    const float a = m == -INFINITY ? 0.f : expf(m - mn);
                    const float w = expf(lse - mn);
                    m = mn;
                    l = l * a + w;
#pragma unroll
                    for (int k = 0; k < E; ++k) acc[k] = acc[k] * a + w * o[k];
                }
            }
            if (last) break;
            cut = next;
            slot = 2 * j;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t orow = static_cast<int64_t>(r.row0 + tok) * p.num_q_heads + r.h * p.group + hd;
#pragma unroll
        for (int k = 0; k < E; k += 4)
            *reinterpret_cast<uint2 *>(p.out + orow * D + k / 4 * 128 + lane * 4) =
                make_uint2(pack_bf16x2(acc[k] * inv, acc[k + 1] * inv),
                           pack_bf16x2(acc[k + 2] * inv, acc[k + 3] * inv));
        if (p.lse_out && lane == 0) p.lse_out[orow] = l == 0.f ? -INFINITY : m + logf(l);
    }
}

template <int D, bool FP8>
static cudaError_t launch(const PrefillLaunch &a) {
    using C = PrefillCfg<D, FP8>;
    auto kernel = prefill_kernel<D, FP8>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    // the warpgroups' register shares must add up to what a CTA is launched with
    static const bool fits = [&] {
        cudaFuncAttributes f;
        return cudaFuncGetAttributes(&f, kernel) == cudaSuccess &&
               f.numRegs * C::THREADS >= C::SOFTMAX_REGS * 256 + C::OTHER_REGS * (C::THREADS - 256);
    }();
    if (!fits) return cudaErrorLaunchOutOfResources;
    const PrefillMaps maps = {a.map_q, a.map_k, a.map_v};
    kernel<<<a.grid, C::THREADS, C::SMEM, a.stream>>>(maps, a.p);
    e = cudaGetLastError();
    if (e != cudaSuccess || !a.p.parts || a.grid < 2) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.grid - 1, kMergeSplit);
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.stream = a.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefill_merge_kernel<D>, a.p, a.grid);
}

cudaError_t launch_prefill(const PrefillLaunch &a) {
    if (a.p.fp8) return launch<128, true>(a);
    return a.p.head_dim == 128 ? launch<128, false>(a) : launch<256, false>(a);
}

}  // namespace pgd
