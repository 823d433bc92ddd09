// pgd_prefill.cu -- launches of prompt attention, and the merge of cut units.
#include "pgd_prefill.cuh"

namespace pgd {

// Merge of the units that share boundaries cut.  The boundary where CTA c
// starts names a unit if it is the first one inside it; the unit's pieces are
// then the second slot of CTA c - 1 and the first slots of CTAs c, c + 1, ...
// as long as their starts lie inside the same unit.  Every block lists those
// units from the records, and the units' query rows are dealt to all warps, R
// at a time:
//   out = sum_j exp(lse_j - M) o_j / sum_j exp(lse_j - M),  M = max_j lse_j
// Latency bounds it: one round of loads for the list, and one for up to U
// pieces of R rows, all issued before the first is used.  Two rows, two pieces
// and 32 warps an SM were the best of R = 1 .. 4, U = 1 .. 4 and 16 .. 64
// warps (a mixed step: 107 us in all, 112 with R = U = 4).
constexpr int kMergeWarps = 16;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps, 2) prefill_merge_kernel(const PrefillParams p,
                                                                         int grid) {
    constexpr int ROWS = D == 128 ? 256 : 128, E4 = D / 128, R = 2 / E4, U = 2;
    constexpr int T = 32 * kMergeWarps;
    // per boundary: the key tile that it cuts at, and whether the one before
    // lies inside the same unit; per unit: its first chunk, boundary and rows
    __shared__ int cut_at[kMaxPrefillCtas + 1];
    __shared__ int first_chunk[kMaxPrefillCtas];
    __shared__ short first_cta[kMaxPrefillCtas];
    __shared__ int4 rows_of[kMaxPrefillCtas];       // row0, ntok, h, tiles
    __shared__ int warp_units[kMergeWarps], warp_chunks[kMergeWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int units = 0, chunks = 0;
    for (int x0 = 1; x0 <= grid; x0 += T) {
        const int x = x0 + threadIdx.x;
        int4 q0 = make_int4(0, 0, 0, 0), q1 = q0, b0 = q0;
        if (x < grid) {
            const int4 *q = reinterpret_cast<const int4 *>(p.parts + x);
            q0 = q[0];                               // unit, cut, tiles
            q1 = q[1];                               // row0, ntok, h
            b0 = *reinterpret_cast<const int4 *>(p.parts + x - 1);
        }
        const bool same = b0.z > 0 && b0.x == q0.x && b0.y == q0.y;
        const bool head = q0.z > 0 && !same;
        const int mine = head ? (q1.y * p.group + R - 1) / R : 0;
        int incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        const unsigned heads = __ballot_sync(0xffffffffu, head);
        __syncthreads();
        if (lane == 31) {
            warp_units[warp] = __popc(heads);
            warp_chunks[warp] = incl;
        }
        __syncthreads();
        int u = units + __popc(heads & ((1u << lane) - 1)), at = chunks + incl - mine;
        for (int w = 0; w < kMergeWarps; ++w) {
            if (w < warp) {
                u += warp_units[w];
                at += warp_chunks[w];
            }
            units += warp_units[w];
            chunks += warp_chunks[w];
        }
        if (head) {
            first_chunk[u] = at;
            first_cta[u] = static_cast<short>(x);
            rows_of[u] = make_int4(q1.x, q1.y, q1.z, q0.w);
        }
        // a continuation is marked by its cut, a head by minus its cut
        if (x <= grid) cut_at[x] = head ? -q0.z : q0.z > 0 ? q0.z : 0;
    }
    __syncthreads();
    const int tpq = 128 / p.group;
    for (int chunk = blockIdx.x * kMergeWarps + warp; chunk < chunks;
         chunk += gridDim.x * kMergeWarps) {
        int a = 0, b = units;                      // the unit of this chunk
        while (b - a > 1) {
            const int mid = (a + b) / 2;
            if (first_chunk[mid] <= chunk) a = mid;
            else b = mid;
        }
        const int c = first_cta[a], i0 = (chunk - first_chunk[a]) * R;
        const int4 unit = rows_of[a];
        const int n = unit.y * p.group;
        int row[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int i = i0 + q, tok = i / p.group;
            row[q] = i < n ? tok / tpq * 128 + (tok % tpq) * p.group + (i - tok * p.group) : -1;
        }
        float m[R], l[R];
        float4 acc[R][E4];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            m[q] = -INFINITY;
            l[q] = 0.f;
#pragma unroll
            for (int k = 0; k < E4; ++k) acc[q][k] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        int start = 0, slot = 2 * (c - 1) + 1, x = c;  // the next piece: [start, cut of x)
        bool more = true;
        while (more) {
            float lse[U][R];
            float4 o[U][R][E4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // the head's cut ends the first piece, a continuation's the others
                const int mark = x == c ? -cut_at[x] : cut_at[x];
                const int end = mark > 0 ? mark : unit.w;
                const bool live = more && end > start;
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    lse[u][q] = -INFINITY;
                    if (live && row[q] >= 0) {
                        const int64_t pr = static_cast<int64_t>(slot) * ROWS + row[q];
                        lse[u][q] = p.lse_part[pr];
#pragma unroll
                        for (int k = 0; k < E4; ++k)
                            o[u][q][k] = *reinterpret_cast<const float4 *>(
                                p.o_part + pr * D + k * 128 + lane * 4);
                    }
                }
                if (mark <= 0) more = false;
                if (more) {
                    start = end;
                    slot = 2 * x;
                    ++x;
                }
            }
#pragma unroll
            for (int q = 0; q < R; ++q) {
                float top = m[q];
#pragma unroll
                for (int u = 0; u < U; ++u) top = fmaxf(top, lse[u][q]);
                const float old = m[q] == -INFINITY ? 0.f : expf(m[q] - top);
                m[q] = top;
                l[q] *= old;
#pragma unroll
                for (int k = 0; k < E4; ++k) {
                    acc[q][k].x *= old; acc[q][k].y *= old; acc[q][k].z *= old; acc[q][k].w *= old;
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    // a NaN or +inf moves no maximum and stays in the sums
                    if (lse[u][q] == -INFINITY) continue;
                    const float w = expf(lse[u][q] - top);
                    l[q] += w;
#pragma unroll
                    for (int k = 0; k < E4; ++k) {
                        acc[q][k].x += w * o[u][q][k].x; acc[q][k].y += w * o[u][q][k].y;
                        acc[q][k].z += w * o[u][q][k].z; acc[q][k].w += w * o[u][q][k].w;
                    }
                }
            }
        }
#pragma unroll
        for (int q = 0; q < R; ++q) {
            if (row[q] < 0) continue;
            const float inv = l[q] == 0.f ? 0.f : 1.f / l[q];
            const int i = i0 + q, tok = i / p.group;
            const int64_t orow = static_cast<int64_t>(unit.x + tok) * p.num_q_heads +
                                 unit.z * p.group + (i - tok * p.group);
#pragma unroll
            for (int k = 0; k < E4; ++k)
                *reinterpret_cast<uint2 *>(p.out + orow * D + k * 128 + lane * 4) =
                    make_uint2(pack_bf16x2(acc[q][k].x * inv, acc[q][k].y * inv),
                               pack_bf16x2(acc[q][k].z * inv, acc[q][k].w * inv));
            if (p.lse_out && lane == 0)
                p.lse_out[orow] = l[q] == 0.f ? -INFINITY : m[q] + logf(l[q]);
        }
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
    cfg.gridDim = dim3(a.sms * 2);
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
