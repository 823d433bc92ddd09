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
// Instruction issue bounded the first forms (a warp's lanes all computed every
// row's weights and addresses: 300 instructions a row, 0.7 of the issue slots,
// 12 us behind a mixed step); here lane r * PB + j has row r's weight of piece
// j, and all lanes load and add 16 bytes of each row.  By itself and with cold
// caches 11.9 us there (0.4 of the issue slots, waiting for loads), 9.3 us of
// the step.
constexpr int kMergeWarps = 16;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps, 2) prefill_merge_kernel(const PrefillParams p,
                                                                         int grid) {
    constexpr int ROWS = D == 128 ? 256 : 128, E4 = D / 128, R = D == 128 ? 4 : 1, PB = 32 / R;
    constexpr int T = 32 * kMergeWarps;
    // per boundary: the key tile that it cuts at, and whether the one before
    // lies inside the same unit; per unit: its first chunk, boundary and rows
    __shared__ int cut_at[kMaxPrefillCtas + 1];
    __shared__ int first_chunk[kMaxPrefillCtas];
    __shared__ short first_cta[kMaxPrefillCtas], pieces_of[kMaxPrefillCtas];
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
    for (int u = threadIdx.x; u < units; u += T) {
        int x = first_cta[u] + 1;
        while (cut_at[x] > 0) ++x;                 // cut_at[grid] is no continuation
        pieces_of[u] = static_cast<short>(x - first_cta[u] + 1);
    }
    __syncthreads();
    const int tpq = 128 / p.group, r = lane / PB, q = lane % PB;
    for (int chunk = blockIdx.x * kMergeWarps + warp; chunk < chunks;
         chunk += gridDim.x * kMergeWarps) {
        int a = 0, b = units;                      // the unit of this chunk
        while (b - a > 1) {
            const int mid = (a + b) / 2;
            if (first_chunk[mid] <= chunk) a = mid;
            else b = mid;
        }
        const int c = first_cta[a], count = pieces_of[a];
        const int4 unit = rows_of[a];
        // the lane's row: of the workspace's slots, and of the output
        const int i = (chunk - first_chunk[a]) * R + r, tok = i / p.group, hd = i - tok * p.group;
        const bool on = i < unit.y * p.group;
        const int tile = tok / tpq, row = tile * 128 + (tok - tile * tpq) * p.group + hd;
        const int64_t orow = static_cast<int64_t>(unit.x + tok) * p.num_q_heads + unit.z * p.group + hd;
        float m = -INFINITY, l = 0.f;
        float4 acc[R][E4];
#pragma unroll
        for (int k = 0; k < R * E4; ++k) acc[k / E4][k % E4] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j0 = 0; j0 < count; j0 += PB) {
            // piece j: the first ends at the head's cut, the others start at
            // CTA c + j - 1's and end at the next one's, the last with the unit
            const int j = j0 + q;
            const int start = j == 0 || j >= count ? 0 : j == 1 ? -cut_at[c] : cut_at[c + j - 1];
            const int end = j >= count ? 0 : j + 1 == count ? unit.w : j == 0 ? -cut_at[c] : cut_at[c + j];
            const int slot = j == 0 ? 2 * (c - 1) + 1 : 2 * (c + j - 1);
            const bool live = end > start;
            const float lse = live && on ? p.lse_part[static_cast<int64_t>(slot) * ROWS + row] : -INFINITY;
            float top = lse;
#pragma unroll
            for (int off = PB / 2; off; off >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            top = fmaxf(top, m);
            const float old = m == -INFINITY ? 0.f : expf(m - top);
            // a NaN or +inf moves no maximum and stays in the sums
            const float w = lse == -INFINITY ? 0.f : expf(lse - top);
            m = top;
            float sum = w;
#pragma unroll
            for (int off = PB / 2; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            l = l * old + sum;
            if (j0 > 0) {
#pragma unroll
                for (int z = 0; z < R; ++z) {
                    const float f = __shfl_sync(0xffffffffu, old, z * PB);
#pragma unroll
                    for (int k = 0; k < E4; ++k) {
                        acc[z][k].x *= f; acc[z][k].y *= f; acc[z][k].z *= f; acc[z][k].w *= f;
                    }
                }
            }
            unsigned left = __ballot_sync(0xffffffffu, live) & (0xffffffffu >> (32 - PB));
            while (left) {
                const int at = __ffs(left) - 1;
                left &= left - 1;
                const float *src = p.o_part +
                    static_cast<int64_t>(__shfl_sync(0xffffffffu, slot, at)) * (ROWS * D) + lane * 4;
                float4 o[R][E4];
#pragma unroll
                for (int z = 0; z < R; ++z) {
                    const int rz = __shfl_sync(0xffffffffu, on ? row : -1, z * PB);
#pragma unroll
                    for (int k = 0; k < E4; ++k) {
                        o[z][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (rz >= 0) o[z][k] = *reinterpret_cast<const float4 *>(src + rz * D + k * 128);
                    }
                }
#pragma unroll
                for (int z = 0; z < R; ++z) {
                    // also for a weight of zero: a piece that is not finite stays so
                    const float f = __shfl_sync(0xffffffffu, w, z * PB + at);
#pragma unroll
                    for (int k = 0; k < E4; ++k) {
                        acc[z][k].x += f * o[z][k].x; acc[z][k].y += f * o[z][k].y;
                        acc[z][k].z += f * o[z][k].z; acc[z][k].w += f * o[z][k].w;
                    }
                }
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int z = 0; z < R; ++z) {
            const float f = __shfl_sync(0xffffffffu, inv, z * PB);
            const int64_t to = __shfl_sync(0xffffffffu, on ? orow : -1ll, z * PB);
            if (to < 0) continue;
#pragma unroll
            for (int k = 0; k < E4; ++k)
                *reinterpret_cast<uint2 *>(p.out + to * D + k * 128 + lane * 4) =
                    make_uint2(pack_bf16x2(acc[z][k].x * f, acc[z][k].y * f),
                               pack_bf16x2(acc[z][k].z * f, acc[z][k].w * f));
        }
        if (p.lse_out && on && q == 0) p.lse_out[orow] = l == 0.f ? -INFINITY : m + logf(l);
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
