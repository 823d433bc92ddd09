// pgd_rows.cu -- the FP8 cache's scales from K/V rows, and rows of a paged
// cache read back.
#include <algorithm>

#include "pgd_prefill.h"
#include "pgd_umma.cuh"

namespace pgd {

// ---------------------------------------------------------------- scales
// scale[h] = max(amax over tokens and elements of |x[t][h][d]| / 448, 2^-40),
// the amax over finite elements.  The absolute value of a bf16 is its low 15
// bits, which order like the values, so the maximum is taken on the bit
// patterns, two per register.  RN(x / 448) is monotone in x: the maximum of
// the quotients is the quotient of the maximum, and positive floats order
// like their bits, so CTAs join by an integer atomicMax whatever their order.
constexpr int kScaleThreads = 256;
constexpr float kMinScale = 0x1p-40f;

__global__ void kv_scales_init_kernel(float *k_scale, float *v_scale, int32_t hkv) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < hkv; i += gridDim.x * blockDim.x) {
        k_scale[i] = kMinScale;
        v_scale[i] = kMinScale;
    }
}

__device__ __forceinline__ uint32_t finite_abs_bf16x2(uint32_t x) {
    const uint32_t y = x & 0x7FFF7FFFu;
    const uint32_t nf = ((y + 0x00800080u) >> 15) & 0x00010001u;   // 1: not finite
    return y & ~(nf * 0xFFFFu);
}

__global__ void __launch_bounds__(kScaleThreads)
kv_quant_scales_kernel(const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new,
                       int32_t num_tokens, int32_t chunks, int32_t lg_head_chunks,
                       float *k_scale, float *v_scale) {
    // blockIdx.y: K or V; blockIdx.z: a group of kScaleThreads columns (16-byte
    // chunks of a token's row); rows narrower than the CTA take several tokens
    const uint4 *__restrict__ src = blockIdx.y ? v_new : k_new;
    const int per = min(chunks, kScaleThreads);
    const int rows = kScaleThreads / per;
    const int r = threadIdx.x / per;
    const int c = blockIdx.z * kScaleThreads + (threadIdx.x - r * per);
    const bool on = r < rows && c < chunks;
    uint32_t m = 0;
    if (on) {
        const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
#pragma unroll 4
        for (int64_t t = static_cast<int64_t>(blockIdx.x) * rows + r; t < num_tokens; t += step) {
            const uint4 x = __ldg(src + t * chunks + c);
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(finite_abs_bf16x2(x.x), finite_abs_bf16x2(x.y)),
                                     __vmaxu2(finite_abs_bf16x2(x.z), finite_abs_bf16x2(x.w))));
        }
    }
    uint32_t v = max(m & 0xFFFFu, m >> 16);
    // a head's chunks (16 or 32) sit in consecutive lanes
    const int width = 1 << lg_head_chunks;
    for (int off = width >> 1; off; off >>= 1)
        v = max(v, __shfl_xor_sync(0xffffffffu, v, off));
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the initialised scales
    if (on && (threadIdx.x & (width - 1)) == 0) {
        const float s = __fdiv_rn(__uint_as_float(v << 16), 448.f);
        atomicMax(reinterpret_cast<int *>((blockIdx.y ? v_scale : k_scale) + (c >> lg_head_chunks)),
                  __float_as_int(s));
    }
}

// Few rows: one CTA per head reads them all and writes its scale, in one
// launch and without atomics.
constexpr int kHeadThreads = 512;

__global__ void __launch_bounds__(kHeadThreads)
kv_head_scales_kernel(const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new,
                      int32_t num_tokens, int32_t chunks, int32_t lg_head_chunks, bool accumulate,
                      float *k_scale, float *v_scale) {
    __shared__ uint32_t warp_max[kHeadThreads / 32];
    const uint4 *__restrict__ src = (blockIdx.y ? v_new : k_new) +
                                    (static_cast<int64_t>(blockIdx.x) << lg_head_chunks) +
                                    (threadIdx.x & ((1 << lg_head_chunks) - 1));
    const int step = kHeadThreads >> lg_head_chunks;
    uint32_t m = 0;
#pragma unroll 8
    for (int t = threadIdx.x >> lg_head_chunks; t < num_tokens; t += step) {
        const uint4 x = __ldg(src + static_cast<int64_t>(t) * chunks);
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(finite_abs_bf16x2(x.x), finite_abs_bf16x2(x.y)),
                                 __vmaxu2(finite_abs_bf16x2(x.z), finite_abs_bf16x2(x.w))));
    }
    const uint32_t w = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = w;
    __syncthreads();
    if (threadIdx.x < 32) {
        const uint32_t v = __reduce_max_sync(
            0xffffffffu, threadIdx.x < kHeadThreads / 32 ? warp_max[threadIdx.x] : 0u);
        if (threadIdx.x == 0) {
            int *out = reinterpret_cast<int *>(blockIdx.y ? v_scale : k_scale) + blockIdx.x;
            const int s = __float_as_int(__fdiv_rn(__uint_as_float(v << 16), 448.f));
            *out = max(s, accumulate ? *out : __float_as_int(kMinScale));
        }
    }
}

// Rows up to which one CTA per head is taken: 200 rows of 8 heads of 128 take
// 3.0 us and one launch, against 3.2 us and two; 1024 rows of 2 heads of 256
// already 8.8 us against 5.4.
constexpr int kHeadTokens = 256;

cudaError_t launch_kv_quant_scales(const void *k_new, const void *v_new, int32_t num_tokens,
                                   int32_t hkv, int32_t head_dim, bool accumulate, float *k_scale,
                                   float *v_scale, int sms, cudaStream_t stream) {
    const int lg_head_chunks = head_dim == 128 ? 4 : 5;
    if (num_tokens <= kHeadTokens && (num_tokens > 0 || !accumulate)) {
        kv_head_scales_kernel<<<dim3(hkv, 2), kHeadThreads, 0, stream>>>(
            static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new), num_tokens,
            hkv * (head_dim / 8), lg_head_chunks, accumulate, k_scale, v_scale);
        return cudaGetLastError();
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    if (!accumulate) {
        kv_scales_init_kernel<<<(hkv + 255) / 256, 256, 0, stream>>>(k_scale, v_scale, hkv);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    if (num_tokens == 0) return cudaSuccess;
    const int chunks = hkv * (head_dim / 8);
    const int groups = (chunks + kScaleThreads - 1) / kScaleThreads;
    const int rows = chunks >= kScaleThreads ? 1 : kScaleThreads / chunks;
    const long long passes = (static_cast<long long>(num_tokens) + rows - 1) / rows;
    const long long want = (static_cast<long long>(sms) * 8 + 2 * groups - 1) / (2 * groups);
    cfg.gridDim = dim3(static_cast<unsigned>(passes < want ? passes : want), 2, groups);
    cfg.blockDim = dim3(kScaleThreads);
    return cudaLaunchKernelEx(&cfg, kv_quant_scales_kernel, static_cast<const uint4 *>(k_new),
                              static_cast<const uint4 *>(v_new), num_tokens, chunks,
                              lg_head_chunks, k_scale, v_scale);
}

// ---------------------------------------------------------------- gather
// Row t of the outputs = row slot % bs of block slot / bs, as bf16: bf16 rows
// are copied, E4M3 rows are the fp32 product e4m3 * scale[h] rounded to
// nearest even.  One thread per 16-byte cache chunk; a CTA takes as many tokens
// as give each thread kGatherLoads chunks, loaded together: memory bounds it
// (65536 tokens of 8 heads of 128: 85 us, 0.96 of the measured copy bandwidth,
// where one token a CTA took 93 us).
constexpr int kGatherThreads = 256;
constexpr int kGatherLoads = 4;
constexpr int kGatherTokens = 64;                   // at most

template <bool FP8>
__global__ void __launch_bounds__(kGatherThreads)
kv_gather_kernel(const uint4 *__restrict__ k_cache, const uint4 *__restrict__ v_cache,
                 const int64_t *__restrict__ slots, int32_t num_tokens, uint4 *k_out, uint4 *v_out,
                 const float *__restrict__ k_scale, const float *__restrict__ v_scale,
                 int32_t hkv, int32_t lg_row, int32_t lg_bs, int64_t pool_slots, int32_t per,
                 bool out32, uint32_t *flags) {
    const int t0 = blockIdx.x * per;
    const int n = hkv << (lg_row + 1);              // chunks of a token, K and V
    __shared__ int64_t row0[kGatherTokens];         // its first cache row, -1: none
    if (threadIdx.x < per) {
        const int t = t0 + threadIdx.x;
        int64_t r = -1;
        if (t < num_tokens) {
            const int64_t slot = __ldg(slots + t);
            if (slot >= pool_slots) raise_flag(flags, kFlagSlot);
            else if (slot >= 0)                      // below: a padding token
                r = (((slot >> lg_bs) * hkv) << lg_bs) + (slot & ((1 << lg_bs) - 1));
        }
        row0[threadIdx.x] = r;
    }
    __syncthreads();
    constexpr int U = kGatherLoads;
    for (int i0 = threadIdx.x; i0 < n * per; i0 += kGatherThreads * U) {
        uint4 x[U];
        int tok[U], at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kGatherThreads;
            tok[u] = i / n;
            at[u] = i - tok[u] * n;
            const int64_t r = i < n * per ? row0[tok[u]] : -1;
            if (r < 0) {
                tok[u] = -1;
                continue;
            }
            const int h = at[u] >> (lg_row + 1), c = at[u] & ((1 << lg_row) - 1);
            const bool isk = !((at[u] >> lg_row) & 1);
            x[u] = __ldg((isk ? k_cache : v_cache) +
                         ((r + (static_cast<int64_t>(h) << lg_bs)) << lg_row) + c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (tok[u] < 0) continue;
            const int h = at[u] >> (lg_row + 1), c = at[u] & ((1 << lg_row) - 1);
            const bool isk = !((at[u] >> lg_row) & 1);
            const int64_t dst = ((static_cast<int64_t>(t0 + tok[u]) * hkv + h) << lg_row) + c;
            uint4 *out = isk ? k_out : v_out;
            if (!FP8) {
                out[dst] = x[u];
            } else {
                const float s = __ldg((isk ? k_scale : v_scale) + h);
                const uint32_t in[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                uint32_t o[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 a = unpack_f16x2(e4m3x2_to_f16x2(in[k] & 0xFFFFu));
                    const float2 b = unpack_f16x2(e4m3x2_to_f16x2(in[k] >> 16));
                    o[2 * k] = pack_bf16x2(a.x * s, a.y * s);
                    o[2 * k + 1] = pack_bf16x2(b.x * s, b.y * s);
                }
                if (out32) {
                    store32(out + 2 * dst, o);
                } else {
                    out[2 * dst] = make_uint4(o[0], o[1], o[2], o[3]);
                    out[2 * dst + 1] = make_uint4(o[4], o[5], o[6], o[7]);
                }
            }
        }
    }
}

cudaError_t launch_kv_gather(const void *k_cache, const void *v_cache, const int64_t *slots,
                             int32_t num_tokens, void *k_out, void *v_out, int32_t hkv,
                             int32_t head_dim, int32_t block_size, int64_t pool_slots, bool fp8,
                             const float *k_scale, const float *v_scale, uint32_t *flags,
                             int sms, cudaStream_t stream) {
    if (num_tokens == 0) return cudaSuccess;
    int lg_row = fp8 ? 3 : 4, lg_bs = block_size == 16 ? 4 : block_size == 32 ? 5 : 6;
    if (head_dim == 256) ++lg_row;
    auto kernel = fp8 ? kv_gather_kernel<true> : kv_gather_kernel<false>;
    // fewer tokens a CTA when there are few: about four CTAs an SM
    const int row = hkv << (lg_row + 1);
    int per = std::max(1, std::min(kGatherTokens, kGatherThreads * kGatherLoads / row));
    per = std::max(1, std::min(per, num_tokens / (4 * sms)));
    const bool out32 = (reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) % 32 == 0;
    kernel<<<static_cast<unsigned>((static_cast<int64_t>(num_tokens) + per - 1) / per),
             kGatherThreads, 0, stream>>>(
        static_cast<const uint4 *>(k_cache), static_cast<const uint4 *>(v_cache), slots,
        num_tokens, static_cast<uint4 *>(k_out), static_cast<uint4 *>(v_out), k_scale, v_scale, hkv, lg_row,
        lg_bs, pool_slots, per, out32, flags);
    return cudaGetLastError();
}

}  // namespace pgd
