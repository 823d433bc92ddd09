// pgd_rows.cu -- the FP8 cache's scales from K/V rows, and rows of a paged
// cache read back.
#include "pgd_prefill.h"
#include "pgd_ptx.cuh"

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

cudaError_t launch_kv_quant_scales(const void *k_new, const void *v_new, int32_t num_tokens,
                                   int32_t hkv, int32_t head_dim, bool accumulate, float *k_scale,
                                   float *v_scale, int sms, cudaStream_t stream) {
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
                              head_dim == 128 ? 4 : 5, k_scale, v_scale);
}

// ---------------------------------------------------------------- gather
// Row t of the outputs = row slot % bs of block slot / bs, as bf16: bf16 rows
// are copied, E4M3 rows are the fp32 product e4m3 * scale[h] rounded to
// nearest even.  One CTA per token, one thread per 16-byte cache chunk.
constexpr int kGatherThreads = 128;

template <bool FP8>
__global__ void __launch_bounds__(kGatherThreads)
kv_gather_kernel(const uint4 *__restrict__ k_cache, const uint4 *__restrict__ v_cache,
                 const int64_t *__restrict__ slots, uint4 *k_out, uint4 *v_out,
                 const float *__restrict__ k_scale, const float *__restrict__ v_scale,
                 int32_t hkv, int32_t lg_row, int32_t lg_bs, int64_t pool_slots,
                 uint32_t *flags) {
    const int t = blockIdx.x;
    const int64_t slot = __ldg(slots + t);
    if (slot < 0) return;                       // padding token
    if (slot >= pool_slots) {
        if (threadIdx.x == 0) raise_flag(flags, kFlagSlot);
        return;
    }
    const int64_t blk = slot >> lg_bs, off = slot & ((1 << lg_bs) - 1);
    const int n = hkv << (lg_row + 1);
    for (int i = threadIdx.x; i < n; i += kGatherThreads) {
        const int h = i >> (lg_row + 1), c = i & ((1 << lg_row) - 1);
        const bool isk = !((i >> lg_row) & 1);
        const int64_t src = ((((blk * hkv + h) << lg_bs) + off) << lg_row) + c;
        const int64_t dst = ((static_cast<int64_t>(t) * hkv + h) << lg_row) + c;
        const uint4 x = __ldg((isk ? k_cache : v_cache) + src);
        uint4 *out = isk ? k_out : v_out;
        if (!FP8) {
            out[dst] = x;
        } else {
            const float s = __ldg((isk ? k_scale : v_scale) + h);
            const uint32_t in[4] = {x.x, x.y, x.z, x.w};
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 a = unpack_f16x2(e4m3x2_to_f16x2(in[k] & 0xFFFFu));
                const float2 b = unpack_f16x2(e4m3x2_to_f16x2(in[k] >> 16));
                o[2 * k] = pack_bf16x2(a.x * s, a.y * s);
                o[2 * k + 1] = pack_bf16x2(b.x * s, b.y * s);
            }
            out[2 * dst] = make_uint4(o[0], o[1], o[2], o[3]);
            out[2 * dst + 1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

cudaError_t launch_kv_gather(const void *k_cache, const void *v_cache, const int64_t *slots,
                             int32_t num_tokens, void *k_out, void *v_out, int32_t hkv,
                             int32_t head_dim, int32_t block_size, int64_t pool_slots, bool fp8,
                             const float *k_scale, const float *v_scale, uint32_t *flags,
                             cudaStream_t stream) {
    if (num_tokens == 0) return cudaSuccess;
    int lg_row = fp8 ? 3 : 4, lg_bs = block_size == 16 ? 4 : block_size == 32 ? 5 : 6;
    if (head_dim == 256) ++lg_row;
    auto kernel = fp8 ? kv_gather_kernel<true> : kv_gather_kernel<false>;
    kernel<<<static_cast<unsigned>(num_tokens), kGatherThreads, 0, stream>>>(
        static_cast<const uint4 *>(k_cache), static_cast<const uint4 *>(v_cache), slots,
        static_cast<uint4 *>(k_out), static_cast<uint4 *>(v_out), k_scale, v_scale, hkv, lg_row,
        lg_bs, pool_slots, flags);
    return cudaGetLastError();
}

}  // namespace pgd
