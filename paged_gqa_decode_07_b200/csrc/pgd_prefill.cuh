// pgd_prefill.cuh -- prompt attention on the 5th-generation tensor cores.
//
// What it computes ("attention kernels", froggydisk: sections "standard
// attention", "FlashAttention", "paged KV and kernels"): for every query row
// (token i, head a) of every sequence
//     out = softmax(scale * q . K_t) V_t  over the visible positions t,
// causal, optionally the last `window` of them, K/V packed or in pages.
//
// Tiles.  A query tile is 128 rows of one KV head: the g heads of its group
// for 128 / g consecutive tokens, so K/V is read once per group and the causal
// diagonal is only 128 / g tokens wide.  A unit is NQ query tiles (2 at
// head_dim 128, 1 at 256) and all keys that they see; keys come in tiles of 128.
//
// Work.  Long contexts: the units of all sequences laid end to end, each as
// long as its keys plus a constant, are cut into one equal share per CTA
// (pgd_prefill_sched.cuh; short ones deal whole units in turn).
// A unit that a boundary cuts leaves one unrounded piece per CTA in the
// workspace; a second kernel merges them by log-sum-exp.
//
// CTA = 2 softmax warpgroups + single warps:
//   warps 0-3, 4-7   softmax; thread = query row (one TMEM lane)
//   warp 8           finds the share, hands its pieces out, and loads: Q and
//                    [128 keys x 128 dims] boxes of K and V into a ring (TMA)
//   warp 9           issues the tcgen05.mma of S = Q K^T and O += P V, the
//                    query tiles in turn (a warp for each let the tiles fall
//                    into step: both in softmax, then both at the tensor cores)
//   the last 2 or 4  keep masked keys out of V (below); for FP8 caches they
//                    also turn the E4M3 boxes and the query rows into f16
// S, P and O live in tensor memory (512 columns):
//   NQ = 2: S0 | S1 | O0 | O1, P_t in the columns of S_t.  One tile's softmax
//     runs while the other's products do, and S_t(j + 1) follows P_t(j) V(j)
//     in issue order, so S_t ready means O_t is at rest.
//   NQ = 1: S0 | S1 | O (256): S(j + 1) is formed while softmax(j) runs.
//
// Softmax, one pass with a running reference m and sum l in fp32: the weights
// are p = 2^(x - m), and m moves (O and l rescaled) only when a score exceeds
// it by more than 8 (weights stay below 2^8, O below 2^8 times its value).
// P enters the product as bf16 (f16 for FP8 caches, whose V is exact there):
// both operands have one type, and a second term for the lost bits would double
// the P V products.  l sums the unrounded weights.  f16 ends at 2^-25: there m
// is put 7 below the maximum, weights reach up to 2^15, and what rounds to zero
// is below 2^-32 of the largest (2^-25 before: n * 2^-25 of the result was lost
// behind one dominant key, with 262144 keys 2^-7).
//
// Masked keys.  A masked weight is zero, but zero times a value that is not
// finite is NaN, and rows of unowned slots may hold anything.  On key tiles
// that some row does not fully see, the V warps zero the rows no query of the
// unit sees before the product reads them, and in rows that only some queries
// see the elements that are not finite; where there was one, the softmax warps
// add those elements to O of the rows that see them (a weight is positive: an
// infinity stays itself, and NaN).  Such tiles are at most seven a unit (the
// diagonal of 256 tokens, and the window's edge), so this takes the same time
// behind any context, and what is added follows from the keys alone.
//
// What bounds it (148 SMs).  A step of two tiles takes the tensor cores 2048
// cycles and ex2 2048, and one tile's chain (softmax 2000 - 2400, products
// 1330) leaves both busy 0.55 - 0.6 of the time.  64 heads over 8, 8192 tokens:
// 975 - 1040 us by itself (1.06 - 1.13 PFLOP/s), 1120 - 1135 in calls one after
// another on changing inputs, at the power cap (992 W, 1.74 GHz), where plain
// matrix products sustain 1.39 PFLOP/s.  Every instruction of the MMA warp
// counts: descriptors built per product (18 instructions each by the code's
// size, 4 now), branches and 64-bit compares before a wait and conditions in
// the loop cost 5400 cycles a step, the straight form 3700.
//
// Tensor-memory loads and stores are warp-wide (.sync.aligned): between two of
// them lanes differ only by predicates and selects, or meet at a __syncwarp.
//
// Every wait is bounded (wait_ns): a role that gives up raises the timeout
// flag and leaves; the producer and the MMA warp then wait for what they have
// in flight, all warps meet, and tensor memory is freed.
#pragma once

#include "pgd_prefill_rows.cuh"
#include "pgd_prefill_sched.cuh"
#include "pgd_umma.cuh"

namespace pgd {

constexpr uint32_t kLine = 128 * 128;         // bytes of a line: 128 rows x 128 B
constexpr uint32_t kBox = 2 * kLine;          // [128 keys][128 dims], 16-bit
constexpr int kBadSlots = 8;                  // units that a mark can be ahead
constexpr uint32_t kMetaBytes = 1024;

// Warps 0-7 are the softmax warpgroups; an FP8 cache takes more warps to
// convert.  Registers: 8 x 184 + 4 x 136 = 12 x 168, 8 x 152 + 8 x 104 = 16 x 128.
template <int D, bool FP8>
struct PrefillCfg {
    static constexpr int THREADS = FP8 ? 512 : 384;
    static constexpr int SOFTMAX_REGS = FP8 ? 152 : 184, OTHER_REGS = FP8 ? 104 : 136;
    static constexpr int V_WARPS = FP8 ? 4 : 2;
    static constexpr int V_WARP0 = THREADS / 32 - V_WARPS;
    static_assert(SOFTMAX_REGS * 256 + OTHER_REGS * (THREADS - 256) <=
                  65536 / THREADS / 8 * 8 * THREADS, "registers of the launch");
    static constexpr int NQ = D == 128 ? 2 : 1;
    static constexpr int LINES = D / 64;              // lines of a Q tile
    static constexpr int BOXES = D / 128;             // boxes of a K or V tile
    static constexpr uint32_t QTILE = LINES * kLine;
    static constexpr int NS = 5;                      // ring of boxes
    static constexpr uint32_t OFF_RING = NQ * QTILE;
    static constexpr uint32_t OFF_META = OFF_RING + NS * kBox;
    static constexpr uint32_t SMEM = OFF_META + kMetaBytes + (FP8 ? 2048 : 0);
    static_assert(SMEM <= 232448, "more shared memory than a CTA has");
};

// Barriers and small state behind the tiles (for FP8, 2 x 256 multipliers of
// the query rows follow).
struct PrefillMeta {
    uint64_t q_full, q_ready, q_empty, drain, pv_done;
    uint64_t s_ready[2], p_ready[2][2], o_done[2];
    uint64_t full[5], empty[5], fixed[5];
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    Piece piece[kPieces];
    Share share;
    uint32_t tmem, bad[kBadSlots];   // units whose V had elements zeroed
};
static_assert(sizeof(PrefillMeta) <= kMetaBytes, "PrefillMeta grew");

struct PrefillMaps {
    CUtensorMap q, k, v;
};

// Whether some row of an active tile does not see all of key tile j (the
// tiles' ranges leave no gap).
__device__ __forceinline__ bool is_partial(const Piece &k, int j) {
    return j < k.part_lo || j >= k.part_hi;
}

// Fill in what each query tile of a piece sees (the producer, once a piece).
template <int NQ>
__device__ __forceinline__ void piece_keys(const PrefillParams &p, Piece &u, int tpq) {
    u.hi = u.pos0 + u.ntok;
    u.lo = first_seen(p, u.pos0);
    u.all_hi = u.pos0 + 1;
    u.all_lo = first_seen(p, u.hi - 1);
    u.part_lo = 0;
    u.part_hi = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        TileKeys &t = u.t[i];
        t.ntok = min(tpq, u.ntok - i * tpq);
        t.p0 = u.pos0 + i * tpq;
        t.kb = t.ke = t.mlo = t.mhi = 0;
        const int hi = t.p0 + t.ntok;
        if (t.ntok > 0 && hi > 0) {
            t.kb = max(first_seen(p, t.p0) / kKeys, u.kb);
            t.ke = max(t.kb, min((hi + kKeys - 1) / kKeys, u.ke));
            t.mlo = (first_seen(p, hi - 1) + kKeys - 1) / kKeys;
            t.mhi = max(0, t.p0 + 1) / kKeys;
            u.part_lo = max(u.part_lo, t.mlo);
            u.part_hi = min(u.part_hi, t.mhi);
        }
    }
}

// ---------------------------------------------------------------- the V warps
// Keep masked keys out of a 16-bit V box: zero the rows outside [lo, hi) of
// the tile's keys, and the non-finite elements of rows that only some query
// rows see, outside [all_lo, all_hi); tells whether there were any.  8 threads
// on one row's 128-byte line.
template <int WARPS>
__device__ __forceinline__ bool clean_box(uint32_t box, int lo, int hi, int all_lo, int all_hi,
                                          int tid) {
    bool bad = false;
    const uint32_t at = box + (tid & 7) * 16;
    const int r0 = tid >> 3;
    for (int r = r0; r < 128; r += WARPS * 4) {
        if (r >= all_lo && r < all_hi) continue;
        const uint32_t a = at + r * 128;
        if (r < lo || r >= hi) {
            sts128(a, 0, 0, 0, 0);
            sts128(a + kLine, 0, 0, 0, 0);
        } else {
            uint32_t x[8], any = 0;
            lds128(a, x[0], x[1], x[2], x[3]);
            lds128(a + kLine, x[4], x[5], x[6], x[7]);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t nf = ((x[k] & 0x7FFF7FFFu) + 0x00800080u) & 0x80008000u;
                any |= nf;
                x[k] &= ~((nf >> 15) * 0xFFFFu);
            }
            if (any) {
                sts128(a, x[0], x[1], x[2], x[3]);
                sts128(a + kLine, x[4], x[5], x[6], x[7]);
                bad = true;
            }
        }
    }
    return bad;
}

// The same for the E4M3 rows of a box that is not converted yet: rows outside
// [lo, hi) become zeros, and so do the NaN of the others (of rows that every
// query sees too: one test less).  A thread takes the bytes that convert_box
// has it read.
template <int WARPS>
__device__ __forceinline__ bool clean_bytes(uint32_t box, int lo, int hi, int tid) {
    bool bad = false;
#pragma unroll 1
    for (int r = tid >> 3; r < 128; r += WARPS * 4) {
        const uint32_t a = box + kLine + r * 128 + (((tid & 7) ^ (r & 7)) << 4);
        uint32_t x[4], any = 0;
        lds128(a, x[0], x[1], x[2], x[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t nan = ((x[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
            any |= nan;
            x[k] &= ~((nan >> 7) * 0xFFu);
        }
        if (r < lo || r >= hi) {
            sts128(a, 0, 0, 0, 0);
        } else if (any) {
            sts128(a, x[0], x[1], x[2], x[3]);
            bad = true;
        }
    }
    return bad;
}

// An E4M3 box to f16, in place: a row's 128 bytes lie where the second half of
// its 128 elements goes, and eight threads of one warp read the whole row
// before they write it.
template <int WARPS>
__device__ __forceinline__ void convert_box(uint32_t box, int tid) {
    constexpr int U = 4;
    const int c = tid & 7, f = c >> 2, o = (c & 3) * 2;
#pragma unroll 1
    for (int r0 = tid >> 3; r0 < 128; r0 += U * WARPS * 4) {
        uint32_t x[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * WARPS * 4;
            lds128(box + kLine + r * 128 + ((c ^ (r & 7)) << 4), x[u][0], x[u][1], x[u][2], x[u][3]);
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * WARPS * 4, sw = r & 7;
            uint32_t y[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                y[2 * k] = e4m3x2_to_f16x2(x[u][k] & 0xFFFFu);
                y[2 * k + 1] = e4m3x2_to_f16x2(x[u][k] >> 16);
            }
            // 16 elements: two chunks of line c / 4; lanes of the second line
            // write theirs in the other order, so that a row's eight lanes hit
            // eight different chunk positions
            const uint32_t row = box + f * kLine + r * 128;
            const uint32_t a0 = row + (((o + f) ^ sw) << 4), a1 = row + (((o + 1 - f) ^ sw) << 4);
            if (f) {
                sts128(a0, y[4], y[5], y[6], y[7]);
                sts128(a1, y[0], y[1], y[2], y[3]);
            } else {
                sts128(a0, y[0], y[1], y[2], y[3]);
                sts128(a1, y[4], y[5], y[6], y[7]);
            }
        }
    }
}

// A query row (eight threads of one warp, two 16-byte chunks each), bf16 ->
// f16 in place, multiplied by the power of two that brings its largest element
// to [2^14, 2^15): exact for every element within 2^-28 of it.  Returns the
// inverse power (1 for a row of zeros or one that is not finite).
__device__ __forceinline__ float convert_q_row(uint32_t tile, int r, int c) {
    const uint32_t a = tile + r * 128 + ((c ^ (r & 7)) << 4);
    uint32_t x[8], m = 0;
    lds128(a, x[0], x[1], x[2], x[3]);
    lds128(a + kLine, x[4], x[5], x[6], x[7]);
#pragma unroll
    for (int k = 0; k < 8; ++k) m = __vmaxu2(m, x[k] & 0x7FFF7FFFu);
#pragma unroll
    for (int off = 4; off; off >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
    const uint32_t top = max(m & 0xFFFFu, m >> 16);
    int e = static_cast<int>(top >> 7) - 127;            // floor(log2) of a normal
    if (top == 0 || top >= 0x7F80u) e = 14;
    if (e < -110) e = -110;                              // keep both powers normal
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float2 v = unpack_bf16x2(x[k]);
        x[k] = pack_f16x2(v.x * up, v.y * up);
    }
    sts128(a, x[0], x[1], x[2], x[3]);
    sts128(a + kLine, x[4], x[5], x[6], x[7]);
    return __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
}

// ---------------------------------------------------------------- softmax
// max(a, b, c), NaN if one is
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Add the elements of V that the V warps zeroed, in the key tiles of this piece,
// to O (at `o`) of the rows that see them; a row sees keys below `hi` (0: no
// row).  One warp, all lanes alike; lane holds elements lane * D / 32 ...
template <int D, bool FP8>
__device__ __forceinline__ void add_bad_values(const PrefillParams &p, const Piece &u,
                                               const TileKeys &tk, int hi, uint32_t o) {
    constexpr int E = D / 32;
    const ValueRows<D, FP8> rows(p, u.seq, u.h, u.kv0);
#pragma unroll 1
    for (int j = tk.kb; j < tk.ke; ++j) {
        if (!is_partial(u, j)) continue;
        const int end = min((j + 1) * kKeys, u.hi);
#pragma unroll 1
        for (int t = max(j * kKeys, u.lo); t < end; ++t) {
            if (!FP8 && t >= u.all_lo && t < u.all_hi) continue;
            float x[E];
            const bool bad = rows.load(t, x);
            const uint32_t found = __ballot_sync(0xffffffffu, bad);
            const bool sees = t < hi && (p.window == 0 || hi - t <= p.window);
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                if (!(found >> (c / E) & ((1u << 16 / E) - 1))) continue;
                uint32_t y[16];
                tmem_ld16(o + c, y);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    asm volatile("" : "+r"(y[i]));
                    const float v = __shfl_sync(0xffffffffu, x[i % E], c / E + i / E);
                    y[i] = sees && !(fabsf(v) < INFINITY)
                               ? __float_as_uint(__uint_as_float(y[i]) + v) : y[i];
                }
                tmem_st16(o + c, y);
                tmem_wait_st();
            }
        }
    }
}

// ---------------------------------------------------------------- the kernel
// A warp's wait for a phase, all lanes or none: false when `limit_ns` ran out
// (the timeout flag is raised).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                          uint32_t *flags) {
    // a try_wait may suspend the thread for a while; a shortened limit polls
    const bool poll = limit_ns < kDefaultWaitNs;
    uint64_t t0 = 0;
    while (!__all_sync(0xffffffffu, poll ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity))) {
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (__any_sync(0xffffffffu, now - t0 > limit_ns)) {
            raise_flag(flags, kFlagTimeout);
            return false;
        }
    }
    return true;
}

// The same where a phase is often over (50 cycles then).
__device__ __forceinline__ bool warp_wait_soon(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                               uint32_t *flags) {
    return __all_sync(0xffffffffu, mbar_test_wait(bar, parity)) ||
           warp_wait(bar, parity, limit_ns, flags);
}

template <int D, bool FP8>
__global__ void __launch_bounds__((PrefillCfg<D, FP8>::THREADS), 1)
prefill_kernel(const __grid_constant__ PrefillMaps maps, const PrefillParams p) {
    using C = PrefillCfg<D, FP8>;
    constexpr int NQ = C::NQ;
    extern __shared__ __align__(1024) uint8_t smem_al[];
    const uint32_t smem = smem_u32(smem_al);
    if (smem & 1023) {                           // the swizzled boxes start on 1024 bytes
        if (threadIdx.x == 0) raise_flag(p.flags, kFlagTimeout);
        return;
    }
    PrefillMeta &meta = *reinterpret_cast<PrefillMeta *>(smem_al + C::OFF_META);
    float *row_mult = reinterpret_cast<float *>(smem_al + C::OFF_META + kMetaBytes);
    const uint32_t ring = smem + C::OFF_RING;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const auto bar = [](uint64_t &b) { return smem_u32(&b); };

    if (threadIdx.x == 0) {
        mbar_init(bar(meta.q_full), 1);
        mbar_init(bar(meta.q_ready), C::V_WARPS);
        mbar_init(bar(meta.q_empty), 1);
        mbar_init(bar(meta.drain), 1);
        mbar_init(bar(meta.pv_done), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(meta.s_ready[i]), 1);
            mbar_init(bar(meta.p_ready[i][0]), 4);
            mbar_init(bar(meta.p_ready[i][1]), 4);
            mbar_init(bar(meta.o_done[i]), 1);
        }
        for (int i = 0; i < 5; ++i) {
            // filled by TMA; an FP8 box goes through the V warps before the
            // MMA warp takes it, a bf16 box is looked at by both
            mbar_init(bar(meta.full[i]), 1);
            mbar_init(bar(meta.empty[i]), FP8 ? 1 : 1 + C::V_WARPS);
            mbar_init(bar(meta.fixed[i]), C::V_WARPS);
        }
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(bar(meta.piece_full[i]), 1);
            mbar_init(bar(meta.piece_empty[i]), 1 + 4 * NQ + C::V_WARPS);   // MMA, softmax, V warps
        }
        for (int i = 0; i < kBadSlots; ++i) meta.bad[i] = 0;
        fence_mbar_init();
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
    }
    if (warp == 9) tmem_alloc(smem_u32(&meta.tmem), 512);
    if (p.parts) find_share<NQ, C::THREADS>(p, meta.share);   // all threads meet in it
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    constexpr uint32_t tmem = 0;                 // all 512 columns start at the first
    constexpr uint32_t kOCol = 256;              // O_t at kOCol + t * 128
    const int tpq = 128 / p.group;
    const uint64_t limit = p.wait_ns;
    int piece = 0;

    // the merge may be placed on SMs that this grid leaves; it waits for the end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const auto wait = [&](uint64_t &b, uint32_t parity) {
        return warp_wait(smem_u32(&b), parity, limit, p.flags);
    };
    // the next piece handed out by the producer; false at the end
    const auto next_piece = [&]() {
        return wait(meta.piece_full[piece % kPieces], (piece / kPieces) & 1) &&
               meta.piece[piece % kPieces].ntok > 0;
    };
    const auto piece_read = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(meta.piece_empty[piece % kPieces]));
        ++piece;
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
        if (warp == 8) {
            // ================================================== producer
            const auto wait = [&](uint64_t &b, uint32_t parity) {
                return warp_wait_soon(smem_u32(&b), parity, limit, p.flags);
            };
            constexpr int N = C::NS;
            const bool paged = p.block_table != nullptr;
            const int bs = p.block_size;
            const int nblk = paged ? kKeys / bs : 1;
            int boxes = 0, units = 0;
            bool ok = true;
            PieceWalk<NQ> walk(p, meta.share);
            UnitDeal<NQ> deal(p);
            while (ok) {
                Piece u;
                const bool more = p.parts ? walk.next(u) : deal.next(u);
                if (more) piece_keys<NQ>(p, u, tpq);
                else u.ntok = 0;
                if (!(ok = wait(meta.piece_empty[piece % kPieces], ((piece / kPieces) & 1) ^ 1))) break;
                if (lane == 0) {
                    meta.piece[piece % kPieces] = u;
                    mbar_arrive(bar(meta.piece_full[piece % kPieces]));
                }
                ++piece;
                if (!more) break;
                if (u.kb >= u.ke) continue;
                const int32_t *table = p.block_table + static_cast<int64_t>(u.seq) * p.max_blocks_per_seq;
                // block ids of key tile j: lane b % nblk holds block b's (or -1)
                const auto ids = [&](int j) {
                    if (!paged || j >= u.ke) return -1;
                    const int key = j * kKeys + (lane % nblk) * bs;
                    if (key + bs <= u.lo || key >= u.hi) return -1;
                    int id = __ldg(table + key / bs);
                    if (id < 0 || id >= p.num_blocks) {
                        raise_flag(p.flags, kFlagBlockId);
                        id = 0;
                    }
                    return id;
                };
                const auto load = [&](const CUtensorMap *map, int j, int half, int id) {
                    const int s = boxes % N;
                    if (!wait(meta.empty[s], ((boxes / N) & 1) ^ 1)) return false;
                    ++boxes;
                    const uint32_t b = bar(meta.full[s]);
                    // E4M3 rows land where their second halves will be
                    const uint32_t dst = ring + s * kBox + (FP8 ? kLine : 0);
                    if (!paged) {
                        if (lane == 0) {
                            mbar_arrive_expect_tx(b, kBox);
#pragma unroll
                            for (int l = 0; l < 2; ++l)
                                tma_load_3d(dst + l * kLine, map, b, (2 * half + l) * 64, u.h,
                                            u.kv0 + j * kKeys);
                        }
                    } else {
                        constexpr int L = FP8 ? 1 : 2;       // loads per block
                        const bool mine = lane < nblk * L && id >= 0;
                        const int cnt = __popc(__ballot_sync(0xffffffffu, mine));
                        if (lane == 0) mbar_arrive_expect_tx(b, cnt * bs * 128);
                        __syncwarp();
                        if (mine) {
                            const int l = lane / nblk;
                            tma_load_4d(dst + l * kLine + (lane % nblk) * bs * 128, map, b, 0, 0,
                                        FP8 ? 0 : 2 * half + l, id * p.num_kv_heads + u.h);
                        }
                    }
                    __syncwarp();
                    return true;
                };
                int id = ids(u.kb), id_next = ids(u.kb + 1);
                if (!(ok = wait(meta.q_empty, (units & 1) ^ 1))) break;
                ++units;
                if (lane == 0) {
                    const uint32_t b = bar(meta.q_full);
                    int tiles = 0;
                    for (int i = 0; i < NQ; ++i) tiles += u.t[i].ntok > 0;
                    mbar_arrive_expect_tx(b, tiles * C::LINES * tpq * p.group * 128);
                    for (int i = 0; i < tiles; ++i)
                        for (int l = 0; l < C::LINES; ++l)
                            tma_load_3d(smem + i * C::QTILE + l * kLine, &maps.q, b, l * 64,
                                        u.h * p.group, u.row0 + i * tpq);
                }
                __syncwarp();
                if (NQ == 2) {
                    for (int j = u.kb; ok && j < u.ke; ++j) {
                        const int id2 = ids(j + 2);
                        ok = load(&maps.k, j, 0, id) && load(&maps.v, j, 0, id);
                        id = id_next;
                        id_next = id2;
                    }
                } else {
                    for (int b = 0; ok && b < C::BOXES; ++b) ok = load(&maps.k, u.kb, b, id);
                    for (int j = u.kb; ok && j < u.ke; ++j) {
                        const int id2 = ids(j + 2);
                        if (j + 1 < u.ke)
                            for (int b = 0; ok && b < C::BOXES; ++b) ok = load(&maps.k, j + 1, b, id_next);
                        for (int b = 0; ok && b < C::BOXES; ++b) ok = load(&maps.v, j, b, id);
                        id = id_next;
                        id_next = id2;
                    }
                }
            }
            // every copy must land before the CTA exits
            bool landed = true;
            for (int i = max(0, boxes - N); i < boxes; ++i)
                landed &= mbar_wait_bounded(bar(meta.full[i % N]), (i / N) & 1, kDrainWaitNs);
            if (units > 0)
                landed &= mbar_wait_bounded(bar(meta.q_full), (units - 1) & 1, kDrainWaitNs);
            if (!landed) raise_flag(p.flags, kFlagTimeout);
        } else if (warp == 9) {
            // ================================================== MMA issue
            constexpr uint32_t kIdS = mma_idesc(128, 128, !FP8, false);
            constexpr uint32_t kIdO = mma_idesc(128, 128, !FP8, true);
            const auto wait = [&](uint64_t &b, uint32_t parity) {
                return warp_wait_soon(smem_u32(&b), parity, limit, p.flags);
            };
            const uint32_t leader = elect_one();
            int units = 0, steps = 0, slot = 0;
            uint32_t phase = 0, fixed_phase = 0;
            uint32_t p_count = 0;                        // parities, bit t of tile t
            bool ok = true;
            // S columns <- Q tile i . K box in slot s, elements 128 * half ...
            const auto qk = [&](uint32_t d, int i, int s, int half) {
                const uint64_t a = smem_desc(smem + i * C::QTILE + half * kBox, 16);
                const uint64_t b = smem_desc(ring + s * kBox, 16);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t off = ((kk >> 2) * kLine + (kk & 3) * 32) >> 4;
                        mma_ss(tmem + d, a + off, b + off, kIdS, kk > 0 || half > 0);
                    }
                }
            };
            // O columns (+)= P (in S columns c) . V box in slot s, one half of the keys
            const auto pv = [&](uint32_t d, uint32_t c, int s, int half, bool acc) {
                const uint64_t b = smem_desc(ring + s * kBox + half * 8192, kLine);
                const uint32_t a = tmem + c + half * 32;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ts(tmem + d, a + kk * 8, b + kk * (2048 >> 4), kIdO, kk > 0 || acc);
                }
            };
            uint64_t *ready = FP8 ? meta.fixed : meta.full;
            // the ring's next box; its slot is returned, -1 after a timeout
            const auto next_box = [&](bool fix) {
                const int s = slot;
                const bool fixed = FP8 || fix;
                const uint32_t parity = !FP8 && fix ? (fixed_phase >> s) & 1 : phase;
                if (!FP8 && fix) fixed_phase ^= 1u << s;
                if (++slot == C::NS) {
                    slot = 0;
                    phase ^= 1;
                }
                return wait(fixed ? meta.fixed[s] : meta.full[s], parity) ? s : -1;
            };
            while (ok && next_piece()) {
                const Piece k = meta.piece[piece % kPieces];
                piece_read();
                if (k.kb >= k.ke) continue;
                if (!(ok = wait(FP8 ? meta.q_ready : meta.q_full, units & 1))) break;
                ++units;
                if (NQ == 2) {
                    int sk = next_box(false);
                    ok = sk >= 0;
                    if (!ok) break;
                    const int kb0 = k.t[0].kb, ke0 = k.t[0].ke;
                    const int kb1 = k.t[NQ - 1].kb, ke1 = k.t[NQ - 1].ke;
#pragma unroll 1
                    for (int i = 0; i < NQ; ++i)
                        if (i ? kb1 == k.kb && kb1 < ke1 : kb0 == k.kb && kb0 < ke0) {
                            qk(i * 128, i, sk, 0);
                            if (leader) mma_commit(bar(meta.s_ready[i]));
                        }
                    if (leader) mma_commit(bar(meta.empty[sk]));
                    if (leader && k.kb + 1 == k.ke) mma_commit(bar(meta.q_empty));
                    // steps in which both tiles finish one key tile and start the
                    // next, and nothing else happens, run without conditions
                    const int steady_lo = max(max(kb0, kb1) + 1, k.part_lo);
                    const int steady_hi = min(min(ke0, ke1), k.part_hi) - 2;
                    for (int j = k.kb; ok && j < k.ke; ++j) {
                        if (j >= steady_lo && j < steady_hi) {
                            const int sv = slot, sn = slot + 1 == C::NS ? 0 : slot + 1;
                            const uint32_t next_phase = phase ^ (slot + 1 == C::NS);
                            ok = false;
                            if (!wait(ready[sv], phase)) break;
                            if (!wait(meta.p_ready[0][0], p_count & 1)) break;
                            tcgen05_fence_after();
                            pv(kOCol, 0, sv, 0, true);
                            if (!wait(meta.p_ready[0][1], p_count & 1)) break;
                            tcgen05_fence_after();
                            pv(kOCol, 0, sv, 1, true);
                            if (!wait(ready[sn], next_phase)) break;
                            qk(0, 0, sn, 0);
                            if (leader) mma_commit(bar(meta.s_ready[0]));
                            if (!wait(meta.p_ready[1][0], p_count >> 1)) break;
                            tcgen05_fence_after();
                            pv(kOCol + 128, 128, sv, 0, true);
                            if (!wait(meta.p_ready[1][1], p_count >> 1)) break;
                            tcgen05_fence_after();
                            pv(kOCol + 128, 128, sv, 1, true);
                            if (leader) mma_commit(bar(meta.empty[sv]));
                            qk(128, 1, sn, 0);
                            if (leader) {
                                mma_commit(bar(meta.s_ready[1]));
                                mma_commit(bar(meta.empty[sn]));
                            }
                            p_count ^= 3;
                            slot = sn + 1 == C::NS ? 0 : sn + 1;
                            phase = next_phase ^ (sn + 1 == C::NS);
                            ok = true;
                            continue;
                        }
                        const bool more = j + 1 < k.ke;
                        const int sv = next_box(is_partial(k, j));
                        ok = sv >= 0;
                        if (!ok) break;
#pragma unroll 1
                        for (int i = 0; i < NQ; ++i) {
                            const int kb = i ? kb1 : kb0, ke = i ? ke1 : ke0;
                            if (j >= kb && j < ke) {
#pragma unroll 1
                                for (int h = 0; h < 2; ++h) {
                                    ok = wait(meta.p_ready[i][h], (p_count >> i) & 1);
                                    if (!ok) break;
                                    tcgen05_fence_after();
                                    pv(kOCol + i * 128, i * 128, sv, h, h > 0 || j > kb);
                                }
                                if (!ok) break;
                                p_count ^= 1u << i;
                                if (j + 1 == ke && leader) mma_commit(bar(meta.o_done[i]));
                            }
                            if (i == NQ - 1 && leader) mma_commit(bar(meta.empty[sv]));
                            if (i == 0 && more) {
                                sk = next_box(false);
                                ok = sk >= 0;
                                if (!ok) break;
                            }
                            if (j + 1 >= kb && j + 1 < ke) {
                                qk(i * 128, i, sk, 0);
                                if (leader) mma_commit(bar(meta.s_ready[i]));
                            }
                        }
                        if (!ok) break;
                        if (leader && more) {
                            mma_commit(bar(meta.empty[sk]));
                            if (j + 2 == k.ke) mma_commit(bar(meta.q_empty));
                        }
                    }
                } else {
                    const auto qk_tile = [&](int step) {
                        for (int b = 0; b < C::BOXES; ++b) {
                            const int s = next_box(false);
                            if (s < 0) return false;
                            qk((step & 1) * 128, 0, s, b);
                            if (leader) {
                                mma_commit(bar(meta.empty[s]));
                                if (b == C::BOXES - 1) mma_commit(bar(meta.s_ready[step & 1]));
                            }
                        }
                        return true;
                    };
                    ok = qk_tile(steps);
                    if (ok && k.kb + 1 == k.ke && leader) mma_commit(bar(meta.q_empty));
                    for (int j = k.kb; ok && j < k.ke; ++j, ++steps) {
                        if (j + 1 < k.ke) {
                            if (!(ok = qk_tile(steps + 1))) break;
                            if (j + 2 == k.ke && leader) mma_commit(bar(meta.q_empty));
                        }
#pragma unroll 1
                        for (int b = 0; b < C::BOXES; ++b) {
                            const int s = next_box(is_partial(k, j));
                            ok = ok && s >= 0;
#pragma unroll 1
                            for (int h = 0; h < 2; ++h) {
                                if (b == 0)
                                    ok = ok && wait(meta.p_ready[steps & 1][h], (steps >> 1) & 1);
                                if (!ok) break;
                                tcgen05_fence_after();
                                pv(kOCol + b * 128, (steps & 1) * 128, s, h, h > 0 || j > k.kb);
                            }
                            if (!ok) break;
                            if (leader) mma_commit(bar(meta.empty[s]));
                        }
                        if (!ok) break;
                        if (leader) mma_commit(bar(meta.pv_done));
                        if (j + 1 == k.ke && leader) mma_commit(bar(meta.o_done[0]));
                    }
                }
            }
            // the tensor cores must be done with shared and tensor memory
            if (leader) mma_commit(bar(meta.drain));
            if (!mbar_wait_bounded(bar(meta.drain), 0, kDrainWaitNs)) raise_flag(p.flags, kFlagTimeout);
            __syncwarp();
        } else if (warp >= C::V_WARP0) {
            // ================================================== V warps
            const int tid = threadIdx.x - C::V_WARP0 * 32;
            int box = 0, units = 0;
            bool ok = true;
            while (ok && next_piece()) {
                const Piece k = meta.piece[piece % kPieces];
                piece_read();
                if (k.kb >= k.ke) continue;
                if (FP8) {
                    if (!(ok = wait(meta.q_full, units & 1))) break;
#pragma unroll 1
                    for (int r = tid >> 3; r < (k.t[NQ - 1].ntok > 0 ? NQ : 1) * 128; r += 4 * C::V_WARPS) {
                        const float back = convert_q_row(smem + (r >> 7) * C::QTILE, r & 127, tid & 7);
                        if ((tid & 7) == 0) row_mult[(units & 1) * 256 + r] = back;
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(meta.q_ready));
                }
                ++units;
                // one box: j its key tile, v whether it is of V
                const auto take = [&](int j, bool v) {
                    const int s = box % C::NS;
                    const bool part = v && is_partial(k, j);
                    const int j0 = j * kKeys;
                    const int lo = part ? k.lo - j0 : 0, hi = part ? k.hi - j0 : kKeys;
                    bool bad = false;
                    if (!wait(meta.full[s], (box / C::NS) & 1)) return false;
                    if (FP8 || part) {
                        if (FP8) {
                            if (part) bad = clean_bytes<C::V_WARPS>(ring + s * kBox, lo, hi, tid);
                            convert_box<C::V_WARPS>(ring + s * kBox, tid);
                        } else {
                            bad = clean_box<C::V_WARPS>(ring + s * kBox, lo, hi, k.all_lo - j0,
                                                        k.all_hi - j0, tid);
                        }
                        fence_proxy_async();
                        if (bad) meta.bad[units % kBadSlots] = units;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(meta.fixed[s]));
                    }
                    if (!FP8) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(meta.empty[s]));
                    }
                    ++box;
                    return true;
                };
                if (NQ == 2) {
                    for (int j = k.kb; ok && j < k.ke; ++j) ok = take(j, false) && take(j, true);
                } else {
                    for (int b = 0; ok && b < C::BOXES; ++b) ok = take(k.kb, false);
                    for (int j = k.kb; ok && j < k.ke; ++j) {
                        if (j + 1 < k.ke)
                            for (int b = 0; ok && b < C::BOXES; ++b) ok = take(j + 1, false);
                        for (int b = 0; ok && b < C::BOXES; ++b) ok = take(j, true);
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFTMAX_REGS));
        if (NQ == 2 || warp < 4) {
            // ================================================== softmax
            const int t = NQ == 2 ? warp >> 2 : 0;
            const int r = threadIdx.x & 127;
            const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // TMEM lane 32 * (warp & 3)
            const int g = p.group;
            const int tok = r / g, hd = r - tok * g;
            constexpr float kLog2e = 1.4426950408889634f;
            int units = 0, steps = 0, done = 0;
            bool ok = true;
            // the piece stays in shared memory until its output is out
            for (; ok && next_piece(); piece_read()) {
                const Piece &u = meta.piece[piece % kPieces];
                const TileKeys tk = u.t[t];
                if (u.kb < u.ke) ++units;
                if (tk.ntok <= 0) continue;
                const bool valid = tok < tk.ntok;
                const int hi = tk.p0 + tok + 1;
                float m = -INFINITY, l = 0.f;
                const bool any = tk.kb < tk.ke;
                if (any) {
                    float mult = 0.f;
                    float2 l2 = make_float2(0.f, 0.f);
                    for (int j = tk.kb; j < tk.ke; ++j, ++steps) {
                        const int sb = NQ == 2 ? t : steps & 1;
                        if (!(ok = wait(meta.s_ready[sb], (NQ == 2 ? steps : steps >> 1) & 1))) break;
                        tcgen05_fence_after();
                        const uint32_t scol = tmem + lanes + sb * 128;
                        if (j == tk.kb) {
                            mult = p.scale * kLog2e;
                            if (FP8) mult *= __ldg(p.k_scale + u.h) * row_mult[((units - 1) & 1) * 256 + t * 128 + r];
                            // a scale of zero: every visible key weighs the same,
                            // and masked scores (-inf) must still vanish
                            mult = mult == 0.f ? 0x1p-149f : mult;
                        }
                        const bool masked = j < tk.mlo || j >= tk.mhi;
                        if (__any_sync(0xffffffffu, masked || mult < 0.f)) {
                            // scores are changed where they lie: hidden ones to
                            // -inf, and all of them negated for a negative scale;
                            // columns [b, a) are the row's
                            const int a = masked ? hi - j * kKeys : kKeys;
                            const int b = masked ? first_seen(p, hi - 1) - j * kKeys : 0;
#pragma unroll 1
                            for (int c = 0; c < 128; c += 32) {
                                if (!__any_sync(0xffffffffu, mult < 0.f || a < c + 32 || b > c)) continue;
                                float s[32];
                                if (!__any_sync(0xffffffffu, valid && a > c)) {
#pragma unroll
                                    for (int i = 0; i < 32; ++i) s[i] = -INFINITY;
                                } else {
                                    tmem_ld32(scol + c, s);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int i = 0; i < 32; ++i) {
                                        asm volatile("" : "+f"(s[i]));
                                        s[i] = mult < 0.f ? -s[i] : s[i];
                                        s[i] = c + i < a && c + i >= b ? s[i] : -INFINITY;
                                    }
                                }
                                tmem_st32(scol + c, s);
                            }
                            tmem_wait_st();
                        }
                        // row maximum
                        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                        for (int c0 = 0; c0 < 128; c0 += 64) {
                            float s[64];
                            tmem_ld32(scol + c0, s);
                            tmem_ld32(scol + c0 + 32, s + 32);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 64; ++c) asm volatile("" : "+f"(s[c]));
#pragma unroll
                            for (int c = 0; c < 64; c += 8)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    m4[i] = max3_nan(m4[i], s[c + i], s[c + 4 + i]);
                        }
                        const float mx = max3_nan(max3_nan(m4[0], m4[1], m4[2]), m4[3], m4[3]);
                        const float am = fabsf(mult);
                        const float top = valid ? mx * am : -INFINITY;
                        // also for NaN, which poisons the row's sum, and +inf
                        constexpr float kBelow = FP8 ? 7.f : 0.f;
                        const bool move = !(top <= m + (8.f + kBelow));
                        if (__any_sync(0xffffffffu, move)) {
                            const float m_new = move ? top - kBelow : m;
                            float alpha = move ? ex2(m - m_new) : 1.f;
                            m = m_new;
                            alpha = top < INFINITY ? alpha : NAN;
                            l2.x = top < INFINITY ? l2.x : NAN;
                            l2 = mul2(l2, make_float2(alpha, alpha));
                            if (j > tk.kb) {
                                if (NQ == 1) {
                                    if (!(ok = wait(meta.pv_done, (steps - 1) & 1))) break;
                                    tcgen05_fence_after();
                                }
                                const uint32_t ocol = tmem + lanes + kOCol + t * 128;
#pragma unroll 1
                                for (int c = 0; c < D; c += 16) {
                                    uint32_t o[16];
                                    tmem_ld16(ocol + c, o);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int i = 0; i < 16; ++i) {
                                        asm volatile("" : "+r"(o[i]));
                                        o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                                    }
                                    tmem_st16(ocol + c, o);
                                }
                            }
                        }
                        const float mu = m == -INFINITY ? 0.f : -m;
                        const float2 k2 = make_float2(am, am), m2 = make_float2(mu, mu);
                        // The scores are read a second time, in a short loop: with
                        // three quarters of them held in registers and the step
                        // unrolled a prompt of 8192 tokens took 951 us instead of
                        // 1007, a mixed step 114 instead of 112 and windowed wide
                        // heads 191 instead of 185.  Every fourth pair of
                        // exponentials as a polynomial on the FMA pipes relieves
                        // ex2 (8 cycles a warp instruction) but took 121 us of the
                        // mixed step, and no less of the prompt.
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int c = 2 * h; c < 2 * h + 2; ++c) {
                                float s[32];
                                uint32_t w[16];
                                tmem_ld32(scol + c * 32, s);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(s[i]));
#pragma unroll
                                for (int i = 0; i < 32; i += 2) {
                                    float2 x = fma2(make_float2(s[i], s[i + 1]), k2, m2);
                                    x.x = ex2(x.x);
                                    x.y = ex2(x.y);
                                    l2 = add2(l2, x);
                                    w[i / 2] = FP8 ? pack_f16x2(x.x, x.y) : pack_bf16x2(x.x, x.y);
                                }
                                tmem_st16(scol + c * 16, w);
                            }
                            tmem_wait_st();
                            tcgen05_fence_before();
                            __syncwarp();
                            mbar_arrive_if(bar(meta.p_ready[sb][h]), lane == 0);
                        }
                    }
                    if (!ok) break;
                    l = l2.x + l2.y;
                    if (!(ok = wait(meta.o_done[t], done & 1))) break;
                    ++done;
                    tcgen05_fence_after();
                    const uint32_t mark = reinterpret_cast<volatile uint32_t *>(meta.bad)[units % kBadSlots];
                    if (__any_sync(0xffffffffu, mark == static_cast<uint32_t>(units)))
                        add_bad_values<D, FP8>(p, u, tk, valid ? hi : 0, tmem + lanes + kOCol + t * 128);
                }
                const float vs = FP8 ? __ldg(p.v_scale + u.h) : 1.f;
                const bool dead = l == 0.f;
                const float inv = dead ? 0.f : vs / l;
                const float lse = dead ? -INFINITY : m * 0.6931471805599453f + logf(l);
                // A thread writes its row, 32 bytes (a sector) at a time.
                const bool part = u.slot >= 0;
                const int64_t orow = part ? (static_cast<int64_t>(u.slot) * NQ + t) * 128 + r
                                          : static_cast<int64_t>(u.row0 + t * tpq + tok) * p.num_q_heads +
                                                u.h * g + hd;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    if (any) {
                        tmem_ld32(tmem + lanes + kOCol + t * 128 + c, o);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(o[i]));
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = dead ? 0.f : o[i] * inv;
                    if (valid && part) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            store32(p.o_part + orow * D + c + i, o + i);
                    } else if (valid) {
#pragma unroll
                        for (int i = 0; i < 32; i += 16) {
                            uint32_t w[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) w[k] = pack_bf16x2(o[i + 2 * k], o[i + 2 * k + 1]);
                            uint16_t *dst = p.out + orow * D + c + i;
                            if (p.out32) {
                                store32(dst, w);
                            } else {
                                *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
                                *reinterpret_cast<uint4 *>(dst + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                            }
                        }
                    }
                    __syncwarp();                // lanes with and without a row meet again
                }
                // the next piece's first P, by the same warps, tells that O was read
                tcgen05_fence_before();
                if (valid) {
                    if (part) p.lse_part[orow] = lse;
                    else if (p.lse_out) p.lse_out[orow] = lse;
                }
            }
        }
    }
    __syncwarp();
    tcgen05_fence_before();
    __syncthreads();
    if (warp == 9) {
        tcgen05_fence_after();
        tmem_dealloc(*reinterpret_cast<volatile uint32_t *>(&meta.tmem), 512);
    }
}

}  // namespace pgd
