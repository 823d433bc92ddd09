// pgd_prefill_sched.cuh -- how the prompt attention kernel deals its work.
//
// A unit is one KV head's NQ query tiles (NQ * (128 / g) consecutive tokens of
// one sequence) over the keys they see together, [lo, hi).  All units lie end
// to end on one axis, sequence by sequence, head by head, tokens ascending, a
// unit hi - lo + kUnitKeys long (its keys, and a constant for the query load,
// the first and the last product and the output).  CTA c of n takes
// [c/n, (c+1)/n) of the axis.  The length of a sequence's first m units has a
// closed form (two arithmetic series clamped at zero), so a CTA finds its
// share with one prefix sum over the sequences and one search, whatever the
// lengths, and no unit list is kept anywhere.
//
// A boundary inside a unit cuts it at a key tile; a unit without keys goes
// whole to the side that has more of it.  Calls that cut nothing (short
// contexts, or no workspace) deal whole units to the CTAs in turn instead,
// which one warp does with 32-bit counts: 2 us less before the first load.
#pragma once

#include "pgd_prefill.h"
#include "pgd_ptx.cuh"

namespace pgd {

constexpr int kMaxThreads = 512;
constexpr int kKeys = 128;           // keys per tile
// A unit's fixed cost, in keys.  Times in us, caches flushed:
//                                          128   256   384   512   768
//   bf16 D 128: prompt of 8192 (64/8)     1022   962   975   986  1015
//               ragged prompts (32/8)      193   170   174   182   194
//               mixed step (32/8)          117   112   114   117   123
//   bf16 D 256: prompt of 4096 (32/2)      367   292   258   263   266
//               ragged prompts (32/4)      367   307   279   291   302
//               mixed step (32/4)          166   155   160   166   172
//   E4M3 D 128: prompt of 4096 (32/8)      215   195   186   186   199
//               ragged prompts (32/8)      247   220   209   215   227
//               mixed step (32/8)          150   131   129   125   135
constexpr int kUnitKeys = 384;
constexpr int kPieces = 4;           // pieces handed out ahead

// The keys that one query tile of a piece sees.
struct TileKeys {
    int ntok;           // query tokens of the tile
    int p0;             // position of the first
    int kb, ke;         // key tiles of this piece
    int mlo, mhi;       // tiles below mlo or from mhi on are not seen whole by every row
};

// One CTA's part of a unit: key tiles [kb, ke) of its query tiles.
struct Piece {
    int seq, h, row0, ntok, pos0, kv0, kb, ke;
    int slot;                        // workspace slot, -1: the whole unit
    int lo, hi;                      // positions that some row sees (whole unit)
    int all_lo, all_hi;              // positions that every row sees
    int part_lo, part_hi;            // as mlo, mhi, of the tiles together
    TileKeys t[2];
};

// Where a CTA's share starts, and how long it is.  More CTAs than the axis is
// long leave shares of no length: they have a start all the same, which the
// merge needs to follow a unit's pieces from CTA to CTA.
struct Share {
    long long at, len;               // offset into the sequence's units, length
    long long seq_start;             // axis position of the sequence
    int seq;                         // num_seqs: no work at all
    long long warp_sum[kMaxThreads / 32];
};

// One sequence, its query rows and its keys (zero rows: nothing to do).
struct SeqRows {
    int row, len, keys;
};

__device__ __forceinline__ SeqRows seq_rows(const PrefillParams &p, int s, bool report) {
    SeqRows r = {0, 0, 0};
    if (s >= p.num_seqs) return r;
    const int a = __ldg(p.cu + s), b = __ldg(p.cu + s + 1);
    int n = p.block_table ? __ldg(p.context_lens + s) : 0;
    if (a == b && a >= 0 && b <= p.num_tokens) return r;       // no rows: no context either
    if (a < 0 || b < a || b > p.num_tokens) {
        if (report) raise_flag(p.flags, kFlagContextLen);
        return r;
    }
    if (p.block_table) {
        const int cap = p.max_blocks_per_seq * p.block_size;
        if (n < 0 || n > cap) {
            if (report) raise_flag(p.flags, kFlagContextLen);
            n = n < 0 ? 0 : cap;
        }
    }
    r.row = a;
    r.len = b - a;
    r.keys = p.block_table ? n : r.len;
    return r;
}

// sum over i < m of max(0, a + i * step)
__device__ __forceinline__ long long ramp(long long a, int step, int m) {
    int i0 = 0;
    if (a < 0) {
        const unsigned q = (static_cast<unsigned>(-a) + step - 1) / step;   // -a <= 2^31
        i0 = q < static_cast<unsigned>(m) ? static_cast<int>(q) : m;
    }
    const long long k = m - i0;
    return k * a + step * ((static_cast<long long>(i0) + m - 1) * k / 2);
}

// Axis length of the first m units of a sequence (of nt, tpu tokens each).
__device__ __forceinline__ long long units_len(const SeqRows &s, int tpu, int nt, int window,
                                               int m) {
    const long long first = static_cast<long long>(s.keys) - s.len;   // position of row 0
    long long x = static_cast<long long>(m) * kUnitKeys;
    if (m == nt && m > 0) x += s.keys + ramp(first + tpu, tpu, m - 1);
    else x += ramp(first + tpu, tpu, m);
    if (window > 0) x -= ramp(first + 1 - window, tpu, m);
    return x;
}

template <int NQ>
__device__ __forceinline__ int tokens_per_unit(const PrefillParams &p) {
    return NQ * (128 / p.group);
}

// The CTA's share (all threads; the caller synchronises before reading it).
template <int NQ, int THREADS>
__device__ void find_share(const PrefillParams &p, Share &share) {
    const int tpu = tokens_per_unit<NQ>(p);
    const int tid = threadIdx.x, lane = tid & 31;
    // inclusive sum over the threads, and the block's total
    const auto scan = [&](long long v, long long &total) {
        long long x = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        __syncthreads();
        if (lane == 31) share.warp_sum[tid >> 5] = x;
        __syncthreads();
        long long before = 0;
        total = 0;
#pragma unroll 4
        for (int w = 0; w < THREADS / 32; ++w) {
            const long long y = share.warp_sum[w];
            if (w < (tid >> 5)) before += y;
            total += y;
        }
        return before + x;
    };
    // first the total, then the sequence that x0 lies in; one copy of the code
    // for both (a cold instruction cache is what a small call waits for)
    const int n = gridDim.x, c = blockIdx.x;
    long long mine = 0, incl = 0, sum = 0, total = 0, base = 0, x0 = 0, x1 = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int s0 = 0; s0 < p.num_seqs; s0 += THREADS) {
            if (pass == 0 || p.num_seqs > THREADS) {
                const SeqRows r = seq_rows(p, s0 + tid, pass == 0 && c == 0);
                const int nt = (r.len + tpu - 1) / tpu;
                mine = nt == 0 ? 0ll : units_len(r, tpu, nt, p.window, nt) * p.num_kv_heads;
                incl = scan(mine, sum);
            }
            if (pass == 0) {
                total += sum;
                continue;
            }
            const long long a = base + incl - mine;
            if (mine > 0 && a <= x0 && x0 < a + mine) {
                share.at = x0 - a;
                share.len = x1 - x0;
                share.seq_start = a;
                share.seq = s0 + tid;
            }
            base += sum;
        }
        if (pass == 0) {
            const long long q = total / n;               // total * c may pass 64 bits
            const unsigned rest = static_cast<unsigned>(total - q * n);
            x0 = q * c + rest * c / n;
            x1 = q * (c + 1) + rest * (c + 1) / n;
            if (tid == 0) {
                share.at = 0;
                share.len = 0;
                share.seq_start = 0;
                share.seq = p.num_seqs;
            }
            __syncthreads();
        }
    }
}

// The first position that a row at position `pos` sees (of those from 0 on);
// `pos` may be negative and the window anything up to 2^31 - 1.
__device__ __forceinline__ int first_seen(const PrefillParams &p, int pos) {
    return p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
}

// A whole unit of a sequence from its token tok0 on; its key tiles as [kb, ke),
// one empty tile for a unit that sees nothing.
__device__ __forceinline__ void unit_piece(const PrefillParams &p, const SeqRows &s, int seq, int h,
                                           int tok0, int tpu, Piece &u, int &lo, int &hi) {
    u.seq = seq;
    u.h = h;
    u.row0 = s.row + tok0;
    u.ntok = min(tpu, s.len - tok0);
    u.pos0 = s.keys - s.len + tok0;
    u.kv0 = s.row;
    u.slot = -1;
    hi = max(0, u.pos0 + u.ntok);
    lo = hi > 0 ? first_seen(p, u.pos0) : 0;
    u.kb = lo / kKeys;
    u.ke = max(u.kb + 1, (hi + kKeys - 1) / kKeys);
}

// Deals whole units, numbered sequence by sequence and head by head, to the
// CTAs in turn; one warp, all lanes alike, 32 sequences at a time.  (The
// queries fit the device's memory, so the numbers fit 31 bits.)
template <int NQ>
struct UnitDeal {
    const PrefillParams &p;
    const int tpu;
    int unit, before, window_units, window_seq, first;
    SeqRows mine;
    int mine_tiles;

    __device__ UnitDeal(const PrefillParams &p_)
        : p(p_), tpu(tokens_per_unit<NQ>(p_)), unit(blockIdx.x), before(0), window_units(0),
          window_seq(-32), first(0), mine_tiles(0) {}

    __device__ __forceinline__ bool next(Piece &u) {
        const int lane = threadIdx.x & 31;
        while (unit >= before + window_units) {
            if (window_seq + 32 >= p.num_seqs) return false;
            before += window_units;
            window_seq += 32;
            mine = seq_rows(p, window_seq + lane, blockIdx.x == 0);
            mine_tiles = (mine.len + tpu - 1) / tpu;
            int incl = mine_tiles * p.num_kv_heads;
            first = incl;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += y;
            }
            first = incl - first;
            window_units = __shfl_sync(0xffffffffu, incl, 31);
        }
        const int at = unit - before;
        // the last lane that starts at or before it (empty sequences start where
        // the next one does)
        const int src = 31 - __clz(__ballot_sync(0xffffffffu, first <= at && mine_tiles > 0));
        SeqRows s;
        s.row = __shfl_sync(0xffffffffu, mine.row, src);
        s.len = __shfl_sync(0xffffffffu, mine.len, src);
        s.keys = __shfl_sync(0xffffffffu, mine.keys, src);
        const int r = at - __shfl_sync(0xffffffffu, first, src);
        const int tiles = __shfl_sync(0xffffffffu, mine_tiles, src), h = r / tiles;
        int lo, hi;
        unit_piece(p, s, window_seq + src, h, (r - h * tiles) * tpu, tpu, u, lo, hi);
        if (hi == 0) u.ke = u.kb;
        unit += gridDim.x;
        return true;
    }
};

// Walks the pieces of the CTA's share; one warp, all lanes alike.  Sequences
// are read 32 at a time, one per lane.
template <int NQ>
struct PieceWalk {
    const PrefillParams &p;
    const int tpu;
    long long len, at;               // what is left; offset into the current unit
    long long unit_start;            // axis position of the current unit
    int seq, h, unit, units;
    SeqRows s, mine;
    int window_seq;

    __device__ PieceWalk(const PrefillParams &p_, const Share &share)
        : p(p_), tpu(tokens_per_unit<NQ>(p_)), len(share.len), at(0),
          unit_start(share.seq_start), seq(share.seq), h(0), unit(0), units(0), window_seq(-64) {
        int cut = 0;
        if (!p.parts) return;
        if (seq < p.num_seqs) {
            load_seq();
            const long long per_head = units_len(s, tpu, units, p.window, units);
            h = static_cast<int>(share.at / per_head);
            const long long x = share.at - h * per_head;
            // the last unit that starts at or before x: 32 probes a round
            int a = 0, b = units;
            while (b - a > 1) {
                const int w = (b - a + 31) / 32;
                const int i = a + w * (threadIdx.x & 31);
                const bool below = i < b && units_len(s, tpu, units, p.window, i) <= x;
                const int top = 31 - __clz(__ballot_sync(0xffffffffu, below));
                b = min(b, a + (top + 1) * w);
                a += top * w;
            }
            unit = a;
            at = x - units_len(s, tpu, units, p.window, a);
            unit_start += h * per_head + (x - at);
            cut = cut_record();
        } else {
            unit_start = -1;
        }
        if ((threadIdx.x & 31) == 0) {
            PartRecord r = {};
            r.unit = unit_start;
            r.cut = cut;
            if (cut) {
                Piece u;
                int lo, hi;
                geometry(u, lo, hi);
                r.tiles = u.ke - u.kb;
                r.row0 = u.row0;
                r.ntok = u.ntok;
                r.h = h;
            }
            p.parts[blockIdx.x] = r;
        }
    }

    __device__ __forceinline__ void load_seq() {
        if (seq < window_seq || seq >= window_seq + 32) {
            window_seq = seq;
            mine = seq_rows(p, seq + (threadIdx.x & 31), false);
        }
        const int src = seq - window_seq;
        s.row = __shfl_sync(0xffffffffu, mine.row, src);
        s.len = __shfl_sync(0xffffffffu, mine.len, src);
        s.keys = __shfl_sync(0xffffffffu, mine.keys, src);
        units = (s.len + tpu - 1) / tpu;
    }

    __device__ __forceinline__ void geometry(Piece &u, int &lo, int &hi) const {
        unit_piece(p, s, seq, h, unit * tpu, tpu, u, lo, hi);
    }

    // The key tile (from the unit's first) at which a boundary x into it cuts.
    __device__ __forceinline__ int cut_at(long long x, int lo, int hi, int tiles) const {
        const long long cost = hi - lo + kUnitKeys;
        if (x <= 0) return 0;
        if (x >= cost) return tiles;
        if (hi == 0) return 2 * x < cost ? 0 : tiles;
        if (x <= kUnitKeys) return 0;
        return static_cast<int>((lo + x - kUnitKeys) / kKeys) - lo / kKeys;
    }

    // The cut of this CTA's first unit by its own start, 0 if that is no cut.
    __device__ __forceinline__ int cut_record() const {
        Piece u;
        int lo, hi;
        geometry(u, lo, hi);
        const int c = cut_at(at, lo, hi, u.ke - u.kb);
        return c < u.ke - u.kb ? c : 0;
    }

    __device__ __forceinline__ bool next(Piece &u) {
        while (len > 0) {
            int lo, hi;
            geometry(u, lo, hi);
            const int tiles = u.ke - u.kb;
            const long long cost = hi - lo + kUnitKeys;
            const long long end = min(cost, at + len);
            const int a = cut_at(at, lo, hi, tiles), b = cut_at(end, lo, hi, tiles);
            len -= end - at;
            at = 0;
            if (len > 0) {                       // on to the next unit
                if (++unit == units) {
                    unit = 0;
                    if (++h == p.num_kv_heads) {
                        h = 0;
                        do {
                            if (++seq >= p.num_seqs) {
                                len = 0;
                                break;
                            }
                            load_seq();
                        } while (units == 0);
                    }
                }
            }
            if (a < b) {
                if (a > 0 || b < tiles) u.slot = 2 * blockIdx.x + (a > 0 ? 0 : 1);
                u.ke = hi == 0 ? u.kb : u.kb + b;
                u.kb += hi == 0 ? 0 : a;
                return true;
            }
        }
        return false;
    }
};

}  // namespace pgd
