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
// A boundary inside a unit cuts it at a key tile when the caller gave a
// workspace; otherwise, and for units without keys, the unit goes whole to the
// side that has more of it.
#pragma once

#include "pgd_prefill.h"
#include "pgd_ptx.cuh"

namespace pgd {

constexpr int kPrefillThreads = 512;
constexpr int kKeys = 128;           // keys per tile
constexpr int kUnitKeys = 128;       // a unit's fixed cost, in keys
constexpr int kPieces = 4;           // pieces handed out ahead

// One CTA's part of a unit: key tiles [kb, ke) of its query tiles.
struct Piece {
    int seq, h, row0, ntok, pos0, kv0, kb, ke;
    int slot;                        // workspace slot, -1: the whole unit
};

// Where a CTA's share starts, and how long it is.
struct Share {
    long long at, len;               // offset into the sequence's units, length
    long long seq_start;             // axis position of the sequence
    int seq;
    long long warp_sum[kPrefillThreads / 32];
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
        const long long q = (-a + step - 1) / step;
        i0 = q < m ? static_cast<int>(q) : m;
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
template <int NQ>
__device__ void find_share(const PrefillParams &p, Share &share) {
    const int tpu = tokens_per_unit<NQ>(p);
    const int tid = threadIdx.x, lane = tid & 31;
    const auto len_of = [&](int s, bool report) {
        const SeqRows r = seq_rows(p, s, report);
        const int nt = (r.len + tpu - 1) / tpu;
        return nt == 0 ? 0ll : units_len(r, tpu, nt, p.window, nt) * p.num_kv_heads;
    };
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
#pragma unroll
        for (int w = 0; w < kPrefillThreads / 32; ++w) {
            const long long y = share.warp_sum[w];
            if (w < (tid >> 5)) before += y;
            total += y;
        }
        return before + x;
    };
    const bool report = blockIdx.x == 0;
    long long mine = len_of(tid, report), sum, total;
    long long incl = scan(mine, sum);
    total = sum;
    for (int s0 = kPrefillThreads; s0 < p.num_seqs; s0 += kPrefillThreads) {
        scan(len_of(s0 + tid, report), sum);
        total += sum;
    }
    if (tid == 0) {
        share.at = 0;
        share.len = 0;
        share.seq_start = 0;
        share.seq = p.num_seqs;
    }
    __syncthreads();
    const long long n = gridDim.x, c = blockIdx.x;
    const long long q = total / n, rest = total - q * n;   // total * n may pass 64 bits
    const long long x0 = q * c + rest * c / n, x1 = q * (c + 1) + rest * (c + 1) / n;
    long long base = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += kPrefillThreads) {
        if (s0 > 0) {
            mine = len_of(s0 + tid, false);
            incl = scan(mine, sum);
        } else if (p.num_seqs > kPrefillThreads) {
            scan(mine, sum);
        }
        const long long a = base + incl - mine;
        if (x0 < x1 && mine > 0 && a <= x0 && x0 < a + mine) {
            share.at = x0 - a;
            share.len = x1 - x0;
            share.seq_start = a;
            share.seq = s0 + tid;
        }
        base += sum;
    }
}

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
        if (len > 0) {
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
            if (p.parts) cut = cut_record();
        } else if (p.parts) {
            unit_start = -1;
        }
        if (p.parts && (threadIdx.x & 31) == 0) {
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

    // The whole current unit; its key tiles as [kb, ke), one empty tile for a
    // unit that sees nothing.
    __device__ __forceinline__ void geometry(Piece &u, int &lo, int &hi) const {
        const int tok0 = unit * tpu;
        u.seq = seq;
        u.h = h;
        u.row0 = s.row + tok0;
        u.ntok = min(tpu, s.len - tok0);
        u.pos0 = s.keys - s.len + tok0;
        u.kv0 = s.row;
        u.slot = -1;
        hi = max(0, u.pos0 + u.ntok);
        lo = p.window > 0 && hi > 0 ? max(0, u.pos0 + 1 - p.window) : 0;
        u.kb = lo / kKeys;
        u.ke = max(u.kb + 1, (hi + kKeys - 1) / kKeys);
    }

    // The key tile (from the unit's first) at which a boundary x into it cuts.
    __device__ __forceinline__ int cut_at(long long x, int lo, int hi, int tiles) const {
        const long long cost = hi - lo + kUnitKeys;
        if (x <= 0) return 0;
        if (x >= cost) return tiles;
        if (!p.parts || hi == 0) return 2 * x < cost ? 0 : tiles;
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
