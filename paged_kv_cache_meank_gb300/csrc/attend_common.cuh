// Work split of the paged attention kernels, shared by all of them.
//
// The work of a call is a line of units: for each sequence, each kv head, each
// tile of RB query rows (row = token * (H/G) + head in the group), one unit per
// `unit` keys that the tile sees (one unit for a tile that sees none, which
// still writes its rows).  The lengths live in device memory, so every CTA
// lays the line out itself, one prefix sum over the sequences, and takes an
// equal run of it: a ragged batch balances without the host knowing a length.  A
// run cuts a tile's keys at its two ends only.  A tile whole within one CTA is
// written at once; the CTAs that share one each leave an unnormalised sum with
// its running maximum and weight, and they are joined in CTA order, so that
// results do not depend on which CTA came last.
#pragma once

#include "kvm_internal.cuh"

namespace kvm {

//
// All of this is run once by one warp before the first load can be issued, from
// an instruction cache that is cold: it is kept small and in 32 bits (the host
// checks that the line is shorter than 2^31 units).
struct SeqInfo {
    int q0, q_len, kv;
};

// The lengths of a sequence; q_len = 0 and *ok = false where they are out of
// their bounds.
__host__ __device__ __forceinline__ SeqInfo seq_info(const BatchArgs &b, int s, bool *ok) {
    SeqInfo i;
    i.q0 = b.q_start[s];
    const int q1 = b.q_start[s + 1];
    i.kv = b.kv_len[s];
    *ok = i.q0 >= 0 && q1 >= i.q0 && q1 <= b.n_tokens && q1 - i.q0 <= b.max_q_len && i.kv >= 0 &&
          i.kv <= b.max_kv_len;
    i.q_len = *ok ? q1 - i.q0 : 0;
    return i;
}

// The token of a query row (row / gqa): `inv` is ceil(2^32 / gqa), or 0 for 1;
// exact while row * gqa < 2^32, which the host checks.
__host__ __device__ __forceinline__ int token_of(int row, uint32_t inv) {
    return inv ? (int)(((uint64_t)(uint32_t)row * inv) >> 32) : row;
}

// A line of units, as laid out (see lay_out).
struct LineInfo {
    int total;     // units of all
    int most;      // the largest row tile's
    int pad;       // units every row tile is counted as, or 0: its own
    int per;       // units of one CTA's run
};

template <int RB, int UNIT>
struct Line {
    // Keys that row tile r of a sequence sees (its last row sees the most).
    __host__ __device__ static __forceinline__ int keys(const SeqInfo &i, const AttendArgs &a, int r) {
        if (!a.causal) return i.kv;
        const int row_end = min(i.q_len * a.gqa, (r + 1) * RB);
        return max(0, min(i.kv, i.kv - i.q_len + token_of(row_end - 1, a.gqa_inv) + 1));
    }
    __host__ __device__ static __forceinline__ int tiles(const SeqInfo &i, const AttendArgs &a) {
        return (i.q_len * a.gqa + RB - 1) / RB;
    }
    __host__ __device__ static __forceinline__ int weight(const SeqInfo &i, const AttendArgs &a, int r) {
        return max(1, (keys(i, a, r) + UNIT - 1) / UNIT);
    }
    // Lays the line out: pre[s] = units of the sequences before s, or with `pad`
    // their row tiles (pre: kPreInts in shared memory, without PAD kPlainPreInts).  By one
    // warp, a lane to a sequence.
    template <bool PAD>
    __device__ static LineInfo lay_out(const AttendArgs &a, int *pre, int n_ctas, int min_units, int join) {
        const int lane = threadIdx.x & 31;
        LineInfo li{0, 1, 0, 0};
        int items = 0;
#pragma unroll 1
        for (int s0 = 0; s0 < a.b.n_seqs; s0 += 32) {
            const int s = s0 + lane;
            int w = 0, n = 0;
            if (s < a.b.n_seqs) {
                bool ok;
                const SeqInfo i = seq_info(a.b, s, &ok);
                if (!ok) atomicOr(a.b.err, kErrBatch);
                n = tiles(i, a);
#pragma unroll 1
                for (int r = 0; r < n; ++r) {
                    const int x = weight(i, a, r);
                    w += x;
                    li.most = max(li.most, x);
                }
            }
            w *= a.b.G;
            n *= a.b.G;
            int last = 0;
            if (a.b.n_seqs > 1) {
                last = 31;
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const int up = __shfl_up_sync(0xffffffffu, w, o);
                    const int un = __shfl_up_sync(0xffffffffu, n, o);
                    if (lane >= o) {
                        w += up;
                        n += un;
                    }
                }
            }
            if (s < a.b.n_seqs) {
                pre[s + 1] = li.total + w;
                if (PAD) pre[kMaxSeqs + 1 + s + 1] = items + n;
            }
            li.total += __shfl_sync(0xffffffffu, w, last);
            items += __shfl_sync(0xffffffffu, n, last);
        }
        if (lane == 0) {
            pre[0] = 0;
            if (PAD) pre[kMaxSeqs + 1] = 0;
        }
        li.most = __reduce_max_sync(0xffffffffu, li.most);
        plan<PAD>(li, items, n_ctas, min_units, join);
        __syncwarp();
        return li;
    }
    // From the row tiles' number, their units and the longest one's: what they are
    // counted as, and the runs.  A join counts as `join` units.
    template <bool PAD>
    __host__ __device__ static void plan(LineInfo &li, int items, int n_ctas, int min_units, int join) {
        const int share = (int)(((uint32_t)li.total + n_ctas - 1) / (uint32_t)n_ctas);
        // shorter runs than min_units do not pay, and a tile of `join` is not cut
        const int least = li.most <= join ? li.most : min_units;
        li.per = max(share, least);
        if (!PAD || items == 0) return;
        // A CTA to a tile, and no joins, where the longest takes less longer than an
        // equal share than a join does: nine ragged sequences of up to 1501 keys took
        // 36.8 us with runs of equal shares, 26.4 so.
        if (items <= n_ctas && li.most <= share + join) {
            li.pad = li.per = li.most;
            li.total = items * li.most;
            return;
        }
        // Where the row tiles are about equally long, they are all counted as `pad`
        // units, at least the longest one's: runs then begin and end at the same few
        // places of every tile.  A CTA meets one tile and not the ends of two, and
        // CTAs that share a head's keys read them at the same time (begun at scattered
        // keys they read 762 MB of a 134 MB cache).
        if ((float)li.total < 0.85f * (float)items * (float)li.most) return;
        int most_per = 0x7FFFFFFF;                       // what another split has to beat
        if (items < n_ctas) {                            // an equal part of a tile to a CTA
            const int parts = min(n_ctas / items, li.most / least);
            li.per = (li.most + parts - 1) / parts;
            li.pad = li.per * parts;
            most_per = (li.per + (parts > 1 ? join : 0)) / 8 * 7 - join;
        }
        // A multiple of a whole tile, its half, third, fourth or sixth: the first of
        // these that gives away at most 1/16 of the share, else the one that gives away
        // least; not where few CTAs are idle with an equal part (512 query tokens over
        // 16384 keys are 96 tiles, and took 210 us by 96 CTAs, 168 by all).
        const int pad = (li.most + 11) / 12 * 12;
        const int per = (int)(((uint32_t)(items * pad) + n_ctas - 1) / (uint32_t)n_ctas);
        if (li.most >= 24 && per < most_per && (float)li.total >= 0.85f * (float)items * (float)pad &&
            (float)items * (float)pad < 2147483647.f) {
            int run = 0x7FFFFFFF;
#pragma unroll 1
            for (int m = 1; m <= 6 && run - per > per / 16; m += m < 4 ? 1 : 2) {
                const int part = pad / m;
                run = min(run, (per + part - 1) / part * part);
            }
            if (run < most_per) {
                li.per = run;
                li.pad = pad;
            }
        }
        if (li.pad) li.total = items * li.pad;
    }
};

constexpr int kPreInts = 2 * (kMaxSeqs + 1), kPlainPreInts = kMaxSeqs + 1;   // shared memory of lay_out

// A walk over one CTA's run of the line.
template <int RB, int UNIT>
struct Walk {
    using LN = Line<RB, UNIT>;
    int x, end, per;         // position, end of the run, units of a run
    int s, g, r, n_tiles;    // sequence, kv head, row tile
    int u0, u1, w, pad;      // the segment's units [u0, u1) of the tile's w (pad: as counted)
    int nk;                  // keys the tile sees
    SeqInfo i;

    // False when the CTA's run is empty.
    __host__ __device__ __forceinline__ bool start(const AttendArgs &a, const int *pre, const LineInfo &li,
                                                   int cta) {
        per = li.per;
        if ((int64_t)cta * per >= li.total) return false;
        x = cta * per;
        end = li.total - x < per ? li.total : x + per;
        pad = li.pad;
        const int unit = pad ? pad : 1;
        if (pad) pre += kMaxSeqs + 1;                   // in row tiles
        int lo = 0, hi = a.b.n_seqs - 1;                // the last s with pre[s] * unit <= x
        while (lo < hi) {
            const int m = (lo + hi + 1) >> 1;
            if (pre[m] * unit <= x) lo = m; else hi = m - 1;
        }
        s = lo;
        bool ok;
        i = seq_info(a.b, s, &ok);
        n_tiles = LN::tiles(i, a);
        int rem = x - pre[s] * unit;
        const int per_head = pad ? n_tiles * pad : (pre[s + 1] - pre[s]) / a.b.G;
        g = rem / per_head;
        rem -= g * per_head;
        r = 0;
        if (pad) {
            if (n_tiles > 1) {
                r = rem / pad;
                rem -= r * pad;
            }
        } else {
            for (int y = LN::weight(i, a, 0); rem >= y; y = LN::weight(i, a, r)) {
                rem -= y;
                ++r;
            }
        }
        u0 = rem;
        fill(a);
        return true;
    }
    __host__ __device__ __forceinline__ void fill(const AttendArgs &a) {
        w = pad ? pad : LN::weight(i, a, r);
        nk = LN::keys(i, a, r);
        u1 = min(w, u0 + (end - x));
    }
    __host__ __device__ __forceinline__ bool next(const AttendArgs &a) {
        x += u1 - u0;
        if (x >= end) return false;
        u0 = 0;
        if (++r == n_tiles) {
            r = 0;
            if (++g == a.b.G) {
                g = 0;
                do {                                    // skips sequences without rows
                    bool ok;
                    i = seq_info(a.b, ++s, &ok);
                    n_tiles = LN::tiles(i, a);
                } while (n_tiles == 0);
            }
        }
        fill(a);
        return true;
    }
    // Key tiles of the segment: its units that hold keys.
    __host__ __device__ __forceinline__ int key_units() const {
        const int real = (nk + UNIT - 1) / UNIT;
        return min(u1, real) - min(u0, real);
    }
    __host__ __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == w; }
    // The first and last CTA that share the segment's tile.
    __host__ __device__ __forceinline__ int first_cta() const { return (x - u0) / per; }
    __host__ __device__ __forceinline__ int last_cta() const { return (x - u0 + w - 1) / per; }
};

// Whether a call's bounds keep the line and the query rows in their 32 bits.
inline bool line_fits(const AttendArgs &a, int rb, int unit) {
    const double rows = (double)a.b.max_q_len * a.gqa;
    const double tiles = (double)a.b.n_seqs * a.b.G * ((int64_t)(rows + rb - 1) / rb);
    return tiles * ((a.b.max_kv_len + (double)unit) / unit + 12) < 2147483647.0 &&
           rows * a.gqa < 4294967296.0;
}

// A CTA's two places for partial results: 1 for a tile that goes on in the next
// CTA and begins in this one, 0 for a tile that began in an earlier one.
__host__ __device__ __forceinline__ size_t part_slot(int cta, bool first) {
    return (size_t)cta * 2 + (first ? 1 : 0);
}

// Rows of partial results, d + 2 floats each: two places a CTA of each form.  The float32
// form may take any call, the other two bf16 queries over bf16 or e4m3 pages.
constexpr int kTileMaxCtas = 160, kTileMaxRows = 256, kSimtMaxRows = 16;
constexpr size_t kTilePartRows = (size_t)kTileMaxCtas * 2 * kTileMaxRows;
constexpr size_t kSimtPartRows = (size_t)kAttendMaxCtas * 2 * kSimtMaxRows;

// attend_decode.cu: up to kDecodeRows query rows of a kv head, the same types.
constexpr int kDecodeRows = 16;
bool attend_decode_supported(int q_dtype, int kv_dtype, const AttendArgs &a);
cudaError_t launch_attend_decode(int kv_dtype, const AttendArgs &a, cudaStream_t s);

// attend_tc.cu: tensor-core tiles of 128 query rows, for bf16 queries over bf16
// or e4m3 pages.
bool attend_tc_supported(int q_dtype, int kv_dtype, const AttendArgs &a);
cudaError_t launch_attend_tc(int kv_dtype, const AttendArgs &a, cudaStream_t s);

}  // namespace kvm
