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

template <int RB, int UNIT>
struct Line {
    // Keys that row tile r of a sequence sees (its last row sees the most).
    __host__ __device__ static __forceinline__ int keys(const SeqInfo &i, int gqa, int causal, int r) {
        if (!causal) return i.kv;
        const int row_end = min(i.q_len * gqa, (r + 1) * RB);
        return max(0, min(i.kv, i.kv - i.q_len + (row_end - 1) / gqa + 1));
    }
    __host__ __device__ static __forceinline__ int tiles(const SeqInfo &i, int gqa) {
        return (i.q_len * gqa + RB - 1) / RB;
    }
    __host__ __device__ static __forceinline__ int weight(const SeqInfo &i, int gqa, int causal, int r) {
        return max(1, (keys(i, gqa, causal, r) + UNIT - 1) / UNIT);
    }
    // A sequence's units by one head, as summed by the lane (few row tiles) or the
    // warp; every lane of the warp calls it with its sequence's lengths.
    __device__ static int64_t units(const SeqInfo &i, int gqa, int causal, int n_here, int lane) {
        const int n = tiles(i, gqa);
        int64_t w = 0;
        if (__all_sync(0xffffffffu, n <= 8)) {
            for (int r = 0; r < n; ++r) w += weight(i, gqa, causal, r);
            return w;
        }
        for (int x = 0; x < n_here; ++x) {
            SeqInfo j;
            j.q0 = 0;
            j.q_len = __shfl_sync(0xffffffffu, i.q_len, x);
            j.kv = __shfl_sync(0xffffffffu, i.kv, x);
            const int m = tiles(j, gqa);
            int64_t sum = 0;
            for (int r = lane; r < m; r += 32) sum += weight(j, gqa, causal, r);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == x) w = sum;
        }
        return w;
    }
    // Lays the line out: pre[s] = units of the sequences before s, pre[n_seqs] =
    // all, pre[n_seqs + 1] = the largest tile's, pre[n_seqs + 2] = the units every
    // tile is counted as, or 0 for its own (see run_units).  By one warp.
    template <bool PAD>
    __device__ static void lay_out(const AttendArgs &a, int64_t *pre, int n_ctas, int min_units) {
        const int lane = threadIdx.x & 31;
        int64_t run = 0, items = 0;
        int most = 1;
        for (int s0 = 0; s0 < a.b.n_seqs; s0 += 32) {
            const int s = s0 + lane;
            SeqInfo i{0, 0, 0};
            bool ok = true;
            if (s < a.b.n_seqs) i = seq_info(a.b, s, &ok);
            if (!ok) atomicOr(a.b.err, kErrBatch);
            const int n = tiles(i, a.gqa);
            if (n > 0) most = max(most, weight(i, a.gqa, a.causal, n - 1));   // the last sees most
            int64_t w = units(i, a.gqa, a.causal, min(32, a.b.n_seqs - s0), lane) * a.b.G;
            int64_t m = (int64_t)n * a.b.G;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t up = __shfl_up_sync(0xffffffffu, w, o);
                const int64_t um = __shfl_up_sync(0xffffffffu, m, o);
                if (lane >= o) {
                    w += up;
                    m += um;
                }
            }
            if (s < a.b.n_seqs) pre[s + 1] = run + w;
            run += __shfl_sync(0xffffffffu, w, 31);
            items += __shfl_sync(0xffffffffu, m, 31);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        int pad = 0;
        if (PAD) pad = padded_weight(items, run, most, n_ctas, min_units);
        if (pad) {
            // every tile counts alike: the prefix sums again, by tiles
            run = 0;
            for (int s0 = 0; s0 < a.b.n_seqs; s0 += 32) {
                const int s = s0 + lane;
                bool ok;
                int64_t w = s < a.b.n_seqs ? (int64_t)tiles(seq_info(a.b, s, &ok), a.gqa) * a.b.G * pad : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t up = __shfl_up_sync(0xffffffffu, w, o);
                    if (lane >= o) w += up;
                }
                if (s < a.b.n_seqs) pre[s + 1] = run + w;
                run += __shfl_sync(0xffffffffu, w, 31);
            }
        }
        if (lane == 0) {
            pre[0] = 0;
            pre[a.b.n_seqs + 1] = most;
            pre[a.b.n_seqs + 2] = pad;
        }
        __syncwarp();
    }
    // Where the row tiles are about equally long, they are all counted as `pad`
    // units, at least the longest one's: runs then begin and end at the same few
    // places of every tile (run_units).  A CTA meets one tile and not the ends of
    // two, and CTAs that share a head's keys read them at the same time (begun at
    // scattered keys they read 762 MB of a 134 MB cache).
    __host__ __device__ static int padded_weight(int64_t items, int64_t total, int most, int n_ctas,
                                                 int min_units) {
        if (items == 0 || total * 100 < items * most * 85) return 0;
        if (items * 4 < (int64_t)n_ctas * 3) {           // several CTAs to a tile
            const int least = most < min_units ? most : min_units;
            int parts = (int)(n_ctas / items);
            if (parts > most / least) parts = most / least;
            return (most + parts - 1) / parts * parts;
        }
        const int pad = (most + 11) / 12 * 12;
        return most >= 24 && total * 100 >= items * pad * 85 ? pad : 0;
    }
};

// a / b, both >= 0: 32-bit division where they fit (a 64-bit one takes about 10
// times as long, and a walk has several before its first load).
__host__ __device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((uint64_t)(a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}

// Units of one CTA's run: an equal share, but not so small that a tile's join
// costs more than its keys, unless whole tiles are smaller.  Of tiles counted
// alike, a CTA takes an equal part of one, or with more tiles than CTAs a
// multiple of a whole, a half, a third or a quarter: the first of these that
// gives away at most 1/16 of the share, else the one that gives away least.
__host__ __device__ __forceinline__ int64_t run_units(const AttendArgs &a, const int64_t *pre, int n_ctas,
                                                      int min_units) {
    const int64_t share = quotient(pre[a.b.n_seqs] + n_ctas - 1, n_ctas);
    const int64_t most = pre[a.b.n_seqs + 1], least = most < min_units ? most : min_units;
    const int64_t pad = pre[a.b.n_seqs + 2];
    if (!pad) return share > least ? share : least;
    const int64_t items = quotient(pre[a.b.n_seqs], pad);
    if (items * 4 < (int64_t)n_ctas * 3) {
        int64_t parts = quotient(n_ctas, items);
        if (parts > quotient(most, least)) parts = quotient(most, least);
        return quotient(pad, parts);
    }
    int64_t best = 0;
    for (int m = 1; m <= 4; ++m) {
        const int64_t part = pad / m, run = quotient(share + part - 1, part) * part;
        if (best == 0 || run < best) best = run;
        if (run * 16 <= share * 17) return run;
    }
    return best;
}

// A walk over one CTA's run of the line.
template <int RB, int UNIT>
struct Walk {
    using LN = Line<RB, UNIT>;
    int64_t x, end, per;     // position, end of the run, units of a run
    int s, g, r, n_tiles;    // sequence, kv head, row tile
    int u0, u1, w, pad;      // the segment's units [u0, u1) of the tile's w (pad: as counted)
    int nk;                  // keys the tile sees
    SeqInfo i;

    // per: units of one CTA's run.  False when the run is empty.
    __host__ __device__ __forceinline__ bool start(const AttendArgs &a, const int64_t *pre, int cta,
                                          int n_ctas, int min_units) {
        const int64_t total = pre[a.b.n_seqs];
        per = run_units(a, pre, n_ctas, min_units);
        if (cta * per >= total) return false;
        start_at(a, pre, cta * per, per);
        end = min(total, x + per);
        fill(a);
        return true;
    }
    // The position of one unit of the line; the run ends with that unit.
    __host__ __device__ __forceinline__ void start_at(const AttendArgs &a, const int64_t *pre,
                                                      int64_t at, int64_t per_) {
        x = at;
        per = per_;
        end = at + 1;
        int lo = 0, hi = a.b.n_seqs - 1;                // the last s with pre[s] <= x
        while (lo < hi) {
            const int m = (lo + hi + 1) >> 1;
            if (pre[m] <= x) lo = m; else hi = m - 1;
        }
        s = lo;
        pad = (int)pre[a.b.n_seqs + 2];
        bool ok;
        i = seq_info(a.b, s, &ok);
        n_tiles = LN::tiles(i, a.gqa);
        int64_t rem = x - pre[s];
        const int64_t per_head = quotient(pre[s + 1] - pre[s], a.b.G);
        g = (int)quotient(rem, per_head);
        rem -= g * per_head;
        r = 0;
        if (pad) {
            r = (int)quotient(rem, pad);
            rem -= (int64_t)r * pad;
            w = pad;
        } else {
            for (w = LN::weight(i, a.gqa, a.causal, 0); rem >= w; w = LN::weight(i, a.gqa, a.causal, r)) {
                rem -= w;
                ++r;
            }
        }
        u0 = (int)rem;
        fill(a);
    }
    __host__ __device__ __forceinline__ void fill(const AttendArgs &a) {
        nk = LN::keys(i, a.gqa, a.causal, r);
        u1 = (int)min((int64_t)w, u0 + (end - x));
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
                    n_tiles = LN::tiles(i, a.gqa);
                } while (n_tiles == 0);
            }
        }
        w = pad ? pad : LN::weight(i, a.gqa, a.causal, r);
        fill(a);
        return true;
    }
    // Key tiles of the segment: its units that hold keys.
    __host__ __device__ __forceinline__ int key_units() const {
        const int real = (nk + UNIT - 1) / UNIT;
        return (u1 < real ? u1 : real) - (u0 < real ? u0 : real);
    }
    __host__ __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == w; }
    // The first and last CTA that share the segment's tile.
    __host__ __device__ __forceinline__ int first_cta() const { return (int)quotient(x - u0, per); }
    __host__ __device__ __forceinline__ int last_cta() const { return (int)quotient(x - u0 + w - 1, per); }
};

// A CTA's two places for partial results: 1 for a tile that goes on in the next
// CTA and begins in this one, 0 for a tile that began in an earlier one.
__host__ __device__ __forceinline__ size_t part_slot(int cta, bool first) {
    return (size_t)cta * 2 + (first ? 1 : 0);
}

// CTAs and query rows of the largest records (the tensor-core tile kernel's).
constexpr int kTileMaxCtas = 160, kTileMaxRows = 256;
constexpr size_t kAttendPartFloats = (size_t)kTileMaxCtas * 2 * kTileMaxRows * 130;

// attend_decode.cu: up to kDecodeRows query rows of a kv head, the same types.
constexpr int kDecodeRows = 16;
bool attend_decode_supported(int q_dtype, int kv_dtype, const AttendArgs &a);
cudaError_t launch_attend_decode(int kv_dtype, const AttendArgs &a, cudaStream_t s);

// attend_tc.cu: tensor-core tiles of 128 query rows, for bf16 queries over bf16
// or e4m3 pages.
bool attend_tc_supported(int q_dtype, int kv_dtype, const AttendArgs &a);
cudaError_t launch_attend_tc(int kv_dtype, const AttendArgs &a, cudaStream_t s);

}  // namespace kvm
