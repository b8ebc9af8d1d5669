// Paged attention on the tensor cores (tcgen05): bf16 queries over bf16 or e4m3
// pages, for more query rows than a decoded token has.
//
// Per kv head, the query rows (token, head of the group) of a sequence are cut
// into tiles of 128; a unit of work is one tile of 128 keys (4 pages).  With S
// and O of a row tile in tensor memory, a unit is
//   S = Q K^T            M = 128 rows, N = 64 keys at a time, operands in shared memory
//   p = 2^(S c - m)      online softmax in log2 units, c = softmax_scale log2 e
//   O += P V             M = 128 rows, N = d; P (bf16) in tensor memory over S, V
//                        read from its [key][d] storage as an MN-major operand
// Two warpgroups of softmax threads, one thread a row, keep the tensor pipe fed:
// while one turns its S into P, the other's products run.
//   PAIR   the groups own two row tiles and meet every key tile together, so K and
//          V are fetched once for 256 rows;
//   SPLIT  (up to 128 rows, and little work: tile_p) both groups own the same rows
//          and take alternate key tiles; their two sums are joined at the end from
//          tensor memory.
// The maximum m is only moved when a tile exceeds it by more than 2^8 (the
// weights then stay below 2^8, well inside bf16 and float32), so O is rescaled a
// few times per row and not per tile.  Weights are rounded to bf16 for the
// product with V (held as the sum of two bf16 they would double those products, 515 of
// 1326 clocks of the tensor pipe that a row tile takes for a key tile); the running weight
// sums the unrounded float32.
//
// e4m3 pages: a fourth warpgroup turns each page's codes into the same swizzled
// tiles in f16 (exact, one instruction for two codes), and the products run in
// f16.  q is divided by a power of two per row first (row_exponent); k_scale goes into the
// factor of the page's scores; the weights times v_scale are kept in f16 against a
// reference of their own, 2^mp.  A weight p = 2^(x - m) becomes p w, w = 2^(log2
// v_scale + m - mp).  mp is kUp below the running maximum: p w is at most 2^(8 + 7), just
// inside f16, and the room is at its lower end, where many small weights can add up
// (what it rounds away is at most 2^-32 of the row's largest p w).  A w beyond float32
// only meets weights below 2^-110, and is bounded (a masked p of 0 times infinity is no
// number).
//
// Warps: 0 TMA producer, 1 and 3 MMA issuers (one for each group), 2 walks the
// CTA's run of the work line and hands its segments to the others, 4-7 and 8-11
// softmax, e4m3: 12-15 convert.  Registers move to the softmax warpgroups
// (setmaxnreg).  One CTA per SM walks its run of the call's work line
// (attend_common.cuh).
// What bounds it: a pair of row tiles on one key tile takes 2 x (811 + 515) =
// 2652 clocks of the tensor pipe as issued (the 64-key products read Q from shared
// memory twice, 405 clocks a half where 256 would do; N = 128 would need the columns
// that let a half be weighed while the other is made), and is passed in about
// 2760: 2048 query tokens over 34816 bf16 keys (1.7 TFLOP) in 1.18 ms, 1440
// TFLOP/s, 0.75 of the measured burst rate.  e4m3 pages add conversions and their
// shared-memory traffic, about 4050 clocks: 32 tokens over 65568 keys 74 us.  Small
// calls are bound by their start (9 thousand clocks to the first scores) and joins.
// Every wait is bounded to a second; on timeout the device error flag (bit 4) is
// raised and the CTA winds down: copies and products under way end before shared and
// tensor memory do.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include "attend_common.cuh"
#include "kvm_vec.cuh"
#include "tc_ptx.cuh"

namespace kvm {

namespace {

constexpr int TK = 128;                     // keys of a tile
constexpr int HK = TK / 2;                  // keys of half a tile
constexpr int TR = 128;                     // query rows of a tile
constexpr int kPagesPerTile = TK / kBlockTokens;
constexpr uint32_t kWaitNs = 1000000000u;   // 1 s
// Key tiles of a CTA's run at least, and what a join costs.  32 query tokens over
// 4096 keys took 18.2 us (e4m3 22.8); with 8 and 16, 22.4 (29.9).  Nine ragged
// sequences of d = 64 took 25.4, with 2 and 4, or 3 and 6, 34.8.
constexpr int kMinTiles = 4, kJoinTiles = 8;
constexpr float kMoveMax = 8.f;             // log2 units a tile may exceed m by
constexpr float kUp = 7.f;
constexpr float kMostW = 127.f;             // log2 of the largest w
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLeast = 1e-37f;            // of a score's factor: 0 * -inf is no mask
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kScales = 4;      // tiles whose pages' scales are kept (see Lay)

template <int D, bool E4, bool PAIR>
struct Lay {
    static constexpr int KA = D / 64;                  // 128-byte atoms of a row
    static constexpr int ATOM = TK * 128;              // one atom of a 128-row tile
    static constexpr int TILE = KA * ATOM;             // a K, V or Q tile in bf16
    static constexpr int Q_TILES = PAIR ? 2 : 1;
    // K / V tiles in flight: bf16 pages in as many slots as fit; of e4m3 pages
    // the raw tiles are what is in flight, the f16 ones a hand-over.  SPLIT needs
    // four: a group meets K of its next tile (two on) before it is done with V.
    static constexpr int SLOTS = E4 ? (D == 64 ? 6 : PAIR ? 3 : 4) : D == 64 ? 8 : PAIR ? 5 : 6;
    static constexpr int RAW = TK * D;                 // an e4m3 K or V tile
    static constexpr int RAW_SLOTS = E4 ? (D == 64 ? 8 : 4) : 0;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_KV = Q_TILES * TILE;
    static constexpr int OFF_RAW = OFF_KV + SLOTS * TILE;
    static constexpr int OFF_ML = OFF_RAW + RAW_SLOTS * RAW;       // SPLIT: group 1's sums
    static constexpr int OFF_QP = OFF_ML + (PAIR ? 0 : TR * 12);   // e4m3: the rows' powers of two
    static constexpr int OFF_BAR = OFF_QP + (E4 ? Q_TILES * TR * 4 : 0);
    static constexpr int SMEM = OFF_BAR + 1024;
    static constexpr int THREADS = E4 ? 512 : 384;
    static_assert(SLOTS * TILE >= kPreInts * 4, "prefix fits the ring");
    // The converter writes the scales of tile t over those of tile t - kScales.  It has
    // filled V of tile t - 1 before, use 2t - 1 of the ring, so every use up to 2t - 1 - SLOTS
    // has been consumed; V of tile t - kScales, use 2 (t - kScales) + 1, is one of them.
    static_assert(!E4 || SLOTS <= 2 * kScales - 2, "a tile's scales are read before they are replaced");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

// A bounded wait (tc::mbar_wait) of a whole warp, whose lanes leave it together: every
// branch goes by a vote.  Tensor memory is read and written by whole warps, so none may
// give up alone.  (A wait of each lane on its own and a vote at the end of the tile took
// 2048 tokens over 34816 e4m3 keys 1515 us against 1433, 32 over 65568 78 against 74.)
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    uint32_t t0 = 0;
    for (uint32_t n = 0; n < (1u << 30); ++n) {
        if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
        if ((n & 63) == 63) {
            const uint32_t t = tc::global_ns_lo();
            if (n == 63)
                t0 = t;
            else if (__any_sync(0xffffffffu, t - t0 > kWaitNs))
                return false;
        }
    }
    return false;
}

// One segment of the CTA's run, as the roles need it.
struct Seg {
    int T;                      // key tiles; 0: no key is seen; -1: the run is over
    int u0;                     // first tile
    int s, g, q0, q_len, kv;    // sequence, kv head, its rows and lengths
    int rbase;                  // first query row of the row tile
    int whole, first;           // all of the tile's keys; the tile begins in this CTA
    int c0, n_ctas;             // the CTAs that share the tile: the first, how many
};

constexpr int kSegs = 4;        // segments handed out ahead

struct Bars {
    uint64_t full[8], empty[8], raw_full[8], raw_empty[8], s_full[2][2], p_full[2][2], pv_done[2][2], sb_free[2], o_full[2], q_full[2];
    uint64_t seg_full[kSegs], seg_empty[kSegs], meet[2], v_clear[8], sc_full[kScales], drained[2];
    Seg seg[kSegs];
    float2 scale[kScales][kPagesPerTile];   // e4m3: (k_scale, v_scale) of a tile's pages
    uint32_t tmem;
    int go;
};
static_assert(sizeof(Bars) <= 1024, "barriers");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return r;
}
// (a, b) * c + d and (a, b) + (c, d), two float32 per instruction.
__device__ __forceinline__ float2 fma2(uint32_t a, uint32_t b, float c, float d) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 z, {%5, %5};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(a), "r"(b), "f"(c), "f"(d));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

__device__ __forceinline__ float2 mul2(float2 a, float c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(c));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two e4m3 codes (low 16 bits) as f16x2: exact.
__device__ __forceinline__ uint32_t e4m3_f16(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}

// 16 bytes to shared memory, zeros when `there` is false (nothing is read).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there = true) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}

// The largest biased exponent of 8 bf16, and the power of two that a query row
// with that largest exponent is divided by on its way to f16: its largest entry comes
// into [2^15, 2^16), the top of f16 (65504; a bf16 has 8 bits, 65280 is the most),
// so that entries down to 2^-32 of it are exact.  Kept where the factors of its
// scores stay normal float32.
__device__ __forceinline__ int max_exponent(uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t e = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) e = max(e, max(w[i] & 0x7F80u, (w[i] >> 16) & 0x7F80u));
    return (int)(e >> 7);
}
__device__ __forceinline__ int row_exponent(int biased) {
    return min(127, max(-101, biased - 127)) - 15;
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
__device__ __forceinline__ uint32_t f16_of_bf16(uint32_t two, float f) {
    return pack_f16(__uint_as_float(two << 16) * f, __uint_as_float(two & 0xFFFF0000u) * f);
}

// This CTA's share (the part-th of n_ctas) of a shared tile's rows, by 256 threads
// (t) that meet(): the parts' sums joined in CTA order.  The parts come through
// shared memory (`buf`, `bytes` of it; ml: 4 floats for each part of each row), all
// of them in flight at once, by loops that are short because they run once, out of
// a cold instruction cache: loaded into registers eight at a time, the joins of nine
// ragged sequences took 10 to 22 thousand cycles.
template <int D, int RB, class Meet>
__device__ __forceinline__ bool join_rows(const AttendArgs &a, const Seg &sh, int part, int t, uint8_t *buf,
                                          int bytes, float *ml, Meet meet) {
    constexpr int QUADS = D / 4;
    constexpr size_t REC = (size_t)RB * (D + 2);
    const int rows = min(RB, sh.q_len * a.gqa - sh.rbase), n = sh.n_ctas;
    const int r0 = rows * part / n, nr = rows * (part + 1) / n - r0;
    if (nr == 0) return true;
    auto record = [&](int p) { return a.part + part_slot(sh.c0 + p, p == 0) * REC; };
    // [part][row]: m and l; then the part's weight w, and w l
    float2 *ml_of = reinterpret_cast<float2 *>(ml), *w_of = ml_of + n * nr;
    // x / y by y_inv = ceil(2^32 / y), where x * y < 2^32 (an x is below 32 (RB + n),
    // a y at most RB); 2^32 is 0 for y = 1
    auto div = [](int x, uint32_t y_inv) { return y_inv ? (int)__umulhi((uint32_t)x, y_inv) : x; };
    const uint32_t nr_inv = ~0u / (uint32_t)nr + 1;
    const int most = min(QUADS, bytes / (n * nr * 16));  // quads of a row at a time
#pragma unroll 1
    for (int q0 = 0; q0 < QUADS; q0 += most) {
        const int nq = min(most, QUADS - q0);
#pragma unroll 4
        for (int x = t; x < n * nq * nr; x += 256) {     // [part][quad][row]
            const int y = div(x, nr_inv), p = div(y, ~0u / (uint32_t)nq + 1);
            copy16(tc::smem_u32(buf) + x * 16, reinterpret_cast<const float4 *>(record(p)) +
                                                   (size_t)(q0 + y - p * nq) * RB + r0 + x - y * nr);
        }
        if (q0 == 0) {
#pragma unroll 1
            for (int x = t; x < n * nr; x += 256) {
                const int p = div(x, nr_inv), r = r0 + x - p * nr;
                const float *rec = record(p) + (size_t)RB * D + r;
                ml_of[x] = make_float2(__ldcg(rec), __ldcg(rec + RB));
            }
            if (!meet()) return false;
#pragma unroll 1
            for (int x = t; x < n * nr; x += 256) {
                const int r = x - div(x, nr_inv) * nr;
                float m = -INFINITY;
#pragma unroll 4
                for (int p = 0; p < n; ++p) m = fmaxf(m, ml_of[p * nr + r].x);
                const float w = ex2(ml_of[x].x - (m == -INFINITY ? 0.f : m));
                w_of[x] = make_float2(w, w * ml_of[x].y);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (!meet()) return false;
#pragma unroll 1
        for (int x = t; x < nr * nq; x += 256) {
            const int q = div(x, nr_inv), r = x - q * nr;
            const float4 *v = reinterpret_cast<const float4 *>(buf) + x;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            float l = 0.f;
#pragma unroll 4
            for (int p = 0; p < n; ++p) {
                const float2 w = w_of[p * nr + r];
                const float4 y = v[p * nq * nr];
                l += w.y;
                o.x += w.x * y.x;
                o.y += w.x * y.y;
                o.z += w.x * y.z;
                o.w += w.x * y.w;
            }
            const float inv = l > 0.f ? __fdividef(1.f, l) : (l == 0.f ? 0.f : l);   // l < 2^32
            const int qrow = sh.rbase + r0 + r, tok = token_of(qrow, a.gqa_inv);
            const int h = sh.g * a.gqa + qrow - tok * a.gqa;
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) +
                                       (int64_t)(sh.q0 + tok) * a.out_stride + (int64_t)h * D + (q0 + q) * 4) =
                make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
            if (q0 + q == 0 && a.lse) {
                float m = -INFINITY;
#pragma unroll 1
                for (int p = 0; p < n; ++p) m = fmaxf(m, ml_of[p * nr + r].x);
                a.lse[(int64_t)(sh.q0 + tok) * a.H + h] = m == -INFINITY ? -INFINITY : m * kLn2 + logf(l);
            }
        }
        if (!meet()) return false;                       // shared memory is free
    }
    return true;
}

}  // namespace

template <int D, bool E4, bool PAIR>
__global__ void __launch_bounds__(Lay<D, E4, PAIR>::THREADS, 1)
attend_tile_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ AttendArgs a) {
    using LY = Lay<D, E4, PAIR>;
    constexpr int RB = PAIR ? 2 * TR : TR;
    constexpr int NS = LY::SLOTS, NR = E4 ? LY::RAW_SLOTS : NS;
    constexpr uint32_t kF16 = E4 ? tc::kIdescF16 : 0u;
    constexpr uint32_t kIdescS = tc::idesc_bf16_f32(TR, HK) & ~kF16;
    constexpr uint32_t kIdescO = (tc::idesc_bf16_f32(TR, D) & ~kF16) | tc::kIdescBMajorMn;
    // the swizzled tiles need 1024-byte alignment, which the start of shared
    // memory has while the kernel declares no static array
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *qs = smem + LY::OFF_Q, *kvs = smem + LY::OFF_KV, *raws = smem + LY::OFF_RAW;
    float2 *ml1 = reinterpret_cast<float2 *>(smem + LY::OFF_ML);
    float *mp1 = reinterpret_cast<float *>(ml1 + TR), *qpow = reinterpret_cast<float *>(smem + LY::OFF_QP);
    Bars *bar = reinterpret_cast<Bars *>(smem + LY::OFF_BAR);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;
    int *err = a.b.err;

    if (tc::smem_u32(smem) & 1023) {
        if (tid == 0) atomicOr(err, 4);
        return;
    }
    if (tid == 0) {
        for (int s = 0; s < 8; ++s) {
            tc::mbar_init(&bar->full[s], E4 ? 128 : 1);
            tc::mbar_init(&bar->empty[s], PAIR ? 2 : 1);
            tc::mbar_init(&bar->v_clear[s], 1);
            tc::mbar_init(&bar->raw_full[s], 1);
            tc::mbar_init(&bar->raw_empty[s], 128);
        }
        for (int s = 0; s < 2; ++s) {
            for (int h = 0; h < 2; ++h) {
                tc::mbar_init(&bar->s_full[s][h], 1);
                tc::mbar_init(&bar->p_full[s][h], 128);
                tc::mbar_init(&bar->pv_done[s][h], 1);
            }
            tc::mbar_init(&bar->sb_free[s], 128);
            tc::mbar_init(&bar->o_full[s], 1);
            tc::mbar_init(&bar->q_full[s], PAIR ? 128 : 256);
            tc::mbar_init(&bar->meet[s], 256);
            tc::mbar_init(&bar->drained[s], 1);
        }
        for (int s = 0; s < kScales; ++s) tc::mbar_init(&bar->sc_full[s], kPagesPerTile);
        for (int s = 0; s < kSegs; ++s) {
            tc::mbar_init(&bar->seg_full[s], 1);
            // producer, MMA issuers, eight softmax warps, four converting warps
            tc::mbar_init(&bar->seg_empty[s], E4 ? 15 : 11);
        }
        tc::fence_mbar_init();
    }
    if (warp == 0 && lane == 0 && !E4) {
        tc::prefetch_map(&kmap);
        tc::prefetch_map(&vmap);
    }
    if (warp == 1) {
        tc::tmem_alloc(&bar->tmem, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = bar->tmem;

    // Each role takes the segments in turn: open() returns false after a wait
    // that gave up; close() hands the place back (one arrival a role's warp).
    auto open = [&](int n) -> const Seg * {
        return tc::mbar_wait(&bar->seg_full[n % kSegs], (n / kSegs) & 1, kWaitNs)
                   ? &bar->seg[n % kSegs]
                   : nullptr;
    };
    auto close = [&](int n) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar->seg_empty[n % kSegs]);
    };

    if (wg == 0) {
        tc::regs_release<E4 ? 64 : 72>();
        if (warp == 0) {
            // ---------------------------------------------------- producer
            int n = 0;                                   // tiles issued: slot and parity
            uint64_t *fb = E4 ? bar->raw_full : bar->full, *eb = E4 ? bar->raw_empty : bar->empty;
            bool ok = true;
            for (int sg = 0; ok; ++sg) {
                const Seg *seg = open(sg);
                if (!__all_sync(0xffffffffu, seg != nullptr)) {
                    ok = false;
                    break;
                }
                int T = seg->T;
                const int u0 = seg->u0, kv_len = seg->kv, g = seg->g;
                const int32_t *table = a.b.page_table + (int64_t)seg->s * a.b.table_stride;
                close(sg);
                if (T < 0) break;
                if (a.stall && blockIdx.x == 0) T = n == 0;   // fault injection: the first key tile alone
                const int n_pages = (kv_len + kBlockTokens - 1) / kBlockTokens;
                int32_t ids = -1;
                for (int j = 0; j < T && ok; ++j) {
                    if (j % 8 == 0) {                    // the page numbers of 8 tiles at once
                        const int p = (u0 + j) * kPagesPerTile + lane;
                        ids = -1;
                        if (p < n_pages && j * kPagesPerTile + lane < T * kPagesPerTile) {
                            ids = table[p];
                            if (ids < 0 || ids >= a.b.n_pages) {
                                atomicOr(err, kErrBatch);
                                ids = -1;
                            }
                        }
                    }
                    const int32_t page =
                        __shfl_sync(0xffffffffu, ids, (j % 8) * kPagesPerTile + (lane & 3));
                    const uint32_t there = __ballot_sync(0xffffffffu, page >= 0) & 15u;
                    const int64_t head =
                        page < 0 ? -1 : ((int64_t)page * a.b.L + a.b.layer) * a.b.G + g;
                    for (int kv = 0; kv < 2; ++kv, ++n) {
                        const int s = n % NR;
                        if (!__all_sync(0xffffffffu,
                                        tc::mbar_wait(&eb[s], ((n / NR) & 1) ^ 1, kWaitNs))) {
                            ok = false;
                            break;
                        }
                        if (lane == 0)
                            tc::mbar_expect_tx(&fb[s], E4 ? __popc(there) * kBlockTokens * D : LY::TILE);
                        __syncwarp();
                        if (lane < kPagesPerTile) {
                            if constexpr (E4) {
                                if (page >= 0)
                                    tc::bulk_load(raws + s * LY::RAW + lane * kBlockTokens * D,
                                                  static_cast<const uint8_t *>(kv ? a.v_pages : a.k_pages) +
                                                      head * kBlockTokens * D,
                                                  kBlockTokens * D, &fb[s]);
                            } else {
                                // a page that is not there is read as zeros (out of the map)
#pragma unroll
                                for (int at = 0; at < LY::KA; ++at)
                                    tc::tma_load_3d(kvs + s * LY::TILE + at * LY::ATOM +
                                                        lane * kBlockTokens * 128,
                                                    kv ? &vmap : &kmap, &fb[s], at * 64, 0, (int)head);
                            }
                        }
                    }
                }
            }
            if (!ok && lane == 0) atomicOr(err, 4);
            // every copy issued lands before the CTA ends
            for (int i = max(0, n - NR); i < n; ++i)
                if (!tc::mbar_wait(&fb[i % NR], (i / NR) & 1, kWaitNs)) {
                    if (lane == 0) atomicOr(err, 4);
                    break;
                }
        } else if (warp != 2) {
            // ---------------------------------------------------- MMA issuers
            // One warp for each group: issuing blocks while the tensor pipe is full, so
            // one warp's waits hide behind the other's products.
            const int gr = warp == 1 ? 0 : 1;
            const uint32_t qbase = tc::smem_u32(qs) + (PAIR ? gr * LY::TILE : 0), kvbase = tc::smem_u32(kvs);
            const uint32_t ts = tmem + gr * TK, to = tmem + 256 + gr * 128;
            uint64_t *q_full = &bar->q_full[PAIR ? gr : 0];
            constexpr int step = PAIR ? 1 : 2;
            int n = 0;                                   // K / V tiles of earlier segments
            uint32_t qn = 0, pn = 0;                     // uses of q_full, p_full
            uint32_t cleared = 0;                        // parity of each slot's v_clear
            bool ok = true;
            // a warp-wide wait: false once one has given up
            auto wait = [&](uint64_t *b, uint32_t parity) {
                if (ok && !__all_sync(0xffffffffu, tc::mbar_wait(b, parity, kWaitNs))) ok = false;
                return ok;
            };
            for (int sg = 0; ok; ++sg) {
                const Seg *seg = open(sg);
                if (!__all_sync(0xffffffffu, seg != nullptr)) {
                    ok = false;
                    break;
                }
                // uniform over the warp, and known to be: descriptors stay in uniform registers
                const int T = __shfl_sync(0xffffffffu, seg->T, 0);
                const int left = __shfl_sync(0xffffffffu, seg->kv - seg->u0 * TK, 0);
                close(sg);
                if (T < 0) break;
                const int j0 = PAIR ? 0 : gr;
                // K tile j is use n + 2j of the ring, V tile j use n + 2j + 1.  A wait by
                // parity means its phase only if the one before is known to be over, so
                // every phase is waited for in turn, the other group's tiles (SPLIT) too.
                auto filled = [&](int use) { return wait(&bar->full[use % NS], (use / NS) & 1); };
                // scores of half of key tile j, into the 64 columns at `col`
                auto qk = [&](int j, int half, uint32_t col) {
                    const int s = (n + 2 * j) % NS;
                    tc::tc_fence_after();
                    const uint32_t qb = tc::desc_lo(qbase, 16);
                    const uint32_t kb = tc::desc_lo(kvbase + s * LY::TILE + half * HK * 128, 16);
                    if (tc::elect_one()) {
#pragma unroll
                        for (int x = 0; x < 4 * LY::KA; ++x) {
                            const uint32_t at = ((x >> 2) * LY::ATOM + (x & 3) * 32) >> 4;
                            tc::mma_16_ss(ts + col, qb + at, tc::kDescHiSw128, kb + at, tc::kDescHiSw128,
                                          kIdescS, x != 0);
                        }
                        tc::mma_commit(&bar->s_full[gr][half]);
                        if (half == 1) tc::mma_commit(&bar->empty[s]);
                    }
                    __syncwarp();
                };
                // the half's weights (32 columns at `col`) times its half of V tile j
                auto pv = [&](int j, int half, uint32_t col) {
                    const int s = (n + 2 * j + 1) % NS;
                    tc::tc_fence_after();
                    const uint32_t vb = tc::desc_lo(kvbase + s * LY::TILE + half * HK * 128, LY::ATOM);
                    if (tc::elect_one()) {
#pragma unroll
                        for (int x = 0; x < HK / 16; ++x)
                            tc::mma_16_ts(to, ts + col + x * 8, vb + (x * 16 * 128 >> 4), tc::kDescHiSw128,
                                          kIdescO, j != j0 || half != 0 || x != 0);
                        tc::mma_commit(&bar->pv_done[gr][half]);
                        if (half == 1) {
                            tc::mma_commit(&bar->empty[s]);
                            if (j + step >= T) tc::mma_commit(&bar->o_full[gr]);
                        }
                    }
                    __syncwarp();
                };
                // rows of V tile j behind the last key may hold anything (0 * NaN): one of
                // the tile's issuers clears them
                auto clear_tail = [&](int j) {
                    const int end = left - j * TK, s = (n + 2 * j + 1) % NS;
                    if (E4 || end >= TK || !(end & 31)) return true;
                    if (!PAIR || gr == 0) {
                        const int rows = 32 - (end & 31);
                        for (int i = lane; i < rows * LY::KA * 8; i += 32) {
                            const int row = end + i / (LY::KA * 8), c = i % (LY::KA * 8);
                            *reinterpret_cast<uint4 *>(kvs + s * LY::TILE + (c >> 3) * LY::ATOM + row * 128 +
                                                       (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                        }
                        tc::fence_proxy_async_smem();
                        __syncwarp();
                        if (PAIR && lane == 0) tc::mbar_arrive(&bar->v_clear[s]);
                    } else if (!wait(&bar->v_clear[s], cleared >> s & 1)) {
                        return false;
                    }
                    cleared ^= 1u << s;
                    return true;
                };
                if (T > 0 && wait(q_full, qn & 1)) {
                    ++qn;
                    if (j0 > 0 && (!filled(n) || !filled(n + 1))) break;
                    if (j0 < T) {
                        if (!filled(n + 2 * j0)) break;
                        qk(j0, 0, HK);
                        qk(j0, 1, 0);
                    }
                    // The 128 columns of S: a tile's first half lies where the last tile's
                    // second half was, free once that is in registers, and its second where
                    // the last tile's weights were.  So the next scores are under way while
                    // these are weighed.  Weights take the place of the first half.
                    uint32_t a_col = HK;
                    for (int j = j0; j < T; j += step, a_col ^= HK) {
                        const bool next = j + step < T;
                        if (!filled(n + 2 * j + 1) || !clear_tail(j)) break;
                        if (!wait(&bar->p_full[gr][0], pn & 1)) break;
                        pv(j, 0, a_col);
                        if (!PAIR && j + 1 < T && (!filled(n + 2 * j + 2) || !filled(n + 2 * j + 3))) break;
                        if (next && !filled(n + 2 * (j + step))) break;
                        if (!wait(&bar->sb_free[gr], pn & 1)) break;
                        if (next) qk(j + step, 0, a_col ^ HK);
                        if (!wait(&bar->p_full[gr][1], pn & 1)) break;
                        pv(j, 1, a_col + HK / 2);
                        if (next) qk(j + step, 1, a_col);
                        ++pn;
                    }
                }
                n += 2 * T;
            }
            // every product issued is done before tensor memory is freed, those of a segment
            // given up part-way too
            if (tc::elect_one()) tc::mma_commit(&bar->drained[gr]);
            __syncwarp();
            if (!tc::mbar_wait(&bar->drained[gr], 0, kWaitNs)) ok = false;
            if (!ok && lane == 0) atomicOr(err, 4);
        } else if (warp == 2) {
            // ---------------------------------------------------- the walk
            using W = Walk<RB, TK>;
            // the prefix sums live in the ring: its first copies follow the first segment
            int *pre = reinterpret_cast<int *>(kvs);
            const LineInfo li = W::LN::template lay_out<true>(a, pre, gridDim.x, kMinTiles, kJoinTiles);
            W k;
            bool any = k.start(a, pre, li, blockIdx.x);
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                for (int n = 0;; ++n) {
                    const int p = n % kSegs;
                    if (!tc::mbar_wait(&bar->seg_empty[p], ((n / kSegs) & 1) ^ 1, kWaitNs)) {
                        atomicOr(err, 4);
                        break;
                    }
                    Seg *seg = &bar->seg[p];
                    if (any) {
                        seg->T = k.key_units();
                        seg->u0 = k.u0;
                        seg->s = k.s;
                        seg->g = k.g;
                        seg->q0 = k.i.q0;
                        seg->q_len = k.i.q_len;
                        seg->kv = k.i.kv;
                        seg->rbase = k.r * RB;
                        seg->whole = k.whole();
                        seg->c0 = k.first_cta();
                        seg->n_ctas = k.last_cta() - seg->c0 + 1;
                        seg->first = seg->c0 == (int)blockIdx.x;
                    } else {
                        seg->T = -1;
                    }
                    tc::mbar_arrive(&bar->seg_full[p]);
                    if (!any) break;
                    any = k.next(a);
                }
        }
    } else if (wg <= 2) {
        // -------------------------------------------------------- softmax
        tc::regs_take<E4 ? 176 : 208>();
        const int gr = wg - 1, row = (warp & 3) * 32 + lane;              // row of the 128
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + gr * TK, to = tmem + lanes + 256 + gr * 128;
        // a negative scale turns the queries' sign, a scale of 0 clears them: c > 0
        const float c0 = a.scale == 0.f ? 1.f : fmaxf(fabsf(a.scale) * kLog2e, kLeast);
        const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
        const uint32_t keep = a.scale == 0.f ? 0u : 0xFFFFFFFFu;
        uint32_t sn = 0, on = 0, on1 = 0, met = 0, met1 = 0, qn = 0, tiles = 0;   // phases met, tiles passed
        bool ok = true;
        auto wait = [&](uint64_t *b, uint32_t parity) {
            if (!warp_wait(b, parity)) ok = false;
            return ok;
        };
        auto meet = [&](int which, uint32_t parity) {    // both groups
            tc::mbar_arrive(&bar->meet[which]);
            // (long waits: lanes polling on their own and one vote disturb the other group less;
            // 32 tokens over 32768 bf16 keys 41.8 us, with warp_wait 42.9)
            if (!__all_sync(0xffffffffu, tc::mbar_wait(&bar->meet[which], parity, kWaitNs))) ok = false;
            return ok;
        };
        Seg shared[2];                                   // the tiles shared with other CTAs
        int n_shared = 0;
        for (int sg = 0; ok; ++sg) {
            const Seg *seg = &bar->seg[sg % kSegs];
            if (!warp_wait(&bar->seg_full[sg % kSegs], (sg / kSegs) & 1)) {
                ok = false;
                break;
            }
            const int T = seg->T;
            if (T < 0) break;
            int vis;
            float c = c0;                                // E4: times the row's power of two
            {
                const int q_len = seg->q_len, kv = seg->kv, rows_all = q_len * a.gqa;
                const int base = seg->rbase + (PAIR ? gr * TR : 0);
                vis = a.causal ? min(kv, kv - q_len + token_of(base + row, a.gqa_inv) + 1) : kv;
                if (T > 0) {
                    // this group's query rows (SPLIT: its half) into the swizzled layout;
                    // nobody reads the last segment's any more
                    const int r0 = PAIR ? 0 : gr * (TR / 2);
                    uint8_t *dst = qs + (PAIR ? gr * LY::TILE : 0);
                    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q) +
                                               (int64_t)seg->q0 * a.q_stride +
                                               (int64_t)seg->g * a.gqa * D;
                    // all of a thread's chunks in flight at once, asked for by a short loop
                    // (four at a time through registers, they took 7 thousand cycles)
                    constexpr int CPR = D / 8, RPP = 128 / CPR;       // chunks of a row, rows of a pass
                    constexpr int N = (PAIR ? TR : TR / 2) / RPP;     // a thread's chunks
                    const int c16 = (tid & 127) % CPR, rr = r0 + (tid & 127) / CPR;
                    src += c16 * 8;
                    dst += (c16 >> 3) * LY::ATOM;
                    auto chunk = [&](int i) {
                        const int r = rr + i * RPP;
                        return reinterpret_cast<uint4 *>(dst + r * 128 + (((c16 & 7) ^ (r & 7)) << 4));
                    };
#pragma unroll 1
                    for (int i = 0; i < N; ++i) {
                        const int qrow = base + rr + i * RPP, t = token_of(qrow, a.gqa_inv);
                        copy16(tc::smem_u32(chunk(i)), src + (int64_t)t * a.q_stride + (qrow - t * a.gqa) * D,
                               qrow < rows_all);
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    if (E4 || flip || !keep) {
                        // each thread's own chunks: the scale's sign; E4: to f16
                        constexpr int B = 4;
#pragma unroll 1
                        for (int i0 = 0; i0 < N; i0 += B) {
                            uint4 x[B];
#pragma unroll
                            for (int i = 0; i < B; ++i) {
                                x[i] = *chunk(i0 + i);
                                x[i] = make_uint4((x[i].x ^ flip) & keep, (x[i].y ^ flip) & keep,
                                                  (x[i].z ^ flip) & keep, (x[i].w ^ flip) & keep);
                            }
                            if constexpr (E4) {
                                int e[B];
#pragma unroll
                                for (int i = 0; i < B; ++i) e[i] = max_exponent(x[i]);
#pragma unroll
                                for (int o = 1; o < CPR; o <<= 1)
#pragma unroll
                                    for (int i = 0; i < B; ++i)
                                        e[i] = max(e[i], __shfl_xor_sync(0xffffffffu, e[i], o));
#pragma unroll
                                for (int i = 0; i < B; ++i) {
                                    const float dn = pow2i(-row_exponent(e[i]));
                                    x[i] = make_uint4(f16_of_bf16(x[i].x, dn), f16_of_bf16(x[i].y, dn),
                                                      f16_of_bf16(x[i].z, dn), f16_of_bf16(x[i].w, dn));
                                    if (c16 == 0)
                                        qpow[(PAIR ? gr * TR : 0) + rr + (i0 + i) * RPP] =
                                            pow2i(row_exponent(e[i]));
                                }
                            }
#pragma unroll
                            for (int i = 0; i < B; ++i) *chunk(i0 + i) = x[i];
                        }
                    }
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive(&bar->q_full[PAIR ? gr : 0]);
                    if constexpr (E4) {                  // the power of two of this thread's row
                        if (!wait(&bar->q_full[PAIR ? gr : 0], qn & 1)) break;
                        c *= qpow[(PAIR ? gr * TR : 0) + row];
                    }
                    ++qn;
                }
                vis -= seg->u0 * TK;                     // from the segment's first key
            }
            // m: reference of the weights (log2).  E4: mp, that of the weights times
            // v_scale, which are what the product with V takes in f16; O is in units
            // of 2^mp.  Both move when a tile exceeds one of them by kMoveMax.
            float m = -INFINITY, mp = -INFINITY, l = 0.f;
            constexpr int step = PAIR ? 1 : 2;
            uint32_t a_col = HK;                         // as the issuer's
            // pv_done phases are met in turn, each before its half's weights are next
            // handed over; `early`: already met, to rescale O
            uint32_t early = 0;
            for (int j = PAIR ? 0 : gr; j < T && ok; j += step, a_col ^= HK, ++sn) {
                const bool head = j < step;              // the group's first tile of the segment
                if constexpr (E4) {
                    const uint32_t tile = tiles + j;
                    if (!warp_wait(&bar->sc_full[tile % kScales], (tile / kScales) & 1)) {
                        ok = false;
                        break;
                    }
                }
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    float kc[2], lv[2];                  // factor of a page's scores, log2 v_scale
                    if constexpr (E4) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 sc = bar->scale[(tiles + j) % kScales][2 * h + i];
                            kc[i] = fmaxf(c * sc.x, kLeast);
                            lv[i] = (float)((int)(__float_as_uint(sc.y) >> 23) - 127);
                        }
                    }
                    if (!warp_wait(&bar->s_full[gr][h], sn & 1)) {
                        ok = false;
                        break;
                    }
                    tc::tc_fence_after();
                    uint32_t s[HK];
                    const uint32_t sc = ts + (h == 0 ? a_col : a_col ^ HK);
                    tc::tmem_ld32_async(sc, s);
                    tc::tmem_ld32_async(sc + 32, s + 32);
#pragma unroll
                    for (int i = 0; i < HK; i += 16) tc::tmem_wait_ld(s + i);
                    if (h == 1) {
                        tc::tc_fence_before();
                        tc::mbar_arrive(&bar->sb_free[gr]);
                    }
                    const int seen = vis - j * TK - h * HK;
                    if (__any_sync(0xffffffffu, seen < HK)) {
#pragma unroll
                        for (int i = 0; i < HK; ++i)
                            if (i >= seen) s[i] = 0xFF800000u;
                    }
                    // The half is weighed against the m so far while its own maxima are
                    // taken (the exponentials leave issue slots free); in the rare one that
                    // exceeds m by kMoveMax, m moves and the half is weighed again.
                    bool settled = false;
                    const bool fresh = __any_sync(0xffffffffu, m == -INFINITY);
                    float sum = 0.f;
                    for (;;) {
                        if (!fresh || settled) {
                            const float off = m == -INFINITY ? 0.f : -m;
                            float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                // E4: from weights to what multiplies V's codes
                                const float w = E4 && m != -INFINITY ? ex2(fminf(lv[y] + m - mp, kMostW)) : 0.f;
                                uint32_t p[16];
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    float2 x = fma2(s[y * 32 + 2 * i], s[y * 32 + 2 * i + 1], E4 ? kc[y] : c,
                                                    off);
                                    x.x = ex2(x.x);
                                    x.y = ex2(x.y);
                                    part[i & 1] = add2(part[i & 1], x);
                                    if constexpr (E4) {
                                        x = mul2(x, w);
                                        p[i] = pack_f16(x.x, x.y);
                                    } else {
                                        p[i] = pack_bf16(x.x, x.y);
                                    }
                                }
                                tc::tmem_st16(ts + a_col + h * 32 + y * 16, p);
                            }
                            sum = (part[0].x + part[0].y) + (part[1].x + part[1].y);
                        }
                        if (settled) break;
                        float mx[8];                     // four of each page
#pragma unroll
                        for (int e = 0; e < 8; ++e) mx[e] = max3(__uint_as_float(s[e * 8]), s[e * 8 + 1], s[e * 8 + 2]);
#pragma unroll
                        for (int i = 3; i < 7; i += 2)
#pragma unroll
                            for (int e = 0; e < 8; ++e) mx[e] = max3(mx[e], s[e * 8 + i], s[e * 8 + i + 1]);
#pragma unroll
                        for (int e = 0; e < 8; ++e) mx[e] = fmaxf(mx[e], __uint_as_float(s[e * 8 + 7]));
                        const float top0 = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                        const float top1 = fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]));
                        float m_new, mp_new;
                        bool grow;
                        if constexpr (E4) {
                            const float x0 = top0 * kc[0], x1 = top1 * kc[1];
                            m_new = fmaxf(m, fmaxf(x0, x1));
                            mp_new = fmaxf(mp, fmaxf(x0 + lv[0], x1 + lv[1]) - kUp);
                            grow = m_new > m + kMoveMax || mp_new > mp + kMoveMax;
                        } else {
                            m_new = mp_new = fmaxf(m, fmaxf(top0, top1) * c);
                            grow = m_new > m + kMoveMax;
                        }
                        if (!fresh && !__any_sync(0xffffffffu, grow)) break;
                        const bool none = m == -INFINITY;
                        l *= none ? 0.f : ex2(m - m_new);
                        if (!head || h == 1) {
                            // O has to hold the products so far: those of the half before are
                            // not implied by these scores (the first half's of a tile: both
                            // of the last tile's).  The first product overwrites O.
                            if (h == 0) {
                                if (!(early & 1) && !warp_wait(&bar->pv_done[gr][0], (sn - 1) & 1)) ok = false;
                                if (!warp_wait(&bar->pv_done[gr][1], (sn - 1) & 1)) ok = false;
                                early = 3;
                            } else {
                                if (!warp_wait(&bar->pv_done[gr][0], sn & 1)) ok = false;
                                early |= 4;
                            }
                            tc::tc_fence_after();
                            const float f = none ? 0.f : ex2(mp - mp_new);
#pragma unroll 1
                            for (int i = 0; i < D; i += 16) {
                                uint32_t o[16];
                                tc::tmem_ld16_async(to + i, o);
                                tc::tmem_wait_ld(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tc::tmem_st16(to + i, o);
                            }
                        }
                        m = m_new;
                        mp = mp_new;
                        settled = true;
                    }
                    l += sum;
                    if (!head && !(early >> h & 1) && !warp_wait(&bar->pv_done[gr][h], (sn - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    tc::tmem_wait_st();
                    tc::tc_fence_before();
                    tc::mbar_arrive(&bar->p_full[gr][h]);
                }
                early >>= 2;
            }
            if (!ok) break;
            tiles += T;
            // ------------------------------------------------ the segment's end
            const bool mine = T > (PAIR ? 0 : gr);      // this group has an O
            if (mine) {
                if (!wait(&bar->o_full[gr], on & 1) ||
                    !(early & 1 || wait(&bar->pv_done[gr][0], (sn - 1) & 1)) ||
                    !wait(&bar->pv_done[gr][1], (sn - 1) & 1))
                    break;
                ++on;
            }
            // O to units of 2^m
            float f0 = E4 && m != -INFINITY ? ex2(mp - m) : 1.f, f1 = 0.f;
            if (!PAIR) {
                if (gr == 1) {
                    ml1[row] = make_float2(m, l);
                    if (E4) mp1[row] = f0;
                }
                if (!meet(0, met & 1)) break;
                if (gr == 0) {                          // group 0 writes the rows
                    const float2 o1 = ml1[row];
                    if (T > 1) {
                        if (!wait(&bar->o_full[1], on1 & 1)) break;
                        ++on1;
                    }
                    const float mm = fmaxf(m, o1.x), base = mm == -INFINITY ? 0.f : mm;
                    const float g0 = ex2(m - base), g1 = ex2(o1.x - base);
                    f0 *= g0;
                    f1 = E4 ? g1 * mp1[row] : g1;
                    l = l * g0 + o1.y * g1;
                    m = mm;
                }
            }
            const bool whole = seg->whole;
            if (PAIR || gr == 0) {
                tc::tc_fence_after();
                const int prow = (PAIR ? gr * TR : 0) + row, qrow = seg->rbase + prow;
                const bool live = qrow < seg->q_len * a.gqa;
                const int tok = token_of(qrow, a.gqa_inv), h = seg->g * a.gqa + qrow - tok * a.gqa;
                float *rec = a.part + part_slot(blockIdx.x, seg->first) * ((size_t)RB * (D + 2));
                if (whole) {
                    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
                    f0 *= inv;
                    f1 *= inv;
                    if (live && a.lse)
                        a.lse[(int64_t)(seg->q0 + tok) * a.H + h] =
                            m == -INFINITY ? -INFINITY : m * kLn2 + logf(l);
                } else if (live) {
                    rec[(size_t)RB * D + prow] = m;
                    rec[(size_t)RB * (D + 1) + prow] = l;
                }
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) +
                                     (int64_t)(seg->q0 + tok) * a.out_stride + (int64_t)h * D;
#pragma unroll 1
                for (int i = 0; i < D; i += 32) {
                    uint32_t o[32];
                    if (mine) {
                        tc::tmem_ld32_async(to + i, o);
                        tc::tmem_wait_ld(o);
                        tc::tmem_wait_ld(o + 16);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f0);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0;
                    }
                    if (!PAIR && T > 1) {
                        uint32_t o1[32];
                        tc::tmem_ld32_async(to + 128 + i, o1);
                        tc::tmem_wait_ld(o1);
                        tc::tmem_wait_ld(o1 + 16);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(
                                fmaf(__uint_as_float(o1[e]), f1, __uint_as_float(o[e])));
                    }
                    if (whole) {
                        if (live) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                float v[8];
#pragma unroll
                                for (int x = 0; x < 8; ++x) v[x] = __uint_as_float(o[e + x]);
                                *reinterpret_cast<uint4 *>(dst + i + e) =
                                    VecTraits<__nv_bfloat16>::pack(v);
                            }
                        }
                    } else if (live) {
                        // four columns of a row, rows adjacent
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<uint4 *>(rec + ((size_t)(i + e) / 4 * RB + prow) * 4) =
                                make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
                tc::tc_fence_before();
            }
            if (!whole) shared[n_shared++ & 1] = *seg;
            // SPLIT: Q and group 1's sums may be overwritten once both are here
            if (!PAIR || !whole) {
                if (!meet(1, met1 & 1)) break;
                ++met1;
                // every thread's part is written and met here: one releases them all
                if (!whole && tid == 128) {
                    __threadfence();
                    tc::red_release_gpu_add(a.count + seg->c0, 1);
                }
            }
            ++met;
            close(sg);
        }
        // ---------------------------------------------------- the shared tiles
        // Once all of a tile's CTAs have left their part, each joins a share of its
        // rows, the parts in CTA order.  All CTAs run at the same time (a cooperative
        // launch), so this waits for no CTA that has yet to start.
        for (int x = 0; x < n_shared && ok; ++x) {
            const Seg &sh = shared[x];
            int *count = a.count + sh.c0, *left = a.count + kAttendMaxCtas + sh.c0;
            if (tid == 128) {
                bool all = tc::ld_acquire_gpu(count) >= sh.n_ctas;
                const uint32_t t0 = tc::global_ns_lo();
                while (!all && tc::global_ns_lo() - t0 < kWaitNs) all = tc::ld_acquire_gpu(count) >= sh.n_ctas;
                __threadfence();                         // the parts, for the CTA that meets next
                bar->go = all;
                if (!all) atomicOr(err, 4);
            }
            if (!meet(1, met1++ & 1)) break;
            const bool all = bar->go != 0;
            auto met_all = [&] { return meet(1, met1++ & 1); };
            if (all && !join_rows<D, RB>(a, sh, blockIdx.x - sh.c0, tid - 128, kvs, NS * LY::TILE,
                                         reinterpret_cast<float *>(qs), met_all))
                break;
            if (!met_all()) break;                       // go and the counters are free
            if (tid == 128) {
                // the last CTA to leave readies the counters for the next call
                __threadfence();
                if (atomicAdd(left, 1) == sh.n_ctas - 1) {
                    *count = 0;
                    *left = 0;
                }
            }
        }
        if (!ok) {
            // what is under way lands before the CTA ends
            asm volatile("cp.async.wait_all;" ::: "memory");
            tc::tmem_wait_st();
            atomicOr(err, 4);
        }
    } else {
        // -------------------------------------------------------- e4m3 -> f16
        if constexpr (E4) {
            tc::regs_release<88>();
            const int w = warp & 3;                      // its page of the tile
            int n = 0;                                   // K / V tiles converted
            bool ok = true;
            for (int sg = 0; ok; ++sg) {
                const Seg *seg = open(sg);
                if (!__all_sync(0xffffffffu, seg != nullptr)) {
                    ok = false;
                    break;
                }
                const int T = seg->T, u0 = seg->u0, kv_len = seg->kv, g = seg->g;
                const int64_t table = (int64_t)seg->s * a.b.table_stride;
                close(sg);
                if (T < 0) break;
                float2 sc_of = make_float2(1.f, 1.f);    // lane i: of the page of tile 32 x + i
                int rows_of = 0;
                for (int j = 0; j < T && ok; ++j) {
                    if ((j & 31) == 0) {                 // the scales of 32 tiles at once
                        const int p = (u0 + j + lane) * kPagesPerTile + w;
                        rows_of = 0;
                        sc_of = make_float2(1.f, 1.f);
                        if (j + lane < T && p * kBlockTokens < kv_len) {
                            const int64_t page = a.b.page_table[table + p];
                            bool there = page >= 0 && page < a.b.n_pages;
                            if (a.k_scale) {
                                const int64_t r = a.b.scale_rows ? (int64_t)a.b.scale_rows[table + p] : page;
                                if (r >= 0 && r < a.b.n_scale_rows) {
                                    const size_t so = ((size_t)r * a.b.L + a.b.layer) * a.b.G + g;
                                    sc_of = make_float2(checked_scale(a.k_scale[so], err),
                                                        checked_scale(a.v_scale[so], err));
                                } else {
                                    atomicOr(err, kErrBatch);
                                    there = false;
                                }
                            }
                            if (there) rows_of = min(kBlockTokens, kv_len - p * kBlockTokens);
                        }
                    }
                    const int rows = __shfl_sync(0xffffffffu, rows_of, j & 31);
                    const float2 sc = make_float2(__shfl_sync(0xffffffffu, sc_of.x, j & 31),
                                                  __shfl_sync(0xffffffffu, sc_of.y, j & 31));
                    for (int kv = 0; kv < 2; ++kv, ++n) {
                        const int rs = n % NR, s = n % NS;
                        if (!__all_sync(0xffffffffu,
                                        tc::mbar_wait(&bar->raw_full[rs], (n / NR) & 1, kWaitNs) &&
                                            tc::mbar_wait(&bar->empty[s], ((n / NS) & 1) ^ 1, kWaitNs))) {
                            ok = false;
                            break;
                        }
                        if (kv == 0 && lane == 0) {
                            // the place of tile t - kScales is free (see Lay)
                            const int x = (n >> 1) % kScales;
                            bar->scale[x][w] = sc;
                            tc::mbar_arrive(&bar->sc_full[x]);
                        }
                        const uint8_t *src = raws + rs * LY::RAW + w * kBlockTokens * D;
                        uint8_t *dst = kvs + s * LY::TILE;
                        constexpr int CPR = D / 16;      // 16-byte pieces of a raw row
                        constexpr int N = kBlockTokens * CPR / 32;
                        uint4 in[N];
#pragma unroll
                        for (int i = 0; i < N; ++i)
                            in[i] = *reinterpret_cast<const uint4 *>(src + (i * 32 + lane) * 16);
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            const int at = i * 32 + lane, r = at / CPR, c = at % CPR;
                            const int key = w * kBlockTokens + r;
                            if (r >= rows) in[i] = make_uint4(0, 0, 0, 0);
                            const uint4 lo = make_uint4(e4m3_f16(in[i].x), e4m3_f16(in[i].x >> 16),
                                                        e4m3_f16(in[i].y), e4m3_f16(in[i].y >> 16));
                            const uint4 hi = make_uint4(e4m3_f16(in[i].z), e4m3_f16(in[i].z >> 16),
                                                        e4m3_f16(in[i].w), e4m3_f16(in[i].w >> 16));
                            // two 16-byte chunks of the row's atom; the lanes of the second
                            // atom write theirs in the other order (bank conflicts)
                            uint8_t *row = dst + (c >> 2) * LY::ATOM + key * 128;
                            const int c0 = (c & 3) * 2, odd = (c >> 2) & 1;
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int h = e ^ odd;
                                *reinterpret_cast<uint4 *>(row + (((c0 + h) ^ (key & 7)) << 4)) = h ? hi : lo;
                            }
                        }
                        tc::fence_proxy_async_smem();
                        tc::mbar_arrive(&bar->raw_empty[rs]);
                        tc::mbar_arrive(&bar->full[s]);
                    }
                }
            }
            if (!ok) atomicOr(err, 4);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- host side

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &qr) == cudaSuccess &&
            qr == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
    }();
    return fn;
}

// bf16 pages as [page, layer, kv head][32][d]; a box is 64 columns of one
// page's rows, and a negative first coordinate reads zeros.
bool page_map(CUtensorMap *m, const void *pages, int d, int64_t heads) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, kBlockTokens, (cuuint64_t)heads};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)kBlockTokens * d * 2};
    cuuint32_t box[3] = {64, kBlockTokens, 1}, estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(pages), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool E4, bool PAIR>
cudaError_t tile_t(const AttendArgs &a, cudaStream_t s) {
    using LY = Lay<D, E4, PAIR>;
    CUtensorMap kmap{}, vmap{};
    if (!E4) {
        const int64_t heads = a.b.n_pages * a.b.L * a.b.G;
        if (!page_map(&kmap, a.k_pages, D, heads) || !page_map(&vmap, a.v_pages, D, heads))
            return cudaErrorInvalidValue;
    }
    auto kern = attend_tile_kernel<D, E4, PAIR>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, LY::SMEM);
    if (e != cudaSuccess) return e;
    const int ctas = min(kTileMaxCtas, sm_count());
    AttendArgs args = a;
    void *params[] = {&kmap, &vmap, &args};
    // CTAs that share a tile wait for one another at the end: all run at once
    e = cudaLaunchCooperativeKernel((const void *)kern, dim3((unsigned)ctas), dim3(LY::THREADS), params,
                                    LY::SMEM, s);
    note_launch();
    return e;
}

template <int D, bool E4>
cudaError_t tile_p(const AttendArgs &a, cudaStream_t s) {
    // Pairs of row tiles fetch (and convert) K and V once for 256 rows; single row tiles
    // are passed in half the time, by both groups, and make twice as many pieces of
    // work.  Those win while there is an SM for each row tile and little work an SM
    // (as bounded by the batch: a call whose bounds are far above its lengths may get the
    // other form, with the same results), us for 8 kv heads of 6 query heads, d = 128:
    //   tokens, keys     bf16 pair / single      e4m3 pair / single
    //   32, 1024              20.8 / 15.5            27.2 / 23.1
    //   32, 4096              21.6 / 17.8            26.4 / 22.7
    //   256, 1024             22.5 / 16.3            29.4 / 25.3
    //   256, 2048             28.0 / 23.9            36.0 / 43.4
    //   256, 4096             36.1 / 39.4            46.5 / 72.9
    //   512, 1024             22.9 / 39.9            29.9 / 56.1
    // d = 64:
    //   32, 4096              18.1 / 15.6            21.6 / 18.1
    //   256, 1024             19.9 / 14.0            24.4 / 17.4
    //   256, 2048             23.9 / 20.1            28.1 / 26.3
    //   256, 4096             31.5 / 33.3            37.9 / 44.1
    //   512, 1024             20.1 / 34.5            25.0 / 41.7
    const int64_t of_seq = ((int64_t)a.b.max_q_len * a.gqa + TR - 1) / TR;
    const int64_t tiles =
        a.b.G * min(a.b.n_seqs * of_seq, (int64_t)a.b.n_tokens * a.gqa / TR + a.b.n_seqs);
    const int64_t units = (a.b.max_kv_len + TK - 1) / TK * tiles;
    const int sms = sm_count();
    const bool single = of_seq == 1 || (tiles <= sms && units <= (int64_t)sms * (E4 ? 6 : 12));
    return single ? tile_t<D, E4, false>(a, s) : tile_t<D, E4, true>(a, s);
}

}  // namespace

bool attend_tc_supported(int q_dtype, int kv_dtype, const AttendArgs &a) {
    // the tensor map's head coordinate is a 32-bit int
    return q_dtype == BF16 && (kv_dtype == BF16 || kv_dtype == E4M3) &&
           (int64_t)a.b.max_q_len * a.gqa > 16 &&
           (kv_dtype == E4M3 ||
            (a.b.n_pages >= 1 && a.b.n_pages <= INT32_MAX / ((int64_t)a.b.L * a.b.G) &&
             encode_fn() != nullptr));
}

cudaError_t launch_attend_tc(int kv_dtype, const AttendArgs &a, cudaStream_t s) {
    if (kv_dtype == E4M3) return a.d == 128 ? tile_p<128, true>(a, s) : tile_p<64, true>(a, s);
    return a.d == 128 ? tile_p<128, false>(a, s) : tile_p<64, false>(a, s);
}

}  // namespace kvm
