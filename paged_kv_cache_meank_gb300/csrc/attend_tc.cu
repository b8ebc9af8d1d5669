// Paged attention on the tensor cores (tcgen05): bf16 queries over bf16 or e4m3
// pages, for more query rows than a decoded token has.
//
// Per kv head, the query rows (token, head of the group) of a sequence are cut
// into tiles of 128; a unit of work is one tile of 128 keys (4 pages).  With S
// and O of a row tile in tensor memory, a unit is
//   S = Q K^T            M = 128 rows, N = 128 keys, both operands in shared memory
//   p = 2^(S c - m)      online softmax in log2 units, c = softmax_scale log2 e
//   O += P V             M = 128 rows, N = d; P (bf16) in tensor memory over S, V
//                        read from its [key][d] storage as an MN-major operand
// Two warpgroups of softmax threads, one thread a row, keep the tensor pipe fed:
// while one turns its S into P, the other's products run.
//   PAIR   (more than 128 rows): the groups own two row tiles and meet every key
//          tile together, so K and V are fetched once for 256 rows;
//   SPLIT  (up to 128 rows): both groups own the same rows and take alternate key
//          tiles; their two sums are joined at the end from tensor memory.
// The maximum m is only moved when a tile exceeds it by more than 2^8 (the
// weights then stay below 2^8, well inside bf16 and float32), so O is rescaled a
// few times per row and not per tile.  Weights are rounded to bf16 for the
// product with V; the running weight sums the unrounded float32.
//
// e4m3 pages: a fourth warpgroup turns each page into the same swizzled bf16
// tiles; with power-of-two scales every value is exact in bf16, so the rest of
// the kernel is the bf16 one.
//
// Warps: 0 TMA producer, 1 MMA issuer, 2 walks the CTA's run of the work line
// and hands its segments to the others, 4-7 and 8-11 softmax, e4m3:
// 12-15 convert.  Registers move to the softmax warpgroups (setmaxnreg).  One CTA
// per SM walks an equal run of the call's work line (attend_common.cuh).
// Every wait is bounded to a second; on timeout the device error flag (bit 4) is
// raised and the CTA winds down as the scoring kernels do.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include "attend_common.cuh"
#include "kvm_vec.cuh"
#include "tc_ptx.cuh"

namespace kvm {

namespace {

constexpr int TK = 128;                     // keys of a tile
constexpr int TR = 128;                     // query rows of a tile
constexpr int kPagesPerTile = TK / kBlockTokens;
constexpr uint32_t kWaitNs = 1000000000u;   // 1 s
constexpr float kMoveMax = 8.f;             // log2 units a tile may exceed m by
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D, bool E4>
struct Lay {
    static constexpr int KA = D / 64;                  // 128-byte atoms of a row
    static constexpr int ATOM = TK * 128;              // one atom of a 128-row tile
    static constexpr int TILE = KA * ATOM;             // a K, V or Q tile in bf16
    // K / V tiles in flight: bf16 pages in as many slots as fit; of e4m3 pages
    // the raw tiles are what is in flight, the bf16 ones a hand-over
    static constexpr int SLOTS = E4 ? 3 : D == 64 ? 8 : 5;
    static constexpr int RAW = TK * D;                 // an e4m3 K or V tile
    static constexpr int RAW_SLOTS = E4 ? (D == 64 ? 8 : 4) : 0;
    static constexpr int OFF_Q = 0;                    // two row tiles
    static constexpr int OFF_KV = 2 * TILE;
    static constexpr int OFF_RAW = OFF_KV + SLOTS * TILE;
    static constexpr int OFF_ML = OFF_RAW + RAW_SLOTS * RAW;       // SPLIT: (m, l) of group 1
    static constexpr int OFF_BAR = OFF_ML + TR * 8;
    static constexpr int SMEM = 1024 + OFF_BAR + 768;
    static constexpr int THREADS = E4 ? 512 : 384;
    static_assert(SLOTS * TILE >= (kMaxSeqs + 1) * 8, "prefix fits the ring");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

// One segment of the CTA's run, as the roles need it.
struct Seg {
    int T;                      // key tiles; 0: no key is seen; -1: the run is over
    int u0;                     // first tile
    int s, g, q0, q_len, kv;    // sequence, kv head, its rows and lengths
    int rbase;                  // first query row of the row tile
    int whole, first;           // all of the tile's keys; the tile begins in this CTA
};

constexpr int kSegs = 4;        // segments handed out ahead

struct Bars {
    uint64_t full[8], empty[8], raw_full[8], raw_empty[8], s_full[2], p_full[2], o_full[2], q_full[2];
    uint64_t seg_full[kSegs], seg_empty[kSegs], meet[2];
    Seg seg[kSegs];
    uint32_t tmem;
};
static_assert(sizeof(Bars) <= 768, "barriers");

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

// Two e4m3 codes in bytes 1 and 3 of t (bytes 0 and 2 zero) as bf16x2 times
// mul.  The code's exponent and mantissa land in bf16's as a value 2^-120 times
// its own (subnormals too), which mul restores together with the block's scale:
// exact for every code and every power-of-two scale that keeps bf16's range.
__device__ __forceinline__ uint32_t e4m3_bf16(uint32_t t, __nv_bfloat162 up, __nv_bfloat162 scale) {
    const uint32_t r = (t & 0x80008000u) | ((t >> 4) & 0x07F007F0u);
    __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162 *>(&r);
    v = __hmul2(__hmul2(v, up), scale);
    return *reinterpret_cast<uint32_t *>(&v);
}

}  // namespace

template <int D, bool E4, bool PAIR>
__global__ void __launch_bounds__(Lay<D, E4>::THREADS, 1)
attend_tile_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ AttendArgs a, int min_units) {
    using LY = Lay<D, E4>;
    constexpr int RB = PAIR ? 2 * TR : TR;
    constexpr int NS = LY::SLOTS, NR = E4 ? LY::RAW_SLOTS : NS;
    constexpr uint32_t kIdescS = tc::idesc_bf16_f32(TR, TK);
    constexpr uint32_t kIdescO = tc::idesc_bf16_f32(TR, D) | tc::kIdescBMajorMn;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *qs = smem + LY::OFF_Q, *kvs = smem + LY::OFF_KV, *raws = smem + LY::OFF_RAW;
    float2 *ml1 = reinterpret_cast<float2 *>(smem + LY::OFF_ML);
    Bars *bar = reinterpret_cast<Bars *>(smem + LY::OFF_BAR);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;
    int *err = a.b.err;

    if (tid == 0) {
        for (int s = 0; s < 8; ++s) {
            tc::mbar_init(&bar->full[s], E4 ? 128 : 1);
            tc::mbar_init(&bar->empty[s], 1);
            tc::mbar_init(&bar->raw_full[s], 1);
            tc::mbar_init(&bar->raw_empty[s], 128);
        }
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(&bar->s_full[s], 1);
            tc::mbar_init(&bar->p_full[s], 128);
            tc::mbar_init(&bar->o_full[s], 1);
            tc::mbar_init(&bar->q_full[s], PAIR ? 128 : 256);
            tc::mbar_init(&bar->meet[s], 256);
        }
        for (int s = 0; s < kSegs; ++s) {
            tc::mbar_init(&bar->seg_full[s], 1);
            // producer, MMA issuer, eight softmax warps, four converting warps
            tc::mbar_init(&bar->seg_empty[s], E4 ? 14 : 10);
        }
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(&bar->tmem, 512);
        tc::tmem_relinquish();
    }
    using W = Walk<RB, TK>;
    {
        // the prefix sums live in the ring until the walk has started
        int64_t *pre = reinterpret_cast<int64_t *>(kvs);
        W::LN::lay_out(a, pre);
    }
    W k;
    bool any = false;
    if (tid == 64)
        any = k.start(a, reinterpret_cast<const int64_t *>(kvs), blockIdx.x, gridDim.x, min_units);
    tc::fence_proxy_async_smem();                        // before the ring's first copies
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = bar->tmem;
    tc::launch_dependents();

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
                const int T = seg->T, u0 = seg->u0, kv_len = seg->kv, g = seg->g;
                const int32_t *table = a.b.page_table + (int64_t)seg->s * a.b.table_stride;
                close(sg);
                if (T < 0) break;
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
        } else if (warp == 1) {
            // ---------------------------------------------------- MMA issuer
            const uint32_t qbase = tc::smem_u32(qs), kvbase = tc::smem_u32(kvs);
            int n = 0;                                   // K / V tiles of earlier segments
            uint32_t qn = 0, pn[2] = {0, 0};             // uses of q_full, p_full
            uint32_t on[2] = {0, 0};                     // segments that ended in o_full
            bool ok = true;
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
                if (T == 0) continue;
                // K tile j is use n + 2j of the ring, V tile j use n + 2j + 1
                auto qk = [&](int gr, int j, bool first) {
                    const int use = n + 2 * j, s = use % NS;
                    if (!wait(&bar->full[s], (use / NS) & 1)) return;
                    if (first && !wait(&bar->q_full[gr], qn & 1)) return;
                    tc::tc_fence_after();
                    const uint32_t qb = tc::desc_lo(qbase + (PAIR ? gr * LY::TILE : 0), 16);
                    const uint32_t kb = tc::desc_lo(kvbase + s * LY::TILE, 16);
                    if (tc::elect_one()) {
#pragma unroll
                        for (int x = 0; x < 4 * LY::KA; ++x) {
                            const uint32_t at = ((x >> 2) * LY::ATOM + (x & 3) * 32) >> 4;
                            tc::mma_16_ss(tmem + gr * TK, qb + at, tc::kDescHiSw128, kb + at,
                                          tc::kDescHiSw128, kIdescS, x != 0);
                        }
                        if (!PAIR || gr == 1) tc::mma_commit(&bar->empty[s]);
                        tc::mma_commit(&bar->s_full[gr]);
                    }
                    __syncwarp();
                };
                auto pv = [&](int gr, int j, bool first, bool last) {
                    const int use = n + 2 * j + 1, s = use % NS;
                    if (!wait(&bar->full[s], (use / NS) & 1)) return;
                    if (!E4 && (!PAIR || gr == 0)) {
                        // rows behind the last key may hold anything (0 * NaN): clear them
                        const int end = left - j * TK;
                        if (end < TK && (end & 31)) {
                            const int rows = 32 - (end & 31);
                            for (int i = lane; i < rows * LY::KA * 8; i += 32) {
                                const int row = end + i / (LY::KA * 8), c = i % (LY::KA * 8);
                                *reinterpret_cast<uint4 *>(kvs + s * LY::TILE + (c >> 3) * LY::ATOM +
                                                           row * 128 + (c & 7) * 16) =
                                    make_uint4(0, 0, 0, 0);
                            }
                            tc::fence_proxy_async_smem();
                            __syncwarp();
                        }
                    }
                    if (!wait(&bar->p_full[gr], pn[gr] & 1)) return;
                    ++pn[gr];
                    tc::tc_fence_after();
                    const uint32_t vb = tc::desc_lo(kvbase + s * LY::TILE, LY::ATOM);
                    if (tc::elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < TK / 16; ++kk)
                            tc::mma_16_ts(tmem + 256 + gr * 128, tmem + gr * TK + kk * 8,
                                          vb + (kk * 16 * 128 >> 4), tc::kDescHiSw128, kIdescO,
                                          !first || kk != 0);
                        if (!PAIR || gr == 1) tc::mma_commit(&bar->empty[s]);
                        if (last) tc::mma_commit(&bar->o_full[gr]);
                    }
                    __syncwarp();
                    if (last) ++on[gr];
                };
                if (PAIR) {
                    qk(0, 0, true);
                    if (ok) qk(1, 0, true);
                    for (int j = 0; j < T && ok; ++j)
                        for (int gr = 0; gr < 2 && ok; ++gr) {
                            pv(gr, j, j == 0, j == T - 1);
                            if (ok && j + 1 < T) qk(gr, j + 1, false);
                        }
                } else {
                    qk(0, 0, true);
                    if (ok && T > 1) qk(1, 1, false);
                    for (int j = 0; j < T && ok; ++j) {
                        const int gr = j & 1;
                        pv(gr, j, j < 2, j + 2 >= T);
                        if (ok && j + 2 < T) qk(gr, j + 2, false);
                    }
                }
                ++qn;
                n += 2 * T;
            }
            if (!ok && lane == 0) atomicOr(err, 4);
            // the last commits cover every MMA issued: done before TMEM is freed
            for (int gr = 0; gr < 2; ++gr)
                if (on[gr] > 0 && !tc::mbar_wait(&bar->o_full[gr], (on[gr] - 1) & 1, kWaitNs))
                    if (lane == 0) atomicOr(err, 4);
        } else if (warp == 2 && lane == 0) {
            // ---------------------------------------------------- the walk
            for (int n = 0;; ++n) {
                const int p = n % kSegs;
                if (!tc::mbar_wait(&bar->seg_empty[p], ((n / kSegs) & 1) ^ 1, kWaitNs)) {
                    atomicOr(err, 4);
                    break;
                }
                Seg *seg = &bar->seg[p];
                if (any) {
                    seg->T = k.nk > 0 ? k.u1 - k.u0 : 0;
                    seg->u0 = k.u0;
                    seg->s = k.s;
                    seg->g = k.g;
                    seg->q0 = k.i.q0;
                    seg->q_len = k.i.q_len;
                    seg->kv = k.i.kv;
                    seg->rbase = k.r * RB;
                    seg->whole = k.whole();
                    seg->first = k.first_cta() == (int)blockIdx.x;
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
        const float c = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
        uint32_t sn = 0, on = 0, on1 = 0, met = 0;
        bool ok = true;
        auto meet = [&](int which) {                     // both groups (SPLIT)
            tc::mbar_arrive(&bar->meet[which]);
            ok = tc::mbar_wait(&bar->meet[which], met & 1, kWaitNs);
            return ok;
        };
        for (int sg = 0; ok; ++sg) {
            const Seg *seg = open(sg);
            if (seg == nullptr) {
                ok = false;
                break;
            }
            const int T = seg->T;
            if (T < 0) break;
            int vis;
            {
                const int q_len = seg->q_len, kv = seg->kv, rows_all = q_len * a.gqa;
                const int base = seg->rbase + (PAIR ? gr * TR : 0);
                vis = a.causal ? min(kv, kv - q_len + (base + row) / a.gqa + 1) : kv;
                if (T > 0) {
                    // this group's query rows (SPLIT: its half) into the swizzled layout;
                    // nobody reads the last segment's any more
                    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
                    const uint32_t keep = a.scale == 0.f ? 0u : 0xFFFFFFFFu;
                    const int r0 = PAIR ? 0 : gr * (TR / 2), n_rows = PAIR ? TR : TR / 2;
                    uint8_t *dst = qs + (PAIR ? gr * LY::TILE : 0);
                    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q) +
                                               (int64_t)seg->q0 * a.q_stride +
                                               (int64_t)seg->g * a.gqa * D;
                    for (int i = tid & 127; i < n_rows * (D / 8); i += 128) {
                        const int r = r0 + i / (D / 8), c16 = i % (D / 8), qrow = base + r;
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (qrow < rows_all) {
                            const int t = qrow / a.gqa, h = qrow - t * a.gqa;
                            v = __ldg(reinterpret_cast<const uint4 *>(src + (int64_t)t * a.q_stride +
                                                                      h * D + c16 * 8));
                            v.x = (v.x ^ flip) & keep;
                            v.y = (v.y ^ flip) & keep;
                            v.z = (v.z ^ flip) & keep;
                            v.w = (v.w ^ flip) & keep;
                        }
                        *reinterpret_cast<uint4 *>(dst + (c16 >> 3) * LY::ATOM + r * 128 +
                                                   (((c16 & 7) ^ (r & 7)) << 4)) = v;
                    }
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive(&bar->q_full[PAIR ? gr : 0]);
                }
                vis -= seg->u0 * TK;                     // from the segment's first key
            }
            float m = -INFINITY, l = 0.f;
            constexpr int step = PAIR ? 1 : 2;
            for (int j = PAIR ? 0 : gr; j < T; j += step) {
                if (!tc::mbar_wait(&bar->s_full[gr], sn & 1, kWaitNs)) {
                    ok = false;
                    break;
                }
                ++sn;
                tc::tc_fence_after();
                uint32_t s[TK];
#pragma unroll
                for (int i = 0; i < TK; i += 32) tc::tmem_ld32_async(ts + i, s + i);
#pragma unroll
                for (int i = 0; i < TK; i += 16) tc::tmem_wait_ld(s + i);
                if (__any_sync(0xffffffffu, (j + 1) * TK > vis)) {
                    const int seen = vis - j * TK;
#pragma unroll
                    for (int i = 0; i < TK; ++i)
                        if (i >= seen) s[i] = 0xFF800000u;
                }
                float mx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) mx[i] = __uint_as_float(s[i]);
#pragma unroll
                for (int i = 4; i < 124; i += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[i + e], s[i + 4 + e]);
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], __uint_as_float(s[124 + e]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                const float m_new = fmaxf(m, top);
                const bool grow = m_new > m + kMoveMax || (m == -INFINITY && m_new > m);
                if (__any_sync(0xffffffffu, grow)) {
                    // s_full follows every earlier product of this thread's group, so O
                    // is complete; the first tile's O is overwritten, not added to
                    const float f = m == -INFINITY ? 0.f : ex2(m - m_new);
                    l *= f;
                    if (j >= step) {
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
                }
                const float off = m == -INFINITY ? 0.f : -m;
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int h = 0; h < TK / 32; ++h) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 x = fma2(s[h * 32 + 2 * i], s[h * 32 + 2 * i + 1], c, off);
                        x.x = ex2(x.x);
                        x.y = ex2(x.y);
                        sum[i & 1] = add2(sum[i & 1], x);
                        p[i] = pack_bf16(x.x, x.y);
                    }
                    tc::tmem_st16(ts + h * 16, p);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tc::tmem_wait_st();
                tc::tc_fence_before();
                tc::mbar_arrive(&bar->p_full[gr]);
            }
            if (!ok) break;
            // ------------------------------------------------ the segment's end
            const bool mine = T > (PAIR ? 0 : gr);      // this group has an O
            if (mine) {
                if (!tc::mbar_wait(&bar->o_full[gr], on & 1, kWaitNs)) {
                    ok = false;
                    break;
                }
                ++on;
            }
            float f0 = 1.f, f1 = 0.f;
            if (!PAIR) {
                if (gr == 1) ml1[row] = make_float2(m, l);
                if (!meet(0)) break;
                if (gr == 0) {                          // group 0 writes the rows
                    const float2 o1 = ml1[row];
                    if (T > 1) {
                        if (!tc::mbar_wait(&bar->o_full[1], on1 & 1, kWaitNs)) {
                            ok = false;
                            break;
                        }
                        ++on1;
                    }
                    const float mm = fmaxf(m, o1.x), base = mm == -INFINITY ? 0.f : mm;
                    f0 = ex2(m - base);
                    f1 = ex2(o1.x - base);
                    l = l * f0 + o1.y * f1;
                    m = mm;
                }
            }
            if (PAIR || gr == 0) {
                tc::tc_fence_after();
                const bool whole = seg->whole;
                const int prow = (PAIR ? gr * TR : 0) + row, qrow = seg->rbase + prow;
                const bool live = qrow < seg->q_len * a.gqa;
                const int tok = qrow / a.gqa, h = seg->g * a.gqa + qrow - tok * a.gqa;
                float *rec = a.part + part_slot(blockIdx.x, seg->first) * ((size_t)RB * (D + 2));
                const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) +
                                     (int64_t)(seg->q0 + tok) * a.out_stride + (int64_t)h * D;
                if (whole) {
                    if (live && a.lse)
                        a.lse[(int64_t)(seg->q0 + tok) * a.H + h] =
                            m == -INFINITY ? -INFINITY : m * kLn2 + logf(l);
                } else {
                    rec[(size_t)RB * D + prow] = m;
                    rec[(size_t)RB * (D + 1) + prow] = l;
                }
#pragma unroll 1
                for (int i = 0; i < D; i += 32) {
                    uint32_t o[32];
                    if (mine) {
                        tc::tmem_ld32_async(to + i, o);
                        tc::tmem_wait_ld(o);
                        tc::tmem_wait_ld(o + 16);
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
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * f0 +
                                                   __uint_as_float(o1[e]) * f1);
                    }
                    if (whole) {
                        if (live) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                float v[8];
#pragma unroll
                                for (int x = 0; x < 8; ++x) v[x] = __uint_as_float(o[e + x]) * inv;
                                *reinterpret_cast<uint4 *>(dst + i + e) =
                                    VecTraits<__nv_bfloat16>::pack(v);
                            }
                        }
                    } else {
                        // four columns of a row, rows adjacent
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<uint4 *>(rec + ((size_t)(i + e) / 4 * RB + prow) * 4) =
                                make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
                tc::tc_fence_before();
            }
            // SPLIT: Q and group 1's sums may be overwritten once both are here
            if (!PAIR) {
                if (!meet(1)) break;
                ++met;
            }
            close(sg);
        }
        if (!ok) atomicOr(err, 4);
    } else {
        // -------------------------------------------------------- e4m3 -> bf16
        if constexpr (E4) {
            tc::regs_release<88>();
            const int w = warp & 3;                      // its page of the tile
            int n = 0;                                   // K / V tiles converted
            bool ok = true;
            const __nv_bfloat162 up = __float2bfloat162_rn(__uint_as_float((120 + 127) << 23));
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
                float ks = 1.f, vs = 1.f;                // lane i: of the page of tile 32 x + i
                int rows_of = 0;
                for (int j = 0; j < T && ok; ++j) {
                    if ((j & 31) == 0) {                 // the scales of 32 tiles at once
                        const int p = (u0 + j + lane) * kPagesPerTile + w;
                        rows_of = 0;
                        if (j + lane < T && p * kBlockTokens < kv_len) {
                            const int64_t page = a.b.page_table[table + p];
                            bool there = page >= 0 && page < a.b.n_pages;
                            if (a.k_scale) {
                                const int64_t r = a.b.scale_rows ? (int64_t)a.b.scale_rows[table + p] : page;
                                if (r >= 0 && r < a.b.n_scale_rows) {
                                    const size_t so = ((size_t)r * a.b.L + a.b.layer) * a.b.G + g;
                                    ks = checked_scale(a.k_scale[so], err);
                                    vs = checked_scale(a.v_scale[so], err);
                                } else {
                                    atomicOr(err, kErrBatch);
                                    there = false;
                                }
                            }
                            if (there) rows_of = min(kBlockTokens, kv_len - p * kBlockTokens);
                        }
                    }
                    const int rows = __shfl_sync(0xffffffffu, rows_of, j & 31);
                    for (int kv = 0; kv < 2; ++kv, ++n) {
                        const int rs = n % NR, s = n % NS;
                        const __nv_bfloat162 scale = __float2bfloat162_rn(
                            __shfl_sync(0xffffffffu, kv ? vs : ks, j & 31));
                        if (!__all_sync(0xffffffffu,
                                        tc::mbar_wait(&bar->raw_full[rs], (n / NR) & 1, kWaitNs) &&
                                            tc::mbar_wait(&bar->empty[s], ((n / NS) & 1) ^ 1, kWaitNs))) {
                            ok = false;
                            break;
                        }
                        const uint8_t *src = raws + rs * LY::RAW + w * kBlockTokens * D;
                        uint8_t *dst = kvs + s * LY::TILE;
                        constexpr int CPR = D / 16;      // 16-byte pieces of a raw row
#pragma unroll
                        for (int i = lane; i < kBlockTokens * CPR; i += 32) {
                            const int r = i / CPR, c = i % CPR, key = w * kBlockTokens + r;
                            uint4 x = *reinterpret_cast<const uint4 *>(src + i * 16);
                            if (r >= rows) x = make_uint4(0, 0, 0, 0);
                            const uint32_t in[4] = {x.x, x.y, x.z, x.w};
                            uint32_t out[8], nan = 0;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                out[2 * e] = e4m3_bf16(__byte_perm(in[e], 0, 0x1404), up, scale);
                                out[2 * e + 1] = e4m3_bf16(__byte_perm(in[e], 0, 0x3424), up, scale);
                                nan |= (in[e] & 0x7F7F7F7Fu) + 0x01010101u;
                            }
                            if (nan & 0x80808080u) {     // a NaN code: S.1111.111
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    if ((in[e >> 2] >> (8 * (e & 3)) & 0x7F) == 0x7F)
                                        out[e >> 1] |= 0x7FC0u << (16 * (e & 1));
                            }
                            // the two 16-byte chunks of the row's atom; the lanes of the
                            // second atom write theirs in the other order (bank conflicts)
                            uint8_t *row = dst + (c >> 2) * LY::ATOM + key * 128;
                            const int c0 = (c & 3) * 2, odd = (c >> 2) & 1;
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int h = e ^ odd;
                                *reinterpret_cast<uint4 *>(row + (((c0 + h) ^ (key & 7)) << 4)) =
                                    h ? make_uint4(out[4], out[5], out[6], out[7])
                                      : make_uint4(out[0], out[1], out[2], out[3]);
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

// Joins the partial sums of the row tiles that several CTAs share: block
// (c, y) takes the tile that begins in CTA c and goes on, rows y, y + ...  The
// work line is laid out as in the kernel before.
template <int D, bool PAIR>
__global__ void __launch_bounds__(256)
attend_join_kernel(const __grid_constant__ AttendArgs a, int n_ctas, int min_units) {
    constexpr int RB = PAIR ? 2 * TR : TR;
    constexpr int ROWS = 32;                             // rows of a block
    constexpr size_t REC = (size_t)RB * (D + 2);
    __shared__ int64_t pre[kMaxSeqs + 1];
    using W = Walk<RB, TK>;
    const int c = blockIdx.x;
    W::LN::lay_out(a, pre);
    const int64_t total = pre[a.b.n_seqs];
    const int64_t per = max((int64_t)min_units, (total + n_ctas - 1) / n_ctas);
    const int64_t end = min(total, (c + 1) * per);
    // every block waits for the kernel before: the stream's next one must not
    // begin while it runs
    tc::wait_prior_grids();
    if (c * per >= end) return;
    // the tile of the run's last unit
    W k;
    k.start_at(a, pre, end - 1, per);
    const int64_t x0 = k.x - k.u0;
    if (x0 < c * per || x0 + k.w <= end) return;         // begun earlier, or complete
    const int c1 = (int)((x0 + k.w - 1) / per);
    const int row = blockIdx.y * ROWS + (threadIdx.x & 31);
    const int qrow = k.r * RB + row;
    if (qrow >= k.i.q_len * a.gqa) return;
    float m = -INFINITY;
    for (int p = c; p <= c1; ++p)
        m = fmaxf(m, __ldcg(a.part + part_slot(p, p == c) * REC + (size_t)RB * D + row));
    const float base = m == -INFINITY ? 0.f : m;
    constexpr int PER = D / 4 / 8;                       // column quads of a thread
    float4 o[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    const int q0 = threadIdx.x >> 5;
    for (int p = c; p <= c1; ++p) {
        const float *rec = a.part + part_slot(p, p == c) * REC;
        const float f = ex2(__ldcg(rec + (size_t)RB * D + row) - base);
        l += f * __ldcg(rec + (size_t)RB * (D + 1) + row);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(rec) + (size_t)(q0 + 8 * i) * RB + row);
            o[i].x += f * v.x;
            o[i].y += f * v.y;
            o[i].z += f * v.z;
            o[i].w += f * v.w;
        }
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    const int tok = qrow / a.gqa, h = k.g * a.gqa + qrow - tok * a.gqa;
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) + (int64_t)(k.i.q0 + tok) * a.out_stride +
                         (int64_t)h * D;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        *reinterpret_cast<uint2 *>(dst + (q0 + 8 * i) * 4) =
            make_uint2(pack_bf16(o[i].x * inv, o[i].y * inv), pack_bf16(o[i].z * inv, o[i].w * inv));
    if (a.lse && q0 == 0)
        a.lse[(int64_t)(k.i.q0 + tok) * a.H + h] = m == -INFINITY ? -INFINITY : m * kLn2 + logf(l);
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
    using LY = Lay<D, E4>;
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
    const int min_units = PAIR ? 2 : 4;
    kern<<<ctas, LY::THREADS, LY::SMEM, s>>>(kmap, vmap, a, min_units);
    note_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas, PAIR ? 8 : 4);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attend_join_kernel<D, PAIR>, a, ctas, min_units);
    note_launch();
    return e;
}

template <int D, bool E4>
cudaError_t tile_p(const AttendArgs &a, cudaStream_t s) {
    return (int64_t)a.b.max_q_len * a.gqa > TR ? tile_t<D, E4, true>(a, s)
                                              : tile_t<D, E4, false>(a, s);
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
