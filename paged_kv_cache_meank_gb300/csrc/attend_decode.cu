// Paged attention for the few query rows of a decoded token (or of a handful of
// drafted ones): bf16 queries over bf16 or e4m3 pages, at most 16 rows of a kv
// head.  The cache is read once and each byte of it meets 16 rows at most, so
// the kernel is bound by HBM; what counts is loads in flight.
//
// A warp owns every fourth (or eighth) stage of its CTA's run of keys (16 or 32 keys of K
// and V, 4-8 KB) with a ring of cp.async stages of its own in shared memory, its
// own running maximum, weight and output, and no barrier until the run's end.
// Keys take the 16-row side of mma.m16n8k16 and query rows the 8-column side, so
// one kv head's 6 or 8 rows fill it:
//   S^T[16 keys][8 rows]  = K Q^T      K by ldmatrix, Q in registers
//   O^T[16 d][8 rows]    += V^T P^T    V by transposing ldmatrix, P^T from S^T by
//                                      movmatrix
// (these products are far from what bounds the kernel, and their operands come
// out of registers: tensor memory would only add round trips).  As in
// attend_tc.cu the maximum moves when a stage exceeds it by 2^8; a vote decides,
// so the usual stage has no shuffles.  A weight goes into the product with V as the
// sum of two bf16 (its rounding, and that of the rest), with two products: the matrix
// pipe is far from busy, and 32768 keys take the same time with one.
//
// e4m3: as in attend_tc.cu codes become f16 (exact) in registers, q is divided by
// a power of two per row, the page's k_scale goes into the factor of the scores
// and the weights times v_scale, by a finite factor, have a reference of their own.
//
// One sequence of 32768 bf16 keys takes 26.8 us, 19.0 of them its 134 MB at the
// 7.06 TB/s that longer sequences add; the start (lengths, page numbers and keys,
// each read before the next can be) takes 5 and leaving and joining the parts 3.  24
// ragged sequences of e4m3 pages (508 MB) take 89.8 us, 5.7 TB/s.
// Three 8 KB or four 4 KB stages a warp; eight to twelve warps an SM.  With fewer
// tiles than SMs they are one CTA, for as few parts to join as can be: one
// sequence of 32768 bf16 keys took 27.4 us against 31.4 with two CTAs of four
// warps, of 65536 e4m3 keys 29.1 against 33.5.  With more, two or three CTAs,
// so that one streams while another joins; the third where rows are narrow and carry
// more arithmetic for their bytes (24 ragged sequences of e4m3 pages: 94.6 us against
// 101.3 with two).
#include <math.h>

#include "attend_common.cuh"
#include "kvm_vec.cuh"
#include "tc_ptx.cuh"

namespace kvm {

namespace {

constexpr float kMoveMax = 8.f, kUp = 7.f, kMostW = 127.f;   // (as in attend_tc.cu)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Pages of a CTA's run at least, and what a join costs.  One sequence of 512, 1024,
// 2048, 4096 bf16 keys takes 6.2, 7.6, 8.2, 9.2 us; with 8 and 16 it took 6.3, 9.0, 9.4,
// 9.0, with 4 and 8, 7.6, 7.8, 8.3, 9.2.
constexpr int kMinPages = 4, kJoinPages = 16;

// W warps a CTA, CTAS of them an SM.
template <int D, bool E4, int NT, int W, int CTAS>
struct Lay {
    static constexpr int RB = 8 * NT;
    static constexpr int ROW = E4 ? D : 2 * D;             // bytes of a K or V row
    static constexpr int KEYS = ROW == 64 ? 32 : 16;       // keys of a stage
    static constexpr int HALF = KEYS * ROW;                // K (or V) of a stage
    static constexpr int STAGE = 2 * HALF;
    static constexpr int STAGES = STAGE == 8192 ? 3 : 4;
    static constexpr int RING = STAGES * STAGE;            // of one warp
    static constexpr int ORS = D + 4;                      // a row of a warp's sums
    static constexpr int REC = RB * ORS + 2 * RB;          // floats: o, m, l
    static constexpr int BYTES = W * (RING > REC * 4 ? RING : REC * 4);
    static constexpr int MAX_CTAS = CTAS * kTileMaxCtas;
    static constexpr int WEIGHTS = MAX_CTAS * RB * 4;      // bytes: of the parts of a join
    static_assert(MAX_CTAS <= kAttendMaxCtas, "counts are for so many");
    static_assert((size_t)MAX_CTAS * 2 * RB <= kTilePartRows, "parts are for so many");
    static constexpr int SMEM = BYTES + kPreInts * 4;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 16 bytes to shared memory, zeros when `there` is false (nothing is read).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t *r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t *r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <bool F16>
__device__ __forceinline__ void mma(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    if constexpr (F16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Four e4m3 codes as two f16x2: exact.
__device__ __forceinline__ void e4m3_f16(uint32_t x, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}

}  // namespace

template <int D, bool E4, int NT, int WARPS, int CTAS>
__global__ void __launch_bounds__(WARPS * 32, CTAS)
attend_decode_kernel(const __grid_constant__ AttendArgs a) {
    using LY = Lay<D, E4, NT, WARPS, CTAS>;
    constexpr int RB = LY::RB, KS = D / 16, MT = D / 16, KEYS = LY::KEYS, S = LY::STAGES;
    constexpr int CH = LY::ROW / 16;                       // 16-byte chunks of a row
    using W = Walk<RB, kBlockTokens>;
    extern __shared__ __align__(1024) uint8_t smem[];
    int *pre = reinterpret_cast<int *>(smem + LY::BYTES);
    __shared__ int is_last;
    __shared__ float part_m[WARPS][RB], part_l[WARPS][RB];
    __shared__ LineInfo line;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g8 = lane >> 2, c4 = lane & 3;               // fragment row and column pair
    const int cta = blockIdx.x;
    if (warp == 0) {
        const LineInfo li = W::LN::template lay_out<true>(a, pre, gridDim.x, kMinPages, kJoinPages);
        if (lane == 0) line = li;
    }
    __syncthreads();
    W k;
    if (!k.start(a, pre, line, cta)) return;
    const uint32_t ring32 = tc::smem_u32(smem + warp * LY::RING);
    const float c = a.scale * kLog2e;
    // a chunk's place in its row: the 8 rows that an ldmatrix phase reads at one
    // chunk fall into distinct banks (rows of 64 bytes: two to a bank line)
    auto place = [](int row, int ch) {
        return row * LY::ROW + ((ch ^ (CH == 4 ? (row >> 1) & 3 : row & 7)) << 4);
    };

    do {
        const int rows_all = k.i.q_len * a.gqa, rbase = k.r * RB;
        const int rows = min(RB, rows_all - rbase);
        // ---- the warp's stages: numbers warp, warp + WARPS, ... of the run
        const int key_first = k.u0 * kBlockTokens;
        const int key_end = min(k.nk, k.u1 * kBlockTokens);
        const int n_all = key_end > key_first ? (key_end - key_first + KEYS - 1) / KEYS : 0;
        const int n = n_all > warp ? (n_all - warp + WARPS - 1) / WARPS : 0;
        // lane i: page and scales of the warp's stage w0 + i
        int w0 = 0;
        int32_t page_of = -1;
        float ks_of = 1.f, vs_of = 1.f;
        auto look_up = [&](int j0) {
            w0 = j0;
            const int j = j0 + lane;
            page_of = -1;
            if (j < n) {
                const int p = (key_first + (warp + j * WARPS) * KEYS) / kBlockTokens;
                const int64_t at = (int64_t)k.s * a.b.table_stride + p;
                const int32_t page = a.b.page_table[at];
                bool ok = page >= 0 && page < a.b.n_pages;
                if (E4 && a.k_scale) {
                    const int64_t r = a.b.scale_rows ? (int64_t)a.b.scale_rows[at] : (int64_t)page;
                    ok = ok && r >= 0 && r < a.b.n_scale_rows;
                    if (ok) {
                        const size_t so = ((size_t)r * a.b.L + a.b.layer) * a.b.G + k.g;
                        ks_of = a.k_scale[so];
                        vs_of = a.v_scale[so];
                    }
                }
                if (ok) page_of = page;
                else atomicOr(a.b.err, kErrBatch);
            }
        };
        // apart from look_up, so that the first stages are asked for before their scales come
        auto check_scales = [&] {
            if (E4 && a.k_scale && page_of >= 0) {
                ks_of = checked_scale(ks_of, a.b.err);
                vs_of = checked_scale(vs_of, a.b.err);
            }
        };
        auto issue = [&](int j, int slot) {
            if (j < n) {
                const int32_t page = __shfl_sync(0xffffffffu, page_of, j - w0);
                const int key0 = key_first + (warp + j * WARPS) * KEYS;
                const int64_t head = ((int64_t)max(page, 0) * a.b.L + a.b.layer) * a.b.G + k.g;
                const int64_t off = (head * kBlockTokens + (key0 & (kBlockTokens - 1))) * LY::ROW + lane * 16;
                const char *kp = static_cast<const char *>(a.k_pages) + off;
                const char *vp = static_cast<const char *>(a.v_pages) + off;
                const uint32_t dst = ring32 + slot * LY::STAGE;
                const int n_rows = page >= 0 ? k.i.kv - key0 : 0;   // rows behind them read as 0
#pragma unroll
                for (int i = 0; i < LY::HALF / 512; ++i) {
                    const int x = i * 32 + lane, row = x / CH, at = place(row, x % CH);
                    copy16(dst + at, kp + i * 512, row < n_rows);
                    copy16(dst + LY::HALF + at, vp + i * 512, row < n_rows);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        look_up(0);
#pragma unroll 1
        for (int i = 0; i < S - 1; ++i) issue(i, i);
        check_scales();

        // ---- the query rows as B fragments, and what each score is multiplied by
        uint32_t qf[NT][KS][2];
        float cm[NT][2];
        int vis[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = t * 8 + g8, row = rbase + r;
            const __nv_bfloat16 *src = nullptr;
            if (r < rows) {
                const int tok = token_of(row, a.gqa_inv), h = row - tok * a.gqa;
                src = static_cast<const __nv_bfloat16 *>(a.q) + (int64_t)(k.i.q0 + tok) * a.q_stride +
                      (int64_t)(k.g * a.gqa + h) * D;
            }
            if constexpr (!E4) {
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        qf[t][s][b] = src ? __ldg(reinterpret_cast<const uint32_t *>(
                                                src + s * 16 + b * 8 + c4 * 2))
                                          : 0u;
                cm[t][0] = cm[t][1] = c;
            } else {
                // d = 16 s + 4 c4 + {0, 1 | 2, 3}: the order a code quad is held in
                uint2 w[KS];
                uint32_t e = 0;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    w[s] = src ? __ldg(reinterpret_cast<const uint2 *>(src + s * 16 + c4 * 4))
                               : make_uint2(0, 0);
                    e = max(e, max(max(w[s].x & 0x7F80u, (w[s].x >> 16) & 0x7F80u),
                                   max(w[s].y & 0x7F80u, (w[s].y >> 16) & 0x7F80u)));
                }
                e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
                e = max(e, __shfl_xor_sync(0xffffffffu, e, 2));
                // the row's largest entry into [2^15, 2^16), as row_exponent in attend_tc.cu
                const int x = min(127, max(-101, (int)(e >> 7) - 127)) - 15;
                const float dn = __uint_as_float((uint32_t)(127 - x) << 23);
                const float up = __uint_as_float((uint32_t)(127 + x) << 23);
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    qf[t][s][0] = pack<true>(__uint_as_float(w[s].x << 16) * dn,
                                             __uint_as_float(w[s].x & 0xFFFF0000u) * dn);
                    qf[t][s][1] = pack<true>(__uint_as_float(w[s].y << 16) * dn,
                                             __uint_as_float(w[s].y & 0xFFFF0000u) * dn);
                }
                cm[t][0] = __shfl_sync(0xffffffffu, up, c4 * 8) * c;
                cm[t][1] = __shfl_sync(0xffffffffu, up, c4 * 8 + 4) * c;
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int q = t * 8 + c4 * 2 + b, tok = token_of(rbase + q, a.gqa_inv);
                vis[t][b] = q >= rows ? 0 : a.causal ? min(k.i.kv, k.i.kv - k.i.q_len + tok + 1) : k.i.kv;
            }
        }
        // keys below `all` are seen by every row of the tile
        const int all = a.causal ? k.i.kv - k.i.q_len + token_of(rbase, a.gqa_inv) + 1 : k.i.kv;
        // m: reference of the weights; mp: of what O holds (e4m3: the weights times
        // v_scale; else the same)
        float m[NT][2], mp[NT][2], l[NT][2], o[MT][NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            m[t][0] = m[t][1] = mp[t][0] = mp[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.f;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][t][e] = 0.f;
        }
        int slot = 0;
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
            __syncwarp();
            {
                // the slot that the previous stage left
                const int jn = j + S - 1;
                if (jn - w0 == 32) {
                    look_up(j);
                    check_scales();
                }
                issue(jn, slot == 0 ? S - 1 : slot - 1);
            }
            float ks = 1.f, lv = 0.f;                      // k_scale, log2 v_scale of the stage
            if constexpr (E4) {
                ks = __shfl_sync(0xffffffffu, ks_of, j - w0);
                lv = (float)((int)(__float_as_uint(__shfl_sync(0xffffffffu, vs_of, j - w0)) >> 23) - 127);
            }
            const int key0 = key_first + (warp + j * WARPS) * KEYS;
            const uint32_t kb = ring32 + slot * LY::STAGE, vb = kb + LY::HALF;
            if (++slot == S) slot = 0;

            // ---- scores of the stage's keys, 16 at a time, in two sums each
            float s[KEYS / 16][NT][4];
#pragma unroll
            for (int u = 0; u < KEYS / 16; ++u) {
                float s2[2][NT][4];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s2[0][t][e] = s2[1][t][e] = 0.f;
                const int row = u * 16 + (lane & 15);
                if constexpr (!E4) {
#pragma unroll
                    for (int x = 0; x < KS; ++x) {
                        uint32_t f[4];
                        ldm4(f, kb + place(row, 2 * x + (lane >> 4)));
#pragma unroll
                        for (int t = 0; t < NT; ++t) mma<false>(s2[x & 1][t], f, qf[t][x][0], qf[t][x][1]);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < KS; x += 2) {
                        uint32_t f[4];
                        ldm4(f, kb + place(row, x + (lane >> 4)));
                        // f[0], f[1]: keys 0-7, 8-15 of chunk x; f[2], f[3]: of chunk x + 1
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            uint32_t fa[4];
                            e4m3_f16(f[2 * y], fa[0], fa[2]);
                            e4m3_f16(f[2 * y + 1], fa[1], fa[3]);
#pragma unroll
                            for (int t = 0; t < NT; ++t)
                                mma<true>(s2[y][t], fa, qf[t][x + y][0], qf[t][x + y][1]);
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[u][t][e] = s2[0][t][e] + s2[1][t][e];
            }
            // ---- scaled, masked, against the running maximum
            const bool edge = key0 + KEYS > all;
            bool grow = false;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float f = E4 ? cm[t][b] * ks : cm[t][b];
                    float top = -INFINITY;
#pragma unroll
                    for (int u = 0; u < KEYS / 16; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float x = s[u][t][2 * h + b] * f;
                            if (edge && key0 + u * 16 + g8 + h * 8 >= vis[t][b]) x = -INFINITY;
                            s[u][t][2 * h + b] = x;
                            top = fmaxf(top, x);
                        }
                    // (a first finite score exceeds the m of -infinity)
                    grow |= top > m[t][b] + kMoveMax || (E4 && top + (lv - kUp) > mp[t][b] + kMoveMax);
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        float x = -INFINITY;
#pragma unroll
                        for (int u = 0; u < KEYS / 16; ++u) x = fmaxf(x, fmaxf(s[u][t][b], s[u][t][b + 2]));
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1)
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
                        const float mn = fmaxf(m[t][b], x), mpn = E4 ? fmaxf(mp[t][b], x + (lv - kUp)) : mn;
                        const bool none = m[t][b] == -INFINITY;
                        const float f = none ? 0.f : ex2(m[t][b] - mn);
                        const float fp = E4 ? (none ? 0.f : ex2(mp[t][b] - mpn)) : f;
                        m[t][b] = mn;
                        mp[t][b] = mpn;
                        l[t][b] *= f;
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            o[i][t][b] *= fp;
                            o[i][t][b + 2] *= fp;
                        }
                    }
            }
            // ---- weights, and the product with V
            // bf16 pages: a weight as the sum of two bf16
            constexpr int PARTS = E4 ? 1 : 2;
            uint32_t pf[PARTS][KEYS / 16][NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float base[2], w[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    base[b] = m[t][b] == -INFINITY ? 0.f : m[t][b];
                    w[b] = !E4 ? 1.f : m[t][b] == -INFINITY ? 0.f : ex2(fminf(lv + m[t][b] - mp[t][b], kMostW));
                }
#pragma unroll
                for (int u = 0; u < KEYS / 16; ++u) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[e] = ex2(s[u][t][e] - base[e & 1]);
                        l[t][e & 1] += p[e];
                        if (E4) p[e] *= w[e & 1];
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t two = pack<E4>(p[2 * h], p[2 * h + 1]);
                        pf[0][u][t][h] = transposed(two);
                        if constexpr (!E4)
                            pf[1][u][t][h] = transposed(
                                pack<false>(p[2 * h] - __uint_as_float(two << 16),
                                            p[2 * h + 1] - __uint_as_float(two & 0xFFFF0000u)));
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < KEYS / 16; ++u) {
                if constexpr (!E4) {
                    const int row = u * 16 + (lane >> 4) * 8 + (lane & 7);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        uint32_t f[4];
                        ldm4t(f, vb + place(row, 2 * i + ((lane >> 3) & 1)));
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int y = 0; y < PARTS; ++y)
                                mma<false>(o[i][t], f, pf[y][u][t][0], pf[y][u][t][1]);
                    }
                } else {
                    const int row = u * 16 + (lane & 15);
#pragma unroll
                    for (int i = 0; i < MT; i += 2) {
                        uint32_t f[4];
                        ldm4t(f, vb + place(row, i + (lane >> 4)));
                        // f[0], f[1]: keys 0-7, 8-15 of chunk i; a register holds two keys'
                        // two adjacent d: the even d's are rows 0-7, the odd ones 8-15
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            uint32_t fa[4];
                            e4m3_f16(__byte_perm(f[2 * y], 0, 0x3120), fa[0], fa[1]);
                            e4m3_f16(__byte_perm(f[2 * y + 1], 0, 0x3120), fa[2], fa[3]);
#pragma unroll
                            for (int t = 0; t < NT; ++t)
                                mma<true>(o[i + y][t], fa, pf[0][u][t][0], pf[0][u][t][1]);
                        }
                    }
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        // ---- the warps' sums, joined through shared memory (the ring is idle)
        __syncthreads();
        float *rec = reinterpret_cast<float *>(smem) + warp * LY::REC;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    l[t][b] += __shfl_xor_sync(0xffffffffu, l[t][b], off);
                const int r = t * 8 + c4 * 2 + b;
                const float f = E4 && m[t][b] != -INFINITY ? ex2(mp[t][b] - m[t][b]) : 1.f;
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        rec[r * LY::ORS + i * 16 + (E4 ? 2 * g8 + h : g8 + 8 * h)] = o[i][t][2 * h + b] * f;
                if (g8 == 0) {
                    rec[RB * LY::ORS + r] = m[t][b];
                    rec[RB * LY::ORS + RB + r] = l[t][b];
                }
            }
        const bool whole = k.whole();
        const int c0 = whole ? cta : k.first_cta(), c1 = whole ? cta : k.last_cta();
        constexpr int QUADS = D / 4;
        auto emit = [&](int r, int q, float4 v, float mm, float ll) {
            const int row = rbase + r, tok = token_of(row, a.gqa_inv);
            const int h = k.g * a.gqa + row - tok * a.gqa;
            const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) +
                                       (int64_t)(k.i.q0 + tok) * a.out_stride + (int64_t)h * D + q * 4) =
                make_uint2(pack<false>(v.x * inv, v.y * inv), pack<false>(v.z * inv, v.w * inv));
            if (q == 0 && a.lse)
                a.lse[(int64_t)(k.i.q0 + tok) * a.H + h] =
                    mm == -INFINITY ? -INFINITY : mm * kLn2 + logf(ll);
        };
        // a part: m and l of RB rows, then the rows
        constexpr size_t PREC = (size_t)RB * (D + 2);
        // ---- the four warps' sums of a row quad; to the output, or to this CTA's part
        __syncthreads();
#pragma unroll 1
        for (int x = tid; x < rows * QUADS; x += WARPS * 32) {
            const int r = x / QUADS, q = x % QUADS;
            const float *all_rec = reinterpret_cast<const float *>(smem);
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) mm = fmaxf(mm, all_rec[w * LY::REC + RB * LY::ORS + r]);
            const float base = mm == -INFINITY ? 0.f : mm;
            float ll = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float *rc = all_rec + w * LY::REC;
                const float f = ex2(rc[RB * LY::ORS + r] - base);
                ll += f * rc[RB * LY::ORS + RB + r];
                const float4 y = *reinterpret_cast<const float4 *>(rc + r * LY::ORS + q * 4);
                v.x += f * y.x;
                v.y += f * y.y;
                v.z += f * y.z;
                v.w += f * y.w;
            }
            if (whole) {
                emit(r, q, v, mm, ll);
            } else {
                float *part = a.part + part_slot(cta, cta == c0) * PREC;
                *reinterpret_cast<float4 *>(part + 2 * RB + r * D + q * 4) = v;
                if (q == 0) {
                    part[r] = mm;
                    part[RB + r] = ll;
                }
            }
        }
        __syncthreads();                                   // the records are free
        if (whole) continue;
        // ---- the last CTA of the tile to leave its part joins them, in the order of
        // the CTAs.  The parts come to shared memory a batch ahead of their use, as
        // many in flight as fit (one CTA reads up to 120 KB from L2), by loops
        // that are short because they run once, out of a cold instruction cache.
        if (tid == 0) {
            int n_before;                                  // (orders the whole CTA's part, met at the barrier)
            asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"
                         : "=r"(n_before)
                         : "l"(a.count + c0)
                         : "memory");
            is_last = n_before == c1 - c0;
            if (is_last) a.count[c0] = 0;                  // ready for the next call
        }
        __syncthreads();
        if (!is_last) continue;
        constexpr int T = WARPS * 32;
        const int pq = rows * QUADS;                       // 16-byte pieces of a part's rows
        const int cap = (LY::BYTES - LY::WEIGHTS) / 32 / pq;   // parts of a batch, two in flight
        float *weight = reinterpret_cast<float *>(smem);   // [part][RB]
        uint8_t *batch = smem + LY::WEIGHTS;
        auto fetch = [&](int p0, int b) {
            const int p1 = min(p0 + cap, c1 + 1);
#pragma unroll 1
            for (int p = p0 + warp; p < p1; p += WARPS) {
                const float4 *src =
                    reinterpret_cast<const float4 *>(a.part + part_slot(p, p == c0) * PREC + 2 * RB);
                const uint32_t dst = tc::smem_u32(batch) + (b * cap + p - p0) * pq * 16;
#pragma unroll 2
                for (int x = lane; x < pq; x += 32) copy16(dst + x * 16, src + x, true);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        fetch(c0, 0);
        fetch(c0 + cap, 1);
        // the rows' m and l over all parts, a thread to a row of every T / RB-th part
        const int jr = tid % RB, jp = tid / RB;
        float mine = -INFINITY, ll = 0.f;
        if (jr < rows)
#pragma unroll 1
            for (int p = c0 + jp; p <= c1; p += T / RB) {
                const float *rc = a.part + part_slot(p, p == c0) * PREC;
                const float pm = __ldcg(rc + jr), pl = __ldcg(rc + RB + jr), mx = fmaxf(mine, pm);
                const float base = mx == -INFINITY ? 0.f : mx;
                weight[(p - c0) * RB + jr] = pm;
                ll = ll * ex2(mine - base) + pl * ex2(pm - base);
                mine = mx;
            }
        float mm = mine;
#pragma unroll
        for (int off = RB; off < 32; off <<= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, off));
        if (lane < RB) part_m[warp][lane] = mm;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WARPS; ++w) mm = fmaxf(mm, part_m[w][jr]);
        const float base = mm == -INFINITY ? 0.f : mm;
        if (jr < rows)
#pragma unroll 1
            for (int p = jp; p <= c1 - c0; p += T / RB)
                weight[p * RB + jr] = ex2(weight[p * RB + jr] - base);
        ll *= ex2(mine - base);
#pragma unroll
        for (int off = RB; off < 32; off <<= 1) ll += __shfl_xor_sync(0xffffffffu, ll, off);
        if (lane < RB) part_l[warp][lane] = ll;
        // the rows' weighted sums, a thread to one or two row quads
        constexpr int PER = RB * QUADS > T ? RB * QUADS / T : 1;
        float4 acc[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        int b = 0;
#pragma unroll 1
        for (int p0 = c0; p0 <= c1; p0 += cap) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncthreads();
            const int np = min(cap, c1 + 1 - p0);
            const float4 *rc = reinterpret_cast<const float4 *>(batch) + b * cap * pq;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int x = tid + i * T;
                if (x >= pq) continue;
                const float *w = weight + (p0 - c0) * RB + x / QUADS;
#pragma unroll 4
                for (int p = 0; p < np; ++p) {
                    const float f = w[p * RB];
                    const float4 y = rc[p * pq + x];
                    acc[i].x += f * y.x;
                    acc[i].y += f * y.y;
                    acc[i].z += f * y.z;
                    acc[i].w += f * y.w;
                }
            }
            __syncthreads();
            fetch(p0 + 2 * cap, b);
            b ^= 1;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int x = tid + i * T, r = x / QUADS;
            if (x >= pq) continue;
            float m_all = -INFINITY, l_all = 0.f;
#pragma unroll 1
            for (int w = 0; w < WARPS; ++w) {
                m_all = fmaxf(m_all, part_m[w][r]);
                l_all += part_l[w][r];
            }
            emit(r, x % QUADS, acc[i], m_all, l_all);
        }
        __syncthreads();                                   // shared memory is the next tile's
    } while (k.next(a));
}

namespace {

template <int D, bool E4, int NT, int WARPS, int CTAS>
cudaError_t decode_t(const AttendArgs &a, cudaStream_t s) {
    using LY = Lay<D, E4, NT, WARPS, CTAS>;
    auto kern = attend_decode_kernel<D, E4, NT, WARPS, CTAS>;
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, LY::SMEM);
    if (e != cudaSuccess) return e;
    const int ctas = min(LY::MAX_CTAS, CTAS * sm_count());
    kern<<<ctas, WARPS * 32, LY::SMEM, s>>>(a);
    note_launch();
    return cudaGetLastError();
}

template <int D, bool E4>
cudaError_t decode_n(const AttendArgs &a, cudaStream_t s) {
    const bool many = (int64_t)a.b.n_seqs * a.b.G >= sm_count();
    if ((int64_t)a.b.max_q_len * a.gqa > 8)
        return many ? decode_t<D, E4, 2, 4, 2>(a, s) : decode_t<D, E4, 2, 8, 1>(a, s);
    return many ? decode_t<D, E4, 1, 4, E4 || D == 64 ? 3 : 2>(a, s) : decode_t<D, E4, 1, 8, 1>(a, s);
}

}  // namespace

bool attend_decode_supported(int q_dtype, int kv_dtype, const AttendArgs &a) {
    return q_dtype == BF16 && (kv_dtype == BF16 || kv_dtype == E4M3) &&
           (int64_t)a.b.max_q_len * a.gqa <= kDecodeRows;
}

cudaError_t launch_attend_decode(int kv_dtype, const AttendArgs &a, cudaStream_t s) {
    if (kv_dtype == E4M3) return a.d == 128 ? decode_n<128, true>(a, s) : decode_n<64, true>(a, s);
    return a.d == 128 ? decode_n<128, false>(a, s) : decode_n<64, false>(a, s);
}

}  // namespace kvm
