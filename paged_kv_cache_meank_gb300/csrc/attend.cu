// Paged attention in float32 on the CUDA cores: every pairing of types that the
// tensor cores do not take (float32 queries or pages), and the dispatch.
//
// One pass over the keys with a running maximum m and weight l per query row
// (online softmax): for a page of 32 keys, s = scale * q.k, m' = max(m, max s),
// p = exp(s - m'), o = o exp(m - m') + p V, l likewise.  A lane holds one key's
// scores of the warp's rows, so a page's maxima and sums are warp shuffles; for
// p V a lane holds D/32 output columns.  Pages are converted to float32 in shared
// memory once and read by all rows of the CTA.  Up to 4 query rows (a decoded
// token), each of the four warps takes every fourth page on its own and the four
// sums are joined at the end; otherwise the four warps take 4 rows each and
// share the pages.
// Bound by the CUDA cores' float32 rate and, for few keys, by latency: one token
// over 77 float32 keys takes 5.9 us, most of it start-up (11.9 with a page's loads
// four at a time).
#include "attend_common.cuh"
#include "kvm_vec.cuh"

namespace kvm {

namespace {

constexpr int kWarps = 4;
constexpr int kRows = 4;                   // rows of a warp

template <typename T>
__device__ inline const T *typed(const void *p) { return static_cast<const T *>(p); }

template <int D, bool KS>
struct Lay {
    static constexpr int RB = KS ? kRows : kRows * kWarps;
    static_assert(RB <= kSimtMaxRows, "parts are for so many");
    static constexpr int KST = D + 4;      // padded K row: lanes' 16-byte reads hit distinct banks
    static constexpr int PAGE = kBlockTokens * (KST + D);
    static constexpr int NBUF = KS ? kWarps : 1;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_P = RB * D;
    static constexpr int FLOATS = OFF_P + NBUF * PAGE;
    static constexpr int SMEM = FLOATS * 4 + kPlainPreInts * 4;
    // CTAs of an SM: equal runs need all of the grid at once.  (The SM has 228 KB, a CTA's
    // own 1 KB and its static variables among them.)
    static constexpr int PER_SM = KS ? (D == 128 ? 1 : 3) : 4;
    static_assert(PER_SM * (SMEM + 1024 + 64) <= 228 * 1024, "the grid runs at once");
};

}  // namespace

template <typename TQ, typename T, int D, bool KS>
__global__ void __launch_bounds__(kWarps * 32)
attend_simt_kernel(AttendArgs a, int min_units) {
    using LY = Lay<D, KS>;
    constexpr int RB = LY::RB, CPL = D / 32;
    using W = Walk<RB, kBlockTokens>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    float *sm = reinterpret_cast<float *>(smem_raw);
    int *pre = reinterpret_cast<int *>(sm + LY::FLOATS);
    __shared__ int is_last;
    __shared__ LineInfo line;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cta = blockIdx.x;
    if (warp == 0) {
        const LineInfo li = W::LN::template lay_out<false>(a, pre, gridDim.x, min_units, 2 * min_units);
        if (lane == 0) line = li;
    }
    __syncthreads();
    W k;
    if (!k.start(a, pre, line, cta)) return;
    const int row0 = KS ? 0 : warp * kRows;     // the warp's rows of the tile
    float *kb = sm + LY::OFF_P + (KS ? warp * LY::PAGE : 0), *vb = kb + kBlockTokens * LY::KST;
    do {
        const int rows_all = k.i.q_len * a.gqa, rbase = k.r * RB;
        const int rows = min(RB, rows_all - rbase);
        __syncthreads();                         // the previous segment is done with shared memory
        for (int i = tid; i < RB * D; i += kWarps * 32) {
            const int r = i / D, row = rbase + r;
            float v = 0.f;
            if (r < rows) {
                const int t = token_of(row, a.gqa_inv), h = row - t * a.gqa;
                v = to_float(typed<TQ>(a.q)[(int64_t)(k.i.q0 + t) * a.q_stride +
                                            (int64_t)(k.g * a.gqa + h) * D + i % D]);
            }
            sm[LY::OFF_Q + i] = v;
        }
        __syncthreads();
        float m[kRows], l[kRows], o[kRows][CPL];
        int vis[kRows];                          // keys row r sees
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
            const int row = rbase + row0 + r, t = token_of(row, a.gqa_inv);
            vis[r] = row0 + r < rows ? (a.causal ? k.i.kv - k.i.q_len + t + 1 : k.i.kv) : 0;
#pragma unroll
            for (int c = 0; c < CPL; ++c) o[r][c] = 0.f;
        }
        for (int u = k.u0 + (KS ? warp : 0); u < k.u1; u += KS ? kWarps : 1) {
            const int key0 = u * kBlockTokens;
            if (key0 >= k.nk) break;             // a tile that sees nothing
            const int64_t at = (int64_t)k.s * a.b.table_stride + u;
            const int64_t page = a.b.page_table[at];
            const int64_t srow = a.k_scale && a.b.scale_rows ? (int64_t)a.b.scale_rows[at] : page;
            const bool ok = page >= 0 && page < a.b.n_pages &&
                            (!a.k_scale || (srow >= 0 && srow < a.b.n_scale_rows));
            if (!ok && lane == 0) atomicOr(a.b.err, kErrBatch);
            if (!KS) __syncthreads();
            float ks = 1.f, vs = 1.f;
            if (ok && a.k_scale) {
                const size_t so = ((size_t)srow * a.b.L + a.b.layer) * a.b.G + k.g;
                ks = checked_scale(a.k_scale[so], a.b.err);
                vs = checked_scale(a.v_scale[so], a.b.err);
            }
            {
                constexpr int N = VecTraits<T>::N, VPR = D / N;
                using V = typename VecTraits<T>::V;
                const size_t base = (((size_t)page * a.b.L + a.b.layer) * a.b.G + k.g) *
                                    kBlockTokens * D;
                // Loads in flight a thread: eight, so that a page's latency is met a few
                // times and not once for each of its 4 KB.  More where a warp reads
                // float32 pages on its own: 20000 keys, d = 64, took 96 us with 8 and 59
                // with 32, d = 128 74 with 8, 70 with 16 and 73 with 32.  (16-bit
                // and 8-bit pages, d = 128: 68 us with 8, 80 with 16.)
                constexpr int TOTAL = 2 * kBlockTokens * VPR, STEP = KS ? 32 : kWarps * 32;
                constexpr int MOST = KS && sizeof(T) == 4 ? (D == 64 ? 32 : 16) : 8;
                constexpr int U = TOTAL / STEP < MOST ? TOTAL / STEP : MOST;
#pragma unroll 1
                for (int i0 = KS ? lane : tid; i0 < TOTAL; i0 += U * STEP) {
                    V v[U];
#pragma unroll
                    for (int x = 0; x < U; ++x) {
                        const int i = i0 + x * STEP, j = i % (kBlockTokens * VPR);
                        if (ok && key0 + j / VPR < k.i.kv)
                            ld_stream_v(typed<T>(i == j ? a.k_pages : a.v_pages) + base + (size_t)j * N, v[x]);
                    }
#pragma unroll
                    for (int x = 0; x < U; ++x) {
                        const int i = i0 + x * STEP, j = i % (kBlockTokens * VPR);
                        const int row = j / VPR, c = (j - row * VPR) * N;
                        float f[N];
                        if (ok && key0 + row < k.i.kv) {
                            VecTraits<T>::unpack(v[x], f);
                            const float sc = i == j ? ks : vs;
#pragma unroll
                            for (int e = 0; e < N; ++e) f[e] *= sc;
                        } else {
#pragma unroll
                            for (int e = 0; e < N; ++e) f[e] = 0.f;
                        }
                        float *dst = i == j ? kb + row * LY::KST + c : vb + row * D + c;
#pragma unroll
                        for (int e = 0; e < N; e += 4)
                            *reinterpret_cast<float4 *>(dst + e) =
                                make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
                    }
                }
            }
            if (KS) __syncwarp(); else __syncthreads();
            float p[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) p[r] = 0.f;
            const float *kr = kb + lane * LY::KST, *qr = sm + LY::OFF_Q + row0 * D;
#pragma unroll 8
            for (int c = 0; c < D; c += 4) {
                const float4 kk = *reinterpret_cast<const float4 *>(kr + c);
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const float4 qq = *reinterpret_cast<const float4 *>(qr + r * D + c);
                    p[r] += qq.x * kk.x;
                    p[r] += qq.y * kk.y;
                    p[r] += qq.z * kk.z;
                    p[r] += qq.w * kk.w;
                }
            }
            const int key = key0 + lane;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float sc = key < vis[r] && key < k.i.kv ? p[r] * a.scale : -INFINITY;
                float mx = sc;
#pragma unroll
                for (int off = 16; off > 0; off >>= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                mx = fmaxf(mx, m[r]);
                const float base = mx == -INFINITY ? 0.f : mx;   // no key seen yet: weights 0
                const float corr = expf(m[r] - base);
                p[r] = expf(sc - base);
                float sum = p[r];
#pragma unroll
                for (int off = 16; off > 0; off >>= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, off);
                l[r] = l[r] * corr + sum;
                m[r] = mx;
#pragma unroll
                for (int c = 0; c < CPL; ++c) o[r][c] *= corr;
            }
#pragma unroll 8
            for (int j = 0; j < kBlockTokens; ++j) {
                float v[CPL];
#pragma unroll
                for (int c = 0; c < CPL; ++c) v[c] = vb[j * D + lane * CPL + c];
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const float w = __shfl_sync(0xffffffffu, p[r], j);
#pragma unroll
                    for (int c = 0; c < CPL; ++c) o[r][c] += w * v[c];
                }
            }
            if (KS) __syncwarp();
        }
        if (KS) {                                // join the four warps' sums in warp 0
            constexpr int REC = kRows * (D + 2);
            __syncthreads();
            float *mine = sm + LY::OFF_P + warp * REC;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
#pragma unroll
                for (int c = 0; c < CPL; ++c) mine[r * D + lane * CPL + c] = o[r][c];
                if (lane == 0) {
                    mine[kRows * D + 2 * r] = m[r];
                    mine[kRows * D + 2 * r + 1] = l[r];
                }
            }
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const float *rec = sm + LY::OFF_P;
                    float mx = -INFINITY;
                    for (int w = 0; w < kWarps; ++w)
                        mx = fmaxf(mx, rec[w * REC + kRows * D + 2 * r]);
                    const float base = mx == -INFINITY ? 0.f : mx;
                    l[r] = 0.f;
#pragma unroll
                    for (int c = 0; c < CPL; ++c) o[r][c] = 0.f;
                    for (int w = 0; w < kWarps; ++w) {
                        const float f = expf(rec[w * REC + kRows * D + 2 * r] - base);
                        l[r] += f * rec[w * REC + kRows * D + 2 * r + 1];
#pragma unroll
                        for (int c = 0; c < CPL; ++c)
                            o[r][c] += f * rec[w * REC + r * D + lane * CPL + c];
                    }
                    m[r] = mx;
                }
            }
        }
        bool write = !KS || warp == 0;
        if (!k.whole()) {
            // leave the partial sums; the last CTA of the tile to do so joins
            // them all, in CTA order
            const int c0 = k.first_cta(), c1 = k.last_cta();
            constexpr size_t REC = (size_t)RB * (D + 2);
            float *rec = a.part + part_slot(cta, cta == c0) * REC;
            if (write) {
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
#pragma unroll
                    for (int c = 0; c < CPL; ++c)
                        rec[(row0 + r) * D + lane * CPL + c] = o[r][c];
                    if (lane == 0) {
                        rec[RB * D + 2 * (row0 + r)] = m[r];
                        rec[RB * D + 2 * (row0 + r) + 1] = l[r];
                    }
                }
            }
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                is_last = atomicAdd(a.count + c0, 1) == c1 - c0;
                if (is_last) a.count[c0] = 0;    // ready for the next call
                __threadfence();
            }
            __syncthreads();
            if (!is_last) write = false;
            if (write) {
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    float mx = -INFINITY;
                    for (int c = c0; c <= c1; ++c)
                        mx = fmaxf(mx, __ldcg(a.part + part_slot(c, c == c0) * REC + RB * D +
                                              2 * (row0 + r)));
                    const float base = mx == -INFINITY ? 0.f : mx;
                    l[r] = 0.f;
#pragma unroll
                    for (int c = 0; c < CPL; ++c) o[r][c] = 0.f;
                    for (int c = c0; c <= c1; ++c) {
                        const float *rc = a.part + part_slot(c, c == c0) * REC;
                        const float f = expf(__ldcg(rc + RB * D + 2 * (row0 + r)) - base);
                        l[r] += f * __ldcg(rc + RB * D + 2 * (row0 + r) + 1);
#pragma unroll
                        for (int e = 0; e < CPL; ++e)
                            o[r][e] += f * __ldcg(rc + (row0 + r) * D + lane * CPL + e);
                    }
                    m[r] = mx;
                }
            }
        }
        if (write) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (row0 + r >= rows) continue;
                const int row = rbase + row0 + r, t = token_of(row, a.gqa_inv), h = k.g * a.gqa + row - t * a.gqa;
                const float inv = l[r] > 0.f ? 1.f / l[r] : (l[r] == 0.f ? 0.f : l[r]);
                TQ *dst = static_cast<TQ *>(a.out) + (int64_t)(k.i.q0 + t) * a.out_stride +
                          (int64_t)h * D + lane * CPL;
#pragma unroll
                for (int c = 0; c < CPL; ++c) dst[c] = from_float<TQ>(o[r][c] * inv);
                if (a.lse && lane == 0)
                    a.lse[(int64_t)(k.i.q0 + t) * a.H + h] = m[r] + logf(l[r]);
            }
        }
    } while (k.next(a));
}

template <typename TQ, typename T, int D, bool KS>
static cudaError_t simt_t(const AttendArgs &a, cudaStream_t s) {
    auto kern = attend_simt_kernel<TQ, T, D, KS>;
    constexpr int smem = Lay<D, KS>::SMEM;
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int ctas = min(kAttendMaxCtas, sm_count() * Lay<D, KS>::PER_SM);
    kern<<<ctas, kWarps * 32, smem, s>>>(a, KS ? 8 : 4);
    note_launch();
    return cudaGetLastError();
}

template <typename TQ, typename T>
static cudaError_t simt_d(const AttendArgs &a, cudaStream_t s) {
    const bool ks = (int64_t)a.b.max_q_len * a.gqa <= kRows;
    if (a.d == 128) return ks ? simt_t<TQ, T, 128, true>(a, s) : simt_t<TQ, T, 128, false>(a, s);
    return ks ? simt_t<TQ, T, 64, true>(a, s) : simt_t<TQ, T, 64, false>(a, s);
}

template <typename TQ>
static cudaError_t simt_q(int kv_dtype, const AttendArgs &a, cudaStream_t s) {
    if (kv_dtype == F32) return simt_d<TQ, float>(a, s);
    if (kv_dtype == BF16) return simt_d<TQ, __nv_bfloat16>(a, s);
    return simt_d<TQ, e4m3>(a, s);
}

size_t attend_scratch_bytes(int q_dtype, int kv_dtype, int d) {
    const bool tensor_cores = q_dtype == BF16 && kv_dtype != F32;
    return (tensor_cores ? max(kTilePartRows, kSimtPartRows) : kSimtPartRows) * (d + 2) * sizeof(float);
}

cudaError_t launch_attend(int q_dtype, int kv_dtype, const AttendArgs &a, cudaStream_t s,
                          bool *too_large) {
    if (attend_decode_supported(q_dtype, kv_dtype, a)) {
        if (!line_fits(a, 8, kBlockTokens)) return *too_large = true, cudaSuccess;
        return launch_attend_decode(kv_dtype, a, s);
    }
    if (attend_tc_supported(q_dtype, kv_dtype, a)) {
        if (!line_fits(a, 128, 128)) return *too_large = true, cudaSuccess;
        return launch_attend_tc(kv_dtype, a, s);
    }
    if (!line_fits(a, 4, kBlockTokens)) return *too_large = true, cudaSuccess;
    return q_dtype == BF16 ? simt_q<__nv_bfloat16>(kv_dtype, a, s) : simt_q<float>(kv_dtype, a, s);
}

}  // namespace kvm
