// Mean-K index of e4m3 pages that carry a scale per (block, layer, kv head).
//
// KVMem (Virtualizing Million-Token Agent Workspaces on a Consumer GPU), §4.3
// and §5: the mean over a block's 32 tokens of its K with RoPE removed, taken
// while the pages are on the GPU.  With scales the index entry is scale * mean
// of the un-rotated codes; the scale is a power of two, so the product is exact
// and the entry is rounded once.  The un-rotated codes themselves are the raw K:
// rotation is linear, so they keep the block's scale.
//
// Layout of meank_kernel: one CTA owns a block and a run of (layer, kv head)
// pairs, with the block's 32 table rows in shared memory; a warp owns whole
// pairs, a lane 8 codes of a half row and their rotate-half partners.  Bound by
// HBM: 32 d bytes read and 32 d written (raw K) a pair.  256 blocks of 64 layers
// and 8 kv heads, d = 128 (1.11 GB), take 187 us, 5.9 TB/s; one block takes 5.9 us.
// Without raw K half the bytes are left and nearly all of the arithmetic: 130 us, bound by
// its issue.
#include "kvm_internal.cuh"
#include "kvm_vec.cuh"

namespace kvm {

constexpr int kScaledWarps = 4;

template <typename TI, int D>
__global__ void __launch_bounds__(kScaledWarps * 32, 6)
meank_scaled_kernel(const e4m3 *__restrict__ k_pages, const float *__restrict__ k_scale,
                    e4m3 *__restrict__ raw_out, TI *__restrict__ index, int64_t index_cap,
                    int64_t first_block, int LG, int lg_per_cta,
                    const float2 *__restrict__ table, int *err) {
    using VT = VecTraits<e4m3>;
    constexpr int N = VT::N, HD = D / 2, TPT = HD / N, TOK = 32 / TPT, ITERS = 32 / TOK;
    constexpr int ROW = N + 2;               // padded: a phase's lanes hit distinct banks
    __shared__ __align__(16) float2 tab[kBlockTokens * TPT * ROW];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c = lane % TPT, t0 = lane / TPT;
    const int64_t b = blockIdx.x, gb = first_block + b;
    const float2 *trow = table + gb * kBlockTokens * HD;
    for (int i = tid; i < kBlockTokens * HD; i += kScaledWarps * 32) {
        const int t = i / HD, j = i - t * HD;
        tab[(t * TPT + j / N) * ROW + j % N] = trow[i];
    }
    __syncthreads();
    const int lg0 = blockIdx.y * lg_per_cta, lg1 = min(LG, lg0 + lg_per_cta);
    for (int lg = lg0 + warp; lg < lg1; lg += kScaledWarps) {
        const size_t base = ((size_t)b * LG + lg) * kBlockTokens * D + (size_t)c * N;
        uint2 vx[ITERS], vy[ITERS];
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const size_t off = base + (size_t)(t0 + i * TOK) * D;
            ld_stream_v(k_pages + off, vx[i]);
            ld_stream_v(k_pages + off + HD, vy[i]);
        }
        const float scale = k_scale[(size_t)b * LG + lg];
        float ax[N], ay[N];
#pragma unroll
        for (int k = 0; k < N; ++k) ax[k] = ay[k] = 0.f;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int t = t0 + i * TOK;
            float x[N], y[N], rx[N], ry[N];
            VT::unpack(vx[i], x);
            VT::unpack(vy[i], y);
            const float4 *cs4 = reinterpret_cast<const float4 *>(tab + (t * TPT + c) * ROW);
#pragma unroll
            for (int k = 0; k < N; k += 2) {
                const float4 w = cs4[k / 2];
                rx[k] = __fadd_rn(__fmul_rn(x[k], w.x), __fmul_rn(y[k], w.y));
                ry[k] = __fsub_rn(__fmul_rn(y[k], w.x), __fmul_rn(x[k], w.y));
                rx[k + 1] = __fadd_rn(__fmul_rn(x[k + 1], w.z), __fmul_rn(y[k + 1], w.w));
                ry[k + 1] = __fsub_rn(__fmul_rn(y[k + 1], w.z), __fmul_rn(x[k + 1], w.w));
            }
#pragma unroll
            for (int k = 0; k < N; ++k) {
                ax[k] += rx[k];
                ay[k] += ry[k];
            }
            if (raw_out != nullptr) {
                const size_t off = base + (size_t)t * D;
                st_stream_v(raw_out + off, VT::pack(rx));
                st_stream_v(raw_out + off + HD, VT::pack(ry));
            }
        }
#pragma unroll
        for (int off = TPT; off < 32; off <<= 1) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                ax[k] += __shfl_xor_sync(0xffffffffu, ax[k], off);
                ay[k] += __shfl_xor_sync(0xffffffffu, ay[k], off);
            }
        }
        if (lane < TPT) {
            const float m = checked_scale(scale, err) * (1.0f / kBlockTokens);
            TI *dst = index + ((size_t)lg * index_cap + gb) * D + (size_t)c * N;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                ax[k] *= m;
                ay[k] *= m;
            }
            store_n<TI, N>(dst, ax);
            store_n<TI, N>(dst + HD, ay);
        }
    }
}

template <typename TI, int D>
static cudaError_t scaled_t(const void *k_pages, const float *k_scale, void *raw_out, void *index,
                            int64_t index_cap, int64_t first_block, int64_t n_blocks, int LG,
                            const float2 *table, int *err, cudaStream_t s) {
    // long runs of pairs amortise the table stage, short ones fill the machine
    int lpc = LG;
    const int64_t want = (int64_t)sm_count() * 16;
    while (lpc > kScaledWarps && n_blocks * ((LG + lpc - 1) / lpc) < want) lpc = (lpc + 1) / 2;
    if (lpc > 64 * kScaledWarps) lpc = 64 * kScaledWarps;
    const int64_t gy = (LG + lpc - 1) / lpc;
    if (n_blocks > 0x7FFFFFFF || gy > 65535) return cudaErrorInvalidValue;
    meank_scaled_kernel<TI, D><<<dim3((unsigned)n_blocks, (unsigned)gy), kScaledWarps * 32, 0, s>>>(
        static_cast<const e4m3 *>(k_pages), k_scale, static_cast<e4m3 *>(raw_out),
        static_cast<TI *>(index), index_cap, first_block, LG, lpc, table, err);
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_meank_scaled(int index_dtype, int d, const void *k_pages, const float *k_scale,
                                void *raw_out, void *index, int64_t index_cap,
                                int64_t first_block, int64_t n_blocks, int LG,
                                const float2 *table, int *err, cudaStream_t s) {
    if (n_blocks <= 0) return cudaSuccess;
#define KVM_SCALED(TI, D)                                                                     \
    return scaled_t<TI, D>(k_pages, k_scale, raw_out, index, index_cap, first_block, n_blocks, \
                           LG, table, err, s)
    if (index_dtype == BF16) {
        if (d == 128) KVM_SCALED(__nv_bfloat16, 128);
        KVM_SCALED(__nv_bfloat16, 64);
    }
    if (d == 128) KVM_SCALED(float, 128);
    KVM_SCALED(float, 64);
#undef KVM_SCALED
}

}  // namespace kvm
