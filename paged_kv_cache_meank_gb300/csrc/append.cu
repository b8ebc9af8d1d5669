// New keys and values into a paged cache, K rotated on the way.
//
// A CTA owns one (sequence, block, kv head): the up to 32 new rows that fall into
// that block, K by four warps and V by the other four.  They read the rows once
// into registers, a 16-byte vector of the first half of a row and its rotate-half
// partners per lane, at most four such pairs (with a warp to a block's K or V the
// rows took 112 to 182 registers, and 8192 tokens of e4m3 pages with raw K 19.2 us
// against 15.6; their 59 MB cannot take less than 8.6.  Into bf16 pages, 12.2 us for 67
// MB, with raw K 13.4 for 84).  For scaled e4m3 pages
// the largest finite entry sets the block's power-of-two scale; no other CTA
// touches the block and head, so the scale, the codes already there and the new
// rows change without atomics.  The scale bounds |k| * sqrt(2), the largest entry
// that any rotation can make, so it holds at every position the block is rotated
// to later (KVMem, "Virtualizing Million-Token Agent Workspaces on a Consumer
// GPU", §4.4: raw K re-rotated at compact positions), and raw K shares it.
// Memory bound: 2 G d elements read and 2 G d (3 with raw K) written a token.
#include "kvm_internal.cuh"
#include "kvm_vec.cuh"

namespace kvm {

constexpr int kParts = 4;                  // warps of a block's K or V, 32 / kParts rows each
constexpr int kAppendThreads = 2 * kParts * 32;
// The largest raw entry a block of scale 1 takes (e4m3: 448 / sqrt(2) rounded
// down for K, 448 for V), as mantissa in [1, 2) times 2^8.
constexpr float kMostK = 316.75f, kMostV = 448.0f;
constexpr int kScaleLeast = -100, kScaleMost = 119;

// The least e with amax <= most * 2^e, clamped; amax finite and >= 0, most in
// [2^8, 2^9).
__device__ inline int scale_exponent(float amax, float most) {
    const int a = (int)(__float_as_uint(amax) >> 23) - 127;
    const uint32_t ma = __float_as_uint(amax) & 0x7FFFFFu, mm = __float_as_uint(most) & 0x7FFFFFu;
    return min(kScaleMost, max(kScaleLeast, a - 8 + (ma > mm ? 1 : 0)));
}
__device__ inline float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

template <typename T, typename TP, int D, bool SCALED>
__global__ void __launch_bounds__(kAppendThreads)
append_kernel(AppendArgs a, int spans) {
    using VI = VecTraits<T>;
    using VP = VecTraits<TP>;
    // a lane's piece of a half row, in elements: the input's vector (8 bf16, or
    // 4 float32; a page vector of 8 e4m3 takes two float32 pieces' place)
    constexpr int N = VI::N, HD = D / 2, TPT = HD / N, RPW = 32 / TPT;
    constexpr int ITERS = kBlockTokens / kParts / RPW;
    using V = typename VI::V;
    const int lane = threadIdx.x & 31, c = lane % TPT, sub = lane / TPT;
    const int seq = blockIdx.x / spans, span = blockIdx.x - seq * spans;
    const int g = blockIdx.y, warp = threadIdx.x >> 5, part = warp % kParts;
    const bool is_k = warp < kParts;
    __shared__ float top[2 * kParts];                   // largest entry of each warp

    const int q0 = a.b.q_start[seq], q1 = a.b.q_start[seq + 1], kv = a.b.kv_len[seq];
    const int q_len = q1 - q0;
    if (q0 < 0 || q1 < q0 || q1 > a.b.n_tokens || q_len > a.b.max_q_len || kv < q_len ||
        kv > a.b.max_kv_len) {
        if (threadIdx.x == 0) atomicOr(a.b.err, kErrBatch);
        return;
    }
    const int first = kv - q_len;                       // logical index of token 0
    const int blk = first / kBlockTokens + span;
    const int lo = max(first, blk * kBlockTokens), hi = min(kv, (blk + 1) * kBlockTokens);
    if (lo >= hi) return;
    const int r0 = lo - blk * kBlockTokens, n = hi - lo;   // rows [r0, r0 + n) of the page
    const int tok0 = q0 + lo - first;

    // the rows are asked for before their page is looked up: one wait, not two
    const T *src = is_k ? static_cast<const T *>(a.k) : static_cast<const T *>(a.v);
    const int64_t stride = is_k ? a.k_stride : a.v_stride;
    V vx[ITERS], vy[ITERS];
    uint32_t on = 0;                                    // bit i: this lane's row i is written
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
        const int j = (part * ITERS + i) * RPW + sub;
        if (j < n) {
            const int64_t pos = a.positions ? (int64_t)a.positions[tok0 + j] : (int64_t)(lo + j);
            if (pos < 0 || pos >= a.max_positions) {
                atomicOr(a.b.err, kErrBatch);
                continue;
            }
            on |= 1u << i;
            const T *p = src + (int64_t)(tok0 + j) * stride + (int64_t)g * D + c * N;
            ld_stream_v(p, vx[i]);
            ld_stream_v(p + HD, vy[i]);
        }
    }
    const int64_t at = (int64_t)seq * a.b.table_stride + blk;
    const int64_t page = a.b.page_table[at];
    const int64_t srow = SCALED && a.b.scale_rows ? (int64_t)a.b.scale_rows[at] : page;
    if (page < 0 || page >= a.b.n_pages || (SCALED && (srow < 0 || srow >= a.b.n_scale_rows))) {
        if (threadIdx.x == 0) atomicOr(a.b.err, kErrBatch);
        return;
    }
    const size_t head = (((size_t)page * a.b.L + a.b.layer) * a.b.G + g) * kBlockTokens * D;
    TP *dst = (is_k ? static_cast<TP *>(a.k_pages) : static_cast<TP *>(a.v_pages)) + head;
    TP *raw = is_k && a.raw_pages ? static_cast<TP *>(a.raw_pages) + head : nullptr;

    float inv = 1.f, most = 448.f;                      // most: what an infinite entry counts as
    bool odd = false;                                   // this lane has infinities or NaN
    if constexpr (SCALED) {
        const size_t so = ((size_t)srow * a.b.L + a.b.layer) * a.b.G + g;
        float *sp = (is_k ? a.k_scale : a.v_scale) + so;
        // read by all before one writes; K's and V's, as the block is left as it was where
        // either is no scale
        const float old_k = r0 > 0 ? a.k_scale[so] : 1.f, old_v = r0 > 0 ? a.v_scale[so] : 1.f;
        // magnitudes compare as integers, infinities and NaN above all others: only where
        // this lane has one of them are they told apart
        uint32_t top_bits = 0;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            if (on >> i & 1) {
                float x[N], y[N];
                VI::unpack(vx[i], x);
                VI::unpack(vy[i], y);
#pragma unroll
                for (int k = 0; k < N; ++k)
                    top_bits = max(top_bits, max(__float_as_uint(x[k]) & 0x7FFFFFFFu,
                                                 __float_as_uint(y[k]) & 0x7FFFFFFFu));
            }
        }
        odd = top_bits >= 0x7F800000u;
        float amax = odd ? 0.f : __uint_as_float(top_bits);
        if (odd) {
#pragma unroll
            for (int i = 0; i < ITERS; ++i) {
                if (on >> i & 1) {
                    float x[N], y[N];
                    VI::unpack(vx[i], x);
                    VI::unpack(vy[i], y);
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        const float ax = fabsf(x[k]), ay = fabsf(y[k]);
                        if (ax < INFINITY) amax = fmaxf(amax, ax);   // NaN compares false
                        if (ay < INFINITY) amax = fmaxf(amax, ay);
                    }
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (lane == 0) top[warp] = amax;
        if (!__syncthreads_or(on != 0)) return;         // (K's and V's positions are the same)
        if (!is_scale(old_k) || !is_scale(old_v)) {     // (the same for all)
            if (threadIdx.x == 0) atomicOr(a.b.err, kErrScale);
            return;
        }
#pragma unroll
        for (int w = 0; w < kParts; ++w) amax = fmaxf(amax, top[warp - part + w]);
        float scale = pow2f(scale_exponent(amax, is_k ? kMostK : kMostV));
        if (r0 > 0) {
            const float had = is_k ? old_k : old_v;
            if (had >= scale) {
                scale = had;
            } else {
                // the codes of the rows before follow the larger scale
                const float f = had / scale;
                const int vecs = r0 * (D / VP::N);
                for (int i = part * 32 + lane; i < vecs; i += kParts * 32) {
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        TP *p = w == 0 ? dst : raw;
                        if (p == nullptr) continue;
                        auto *vp = reinterpret_cast<typename VP::V *>(p) + i;
                        float x[VP::N];
                        VP::unpack(*vp, x);
#pragma unroll
                        for (int k = 0; k < VP::N; ++k) x[k] *= f;
                        *vp = VP::pack(x);
                    }
                }
            }
        }
        if (part == 0 && lane == 0) *sp = scale;
        inv = 1.f / scale;                              // exact: a power of two
        most = 448.f * scale;
    }

#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
        const int j = (part * ITERS + i) * RPW + sub;
        if (!(on >> i & 1)) continue;
        float x[N], y[N], ox[N], oy[N];
        VI::unpack(vx[i], x);
        VI::unpack(vy[i], y);
        TP *row = dst + (size_t)(r0 + j) * D + c * N;
        if (is_k) {
            // infinity times a sine of 0, or infinity less infinity, would be NaN
            if (SCALED && odd) {
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    if (fabsf(x[k]) == INFINITY) x[k] = copysignf(most, x[k]);
                    if (fabsf(y[k]) == INFINITY) y[k] = copysignf(most, y[k]);
                }
            }
            const int64_t pos = a.positions ? (int64_t)a.positions[tok0 + j] : (int64_t)(lo + j);
            const float4 *t = reinterpret_cast<const float4 *>(a.table + pos * HD + c * N);
#pragma unroll
            for (int k = 0; k < N; k += 2) {
                const float4 w = __ldg(t + k / 2);
                ox[k] = __fsub_rn(__fmul_rn(x[k], w.x), __fmul_rn(y[k], w.y)) * inv;
                oy[k] = __fadd_rn(__fmul_rn(x[k], w.y), __fmul_rn(y[k], w.x)) * inv;
                ox[k + 1] = __fsub_rn(__fmul_rn(x[k + 1], w.z), __fmul_rn(y[k + 1], w.w)) * inv;
                oy[k + 1] = __fadd_rn(__fmul_rn(x[k + 1], w.w), __fmul_rn(y[k + 1], w.z)) * inv;
            }
            if (raw != nullptr) {
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    x[k] *= inv;
                    y[k] *= inv;
                }
                TP *rr = raw + (size_t)(r0 + j) * D + c * N;
                store_n<TP, N>(rr, x);
                store_n<TP, N>(rr + HD, y);
            }
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                ox[k] = x[k] * inv;
                oy[k] = y[k] * inv;
            }
        }
        store_n<TP, N>(row, ox);
        store_n<TP, N>(row + HD, oy);
    }
}

template <typename T, typename TP, int D, bool SCALED>
static cudaError_t append_t(const AppendArgs &a, cudaStream_t s) {
    const int spans = append_spans(a.b.max_q_len);      // (the host has checked the grid's size)
    append_kernel<T, TP, D, SCALED>
        <<<dim3((unsigned)(a.b.n_seqs * spans), (unsigned)a.b.G), kAppendThreads, 0, s>>>(a, spans);
    note_launch();
    return cudaGetLastError();
}

template <typename T, int D>
static cudaError_t append_kv(int kv_dtype, const AppendArgs &a, cudaStream_t s) {
    if (kv_dtype == F32) return append_t<T, float, D, false>(a, s);
    if (kv_dtype == BF16) return append_t<T, __nv_bfloat16, D, false>(a, s);
    return a.k_scale ? append_t<T, e4m3, D, true>(a, s) : append_t<T, e4m3, D, false>(a, s);
}

cudaError_t launch_append(int q_dtype, int kv_dtype, int d, const AppendArgs &a, cudaStream_t s) {
    if (a.b.n_seqs <= 0 || a.b.n_tokens <= 0 || a.b.max_q_len <= 0) return cudaSuccess;
    if (q_dtype == BF16)
        return d == 128 ? append_kv<__nv_bfloat16, 128>(kv_dtype, a, s)
                        : append_kv<__nv_bfloat16, 64>(kv_dtype, a, s);
    return d == 128 ? append_kv<float, 128>(kv_dtype, a, s) : append_kv<float, 64>(kv_dtype, a, s);
}

}  // namespace kvm
