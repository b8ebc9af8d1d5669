// Queries and keys normalised per head and rotated, in one pass.
//
// y = x * rsqrt(mean(x^2) + eps) * w over a head's d entries, then rotate-half
// RoPE at the token's position.  Both the RoPE-free y (what KVMem's block
// scoring, Eq. (10) of "KVMem: Virtualizing Million-Token Agent Workspaces on a
// Consumer GPU" §4.3, takes as queries, and what is kept as raw K) and the
// rotated R_p y (what attention takes) come out of one read of x.
//
// A head is d entries of one token: D/2/N lanes hold it, each a 16-byte vector
// of the first half and its rotate-half partners in the second, so the sum of
// squares needs log2(lanes) shuffles and the rotation none.  A warp stays with
// one token for a run of heads, so the token's cos/sin are read once into
// registers.  Memory bound: (1 + outputs) * (H + G) * d elements a token.  8192
// tokens of 48 + 8 heads of 128 in bf16 with both outputs (357 MB) take 59 us, 6.0
// TB/s; one token takes 2.6 us, split over warps down to one load of each lane.
#include "kvm_internal.cuh"
#include "kvm_vec.cuh"

namespace kvm {

constexpr int kNormWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kNormWarps * 32)
norm_rope_kernel(NormArgs a, int chunk, int n_chunks) {
    using VT = VecTraits<T>;
    using V = typename VT::V;
    constexpr int N = VT::N, HD = D / 2, TPT = HD / N, RPW = 32 / TPT;
    const int lane = threadIdx.x & 31, c = lane % TPT, sub = lane / TPT;
    const int64_t unit = (int64_t)blockIdx.x * kNormWarps + (threadIdx.x >> 5);
    const int64_t tok = unit / n_chunks;
    if (tok >= a.n_tokens) return;
    const int h0 = (int)(unit - tok * n_chunks) * chunk;
    const int Hq = a.q != nullptr ? a.H : 0, Hall = Hq + (a.k != nullptr ? a.G : 0);
    const int64_t pos = a.positions[tok];
    if (pos < 0 || pos >= a.max_positions) {
        if (lane == 0) atomicOr(a.err, kErrBatch);
        return;
    }
    float cs[N], sn[N];
    {
        const float4 *t4 = reinterpret_cast<const float4 *>(a.table + pos * HD + c * N);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float4 w = __ldg(t4 + i);
            cs[2 * i] = w.x;
            sn[2 * i] = w.y;
            cs[2 * i + 1] = w.z;
            sn[2 * i + 1] = w.w;
        }
    }
    const int h1 = min(Hall, h0 + chunk);
    for (int hb = h0; hb < h1; hb += RPW) {
        const int h = hb + sub;
        const bool on = h < h1;
        const bool is_q = h < Hq;
        const int hh = is_q ? h : h - Hq;
        float x[N], y[N];
        if (on) {
            const T *src = is_q ? static_cast<const T *>(a.q) + tok * a.q_stride
                                : static_cast<const T *>(a.k) + tok * a.k_stride;
            V vx, vy;
            ld_stream_v(src + (size_t)hh * D + c * N, vx);
            ld_stream_v(src + (size_t)hh * D + HD + c * N, vy);
            VT::unpack(vx, x);
            VT::unpack(vy, y);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = y[i] = 0.f;
        }
        const T *w = static_cast<const T *>(is_q ? a.q_weight : a.k_weight);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) ss += x[i] * x[i] + y[i] * y[i];
#pragma unroll
        for (int o = TPT / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (!on) continue;
        if (w != nullptr) {
            const float r = rsqrtf(ss * (1.0f / D) + a.eps);
            float wx[N], wy[N];
            VT::unpack(__ldg(reinterpret_cast<const V *>(w + c * N)), wx);
            VT::unpack(__ldg(reinterpret_cast<const V *>(w + HD + c * N)), wy);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                x[i] = x[i] * r * wx[i];
                y[i] = y[i] * r * wy[i];
            }
        }
        const size_t off = ((size_t)tok * (is_q ? a.H : a.G) + hh) * D + c * N;
        T *free_out = static_cast<T *>(is_q ? a.q_free : a.k_free);
        T *rot_out = static_cast<T *>(is_q ? a.q_rot : a.k_rot);
        if (free_out != nullptr) {
            *reinterpret_cast<V *>(free_out + off) = VT::pack(x);
            *reinterpret_cast<V *>(free_out + off + HD) = VT::pack(y);
        }
        if (rot_out != nullptr) {
            float ox[N], oy[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                ox[i] = __fsub_rn(__fmul_rn(x[i], cs[i]), __fmul_rn(y[i], sn[i]));
                oy[i] = __fadd_rn(__fmul_rn(x[i], sn[i]), __fmul_rn(y[i], cs[i]));
            }
            *reinterpret_cast<V *>(rot_out + off) = VT::pack(ox);
            *reinterpret_cast<V *>(rot_out + off + HD) = VT::pack(oy);
        }
    }
}

template <typename T, int D>
static cudaError_t norm_t(const NormArgs &a, cudaStream_t s) {
    constexpr int RPW = 32 / (D / 2 / VecTraits<T>::N);
    const int heads = (a.q ? a.H : 0) + (a.k ? a.G : 0);
    int chunk = heads;
    // few tokens: a warp takes fewer heads, down to one load of each lane
    while (chunk > RPW &&
           (int64_t)a.n_tokens * ((heads + chunk - 1) / chunk) < (int64_t)sm_count() * 64)
        chunk = ((chunk + 1) / 2 + RPW - 1) / RPW * RPW;
    const int n_chunks = (heads + chunk - 1) / chunk;
    const int64_t units = (int64_t)a.n_tokens * n_chunks;
    const int64_t ctas = (units + kNormWarps - 1) / kNormWarps;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
    norm_rope_kernel<T, D><<<(unsigned)ctas, kNormWarps * 32, 0, s>>>(a, chunk, n_chunks);
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_norm_rope(int dtype, const NormArgs &a, cudaStream_t s) {
    if (a.n_tokens <= 0) return cudaSuccess;
    if (dtype == BF16)
        return a.d == 128 ? norm_t<__nv_bfloat16, 128>(a, s) : norm_t<__nv_bfloat16, 64>(a, s);
    return a.d == 128 ? norm_t<float, 128>(a, s) : norm_t<float, 64>(a, s);
}

}  // namespace kvm
