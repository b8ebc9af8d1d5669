// The C ABI around the recall of one layer's attention (include/kvm.h): argument
// checks on the host, then one launch on the caller's stream.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "kvm.h"
#include "kvm_internal.cuh"

namespace {

kvm_status fail(kvm_status s, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    try {   // no exception crosses the C ABI
        kvm::set_last_error(buf);
    } catch (...) {
    }
    return s;
}

kvm_status launched(cudaError_t e, const char *what) {
    return e == cudaSuccess ? KVM_OK : fail(KVM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

int64_t elt_bytes(int dt) { return dt == KVM_E4M3 ? 1 : dt == KVM_BF16 ? 2 : 4; }

kvm_status aligned(const void *p, const char *what, bool vec) {
    if (vec && ((uintptr_t)p & 15) != 0)
        return fail(KVM_ERR_INVALID_ARG, "%s: not 16-byte aligned", what);
    if (!vec && ((uintptr_t)p & 3) != 0)
        return fail(KVM_ERR_INVALID_ARG, "%s: not 4-byte aligned", what);
    return KVM_OK;
}

// A buffer of these calls: device memory of the context's device (managed
// memory counts), 16-byte aligned where `vec`.
kvm_status on_device(const void *p, const kvm::CtxView &c, const char *what, bool vec = true) {
    if (!p) return KVM_OK;
    if (const kvm_status st = aligned(p, what, vec); st != KVM_OK) return st;
    cudaPointerAttributes a{};
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return fail(KVM_ERR_INVALID_ARG, "%s: not an address the GPU can use", what);
    }
    if (a.type == cudaMemoryTypeManaged) return KVM_OK;
    if (a.type != cudaMemoryTypeDevice)
        return fail(KVM_ERR_INVALID_ARG, "%s: not device memory", what);
    if (a.device != c.device)
        return fail(KVM_ERR_INVALID_ARG, "%s: memory of device %d, the context's is %d", what,
                    a.device, c.device);
    return KVM_OK;
}

// A buffer that may be pinned host memory too: the address a kernel uses.
kvm_status kernel_buffer(const void *p, const void **out, const char *what, bool vec = true) {
    if (const kvm_status st = aligned(p, what, vec); st != KVM_OK) return st;
    return static_cast<kvm_status>(kvm::resolve_kernel_ptr(p, out, what));
}

// The context's device has to be the current one: the launches go there.
kvm_status current_device(const kvm::CtxView &c) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return fail(KVM_ERR_CUDA, "no current device");
    }
    if (dev != c.device)
        return fail(KVM_ERR_INVALID_ARG, "current device %d, the context's is %d", dev, c.device);
    return KVM_OK;
}

kvm_status row_stride(int64_t stride, int64_t heads, int d, int dtype, const char *what) {
    if (stride < heads * d)
        return fail(KVM_ERR_INVALID_ARG, "%s: row stride %lld below a row's %lld elements", what,
                    (long long)stride, (long long)(heads * d));
    if ((stride * elt_bytes(dtype)) % 16 != 0)
        return fail(KVM_ERR_INVALID_ARG, "%s: row stride is not a multiple of 16 bytes", what);
    if (stride > ((int64_t)1 << 40))
        return fail(KVM_ERR_INVALID_ARG, "%s: row stride out of range", what);
    return KVM_OK;
}

#define KVM_TRY(call)                          \
    do {                                       \
        const kvm_status st_ = (call);         \
        if (st_ != KVM_OK) return st_;         \
    } while (0)

// Checks a batch and a cache and fills `b`.  *empty: nothing to do.
kvm_status batch_args(const kvm::CtxView &c, const kvm_batch *batch, const kvm_cache *cache,
                      int32_t layer, kvm::BatchArgs *b, bool *empty) {
    *empty = false;
    if (!batch || !cache) return fail(KVM_ERR_INVALID_ARG, "batch and cache are required");
    if (batch->n_seqs < 0 || batch->n_tokens < 0 || batch->max_q_len < 0 || batch->max_kv_len < 0)
        return fail(KVM_ERR_INVALID_ARG, "batch: negative size");
    if (batch->n_seqs > kvm::kMaxSeqs)
        return fail(KVM_ERR_CAPACITY, "batch: %d sequences, at most %d", batch->n_seqs,
                    kvm::kMaxSeqs);
    if (layer < 0 || layer >= c.L)
        return fail(KVM_ERR_INVALID_ARG, "layer %d of %d", layer, c.L);
    if (cache->n_pages < 0 || cache->n_scale_rows < 0)
        return fail(KVM_ERR_INVALID_ARG, "cache: negative size");
    if ((cache->k_scale == nullptr) != (cache->v_scale == nullptr))
        return fail(KVM_ERR_INVALID_ARG, "k_scale and v_scale must both be set or both be NULL");
    if (cache->k_scale && c.kv_dtype != KVM_E4M3)
        return fail(KVM_ERR_INVALID_ARG, "scales are for KVM_E4M3 pages");
    if (!cache->k_scale && (cache->n_scale_rows != 0 || batch->scale_rows))
        return fail(KVM_ERR_INVALID_ARG, "scale rows without scales");
    if (batch->n_seqs == 0 || batch->n_tokens == 0 || batch->max_q_len == 0) {
        *empty = true;
        return KVM_OK;
    }
    if (!batch->q_start || !batch->kv_len || !batch->page_table)
        return fail(KVM_ERR_INVALID_ARG, "batch: q_start, kv_len and page_table are required");
    if (!cache->k_pages || !cache->v_pages)
        return fail(KVM_ERR_INVALID_ARG, "cache: k_pages and v_pages are required");
    if (batch->table_stride < 1 ||
        ((int64_t)batch->max_kv_len + kvm::kBlockTokens - 1) / kvm::kBlockTokens >
            batch->table_stride)
        return fail(KVM_ERR_INVALID_ARG, "batch: max_kv_len %d beyond %lld page table entries",
                    batch->max_kv_len, (long long)batch->table_stride);
    // logical indexes, row numbers and work units are 32-bit
    if (batch->max_kv_len > 0x7FFFFFFF - 256 ||
        (int64_t)batch->max_q_len * (c.H / c.G) > 0x7FFFFFFF - 512)
        return fail(KVM_ERR_CAPACITY, "batch: max_kv_len or max_q_len out of range");
    KVM_TRY(current_device(c));
    KVM_TRY(on_device(batch->q_start, c, "q_start", false));
    KVM_TRY(on_device(batch->kv_len, c, "kv_len", false));
    KVM_TRY(on_device(batch->page_table, c, "page_table", false));
    KVM_TRY(on_device(batch->scale_rows, c, "scale_rows", false));
    KVM_TRY(on_device(cache->k_pages, c, "k_pages"));
    KVM_TRY(on_device(cache->v_pages, c, "v_pages"));
    KVM_TRY(on_device(cache->k_scale, c, "k_scale", false));
    KVM_TRY(on_device(cache->v_scale, c, "v_scale", false));
    b->n_seqs = batch->n_seqs;
    b->n_tokens = batch->n_tokens;
    b->max_q_len = batch->max_q_len;
    b->max_kv_len = batch->max_kv_len;
    b->q_start = batch->q_start;
    b->kv_len = batch->kv_len;
    b->page_table = batch->page_table;
    b->scale_rows = batch->scale_rows;
    b->table_stride = batch->table_stride;
    b->n_pages = cache->n_pages;
    b->n_scale_rows = cache->n_scale_rows;
    b->L = c.L;
    b->G = c.G;
    b->layer = layer;
    b->err = c.err;
    return KVM_OK;
}

}  // namespace

extern "C" {

kvm_status kvm_qk_norm_rope(kvm_ctx *ctx, int32_t n_tokens, const int32_t *positions,
                            const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                            const void *q_weight, const void *k_weight, float eps, void *q_free,
                            void *q_rot, void *k_free, void *k_rot, kvm_stream stream) {
    if (!ctx) return fail(KVM_ERR_INVALID_ARG, "ctx is NULL");
    const kvm::CtxView c = kvm::ctx_view(ctx);
    if (n_tokens < 0) return fail(KVM_ERR_INVALID_ARG, "n_tokens < 0");
    if (n_tokens == 0) return KVM_OK;   // (buffers of no tokens may have no address)
    if (!q && !k) return fail(KVM_ERR_INVALID_ARG, "q or k is required");
    if ((q != nullptr) != (q_free || q_rot) || (k != nullptr) != (k_free || k_rot))
        return fail(KVM_ERR_INVALID_ARG, "each given side needs an output, and only it");
    if ((!q && q_weight) || (!k && k_weight))
        return fail(KVM_ERR_INVALID_ARG, "a weight without its side");
    if ((q_free && q_free == q_rot) || (k_free && k_free == k_rot))
        return fail(KVM_ERR_INVALID_ARG, "free and rot outputs must differ");
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(KVM_ERR_INVALID_ARG, "eps must be >= 0");
    if (q) KVM_TRY(row_stride(q_stride, c.H, c.d, c.q_dtype, "q"));
    if (k) KVM_TRY(row_stride(k_stride, c.G, c.d, c.q_dtype, "k"));
    if (!positions) return fail(KVM_ERR_INVALID_ARG, "positions are required");
    // an output that is its own input has to have the input's rows
    if ((q && (q == q_free || q == q_rot) && q_stride != (int64_t)c.H * c.d) ||
        (k && (k == k_free || k == k_rot) && k_stride != (int64_t)c.G * c.d))
        return fail(KVM_ERR_INVALID_ARG, "in place needs packed rows");
    KVM_TRY(current_device(c));
    KVM_TRY(on_device(positions, c, "positions", false));
    KVM_TRY(on_device(q, c, "q"));
    KVM_TRY(on_device(k, c, "k"));
    KVM_TRY(on_device(q_weight, c, "q_weight"));
    KVM_TRY(on_device(k_weight, c, "k_weight"));
    KVM_TRY(on_device(q_free, c, "q_free"));
    KVM_TRY(on_device(q_rot, c, "q_rot"));
    KVM_TRY(on_device(k_free, c, "k_free"));
    KVM_TRY(on_device(k_rot, c, "k_rot"));
    kvm::NormArgs a{};
    a.n_tokens = n_tokens;
    a.H = c.H;
    a.G = c.G;
    a.d = c.d;
    a.positions = positions;
    a.q = q;
    a.k = k;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.eps = eps;
    a.q_free = q_free;
    a.q_rot = q_rot;
    a.k_free = k_free;
    a.k_rot = k_rot;
    a.table = c.table;
    a.max_positions = c.max_positions;
    a.err = c.err;
    return launched(kvm::launch_norm_rope(c.q_dtype, a, reinterpret_cast<cudaStream_t>(stream)),
                    "norm + rope launch");
}

kvm_status kvm_append_kv(kvm_ctx *ctx, const kvm_batch *batch, const kvm_cache *cache,
                         int32_t layer, const void *k, int64_t k_stride, const void *v,
                         int64_t v_stride, const int32_t *positions, void *raw_k_pages,
                         kvm_stream stream) {
    if (!ctx) return fail(KVM_ERR_INVALID_ARG, "ctx is NULL");
    const kvm::CtxView c = kvm::ctx_view(ctx);
    kvm::AppendArgs a{};
    bool empty;
    KVM_TRY(batch_args(c, batch, cache, layer, &a.b, &empty));
    if (empty) return KVM_OK;
    if (!k || !v) return fail(KVM_ERR_INVALID_ARG, "k and v are required");
    if (cache->k_pages == cache->v_pages || raw_k_pages == cache->k_pages ||
        raw_k_pages == cache->v_pages)
        return fail(KVM_ERR_INVALID_ARG, "K, V and raw K pages must differ");
    if (cache->k_scale && cache->k_scale == cache->v_scale)
        return fail(KVM_ERR_INVALID_ARG, "k_scale and v_scale must differ");
    if ((int64_t)a.b.n_seqs * kvm::append_spans(a.b.max_q_len) > 0x7FFFFFFF || c.G > 65535)
        return fail(KVM_ERR_CAPACITY, "batch: %d sequences of up to %d new tokens are too much for one call",
                    batch->n_seqs, batch->max_q_len);
    KVM_TRY(row_stride(k_stride, c.G, c.d, c.q_dtype, "k"));
    KVM_TRY(row_stride(v_stride, c.G, c.d, c.q_dtype, "v"));
    KVM_TRY(on_device(k, c, "k"));
    KVM_TRY(on_device(v, c, "v"));
    KVM_TRY(on_device(positions, c, "positions", false));
    KVM_TRY(on_device(raw_k_pages, c, "raw_k_pages"));
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.positions = positions;
    a.k_pages = cache->k_pages;
    a.v_pages = cache->v_pages;
    a.raw_pages = raw_k_pages;
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    a.table = c.table;
    a.max_positions = c.max_positions;
    return launched(kvm::launch_append(c.q_dtype, c.kv_dtype, c.d, a,
                                       reinterpret_cast<cudaStream_t>(stream)),
                    "append launch");
}

kvm_status kvm_attend(kvm_ctx *ctx, const kvm_batch *batch, const kvm_cache *cache,
                      int32_t layer, const void *q, int64_t q_stride, float softmax_scale,
                      int32_t causal, void *out, int64_t out_stride, float *lse,
                      kvm_stream stream) {
    if (!ctx) return fail(KVM_ERR_INVALID_ARG, "ctx is NULL");
    const kvm::CtxView c = kvm::ctx_view(ctx);
    kvm::AttendArgs a{};
    bool empty;
    KVM_TRY(batch_args(c, batch, cache, layer, &a.b, &empty));
    if (empty) return KVM_OK;
    if (!q || !out) return fail(KVM_ERR_INVALID_ARG, "q and out are required");
    if (causal != 0 && causal != 1) return fail(KVM_ERR_INVALID_ARG, "causal must be 0 or 1");
    // (beyond that, the factor in log2 units could overflow)
    if (!(std::fabs(softmax_scale) <= 1e30f))
        return fail(KVM_ERR_INVALID_ARG, "softmax_scale must be at most 1e30 in magnitude");
    KVM_TRY(row_stride(q_stride, c.H, c.d, c.q_dtype, "q"));
    KVM_TRY(row_stride(out_stride, c.H, c.d, c.q_dtype, "out"));
    if (q == out) return fail(KVM_ERR_INVALID_ARG, "out must not be q");
    KVM_TRY(on_device(q, c, "q"));
    KVM_TRY(on_device(out, c, "out"));
    KVM_TRY(on_device(lse, c, "lse", false));
    a.H = c.H;
    a.gqa = c.H / c.G;
    a.gqa_inv = a.gqa > 1 ? (uint32_t)(((1ull << 32) + a.gqa - 1) / a.gqa) : 0;
    a.d = c.d;
    a.q = q;
    a.q_stride = q_stride;
    a.k_pages = cache->k_pages;
    a.v_pages = cache->v_pages;
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    a.scale = softmax_scale;
    a.causal = causal;
    a.out = out;
    a.out_stride = out_stride;
    a.lse = lse;
    a.part = c.attend_part;
    a.count = c.attend_count;
    a.stall = kvm::take_injection(ctx, 4) ? 1 : 0;
    bool too_large = false;
    const cudaError_t e = kvm::launch_attend(c.q_dtype, c.kv_dtype, a,
                                             reinterpret_cast<cudaStream_t>(stream), &too_large);
    if (too_large)
        return fail(KVM_ERR_CAPACITY, "batch: %d sequences of up to %d x %d tokens are too much for one call",
                    batch->n_seqs, batch->max_q_len, batch->max_kv_len);
    return launched(e, "attention launch");
}

kvm_status kvm_build_index_scaled(kvm_ctx *ctx, const void *k_pages, const float *k_scale,
                                  int64_t first_block, int64_t n_blocks, void *index,
                                  void *raw_k_out, kvm_stream stream) {
    if (!ctx) return fail(KVM_ERR_INVALID_ARG, "ctx is NULL");
    const kvm::CtxView c = kvm::ctx_view(ctx);
    if (c.kv_dtype != KVM_E4M3)
        return fail(KVM_ERR_INVALID_ARG, "scales are for KVM_E4M3 pages");
    if (!k_pages || !k_scale || !index)
        return fail(KVM_ERR_INVALID_ARG, "k_pages, k_scale and index are required");
    if (first_block < 0 || n_blocks < 0)
        return fail(KVM_ERR_INVALID_ARG, "negative block range");
    if (first_block > c.max_blocks || n_blocks > c.max_blocks - first_block)
        return fail(KVM_ERR_CAPACITY, "blocks [%lld, +%lld) beyond max_blocks %lld",
                    (long long)first_block, (long long)n_blocks, (long long)c.max_blocks);
    if ((first_block + n_blocks) * kvm::kBlockTokens > c.max_positions)
        return fail(KVM_ERR_CAPACITY, "positions up to %lld beyond max_positions %lld",
                    (long long)((first_block + n_blocks) * kvm::kBlockTokens),
                    (long long)c.max_positions);
    if (n_blocks == 0) return KVM_OK;
    KVM_TRY(current_device(c));
    // buffers as kvm_build_index takes them: pinned host memory too
    const void *pages, *scales, *idx, *raw;
    KVM_TRY(kernel_buffer(k_pages, &pages, "k_pages"));
    KVM_TRY(kernel_buffer(k_scale, &scales, "k_scale", false));
    KVM_TRY(kernel_buffer(index, &idx, "index"));
    KVM_TRY(kernel_buffer(raw_k_out, &raw, "raw_k_out"));
    return launched(
        kvm::launch_meank_scaled(c.index_dtype, c.d, pages, static_cast<const float *>(scales),
                                 const_cast<void *>(raw), const_cast<void *>(idx), c.max_blocks,
                                 first_block, n_blocks, c.L * c.G, c.table, c.err,
                                 reinterpret_cast<cudaStream_t>(stream)),
        "scaled meank launch");
}

}  // extern "C"
