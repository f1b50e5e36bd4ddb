// kv4_api.cu -- the C entry points of the 4-bit paged KV cache (declared in
// include/nmspmv.h): argument checks and dispatch.
#include <cmath>

#include "kv4.cuh"

namespace nm {
namespace {

bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

bool sizes_ok(int page_tokens, int n_layers, int n_kv_heads, int head_dim)
{
    return (page_tokens == 16 || page_tokens == 32 || page_tokens == 64 || page_tokens == 128) && n_layers > 0 &&
           n_kv_heads > 0 && n_layers <= 65536 && n_kv_heads <= 65536 && (head_dim == 64 || head_dim == 128);
}

int64_t round_up(int64_t x, int64_t n) { return (x + n - 1) / n * n; }

// The cache's own arguments; *c, *w: what the kernels get. The status word is
// looked up last, so that every refusal comes before the first CUDA call.
nm_status check_cache(const nm_kv4_cache *k, bool need_pool)
{
    if (!k)
        return NM_ERR_INVALID_ARG;
    if (!sizes_ok(k->page_tokens, k->n_layers, k->n_kv_heads, k->head_dim))
        return NM_ERR_UNSUPPORTED;
    if (k->n_pages < 0 || k->n_pages > 0x3FFFFFFF || k->max_seqs < 0 || k->max_pages < 0 ||
        (int64_t)k->max_pages * k->page_tokens > 0x3FFFFFFF)
        return NM_ERR_SHAPE;
    if (!k->info || !k->lens || !k->refs || !k->tables || !k->workspace || (need_pool && k->n_pages > 0 && !k->pool))
        return NM_ERR_INVALID_ARG;
    if (!aligned(k->info, 16) || !aligned(k->lens, 16) || !aligned(k->refs, 16) || !aligned(k->tables, 16) ||
        !aligned(k->workspace, 256) || !aligned(k->pool, 128))
        return NM_ERR_ALIGN;
    if (k->workspace_bytes < nm_kv4_workspace_bytes(k->n_pages, k->head_dim))
        return NM_ERR_SHAPE;
    return NM_OK;
}

nm_status view(const nm_kv4_cache *k, Kv4 *c, Kv4Work *w, int *num_sms)
{
    nm_status s = library_status_word(&c->status);
    if (s != NM_OK)
        return s;
    static std::atomic<int> sms[kMaxDevices] = {}; // 0: not asked for yet; threads that ask at once get the same
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return NM_ERR_CUDA;
    int n = sms[dev].load(std::memory_order_relaxed);
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            return NM_ERR_CUDA;
        sms[dev].store(n, std::memory_order_relaxed);
    }
    w->device = dev;
    w->num_sms = *num_sms = n;
    if (2 * *num_sms > (int)kKv4Counters / 4)
        return NM_ERR_UNSUPPORTED;
    c->pool = (uint8_t *)k->pool;
    c->n_pages = k->n_pages;
    c->page_bytes = nm_kv4_page_bytes(k->page_tokens, k->n_layers, k->n_kv_heads, k->head_dim);
    c->page_tokens = k->page_tokens;
    c->page_shift = k->page_tokens == 16 ? 4 : k->page_tokens == 32 ? 5 : k->page_tokens == 64 ? 6 : 7;
    c->n_layers = k->n_layers;
    c->n_kv_heads = k->n_kv_heads;
    c->head_dim = k->head_dim;
    c->max_seqs = k->max_seqs;
    c->max_pages = k->max_pages;
    c->info = k->info;
    c->lens = k->lens;
    c->refs = k->refs;
    c->tables = k->tables;
    uint8_t *p = (uint8_t *)k->workspace;
    w->counters = (uint32_t *)p;
    p += kKv4Counters * 4;
    w->list = (int32_t *)p;
    p += round_up((64 + 2 * k->n_pages + kKv4MaxSeqs) * 4, 256);
    w->partials = (float *)p;
    return NM_OK;
}

nm_status check_list(int n, bool have)
{
    if (n < 0)
        return NM_ERR_INVALID_ARG;
    if (n > kKv4MaxSeqs)
        return NM_ERR_UNSUPPORTED;
    return n > 0 && !have ? NM_ERR_INVALID_ARG : NM_OK;
}

// n_seqs, starts and n_tokens of a call over token arrays.
nm_status check_batch(const int32_t *starts, int n_seqs, int64_t n_tokens)
{
    nm_status s = check_list(n_seqs, true);
    if (s != NM_OK)
        return s;
    if (n_tokens < 0 || n_tokens > 0x3FFFFFFF || (!starts && n_tokens != n_seqs))
        return NM_ERR_SHAPE;
    return NM_OK;
}

// A token array of `heads` heads with token stride `stride`.
nm_status check_tokens(const void *p, int64_t stride, int64_t heads, int head_dim)
{
    if (!p)
        return NM_ERR_INVALID_ARG;
    if (!aligned(p, 16))
        return NM_ERR_ALIGN;
    return stride % 8 != 0 || stride < heads * head_dim ? NM_ERR_SHAPE : NM_OK;
}

__global__ void __launch_bounds__(256) init_kernel(const Kv4 c, uint32_t *counters)
{
    const int64_t i0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = i0; i < (int64_t)c.max_seqs * c.max_pages; i += step)
        c.tables[i] = -1;
    for (int64_t i = i0; i < c.n_pages; i += step)
        c.refs[i] = 0;
    for (int64_t i = i0; i < c.max_seqs; i += step)
        c.lens[i] = 0;
    for (int64_t i = i0; i < 16; i += step)
        c.info[i] = i == 0 ? (int32_t)c.n_pages : 0;
    for (int64_t i = i0; i < (int64_t)kKv4Counters; i += step)
        counters[i] = 0;
}

} // namespace
} // namespace nm

using namespace nm;

extern "C" {

int64_t nm_kv4_page_bytes(int page_tokens, int n_layers, int n_kv_heads, int head_dim)
{
    if (!sizes_ok(page_tokens, n_layers, n_kv_heads, head_dim))
        return 0;
    const int64_t cell = head_dim == 128 ? Kv4Cell<128>::kBytes : Kv4Cell<64>::kBytes;
    return (int64_t)n_layers * n_kv_heads * (page_tokens / kKv4Cell) * cell;
}

int64_t nm_kv4_workspace_bytes(int64_t n_pages, int head_dim)
{
    if (n_pages < 0 || n_pages > 0x3FFFFFFF || (head_dim != 64 && head_dim != 128))
        return 0;
    return (int64_t)kKv4Counters * 4 + round_up((64 + 2 * n_pages + kKv4MaxSeqs) * 4, 256) +
           (int64_t)kv4_partial_bytes(head_dim);
}

nm_status nm_kv4_init(const nm_kv4_cache *cache, void *stream)
{
    NvtxRange nvtx_("nm_kv4_init");
    nm_status s = check_cache(cache, false);
    if (s != NM_OK)
        return s;
    Kv4 c;
    Kv4Work w;
    int sms;
    if ((s = view(cache, &c, &w, &sms)) != NM_OK)
        return s;
    init_kernel<<<sms, 256, 0, (cudaStream_t)stream>>>(c, w.counters);
    return cudaGetLastError() == cudaSuccess ? NM_OK : NM_ERR_CUDA;
}

nm_status nm_kv4_reserve(const nm_kv4_cache *cache, const int32_t *seqs, const int32_t *starts, int n_seqs,
                         void *stream)
{
    NvtxRange nvtx_("nm_kv4_reserve");
    nm_status s = check_cache(cache, false);
    if (s != NM_OK || (s = check_list(n_seqs, true)) != NM_OK)
        return s;
    Kv4 c;
    Kv4Work w;
    int sms;
    if ((s = view(cache, &c, &w, &sms)) != NM_OK)
        return s;
    return kv4_launch_reserve(c, seqs, starts, n_seqs, w, (cudaStream_t)stream);
}

nm_status nm_kv4_fork(const nm_kv4_cache *cache, const int32_t *src, const int32_t *dst, int n, void *stream)
{
    NvtxRange nvtx_("nm_kv4_fork");
    nm_status s = check_cache(cache, true);
    if (s != NM_OK || (s = check_list(n, src && dst)) != NM_OK)
        return s;
    Kv4 c;
    Kv4Work w;
    int sms;
    if ((s = view(cache, &c, &w, &sms)) != NM_OK)
        return s;
    return kv4_launch_fork(c, src, dst, n, w, sms, (cudaStream_t)stream);
}

nm_status nm_kv4_free(const nm_kv4_cache *cache, const int32_t *seqs, int n, void *stream)
{
    NvtxRange nvtx_("nm_kv4_free");
    nm_status s = check_cache(cache, false);
    if (s != NM_OK || (s = check_list(n, true)) != NM_OK || n == 0)
        return s;
    Kv4 c;
    Kv4Work w;
    int sms;
    if ((s = view(cache, &c, &w, &sms)) != NM_OK)
        return s;
    return kv4_launch_free(c, seqs, n, (cudaStream_t)stream);
}

nm_status nm_kv4_compact(const nm_kv4_cache *cache, void *stream)
{
    NvtxRange nvtx_("nm_kv4_compact");
    nm_status s = check_cache(cache, true);
    if (s != NM_OK || cache->n_pages == 0)
        return s;
    Kv4 c;
    Kv4Work w;
    int sms;
    if ((s = view(cache, &c, &w, &sms)) != NM_OK)
        return s;
    return kv4_launch_compact(c, w, sms, (cudaStream_t)stream);
}

nm_status nm_kv4_copy_pages(const nm_kv4_cache *src, const int32_t *src_pages, const nm_kv4_cache *dst,
                            const int32_t *dst_pages, int64_t n, void *stream)
{
    NvtxRange nvtx_("nm_kv4_copy_pages");
    nm_status s = check_cache(src, true);
    if (s != NM_OK || (s = check_cache(dst, true)) != NM_OK)
        return s;
    if (src->page_tokens != dst->page_tokens || src->n_layers != dst->n_layers ||
        src->n_kv_heads != dst->n_kv_heads || src->head_dim != dst->head_dim || n < 0 || n > 0x3FFFFFFF)
        return NM_ERR_SHAPE;
    if (n == 0)
        return NM_OK;
    if (!src_pages || !dst_pages)
        return NM_ERR_INVALID_ARG;
    Kv4 c;
    Kv4Work w;
    int sms;
    if ((s = view(src, &c, &w, &sms)) != NM_OK)
        return s;
    return kv4_launch_copy(c.pool, c.n_pages, src_pages, (uint8_t *)dst->pool, dst->n_pages, dst_pages, c.page_bytes, n,
                           c.status, sms, (cudaStream_t)stream);
}

nm_status nm_kv4_append(const nm_kv4_cache *cache, int layer, const int32_t *seqs, const int32_t *starts, int n_seqs,
                        int64_t n_tokens, const void *k_bf16, int64_t k_stride, const void *v_bf16, int64_t v_stride,
                        const void *q_bf16, int64_t q_stride, int n_q_heads, void *q_out_bf16, int64_t q_out_stride,
                        const float *rope, int64_t rope_rows, void *stream)
{
    NvtxRange nvtx_("nm_kv4_append");
    nm_status s = check_cache(cache, true);
    if (s != NM_OK || (s = check_batch(starts, n_seqs, n_tokens)) != NM_OK)
        return s;
    if (layer < 0 || layer >= cache->n_layers || n_q_heads < 0 || n_q_heads > 65536 || rope_rows < 0)
        return NM_ERR_SHAPE;
    if (n_tokens == 0)
        return NM_OK;
    const int D = cache->head_dim;
    if ((s = check_tokens(k_bf16, k_stride, cache->n_kv_heads, D)) != NM_OK ||
        (s = check_tokens(v_bf16, v_stride, cache->n_kv_heads, D)) != NM_OK)
        return s;
    const bool q = q_bf16 && n_q_heads > 0;
    if (q && ((s = check_tokens(q_bf16, q_stride, n_q_heads, D)) != NM_OK ||
              (s = check_tokens(q_out_bf16, q_out_stride, n_q_heads, D)) != NM_OK))
        return s;
    if (q && q_bf16 == q_out_bf16 && q_stride != q_out_stride)
        return NM_ERR_SHAPE;
    if (rope && !aligned(rope, 16))
        return NM_ERR_ALIGN;
    Kv4 c;
    Kv4Work w;
    int sms;
    if ((s = view(cache, &c, &w, &sms)) != NM_OK)
        return s;
    const Kv4Batch b{seqs, starts, n_seqs, n_tokens};
    return kv4_launch_append(c, b, layer, k_bf16, k_stride, v_bf16, v_stride, q ? q_bf16 : nullptr, q_stride,
                             n_q_heads, q_out_bf16, q_out_stride, rope, rope_rows, (cudaStream_t)stream);
}

nm_status nm_kv4_read(const nm_kv4_cache *cache, int layer, const int32_t *seqs, const int32_t *starts, int n_seqs,
                      int64_t n_tokens, void *k, void *v, int f32, void *stream)
{
    NvtxRange nvtx_("nm_kv4_read");
    nm_status s = check_cache(cache, true);
    if (s != NM_OK || (s = check_batch(starts, n_seqs, n_tokens)) != NM_OK)
        return s;
    if (layer < 0 || layer >= cache->n_layers)
        return NM_ERR_SHAPE;
    if (n_tokens == 0 || (!k && !v))
        return NM_OK;
    if (!aligned(k, 16) || !aligned(v, 16))
        return NM_ERR_ALIGN;
    Kv4 c;
    Kv4Work w;
    int sms;
    if ((s = view(cache, &c, &w, &sms)) != NM_OK)
        return s;
    const Kv4Batch b{seqs, starts, n_seqs, n_tokens};
    return kv4_launch_read(c, b, layer, k, v, f32 != 0, (cudaStream_t)stream);
}

nm_status nm_kv4_attention(const nm_kv4_cache *cache, int layer, const int32_t *seqs, const int32_t *starts,
                           int n_seqs, int64_t n_tokens, int64_t max_new, const void *q_bf16, int64_t q_stride,
                           int n_q_heads, float scale, void *out_bf16, int64_t out_stride, float *lse, void *stream)
{
    NvtxRange nvtx_("nm_kv4_attention");
    nm_status s = check_cache(cache, true);
    if (s != NM_OK || (s = check_batch(starts, n_seqs, n_tokens)) != NM_OK)
        return s;
    if (layer < 0 || layer >= cache->n_layers || n_q_heads <= 0 || n_q_heads % cache->n_kv_heads != 0)
        return NM_ERR_SHAPE;
    if (n_q_heads / cache->n_kv_heads > 64)
        return NM_ERR_UNSUPPORTED;
    if (max_new < 1 || !std::isfinite(scale))
        return NM_ERR_INVALID_ARG;
    if (n_tokens * n_q_heads > 0x3FFFFFFF)
        return NM_ERR_SHAPE;
    if (n_tokens == 0)
        return NM_OK;
    const int D = cache->head_dim;
    if ((s = check_tokens(q_bf16, q_stride, n_q_heads, D)) != NM_OK ||
        (s = check_tokens(out_bf16, out_stride, n_q_heads, D)) != NM_OK)
        return s;
    if (lse && !aligned(lse, 16))
        return NM_ERR_ALIGN;
    Kv4 c;
    Kv4Work w;
    int sms;
    if ((s = view(cache, &c, &w, &sms)) != NM_OK)
        return s;
    const Kv4Batch b{seqs, starts, n_seqs, n_tokens};
    const Kv4Attn a{layer, q_bf16, q_stride, n_q_heads, scale, out_bf16, out_stride, lse};
    return kv4_launch_attention(c, b, a, starts ? max_new : 1, w, (cudaStream_t)stream);
}

} // extern "C"
