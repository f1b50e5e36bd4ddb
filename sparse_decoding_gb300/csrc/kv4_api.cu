// kv4_api.cu -- the C entry points of the 4-bit paged KV cache (declared in
// include/nmspmv.h), and the bookkeeping and the checks of arguments of every paged cache.
#include "kv_args.cuh"

namespace nm {
namespace {

const KvFormat kFormat{
    [](int head_dim) { return (int64_t)(head_dim == 128 ? Kv4Cell<128>::kBytes : Kv4Cell<64>::kBytes); },
    [](int) { return (int64_t)0; }, kv4_partial_bytes};

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

nm_status kv_init(const KvFormat &f, const nm_kv4_cache *cache, cudaStream_t st)
{
    nm_status s = check_cache(f, cache, false);
    if (s != NM_OK)
        return s;
    Kv4 c;
    Kv4Work w;
    int sms;
    if ((s = view(f, cache, &c, &w, &sms)) != NM_OK)
        return s;
    init_kernel<<<sms, 256, 0, st>>>(c, w.counters);
    return cudaGetLastError() == cudaSuccess ? NM_OK : NM_ERR_CUDA;
}

nm_status kv_reserve(const KvFormat &f, const nm_kv4_cache *cache, const int32_t *seqs, const int32_t *starts, int n_seqs,
                     cudaStream_t st)
{
    nm_status s = check_cache(f, cache, false);
    if (s != NM_OK || (s = check_list(n_seqs, true)) != NM_OK)
        return s;
    Kv4 c;
    Kv4Work w;
    int sms;
    if ((s = view(f, cache, &c, &w, &sms)) != NM_OK)
        return s;
    return kv4_launch_reserve(c, seqs, starts, n_seqs, w, st);
}

nm_status kv_fork(const KvFormat &f, const nm_kv4_cache *cache, const int32_t *src, const int32_t *dst, int n,
                  cudaStream_t st)
{
    nm_status s = check_cache(f, cache, true);
    if (s != NM_OK || (s = check_list(n, src && dst)) != NM_OK)
        return s;
    Kv4 c;
    Kv4Work w;
    int sms;
    if ((s = view(f, cache, &c, &w, &sms)) != NM_OK)
        return s;
    return kv4_launch_fork(c, src, dst, n, w, (int)f.cell_bytes(c.head_dim), sms, st);
}

nm_status kv_free(const KvFormat &f, const nm_kv4_cache *cache, const int32_t *seqs, int n, cudaStream_t st)
{
    nm_status s = check_cache(f, cache, false);
    if (s != NM_OK || (s = check_list(n, true)) != NM_OK || n == 0)
        return s;
    Kv4 c;
    Kv4Work w;
    int sms;
    if ((s = view(f, cache, &c, &w, &sms)) != NM_OK)
        return s;
    return kv4_launch_free(c, seqs, n, st);
}

nm_status kv_compact(const KvFormat &f, const nm_kv4_cache *cache, cudaStream_t st)
{
    nm_status s = check_cache(f, cache, true);
    if (s != NM_OK || cache->n_pages == 0)
        return s;
    Kv4 c;
    Kv4Work w;
    int sms;
    if ((s = view(f, cache, &c, &w, &sms)) != NM_OK)
        return s;
    return kv4_launch_compact(c, w, sms, st);
}

nm_status kv_copy_pages(const KvFormat &f, const nm_kv4_cache *src, const int32_t *src_pages, const nm_kv4_cache *dst,
                        const int32_t *dst_pages, int64_t n, cudaStream_t st)
{
    nm_status s = check_cache(f, src, true);
    if (s != NM_OK || (s = check_cache(f, dst, true)) != NM_OK)
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
    if ((s = view(f, src, &c, &w, &sms)) != NM_OK)
        return s;
    return kv4_launch_copy(c.pool, c.n_pages, src_pages, (uint8_t *)dst->pool, dst->n_pages, dst_pages, c.page_bytes, n,
                           c.status, sms, st);
}

nm_status kv_append_args(const KvFormat &f, KvCall *o, const nm_kv4_cache *cache, int layer, const int32_t *seqs,
                         const int32_t *starts, int n_seqs, int64_t n_tokens, const void *k, int64_t k_stride,
                         const void *v, int64_t v_stride, const void *q, int64_t q_stride, int n_q_heads,
                         const void *q_out, int64_t q_out_stride, const float *rope, int64_t rope_rows)
{
    nm_status s = check_cache(f, cache, true);
    if (s != NM_OK || (s = check_batch(starts, n_seqs, n_tokens)) != NM_OK)
        return s;
    if (layer < 0 || layer >= cache->n_layers || n_q_heads < 0 || n_q_heads > 65536 || rope_rows < 0)
        return NM_ERR_SHAPE;
    o->done = n_tokens == 0;
    if (o->done)
        return NM_OK;
    const int D = cache->head_dim;
    if ((s = check_tokens(k, k_stride, cache->n_kv_heads, D)) != NM_OK ||
        (s = check_tokens(v, v_stride, cache->n_kv_heads, D)) != NM_OK)
        return s;
    const bool have_q = q && n_q_heads > 0;
    if (have_q && ((s = check_tokens(q, q_stride, n_q_heads, D)) != NM_OK ||
                   (s = check_tokens(q_out, q_out_stride, n_q_heads, D)) != NM_OK))
        return s;
    if (have_q && q == q_out && q_stride != q_out_stride)
        return NM_ERR_SHAPE;
    if (rope && !aligned(rope, 16))
        return NM_ERR_ALIGN;
    return kv_open(f, o, cache, seqs, starts, n_seqs, n_tokens);
}

nm_status kv_read_args(const KvFormat &f, KvCall *o, const nm_kv4_cache *cache, int layer, const int32_t *seqs,
                       const int32_t *starts, int n_seqs, int64_t n_tokens, const void *k, const void *v)
{
    nm_status s = check_cache(f, cache, true);
    if (s != NM_OK || (s = check_batch(starts, n_seqs, n_tokens)) != NM_OK)
        return s;
    if (layer < 0 || layer >= cache->n_layers)
        return NM_ERR_SHAPE;
    o->done = n_tokens == 0 || (!k && !v);
    if (o->done)
        return NM_OK;
    if (!aligned(k, 16) || !aligned(v, 16))
        return NM_ERR_ALIGN;
    return kv_open(f, o, cache, seqs, starts, n_seqs, n_tokens);
}

nm_status kv_attention_args(const KvFormat &f, KvCall *o, const nm_kv4_cache *cache, int layer, const int32_t *starts,
                            int n_seqs, int64_t n_tokens, int64_t max_new, const void *q,
                            int64_t q_stride, int n_q_heads, float scale, const void *out, int64_t out_stride,
                            const float *lse)
{
    nm_status s = check_cache(f, cache, true);
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
    o->done = n_tokens == 0;
    if (o->done)
        return NM_OK;
    const int D = cache->head_dim;
    if ((s = check_tokens(q, q_stride, n_q_heads, D)) != NM_OK ||
        (s = check_tokens(out, out_stride, n_q_heads, D)) != NM_OK)
        return s;
    if (lse && !aligned(lse, 16))
        return NM_ERR_ALIGN;
    return NM_OK;
}

nm_status kv_open(const KvFormat &f, KvCall *o, const nm_kv4_cache *cache, const int32_t *seqs, const int32_t *starts,
                  int n_seqs, int64_t n_tokens)
{
    int sms;
    const nm_status s = view(f, cache, &o->c, &o->w, &sms);
    o->b = Kv4Batch{seqs, starts, n_seqs, n_tokens};
    return s;
}

} // namespace nm

using namespace nm;

extern "C" {

int64_t nm_kv4_page_bytes(int page_tokens, int n_layers, int n_kv_heads, int head_dim)
{
    return page_bytes(kFormat, page_tokens, n_layers, n_kv_heads, head_dim);
}

int64_t nm_kv4_workspace_bytes(int64_t n_pages, int head_dim) { return workspace_bytes(kFormat, n_pages, head_dim); }

nm_status nm_kv4_init(const nm_kv4_cache *cache, void *stream)
{
    NvtxRange nvtx_("nm_kv4_init");
    return kv_init(kFormat, cache, (cudaStream_t)stream);
}

nm_status nm_kv4_reserve(const nm_kv4_cache *cache, const int32_t *seqs, const int32_t *starts, int n_seqs,
                         void *stream)
{
    NvtxRange nvtx_("nm_kv4_reserve");
    return kv_reserve(kFormat, cache, seqs, starts, n_seqs, (cudaStream_t)stream);
}

nm_status nm_kv4_fork(const nm_kv4_cache *cache, const int32_t *src, const int32_t *dst, int n, void *stream)
{
    NvtxRange nvtx_("nm_kv4_fork");
    return kv_fork(kFormat, cache, src, dst, n, (cudaStream_t)stream);
}

nm_status nm_kv4_free(const nm_kv4_cache *cache, const int32_t *seqs, int n, void *stream)
{
    NvtxRange nvtx_("nm_kv4_free");
    return kv_free(kFormat, cache, seqs, n, (cudaStream_t)stream);
}

nm_status nm_kv4_compact(const nm_kv4_cache *cache, void *stream)
{
    NvtxRange nvtx_("nm_kv4_compact");
    return kv_compact(kFormat, cache, (cudaStream_t)stream);
}

nm_status nm_kv4_copy_pages(const nm_kv4_cache *src, const int32_t *src_pages, const nm_kv4_cache *dst,
                            const int32_t *dst_pages, int64_t n, void *stream)
{
    NvtxRange nvtx_("nm_kv4_copy_pages");
    return kv_copy_pages(kFormat, src, src_pages, dst, dst_pages, n, (cudaStream_t)stream);
}

nm_status nm_kv4_append(const nm_kv4_cache *cache, int layer, const int32_t *seqs, const int32_t *starts, int n_seqs,
                        int64_t n_tokens, const void *k_bf16, int64_t k_stride, const void *v_bf16, int64_t v_stride,
                        const void *q_bf16, int64_t q_stride, int n_q_heads, void *q_out_bf16, int64_t q_out_stride,
                        const float *rope, int64_t rope_rows, void *stream)
{
    NvtxRange nvtx_("nm_kv4_append");
    KvCall o;
    const nm_status s = kv_append_args(kFormat, &o, cache, layer, seqs, starts, n_seqs, n_tokens, k_bf16, k_stride, v_bf16,
                                       v_stride, q_bf16, q_stride, n_q_heads, q_out_bf16, q_out_stride, rope, rope_rows);
    if (s != NM_OK || o.done)
        return s;
    return kv4_launch_append(o.c, o.b, layer, k_bf16, k_stride, v_bf16, v_stride, n_q_heads > 0 ? q_bf16 : nullptr,
                             q_stride, n_q_heads, q_out_bf16, q_out_stride, rope, rope_rows, (cudaStream_t)stream);
}

nm_status nm_kv4_read(const nm_kv4_cache *cache, int layer, const int32_t *seqs, const int32_t *starts, int n_seqs,
                      int64_t n_tokens, void *k, void *v, int f32, void *stream)
{
    NvtxRange nvtx_("nm_kv4_read");
    KvCall o;
    const nm_status s = kv_read_args(kFormat, &o, cache, layer, seqs, starts, n_seqs, n_tokens, k, v);
    if (s != NM_OK || o.done)
        return s;
    return kv4_launch_read(o.c, o.b, layer, k, v, f32 != 0, (cudaStream_t)stream);
}

nm_status nm_kv4_attention(const nm_kv4_cache *cache, int layer, const int32_t *seqs, const int32_t *starts,
                           int n_seqs, int64_t n_tokens, int64_t max_new, const void *q_bf16, int64_t q_stride,
                           int n_q_heads, float scale, void *out_bf16, int64_t out_stride, float *lse, void *stream)
{
    NvtxRange nvtx_("nm_kv4_attention");
    KvCall o;
    nm_status s = kv_attention_args(kFormat, &o, cache, layer, starts, n_seqs, n_tokens, max_new, q_bf16, q_stride,
                                    n_q_heads, scale, out_bf16, out_stride, lse);
    if (s != NM_OK || o.done || (s = kv_open(kFormat, &o, cache, seqs, starts, n_seqs, n_tokens)) != NM_OK)
        return s;
    const Kv4Attn a{layer, q_bf16, q_stride, n_q_heads, scale, out_bf16, out_stride, lse};
    return kv4_launch_attention(o.c, o.b, a, starts ? max_new : 1, o.w, (cudaStream_t)stream);
}

} // extern "C"
