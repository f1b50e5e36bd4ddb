// kv8_api.cu -- the C entry points of the 8-bit paged KV cache (declared in
// include/nmspmv.h): argument checks and dispatch.
#include "kv8.cuh"
#include "kv_args.cuh"

using namespace nm;

namespace {

const KvFormat kFormat{
    [](int head_dim) { return (int64_t)(head_dim == 128 ? Kv8Cell<128>::kBytes : Kv8Cell<64>::kBytes); },
    [](int head_dim) { return (int64_t)(head_dim == 128 ? Kv8Cell<128>::kTail : Kv8Cell<64>::kTail); }, kv8_partial_bytes};

// The lists of a selection: [n_tokens][n_kv_heads][n_list].
nm_status check_pages(const nm_kv8_cache *cache, const int32_t *pages, int n_list)
{
    if (n_list < 1)
        return NM_ERR_INVALID_ARG;
    if (n_list > kKv8SelectPages || (int64_t)n_list * cache->page_tokens > 0x3FFFFFFF)
        return NM_ERR_UNSUPPORTED;
    return aligned(pages, 4) ? NM_OK : NM_ERR_ALIGN;
}

} // namespace

extern "C" {

int64_t nm_kv8_page_bytes(int page_tokens, int n_layers, int n_kv_heads, int head_dim)
{
    return page_bytes(kFormat, page_tokens, n_layers, n_kv_heads, head_dim);
}

int64_t nm_kv8_workspace_bytes(int64_t n_pages, int head_dim) { return workspace_bytes(kFormat, n_pages, head_dim); }

nm_status nm_kv8_init(const nm_kv8_cache *cache, void *stream)
{
    NvtxRange nvtx_("nm_kv8_init");
    return kv_init(kFormat, cache, (cudaStream_t)stream);
}

nm_status nm_kv8_reserve(const nm_kv8_cache *cache, const int32_t *seqs, const int32_t *starts, int n_seqs,
                         void *stream)
{
    NvtxRange nvtx_("nm_kv8_reserve");
    return kv_reserve(kFormat, cache, seqs, starts, n_seqs, (cudaStream_t)stream);
}

nm_status nm_kv8_fork(const nm_kv8_cache *cache, const int32_t *src, const int32_t *dst, int n, void *stream)
{
    NvtxRange nvtx_("nm_kv8_fork");
    return kv_fork(kFormat, cache, src, dst, n, (cudaStream_t)stream);
}

nm_status nm_kv8_free(const nm_kv8_cache *cache, const int32_t *seqs, int n, void *stream)
{
    NvtxRange nvtx_("nm_kv8_free");
    return kv_free(kFormat, cache, seqs, n, (cudaStream_t)stream);
}

nm_status nm_kv8_compact(const nm_kv8_cache *cache, void *stream)
{
    NvtxRange nvtx_("nm_kv8_compact");
    return kv_compact(kFormat, cache, (cudaStream_t)stream);
}

nm_status nm_kv8_copy_pages(const nm_kv8_cache *src, const int32_t *src_pages, const nm_kv8_cache *dst,
                            const int32_t *dst_pages, int64_t n, void *stream)
{
    NvtxRange nvtx_("nm_kv8_copy_pages");
    return kv_copy_pages(kFormat, src, src_pages, dst, dst_pages, n, (cudaStream_t)stream);
}

nm_status nm_kv8_append(const nm_kv8_cache *cache, int layer, const int32_t *seqs, const int32_t *starts, int n_seqs,
                        int64_t n_tokens, const void *k_bf16, int64_t k_stride, const void *v_bf16, int64_t v_stride,
                        const void *q_bf16, int64_t q_stride, int n_q_heads, void *q_out_bf16, int64_t q_out_stride,
                        const float *rope, int64_t rope_rows, void *stream)
{
    NvtxRange nvtx_("nm_kv8_append");
    KvCall o;
    const nm_status s = kv_append_args(kFormat, &o, cache, layer, seqs, starts, n_seqs, n_tokens, k_bf16, k_stride, v_bf16,
                                       v_stride, q_bf16, q_stride, n_q_heads, q_out_bf16, q_out_stride, rope, rope_rows);
    if (s != NM_OK || o.done)
        return s;
    return kv8_launch_append(o.c, o.b, layer, k_bf16, k_stride, v_bf16, v_stride, n_q_heads > 0 ? q_bf16 : nullptr,
                             q_stride, n_q_heads, q_out_bf16, q_out_stride, rope, rope_rows, (cudaStream_t)stream);
}

nm_status nm_kv8_read(const nm_kv8_cache *cache, int layer, const int32_t *seqs, const int32_t *starts, int n_seqs,
                      int64_t n_tokens, void *k, void *v, int f32, void *stream)
{
    NvtxRange nvtx_("nm_kv8_read");
    KvCall o;
    const nm_status s = kv_read_args(kFormat, &o, cache, layer, seqs, starts, n_seqs, n_tokens, k, v);
    if (s != NM_OK || o.done)
        return s;
    return kv8_launch_read(o.c, o.b, layer, k, v, f32 != 0, (cudaStream_t)stream);
}

nm_status nm_kv8_attention(const nm_kv8_cache *cache, int layer, const int32_t *seqs, const int32_t *starts,
                           int n_seqs, int64_t n_tokens, int64_t max_new, const void *q_bf16, int64_t q_stride,
                           int n_q_heads, float scale, const int32_t *pages, int n_list, void *out_bf16,
                           int64_t out_stride, float *lse, void *stream)
{
    NvtxRange nvtx_("nm_kv8_attention");
    KvCall o;
    nm_status s = kv_attention_args(kFormat, &o, cache, layer, starts, n_seqs, n_tokens, pages ? 1 : max_new, q_bf16,
                                    q_stride, n_q_heads, scale, out_bf16, out_stride, lse);
    if (s != NM_OK || o.done || (pages && (s = check_pages(cache, pages, n_list)) != NM_OK) ||
        (s = kv_open(kFormat, &o, cache, seqs, starts, n_seqs, n_tokens)) != NM_OK)
        return s;
    const Kv4Attn a{layer, q_bf16, q_stride, n_q_heads, scale, out_bf16, out_stride, lse};
    return kv8_launch_attention(o.c, o.b, a, starts ? max_new : 1, pages, n_list, o.w, (cudaStream_t)stream);
}

nm_status nm_kv8_select(const nm_kv8_cache *cache, int layer, const int32_t *seqs, const int32_t *starts, int n_seqs,
                        int64_t n_tokens, const void *q_bf16, int64_t q_stride, int n_q_heads, int n_list, int first,
                        int last, int32_t *pages, void *stream)
{
    NvtxRange nvtx_("nm_kv8_select");
    KvCall o;
    // q alone is read: its checks are attention's
    nm_status s = kv_attention_args(kFormat, &o, cache, layer, starts, n_seqs, n_tokens, 1, q_bf16, q_stride, n_q_heads,
                                    1.0f, q_bf16, q_stride, nullptr);
    if (s != NM_OK || o.done)
        return s;
    if (!pages || first < 0 || last < 1)
        return NM_ERR_INVALID_ARG;
    if ((s = check_pages(cache, pages, n_list)) != NM_OK)
        return s;
    if ((int64_t)first + last > n_list)
        return NM_ERR_INVALID_ARG;
    if (cache->max_pages > kKv8SelectPages)
        return NM_ERR_UNSUPPORTED;
    if ((s = kv_open(kFormat, &o, cache, seqs, starts, n_seqs, n_tokens)) != NM_OK)
        return s;
    const Kv8Select a{layer, n_q_heads, n_list, first, last, q_bf16, q_stride, pages};
    return kv8_launch_select(o.c, o.b, a, o.w, (cudaStream_t)stream);
}

} // extern "C"
