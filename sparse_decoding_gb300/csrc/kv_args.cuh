// kv_args.cuh -- what the C entry points of the paged caches share: checks of their
// arguments, and the bookkeeping calls.
#pragma once

#include <cmath>

#include "kv4.cuh"

namespace nm {

// What a format decides: the bytes of a cell, of a kv head's share of a page beside its
// cells, and of the workspace's attention parts.
struct KvFormat {
    int64_t (*cell_bytes)(int head_dim);
    int64_t (*tail_bytes)(int head_dim);
    size_t (*partial_bytes)(int head_dim);
};

inline bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

inline bool sizes_ok(int page_tokens, int n_layers, int n_kv_heads, int head_dim)
{
    return (page_tokens == 16 || page_tokens == 32 || page_tokens == 64 || page_tokens == 128) && n_layers > 0 &&
           n_kv_heads > 0 && n_layers <= 65536 && n_kv_heads <= 65536 && (head_dim == 64 || head_dim == 128);
}

inline int64_t round_up(int64_t x, int64_t n) { return (x + n - 1) / n * n; }

inline int64_t page_bytes(const KvFormat &f, int page_tokens, int n_layers, int n_kv_heads, int head_dim)
{
    if (!sizes_ok(page_tokens, n_layers, n_kv_heads, head_dim))
        return 0;
    return (int64_t)n_layers * n_kv_heads * ((page_tokens / kKv4Cell) * f.cell_bytes(head_dim) + f.tail_bytes(head_dim));
}

inline int64_t workspace_bytes(const KvFormat &f, int64_t n_pages, int head_dim)
{
    if (n_pages < 0 || n_pages > 0x3FFFFFFF || (head_dim != 64 && head_dim != 128))
        return 0;
    return (int64_t)kKv4Counters * 4 + round_up((64 + 2 * n_pages + kKv4MaxSeqs) * 4, 256) +
           (int64_t)f.partial_bytes(head_dim);
}

// The cache's own arguments; *c, *w: what the kernels get. The status word is
// looked up last, so that every refusal comes before the first CUDA call.
inline nm_status check_cache(const KvFormat &f, const nm_kv4_cache *k, bool need_pool)
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
    if (k->workspace_bytes < workspace_bytes(f, k->n_pages, k->head_dim))
        return NM_ERR_SHAPE;
    return NM_OK;
}

inline nm_status view(const KvFormat &f, const nm_kv4_cache *k, Kv4 *c, Kv4Work *w, int *num_sms)
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
    c->page_bytes = page_bytes(f, k->page_tokens, k->n_layers, k->n_kv_heads, k->head_dim);
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

inline nm_status check_list(int n, bool have)
{
    if (n < 0)
        return NM_ERR_INVALID_ARG;
    if (n > kKv4MaxSeqs)
        return NM_ERR_UNSUPPORTED;
    return n > 0 && !have ? NM_ERR_INVALID_ARG : NM_OK;
}

// n_seqs, starts and n_tokens of a call over token arrays.
inline nm_status check_batch(const int32_t *starts, int n_seqs, int64_t n_tokens)
{
    nm_status s = check_list(n_seqs, true);
    if (s != NM_OK)
        return s;
    if (n_tokens < 0 || n_tokens > 0x3FFFFFFF || (!starts && n_tokens != n_seqs))
        return NM_ERR_SHAPE;
    return NM_OK;
}

// A token array of `heads` heads with token stride `stride`.
inline nm_status check_tokens(const void *p, int64_t stride, int64_t heads, int head_dim)
{
    if (!p)
        return NM_ERR_INVALID_ARG;
    if (!aligned(p, 16))
        return NM_ERR_ALIGN;
    return stride % 8 != 0 || stride < heads * head_dim ? NM_ERR_SHAPE : NM_OK;
}

// ---- the bookkeeping calls, the same in every format (kv4_api.cu) ----

nm_status kv_init(const KvFormat &f, const nm_kv4_cache *cache, cudaStream_t st);
nm_status kv_reserve(const KvFormat &f, const nm_kv4_cache *cache, const int32_t *seqs, const int32_t *starts, int n_seqs,
                     cudaStream_t st);
nm_status kv_fork(const KvFormat &f, const nm_kv4_cache *cache, const int32_t *src, const int32_t *dst, int n,
                  cudaStream_t st);
nm_status kv_free(const KvFormat &f, const nm_kv4_cache *cache, const int32_t *seqs, int n, cudaStream_t st);
nm_status kv_compact(const KvFormat &f, const nm_kv4_cache *cache, cudaStream_t st);
nm_status kv_copy_pages(const KvFormat &f, const nm_kv4_cache *src, const int32_t *src_pages, const nm_kv4_cache *dst,
                        const int32_t *dst_pages, int64_t n, cudaStream_t st);

// Of append, read and attention: their arguments checked. done: there is nothing to do. kv_open fills
// in the rest; it asks CUDA first, so it comes after every refusal (append's and read's checks end with it).
struct KvCall {
    Kv4 c;
    Kv4Work w;
    Kv4Batch b;
    bool done;
};
nm_status kv_open(const KvFormat &f, KvCall *o, const nm_kv4_cache *cache, const int32_t *seqs, const int32_t *starts,
                  int n_seqs, int64_t n_tokens);
nm_status kv_append_args(const KvFormat &f, KvCall *o, const nm_kv4_cache *cache, int layer, const int32_t *seqs,
                         const int32_t *starts, int n_seqs, int64_t n_tokens, const void *k, int64_t k_stride,
                         const void *v, int64_t v_stride, const void *q, int64_t q_stride, int n_q_heads,
                         const void *q_out, int64_t q_out_stride, const float *rope, int64_t rope_rows);
nm_status kv_read_args(const KvFormat &f, KvCall *o, const nm_kv4_cache *cache, int layer, const int32_t *seqs,
                       const int32_t *starts, int n_seqs, int64_t n_tokens, const void *k, const void *v);
nm_status kv_attention_args(const KvFormat &f, KvCall *o, const nm_kv4_cache *cache, int layer, const int32_t *starts,
                            int n_seqs, int64_t n_tokens, int64_t max_new, const void *q,
                            int64_t q_stride, int n_q_heads, float scale, const void *out, int64_t out_stride,
                            const float *lse);

} // namespace nm
