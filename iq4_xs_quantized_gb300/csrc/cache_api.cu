// cache_api.cu -- the extern "C" entry points of the attention side
// (include/iq4xs.h): checks of the arguments on the host, before any launch.
#include "cache.cuh"

using namespace iq4xs;

namespace {

constexpr int64_t kMaxRows = 32768;
constexpr int64_t kMaxSequences = 65535;
constexpr int64_t kMaxStride = int64_t(1) << 44;
constexpr int64_t kMaxExtent = int64_t(1) << 59;  // elements of an axis

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int from_cuda(cudaError_t e) { return e == cudaSuccess ? IQ4XS_OK : IQ4XS_ERR_CUDA; }

int view_cache(const iq4xs_kv_cache* c, CacheView* out) {
    if (!c || !c->k || !c->v) return IQ4XS_ERR_ARG;
    if (c->dtype != IQ4XS_KV_F16 && c->dtype != IQ4XS_KV_BF16) return IQ4XS_ERR_ARG;
    if (c->layers < 1 || c->layers > 65535 || c->pages < 1 || c->pages > INT32_MAX || c->heads < 1 ||
        c->heads > 1024)
        return IQ4XS_ERR_SHAPE;
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return IQ4XS_ERR_SHAPE;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return IQ4XS_ERR_SHAPE;
    const int64_t strides[4] = {c->layer_stride, c->page_stride, c->head_stride, c->slot_stride};
    for (int64_t s : strides)
        if (s < 0 || s > kMaxStride || s % 8) return IQ4XS_ERR_ARG;
    // (offsets are 64-bit elements: the last one's may not pass them)
    const int64_t last[4] = {c->layers - 1, c->pages - 1, c->heads - 1, c->page_size - 1};
    for (int i = 0; i < 4; ++i)
        if (last[i] > 0 && strides[i] > kMaxExtent / last[i]) return IQ4XS_ERR_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return IQ4XS_ERR_ALIGN;
    out->k = static_cast<uint16_t*>(c->k);
    out->v = static_cast<uint16_t*>(c->v);
    out->layer_stride = c->layer_stride;
    out->page_stride = c->page_stride;
    out->head_stride = c->head_stride;
    out->slot_stride = c->slot_stride;
    out->extent = 2 * ((c->layers - 1) * c->layer_stride + (c->pages - 1) * c->page_stride +
                       (c->heads - 1) * c->head_stride + (c->page_size - 1) * c->slot_stride + c->head_dim);
    out->layers = (int)c->layers;
    out->pages = (int)c->pages;
    out->heads = (int)c->heads;
    out->page_size = (int)c->page_size;
    out->page_shift = 0;
    while ((1 << out->page_shift) < out->page_size) ++out->page_shift;
    out->head_dim = (int)c->head_dim;
    return IQ4XS_OK;
}

}  // namespace

int iq4xs::view_batch(const iq4xs_kv_batch* b, BatchView* out) {
    if (!b) return IQ4XS_ERR_ARG;
    if (b->sequences < 0 || b->sequences > kMaxSequences) return IQ4XS_ERR_SHAPE;
    if (b->table_width < 1 || b->table_width > (1 << 20)) return IQ4XS_ERR_SHAPE;
    if (b->table_stride < b->table_width || b->table_stride > kMaxStride) return IQ4XS_ERR_ARG;
    if (!b->row_offsets || (b->sequences > 0 && (!b->lens || !b->held || !b->page_table))) return IQ4XS_ERR_ARG;
    if (!aligned(b->row_offsets, 4) || !aligned(b->lens, 4) || !aligned(b->held, 4) || !aligned(b->page_table, 4))
        return IQ4XS_ERR_ALIGN;
    out->row_offsets = b->row_offsets;
    out->lens = b->lens;
    out->held = b->held;
    out->page_table = b->page_table;
    out->table_stride = b->table_stride;
    out->table_width = (int)b->table_width;
    out->sequences = (int)b->sequences;
    return IQ4XS_OK;
}

extern "C" {

int iq4xs_qk_norm_rope(const iq4xs_qk_norm_rope_args* a, const iq4xs_kv_cache* cache, const iq4xs_kv_batch* batch,
                       int64_t stream) {
    if (!a || !a->q || !a->k || !a->v || !a->q_out) return IQ4XS_ERR_ARG;
    CacheView c;
    BatchView b;
    int rc = view_cache(cache, &c);
    if (rc || (rc = view_batch(batch, &b))) return rc;
    if (a->rows < 1 || a->rows > kMaxRows || a->q_heads < 1 || a->q_heads > 1024) return IQ4XS_ERR_SHAPE;
    if (a->layer < 0 || a->layer >= c.layers) return IQ4XS_ERR_ARG;
    if (!(a->eps >= 0)) return IQ4XS_ERR_ARG;
    const int64_t strides[6] = {a->q_row_stride, a->q_head_stride, a->k_row_stride,
                                a->k_head_stride, a->v_row_stride, a->v_head_stride};
    for (int64_t s : strides)
        if (s < 0 || s > kMaxStride || s % 4) return IQ4XS_ERR_ARG;
    if (a->q_out_row_stride < a->q_heads * c.head_dim || a->q_out_row_stride > kMaxStride || a->q_out_row_stride % 8)
        return IQ4XS_ERR_ARG;
    if (a->rope ? (a->rope_positions < 1 || a->rot_dim < 8) : a->rot_dim != 0) return IQ4XS_ERR_ARG;
    if (a->rot_dim % 8 || a->rot_dim > c.head_dim) return IQ4XS_ERR_SHAPE;
    if (a->interleaved != 0 && a->interleaved != 1) return IQ4XS_ERR_ARG;
    if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->q_weight, 16) ||
        !aligned(a->k_weight, 16) || !aligned(a->rope, 16) || !aligned(a->positions, 4) || !aligned(a->q_out, 16))
        return IQ4XS_ERR_ALIGN;
    int *err, sms;
    void* encode;
    if ((rc = device_context(&err, &sms, &encode))) return rc;
    if (b.sequences == 0) return IQ4XS_OK;
    return from_cuda(launch_qk_norm_rope(*a, c, b, cache->dtype == IQ4XS_KV_BF16, err, sms,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

int64_t iq4xs_tree_attention_workspace_bytes(int64_t rows, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                             int64_t sequences) {
    if (rows < 1 || rows > kMaxRows || kv_heads < 1 || kv_heads > 1024 || q_heads < 1 || q_heads > 1024 ||
        q_heads % kv_heads || sequences < 0 || sequences > kMaxSequences)
        return 0;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
    int *err, sms;
    void* encode;
    if (device_context(&err, &sms, &encode)) return 0;
    return tree_attention_workspace(rows, q_heads, kv_heads, head_dim, sequences, sms);
}

int iq4xs_tree_attention(const iq4xs_tree_attention_args* a, const iq4xs_kv_cache* cache, const iq4xs_kv_batch* batch,
                         int64_t stream) {
    if (!a || !a->q || !a->out || !a->workspace) return IQ4XS_ERR_ARG;
    CacheView c;
    BatchView b;
    int rc = view_cache(cache, &c);
    if (rc || (rc = view_batch(batch, &b))) return rc;
    if (a->rows < 1 || a->rows > kMaxRows || a->q_heads < 1 || a->q_heads > 1024 || a->q_heads % c.heads)
        return IQ4XS_ERR_SHAPE;
    if (a->layer < 0 || a->layer >= c.layers) return IQ4XS_ERR_ARG;
    const int64_t width = a->q_heads * c.head_dim;
    if (a->q_row_stride < width || a->q_row_stride % 8 || a->out_row_stride < width || a->out_row_stride % 4)
        return IQ4XS_ERR_ARG;
    if (a->q_row_stride > kMaxStride || a->out_row_stride > kMaxStride) return IQ4XS_ERR_ARG;
    if (!(a->scale > -1e30 && a->scale < 1e30)) return IQ4XS_ERR_ARG;
    if (a->tree_mask ? (a->mask_words < 1 || a->mask_words > 512) : a->mask_words != 0) return IQ4XS_ERR_ARG;
    if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->tree_mask, 8) || !aligned(a->workspace, 32))
        return IQ4XS_ERR_ALIGN;
    int *err, sms;
    void* encode;
    if ((rc = device_context(&err, &sms, &encode))) return rc;
    if (a->workspace_bytes < tree_attention_workspace(a->rows, a->q_heads, c.heads, c.head_dim, b.sequences, sms))
        return IQ4XS_ERR_ARG;
    if (b.sequences == 0) return IQ4XS_OK;
    return from_cuda(launch_tree_attention(*a, c, b, cache->dtype == IQ4XS_KV_BF16, encode, err, sms,
                                           take_skip_stage(), reinterpret_cast<cudaStream_t>(stream)));
}

int iq4xs_cache_reserve(const iq4xs_kv_batch* batch, int64_t page_size, int32_t* refs, int64_t pages, int32_t* status,
                        int64_t stream) {
    BatchView b;
    int rc = view_batch(batch, &b);
    if (rc) return rc;
    if (!refs || (!status && b.sequences > 0)) return IQ4XS_ERR_ARG;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) || pages < 1 || pages > INT32_MAX)
        return IQ4XS_ERR_SHAPE;
    if (!aligned(refs, 16) || !aligned(status, 4)) return IQ4XS_ERR_ALIGN;
    int *err, sms;
    void* encode;
    if ((rc = device_context(&err, &sms, &encode))) return rc;
    if (b.sequences == 0) return IQ4XS_OK;
    return from_cuda(launch_cache_reserve(b, (int)page_size, refs, (int)pages, status, err,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

int iq4xs_cache_commit(const iq4xs_kv_cache* cache, const iq4xs_kv_batch* batch, int32_t* refs, const int32_t* paths,
                       int64_t path_width, const int32_t* accepted, int32_t* new_lens, int64_t stream) {
    CacheView c;
    BatchView b;
    int rc = view_cache(cache, &c);
    if (rc || (rc = view_batch(batch, &b))) return rc;
    if (!refs || (b.sequences > 0 && (!paths || !accepted || !new_lens))) return IQ4XS_ERR_ARG;
    if (path_width < 1 || path_width > kMaxRows) return IQ4XS_ERR_SHAPE;
    if (!aligned(refs, 16) || !aligned(paths, 4) || !aligned(accepted, 4) || !aligned(new_lens, 4))
        return IQ4XS_ERR_ALIGN;
    int *err, sms;
    void* encode;
    if ((rc = device_context(&err, &sms, &encode))) return rc;
    if (b.sequences == 0) return IQ4XS_OK;
    return from_cuda(launch_cache_commit(c, b, refs, paths, (int)path_width, accepted, new_lens, err,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

int iq4xs_cache_fork(const iq4xs_kv_cache* cache, const iq4xs_kv_batch* batch, int32_t* refs, const int32_t* parents,
                     const int32_t* children, int64_t count, int32_t* status, int64_t stream) {
    CacheView c;
    BatchView b;
    int rc = view_cache(cache, &c);
    if (rc || (rc = view_batch(batch, &b))) return rc;
    if (!refs || (count > 0 && (!parents || !children || !status))) return IQ4XS_ERR_ARG;
    if (count < 0 || count > kMaxSequences) return IQ4XS_ERR_SHAPE;
    if (!aligned(refs, 16) || !aligned(parents, 4) || !aligned(children, 4) || !aligned(status, 4))
        return IQ4XS_ERR_ALIGN;
    int *err, sms;
    void* encode;
    if ((rc = device_context(&err, &sms, &encode))) return rc;
    if (count == 0) return IQ4XS_OK;
    return from_cuda(launch_cache_fork(c, b, refs, parents, children, (int)count, status, err,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

int iq4xs_cache_release(const iq4xs_kv_batch* batch, int32_t* refs, int64_t pages, const int32_t* rows, int64_t count,
                        int64_t stream) {
    BatchView b;
    int rc = view_batch(batch, &b);
    if (rc) return rc;
    if (!refs || (count > 0 && !rows)) return IQ4XS_ERR_ARG;
    if (pages < 1 || pages > INT32_MAX || count < 0 || count > kMaxSequences) return IQ4XS_ERR_SHAPE;
    if (!aligned(refs, 16) || !aligned(rows, 4)) return IQ4XS_ERR_ALIGN;
    int *err, sms;
    void* encode;
    if ((rc = device_context(&err, &sms, &encode))) return rc;
    if (count == 0) return IQ4XS_OK;
    return from_cuda(launch_cache_release(b, refs, (int)pages, rows, (int)count, err,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

int iq4xs_cache_copy_pages(const iq4xs_kv_cache* cache, const int32_t* src, const int32_t* dst, int64_t count,
                           int64_t stream) {
    CacheView c;
    int rc = view_cache(cache, &c);
    if (rc) return rc;
    if (count > 0 && (!src || !dst)) return IQ4XS_ERR_ARG;
    if (count < 0 || count > kMaxSequences) return IQ4XS_ERR_SHAPE;
    if (!aligned(src, 4) || !aligned(dst, 4)) return IQ4XS_ERR_ALIGN;
    int *err, sms;
    void* encode;
    if ((rc = device_context(&err, &sms, &encode))) return rc;
    if (count == 0) return IQ4XS_OK;
    return from_cuda(
        launch_cache_copy_pages(c, src, dst, (int)count, err, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
