// delta_api.cu -- the extern "C" entry points of the recurrent layers and of a
// step's verification (include/iq4xs.h): checks of the arguments on the host,
// before any launch.
#include "delta.cuh"

using namespace iq4xs;

namespace {

constexpr int64_t kMaxRows = 32768;
constexpr int64_t kMaxStride = int64_t(1) << 37;  // elements (tensor maps hold strides of up to 2^40 bytes)
constexpr int64_t kMaxExtent = int64_t(1) << 59;  // elements of an axis

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int from_cuda(cudaError_t e) { return e == cudaSuccess ? IQ4XS_OK : IQ4XS_ERR_CUDA; }
inline bool in_stride(int64_t s, int64_t least, int64_t unit) { return s >= least && s <= kMaxStride && s % unit == 0; }
inline bool fits(int64_t n, int64_t stride) { return n < 2 || stride <= kMaxExtent / (n - 1); }

int view_state(const iq4xs_delta_state* c, const BatchView& b, DeltaView* out) {
    if (!c || !c->s) return IQ4XS_ERR_ARG;
    if (c->layers < 1 || c->layers > 65535 || c->slots < 1 || c->slots > INT32_MAX || c->key_heads < 1 ||
        c->heads < 1 || c->heads > 1024 || c->heads % c->key_heads)
        return IQ4XS_ERR_SHAPE;
    if ((c->key_dim != 64 && c->key_dim != 128) || (c->value_dim != 64 && c->value_dim != 128)) return IQ4XS_ERR_SHAPE;
    if (!c->slot_of && b.sequences > c->slots) return IQ4XS_ERR_SHAPE;
    const int64_t size = c->heads * c->key_dim * c->value_dim;
    const int64_t channels = 2 * c->key_heads * c->key_dim + c->heads * c->value_dim;
    // (the stride of an axis of one is of no account)
    if ((c->slots > 1 && !in_stride(c->s_slot_stride, size, 4)) ||
        (c->layers > 1 && !in_stride(c->s_layer_stride, size, 4)) || !fits(c->slots, c->s_slot_stride) ||
        !fits(c->layers, c->s_layer_stride))
        return IQ4XS_ERR_ARG;
    if (c->conv && ((c->slots > 1 && !in_stride(c->conv_slot_stride, (kConvTaps - 1) * channels, 4)) ||
                    (c->layers > 1 && !in_stride(c->conv_layer_stride, (kConvTaps - 1) * channels, 4)) ||
                    !fits(c->slots, c->conv_slot_stride) || !fits(c->layers, c->conv_layer_stride)))
        return IQ4XS_ERR_ARG;
    if (!aligned(c->s, 16) || !aligned(c->conv, 16) || !aligned(c->slot_of, 4)) return IQ4XS_ERR_ALIGN;
    out->s = c->s;
    out->conv = c->conv;
    out->slot_of = c->slot_of;
    out->s_slot_stride = c->slots > 1 ? c->s_slot_stride : 0;
    out->s_layer_stride = c->layers > 1 ? c->s_layer_stride : 0;
    out->conv_slot_stride = c->slots > 1 ? c->conv_slot_stride : 0;
    out->conv_layer_stride = c->layers > 1 ? c->conv_layer_stride : 0;
    out->s_extent = 4 * ((c->layers - 1) * out->s_layer_stride + (c->slots - 1) * out->s_slot_stride + size);
    out->conv_extent = 4 * ((c->layers - 1) * out->conv_layer_stride + (c->slots - 1) * out->conv_slot_stride +
                            (kConvTaps - 1) * channels);
    out->layers = (int)c->layers;
    out->slots = (int)c->slots;
    out->key_heads = (int)c->key_heads;
    out->heads = (int)c->heads;
    out->key_dim = (int)c->key_dim;
    out->value_dim = (int)c->value_dim;
    out->channels = (int)channels;
    return IQ4XS_OK;
}

inline bool good_mask(const uint64_t* mask, int64_t words) {
    return mask ? (words >= 1 && words <= 512) : words == 0;
}

}  // namespace

extern "C" {

int iq4xs_delta_inputs(const iq4xs_delta_inputs_args* a, const iq4xs_delta_state* state, const iq4xs_kv_batch* batch,
                       int64_t stream) {
    if (!a || !a->x || !a->conv_weight || !a->a || !a->b || !a->a_log || !a->dt_bias || !a->q || !a->k || !a->v ||
        !a->g || !a->beta)
        return IQ4XS_ERR_ARG;
    BatchView b;
    DeltaView d;
    int rc = view_batch(batch, &b);
    if (rc || (rc = view_state(state, b, &d))) return rc;
    if (a->rows < 1 || a->rows > kMaxRows) return IQ4XS_ERR_SHAPE;
    if (!d.conv || a->layer < 0 || a->layer >= d.layers) return IQ4XS_ERR_ARG;
    if (a->dtype != IQ4XS_KV_F16 && a->dtype != IQ4XS_KV_BF16) return IQ4XS_ERR_ARG;
    if (!(a->eps >= 0)) return IQ4XS_ERR_ARG;
    const int64_t keys = (int64_t)d.key_heads * d.key_dim;
    if (!in_stride(a->x_row_stride, d.channels, 4) || !in_stride(a->a_row_stride, d.heads, 1) ||
        !in_stride(a->b_row_stride, d.heads, 1) || !in_stride(a->q_row_stride, keys, 8) ||
        !in_stride(a->k_row_stride, keys, 8) || !in_stride(a->v_row_stride, (int64_t)d.heads * d.value_dim, 8))
        return IQ4XS_ERR_ARG;
    if (!good_mask(a->tree_mask, a->mask_words)) return IQ4XS_ERR_ARG;
    if (a->advance != 0 && (a->advance != 1 || a->tree_mask)) return IQ4XS_ERR_ARG;
    if (!aligned(a->x, 16) || !aligned(a->conv_weight, 16) || !aligned(a->a, 4) || !aligned(a->b, 4) ||
        !aligned(a->a_log, 4) || !aligned(a->dt_bias, 4) || !aligned(a->q, 16) || !aligned(a->k, 16) ||
        !aligned(a->v, 16) || !aligned(a->g, 4) || !aligned(a->beta, 4) || !aligned(a->tree_mask, 8))
        return IQ4XS_ERR_ALIGN;
    int *err, sms;
    void* encode;
    if ((rc = device_context(&err, &sms, &encode))) return rc;
    if (b.sequences == 0) return IQ4XS_OK;
    return from_cuda(launch_delta_inputs(*a, d, b, err, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int iq4xs_delta_rule(const iq4xs_delta_rule_args* a, const iq4xs_delta_state* state, const iq4xs_kv_batch* batch,
                     int64_t stream) {
    if (!a || !a->q || !a->k || !a->v || !a->g || !a->beta || !a->out) return IQ4XS_ERR_ARG;
    BatchView b;
    DeltaView d;
    int rc = view_batch(batch, &b);
    if (rc || (rc = view_state(state, b, &d))) return rc;
    if (a->rows < 1 || a->rows > kMaxRows) return IQ4XS_ERR_SHAPE;
    if (a->layer < 0 || a->layer >= d.layers) return IQ4XS_ERR_ARG;
    if (a->dtype != IQ4XS_KV_F16 && a->dtype != IQ4XS_KV_BF16) return IQ4XS_ERR_ARG;
    if (!(a->scale > -1e30 && a->scale < 1e30)) return IQ4XS_ERR_ARG;
    const int64_t keys = (int64_t)d.key_heads * d.key_dim, values = (int64_t)d.heads * d.value_dim;
    if (!in_stride(a->q_row_stride, keys, 8) || !in_stride(a->k_row_stride, keys, 8) ||
        !in_stride(a->v_row_stride, values, 8) || !in_stride(a->out_row_stride, values, 4))
        return IQ4XS_ERR_ARG;
    if (!good_mask(a->tree_mask, a->mask_words) || (a->tree_mask && !a->u)) return IQ4XS_ERR_ARG;
    if (a->max_rows < 0 || a->max_rows > kMaxRows) return IQ4XS_ERR_SHAPE;
    if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->g, 4) || !aligned(a->beta, 4) ||
        !aligned(a->out, 16) || !aligned(a->u, 16) || !aligned(a->tree_mask, 8))
        return IQ4XS_ERR_ALIGN;
    int *err, sms;
    void* encode;
    if ((rc = device_context(&err, &sms, &encode))) return rc;
    if (b.sequences == 0) return IQ4XS_OK;
    DeltaRule p;
    p.q = static_cast<const uint16_t*>(a->q);
    p.k = static_cast<const uint16_t*>(a->k);
    p.v = static_cast<const uint16_t*>(a->v);
    p.q_row_stride = a->q_row_stride;
    p.k_row_stride = a->k_row_stride;
    p.v_row_stride = a->v_row_stride;
    p.g = a->g;
    p.beta = a->beta;
    p.out = a->out;
    p.out_row_stride = a->out_row_stride;
    p.u = a->u;
    p.tree_mask = a->tree_mask;
    p.mask_words = (int)a->mask_words;
    p.s_offset = a->layer * d.s_layer_stride;
    p.scale = (float)a->scale;
    p.rows = (int)a->rows;
    p.bf16 = a->dtype == IQ4XS_KV_BF16;
    p.skip_block = take_skip_stage();
    // The most rows that a sequence can have; the kernels skip one with more.
    p.max_rows = (int)(a->max_rows > 0 && a->max_rows < a->rows ? a->max_rows : a->rows);
    p.max_given = a->max_rows > 0;
    p.few_rows = 0;
    if (a->u && p.max_rows > kDeltaTreeRows) p.max_rows = kDeltaTreeRows;
    return from_cuda(launch_delta_rule(p, d, b, encode, err, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int iq4xs_delta_commit(const iq4xs_delta_commit_args* a, const iq4xs_delta_state* state, const iq4xs_kv_batch* batch,
                       int64_t stream) {
    if (!a || !a->k || !a->g || !a->u) return IQ4XS_ERR_ARG;
    BatchView b;
    DeltaView d;
    int rc = view_batch(batch, &b);
    if (rc || (rc = view_state(state, b, &d))) return rc;
    if (b.sequences > 0 && (!a->paths || !a->accepted)) return IQ4XS_ERR_ARG;
    if ((a->x != nullptr) != (d.conv != nullptr)) return IQ4XS_ERR_ARG;
    if (a->rows < 1 || a->rows > kMaxRows || a->path_width < 1 || a->path_width > kMaxRows) return IQ4XS_ERR_SHAPE;
    if (a->dtype != IQ4XS_KV_F16 && a->dtype != IQ4XS_KV_BF16) return IQ4XS_ERR_ARG;
    if (!in_stride(a->k_row_stride, (int64_t)d.key_heads * d.key_dim, 8)) return IQ4XS_ERR_ARG;
    if (a->x && !in_stride(a->x_row_stride, d.channels, 4)) return IQ4XS_ERR_ARG;
    if (d.layers > 1 && (!in_stride(a->k_layer_stride, 8, 8) || !in_stride(a->g_layer_stride, 1, 1) ||
                         !in_stride(a->u_layer_stride, 4, 4) || (a->x && !in_stride(a->x_layer_stride, 4, 4)) ||
                         !fits(d.layers, a->k_layer_stride) || !fits(d.layers, a->g_layer_stride) ||
                         !fits(d.layers, a->u_layer_stride) || (a->x && !fits(d.layers, a->x_layer_stride))))
        return IQ4XS_ERR_ARG;
    if (!aligned(a->k, 16) || !aligned(a->g, 4) || !aligned(a->u, 16) || !aligned(a->x, 16) ||
        !aligned(a->paths, 4) || !aligned(a->accepted, 4))
        return IQ4XS_ERR_ALIGN;
    int *err, sms;
    void* encode;
    if ((rc = device_context(&err, &sms, &encode))) return rc;
    if (b.sequences == 0) return IQ4XS_OK;
    return from_cuda(launch_delta_commit(*a, d, b, err, reinterpret_cast<cudaStream_t>(stream)));
}

int iq4xs_token_probs(const float* logits, int64_t logits_stride, int64_t rows, int64_t vocab,
                      const float* temperature, float* probs, int64_t probs_stride, int64_t stream) {
    if (!logits || !probs) return IQ4XS_ERR_ARG;
    if (rows < 1 || rows > kMaxRows || vocab < 1 || vocab > (1 << 20)) return IQ4XS_ERR_SHAPE;
    if (!in_stride(logits_stride, vocab, 1) || !in_stride(probs_stride, vocab, 1)) return IQ4XS_ERR_ARG;
    if (!aligned(logits, 4) || !aligned(probs, 4) || !aligned(temperature, 4)) return IQ4XS_ERR_ALIGN;
    int *err, sms;
    void* encode;
    const int rc = device_context(&err, &sms, &encode);
    if (rc) return rc;
    return from_cuda(launch_token_probs(logits, logits_stride, rows, vocab, temperature, probs, probs_stride, err, sms,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

int iq4xs_verify_drafts(const iq4xs_verify_drafts_args* a, const iq4xs_kv_batch* batch, int64_t stream) {
    if (!a || !a->probs || !a->tokens || !a->accept_u) return IQ4XS_ERR_ARG;
    BatchView b;
    int rc = view_batch(batch, &b);
    if (rc) return rc;
    if (b.sequences > 0 && (!a->draw_u || !a->paths || !a->accepted || !a->next)) return IQ4XS_ERR_ARG;
    if (a->rows < 1 || a->rows > kMaxRows || a->vocab < 1 || a->vocab > (1 << 20) || a->path_width < 1 ||
        a->path_width > kMaxRows)
        return IQ4XS_ERR_SHAPE;
    if (!in_stride(a->probs_stride, a->vocab, 1) || (a->draft_probs && !in_stride(a->draft_stride, a->vocab, 1)))
        return IQ4XS_ERR_ARG;
    if (!good_mask(a->tree_mask, a->mask_words)) return IQ4XS_ERR_ARG;
    if (!aligned(a->probs, 4) || !aligned(a->draft_probs, 4) || !aligned(a->tokens, 4) || !aligned(a->tree_mask, 8) ||
        !aligned(a->accept_u, 4) || !aligned(a->draw_u, 4) || !aligned(a->paths, 4) || !aligned(a->accepted, 4) ||
        !aligned(a->next, 4))
        return IQ4XS_ERR_ALIGN;
    int *err, sms;
    void* encode;
    if ((rc = device_context(&err, &sms, &encode))) return rc;
    if (b.sequences == 0) return IQ4XS_OK;
    return from_cuda(launch_verify_drafts(*a, b, err, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
