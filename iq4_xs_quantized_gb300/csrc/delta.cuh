// delta.cuh -- the recurrent layers' state as kernels see it (layouts:
// include/iq4xs.h), and what their kernels share.
#pragma once

#include "cache.cuh"

namespace iq4xs {

struct DeltaView {
    float* s;
    float* conv;
    const int32_t* slot_of;
    int64_t s_slot_stride, conv_slot_stride;    // elements
    int64_t s_layer_stride, conv_layer_stride;
    int64_t s_extent, conv_extent;              // bytes from the first element to behind the last
    int layers, slots, key_heads, heads, key_dim, value_dim, channels;
};

constexpr int kConvTaps = 4;
constexpr int kDeltaTreeRows = 64;  // rows of a sequence whose state stays

// Sequence s: its rows (n = 0 where the offsets are out of order or of range),
// its length and slot (-1 where out of range).  All four values are asked for
// before the first is looked at: a look that may record keeps later loads behind it.
struct DeltaSequence {
    int first, n, len, slot;
};
__device__ __forceinline__ DeltaSequence delta_sequence(const BatchView& b, const DeltaView& d, int s, int rows, int* err) {
    const int32_t* const at_slot = d.slot_of != nullptr ? d.slot_of + s : b.lens + s;
    const int first = b.row_offsets[s], end = b.row_offsets[s + 1], len = b.lens[s], mapped = *at_slot;
    const int slot = d.slot_of != nullptr ? mapped : s;
    const bool rows_fit = first >= 0 && end >= first && end <= rows, slot_fits = slot >= 0 && slot < d.slots;
    if (!rows_fit) data_error(err, kDataOffsets);
    if (len < 0) data_error(err, kDataLens);
    if (!slot_fits) data_error(err, kDataSlot);
    return {first, rows_fit ? end - first : 0, max(len, -1), slot_fits ? slot : -1};
}

// Eight 16-bit values -> fp32.
template <class T>
__device__ __forceinline__ void unpack8(const uint4& w, float* x) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = T::unpack(v[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void unpack8(bool bf16, const uint4& w, float* x) {
    if (bf16) unpack8<KvBf16>(w, x);
    else unpack8<KvF16>(w, x);
}

// A value as two parts that tf32 holds: without its last 13 bits, and the remainder.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
    hi = __float_as_uint(x) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}
// The same with the remainder rounded to the 11 bits that the MMA takes of it (the
// last 13 are not looked at): together 2^-22 of the value off at most, where cut ones are
// 3 2^-23 and never above.
__device__ __forceinline__ void split_tf32_near(float x, uint32_t& hi, uint32_t& lo) {
    hi = __float_as_uint(x) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi)) + 0x1000u;
}
// D += A B of a 16 x 8 x 8 tile by the warp-level MMA on tf32.
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint2& b) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}

struct DeltaRule {  // iq4xs_delta_rule_args as its kernels see them
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    int64_t q_row_stride, k_row_stride, v_row_stride;
    const float* g;
    const float* beta;
    float* out;
    int64_t out_row_stride;
    float* u;
    const uint64_t* tree_mask;
    int64_t s_offset;  // of the layer
    float scale;
    int mask_words, max_rows, rows, bf16;
    int max_given;   // the caller said so
    int few_rows;    // sequences of more rows go in blocks of 64
    int skip_block;  // (a test's) copies of this block, or item, of every CTA stay out; -1: none
};

// The new tokens before t that row row0 + t comes from, as bits (of 64).
__device__ __forceinline__ uint64_t delta_seen(const uint64_t* mask, int words, int rows, int row0, int t,
                                               const Bc& bc) {
    const uint64_t before = (1ull << t) - 1;
    if (mask == nullptr) return before;
    const uint64_t* at = mask + (int64_t)(row0 + t) * words;
    if (!bc_global(bc, at, 8, mask, 8 * (int64_t)rows * words, kBcDeltaMask)) return 0;
    return *at & before;
}

cudaError_t launch_delta_inputs(const iq4xs_delta_inputs_args& a, const DeltaView& d, const BatchView& b, int* err,
                                int num_sms, cudaStream_t stream);
cudaError_t launch_delta_rule(DeltaRule p, const DeltaView& d, const BatchView& b, void* encode, int* err, int num_sms,
                              cudaStream_t stream);
cudaError_t launch_delta_chunk(const DeltaRule& p, const DeltaView& d, const BatchView& b, void* encode, int* err,
                               cudaStream_t stream);
cudaError_t launch_delta_commit(const iq4xs_delta_commit_args& a, const DeltaView& d, const BatchView& b, int* err,
                                cudaStream_t stream);
cudaError_t launch_token_probs(const float* logits, int64_t logits_stride, int64_t rows, int64_t vocab,
                               const float* temperature, float* probs, int64_t probs_stride, int* err, int num_sms,
                               cudaStream_t stream);
cudaError_t launch_verify_drafts(const iq4xs_verify_drafts_args& a, const BatchView& b, int* err, int num_sms,
                                 cudaStream_t stream);

}  // namespace iq4xs
