// attention.cu -- tree attention over the paged cache: tensor maps, the
// choice of the form, and the join of items that the split cut.
#include "attention.cuh"

#include <math.h>

namespace iq4xs {
namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Where no sequence can be longer than this (the table's width), in tokens:
// items are not cut; or from kAloneTokens on a cluster shares an item, if the
// SMs hold all items' clusters.  Measured for one token, 24/4 heads of 256, as
// a cluster / not cut / cut and joined: 100 cached tokens 8.7 / 7.7 us, 517
// 9.0 / 19.5 / 10.4, 2000 10.5 / 53 / 10.8, 8000 19.2 / - / 14.4.
constexpr int64_t kWholeTokens = 512, kAloneTokens = 128, kClusterTokens = 2048;
static_assert(sizeof(CutItem) == 32, "partial results stay aligned");

// One map over K or V of a layer: 64 channels, slots, 64-channel chunks, heads,
// pages.  A box is up to `slots` slots of a page by `chunks` chunks, and lies
// in shared memory as [chunk][slot][128 bytes].
bool encode_kv(EncodeTiledFn enc, uint16_t* base, const CacheView& c, bool bf16, int slots, int chunks,
               CUtensorMap* map) {
    const cuuint64_t gdim[5] = {64, (cuuint64_t)c.page_size, (cuuint64_t)c.head_dim / 64, (cuuint64_t)c.heads,
                                (cuuint64_t)c.pages};
    const cuuint64_t gstride[4] = {(cuuint64_t)c.slot_stride * 2, 128, (cuuint64_t)c.head_stride * 2,
                                   (cuuint64_t)c.page_stride * 2};
    const cuuint32_t box[5] = {64, (cuuint32_t)slots, (cuuint32_t)chunks, 1, 1};
    const cuuint32_t estride[5] = {1, 1, 1, 1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, base, gdim, gstride,
               box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ------------------------------------------------------------------- join
// The partial results of cut items, weighted by exp2(m_i - m), over the joined
// sum; a CTA per cut item and some of its rows, whose addresses the attention
// kernel left.  Groups of D / 4 threads own the D channels of a row: with few
// parts an item (kByRows) the groups take rows, with many they take parts of
// one row, kJoinBatch in flight each, and add up in shared memory.  Sums have
// a fixed order.  Measured: about 4 us behind 152 CTAs, most of it the launch
// and two loads in a row; over all rows instead of the cut items up to 60 us.
constexpr int kJoinThreads = 256, kJoinBatch = 8, kJoinRows = 8;
constexpr int kMaxParts = 256;

template <int D, bool kByRows>
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(const AttnParams p, int* err) {
    constexpr int kAcross = D / 4, kGroups = kJoinThreads / kAcross;
    __shared__ float4 acc_s[kByRows ? 1 : kJoinThreads];
    __shared__ float2 ml_s[kByRows ? 1 : kMaxParts];
    griddep_wait();
    griddep_launch_dependents();
    const CutItem cut = p.cuts[blockIdx.x];
    const int row0 = blockIdx.y * (kByRows ? kJoinRows : 1);
    if (cut.first < 0 || row0 >= cut.rows) return;
    const int n = (int)blockIdx.x - cut.first + 1;  // (at most the CTAs, which kMaxParts holds)
    const int lane = threadIdx.x & 31, group = threadIdx.x / kAcross, col = threadIdx.x % kAcross * 4;
    const Bc bc = bc_open(err);
    const auto slot_of = [&](int i) { return 2 * (cut.first + i) + (i == 0); };
    const auto sum_of = [&](int i, int r) {
        const float2* at = part_sum(p, slot_of(i), r, bc);
        return at != nullptr ? *at : make_float2(-INFINITY, 0.f);
    };
    const auto part_of = [&](int i, int r) {
        const float* at = part_row(p, slot_of(i), r, col, 4, bc);
        return at != nullptr ? *reinterpret_cast<const float4*>(at) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    const auto add = [](float4& a, float4 v, float f) {
        a.x = fmaf(v.x, f, a.x);
        a.y = fmaf(v.y, f, a.y);
        a.z = fmaf(v.z, f, a.z);
        a.w = fmaf(v.w, f, a.w);
    };
    const auto put = [&](int r, float4 a, float sum) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row that sees nothing: zeros
        const int row = cut.first_row + r, t = token_of(p, row);
        float* dst = p.out + (cut.row0 + t) * p.out_row_stride + ((int64_t)cut.head * p.group + row - t * p.group) * D + col;
        if (bc_global(bc, dst, 16, p.out, 4 * ((p.rows - 1) * p.out_row_stride + (int64_t)p.group * p.kv_heads * D),
                      kBcAttnOut))
            *reinterpret_cast<float4*>(dst) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    };
    if constexpr (kByRows) {
        for (int r = row0 + group; r < min(row0 + kJoinRows, cut.rows); r += kGroups) {
            float top = -INFINITY, sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i0 = 0; i0 < n; i0 += kJoinBatch) {
                float2 ml[kJoinBatch];
                float4 v[kJoinBatch];
#pragma unroll
                for (int k = 0; k < kJoinBatch; ++k) {  // (the last part again instead of a branch)
                    ml[k] = sum_of(min(i0 + k, n - 1), r);
                    v[k] = part_of(min(i0 + k, n - 1), r);
                }
                float most = top;
#pragma unroll
                for (int k = 0; k < kJoinBatch; ++k) most = fmaxf(most, ml[k].x);
                if (most > top) {
                    const float f = fast_exp2(top - most);
                    sum *= f;
                    acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
                    top = most;
                }
#pragma unroll
                for (int k = 0; k < kJoinBatch; ++k)
                    if (i0 + k < n) {
                        const bool none = ml[k].x == -INFINITY;  // (nothing seen: sum 0, or NaN)
                        const float f = none ? ml[k].y : fast_exp2(ml[k].x - top);
                        sum += none ? ml[k].y : ml[k].y * f;
                        add(acc, v[k], f);
                    }
            }
            put(r, acc, sum);
        }
    } else {
        const int r = row0;
        for (int i = threadIdx.x; i < n; i += kJoinThreads) ml_s[i] = sum_of(i, r);
        float4 v[kJoinBatch];
#pragma unroll
        for (int k = 0; k < kJoinBatch; ++k)
            v[k] = part_of(min(group + k * kGroups, n - 1), r);
        __syncthreads();
        float top = -INFINITY, sum = 0.f;
        for (int i = lane; i < n; i += 32) top = fmaxf(top, ml_s[i].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        for (int i = lane; i < n; i += 32) {
            const float2 t = ml_s[i];
            sum += t.x == -INFINITY ? t.y : t.y * fast_exp2(t.x - top);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = group; i0 < n; i0 += kJoinBatch * kGroups) {
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k)
                if (i0 + k * kGroups < n) {
                    const float2 t = ml_s[i0 + k * kGroups];
                    add(acc, v[k], t.x == -INFINITY ? t.y : fast_exp2(t.x - top));
                }
            if (i0 + kJoinBatch * kGroups < n) {
#pragma unroll
                for (int k = 0; k < kJoinBatch; ++k)
                    v[k] = part_of(min(i0 + (kJoinBatch + k) * kGroups, n - 1), r);
            }
        }
        acc_s[threadIdx.x] = acc;
        __syncthreads();
        if (group != 0) return;
#pragma unroll
        for (int i = 1; i < kGroups; ++i) add(acc, acc_s[i * kAcross + threadIdx.x], 1.f);
        put(r, acc, sum);
    }
}

// By rows on tcgen05, whose items have many rows and few parts.
template <int D>
cudaError_t launch_join_width(bool tc, const AttnParams& p, int* err, cudaStream_t stream) {
    const unsigned rows = (unsigned)p.slot_rows, ctas = (unsigned)p.ctas;
    if (tc)
        return launch_chained(attention_join_kernel<D, true>, dim3(ctas, (rows + kJoinRows - 1) / kJoinRows),
                              dim3(kJoinThreads), 0, stream, 1, p, err);
    return launch_chained(attention_join_kernel<D, false>, dim3(ctas, rows), dim3(kJoinThreads), 0, stream, 1, p, err);
}
cudaError_t launch_join(bool tc, const AttnParams& p, int* err, cudaStream_t stream) {
    switch (p.head_dim) {
        case 64: return launch_join_width<64>(tc, p, err, stream);
        case 128: return launch_join_width<128>(tc, p, err, stream);
        case 256: return launch_join_width<256>(tc, p, err, stream);
        default: return cudaErrorInvalidValue;
    }
}

inline int64_t slot_rows(int64_t row_tile, int64_t rows, int64_t group) {
    return rows * group < row_tile ? rows * group : row_tile;
}
inline int64_t align32(int64_t v) { return (v + 31) / 32 * 32; }

}  // namespace

int64_t tree_attention_workspace(int64_t rows, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t,
                                 int num_sms) {
    // that of the largest row tile: a call's own rows choose the form
    const int64_t n = 2 * (int64_t)num_sms * slot_rows(TcForm<64>::kRows, rows, q_heads / kv_heads);
    return (int64_t)sizeof(CutItem) * num_sms + align32(n * 8) + n * head_dim * 4;
}

cudaError_t launch_tree_attention(const iq4xs_tree_attention_args& a, const CacheView& c, const BatchView& b, bool bf16,
                                  void* encode, int* err, int num_sms, int skip_stage, cudaStream_t stream) {
    AttnParams p;
    const int group = (int)(a.q_heads / c.heads);
    p.q = static_cast<const uint16_t*>(a.q);
    p.out = a.out;
    p.mask = a.tree_mask;
    p.q_row_stride = a.q_row_stride;
    p.out_row_stride = a.out_row_stride;
    p.rows = a.rows;
    p.layer_offset = a.layer * c.layer_stride;
    p.scale_log2 = a.scale == 0 ? 1.f : (float)(fabs(a.scale) * 1.4426950408889634);
    p.q_and = a.scale == 0 ? 0u : 0xffffffffu;
    p.q_xor = a.scale < 0 ? 0x80008000u : 0u;
    p.group = group;
    p.group_magic = ((uint64_t(1) << 38) + group - 1) / group;
    p.wide_out = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.out_row_stride % 8 == 0;
    p.kv_heads = c.heads;
    p.mask_words = (int)a.mask_words;
    p.head_dim = c.head_dim;
    p.skip_stage = skip_stage;
    // The warp-level form up to 8 rows a sequence and key/value head (7
    // sequences of 9,000 tokens, 8 rows, 128 channels, bf16: 42.7 us, tcgen05
    // 47.4), and up to 16 at 256 channels (12 rows, fp16: 45.6 and 49.2) or
    // where the items are few (16 rows of one sequence of 30,000, 128 channels:
    // 34.3 and 36.1; of 4 sequences 82.6 and 69.3, of 7 of 9,000 57.3 and 47.8);
    // tcgen05 with tiles of 128 beyond (20 rows of 64 channels: 34.5 us, 45.2 by
    // warp-level tiles of 24).
    const int64_t mean_rows = (a.rows + b.sequences - 1) / b.sequences * group;
    // Items there can be at most: a row tile more than whole ones a sequence.
    const auto items = [&](int rows) {
        return c.heads * ((a.rows < b.sequences ? a.rows : b.sequences) + a.rows * group / rows);
    };
    const auto few = [&](int64_t n) { return n * (kMaxCluster + 1) <= num_sms; };  // a cluster for each fits
    const int row_tile = mean_rows <= 8                                             ? 8
                         : mean_rows <= 16 && (c.head_dim == 256 || few(items(16))) ? 16
                                                                                    : 128;
    const bool tc = row_tile == 128;
    p.ctas = num_sms < kMaxParts ? num_sms : kMaxParts;
    p.cluster = 1;
    const int64_t tokens = (int64_t)b.table_width * c.page_size;  // no sequence is longer
    p.whole_items = tokens <= kWholeTokens;
    if (!tc && tokens > kAloneTokens && tokens <= kClusterTokens && few(items(row_tile))) {
        p.cluster = kMaxCluster;  // (one more in `few`: a GPC's SMs are no multiple of eight)
        p.ctas = (int)items(row_tile);
        p.whole_items = 1;
    }
    p.slot_rows = (int)slot_rows(row_tile, a.rows, group);
    // Measured: starting and ending a part costs about 8 key tiles on tcgen05, 3 on the warp-level form.
    p.part_tiles = tc ? 8 : 3;
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    p.cuts = reinterpret_cast<CutItem*>(ws);
    ws += sizeof(CutItem) * num_sms;
    p.part_ml = reinterpret_cast<float2*>(ws);
    p.part_o = reinterpret_cast<float*>(ws + align32(2 * (int64_t)p.ctas * p.slot_rows * 8));
    CUtensorMap tk, tv;
    const EncodeTiledFn enc = reinterpret_cast<EncodeTiledFn>(encode);
    // Boxes of whole pages' rows where the form's tiles can take them (one
    // copy instead of one a chunk); the tcgen05 tiles cannot where a page is
    // shorter than a tile, for all of a chunk's keys lie together there.
    const int tile = !tc ? MmaForm<1>::kKeys : c.head_dim == 256 ? TcForm<256>::kKeys : TcForm<128>::kKeys;
    p.box_slots = c.page_size < tile ? c.page_size : tile;
    p.box_chunks = tc && c.page_size < tile ? 1 : c.head_dim / 64;
    if (!encode_kv(enc, c.k + p.layer_offset, c, bf16, p.box_slots, p.box_chunks, &tk) ||
        !encode_kv(enc, c.v + p.layer_offset, c, bf16, p.box_slots, p.box_chunks, &tv))
        return cudaErrorInvalidValue;
    const cudaError_t e = tc ? launch_attention_tc(p, &tk, &tv, c, b, bf16, err, stream)
                             : launch_attention_mma(row_tile, p, &tk, &tv, c, b, bf16, err, stream);
    if (e != cudaSuccess || p.whole_items) return e;
    return launch_join(tc, p, err, stream);
}

}  // namespace iq4xs
