// append.cu -- from the projections' fp32 rows to attention's operands in one
// pass: per-head RMS norm of q and k, rotation of the first rot_dim channels,
// one rounding to the cache's 16-bit type, q to its buffer and k, v into the
// paged cache.
//
//   y_i = x_i * w_i / sqrt(mean(x^2) + eps);  (a, b) -> (a cos - b sin, a sin + b cos)
//
// Every value is read once (4 bytes) and written once (2 bytes), so HBM
// bounds it.  A warp owns several heads of one row: their loads are in flight
// together, the row's sequence, position and rotation are looked up once, a
// head's values stay in the warp's registers, the mean is five shuffles, and
// a rotation partner is a shuffle (or the lane's next value) away.
#include "cache.cuh"

namespace iq4xs {
namespace {

constexpr int kAppendThreads = 256;

struct AppendParams {
    const float* x[3];        // q, k, v
    int64_t row_stride[3];
    int64_t head_stride[3];
    const float* weight[2];   // q, k
    const float* rope;
    const int32_t* positions;
    uint16_t* q_out;
    int64_t q_out_row_stride;
    int64_t layer_offset;     // elements
    int64_t rope_positions;
    float eps;
    int rot_half, rows, q_heads;
};

// Heads of a row that a warp takes: 2 KB of fp32 in flight (measured at 12289
// rows of 48 heads of 128: one head a warp 142 us).
template <int D>
constexpr int heads_of() { return D == 64 ? 8 : D == 128 ? 4 : 2; }

template <int D, class T, bool kInter>
__global__ void __launch_bounds__(kAppendThreads)
    qk_norm_rope_kernel(const AppendParams p, const CacheView c, const BatchView b, int* err) {
    constexpr int kVec = D >= 128 ? 4 : 2;       // consecutive channels of a lane
    constexpr int kBlocks = D / (32 * kVec);     // such runs, 32 * kVec channels apart
    constexpr int kHeads = heads_of<D>();
    griddep_launch_dependents();
    griddep_wait();  // the projections (and lengths, tables) may come from the preceding grid
    const Bc bc = bc_open(err);
    const int lane = threadIdx.x & 31;
    const int heads = p.q_heads + 2 * c.heads, groups = (heads + kHeads - 1) / kHeads;
    const int unit = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const int row = unit / groups;
    if (row >= p.rows) return;
    const int h0 = (unit - row * groups) * kHeads;

    float v[kHeads][kBlocks][kVec];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i;
        const int kind = h < p.q_heads ? 0 : h < p.q_heads + c.heads ? 1 : 2;
        const int in_kind = h - (kind == 0 ? 0 : kind == 1 ? p.q_heads : p.q_heads + c.heads);
        const float* x = p.x[kind] + row * p.row_stride[kind] + in_kind * p.head_stride[kind];
        const int64_t extent = 4 * ((p.rows - 1) * p.row_stride[kind] +
                                    ((kind == 0 ? p.q_heads : c.heads) - 1) * p.head_stride[kind] + D);
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            const float* src = x + (j * 32 + lane) * kVec;
            const bool ok = h < heads && bc_global(bc, src, 4 * kVec, p.x[kind], extent, kBcAppX);
            if constexpr (kVec == 4) {
                const float4 f = ok ? __ldcs(reinterpret_cast<const float4*>(src)) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[i][j][0] = f.x; v[i][j][1] = f.y; v[i][j][2] = f.z; v[i][j][3] = f.w;
            } else {
                const float2 f = ok ? __ldcs(reinterpret_cast<const float2*>(src)) : make_float2(0.f, 0.f);
                v[i][j][0] = f.x; v[i][j][1] = f.y;
            }
        }
    }

    // The row's sequence: the sequences that end at or before it come first
    // (offsets do not fall), so it is their number; 32 offsets a step.
    const int given = p.positions != nullptr ? p.positions[row] : 0;
    int s = 0;
    for (int s0 = 0; s0 < b.sequences; s0 += 32) {
        const int i = s0 + lane;
        const unsigned done = __ballot_sync(0xffffffffu, i < b.sequences && b.row_offsets[i + 1] <= row);
        s += __popc(done);
        if (done != 0xffffffffu) break;
    }
    if (s >= b.sequences || row < b.row_offsets[0]) return;  // a row of no sequence
    int first;
    const int n = batch_rows(b, s, p.rows, &first, err);
    const int len = batch_len(b, s, err);
    if (n == 0 || len < 0 || row < first || len > INT32_MAX - n) return;
    const int at = len + (row - first);

    // The rotation of the lane's channels: (cos, sin) of their pairs.
    constexpr int kPairs = kInter ? kVec / 2 : kVec;
    float2 turn[kBlocks][kPairs];
    const int pos = p.positions != nullptr ? given : at;
    if (p.rot_half > 0 && h0 < p.q_heads + c.heads) {
        if (pos < 0 || pos >= p.rope_positions) {
            data_error(err, kDataPosition);
            return;
        }
        const float* cs = p.rope + (int64_t)pos * 2 * p.rot_half;
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            const int i = (j * 32 + lane) * kVec;
            const int pair = kInter ? i / 2 : i < p.rot_half ? i : i - p.rot_half;
#pragma unroll
            for (int e = 0; e < kPairs; ++e)
                turn[j][e] = i < 2 * p.rot_half && bc_global(bc, cs + 2 * (pair + e), 8, p.rope,
                                                             p.rope_positions * 8 * p.rot_half, kBcAppRope)
                                 ? __ldg(reinterpret_cast<const float2*>(cs + 2 * (pair + e)))
                                 : make_float2(1.f, 0.f);
        }
    }
    int page = -1;
    if (h0 + kHeads > p.q_heads) {
        page = page_of(c, b, s, at, err);
        if (page < 0 && h0 >= p.q_heads) return;
    }

#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i;
        if (h >= heads) break;
        const int kind = h < p.q_heads ? 0 : h < p.q_heads + c.heads ? 1 : 2;
        const int in_kind = h - (kind == 0 ? 0 : kind == 1 ? p.q_heads : p.q_heads + c.heads);
        if (kind < 2) {
            if (p.weight[kind] != nullptr) {
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < kBlocks; ++j)
#pragma unroll
                    for (int e = 0; e < kVec; ++e) sum = fmaf(v[i][j][e], v[i][j][e], sum);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const float r = 1.0f / sqrtf(sum * (1.0f / D) + p.eps);
#pragma unroll
                for (int j = 0; j < kBlocks; ++j) {
                    const float* w = p.weight[kind] + (j * 32 + lane) * kVec;
                    if (bc_global(bc, w, 4 * kVec, p.weight[kind], 4 * D, kBcAppW)) {
#pragma unroll
                        for (int e = 0; e < kVec; ++e) v[i][j][e] = v[i][j][e] * r * __ldg(w + e);
                    }
                }
            }
            if (p.rot_half > 0) {
                if constexpr (kInter) {
#pragma unroll
                    for (int j = 0; j < kBlocks; ++j)
#pragma unroll
                        for (int e = 0; e < kPairs; ++e) {
                            const float a0 = v[i][j][2 * e], a1 = v[i][j][2 * e + 1];
                            v[i][j][2 * e] = a0 * turn[j][e].x - a1 * turn[j][e].y;
                            v[i][j][2 * e + 1] = a0 * turn[j][e].y + a1 * turn[j][e].x;
                        }
                } else {
                    // The partner of channel k is k + half (k < half) or k - half:
                    // rot_half is a multiple of kVec, so a lane's run has its
                    // partners in one lane's run.  (Channels behind the rotated
                    // ones meet cos 1, sin 0 and some finite or infinite partner:
                    // they are left out.)
                    float q[kBlocks][kVec];
#pragma unroll
                    for (int j = 0; j < kBlocks; ++j) {
                        const int k = (j * 32 + lane) * kVec;
                        const int from = (k < p.rot_half ? k + p.rot_half : k - p.rot_half) & (D - 1);
                        const int src_lane = (from / kVec) & 31, src_block = from / (32 * kVec);
#pragma unroll
                        for (int e = 0; e < kVec; ++e) {
                            float got = __shfl_sync(0xffffffffu, v[i][0][e], src_lane);
                            if constexpr (kBlocks == 2) {
                                const float other = __shfl_sync(0xffffffffu, v[i][1][e], src_lane);
                                got = src_block ? other : got;
                            }
                            q[j][e] = got;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < kBlocks; ++j) {
                        const int k = (j * 32 + lane) * kVec;
                        if (k < 2 * p.rot_half) {
#pragma unroll
                            for (int e = 0; e < kVec; ++e) {
                                const float2 t = turn[j][e];
                                v[i][j][e] = k < p.rot_half ? v[i][j][e] * t.x - q[j][e] * t.y
                                                            : q[j][e] * t.y + v[i][j][e] * t.x;
                            }
                        }
                    }
                }
            }
        }
        uint16_t *dst, *base;
        int64_t extent;
        if (kind == 0) {
            base = p.q_out;
            dst = base + row * p.q_out_row_stride + (int64_t)in_kind * D;
            extent = 2 * ((p.rows - 1) * p.q_out_row_stride + (int64_t)p.q_heads * D);
        } else {
            if (page < 0) continue;
            base = kind == 1 ? c.k : c.v;
            dst = base + p.layer_offset + page * c.page_stride + in_kind * c.head_stride +
                  (at & (c.page_size - 1)) * c.slot_stride;
            extent = c.extent;
        }
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            uint16_t* to = dst + (j * 32 + lane) * kVec;
            if (!bc_global(bc, to, 2 * kVec, base, extent, kind == 0 ? kBcAppQ : kBcAppKv)) continue;
            if constexpr (kVec == 4)
                *reinterpret_cast<uint2*>(to) =
                    make_uint2(T::pack(v[i][j][0], v[i][j][1]), T::pack(v[i][j][2], v[i][j][3]));
            else
                *reinterpret_cast<uint32_t*>(to) = T::pack(v[i][j][0], v[i][j][1]);
        }
    }
}

template <int D, class T>
cudaError_t launch_width(const AppendParams& p, const CacheView& c, const BatchView& b, bool inter, int* err,
                         cudaStream_t stream) {
    const int heads = p.q_heads + 2 * c.heads;
    const int64_t units = (int64_t)p.rows * ((heads + heads_of<D>() - 1) / heads_of<D>());
    const dim3 grid((unsigned)((units + kAppendThreads / 32 - 1) / (kAppendThreads / 32)));
    return inter ? launch_chained(qk_norm_rope_kernel<D, T, true>, grid, dim3(kAppendThreads), 0, stream, 1, p, c, b, err)
                 : launch_chained(qk_norm_rope_kernel<D, T, false>, grid, dim3(kAppendThreads), 0, stream, 1, p, c, b, err);
}

template <class T>
cudaError_t launch_type(const AppendParams& p, const CacheView& c, const BatchView& b, bool inter, int* err,
                        cudaStream_t stream) {
    switch (c.head_dim) {
        case 64: return launch_width<64, T>(p, c, b, inter, err, stream);
        case 128: return launch_width<128, T>(p, c, b, inter, err, stream);
        case 256: return launch_width<256, T>(p, c, b, inter, err, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const iq4xs_qk_norm_rope_args& a, const CacheView& c, const BatchView& b, bool bf16,
                                int* err, cudaStream_t stream) {
    AppendParams p;
    p.x[0] = a.q; p.x[1] = a.k; p.x[2] = a.v;
    p.row_stride[0] = a.q_row_stride; p.row_stride[1] = a.k_row_stride; p.row_stride[2] = a.v_row_stride;
    p.head_stride[0] = a.q_head_stride; p.head_stride[1] = a.k_head_stride; p.head_stride[2] = a.v_head_stride;
    p.weight[0] = a.q_weight; p.weight[1] = a.k_weight;
    p.rope = a.rope;
    p.positions = a.positions;
    p.q_out = static_cast<uint16_t*>(a.q_out);
    p.q_out_row_stride = a.q_out_row_stride;
    p.layer_offset = a.layer * c.layer_stride;
    p.rope_positions = a.rope_positions;
    p.eps = (float)a.eps;
    p.rot_half = (int)(a.rot_dim / 2);
    p.rows = (int)a.rows;
    p.q_heads = (int)a.q_heads;
    return bf16 ? launch_type<KvBf16>(p, c, b, a.interleaved != 0, err, stream)
                : launch_type<KvF16>(p, c, b, a.interleaved != 0, err, stream);
}

}  // namespace iq4xs
