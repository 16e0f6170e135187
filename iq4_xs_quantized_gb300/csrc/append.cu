// append.cu -- from the projections' fp32 rows to attention's operands in one
// pass: per-head RMS norm of q and k, rotation of the first rot_dim channels,
// one rounding to the cache's 16-bit type, q to its buffer and k, v into the
// paged cache.
//
//   y_i = x_i * w_i / sqrt(mean(x^2) + eps);  (a, b) -> (a cos - b sin, a sin + b cos)
//
// Every value is read once (4 bytes) and written once (2 bytes), so HBM
// bounds it, and the instructions a value takes come next.  D / 8 lanes own a
// head, eight channels each (four from the head's first half, four from its
// second), and a warp several heads of one row: their loads are in flight
// together, the row's sequence, position and rotation are looked up once, the
// mean is three to five shuffles for all of them, and a rotation partner is
// the lane's own other half, its next value, or a shuffle away.  With many rows
// a warp goes on to further heads of its row: the looking up is half of a
// step's instructions.
//
// Measured: 12,289 rows of 32 + 2 x 8 heads of 128 channels, all rotated, bf16:
// 459 MB in 71.7 us, 6.4 TB/s, 94 % of a copy's rate (a step a warp 79, a warp
// a head 142); 8,000 rows of 24 + 2 x 4 heads of 256: 393 MB in 69 us, 84 % (86).
// One row of the latter: 2.7 us, a launch and three loads that wait for one
// another.  One step of four heads instead of two at a time: the same on many
// rows, 3.5 us on one.
#include "cache.cuh"

namespace iq4xs {
namespace {

constexpr int kAppendThreads = 128;

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
    int steps;  // of AppendShape::kHeads heads that a warp takes
};

// A warp's heads: side by side, and one after another (2 KB of fp32 in flight).
template <int D>
struct AppendShape {
    static constexpr int kLanes = D / 8;          // of a head
    static constexpr int kAbreast = 32 / kLanes;
    static constexpr int kDeep = 2;
    static constexpr int kHeads = kAbreast * kDeep;
};

template <int D, class T, bool kInter>
__global__ void __launch_bounds__(kAppendThreads)
    qk_norm_rope_kernel(const AppendParams p, const CacheView c, const BatchView b, int* err) {
    using S = AppendShape<D>;
    constexpr int kL = S::kLanes, kDeep = S::kDeep;
    griddep_launch_dependents();
    griddep_wait();  // the projections (and lengths, tables) may come from the preceding grid
    const Bc bc = bc_open(err);
    const int lane = threadIdx.x & 31, l = lane % kL;
    const int heads = p.q_heads + 2 * c.heads, span = p.steps * S::kHeads, parts = (heads + span - 1) / span;
    const int unit = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const int row = unit / parts;
    if (row >= p.rows) return;
    int h0 = (unit - row * parts) * span;
    const int h_end = min(heads, h0 + span);

    // The lane's channels: 4 l + e of the head's first half (block 0) and second.
    float v[kDeep][2][4];
    int kind[kDeep], in_kind[kDeep];
    const auto load = [&] {
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const int h = min(h0 + i * S::kAbreast + lane / kL, heads - 1);  // (the last again instead of a branch)
            kind[i] = h < p.q_heads ? 0 : h < p.q_heads + c.heads ? 1 : 2;
            in_kind[i] = h - (kind[i] == 0 ? 0 : kind[i] == 1 ? p.q_heads : p.q_heads + c.heads);
            const float* base = kind[i] == 0 ? p.x[0] : kind[i] == 1 ? p.x[1] : p.x[2];
            const int64_t rs = kind[i] == 0 ? p.row_stride[0] : kind[i] == 1 ? p.row_stride[1] : p.row_stride[2];
            const int64_t hs = kind[i] == 0 ? p.head_stride[0] : kind[i] == 1 ? p.head_stride[1] : p.head_stride[2];
            const float* x = base + row * rs + in_kind[i] * hs + 4 * l;
            const int64_t extent = 4 * ((p.rows - 1) * rs + ((kind[i] == 0 ? p.q_heads : c.heads) - 1) * hs + D);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const bool ok = bc_global(bc, x + j * (D / 2), 16, base, extent, kBcAppX);
                const float4 f =
                    ok ? __ldcs(reinterpret_cast<const float4*>(x + j * (D / 2))) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[i][j][0] = f.x; v[i][j][1] = f.y; v[i][j][2] = f.z; v[i][j][3] = f.w;
            }
        }
    };
    load();

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
    constexpr int kPairs = kInter ? 2 : 4;
    float2 turn[2][kPairs];
    const int pos = p.positions != nullptr ? given : at;
    bool placed = true;  // (else the row's q and k stay unwritten)
    if (p.rot_half > 0 && h0 < p.q_heads + c.heads) {
        if (pos < 0 || pos >= p.rope_positions) {
            data_error(err, kDataPosition);
            placed = false;
        }
        const float* cs = p.rope + (int64_t)pos * 2 * p.rot_half;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = j * (D / 2) + 4 * l;
            const float* from = cs + (kInter ? k : 2 * (k < p.rot_half ? k : k - p.rot_half));
#pragma unroll
            for (int e = 0; e < kPairs; e += 2) {
                float4 t = make_float4(1.f, 0.f, 1.f, 0.f);
                if (placed && k < 2 * p.rot_half &&
                    bc_global(bc, from + 2 * e, 16, p.rope, p.rope_positions * 8 * p.rot_half, kBcAppRope))
                    t = *reinterpret_cast<const float4*>(from + 2 * e);
                turn[j][e] = make_float2(t.x, t.y);
                turn[j][e + 1] = make_float2(t.z, t.w);
            }
        }
    }
    int page = -1;
    if (h_end > p.q_heads) page = page_of(c, b, s, at, err);

    for (;;) {
        // Step by step over all heads, so that their chains run side by side.
        float sum[kDeep];
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            sum[i] = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[i] = fmaf(v[i][j][e], v[i][j][e], sum[i]);
        }
#pragma unroll
        for (int o = kL / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < kDeep; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const float* weight = kind[i] == 0 ? p.weight[0] : kind[i] == 1 ? p.weight[1] : nullptr;
            if (weight == nullptr) continue;  // (v, or no norm)
            const float r = rsqrtf(sum[i] * (1.0f / D) + p.eps);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float* w = weight + j * (D / 2) + 4 * l;
                if (!bc_global(bc, w, 16, weight, 4 * D, kBcAppW)) continue;
                const float4 t = *reinterpret_cast<const float4*>(w);
                v[i][j][0] *= r * t.x;
                v[i][j][1] *= r * t.y;
                v[i][j][2] *= r * t.z;
                v[i][j][3] *= r * t.w;
            }
        }
        if (p.rot_half > 0) {
#pragma unroll
            for (int i = 0; i < kDeep; ++i) {
                const bool turns = kind[i] < 2;
                if constexpr (kInter) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < kPairs; ++e) {
                            const bool here = turns && j * (D / 2) + 4 * l < 2 * p.rot_half;
                            const float a0 = v[i][j][2 * e], a1 = v[i][j][2 * e + 1];
                            v[i][j][2 * e] = here ? a0 * turn[j][e].x - a1 * turn[j][e].y : a0;
                            v[i][j][2 * e + 1] = here ? a0 * turn[j][e].y + a1 * turn[j][e].x : a1;
                        }
                } else {
                    // The partner of channel k is k + half (k < half) or k - half;
                    // half is a multiple of 4, so a lane's four have theirs in one
                    // lane's four: its own other ones where all channels turn.
                    // Channels behind the rotated ones stay as they are.
                    float q[2][4];
                    if (p.rot_half == D / 2) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            q[0][e] = v[i][1][e];
                            q[1][e] = v[i][0][e];
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int k = j * (D / 2) + 4 * l;
                            const int from = (k < p.rot_half ? k + p.rot_half : k - p.rot_half) & (D - 1);
                            const int src = lane / kL * kL + from / 4 % kL;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float a0 = __shfl_sync(0xffffffffu, v[i][0][e], src);
                                const float a1 = __shfl_sync(0xffffffffu, v[i][1][e], src);
                                q[j][e] = from >= D / 2 ? a1 : a0;
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int k = j * (D / 2) + 4 * l;
                        const bool first_half = k < p.rot_half, here = turns && k < 2 * p.rot_half;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 t = turn[j][e];
                            const float x = v[i][j][e] * t.x + (first_half ? -q[j][e] : q[j][e]) * t.y;
                            v[i][j][e] = here ? x : v[i][j][e];
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            uint16_t* base = kind[i] == 0 ? p.q_out : kind[i] == 1 ? c.k : c.v;
            const int64_t offset = kind[i] == 0 ? row * p.q_out_row_stride + in_kind[i] * D
                                                : p.layer_offset + page * c.page_stride + in_kind[i] * c.head_stride +
                                                      (at & (c.page_size - 1)) * c.slot_stride;
            const int64_t extent =
                kind[i] == 0 ? 2 * ((p.rows - 1) * p.q_out_row_stride + (int64_t)p.q_heads * D) : c.extent;
            if (h0 + i * S::kAbreast + lane / kL >= h_end || (kind[i] > 0 && page < 0) || (kind[i] < 2 && !placed))
                continue;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint16_t* to = base + offset + j * (D / 2) + 4 * l;
                if (bc_global(bc, to, 8, base, extent, kind[i] == 0 ? kBcAppQ : kBcAppKv))
                    *reinterpret_cast<uint2*>(to) =
                        make_uint2(T::pack(v[i][j][0], v[i][j][1]), T::pack(v[i][j][2], v[i][j][3]));
            }
        }
        h0 += S::kHeads;
        if (h0 >= h_end) break;
        load();
    }
}

template <int D, class T>
cudaError_t launch_width(AppendParams& p, const CacheView& c, const BatchView& b, bool inter, int* err, int num_sms,
                         cudaStream_t stream) {
    constexpr int kHeads = AppendShape<D>::kHeads, kWarps = 96;
    const int heads = p.q_heads + 2 * c.heads, groups = (heads + kHeads - 1) / kHeads;
    // A warp takes several steps of heads, one look at its row for all of
    // them, while kWarps warps an SM remain; even shares.
    const int64_t want = ((int64_t)kWarps * num_sms + p.rows - 1) / p.rows;
    const int parts = want < groups ? (int)want : groups;
    p.steps = (groups + parts - 1) / parts;
    const int64_t units = (int64_t)p.rows * ((groups + p.steps - 1) / p.steps);
    const dim3 grid((unsigned)((units + kAppendThreads / 32 - 1) / (kAppendThreads / 32)));
    return inter ? launch_chained(qk_norm_rope_kernel<D, T, true>, grid, dim3(kAppendThreads), 0, stream, 1, p, c, b, err)
                 : launch_chained(qk_norm_rope_kernel<D, T, false>, grid, dim3(kAppendThreads), 0, stream, 1, p, c, b, err);
}

template <class T>
cudaError_t launch_type(AppendParams& p, const CacheView& c, const BatchView& b, bool inter, int* err, int num_sms,
                        cudaStream_t stream) {
    switch (c.head_dim) {
        case 64: return launch_width<64, T>(p, c, b, inter, err, num_sms, stream);
        case 128: return launch_width<128, T>(p, c, b, inter, err, num_sms, stream);
        case 256: return launch_width<256, T>(p, c, b, inter, err, num_sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const iq4xs_qk_norm_rope_args& a, const CacheView& c, const BatchView& b, bool bf16,
                                int* err, int num_sms, cudaStream_t stream) {
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
    return bf16 ? launch_type<KvBf16>(p, c, b, a.interleaved != 0, err, num_sms, stream)
                : launch_type<KvF16>(p, c, b, a.interleaved != 0, err, num_sms, stream);
}

}  // namespace iq4xs
