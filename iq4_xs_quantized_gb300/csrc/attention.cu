// attention.cu -- attention of new tokens over the paged cache under a tree
// mask, in its simplest form: a CTA per (row, query head), a warp per key.
//
//   o = sum_p w_p v_p / sum_p w_p,  w_p = exp(scale q.k_p - m)
//
// one pass with a running maximum m and sum; the warps' partial results are
// joined at the end.
#include "cache.cuh"

namespace iq4xs {
namespace {

constexpr int kThreads = 128;

template <int D, class T>
__global__ void __launch_bounds__(kThreads)
    attention_kernel(const iq4xs_tree_attention_args a, const CacheView c, const BatchView b, int* err) {
    constexpr int kPer = D / 32;  // channels of a lane, 2 adjacent ones 64 apart
    __shared__ float part[kThreads / 32][D + 2];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int row = blockIdx.x, h = blockIdx.y, kvh = h / (int)(a.q_heads / c.heads);
    int s = 0;
    for (int s0 = 0; s0 < b.sequences; s0 += 32) {
        const unsigned done =
            __ballot_sync(0xffffffffu, s0 + lane < b.sequences && b.row_offsets[s0 + lane + 1] <= row);
        s += __popc(done);
        if (done != 0xffffffffu) break;
    }
    if (s >= b.sequences || row < b.row_offsets[0]) return;
    int first;
    const int n = batch_rows(b, s, a.rows, &first, err), len = batch_len(b, s, err), t = row - first;
    if (n == 0 || len < 0 || t < 0 || len > INT32_MAX - n) return;

    const uint16_t* q = static_cast<const uint16_t*>(a.q) + row * a.q_row_stride + (int64_t)h * D;
    float qv[kPer], o[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
        const float2 f = T::unpack(*reinterpret_cast<const uint32_t*>(q + 32 * i + 2 * lane));
        qv[i] = f.x * (float)a.scale;
        qv[i + 1] = f.y * (float)a.scale;
        o[i] = o[i + 1] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int p = w; p < len + n; p += kThreads / 32) {
        const int j = p - len;
        if (j >= 0) {
            const bool seen = a.tree_mask == nullptr ? j <= t
                              : j < 64 * a.mask_words && (a.tree_mask[row * a.mask_words + (j >> 6)] >> (j & 63) & 1);
            if (!seen) continue;
        }
        const int page = page_of(c, b, s, p, err);
        if (page < 0) continue;
        const int64_t at = a.layer * c.layer_stride + page * c.page_stride + kvh * c.head_stride +
                           (p & (c.page_size - 1)) * c.slot_stride;
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; i += 2) {
            const float2 f = T::unpack(*reinterpret_cast<const uint32_t*>(c.k + at + 32 * i + 2 * lane));
            x = fmaf(qv[i], f.x, fmaf(qv[i + 1], f.y, x));
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        const float m2 = fmaxf(m, x);
        const float old = m2 == -INFINITY ? 1.f : expf(m - m2), e = m2 == -INFINITY ? 0.f : expf(x - m2);
        l = l * old + e;
#pragma unroll
        for (int i = 0; i < kPer; i += 2) {
            const float2 f = T::unpack(*reinterpret_cast<const uint32_t*>(c.v + at + 32 * i + 2 * lane));
            o[i] = o[i] * old + e * f.x;
            o[i + 1] = o[i + 1] * old + e * f.y;
        }
        m = m2;
    }
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
        part[w][32 * i + 2 * lane] = o[i];
        part[w][32 * i + 2 * lane + 1] = o[i + 1];
    }
    if (lane == 0) {
        part[w][D] = m;
        part[w][D + 1] = l;
    }
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
    for (int i = 0; i < kThreads / 32; ++i) top = fmaxf(top, part[i][D]);
    for (int i = 0; i < kThreads / 32; ++i) sum += top == -INFINITY ? 0.f : part[i][D + 1] * expf(part[i][D] - top);
    for (int d = threadIdx.x; d < D; d += kThreads) {
        float v = 0.f;
        for (int i = 0; i < kThreads / 32; ++i)
            v += top == -INFINITY || part[i][D + 1] == 0.f ? 0.f : part[i][d] * expf(part[i][D] - top);
        a.out[row * a.out_row_stride + (int64_t)h * D + d] = sum == 0.f ? 0.f : v / sum;
    }
}

template <class T>
cudaError_t launch_type(const iq4xs_tree_attention_args& a, const CacheView& c, const BatchView& b, int* err,
                        cudaStream_t stream) {
    const dim3 grid((unsigned)a.rows, (unsigned)a.q_heads);
    switch (c.head_dim) {
        case 64: return launch_chained(attention_kernel<64, T>, grid, dim3(kThreads), 0, stream, a, c, b, err);
        case 128: return launch_chained(attention_kernel<128, T>, grid, dim3(kThreads), 0, stream, a, c, b, err);
        case 256: return launch_chained(attention_kernel<256, T>, grid, dim3(kThreads), 0, stream, a, c, b, err);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

int64_t tree_attention_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int) { return 16; }

cudaError_t launch_tree_attention(const iq4xs_tree_attention_args& a, const CacheView& c, const BatchView& b, bool bf16,
                                  void*, int* err, int, cudaStream_t stream) {
    return bf16 ? launch_type<KvBf16>(a, c, b, err, stream) : launch_type<KvF16>(a, c, b, err, stream);
}

}  // namespace iq4xs
