// token_probs.cu -- the target's probabilities from its logits.
//
//   p_i = e^((l_i - top) / T) / sum_j e^((l_j - top) / T)
//
// or, T not above 0, 1 at the first of the largest logits.  A row is read once,
// by a cluster of CTAs that keep their parts in registers and exchange maximum
// and sum through distributed shared memory, and written once: HBM bounds it.
// Rows start at any multiple of four bytes; a part's units of four values lie on
// 16-byte boundaries of the logits, cut at the row's ends.
#include "cache.cuh"
#include "delta.cuh"

namespace iq4xs {
namespace {

constexpr int kProbThreads = 512;
constexpr int kProbUnits = 8;  // of four logits that a thread keeps
constexpr int kProbPart = 4 * kProbThreads * kProbUnits;
constexpr int kProbCluster = 8;

struct Top {
    float x;   // largest logit
    int at;    // where it stands first
    float sum; // of e^((l - x) / T)
};
__device__ __forceinline__ uint32_t rank_addr(const void* p, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float ld_rank(const float* p, int rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(rank_addr(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ int ld_rank(const int* p, int rank) {
    int v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(rank_addr(p, rank)) : "memory");
    return v;
}

__global__ void __launch_bounds__(kProbThreads) token_probs_kernel(const float* logits, int64_t logits_stride,
                                                                   int64_t rows, int vocab, const float* temperature,
                                                                   float* probs, int64_t probs_stride, int ranks,
                                                                   int* err) {
    __shared__ float tops[kProbThreads / 32], sums[kProbThreads / 32], mine[2];
    __shared__ int places[kProbThreads / 32], my_place;
    griddep_launch_dependents();
    griddep_wait();
    const Bc bc = bc_open(err);
    const int rank = blockIdx.x % ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / ranks;
    const float* const in = logits + row * logits_stride;
    float* const out = probs + row * probs_stride;
    const int64_t in_extent = 4 * ((rows - 1) * logits_stride + vocab), out_extent = 4 * ((rows - 1) * probs_stride + vocab);
    // unit u holds values 4 u - skew .. + 3
    const int skew = (int)(reinterpret_cast<uintptr_t>(in) >> 2 & 3);
    const bool same = (int)(reinterpret_cast<uintptr_t>(out) >> 2 & 3) == skew;
    const int units = (vocab + skew + 3) / 4, each = (units + ranks - 1) / ranks;
    const int u0 = rank * each, u1 = min(units, u0 + each);
    float t = 1.f;
    if (temperature != nullptr && bc_global(bc, temperature + row, 4, temperature, 4 * rows, kBcTemp)) t = temperature[row];
    const bool greedy = !(t > 0.f);
    auto load = [&](int u, float (&x)[4]) {
        const int i0 = 4 * u - skew;
        if (i0 >= 0 && i0 + 4 <= vocab) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (bc_global(bc, in + i0, 16, logits, in_extent, kBcLogits)) v = *reinterpret_cast<const float4*>(in + i0);
            x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = -INFINITY;
                if (i0 + e >= 0 && i0 + e < vocab && bc_global(bc, in + i0 + e, 4, logits, in_extent, kBcLogits))
                    x[e] = in[i0 + e];
            }
        }
    };
    float x[kProbUnits][4];
    float top = -INFINITY;
    int place = INT32_MAX;
    bool odd = false;  // a NaN
    auto look = [&](const float (&v)[4], int u) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            odd |= isnan(v[e]);
            if (v[e] > top) {  // (places rise)
                top = v[e];
                place = 4 * u - skew + e;
            }
        }
    };
#pragma unroll
    for (int k = 0; k < kProbUnits; ++k) {
        const int u = u0 + k * kProbThreads + tid;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[k][e] = -INFINITY;
        if (u < u1) load(u, x[k]);
    }
#pragma unroll
    for (int k = 0; k < kProbUnits; ++k) look(x[k], u0 + k * kProbThreads + tid);
    for (int u = u0 + kProbUnits * kProbThreads + tid; u < u1; u += kProbThreads) {  // what registers do not hold
        float v[4];
        load(u, v);
        look(v, u);
    }
    auto first_top = [&](float other, int at) {
        if (other > top || (other == top && at < place)) {
            top = other;
            place = at;
        }
    };
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        first_top(__shfl_xor_sync(0xffffffffu, top, o), __shfl_xor_sync(0xffffffffu, place, o));
    if (lane == 0) {
        tops[warp] = top;
        places[warp] = place;
    }
    odd = __syncthreads_or(odd);
    for (int w = 0; w < kProbThreads / 32; ++w) first_top(tops[w], places[w]);
    // The part's sum against its own maximum; the row's is made of the parts'.
    const float scale = 1.f / t;
    float sum = 0.f;
    auto add = [&](const float (&v)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += v[e] == -INFINITY ? 0.f : expf((v[e] - top) / t);
    };
    (void)scale;
    if (!greedy) {
#pragma unroll
        for (int k = 0; k < kProbUnits; ++k) add(x[k]);
        for (int u = u0 + kProbUnits * kProbThreads + tid; u < u1; u += kProbThreads) {
            float v[4];
            load(u, v);
            add(v);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sums[warp] = sum;
    __syncthreads();
    sum = 0.f;
    for (int w = 0; w < kProbThreads / 32; ++w) sum += sums[w];
    if (odd) sum = NAN;
    if (ranks > 1) {
        if (tid == 0) {
            mine[0] = top;
            mine[1] = sum;
            my_place = place;
        }
        cluster_arrive_release();
        cluster_wait();
        float all = 0.f;
        for (int r = 0; r < ranks; ++r) first_top(ld_rank(&mine[0], r), ld_rank(&my_place, r));
        for (int r = 0; r < ranks; ++r) {
            const float part_top = ld_rank(&mine[0], r), part = ld_rank(&mine[1], r);
            all += greedy || part_top == -INFINITY ? (isnan(part) ? part : 0.f) : part * expf((part_top - top) / t);
        }
        sum = all;
        cluster_arrive_release();  // (no CTA ends while another reads its part)
    }
    const bool nothing = top == -INFINITY && !isnan(sum), bad = isnan(sum) || (!greedy && top == INFINITY);
    const float inverse = 1.f / sum;
    auto put = [&](const float (&v)[4], int u) {
        const int i0 = 4 * u - skew;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[e] = bad ? NAN
                   : nothing || v[e] == -INFINITY ? 0.f
                   : greedy ? (i0 + e == place ? 1.f : 0.f)
                            : expf((v[e] - top) / t) * inverse;
        if (same && i0 >= 0 && i0 + 4 <= vocab) {
            if (bc_global(bc, out + i0, 16, probs, out_extent, kBcProbs))
                *reinterpret_cast<float4*>(out + i0) = make_float4(y[0], y[1], y[2], y[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i0 + e >= 0 && i0 + e < vocab && bc_global(bc, out + i0 + e, 4, probs, out_extent, kBcProbs))
                    out[i0 + e] = y[e];
        }
    };
#pragma unroll
    for (int k = 0; k < kProbUnits; ++k) {
        const int u = u0 + k * kProbThreads + tid;
        if (u < u1) put(x[k], u);
    }
    for (int u = u0 + kProbUnits * kProbThreads + tid; u < u1; u += kProbThreads) {
        float v[4];
        load(u, v);
        put(v, u);
    }
    if (ranks > 1) cluster_wait();
}

}  // namespace

cudaError_t launch_token_probs(const float* logits, int64_t logits_stride, int64_t rows, int64_t vocab,
                               const float* temperature, float* probs, int64_t probs_stride, int* err,
                               cudaStream_t stream) {
    int ranks = 1;
    while (ranks < kProbCluster && (int64_t)ranks * kProbPart < vocab + 3) ranks *= 2;
    return launch_chained(token_probs_kernel, dim3((unsigned)(rows * ranks)), dim3(kProbThreads), 0, stream, ranks, logits,
                          logits_stride, rows, (int)vocab, temperature, probs, probs_stride, ranks, err);
}

}  // namespace iq4xs
