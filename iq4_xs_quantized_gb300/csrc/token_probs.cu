// token_probs.cu -- the target's probabilities from its logits.
//
//   p_i = e^((l_i - top) / T) / sum_j e^((l_j - top) / T)
//
// or, T not above 0, 1 at the first of the largest logits.  A cluster of CTAs shares a
// row and exchanges maximum and sum through distributed shared memory, in one of
// two forms.  Where registers hold the rows under way, a row is read once, kept, and
// written: one row of 32,000 3.8 us, a launch, the loads and the exchange.  Of a
// batch whose rows they do not hold, each part is read with a running maximum and sum
// and read again, out of L2, when the row's are known: 96 rows of 131,073 23.7 us from
// HBM, 4.3 TB/s of the 6.8 of a copy (18.8 with the logits in L2).  All its rows are read
// before the first is written, which bounds it: HBM is busy for 28 % of the capture's
// cycles, loads are what warps wait for (CTAs of 256 threads 24.9 to 34.8, of
// 1,024 30 and more; two and eight units abreast 24.5 and 29.4).
// Rows start at any multiple of four bytes; a part's units of four values lie on
// 16-byte boundaries of the logits, cut at the row's ends.
#include "attention.cuh"
#include "delta.cuh"

namespace iq4xs {
namespace {

constexpr int kProbThreads = 512;
constexpr int kProbWarps = kProbThreads / 32;
constexpr int kProbUnits = 4;  // of four logits that a thread keeps
constexpr int kAhead = 4;      // or has in flight
constexpr int kProbPart = 4 * kProbThreads * kProbUnits;
constexpr int kProbCluster = 8;
constexpr int kProbMost = 40000;  // logits of a part that is read twice

__device__ __forceinline__ uint32_t rank_addr(const void* p, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ uint4 ld_rank(const uint4* p, int rank) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(rank_addr(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool kGreedy, bool kHold>
__device__ __forceinline__ void row_probs(const float* logits, const float* in, int64_t in_extent, float* probs, float* out,
                                          int64_t out_extent, int vocab, float t, int rank, int ranks, const Bc& bc) {
    __shared__ float tops[kProbWarps], sums[kProbWarps];
    __shared__ int places[kProbWarps];
    __shared__ uint4 mine;  // the part's largest, where it stands, its sum
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // unit u holds values 4 u - skew .. + 3
    const int skew = (int)(reinterpret_cast<uintptr_t>(in) >> 2 & 3);
    const bool same = (int)(reinterpret_cast<uintptr_t>(out) >> 2 & 3) == skew;
    const int units = (vocab + skew + 3) / 4, each = (units + ranks - 1) / ranks;
    const int u0 = rank * each, u1 = min(units, u0 + each);
    auto load = [&](int u, float (&x)[4]) {
        const int i0 = 4 * u - skew;
        if (u < u1 && i0 >= 0 && i0 + 4 <= vocab) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (bc_global(bc, in + i0, 16, logits, in_extent, kBcLogits)) v = *reinterpret_cast<const float4*>(in + i0);
            x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = -INFINITY;
                if (u < u1 && i0 + e >= 0 && i0 + e < vocab && bc_global(bc, in + i0 + e, 4, logits, in_extent, kBcLogits))
                    x[e] = in[i0 + e];
            }
        }
    };
    float x[kHold ? kProbUnits : 1][4];
    if constexpr (kHold) {
#pragma unroll
        for (int k = 0; k < kProbUnits; ++k) load(u0 + k * kProbThreads + tid, x[k]);
    }
    // e^(d / T), d not above 0, with one rounding of the exponent: log2(e) / T, within
    // fp32's range (equal values then give 1 at any T), as a number 2^-20 below it and
    // what that lacks, above 0 so that -inf stays -inf.
    float inverse;
    asm("rcp.approx.f32 %0, %1;" : "=f"(inverse) : "f"(t));
    const float rate = 1.4426936f * inverse, c = fminf(fmaxf(rate, 1.17549435e-38f), 3.40282347e38f);
    const float lack = (fmaf(-c, t, 1.44269502f) + 1.9259630e-8f) * inverse;
    const float c2 = c == rate && lack > 0.f ? lack : 0x1p-149f;
    auto power = [&](float d) { return exp2_of(fmaf(d, c, d * c2)); };
    float top = -INFINITY, sum = 0.f;
    int place = INT32_MAX;
    auto look = [&](const float (&v)[4], int u) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (kGreedy) {
                if (isnan(v[e])) sum = v[e];
                if (v[e] > top) {  // (places rise)
                    top = v[e];
                    place = 4 * u - skew + e;
                }
            } else {
                top = fmaxf(top, v[e]);
            }
        }
    };
    auto first_top = [&](float other, int at) {
        if (kGreedy && (other > top || (other == top && at < place))) place = at;
        top = fmaxf(top, other);
    };
    float own = -INFINITY;  // what a thread's weights (or sum) are taken against
    auto weigh = [&](float (&v)[4]) {
        const float shift = own == -INFINITY ? 0.f : own;
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const float2 d = add2(make_float2(v[e], v[e + 1]), make_float2(-shift, -shift));
            const float2 z = fma2(d, make_float2(c, c), fma2(d, make_float2(c2, c2), make_float2(-0.f, -0.f)));
            v[e] = exp2_of(z.x);
            v[e + 1] = exp2_of(z.y);
        }
    };
    if constexpr (kHold) {
#pragma unroll
        for (int k = 0; k < kProbUnits; ++k) look(x[k], u0 + k * kProbThreads + tid);
    } else {
        for (int u = u0 + tid; u < u1; u += kAhead * kProbThreads) {
            float v[kAhead][4];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) load(u + k * kProbThreads, v[k]);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) look(v[k], u + k * kProbThreads);
            if (!kGreedy) {  // a running sum
                sum = top > own && own != -INFINITY ? sum * power(own - top) : sum;
                own = top;
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    weigh(v[k]);
                    sum += (v[k][0] + v[k][1]) + (v[k][2] + v[k][3]);
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, top, o);
        first_top(other, kGreedy ? __shfl_xor_sync(0xffffffffu, place, o) : 0);
    }
    if (lane == 0) {
        tops[warp] = top;
        places[warp] = place;
    }
    __syncthreads();
    for (int w = 0; w < kProbWarps; ++w) first_top(tops[w], places[w]);
    // The part's sum against its own maximum; the row's is made of the parts'.
    if (!kGreedy) {
        if constexpr (kHold) {  // weights in the logits' place
            own = top;
#pragma unroll
            for (int k = 0; k < kProbUnits; ++k) {
                weigh(x[k]);
                sum += (x[k][0] + x[k][1]) + (x[k][2] + x[k][3]);
            }
        } else {
            sum = own == -INFINITY ? sum : sum * power(own - top);
            own = top;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sums[warp] = sum;
    __syncthreads();
    sum = 0.f;
    for (int w = 0; w < kProbWarps; ++w) sum += sums[w];
    if (ranks > 1) {
        if (tid == 0) mine = make_uint4(__float_as_uint(top), (uint32_t)place, __float_as_uint(sum), 0);
        __syncwarp();  // (the barrier wants warps whole)
        cluster_arrive_release();
        cluster_wait();
        for (int r = 0; r < ranks; ++r) {
            const uint4 part = ld_rank(&mine, r);
            first_top(__uint_as_float(part.x), (int)part.y);
        }
        sum = 0.f;
        for (int r = 0; r < ranks; ++r) {
            const uint4 part = ld_rank(&mine, r);
            const float of = __uint_as_float(part.z), its = __uint_as_float(part.x);
            sum += kGreedy ? of : its == -INFINITY ? of : of * power(its - top);
        }
        cluster_arrive_release();  // (no CTA ends while another reads its part)
    }
    // A weight times this is the probability (a part without any: zeros, unless the row is NaN).
    const float factor = own == -INFINITY ? sum * 0.f : own == top ? 1.f / sum : power(own - top) / sum;
    auto put = [&](const float (&v)[4], int u) {
        const int i0 = 4 * u - skew;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[e] = kGreedy ? (isnan(sum) ? sum : i0 + e == place ? 1.f : 0.f) : v[e] * factor;
        if (same && i0 >= 0 && i0 + 4 <= vocab) {
            if (bc_global(bc, out + i0, 16, probs, out_extent, kBcProbs))
                __stcs(reinterpret_cast<float4*>(out + i0), make_float4(y[0], y[1], y[2], y[3]));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i0 + e >= 0 && i0 + e < vocab && bc_global(bc, out + i0 + e, 4, probs, out_extent, kBcProbs))
                    out[i0 + e] = y[e];
        }
    };
    if constexpr (kHold) {
#pragma unroll
        for (int k = 0; k < kProbUnits; ++k) {
            const int u = u0 + k * kProbThreads + tid;
            if (u < u1) put(x[k], u);
        }
    } else {
        for (int u = u0 + tid; u < u1; u += kAhead * kProbThreads) {
            float v[kAhead][4];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (!kGreedy) load(u + k * kProbThreads, v[k]);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (!kGreedy) weigh(v[k]);
                if (u + k * kProbThreads < u1) put(v[k], u + k * kProbThreads);
            }
        }
    }
    if (ranks > 1) {
        __syncwarp();
        cluster_wait();
    }
}

template <bool kHold>
__global__ void __launch_bounds__(kProbThreads, kHold ? 2 : 3)
    token_probs_kernel(const float* logits, int64_t logits_stride, int64_t rows, int vocab, const float* temperature,
                       float* probs, int64_t probs_stride, int ranks, int* err) {
    griddep_launch_dependents();
    griddep_wait();
    const Bc bc = bc_open(err);
    const int rank = blockIdx.x % ranks;
    const int64_t row = blockIdx.x / ranks;
    const float* const in = logits + row * logits_stride;
    float* const out = probs + row * probs_stride;
    const int64_t in_extent = 4 * ((rows - 1) * logits_stride + vocab), out_extent = 4 * ((rows - 1) * probs_stride + vocab);
    float t = 1.f;
    if (temperature != nullptr && bc_global(bc, temperature + row, 4, temperature, 4 * rows, kBcTemp)) t = temperature[row];
    if (t > 0.f) row_probs<false, kHold>(logits, in, in_extent, probs, out, out_extent, vocab, t, rank, ranks, bc);
    else row_probs<true, kHold>(logits, in, in_extent, probs, out, out_extent, vocab, 1.f, rank, ranks, bc);
}

}  // namespace

cudaError_t launch_token_probs(const float* logits, int64_t logits_stride, int64_t rows, int64_t vocab,
                               const float* temperature, float* probs, int64_t probs_stride, int* err, int num_sms,
                               cudaStream_t stream) {
    // In registers where one CTA holds a row, or all rows are under way at once, in as
    // few parts as hold it (one row of 8,000: 2.8 us by one CTA, 3.4 by four, 32,000
    // 3.9 by four and 4.1 by eight); else read twice, the second time from L2 (600 rows of
    // 8,000 6.7 us in registers, 7.1 read twice; of 32,000 8 4.4 and 5.0, 48 5.7 and 9.6, 96 9.4
    // and 8.1, 192 14.1 and 10.2).
    int ranks = 1;
    while (ranks < kProbCluster && (int64_t)ranks * kProbPart < vocab + 3) ranks *= 2;
    const bool hold = (int64_t)ranks * kProbPart >= vocab + 3 && (ranks == 1 || ranks * rows <= 2 * num_sms);
    // Read twice, as many parts as are resident at once (32,000: 96 rows 8.0, 8.8, 8.2 and 15.9 us
    // by 1, 2, 4 and 8, 200 10.9, 10.3, 14.2, 28.6, 400 14.3, 18.9, 25.1, 52.6; 131,073: one row 20.0, 12.8,
    // 8.7, 6.8), of at most 40,000 (200 rows of 131,073: 59.3, 51.1, 44.3, 53.7).
    if (!hold) {
        ranks = 1;
        while (ranks < kProbCluster && (int64_t)ranks * 4 * kProbThreads < vocab &&
               (2 * ranks * rows <= 3 * num_sms || (int64_t)ranks * kProbMost < vocab))
            ranks *= 2;
    }
    return launch_chained(hold ? token_probs_kernel<true> : token_probs_kernel<false>, dim3((unsigned)(rows * ranks)),
                          dim3(kProbThreads), 0, stream, ranks, logits, logits_stride, rows, (int)vocab, temperature, probs,
                          probs_stride, ranks, err);
}

}  // namespace iq4xs
