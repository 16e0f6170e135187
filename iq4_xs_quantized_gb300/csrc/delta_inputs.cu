// delta_inputs.cu -- from the projection's fp32 rows to the delta rule's
// operands in one pass: causal convolution over four inputs along a row's
// ancestors, SiLU, unit norm of every query and key head, one rounding to 16
// bits; decay and step size of every head; the state's last inputs.
//
// A thread takes four channels of a run of one sequence's rows and keeps the
// last three inputs in registers (chains), so that HBM reads each value once
// (4 bytes) and writes it once (2 bytes), which bounds it.  The first run of a
// sequence alone reads the state's inputs, and writes them anew: its rows are
// at least the three that need them.  A drafted tree's rows read their
// ancestors' inputs instead, out of L1 or L2.
//
// Four rows' loads are in flight together and the next four's are asked for
// before these are worked on (6,147 rows of 16 + 16 + 48 heads of 128: 74 us, 5.1 TB/s of
// the 6.8 of a copy; two abreast 82, CTAs of 256 threads 84).  Half of
// the issue slots are used then (packed arithmetic took 5 us off) and loads are
// what warps wait for; the smallest calls are a launch and three dependent loads.
#include "attention.cuh"
#include "delta.cuh"

namespace iq4xs {
namespace {

constexpr int kInputThreads = 128;
constexpr int kInputCols = 4 * kInputThreads;  // channels of a CTA
constexpr int kAbreast = 4;                    // rows whose loads are in flight together
constexpr int kLeastRun = 4, kShortRun = 16, kLongRun = 32;  // rows of one CTA
static_assert(kLeastRun >= kConvTaps - 1, "the first run alone touches the state");

struct InputParams {
    const float* x;
    const float* weight;
    const float* a;
    const float* b;
    const float* a_log;
    const float* dt_bias;
    uint16_t* out[3];          // q, k, v
    int64_t out_stride[3];
    float* g;
    float* beta;
    const uint64_t* tree_mask;
    int64_t x_stride, a_stride, b_stride, conv_offset;
    float eps;
    int mask_words, advance, rows, run, col_parts, key_lanes;
};

// Four channels, as two pairs for packed arithmetic.
struct Four {
    float2 a, b;
};
__device__ __forceinline__ Four as_four(const float4& x) { return {make_float2(x.x, x.y), make_float2(x.z, x.w)}; }
__device__ __forceinline__ void tap(Four& y, const Four& w, const Four& x) {
    y.a = fma2(w.a, x.a, y.a);
    y.b = fma2(w.b, x.b, y.b);
}
// y / (1 + e^-y) by the approximate power and reciprocal.  The exponent is rounded once,
// and so the result is off by about (8 + 1.2 |y|) 2^-24 of itself for y below 0 (8 2^-24
// above); below -87.3 the reciprocal is flushed and the result 0 (1e-36 and less).  A
// rounding to 16 bits comes behind it: fp16 holds nothing of y below -20 (2^-19 there for
// half a step of 2^-11), bf16 2^-17 at -87 for half a step of 2^-8.
__device__ __forceinline__ float2 silu(float2 y) {
    const float2 z = fma2(y, make_float2(-1.44269504088896340736f, -1.44269504088896340736f), make_float2(-0.f, -0.f));
    const float2 e = add2(make_float2(fast_exp2(z.x), fast_exp2(z.y)), make_float2(1.f, 1.f));
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
    return fma2(y, r, make_float2(-0.f, -0.f));
}

template <class T>
__global__ void __launch_bounds__(kInputThreads, 6) delta_inputs_kernel(const InputParams p, const DeltaView d,
                                                                     const BatchView b, int* err) {
    griddep_launch_dependents();
    griddep_wait();
    const Bc bc = bc_open(err);
    const int lane = threadIdx.x & 31, part = blockIdx.x % p.col_parts, at = blockIdx.x / p.col_parts;
    // Sequence s's runs begin at place row_offsets[s] / run + s: enough places
    // for them all, and the last sequence that begins at or before `at` is this one's.
    int s = -1;
    for (int s0 = 0; s0 < b.sequences; s0 += 32) {
        const int i = s0 + lane;
        const unsigned begun = __ballot_sync(0xffffffffu, i < b.sequences && b.row_offsets[i] / p.run + i <= at);
        s += __popc(begun);
        if (begun != 0xffffffffu) break;
    }
    if (s < 0) return;
    const DeltaSequence seq = delta_sequence(b, d, s, p.rows, err);
    const int first = seq.first, n = seq.n, len = seq.len, slot = seq.slot;
    const int t0 = (at - (first / p.run + s)) * p.run, t1 = min(n, t0 + p.run);
    if (len < 0 || slot < 0 || t0 < 0 || t0 >= n) return;

    if (part == p.col_parts - 1) {  // the gates
        const int64_t extent = 4 * (int64_t)p.rows * d.heads;
        for (int i = threadIdx.x; i < (t1 - t0) * d.heads; i += kInputThreads) {
            const int row = first + t0 + i / d.heads, h = i % d.heads;
            const float* a = p.a + row * p.a_stride + h;
            const float* c = p.b + row * p.b_stride + h;
            if (!bc_global(bc, a, 4, p.a, 4 * ((p.rows - 1) * p.a_stride + d.heads), kBcDeltaGate) ||
                !bc_global(bc, c, 4, p.b, 4 * ((p.rows - 1) * p.b_stride + d.heads), kBcDeltaGate))
                continue;
            float rate = 0.f, bias = 0.f;
            if (bc_global(bc, p.a_log + h, 4, p.a_log, 4 * (int64_t)d.heads, kBcDeltaGate)) rate = p.a_log[h];
            if (bc_global(bc, p.dt_bias + h, 4, p.dt_bias, 4 * (int64_t)d.heads, kBcDeltaGate)) bias = p.dt_bias[h];
            const float z = *a + bias;
            const float g = -expf(rate) * (fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))));
            const int64_t to = (int64_t)row * d.heads + h;
            if (bc_global(bc, p.g + to, 4, p.g, extent, kBcDeltaGate)) p.g[to] = g;
            if (bc_global(bc, p.beta + to, 4, p.beta, extent, kBcDeltaGate)) p.beta[to] = 1.f / (1.f + expf(-*c));
        }
        return;
    }
    const int c = part * kInputCols + 4 * threadIdx.x;
    const bool here = c < d.channels;  // (lanes behind the last channel take part in the shuffles)
    const int64_t x_extent = 4 * ((p.rows - 1) * p.x_stride + d.channels);
    const Four zero = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    auto input = [&](int row) {
        const float* from = p.x + row * p.x_stride + c;
        return here && bc_global(bc, from, 16, p.x, x_extent, kBcDeltaX) ? as_four(*reinterpret_cast<const float4*>(from)) : zero;
    };
    float* const at_conv = d.conv + p.conv_offset + slot * d.conv_slot_stride;
    auto before = [&](int i) {  // input i of the state's, oldest first
        const float* from = at_conv + (int64_t)i * d.channels + c;
        return here && len > 0 && bc_global(bc, from, 16, d.conv, d.conv_extent, kBcDeltaConv)
                   ? as_four(*reinterpret_cast<const float4*>(from)) : zero;
    };
    Four w[4];  // of a tap
    {
        float4 of[4];  // of a channel
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* from = p.weight + 4 * (int64_t)(c + i);
            of[i] = here && bc_global(bc, from, 16, p.weight, 16 * (int64_t)d.channels, kBcDeltaW)
                        ? *reinterpret_cast<const float4*>(from) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        w[0] = {make_float2(of[0].x, of[1].x), make_float2(of[2].x, of[3].x)};
        w[1] = {make_float2(of[0].y, of[1].y), make_float2(of[2].y, of[3].y)};
        w[2] = {make_float2(of[0].z, of[1].z), make_float2(of[2].z, of[3].z)};
        w[3] = {make_float2(of[0].w, of[1].w), make_float2(of[2].w, of[3].w)};
    }
    const int keys = d.key_heads * d.key_dim, kind = c < keys ? 0 : c < 2 * keys ? 1 : 2;
    const bool unit_norm = part * kInputCols + 4 * (threadIdx.x & ~31) < 2 * keys;
    uint16_t* const base = p.out[kind];
    const int64_t out_stride = p.out_stride[kind];
    const int64_t out_extent = 2 * ((p.rows - 1) * out_stride + (kind < 2 ? keys : d.heads * d.value_dim));
    uint16_t* to = base + (first + t0) * out_stride + c - kind * keys;  // of the next row finished
    // Four rows side by side: SiLU, unit norm, rounding (rows t .. t1 - 1).
    auto finish = [&](int t, Four (&y)[kAbreast]) {
#pragma unroll
        for (int i = 0; i < kAbreast; ++i) y[i] = {silu(y[i].a), silu(y[i].b)};
        if (unit_norm) {  // (some lane of the warp has a query's or key's channels)
            float sum[kAbreast];
#pragma unroll
            for (int i = 0; i < kAbreast; ++i)
                sum[i] = fmaf(y[i].a.x, y[i].a.x, fmaf(y[i].a.y, y[i].a.y, fmaf(y[i].b.x, y[i].b.x, y[i].b.y * y[i].b.y)));
            for (int o = p.key_lanes / 2; o > 0; o >>= 1)
#pragma unroll
                for (int i = 0; i < kAbreast; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
#pragma unroll
            for (int i = 0; i < kAbreast; ++i) {
                const float r = kind < 2 ? rsqrtf(sum[i] + p.eps) : 1.f;
                const float2 r2 = make_float2(r, r);
                y[i] = {fma2(y[i].a, r2, make_float2(-0.f, -0.f)), fma2(y[i].b, r2, make_float2(-0.f, -0.f))};
            }
        }
#pragma unroll
        for (int i = 0; i < kAbreast; ++i, to += out_stride)
            if (here && t + i < t1 && bc_global(bc, to, 8, base, out_extent, kBcDeltaQkv))
                *reinterpret_cast<uint2*>(to) = make_uint2(T::pack(y[i].a.x, y[i].a.y), T::pack(y[i].b.x, y[i].b.y));
    };
    auto past = [&](int t) { return t >= 0 ? input(first + t) : before(kConvTaps - 1 + t); };
    if (p.tree_mask == nullptr) {
        Four x0 = past(t0 - 3), x1 = past(t0 - 2), x2 = past(t0 - 1);
        Four new0 = zero, new1 = zero, new2 = zero;
        const bool moves = p.advance && t0 == 0;
        if (moves) {  // (the state's inputs are read before they are written)
            new0 = past(n - 3);
            new1 = past(n - 2);
            new2 = past(n - 1);
        }
        Four ahead[kAbreast];
        const float* from = p.x + (first + t0) * p.x_stride + c;
        auto ask = [&](int t) {
#pragma unroll
            for (int i = 0; i < kAbreast; ++i, from += p.x_stride)
                ahead[i] = here && t + i < t1 && bc_global(bc, from, 16, p.x, x_extent, kBcDeltaX)
                               ? as_four(*reinterpret_cast<const float4*>(from)) : zero;
        };
        ask(t0);
        for (int t = t0; t < t1; t += kAbreast) {
            Four y[kAbreast];
#pragma unroll
            for (int i = 0; i < kAbreast; ++i) {
                y[i] = zero;
                tap(y[i], w[0], x0);
                tap(y[i], w[1], x1);
                tap(y[i], w[2], x2);
                tap(y[i], w[3], ahead[i]);
                x0 = x1;
                x1 = x2;
                x2 = ahead[i];
            }
            ask(t + kAbreast);  // (the next rows' loads are in flight while these are finished)
            finish(t, y);
        }
        if (moves && here && bc_global(bc, at_conv + c, 16, d.conv, d.conv_extent, kBcDeltaConv) &&
            bc_global(bc, at_conv + 2 * (int64_t)d.channels + c, 16, d.conv, d.conv_extent, kBcDeltaConv)) {
            const Four moved[3] = {new0, new1, new2};
#pragma unroll
            for (int i = 0; i < 3; ++i)
                *reinterpret_cast<float4*>(at_conv + (int64_t)i * d.channels + c) =
                    make_float4(moved[i].a.x, moved[i].a.y, moved[i].b.x, moved[i].b.y);
        }
        return;
    }
    // The parent of row t (below 0: an input of the state's).
    auto parent = [&](int t) {
        if (t < 0) return t - 1;
        for (int i = min(p.mask_words - 1, t >> 6); i >= 0; --i) {
            const uint64_t* from = p.tree_mask + (int64_t)(first + t) * p.mask_words + i;
            uint64_t bits = bc_global(bc, from, 8, p.tree_mask, 8 * (int64_t)p.rows * p.mask_words, kBcDeltaMask) ? *from : 0;
            if (i == t >> 6) bits &= (1ull << (t & 63)) - 1;
            if (bits != 0) return 64 * i + 63 - __clzll(bits);
        }
        return -1;
    };
    for (int t = t0; t < t1; t += kAbreast) {
        Four y[kAbreast];
        int from[kAbreast];
#pragma unroll
        for (int i = 0; i < kAbreast; ++i) {
            from[i] = min(t + i, t1 - 1);
            y[i] = zero;
            tap(y[i], w[3], input(first + from[i]));
        }
#pragma unroll
        for (int j = 2; j >= 0; --j)
#pragma unroll
            for (int i = 0; i < kAbreast; ++i) {
                from[i] = parent(from[i]);
                tap(y[i], w[j], past(from[i]));
            }
        finish(t, y);
    }
}

}  // namespace

cudaError_t launch_delta_inputs(const iq4xs_delta_inputs_args& a, const DeltaView& d, const BatchView& b, int* err,
                                int num_sms, cudaStream_t stream) {
    InputParams p;
    p.x = a.x;
    p.weight = a.conv_weight;
    p.a = a.a;
    p.b = a.b;
    p.a_log = a.a_log;
    p.dt_bias = a.dt_bias;
    p.out[0] = static_cast<uint16_t*>(a.q);
    p.out[1] = static_cast<uint16_t*>(a.k);
    p.out[2] = static_cast<uint16_t*>(a.v);
    p.out_stride[0] = a.q_row_stride;
    p.out_stride[1] = a.k_row_stride;
    p.out_stride[2] = a.v_row_stride;
    p.g = a.g;
    p.beta = a.beta;
    p.tree_mask = a.tree_mask;
    p.x_stride = a.x_row_stride;
    p.a_stride = a.a_row_stride;
    p.b_stride = a.b_row_stride;
    p.conv_offset = a.layer * d.conv_layer_stride;
    p.eps = (float)a.eps;
    p.mask_words = (int)a.mask_words;
    p.advance = (int)a.advance;
    p.rows = (int)a.rows;
    p.key_lanes = d.key_dim / 4;
    p.col_parts = (d.channels + kInputCols - 1) / kInputCols + 1;
    // Rows of a run, at least the three that read the state's inputs: few while about
    // all CTAs are resident at once, for a CTA's rows come one behind the other (48
    // heads, runs of 4, 8 and 16: 96 rows 5.4, 5.8 and 7.5 us, 300 8.2, 7.1 and 8.8, 1,000
    // 19.9, 15.2 and 14.1); 32 where SMs keep several rounds all the same, for runs look
    // their sequence up and read three rows again (of 16 and 32: 2,048 rows 27.1 and 28.4,
    // 4,000 48.4 and 46.1, 6,147 71.2 and 69.7; of 64 71.4).
    p.run = kLeastRun;
    while (p.run < kShortRun && a.rows * p.col_parts > (int64_t)p.run * 7 * num_sms) p.run *= 2;
    if (a.rows * p.col_parts >= (int64_t)kLongRun * 16 * num_sms) p.run = kLongRun;
    const int64_t blocks = (a.rows / p.run + b.sequences) * p.col_parts;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks);
    return a.dtype == IQ4XS_KV_BF16
               ? launch_chained(delta_inputs_kernel<KvBf16>, grid, dim3(kInputThreads), 0, stream, 1, p, d, b, err)
               : launch_chained(delta_inputs_kernel<KvF16>, grid, dim3(kInputThreads), 0, stream, 1, p, d, b, err);
}

}  // namespace iq4xs
