// delta_chunk.cu -- the gated delta rule over many rows a sequence (prompt
// chunks, wide drafted trees) on tcgen05: blocks of 64 rows.
//
// With S the state before a block, k_t and q_t its rows, F_tj the decay from j to
// t and G_t from the block's start, the rule over the block is (u, r rows of DV)
//
//   r_t = beta_t (v_t - G_t S^T k_t)                     products 1: S with [K; Q]
//   u = T r,  T = (1 + A)^-1,  A_tj = beta_t F_tj k_t.k_j  (j before t)   product 2
//   o_t = scale (G_t S^T q_t + sum_j F_tj (q_t.k_j) u_j)   product 3a: U with P
//   S <- G S + sum_j k_j (F_nj u_j)^T                      product 3b: U F with K
//
// A CTA takes a head of a sequence.  A lane of tensor memory is a value channel:
// S, r and u are the products' left operands, written there by the two threads of
// the lane, who keep S in registers; [K; Q], T and P are the right ones, in shared
// memory.  Four more warps prepare the next block meanwhile: K and Q in shared
// memory, their products [K; Q] K^T, decays (by walking back from every row, so
// that no difference of long sums enters), A, T by forward substitution in halves,
// and P.
//
// Precision.  The products take fp16.  K and Q of 16 bits are exact (bf16 rows
// times a power of two; what is 2^-38 below a row's largest is cut), all else goes
// in two parts, a value and its remainder, 22 bits, with a power of two for each
// row that brings its largest to 2^13: one part would be the largest error of the
// result.  Every product starts from zero and joins fp32 registers by rounded
// arithmetic (the tensor core cuts its sums off).
//
// A row that holds NaN or infinities (or meets them in S) gives zeros to the
// products and is marked; u and o of rows that come from it are made NaN after them.
#include "attention.cuh"
#include "delta.cuh"

namespace iq4xs {
namespace {

constexpr int kRows = kDeltaTreeRows;  // of a block
constexpr int kMainWarps = 8, kPrepWarps = 4;
constexpr int kMainThreads = 32 * kMainWarps, kPrepThreads = 32 * kPrepWarps;
constexpr int kChunkThreads = kMainThreads + kPrepThreads;
constexpr int kPitch = kRows + 4;      // of A and T in fp32
static_assert(kRows == 64, "a row of T or P is one swizzle row; the halves of the substitution are 32");

// What a block's rows say, one set a buffer.
struct Gates {
    float beta[kRows];
    float gk[kRows];    // G_t, less the scale of k_t
    float gq[kRows];    // scale G_t, less that of q_t
    float left[kRows];  // F_nj, less the scale of k_j
    float ct[kRows];    // what the rows of T and P were divided by
    float cp[kRows];
    unsigned long long seen[kRows];
    unsigned long long odd;  // rows whose k or gates are not finite
    float decay;             // G_n
    int pad;
};

template <int DK, int DV>
struct ChunkShape {
    static constexpr int kKqBytes = 2 * kRows * DK * 2;   // K rows, then Q rows; chunks of 64 channels
    static constexpr int kPartBytes = kRows * kRows * 2;  // T or P, one part
    static constexpr int kVBytes = kRows * DV * 2;
    static constexpr int kKq = 0;
    static constexpr int kT = kKq + 2 * kKqBytes;         // [buffer][hi, lo]
    static constexpr int kP = kT + 4 * kPartBytes;
    static constexpr int kV = kP + 4 * kPartBytes;
    static constexpr int kA = kV + 2 * kVBytes;           // fp32
    static constexpr int kTs = kA + kRows * kPitch * 4;
    static constexpr int kX = kTs + kRows * kPitch * 4;   // [32][32]
    static constexpr int kGates = kX + 32 * 32 * 4;
    static constexpr int kTops = kGates + 2 * (int)sizeof(Gates);  // [S, r, u, u F][share][128] largest
    static constexpr int kOdd = kTops + 4 * 2 * 128 * 4;           // [r, u][share][128] rows not finite
    static constexpr int kScales = kOdd + 2 * 2 * 128 * 4;         // [128] of K's and Q's rows; then their g
    static constexpr int kBars = kScales + 2 * kRows * 4 + kRows * 4;
    static constexpr int kMisc = kBars + 16 * 8;
    static constexpr int kSmem = kMisc + 16;
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(sizeof(Gates) % 16 == 0 && kGates % 16 == 0 && kBars % 8 == 0 && kKqBytes % 1024 == 0, "alignment");
    // tensor memory columns: S's parts, then those of u and u F; S^T [K; Q], u and
    // o in turn; r's parts; the state's part; [K; Q] K^T of the next block
    static constexpr int kParts = 0, kD = 128, kR = 256, kNew = 320, kPairs = 448;
    static_assert(kPairs + kRows <= 512 && DK <= 128, "tensor memory");
    static constexpr int kHalf = DK / 2;   // key channels a thread
    static constexpr int kQuads = DV / 32; // quadrants with value channels
};

__device__ __forceinline__ void pair_sync(int quad) { asm volatile("bar.sync %0, 64;" ::"r"(quad + 1) : "memory"); }
__device__ __forceinline__ void main_sync() { asm volatile("bar.sync 5, %0;" ::"n"(kMainThreads) : "memory"); }
__device__ __forceinline__ void prep_sync() { asm volatile("bar.sync 6, %0;" ::"n"(kPrepThreads) : "memory"); }
// Whether x holds for any of the threads: one answer for all of them.
template <int kBar, int kThreads>
__device__ __forceinline__ bool any_of(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "n"(kBar), "n"(kThreads)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {  // the rest of 16: zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// A power of two that brings `top` to 2^13 .. 2^14, and its inverse; 1 where it is 0 or not finite.
__device__ __forceinline__ float2 fit(float top) {
    const int e = (int)(__float_as_uint(top) >> 23);
    if (e == 255 || top == 0.f) return make_float2(1.f, 1.f);
    const int f = min(252, 267 - e);
    return make_float2(__uint_as_float((uint32_t)f << 23), __uint_as_float((uint32_t)(254 - f) << 23));
}
// Two values as two fp16 parts.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = KvF16::pack(a, b);
    const float2 r = KvF16::unpack(hi);
    lo = KvF16::pack(a - r.x, b - r.y);
}
__device__ __forceinline__ bool odd_value(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }

template <int DK, int DV>
__global__ void __launch_bounds__(kChunkThreads, 1) delta_chunk_kernel(const __grid_constant__ DeltaRule p,
                                                                       const __grid_constant__ DeltaView d,
                                                                       const __grid_constant__ BatchView b, int* err) {
    using C = ChunkShape<DK, DV>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    if ((base & 1023) != 0) {  // (no static shared memory: the swizzle atoms' alignment)
        if (threadIdx.x == 0) atomicCAS(err, 0, kDevErrLayout);
        return;
    }
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBars);  // [2] a block is prepared
    uint64_t* empty = full + 2;                                     // [2] and used
    uint64_t* done1 = empty + 2;
    uint64_t* done2 = done1 + 1;
    uint64_t* done_s = done2 + 1;
    uint64_t* done_o = done_s + 1;
    uint64_t* done_pairs = done_o + 1;
    uint64_t* drained = done_pairs + 1;  // [2]
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_at + 1);
    Gates* gates = reinterpret_cast<Gates*>(smem + C::kGates);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_launch_dependents();
    griddep_wait();
    const Bc bc = bc_open(err);
    const int head = blockIdx.x % d.heads, s = blockIdx.x / d.heads;
    int row0;
    const int n = batch_rows(b, s, p.rows, &row0, err);
    const int len = batch_len(b, s, err), slot = delta_slot(d, s, err);
    if (n == 0 || len < 0 || slot < 0) return;
    if (n > p.max_rows) {
        if (tid == 0) data_error(err, kDataCount);
        return;
    }
    const bool keep = p.u != nullptr;
    const int blocks = (n + kRows - 1) / kRows;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(full + i, kPrepThreads);
            mbar_init(empty + i, kMainWarps);
            mbar_init(drained + i, 1);
        }
        mbar_init(done1, 1);
        mbar_init(done2, 1);
        mbar_init(done_s, 1);
        mbar_init(done_o, 1);
        mbar_init(done_pairs, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0) tmem_alloc(tmem_at, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_at);
    const int key_head = head / (d.heads / d.key_heads);
    const int64_t keys = (int64_t)d.key_heads * DK, values = (int64_t)d.heads * DV;

    if (warp >= kMainWarps) {
        // ------------------------------------------------ the next block's operands
        const int id = tid - kMainThreads;
        constexpr int kUnits = DK / 8, kDown = kPrepThreads / kUnits, kTimes = 2 * kRows / kDown;
        const int unit = id % kUnits;
        float* const scales = reinterpret_cast<float*>(smem + C::kScales);  // what K's and Q's rows are to be divided by
        float* const g_at = scales + 2 * kRows;
        float* const A = reinterpret_cast<float*>(smem + C::kA);
        float* const Ts = reinterpret_cast<float*>(smem + C::kTs);
        float* const X = reinterpret_cast<float*>(smem + C::kX);
        uint4 raw[kTimes];
        auto load = [&](int t0) {
#pragma unroll
            for (int i = 0; i < kTimes; ++i) {
                const int r = id / kUnits + i * kDown, t = r % kRows;
                const uint16_t* from = r < kRows ? p.k : p.q;
                const int64_t stride = r < kRows ? p.k_row_stride : p.q_row_stride;
                const uint16_t* at = from + (row0 + t0 + t) * stride + key_head * DK + 8 * unit;
                raw[i] = make_uint4(0, 0, 0, 0);
                if (t0 + t < n && bc_global(bc, at, 16, from, 2 * ((p.rows - 1) * stride + keys), kBcDeltaQkv))
                    raw[i] = *reinterpret_cast<const uint4*>(at);
            }
        };
        load(0);
        for (int c = 0; c < blocks; ++c) {
            const int buf = c & 1, t0 = c * kRows, m = min(kRows, n - t0);
            Gates& gt = gates[buf];
            bool lost = c >= 2 && !kv_wait(empty + buf, (c / 2 - 1) & 1, abort_flag, err, kDevErrTimeoutDelta);
            if (any_of<6, kPrepThreads>(lost)) break;  // (all leave together)
            // V as it lies
            for (int i = id; i < kRows * (DV / 8); i += kPrepThreads) {
                const int t = i / (DV / 8), u = i % (DV / 8);
                const uint16_t* at = p.v + (row0 + t0 + min(t, m - 1)) * p.v_row_stride + head * DV + 8 * u;
                const bool in = t < m && bc_global(bc, at, 16, p.v, 2 * ((p.rows - 1) * p.v_row_stride + values), kBcDeltaQkv);
                cp_async16(base + C::kV + buf * C::kVBytes + (t * DV + 8 * u) * 2, at, in ? 16 : 0);
            }
            if (id == 0) gt.odd = 0;
            prep_sync();
            if (id < kRows) {
                const int64_t at = (int64_t)(row0 + t0 + id) * d.heads + head, extent = 4 * (int64_t)p.rows * d.heads;
                float g = 0.f, beta = 0.f;
                uint64_t seen = 0;
                if (id < m) {
                    if (bc_global(bc, p.g + at, 4, p.g, extent, kBcDeltaGate)) g = p.g[at];
                    if (bc_global(bc, p.beta + at, 4, p.beta, extent, kBcDeltaGate)) beta = p.beta[at];
                    seen = delta_seen(p.tree_mask, p.mask_words, p.rows, row0, id, bc);
                    if (odd_value(beta) || isnan(g) || g == INFINITY) {
                        g = beta = 0.f;
                        atomicOr(&gt.odd, 1ull << id);
                    }
                }
                g_at[id] = g;
                gt.beta[id] = beta;
                gt.seen[id] = seen;
                gt.left[id] = 0.f;
            }
            // K and Q: fp16 as it is, bf16 with its row's largest at 2^13; a row of K that is not finite: zeros
#pragma unroll
            for (int i = 0; i < kTimes; ++i) {
                const int r = id / kUnits + i * kDown;
                uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                const uint32_t exp = p.bf16 ? 0x7f80u : 0x7c00u;
                bool odd = false;
#pragma unroll
                for (int e = 0; e < 4; ++e) odd |= (w[e] & exp) == exp || (w[e] >> 16 & exp) == exp;
                const unsigned odd_lanes = __ballot_sync(0xffffffffu, odd) >> (lane / kUnits * kUnits) &
                                           (kUnits == 32 ? 0xffffffffu : (1u << kUnits) - 1);
                float inverse = 1.f;
                if (p.bf16) {
                    float x[8], top = 0.f;
                    unpack8<KvBf16>(raw[i], x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
#pragma unroll
                    for (int o = kUnits / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    const float2 f = fit(top);
                    inverse = f.y;
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = KvF16::pack(x[2 * e] * f.x, x[2 * e + 1] * f.x);
                }
                if (odd_lanes != 0 && r < kRows) {
                    w[0] = w[1] = w[2] = w[3] = 0;
                    if (unit == 0) atomicOr(&gt.odd, 1ull << r);
                }
                sts_u128(base + C::kKq + buf * C::kKqBytes + unit_at(r, unit, 2 * kRows), make_uint4(w[0], w[1], w[2], w[3]));
                if (unit == 0) scales[r] = inverse;
            }
            fence_proxy_async_smem();
            prep_sync();
            if (id == 0) {
                tc_fence_after();
                const uint64_t kq = desc_sw128(base + C::kKq + buf * C::kKqBytes, 16, 1024);
#pragma unroll
                for (int k = 0; k < DK / 16; ++k) {
                    const uint64_t at = kq + (((k / 4) * 2 * kRows * kChunkBytes + (k % 4) * 32) >> 4);
                    tc_mma_f16(tmem + C::kPairs, at, at, idesc_kv(kRows, 0, false), k > 0);
                }
                tc_commit(done_pairs);
            }
            if (c + 1 < blocks) load(t0 + kRows);
            // Row t of the pairs: A from the rows of K, P from those of Q.
            const int t = id % kRows;
            const bool is_q = id >= kRows;
            lost = !kv_wait(done_pairs, c & 1, abort_flag, err, kDevErrTimeoutDelta);
            tc_fence_after();
            {
                uint32_t x[kRows];
                const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + C::kPairs;
                tmem_ld32_wait(at, x);
                tmem_ld32_wait(at + 32, x + 32);
                const uint64_t seen = gt.seen[t];
                const float mine = scales[id];
                const float factor = (is_q ? p.scale : gt.beta[t]) * mine;
                float sum = 0.f, before = g_at[t], top = 0.f;
#pragma unroll
                for (int j = kRows - 1; j >= 0; --j) {
                    const bool from = seen >> j & 1, self = j == t;
                    if (from) {
                        sum += before;
                        before = g_at[j];
                    }
                    const float far = self ? 1.f : expf(sum);
                    const float scaled = far * scales[j];
                    const float y = from || (self && is_q) ? __uint_as_float(x[j]) * (factor * scaled) : 0.f;
                    x[j] = __float_as_uint(y);
                    top = fmaxf(top, fabsf(y));
                    if (!is_q && t == m - 1 && (from || self)) gt.left[j] = scaled;
                }
                const float all = expf(sum + before);  // from the block's start
                if (is_q) {
                    gt.gq[t] = p.scale * all * mine;
                    const float2 f = fit(top);
                    gt.cp[t] = f.y;
                    const uint32_t to = base + C::kP + buf * 2 * C::kPartBytes;
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            split2(__uint_as_float(x[8 * u + 2 * e]) * f.x, __uint_as_float(x[8 * u + 2 * e + 1]) * f.x, hi[e], lo[e]);
                        sts_u128(to + unit_at(t, u, kRows), make_uint4(hi[0], hi[1], hi[2], hi[3]));
                        sts_u128(to + C::kPartBytes + unit_at(t, u, kRows), make_uint4(lo[0], lo[1], lo[2], lo[3]));
                    }
                } else {
                    gt.gk[t] = all * mine;
                    if (t == m - 1) gt.decay = all;
#pragma unroll
                    for (int j = 0; j < kRows; j += 4)
                        *reinterpret_cast<uint4*>(A + t * kPitch + j) = make_uint4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                }
            }
            tc_fence_before();
            prep_sync();
            // T's diagonal halves, a column a thread.
            if (id < kRows) {
                const float* a = A + (id & 32) * (kPitch + 1);
                float x[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float y[4] = {i == lane ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < i; j += 4) {
                        const float4 w = *reinterpret_cast<const float4*>(a + i * kPitch + j);
                        y[0] = fmaf(-w.x, x[j], y[0]);
                        if (j + 1 < i) y[1] = fmaf(-w.y, x[j + 1], y[1]);
                        if (j + 2 < i) y[2] = fmaf(-w.z, x[j + 2], y[2]);
                        if (j + 3 < i) y[3] = fmaf(-w.w, x[j + 3], y[3]);
                    }
                    x[i] = (y[0] + y[1]) + (y[2] + y[3]);
                    Ts[((id & 32) + i) * kPitch + id] = x[i];
                }
            }
            prep_sync();
            // The half below: -T22 (A21 T11), eight rows of a column a thread.
            auto product = [&](const float* left, int pitch, const float* right, int right_pitch, float (&y)[8]) {
                float x[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) x[j] = right[j * right_pitch + lane];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 w = *reinterpret_cast<const float4*>(left + i * pitch + j);
                        z[0] = fmaf(w.x, x[j], z[0]);
                        z[1] = fmaf(w.y, x[j + 1], z[1]);
                        z[2] = fmaf(w.z, x[j + 2], z[2]);
                        z[3] = fmaf(w.w, x[j + 3], z[3]);
                    }
                    y[i] = (z[0] + z[1]) + (z[2] + z[3]);
                }
            };
            const int r8 = 8 * (warp - kMainWarps);
            if (m > 32) {  // (else the half below is of empty rows)
                float y[8];
                product(A + (32 + r8) * kPitch, kPitch, Ts, kPitch, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) X[(r8 + i) * 32 + lane] = y[i];
                prep_sync();
                product(Ts + (32 + r8) * kPitch + 32, kPitch, X, 32, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) Ts[(32 + r8 + i) * kPitch + lane] = -y[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) Ts[(32 + r8 + i) * kPitch + lane] = 0.f;
            }
            prep_sync();
            {
                const int row = id / 2, half = id % 2;
                const bool zero = row < 32 && half == 1;
                float x[32], top = 0.f;
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 w = zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                                          : *reinterpret_cast<const float4*>(Ts + row * kPitch + 32 * half + j);
                    x[j] = w.x; x[j + 1] = w.y; x[j + 2] = w.z; x[j + 3] = w.w;
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) top = fmaxf(top, fabsf(x[j]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                const float2 f = fit(top);
                if (half == 0) gt.ct[row] = f.y;
                const uint32_t to = base + C::kT + buf * 2 * C::kPartBytes;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) split2(x[8 * u + 2 * e] * f.x, x[8 * u + 2 * e + 1] * f.x, hi[e], lo[e]);
                    sts_u128(to + unit_at(row, 4 * half + u, kRows), make_uint4(hi[0], hi[1], hi[2], hi[3]));
                    sts_u128(to + C::kPartBytes + unit_at(row, 4 * half + u, kRows), make_uint4(lo[0], lo[1], lo[2], lo[3]));
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            if (any_of<6, kPrepThreads>(lost)) break;
            mbar_arrive(full + buf);
        }
        // Tensor memory is given back only when every product is done.
        if (*abort_flag && id == 0) {
            tc_commit(drained + 1);
            int no_abort = 0;
            kv_wait(drained + 1, 0, &no_abort, err, kDevErrTimeoutDelta);
        }
    } else {
        // ------------------------------------------------------------ the blocks
        const int quad = warp & 3, share = warp >> 2, at_lane = quad * 32 + lane;
        const bool busy = quad < C::kQuads;  // the warp has value channels
        const uint32_t lane_at = tmem + ((uint32_t)(quad * 32) << 16);
        float* const tops = reinterpret_cast<float*>(smem + C::kTops);
        uint32_t* const odds = reinterpret_cast<uint32_t*>(smem + C::kOdd);
        float* const at_s = d.s + p.s_offset + slot * d.s_slot_stride + ((int64_t)head * DK + share * C::kHalf) * DV + at_lane;
        auto largest = [&](int what, float mine) {  // of the lane's two threads, behind a pair_sync
            tops[(what * 2 + share) * 128 + at_lane] = mine;
        };
        auto largest_of = [&](int what) { return fmaxf(tops[what * 256 + at_lane], tops[what * 256 + 128 + at_lane]); };
        float S[C::kHalf];
#pragma unroll
        for (int i = 0; i < C::kHalf; ++i) {
            const float* from = at_s + i * DV;
            S[i] = busy && len > 0 && bc_global(bc, from, 4, d.s, d.s_extent, kBcDeltaS) ? *from : 0.f;
        }
        float inverse_s = 1.f;
        // S into its parts.
        auto put_state = [&] {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < C::kHalf; ++i) top = fmaxf(top, fabsf(S[i]));
            largest(0, top);
            pair_sync(quad);
            const float2 f = fit(largest_of(0));
            inverse_s = f.y;
#pragma unroll
            for (int i = 0; i < C::kHalf; i += 32) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) split2(S[i + 2 * e] * f.x, S[i + 2 * e + 1] * f.x, hi[e], lo[e]);
                tmem_st16(lane_at + C::kParts + (share * C::kHalf + i) / 2, hi);
                tmem_st16(lane_at + C::kParts + DK / 2 + (share * C::kHalf + i) / 2, lo);
            }
            tmem_wait_st();
        };
        if (busy) put_state();
        bool lost = false;
        float o[32];
        int o_rows = 0;          // rows of `o` on their way out
        int64_t o_first = 0;
        auto put_rows = [&] {
            if (!busy) return;
            float* to = p.out + o_first * p.out_row_stride + head * DV + at_lane;
#pragma unroll
            for (int i = 0; i < 32; ++i, to += p.out_row_stride)
                if (i < o_rows && bc_global(bc, to, 4, p.out, 4 * ((p.rows - 1) * p.out_row_stride + values), kBcDeltaOut))
                    *to = o[i];
        };
        for (int c = 0; c < blocks; ++c) {
            const int buf = c & 1, t0 = c * kRows, m = min(kRows, n - t0);
            const Gates& gt = gates[buf];
            lost |= !kv_wait(full + buf, (c / 2) & 1, abort_flag, err, kDevErrTimeoutDelta);
            tc_fence_before();
            if (any_of<5, kMainThreads>(lost)) break;
            const uint64_t kq = desc_sw128(base + C::kKq + buf * C::kKqBytes, 16, 1024);
            const uint64_t td = desc_sw128(base + C::kT + buf * 2 * C::kPartBytes, 16, 1024);
            const uint64_t pd = desc_sw128(base + C::kP + buf * 2 * C::kPartBytes, 16, 1024);
            if (tid == 0) {
                tc_fence_after();
#pragma unroll
                for (int part = 1; part >= 0; --part)  // the smaller parts first
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k)
                        tc_mma_f16_ta(tmem + C::kD, tmem + C::kParts + part * DK / 2 + 8 * k,
                                      kq + (((k / 4) * 2 * kRows * kChunkBytes + (k % 4) * 32) >> 4),
                                      idesc_kv(2 * kRows, 0, false), part == 0 || k > 0);
                tc_commit(done1);
            }
            put_rows();  // (the last block's)
            const int first = 32 * share;  // the thread's rows of the block
            lost |= !kv_wait(done1, c & 1, abort_flag, err, kDevErrTimeoutDelta);
            float inverse_r = 1.f;
            uint64_t odd = gt.odd;
            if (busy) {
                tc_fence_after();
                uint32_t x[32];
                tmem_ld32_wait(lane_at + C::kD + first, x);
                const uint16_t* v = reinterpret_cast<const uint16_t*>(smem + C::kV + buf * C::kVBytes) + first * DV + at_lane;
                float top = 0.f;
                uint32_t bits = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const uint32_t raw = v[i * DV];
                    const float value = p.bf16 ? __uint_as_float(raw << 16) : KvF16::unpack(raw).x;
                    const float y = gt.beta[first + i] * (value - gt.gk[first + i] * (inverse_s * __uint_as_float(x[i])));
                    if (odd_value(y)) bits |= 1u << i;
                    x[i] = odd_value(y) ? 0 : __float_as_uint(y);
                    top = fmaxf(top, fabsf(__uint_as_float(x[i])));
                }
                largest(1, top);
                odds[share * 128 + at_lane] = bits;
                pair_sync(quad);
                odd |= (uint64_t)odds[128 + at_lane] << 32 | odds[at_lane];
                const float2 f = fit(largest_of(1));
                inverse_r = f.y;
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    split2(__uint_as_float(x[2 * e]) * f.x, __uint_as_float(x[2 * e + 1]) * f.x, hi[e], lo[e]);
                tmem_st16(lane_at + C::kR + first / 2, hi);
                tmem_st16(lane_at + C::kR + kRows / 2 + first / 2, lo);
                tmem_wait_st();
            }
            tc_fence_before();
            main_sync();
            if (tid == 0) {
                tc_fence_after();
                constexpr uint32_t kId = idesc_kv(kRows, 0, false);
#pragma unroll
                for (int pass = 0; pass < 3; ++pass)  // remainder by value, value by remainder, value by value
#pragma unroll
                    for (int k = 0; k < kRows / 16; ++k)
                        tc_mma_f16_ta(tmem + C::kD, tmem + C::kR + (pass == 0 ? kRows / 2 : 0) + 8 * k,
                                      td + (((pass == 1 ? C::kPartBytes : 0) + k * 32) >> 4), kId, pass > 0 || k > 0);
                tc_commit(done2);
            }
            lost |= !kv_wait(done2, c & 1, abort_flag, err, kDevErrTimeoutDelta);
            float inverse_u = 1.f, inverse_f = 1.f;
            if (busy) {
                tc_fence_after();
                uint32_t x[32];
                tmem_ld32_wait(lane_at + C::kD + first, x);
                float top = 0.f, top_f = 0.f;
                uint32_t bits = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float y = __uint_as_float(x[i]) * inverse_r * gt.ct[first + i];
                    if (odd_value(y)) bits |= 1u << i;
                    x[i] = odd_value(y) ? 0 : __float_as_uint(y);
                }
                odds[256 + share * 128 + at_lane] = bits;
                if (odd != 0) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if ((gt.seen[first + i] | 1ull << (first + i)) & odd) {
                            bits |= 1u << i;
                            x[i] = 0;
                        }
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    top = fmaxf(top, fabsf(__uint_as_float(x[i])));
                    top_f = fmaxf(top_f, fabsf(__uint_as_float(x[i]) * gt.left[first + i]));
                }
                if (keep) {
                    float* to = p.u + ((int64_t)(row0 + t0 + first) * d.heads + head) * DV + at_lane;
#pragma unroll
                    for (int i = 0; i < 32; ++i, to += values)
                        if (first + i < m && bc_global(bc, to, 4, p.u, 4 * p.rows * values, kBcDeltaU))
                            *to = bits >> i & 1 ? NAN : __uint_as_float(x[i]);
                }
                largest(2, top);
                largest(3, top_f);
                pair_sync(quad);
                odd |= (uint64_t)odds[256 + 128 + at_lane] << 32 | odds[256 + at_lane];
                const float2 f = fit(largest_of(2)), ff = fit(largest_of(3));
                inverse_u = f.y;
                inverse_f = ff.y;
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    split2(__uint_as_float(x[2 * e]) * f.x, __uint_as_float(x[2 * e + 1]) * f.x, hi[e], lo[e]);
                tmem_st16(lane_at + C::kParts + first / 2, hi);
                tmem_st16(lane_at + C::kParts + kRows / 2 + first / 2, lo);
                if (!keep) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        split2(__uint_as_float(x[2 * e]) * gt.left[first + 2 * e] * ff.x,
                               __uint_as_float(x[2 * e + 1]) * gt.left[first + 2 * e + 1] * ff.x, hi[e], lo[e]);
                    tmem_st16(lane_at + C::kParts + kRows + first / 2, hi);
                    tmem_st16(lane_at + C::kParts + kRows + kRows / 2 + first / 2, lo);
                }
                tmem_wait_st();
            }
            tc_fence_before();
            main_sync();
            if (tid == 0) {
                tc_fence_after();
                if (!keep) {
                    const uint64_t kn = desc_sw128(base + C::kKq + buf * C::kKqBytes, 2 * kRows * kChunkBytes, 1024);
#pragma unroll
                    for (int part = 1; part >= 0; --part)
#pragma unroll
                        for (int k = 0; k < kRows / 16; ++k)
                            tc_mma_f16_ta(tmem + C::kNew, tmem + C::kParts + kRows + part * kRows / 2 + 8 * k,
                                          kn + ((k * 16 * kChunkBytes) >> 4), idesc_kv(DK, 0, true), part == 0 || k > 0);
                    tc_commit(done_s);
                }
                constexpr uint32_t kId = idesc_kv(kRows, 0, false);
#pragma unroll
                for (int pass = 0; pass < 3; ++pass)
#pragma unroll
                    for (int k = 0; k < kRows / 16; ++k)
                        tc_mma_f16_ta(tmem + C::kD, tmem + C::kParts + (pass == 0 ? kRows / 2 : 0) + 8 * k,
                                      pd + (((pass == 1 ? C::kPartBytes : 0) + k * 32) >> 4), kId, pass > 0 || k > 0);
                tc_commit(done_o);
            }
            if (!keep) {
                lost |= !kv_wait(done_s, c & 1, abort_flag, err, kDevErrTimeoutDelta);
                if (busy) {
                    tc_fence_after();
                    const float decay = gt.decay;
#pragma unroll
                    for (int i = 0; i < C::kHalf; i += 32) {
                        uint32_t x[32];
                        tmem_ld32_wait(lane_at + C::kNew + share * C::kHalf + i, x);
#pragma unroll
                        for (int e = 0; e < 32; ++e) S[i + e] = fmaf(decay, S[i + e], inverse_f * __uint_as_float(x[e]));
                    }
                    if (odd != 0) {
#pragma unroll
                        for (int i = 0; i < C::kHalf; ++i) S[i] = NAN;
                    }
                }
            }
            lost |= !kv_wait(done_o, c & 1, abort_flag, err, kDevErrTimeoutDelta);
            if (busy) {
                tc_fence_after();
                uint32_t x[32], y[32];
                tmem_ld32_wait(lane_at + C::kD + first, x);
                tmem_ld32_wait(lane_at + C::kD + kRows + first, y);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    o[i] = fmaf(gt.gq[first + i] * inverse_s, __uint_as_float(y[i]),
                                gt.cp[first + i] * inverse_u * __uint_as_float(x[i]));
                if (odd != 0) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if ((gt.seen[first + i] | 1ull << (first + i)) & odd) o[i] = NAN;
                }
                o_rows = m - first;
                o_first = row0 + t0 + first;
                if (c + 1 < blocks) put_state();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + buf);
        }
        put_rows();
        if (!keep && busy && !lost) {
#pragma unroll
            for (int i = 0; i < C::kHalf; ++i)
                if (bc_global(bc, at_s + i * DV, 4, d.s, d.s_extent, kBcDeltaS)) at_s[i * DV] = S[i];
        }
        if (*abort_flag && tid == 0) {
            tc_commit(drained);
            int no_abort = 0;
            kv_wait(drained, 0, &no_abort, err, kDevErrTimeoutDelta);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int DK, int DV>
cudaError_t launch_chunk(const DeltaRule& p, const DeltaView& d, const BatchView& b, int* err, cudaStream_t stream) {
    using C = ChunkShape<DK, DV>;
    const cudaError_t e = allow_smem<delta_chunk_kernel<DK, DV>>(C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_chained(delta_chunk_kernel<DK, DV>, dim3((unsigned)((int64_t)b.sequences * d.heads)), dim3(kChunkThreads),
                          C::kSmem, stream, 1, p, d, b, err);
}

}  // namespace

cudaError_t launch_delta_chunk(const DeltaRule& p, const DeltaView& d, const BatchView& b, int* err, cudaStream_t stream) {
    if (d.key_dim == 64) return d.value_dim == 64 ? launch_chunk<64, 64>(p, d, b, err, stream) : launch_chunk<64, 128>(p, d, b, err, stream);
    return d.value_dim == 64 ? launch_chunk<128, 64>(p, d, b, err, stream) : launch_chunk<128, 128>(p, d, b, err, stream);
}

}  // namespace iq4xs
