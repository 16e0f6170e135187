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
// memory.  Eight more warps prepare the next block meanwhile: K and Q in shared
// memory, their products [K; Q] K^T, decays (by walking back from every row, so
// that no difference of long sums enters), A and P; T's diagonal blocks of 16 by
// substitution, what is below them, -T22 A21 T11, by the warp-level MMA on tf32, three
// terms of two parts (with decays from a scan and rows asked into L2: 231 to 210 us).
//
// Measured: 6,147 rows of 3 sequences, 48 heads of 128 x 128: 212 us, floor of the bytes
// 44; 144 CTAs, 33 blocks of 12,300 cycles in a row, the first behind 8 us.  What bounds
// it is that chain: preparing a block takes 11,300 cycles (copies landing 1,000,
// conversion 2,900, the pairs' product 1,900, decays 1,600, substitution 1,500, the rest
// of T 3,700), the block itself 10,500 (S^T [K; Q] and the last block's out 2,400, r
// 2,000, u 3,600, S 2,500), the tensor core busy 20 % of the time.  Tried: copies issued by
// other warps and as soon as the block lets go of K, Q and V (medians of a CTA 196 us
// instead of 198, but the slowest 203 to 233 instead of 201: 213 to 230 in all); polling
// instead of sleeping waits (216); the gates under the pairs' product, three sums for T's
// terms, the last two products issued by two warps (no difference).
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
// So is a row whose A or T passes fp32's range (keys of norms whose product is 2^127):
// T is then made again, column by column over the rows that come from one another
// alone, for 0 times infinity in a row of another branch is NaN.
#include <type_traits>

#include "attention.cuh"
#include "delta.cuh"

namespace iq4xs {
namespace {

constexpr int kRows = kDeltaTreeRows;  // of a block
constexpr int kMainWarps = 8, kPrepWarps = 8;
constexpr int kMainThreads = 32 * kMainWarps, kPrepThreads = 32 * kPrepWarps;
constexpr int kChunkThreads = kMainThreads + kPrepThreads;
constexpr int kPitch = kRows + 4;      // of A and T in fp32
// The main warps keep S; the others give up registers (the sum is the launch's).
constexpr int kMainRegs = 168, kPrepRegs = 88;
static_assert(kMainWarps * kMainRegs + kPrepWarps * kPrepRegs <= (kMainWarps + kPrepWarps) * 128, "register split");
static_assert(kRows == 64, "a row of T or P is one swizzle row; the halves of the substitution are 32");

// What a block's rows say, one set a buffer.
struct __align__(16) Gates {
    float beta[kRows];
    float bg[kRows];    // -beta G_t, less the scale of k_t
    float gq[kRows];    // scale G_t, less that of q_t
    float left[kRows];  // F_nj, less the scale of k_j
    float ct[kRows];    // what the rows of T and P are to be multiplied by
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
    static constexpr int kA = kV + 2 * kVBytes;           // A and P in fp32
    static constexpr int kTs = kA + 2 * kRows * kPitch * 4;
    static constexpr int kGates = kTs + kRows * kPitch * 4;
    static constexpr int kTops = kGates + 2 * (int)sizeof(Gates);  // [S, r, u, u F][share][128] largest
    static constexpr int kOdd = kTops + 4 * 2 * 128 * 4;           // [r, u][share][128] rows not finite
    static constexpr int kScales = kOdd + 2 * 2 * 128 * 4;         // [128] of K's and Q's rows; their g and beta; P's largest; g summed up
    static constexpr int kSeen = kScales + 7 * kRows * 4;           // [64] 64-bit, and the rows that are not finite
    static constexpr int kBars = kSeen + kRows * 8 + 8;
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
__device__ __forceinline__ void prefetch_2d(const void* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
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
// Two bf16 values times a power of two (twice, side by side) in fp16.
__device__ __forceinline__ uint32_t scaled16(uint32_t w, uint32_t f) {
    uint32_t y;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(w), "r"(f), "r"(0x80008000u));
    const float2 x = KvBf16::unpack(y);
    return KvF16::pack(x.x, x.y);
}
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("max.u16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
__device__ __forceinline__ uint4 lds_u128(uint32_t at) {
    uint4 w;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at) : "memory");
    return w;
}
// Products issued by a whole warp, of which one lane (`one`) counts: descriptors
// and columns then stay in uniform registers.
__device__ __forceinline__ void mma_ta(bool one, uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 q, %0, 0;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], %3, %4, p;\n\t}" ::"r"((uint32_t)one),
        "r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_ss(bool one, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 q, %0, 0;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%1], %2, %3, %4, p;\n\t}" ::"r"((uint32_t)one),
        "r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void commit_one(bool one, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %0, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"((uint32_t)one),
        "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ bool odd_value(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return fma2(a, b, make_float2(-0.f, -0.f)); }
__device__ __forceinline__ float max3(float top, float a, float b) {  // of magnitudes
    asm("max.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(fabsf(a)), "f"(fabsf(b)));
    return top;
}
// Values that are not finite become 0; their places as bits, and the largest of
// the others.  (Out of line, and called on a copy: the values stay in registers.)
__device__ __noinline__ float take_odd_at(float2* x, uint32_t* places) {
    float top = 0.f;
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (odd_value(x[i].x)) {
            bits |= 1u << (2 * i);
            x[i].x = 0.f;
        }
        if (odd_value(x[i].y)) {
            bits |= 2u << (2 * i);
            x[i].y = 0.f;
        }
        top = fmaxf(top, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
    }
    *places = bits;
    return top;
}
__device__ __forceinline__ float take_odd(float2 (&x)[16], uint32_t& bits) {
    float2 copy[16];
    uint32_t places;
#pragma unroll
    for (int i = 0; i < 16; ++i) copy[i] = x[i];
    const float top = take_odd_at(copy, &places);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = copy[i];
    bits = places;
    return top;
}
// Of rows first .. first + 31 those that come from rows marked in `odd`: zeros, and their places as bits.
__device__ __noinline__ uint32_t hidden(const Gates& gt, int first, uint64_t odd) {
    uint32_t bits = 0;
    for (int i = 0; i < 32; ++i)
        if ((gt.seen[first + i] | 1ull << (first + i)) & odd) bits |= 1u << i;
    return bits;
}
__device__ __forceinline__ uint32_t hide(float2 (&x)[16], const Gates& gt, int first, uint64_t odd) {
    const uint32_t bits = hidden(gt, first, odd);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (bits >> (2 * i) & 1) x[i].x = 0.f;
        if (bits >> (2 * i + 1) & 1) x[i].y = 0.f;
    }
    return bits;
}

__device__ __forceinline__ float max3_nan(float top, float a, float b) {  // NaN where one is
    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(fabsf(a)), "f"(fabsf(b)));
    return top;
}
// A column of T again, from the rows that come from one another alone (and the
// zeros above the diagonal that the substitution wrote).  What is not finite
// becomes 0, its row is marked.
__device__ __noinline__ void careful_column(const float* A, float* T, const unsigned long long* seen, unsigned long long* odd,
                                            int col) {
#pragma unroll 1
    for (int i = col & ~15; i < kRows; ++i) {
        float x = i == col ? 1.f : 0.f;
#pragma unroll 1
        for (int j = col; j < i; ++j)
            if (seen[i] >> j & 1) x = fmaf(-A[i * kPitch + j], T[j * kPitch + col], x);
        if (odd_value(x)) {
            atomicOr(odd, 1ull << i);
            x = 0.f;
        }
        T[i * kPitch + col] = x;
    }
}

// A tile (16 rows from `rows`, 8 columns from `cols`) of an N x N block below T's
// diagonal at `at`: pass 0, X = A21 T11; pass 1, T21 = -T22 X.
template <int N>
__device__ __forceinline__ void below_tile(const float* A, float* T, float* X, int at, int rows, int cols, int lane, int pass) {
    const int g = lane / 4, t = lane % 4;
    const float* left = (pass == 0 ? A : T + N) + (at + N + rows + g) * kPitch + at + t;
    const float* right = (pass == 0 ? T + at * kPitch + at : X) + t * kPitch + cols + g;
    float d[2][4] = {};
#pragma unroll
    for (int k = 0; k < N; k += 8) {
        uint32_t a[2][4];
        uint2 b[2];
        split_tf32(left[k], a[0][0], a[1][0]);
        split_tf32(left[k + 8 * kPitch], a[0][1], a[1][1]);
        split_tf32(left[k + 4], a[0][2], a[1][2]);
        split_tf32(left[k + 4 + 8 * kPitch], a[0][3], a[1][3]);
        split_tf32(right[k * kPitch], b[0].x, b[1].x);
        split_tf32(right[(k + 4) * kPitch], b[0].y, b[1].y);
        mma_tf32(d[1], a[1], b[0]);
        mma_tf32(d[1], a[0], b[1]);
        mma_tf32(d[0], a[0], b[0]);
    }
    float* to = (pass == 0 ? X + rows * kPitch : T + (at + N + rows) * kPitch + at) + g * kPitch + cols + 2 * t;
    const float sign = pass == 0 ? 1.f : -1.f;
    *reinterpret_cast<float2*>(to) = make_float2(sign * (d[0][0] + d[1][0]), sign * (d[0][1] + d[1][1]));
    *reinterpret_cast<float2*>(to + 8 * kPitch) = make_float2(sign * (d[0][2] + d[1][2]), sign * (d[0][3] + d[1][3]));
}

template <int DK, int DV, bool kBf16>
__global__ void __launch_bounds__(kChunkThreads, 1) delta_chunk_kernel(const __grid_constant__ CUtensorMap map_q,
                                                                       const __grid_constant__ CUtensorMap map_k,
                                                                       const __grid_constant__ CUtensorMap map_v,
                                                                       const __grid_constant__ DeltaRule p,
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
    uint64_t* landed = empty + 2;                                   // [2] its rows have come
    uint64_t* unread = landed + 2;                                  // [2] and are not needed any more
    uint64_t* done1 = unread + 2;
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
    const DeltaSequence seq = delta_sequence(b, d, s, p.rows, err);
    const int row0 = seq.first, n = seq.n, len = seq.len, slot = seq.slot;
    if (n <= p.few_rows || len < 0 || slot < 0) return;
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
            mbar_init(landed + i, 1);
            mbar_init(unread + i, 1);
            mbar_init(drained + i, 1);
        }
        mbar_init(done1, 1);
        mbar_init(done2, 1);
        mbar_init(done_s, 1);
        mbar_init(done_o, 1);
        mbar_init(done_pairs, 1);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tmap(&map_q);
        prefetch_tmap(&map_k);
        prefetch_tmap(&map_v);
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
        // (Loops are kept small: a block's instructions are run through once,
        // and unrolled they came from beyond the instruction caches.)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPrepRegs));
        const int id = tid - kMainThreads;
        constexpr int kLanes = 8, kDown = kPrepThreads / kLanes;  // of a row, one or two of its 16-byte units each
        constexpr int kTimes = 2 * kRows / kDown, kEach = DK / 64;
        const int unit = id % kLanes;
        float* const scales = reinterpret_cast<float*>(smem + C::kScales);  // what K's and Q's rows are to be multiplied by
        float* const g_at = scales + 2 * kRows;                             // in log2
        float* const beta_at = g_at + kRows;
        float* const maxima = beta_at + kRows;  // [half] of P's rows
        float* const scan = maxima + 2 * kRows;
        unsigned long long* const seen_at = reinterpret_cast<unsigned long long*>(smem + C::kSeen);
        unsigned long long* const odd_at = seen_at + kRows;
        float* const A = reinterpret_cast<float*>(smem + C::kA);
        float* const Ts = reinterpret_cast<float*>(smem + C::kTs);
        float* const X = A + 32;  // (A's rows 0 .. 31 have no columns there)
        for (int i = id; i < kRows * kPitch; i += kPrepThreads) Ts[i] = 0.f;  // (above the diagonal nothing is written)
        const bool one = elect_one();
        int staged = -1;  // the last block whose rows the first thread has asked for
        // K, Q and V of a block as they lie; what comes behind its last row is another's, or zeros
        auto stage = [&](int c) {
            const int buf = c & 1, row = row0 + c * kRows;
            staged = c;
            if (c == p.skip_block) return;
            mbar_arrive_expect_tx(landed + buf, C::kKqBytes + C::kVBytes);
            uint8_t* const kq = smem + C::kKq + buf * C::kKqBytes;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int x = key_head * DK + 64 * i;
                bc_tma(bc, x, 2, 64, keys, row, p.rows, kBcDeltaQkv, kBcDeltaQkv);
                tma_load_2d(kq + i * 2 * kRows * kChunkBytes, &map_k, x, row, landed + buf);
                tma_load_2d(kq + (i * 2 + 1) * kRows * kChunkBytes, &map_q, x, row, landed + buf);
            }
            bc_tma(bc, head * DV, 2, DV, values, row, p.rows, kBcDeltaQkv, kBcDeltaQkv);
            tma_load_2d(smem + C::kV + buf * C::kVBytes, &map_v, head * DV, row, landed + buf);
            if (c + 1 < blocks) {  // the next block's on their way to L2: its copies start late
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    prefetch_2d(&map_k, key_head * DK + 64 * i, row + kRows);
                    prefetch_2d(&map_q, key_head * DK + 64 * i, row + kRows);
                }
                prefetch_2d(&map_v, head * DV, row + kRows);
            }
        };
        // The block's gates, asked for ahead of their use.
        float g_next = 0.f, beta_next = 0.f;
        auto load_gates = [&](int t0) {
            g_next = beta_next = 0.f;
            if (id < kRows && t0 + id < n) {
                const int64_t at = (int64_t)(row0 + t0 + id) * d.heads + head, extent = 4 * (int64_t)p.rows * d.heads;
                if (bc_global(bc, p.g + at, 4, p.g, extent, kBcDeltaGate)) g_next = p.g[at];
                if (bc_global(bc, p.beta + at, 4, p.beta, extent, kBcDeltaGate)) beta_next = p.beta[at];
            }
        };
        load_gates(0);
        for (int c = 0; c < blocks; ++c) {
            const int buf = c & 1, t0 = c * kRows, m = min(kRows, n - t0);
            Gates& gt = gates[buf];
            const uint32_t kq_at = base + C::kKq + buf * C::kKqBytes;
            bool lost = false;
            if (id == 0 && staged != c) {
                lost = c >= 2 && !kv_wait(unread + buf, (c / 2 - 1) & 1, abort_flag, err, kDevErrTimeoutDelta);
                if (!lost) stage(c);
            }
            if (any_of<6, kPrepThreads>(lost)) break;  // (all leave together)
            if (id < kRows) {
                float g = g_next, beta = beta_next;
                const bool odd = odd_value(beta) || isnan(g) || g == INFINITY;
                if (odd) g = beta = 0.f;
                g_at[id] = g * 1.44269504088896340736f;
                beta_at[id] = beta;
                seen_at[id] = id < m ? delta_seen(p.tree_mask, p.mask_words, p.rows, row0, id, bc) : 0;
                const unsigned bits = __ballot_sync(0xffffffffu, odd);
                if (lane == 0) reinterpret_cast<unsigned*>(odd_at)[id / 32] = bits;
                float upto = g_at[id];  // of a half's rows, up to and with this one
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float y = __shfl_up_sync(0xffffffffu, upto, o);
                    upto += lane >= o ? y : 0.f;
                }
                scan[id] = upto;
            }
            lost = !kv_wait(landed + buf, (c / 2) & 1, abort_flag, err, kDevErrTimeoutDeltaRows);
            prep_sync();
            // K and Q for the products: fp16 as it is, bf16 with its row's largest
            // brought to 2^13; a row of K that is not finite, or behind the last: zeros
            {
                uint4 w[kTimes][kEach];
                uint32_t top[kTimes];
#pragma unroll
                for (int i = 0; i < kTimes; ++i)
#pragma unroll
                    for (int e = 0; e < kEach; ++e)
                        w[i][e] = lds_u128(kq_at + unit_at(id / kLanes + i * kDown, unit + 8 * e, 2 * kRows));
#pragma unroll
                for (int i = 0; i < kTimes; ++i) {
                    top[i] = 0;
#pragma unroll
                    for (int e = 0; e < kEach; ++e)
                        top[i] = max16x2(top[i], max16x2(max16x2(w[i][e].x & 0x7fff7fffu, w[i][e].y & 0x7fff7fffu),
                                                         max16x2(w[i][e].z & 0x7fff7fffu, w[i][e].w & 0x7fff7fffu)));
                }
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
                    for (int i = 0; i < kTimes; ++i) top[i] = max16x2(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
#pragma unroll
                for (int i = 0; i < kTimes; ++i) {
                    const int r = id / kLanes + i * kDown;
                    const uint32_t most = max(top[i] & 0xffffu, top[i] >> 16);
                    const bool odd = most >= (kBf16 ? 0x7f80u : 0x7c00u), gone = r % kRows >= m || (odd && r < kRows);
                    float2 f = make_float2(1.f, 1.f);
                    if (kBf16) {
                        f = fit(__uint_as_float(most << 16));
                        const uint32_t f2 = (__float_as_uint(f.x) >> 16) * 0x10001u;  // (a power of two is a bf16)
#pragma unroll
                        for (int e = 0; e < kEach; ++e)
                            w[i][e] = make_uint4(scaled16(w[i][e].x, f2), scaled16(w[i][e].y, f2), scaled16(w[i][e].z, f2),
                                                 scaled16(w[i][e].w, f2));
                    }
                    if (odd && r < m && unit == 0) atomicOr(odd_at, 1ull << r);
                    if (kBf16 || gone)
#pragma unroll
                        for (int e = 0; e < kEach; ++e)
                            sts_u128(kq_at + unit_at(r, unit + 8 * e, 2 * kRows), gone ? make_uint4(0, 0, 0, 0) : w[i][e]);
                    if (unit == 0) scales[r] = gone ? 1.f : f.y;
                }
            }
            fence_proxy_async_smem();
            prep_sync();
            if (warp == kMainWarps) {
                tc_fence_after();
                const uint64_t kq = desc_sw128(kq_at, 16, 1024);
#pragma unroll
                for (int k = 0; k < DK / 16; ++k) {
                    const uint64_t at = kq + (((k / 4) * 2 * kRows * kChunkBytes + (k % 4) * 32) >> 4);
                    mma_ss(one, tmem + C::kPairs, at, at, idesc_kv(kRows, 0, false), k > 0);
                }
                commit_one(one, done_pairs);
            }
            // Half a row of the pairs: A from the rows of K, P from those of Q.
            const int pair_row = (warp & 3) * 32 + lane, t = pair_row % kRows, half = (warp - kMainWarps) >> 2;
            const bool is_q = pair_row >= kRows;
            const uint64_t from = seen_at[t] | 1ull << t;  // and the row itself
            const uint32_t bits = (uint32_t)(from >> (32 - 32 * half));  // half 0: columns 32 .. 63, half 1: 0 .. 31
            const float mine = scales[pair_row], factor = (is_q ? p.scale : beta_at[t]) * mine;
            const bool last = !is_q && t == m - 1;
            float run = 0.f, top = 0.f;  // the logarithm of the decay from behind the column
            if (half == 1 && p.tree_mask == nullptr) {
                run = t >= 32 ? scan[t] : 0.f;
            } else if (half == 1) {
                const uint32_t above = (uint32_t)(from >> 32);
#pragma unroll 2
                for (int j = kRows - 4; j >= 32; j -= 4) {
                    const float4 g = *reinterpret_cast<const float4*>(g_at + j);
                    run += above >> (j - 29) & 1 ? g.w : 0.f;
                    run += above >> (j - 30) & 1 ? g.z : 0.f;
                    run += above >> (j - 31) & 1 ? g.y : 0.f;
                    run += above >> (j - 32) & 1 ? g.x : 0.f;
                }
            }
            float* const my_row = A + pair_row * kPitch;
            lost |= !kv_wait(done_pairs, c & 1, abort_flag, err, kDevErrTimeoutDelta);
            // (the block before the last has been used, its gates too)
            lost |= c >= 2 && !kv_wait(empty + buf, (c / 2 - 1) & 1, abort_flag, err, kDevErrTimeoutDelta);
            tc_fence_after();
#pragma unroll 1
            for (int j0 = 16; j0 >= 0; j0 -= 16) {
                const int col = 32 - 32 * half + j0;
                uint32_t x[16];
                tmem_ld16_wait(tmem + ((uint32_t)((warp & 3) * 32) << 16) + C::kPairs + col, x);
                float f[16], g[16];
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 a = *reinterpret_cast<const float4*>(scales + col + j), e = *reinterpret_cast<const float4*>(g_at + col + j);
                    f[j] = a.x; f[j + 1] = a.y; f[j + 2] = a.z; f[j + 3] = a.w;
                    g[j] = e.x; g[j + 1] = e.y; g[j + 2] = e.z; g[j + 3] = e.w;
                }
                const uint32_t here = bits >> j0;
#pragma unroll
                for (int j = 15; j >= 0; --j) {
                    const bool with = here >> j & 1;
                    f[j] = with ? f[j] * fast_exp2(run) : 0.f;
                    run += with ? g[j] : 0.f;
                    const float y = __uint_as_float(x[j]) * (factor * f[j]);  // (A's diagonal is not read)
                    x[j] = __float_as_uint(y);
                    top = fmaxf(top, fabsf(y));
                }
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    *reinterpret_cast<uint4*>(my_row + col + j) = make_uint4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                    if (last) *reinterpret_cast<float4*>(gt.left + col + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
                }
            }
            if (half == 1) {
                const float all = fast_exp2(run);  // from the block's start
                if (is_q) gt.gq[t] = p.scale * all * mine;
                else gt.bg[t] = -beta_at[t] * all * mine;
                if (last) gt.decay = all;
            }
            if (is_q) {
                maxima[half * kRows + t] = top;
            } else if (half == 0) {
                gt.beta[t] = beta_at[t];
                gt.seen[t] = seen_at[t];
                if (t == 0) gt.odd = *odd_at;
            }
            tc_fence_before();
            // Part of a row in fp32 -> its parts
            auto put_parts = [&](const float* row, int u0, int u1, float scale, uint32_t to, int r) {
#pragma unroll 1
                for (int u = u0; u < u1; ++u) {
                    const float4 a = *reinterpret_cast<const float4*>(row + 8 * u), e = *reinterpret_cast<const float4*>(row + 8 * u + 4);
                    uint32_t hi[4], lo[4];
                    split2(a.x * scale, a.y * scale, hi[0], lo[0]);
                    split2(a.z * scale, a.w * scale, hi[1], lo[1]);
                    split2(e.x * scale, e.y * scale, hi[2], lo[2]);
                    split2(e.z * scale, e.w * scale, hi[3], lo[3]);
                    sts_u128(to + unit_at(r, u, kRows), make_uint4(hi[0], hi[1], hi[2], hi[3]));
                    sts_u128(to + C::kPartBytes + unit_at(r, u, kRows), make_uint4(lo[0], lo[1], lo[2], lo[3]));
                }
            };
            prep_sync();
            // T by halves: its diagonal blocks of 16 by substitution, a column a
            // thread; then the blocks below, -T22 (A21 T11), of 16 and of 32.
            if (is_q) {
                const float2 f = fit(fmaxf(maxima[t], maxima[kRows + t]));
                gt.cp[t] = f.y;
                put_parts(my_row, 4 - 4 * half, 8 - 4 * half, f.x, base + C::kP + buf * 2 * C::kPartBytes, t);
            } else if (half == 0) {
                const int at = t / 16 * 16, col = t % 16;
                const float* a = A + at * (kPitch + 1);
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float y[4] = {i == col ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < i; j += 4) {
                        const float4 w = *reinterpret_cast<const float4*>(a + i * kPitch + j);
                        y[0] = fmaf(-w.x, x[j], y[0]);
                        if (j + 1 < i) y[1] = fmaf(-w.y, x[j + 1], y[1]);
                        if (j + 2 < i) y[2] = fmaf(-w.z, x[j + 2], y[2]);
                        if (j + 3 < i) y[3] = fmaf(-w.w, x[j + 3], y[3]);
                    }
                    x[i] = (y[0] + y[1]) + (y[2] + y[3]);
                    Ts[(at + i) * kPitch + t] = x[i];
                }
            }
            load_gates(t0 + kRows);
            if (id == 0 && c + 1 < blocks && (c < 1 || mbar_try_wait(smem_u32(unread + (buf ^ 1)), ((c + 1) / 2 - 1) & 1)))
                stage(c + 1);
            prep_sync();
            // The blocks below, N x N: X = A21 T11, then T21 = -T22 X, a tile of 16 x 8 a warp.
            const int tile = warp - kMainWarps;
            if (tile < 4) below_tile<16>(A, Ts, X + tile / 2 * 16, tile / 2 * 32, 0, tile % 2 * 8, lane, 0);
            prep_sync();
            if (tile < 4) below_tile<16>(A, Ts, X + tile / 2 * 16, tile / 2 * 32, 0, tile % 2 * 8, lane, 1);
            prep_sync();
            below_tile<32>(A, Ts, X, 0, tile / 4 * 16, tile % 4 * 8, lane, 0);
            prep_sync();
            below_tile<32>(A, Ts, X, 0, tile / 4 * 16, tile % 4 * 8, lane, 1);
            prep_sync();
            // T's parts, a quarter of a row a thread; once more where T was not finite.
            bool stop = false;
#pragma unroll 1
            for (bool again = false;; again = true) {
                const int row = id / 4, quarter = id % 4;
                float most = 0.f;
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 w = *reinterpret_cast<const float4*>(Ts + row * kPitch + 16 * quarter + j);
                    most = max3_nan(max3_nan(most, w.x, w.y), w.z, w.w);
                }
                const bool odd = odd_value(most);
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
                const float2 f = fit(most);
                if (quarter == 0) gt.ct[row] = f.y;
                put_parts(Ts + row * kPitch, 2 * quarter, 2 * quarter + 2, f.x, base + C::kT + buf * 2 * C::kPartBytes, row);
                fence_proxy_async_smem();
                if (!any_of<6, kPrepThreads>(lost || odd) || again) break;
                stop = any_of<6, kPrepThreads>(lost);
                if (stop) break;
                if (id < kRows) careful_column(A, Ts, seen_at, odd_at, id);
                prep_sync();
                if (id == 0) gt.odd = *odd_at;
            }
            if (stop) break;
            mbar_arrive(full + buf);
        }
        // Tensor memory is given back only when every product is done.
        // And no copy may be in flight when the CTA ends.
        if (*abort_flag && warp == kMainWarps && one) {
            tc_commit(drained + 1);
            int no_abort = 0;
            kv_wait(drained + 1, 0, &no_abort, err, kDevErrTimeoutDelta);
        }
        if (*abort_flag && id == 0) {
            int no_abort = 0;
            for (int c = max(0, staged - 1); c <= staged; ++c)
                kv_wait(landed + (c & 1), (c / 2) & 1, &no_abort, err, kDevErrTimeoutDeltaRows);
        }
    } else {
        // ------------------------------------------------------------ the blocks
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMainRegs));
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
        float2 S[C::kHalf / 2];
#pragma unroll
        for (int i = 0; i < C::kHalf; ++i) {
            const float* from = at_s + i * DV;
            const float x = busy && len > 0 && bc_global(bc, from, 4, d.s, d.s_extent, kBcDeltaS) ? *from : 0.f;
            (i & 1 ? S[i / 2].y : S[i / 2].x) = x;
        }
        float inverse_s = 1.f;
        // Two neighbouring values -> their parts.
        auto split = [&](float2 x, float scale, uint32_t& hi, uint32_t& lo) {
            x = mul2(x, make_float2(scale, scale));
            hi = KvF16::pack(x.x, x.y);
            const float2 r = fma2(KvF16::unpack(hi), make_float2(-1.f, -1.f), x);
            lo = KvF16::pack(r.x, r.y);
        };
        // S into its parts.
        auto put_state = [&] {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < C::kHalf / 2; ++i) top = max3(top, S[i].x, S[i].y);
            largest(0, top);
            pair_sync(quad);
            const float2 f = fit(largest_of(0));
            inverse_s = f.y;
#pragma unroll
            for (int i = 0; i < C::kHalf / 2; i += 16) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) split(S[i + e], f.x, hi[e], lo[e]);
                tmem_st16(lane_at + C::kParts + share * C::kHalf / 2 + i, hi);
                tmem_st16(lane_at + C::kParts + DK / 2 + share * C::kHalf / 2 + i, lo);
            }
            tmem_wait_st();
        };
        if (busy) put_state();
        const bool one = elect_one();
        bool lost = false;
        // o of the last block: S^T q's and U's parts lie in its columns until the block after next writes there.
        auto take_rows = [&](int c, uint64_t odd, float scale_s, float scale_u) {
            const int buf = c & 1, m = min(kRows, n - c * kRows), first = 32 * share;
            const uint32_t at_d = buf ? C::kNew : C::kD;
            const Gates& gt = gates[buf];
            float2 o[16];
            if (busy) {
                tc_fence_after();
                const float2 inv_s = make_float2(scale_s, scale_s), inv_u = make_float2(scale_u, scale_u);
#pragma unroll
                for (int h = 0; h < 32; h += 16) {
                    uint32_t x[16], y[16];
                    tmem_ld16_wait(lane_at + at_d + first + h, x);
                    tmem_ld16_wait(lane_at + at_d + kRows + first + h, y);
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 gq = *reinterpret_cast<const float4*>(gt.gq + first + h + i);
                        const float4 cp = *reinterpret_cast<const float4*>(gt.cp + first + h + i);
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const float2 xs = make_float2(__uint_as_float(x[i + e]), __uint_as_float(x[i + e + 1]));
                            const float2 ys = make_float2(__uint_as_float(y[i + e]), __uint_as_float(y[i + e + 1]));
                            o[(h + i + e) / 2] = fma2(mul2(ys, inv_s), e ? make_float2(gq.z, gq.w) : make_float2(gq.x, gq.y),
                                                      mul2(mul2(xs, inv_u), e ? make_float2(cp.z, cp.w) : make_float2(cp.x, cp.y)));
                        }
                    }
                }
                if (odd != 0) {
                    const uint32_t gone = hide(o, gt, first, odd);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (gone >> (2 * i) & 1) o[i].x = NAN;
                        if (gone >> (2 * i + 1) & 1) o[i].y = NAN;
                    }
                }
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + buf);
            if (!busy) return;
            float* to = p.out + (row0 + c * kRows + first) * p.out_row_stride + head * DV + at_lane;
            if (m - first >= 32 && !kBoundsCheck) {
#pragma unroll
                for (int i = 0; i < 32; ++i, to += p.out_row_stride) *to = i & 1 ? o[i / 2].y : o[i / 2].x;
                return;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i, to += p.out_row_stride)
                if (first + i < m && bc_global(bc, to, 4, p.out, 4 * ((p.rows - 1) * p.out_row_stride + values), kBcDeltaOut))
                    *to = i & 1 ? o[i / 2].y : o[i / 2].x;
        };
        uint64_t odd_last = 0;
        float scale_s = 1.f, scale_u = 1.f;
        for (int c = 0; c < blocks; ++c) {
            const int buf = c & 1, t0 = c * kRows, m = min(kRows, n - t0);
            const uint32_t at_d = buf ? C::kNew : C::kD, at_new = buf ? C::kD : C::kNew;  // (in turn)
            const Gates& gt = gates[buf];
            lost |= !kv_wait(full + buf, (c / 2) & 1, abort_flag, err, kDevErrTimeoutDelta);
            tc_fence_before();
            if (any_of<5, kMainThreads>(lost)) break;
            const uint64_t kq = desc_sw128(base + C::kKq + buf * C::kKqBytes, 16, 1024);
            const uint64_t td = desc_sw128(base + C::kT + buf * 2 * C::kPartBytes, 16, 1024);
            const uint64_t pd = desc_sw128(base + C::kP + buf * 2 * C::kPartBytes, 16, 1024);
            if (warp == 0) {
                tc_fence_after();
#pragma unroll
                for (int part = 1; part >= 0; --part)  // the smaller parts first
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k)
                        mma_ta(one, tmem + at_d, tmem + C::kParts + part * DK / 2 + 8 * k,
                                      kq + (((k / 4) * 2 * kRows * kChunkBytes + (k % 4) * 32) >> 4),
                                      idesc_kv(2 * kRows, 0, false), part == 0 || k > 0);
                commit_one(one, done1);
            }
            if (c > 0) take_rows(c - 1, odd_last, scale_s, scale_u);  // (under the product)
            const int first = 32 * share;  // the thread's rows of the block
            lost |= !kv_wait(done1, c & 1, abort_flag, err, kDevErrTimeoutDelta);
            float inverse_r = 1.f;
            uint64_t odd = gt.odd;
            const uint64_t rows_in = ~0ull >> (kRows - m);  // (V behind them is another's)
            if (busy) {
                tc_fence_after();
                uint32_t x[32];
                tmem_ld32_wait(lane_at + at_d + first, x);
                const uint16_t* v = reinterpret_cast<const uint16_t*>(smem + C::kV + buf * C::kVBytes) + first * DV + at_lane;
                const float2 inverse2 = make_float2(inverse_s, inverse_s);
                float2 r[16], zero = make_float2(0.f, 0.f);
                float top = 0.f;
                uint32_t bits = 0;
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float4 beta = *reinterpret_cast<const float4*>(gt.beta + first + 2 * i);
                    const float4 bg = *reinterpret_cast<const float4*>(gt.bg + first + 2 * i);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t both = v[(2 * (i + e)) * DV] | (uint32_t)v[(2 * (i + e) + 1) * DV] << 16;
                        const float2 value = kBf16 ? KvBf16::unpack(both) : KvF16::unpack(both);
                        const float2 xs = make_float2(__uint_as_float(x[2 * (i + e)]), __uint_as_float(x[2 * (i + e) + 1]));
                        r[i + e] = fma2(mul2(xs, inverse2), e ? make_float2(bg.z, bg.w) : make_float2(bg.x, bg.y),
                                        mul2(value, e ? make_float2(beta.z, beta.w) : make_float2(beta.x, beta.y)));
                        zero = fma2(r[i + e], make_float2(0.f, 0.f), zero);
                        top = max3(top, r[i + e].x, r[i + e].y);
                    }
                }
                if (!(zero.x + zero.y == 0.f)) top = take_odd(r, bits);  // (NaN)
                largest(1, top);
                odds[share * 128 + at_lane] = bits;
                pair_sync(quad);
                odd |= ((uint64_t)odds[128 + at_lane] << 32 | odds[at_lane]) & rows_in;
                const float2 f = fit(largest_of(1));
                inverse_r = f.y;
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) split(r[e], f.x, hi[e], lo[e]);
                tmem_st16(lane_at + C::kR + first / 2, hi);
                tmem_st16(lane_at + C::kR + kRows / 2 + first / 2, lo);
                tmem_wait_st();
            }
            tc_fence_before();
            main_sync();
            if (warp == 0) {
                tc_fence_after();
                constexpr uint32_t kId = idesc_kv(kRows, 0, false);
#pragma unroll
                for (int pass = 0; pass < 3; ++pass)  // remainder by value, value by remainder, value by value
#pragma unroll
                    for (int k = 0; k < kRows / 16; ++k)
                        mma_ta(one, tmem + at_d, tmem + C::kR + (pass == 0 ? kRows / 2 : 0) + 8 * k,
                                      td + (((pass == 1 ? C::kPartBytes : 0) + k * 32) >> 4), kId, pass > 0 || k > 0);
                commit_one(one, done2);
            }
            lost |= !kv_wait(done2, c & 1, abort_flag, err, kDevErrTimeoutDelta);
            float inverse_u = 1.f, inverse_f = 1.f;
            if (busy) {
                tc_fence_after();
                uint32_t x[32];
                tmem_ld32_wait(lane_at + at_d + first, x);
                float2 u[16], zero = make_float2(0.f, 0.f);
                const float2 inverse2 = make_float2(inverse_r, inverse_r);
                uint32_t bits = 0;
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float4 ct = *reinterpret_cast<const float4*>(gt.ct + first + 2 * i);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 xs = make_float2(__uint_as_float(x[2 * (i + e)]), __uint_as_float(x[2 * (i + e) + 1]));
                        u[i + e] = mul2(mul2(xs, inverse2), e ? make_float2(ct.z, ct.w) : make_float2(ct.x, ct.y));
                        zero = fma2(u[i + e], make_float2(0.f, 0.f), zero);
                    }
                }
                if (!(zero.x + zero.y == 0.f)) take_odd(u, bits);
                odds[256 + share * 128 + at_lane] = bits;
                if (odd != 0) bits |= hide(u, gt, first, odd);
                if (keep) {
                    float* to = p.u + ((int64_t)(row0 + t0 + first) * d.heads + head) * DV + at_lane;
#pragma unroll
                    for (int i = 0; i < 32; ++i, to += values)
                        if (first + i < m && bc_global(bc, to, 4, p.u, 4 * p.rows * values, kBcDeltaU))
                            *to = bits >> i & 1 ? NAN : i & 1 ? u[i / 2].y : u[i / 2].x;
                }
                float top = 0.f, top_f = 0.f;
                float2 w[16];
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float4 left = *reinterpret_cast<const float4*>(gt.left + first + 2 * i);
                    w[i] = mul2(u[i], make_float2(left.x, left.y));
                    w[i + 1] = mul2(u[i + 1], make_float2(left.z, left.w));
                    top = max3(max3(top, u[i].x, u[i].y), u[i + 1].x, u[i + 1].y);
                    top_f = max3(max3(top_f, w[i].x, w[i].y), w[i + 1].x, w[i + 1].y);
                }
                largest(2, top);
                largest(3, top_f);
                pair_sync(quad);
                odd |= ((uint64_t)odds[256 + 128 + at_lane] << 32 | odds[256 + at_lane]) & rows_in;
                const float2 f = fit(largest_of(2)), ff = fit(largest_of(3));
                inverse_u = f.y;
                inverse_f = ff.y;
                uint32_t hi[16], lo[16];
                if (!keep) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) split(w[e], ff.x, hi[e], lo[e]);
                    tmem_st16(lane_at + C::kParts + kRows + first / 2, hi);
                    tmem_st16(lane_at + C::kParts + kRows + kRows / 2 + first / 2, lo);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) split(u[e], f.x, hi[e], lo[e]);
                tmem_st16(lane_at + C::kParts + first / 2, hi);
                tmem_st16(lane_at + C::kParts + kRows / 2 + first / 2, lo);
                tmem_wait_st();
            }
            tc_fence_before();
            main_sync();
            if (warp == 0) {
                tc_fence_after();
                if (!keep) {
                    const uint64_t kn = desc_sw128(base + C::kKq + buf * C::kKqBytes, 2 * kRows * kChunkBytes, 1024);
#pragma unroll
                    for (int part = 1; part >= 0; --part)
#pragma unroll
                        for (int k = 0; k < kRows / 16; ++k)
                            mma_ta(one, tmem + at_new, tmem + C::kParts + kRows + part * kRows / 2 + 8 * k,
                                          kn + ((k * 16 * kChunkBytes) >> 4), idesc_kv(DK, 0, true), part == 0 || k > 0);
                    commit_one(one, done_s);
                }
                constexpr uint32_t kId = idesc_kv(kRows, 0, false);
#pragma unroll
                for (int pass = 0; pass < 3; ++pass)
#pragma unroll
                    for (int k = 0; k < kRows / 16; ++k)
                        mma_ta(one, tmem + at_d, tmem + C::kParts + (pass == 0 ? kRows / 2 : 0) + 8 * k,
                                      pd + (((pass == 1 ? C::kPartBytes : 0) + k * 32) >> 4), kId, pass > 0 || k > 0);
                commit_one(one, done_o);
                commit_one(one, unread + buf);
            }
            if (!keep) {
                lost |= !kv_wait(done_s, c & 1, abort_flag, err, kDevErrTimeoutDelta);
                if (busy) {
                    tc_fence_after();
                    const float2 decay2 = make_float2(gt.decay, gt.decay), inverse2 = make_float2(inverse_f, inverse_f);
#pragma unroll
                    for (int i = 0; i < C::kHalf; i += 32) {
                        uint32_t x[32];
                        tmem_ld32_wait(lane_at + at_new + share * C::kHalf + i, x);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            S[i / 2 + e] = fma2(S[i / 2 + e], decay2,
                                                mul2(inverse2, make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]))));
                    }
                    if (odd != 0) {
#pragma unroll
                        for (int i = 0; i < C::kHalf / 2; ++i) S[i] = make_float2(NAN, NAN);
                    }
                }
            }
            lost |= !kv_wait(done_o, c & 1, abort_flag, err, kDevErrTimeoutDelta);
            odd_last = odd;
            scale_s = inverse_s;
            scale_u = inverse_u;
            if (busy && c + 1 < blocks) {
                tc_fence_after();
                put_state();
            }
            tc_fence_before();
        }
        lost = any_of<5, kMainThreads>(lost);  // one answer: what follows is a warp's work
        if (!lost) take_rows(blocks - 1, odd_last, scale_s, scale_u);
        if (!keep && busy && !lost) {
#pragma unroll
            for (int i = 0; i < C::kHalf; ++i)
                if (bc_global(bc, at_s + i * DV, 4, d.s, d.s_extent, kBcDeltaS))
                    at_s[i * DV] = i & 1 ? S[i / 2].y : S[i / 2].x;
        }
        if (*abort_flag && warp == 0 && one) {
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

// Rows of `width` 16-bit values, in boxes of kRows rows by `box`.
bool encode_rows(void* enc, const uint16_t* base, int64_t width, int64_t rows, int64_t stride, int box, CUtensorMapSwizzle swizzle,
                 CUtensorMap* map) {
    const cuuint64_t gdim[2] = {(cuuint64_t)width, (cuuint64_t)rows}, gstride[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box_dim[2] = {(cuuint32_t)box, (cuuint32_t)kRows}, estride[2] = {1, 1};
    return reinterpret_cast<EncodeTiledFn>(enc)(
               map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<uint16_t*>(base), gdim, gstride, box_dim, estride,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV, bool kBf16>
cudaError_t launch_type(const DeltaRule& p, const DeltaView& d, const BatchView& b, void* encode, int* err,
                        cudaStream_t stream) {
    using C = ChunkShape<DK, DV>;
    CUtensorMap q, k, v;
    const int64_t keys = (int64_t)d.key_heads * DK, values = (int64_t)d.heads * DV;
    if (!encode_rows(encode, p.q, keys, p.rows, p.q_row_stride, 64, CU_TENSOR_MAP_SWIZZLE_128B, &q) ||
        !encode_rows(encode, p.k, keys, p.rows, p.k_row_stride, 64, CU_TENSOR_MAP_SWIZZLE_128B, &k) ||
        !encode_rows(encode, p.v, values, p.rows, p.v_row_stride, DV, CU_TENSOR_MAP_SWIZZLE_NONE, &v))
        return cudaErrorInvalidValue;
    const cudaError_t e = allow_smem<delta_chunk_kernel<DK, DV, kBf16>>(C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_chained(delta_chunk_kernel<DK, DV, kBf16>, dim3((unsigned)((int64_t)b.sequences * d.heads)),
                          dim3(kChunkThreads), C::kSmem, stream, 1, q, k, v, p, d, b, err);
}
template <int DK, int DV>
cudaError_t launch_chunk(const DeltaRule& p, const DeltaView& d, const BatchView& b, void* encode, int* err,
                         cudaStream_t stream) {
    return p.bf16 ? launch_type<DK, DV, true>(p, d, b, encode, err, stream)
                  : launch_type<DK, DV, false>(p, d, b, encode, err, stream);
}

}  // namespace

cudaError_t launch_delta_chunk(const DeltaRule& p, const DeltaView& d, const BatchView& b, void* encode, int* err,
                               cudaStream_t stream) {
    if (d.key_dim == 64)
        return d.value_dim == 64 ? launch_chunk<64, 64>(p, d, b, encode, err, stream)
                                 : launch_chunk<64, 128>(p, d, b, encode, err, stream);
    return d.value_dim == 64 ? launch_chunk<128, 64>(p, d, b, encode, err, stream)
                             : launch_chunk<128, 128>(p, d, b, encode, err, stream);
}

}  // namespace iq4xs
