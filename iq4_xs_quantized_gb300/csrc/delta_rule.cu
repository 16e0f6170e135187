// delta_rule.cu -- the gated delta rule over few rows a sequence: a decode
// step's single tokens, drafted chains and trees; and the choice of the form.
//
// A block of rows of one sequence and head at once, S its state before them:
//
//   u_t = beta_t (v_t - G_t S^T k_t) - sum_j A_tj u_j   A_tj = beta_t F_tj k_t.k_j
//   o_t = scale (G_t S^T q_t + sum_j F_tj (q_t.k_j) u_j)
//   S  <- G_n S + sum_j F_nj k_j u_j^T
//
// j over the rows that t comes from (o: and t itself), F_tj = e^(sum of g behind
// j up to t), G_t the same from the block's start; the sums of g are taken over
// the rows between, so that no difference of long sums enters.
//
// A CTA holds a head's S, or a slice of its columns, in registers for all of a
// sequence's rows: HBM reads it once and, where it moves on, writes it once,
// which bounds single rows (45 sequences of 48 heads of 128 x 128, 283 MB: 45.1 us, 6.3 TB/s, 92 %
// of a copy; one sequence 3.2 us, of which a launch and two loads that wait for one another
// are most).
#include "attention.cuh"
#include "delta.cuh"

namespace iq4xs {
namespace {

// ------------------------------------------------------------- single rows
// Row by row, VS columns a CTA: fp32 throughout, a thread some key channels of
// four columns, the CTA's parts of S^T k and S^T q joined in shared memory.
constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32;

__device__ __forceinline__ void axpy(float4& y, float a, const float4& x) {
    y.x = fmaf(a, x.x, y.x);
    y.y = fmaf(a, x.y, y.y);
    y.z = fmaf(a, x.z, y.z);
    y.w = fmaf(a, x.w, y.w);
}

template <int DK, int VS>
__global__ void __launch_bounds__(kRowThreads, 4) delta_row_kernel(const DeltaRule p, const DeltaView d,
                                                                   const BatchView b, int* err) {
    constexpr int kCols = VS / 4, kKeys = DK / (kRowThreads / kCols);  // threads across; key channels a thread
    static_assert(kKeys >= 2 && kCols <= 16, "a warp's groups of columns are joined by shuffles");
    __shared__ __align__(16) float kq[2][DK];
    __shared__ __align__(16) float parts[kRowWarps][2][VS];
    __shared__ __align__(16) float u_at[VS];
    __shared__ float qk_at;
    griddep_launch_dependents();
    griddep_wait();
    const Bc bc = bc_open(err);
    const int slices = d.value_dim / VS;
    const int slice = blockIdx.x % slices, head = blockIdx.x / slices % d.heads, s = blockIdx.x / slices / d.heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int col = tid % kCols * 4, group = tid / kCols;
    const DeltaSequence seq = delta_sequence(b, d, s, p.rows, err);
    const int row0 = seq.first, n = seq.n, len = seq.len, slot = seq.slot;
    if (n == 0 || len < 0 || slot < 0) return;
    if (n > p.max_rows) {
        if (tid == 0) data_error(err, kDataCount);
        return;
    }
    const int key_head = head / (d.heads / d.key_heads), v0 = slice * VS;
    float* const at_s = d.s + p.s_offset + slot * d.s_slot_stride + ((int64_t)head * DK + group * kKeys) * d.value_dim + v0 + col;
    float4 S[kKeys];
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
        const float* from = at_s + i * d.value_dim;
        S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (len > 0 && bc_global(bc, from, 16, d.s, d.s_extent, kBcDeltaS)) S[i] = *reinterpret_cast<const float4*>(from);
    }
    const int64_t keys = (int64_t)d.key_heads * DK, values = (int64_t)d.heads * d.value_dim;
    for (int t = 0; t < n; ++t) {
        const int row = row0 + t;
        if (t > 0) __syncthreads();  // the last row's keys have been used
        if (tid < 2 * (DK / 8)) {
            const int which = tid / (DK / 8), c = tid % (DK / 8) * 8;
            const uint16_t* base = which ? p.q : p.k;
            const int64_t stride = which ? p.q_row_stride : p.k_row_stride;
            const uint16_t* from = base + row * stride + key_head * DK + c;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (bc_global(bc, from, 16, base, 2 * ((p.rows - 1) * stride + keys), kBcDeltaQkv))
                w = *reinterpret_cast<const uint4*>(from);
            unpack8(p.bf16, w, &kq[which][c]);
        }
        const int64_t at = (int64_t)row * d.heads + head, extent = 4 * (int64_t)p.rows * d.heads;
        float g = 0.f, beta = 0.f, v = 0.f;
        if (bc_global(bc, p.g + at, 4, p.g, extent, kBcDeltaGate)) g = p.g[at];
        if (tid < VS) {
            if (bc_global(bc, p.beta + at, 4, p.beta, extent, kBcDeltaGate)) beta = p.beta[at];
            const uint16_t* from = p.v + row * p.v_row_stride + head * d.value_dim + v0 + tid;
            if (bc_global(bc, from, 2, p.v, 2 * ((p.rows - 1) * p.v_row_stride + values), kBcDeltaQkv))
                v = p.bf16 ? KvBf16::unpack(*from).x : KvF16::unpack(*from).x;
        }
        const float decay = expf(g);
        __syncthreads();
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), c = a;
#pragma unroll
        for (int i = 0; i < kKeys; i += 2) {
            const float2 k2 = *reinterpret_cast<const float2*>(&kq[0][group * kKeys + i]);
            const float2 q2 = *reinterpret_cast<const float2*>(&kq[1][group * kKeys + i]);
            axpy(a, k2.x, S[i]);
            axpy(c, q2.x, S[i]);
            axpy(a, k2.y, S[i + 1]);
            axpy(c, q2.y, S[i + 1]);
        }
        // over the warp's groups: the lower lanes the key's sums, the upper the query's
        const bool low = lane < 16;
        float4 mine = low ? a : c, other = low ? c : a;
        mine.x += __shfl_xor_sync(0xffffffffu, other.x, 16);
        mine.y += __shfl_xor_sync(0xffffffffu, other.y, 16);
        mine.z += __shfl_xor_sync(0xffffffffu, other.z, 16);
        mine.w += __shfl_xor_sync(0xffffffffu, other.w, 16);
        if (kCols == 8) {
            mine.x += __shfl_xor_sync(0xffffffffu, mine.x, 8);
            mine.y += __shfl_xor_sync(0xffffffffu, mine.y, 8);
            mine.z += __shfl_xor_sync(0xffffffffu, mine.z, 8);
            mine.w += __shfl_xor_sync(0xffffffffu, mine.w, 8);
        }
        if (lane % 16 < kCols) *reinterpret_cast<float4*>(&parts[warp][low ? 0 : 1][col]) = mine;
        if (warp == kRowWarps - 1) {
            float qk = 0.f;
#pragma unroll
            for (int i = 0; i < DK; i += 32) qk = fmaf(kq[0][lane + i], kq[1][lane + i], qk);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) qk += __shfl_xor_sync(0xffffffffu, qk, o);
            if (lane == 0) qk_at = qk;
        }
        __syncthreads();
        if (tid < VS) {
            float sk = 0.f, sq = 0.f;
#pragma unroll
            for (int w = 0; w < kRowWarps; ++w) {
                sk += parts[w][0][tid];
                sq += parts[w][1][tid];
            }
            const float u = beta * (v - decay * sk);
            u_at[tid] = u;
            float* to = p.out + row * p.out_row_stride + head * d.value_dim + v0 + tid;
            if (bc_global(bc, to, 4, p.out, 4 * ((p.rows - 1) * p.out_row_stride + values), kBcDeltaOut))
                *to = p.scale * fmaf(qk_at, u, decay * sq);
            if (p.u != nullptr) {
                to = p.u + at * d.value_dim + v0 + tid;
                if (bc_global(bc, to, 4, p.u, 4 * p.rows * values, kBcDeltaU)) *to = u;
            }
        }
        if (p.u == nullptr) {
            __syncthreads();
            const float4 u = *reinterpret_cast<const float4*>(u_at + col);
#pragma unroll
            for (int i = 0; i < kKeys; i += 2) {
                const float2 k2 = *reinterpret_cast<const float2*>(&kq[0][group * kKeys + i]);
                S[i] = make_float4(decay * S[i].x, decay * S[i].y, decay * S[i].z, decay * S[i].w);
                S[i + 1] = make_float4(decay * S[i + 1].x, decay * S[i + 1].y, decay * S[i + 1].z, decay * S[i + 1].w);
                axpy(S[i], k2.x, u);
                axpy(S[i + 1], k2.y, u);
            }
        }
    }
    if (p.u == nullptr) {
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            float* to = at_s + i * d.value_dim;
            if (bc_global(bc, to, 16, d.s, d.s_extent, kBcDeltaS)) *reinterpret_cast<float4*>(to) = S[i];
        }
    }
}

// ------------------------------------------------------------- a few rows
// Blocks of TB rows, 16 columns a warp, by the warp-level MMA on tf32: S^T is its
// left operand and lies in the layout that the state's update gives as a result
// (key channels 2 t and 2 t + 1 of eight stand for the operand's t and t + 4), so
// it stays where it is.  K and Q of 16 bits are exact in tf32; S and u go in two
// parts, a value without its last 13 bits and the remainder, rounded to the 11 bits
// that the MMA takes of it (2^-22 of a value); the MMA cuts its sums off, so S^T k and
// S^T q are made of three (the remainders', each half of the channels'), which are
// joined, and S is moved on, by fp32 arithmetic that rounds.  12 trees of 8 are then off
// by 2.8e-7 of the largest output and 2.0e-7 of their norm, fp32 throughout by 2.8e-7 and
// 1.7e-7; with cut remainders and one sum for both halves 5.5e-7 and 4.1e-7 (trees
// no faster, 48 chains of 16 103 us instead of 107).
//
// CTAs stay for several items (a head's columns of a sequence): S comes to shared
// memory by TMA, goes to registers, and the next item's is on its way meanwhile.
// (CTAs of one item each load together and then compute together: 16.3 us where these
// took 15.1 for 12 trees of 8 of 48 heads of 128 x 128 with the states in L2; 11.7 now, 15.0 from
// HBM, 40 MB: 2.7 TB/s; FFMA instead
// of the MMA 17.8.)  What bounds it: an item's chain of six steps between barriers,
// about 2.9 us, two CTAs an SM; S in two parts is a third of its instructions.
constexpr int kFewPad = 8;  // floats behind a row in shared memory: rows an operand reads together on all banks

template <int DK, int kWarps, int TB>
struct FewShape {
    static constexpr int kThreads = 32 * kWarps, VS = 16 * kWarps;
    static constexpr int kPitch = DK + kFewPad, kVPitch = VS + kFewPad;
    // shared memory, in floats
    static constexpr int kBoxes = VS / 32;             // of 32 columns, 128 bytes a key channel, swizzled
    static constexpr int kS = 0;
    static constexpr int kK = kS + DK * VS;            // [TB][pitch]
    static constexpr int kQ = kK + TB * kPitch;
    static constexpr int kU = kQ + TB * kPitch;        // [TB] S^T k, then u
    static constexpr int kO = kU + TB * kVPitch;       // [TB] S^T q
    static constexpr int kA = kO + TB * kVPitch;       // [TB][TB]
    static constexpr int kP = kA + TB * TB;
    static constexpr int kGates = kP + TB * TB;        // [TB] g, beta, G, F of the last row
    static constexpr int kSeen = kGates + 4 * TB;      // [TB]
    static constexpr int kBar = kSeen + TB;            // the barrier S lands on, and whether a wait ran out
    static constexpr int kSmem = (kBar + 4) * 4;
    static constexpr int kTiles = TB / 8;
    static_assert(kBar % 2 == 0, "barrier's alignment");
};

// x + a u where `with` holds (a selection, not a branch).
__device__ __forceinline__ float take(bool with, float a, float u, float x) {
    const float y = fmaf(a, u, x);
    return with ? y : x;
}

struct FewItem {
    int row0, n, len, slot, head, v0;  // n = 0: nothing to do
};

template <int DK, int kWarps, int TB, bool kMoves>
__global__ void __launch_bounds__(FewShape<DK, kWarps, TB>::kThreads, 16 / kWarps)
    delta_few_kernel(const __grid_constant__ CUtensorMap map_s, const __grid_constant__ DeltaRule p,
                     const __grid_constant__ DeltaView d, const __grid_constant__ BatchView b, int items, int* err) {
    using C = FewShape<DK, kWarps, TB>;
    constexpr int kSteps = DK / 8, VS = C::VS, kTiles = C::kTiles;
    extern __shared__ __align__(1024) float sm[];
    uint32_t* const seen = reinterpret_cast<uint32_t*>(sm + C::kSeen);
    uint64_t* const landed = reinterpret_cast<uint64_t*>(sm + C::kBar);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(landed + 1);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane / 4, t4 = lane % 4;
    if ((smem_u32(sm) & 1023) != 0) {  // (no static shared memory: the swizzle atoms' alignment)
        if (tid == 0) atomicCAS(err, 0, kDevErrLayout);
        return;
    }
    if (tid == 0) {
        mbar_init(landed, 1);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tmap(&map_s);
    }
    __syncthreads();
    griddep_launch_dependents();
    griddep_wait();
    const Bc bc = bc_open(err);
    const int slices = d.value_dim / VS;
    const int64_t keys = (int64_t)d.key_heads * DK, values = (int64_t)d.heads * d.value_dim;
    auto look = [&](int item) {
        FewItem it = {};
        if (item >= items) return it;
        const int s = item / slices / d.heads;
        it.head = item / slices % d.heads;
        it.v0 = item % slices * VS;
        const DeltaSequence seq = delta_sequence(b, d, s, p.rows, err);
        const int n = seq.n;
        it.row0 = seq.first;
        it.len = seq.len;
        it.slot = seq.slot;
        if (n > p.max_rows && tid == 0) data_error(err, kDataCount);
        it.n = it.len < 0 || it.slot < 0 || n > p.max_rows || n > p.few_rows ? 0 : n;
        return it;
    };
    int fetched = 0;
    auto fetch = [&](const FewItem& it) {  // by one thread
        if (it.n == 0 || it.len == 0 || fetched++ == p.skip_block) return;
        mbar_arrive_expect_tx(landed, DK * VS * 4);
        bc_tma(bc, it.v0, 4, VS, d.value_dim, it.head * DK, (int64_t)d.heads * DK, kBcDeltaS, kBcDeltaS);
#pragma unroll
        for (int i = 0; i < C::kBoxes; ++i)
            tma_load_3d(sm + C::kS + i * DK * 32, &map_s, it.v0 + 32 * i, it.head * DK, it.slot, landed);
    };
    FewItem now = look(blockIdx.x);
    if (tid == 0) fetch(now);
    uint32_t phase = 0;
    bool lost = false;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int n = now.n, row0 = now.row0, len = now.len, slot = now.slot, head = now.head, v0 = now.v0;
        const int key_head = head / (d.heads / d.key_heads);
        // A block's rows: asked for before the next item's state, behind which they would wait.
        constexpr int kAll = TB * 2 * (DK / 8), kUnits = (kAll + C::kThreads - 1) / C::kThreads;
        uint4 kq[kUnits];
        uint16_t v[TB];  // of a column, where the thread has one
        float gate = 0.f, beta = 0.f;
        auto ask = [&](int t0) {
            const int m = min(TB, n - t0), first = row0 + t0;
#pragma unroll
            for (int x = 0; x < kUnits; ++x) {  // (rows behind the last: zeros)
                const int i = tid + x * C::kThreads, c = i % (DK / 8) * 8, which = i / (DK / 8) % 2, t = i / (DK / 8) / 2;
                const uint16_t* base = which ? p.q : p.k;
                const int64_t stride = which ? p.q_row_stride : p.k_row_stride;
                const uint16_t* from = base + (first + t) * stride + key_head * DK + c;
                kq[x] = make_uint4(0, 0, 0, 0);
                if (t < m && bc_global(bc, from, 16, base, 2 * ((p.rows - 1) * stride + keys), kBcDeltaQkv))
                    kq[x] = *reinterpret_cast<const uint4*>(from);
            }
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                const uint16_t* from = p.v + (first + t) * p.v_row_stride + head * d.value_dim + v0 + tid;
                v[t] = 0;
                if (tid < VS && t < m && bc_global(bc, from, 2, p.v, 2 * ((p.rows - 1) * p.v_row_stride + values), kBcDeltaQkv))
                    v[t] = *from;
            }
            if (tid < m) {
                const int64_t at = (int64_t)(first + tid) * d.heads + head, extent = 4 * (int64_t)p.rows * d.heads;
                if (bc_global(bc, p.g + at, 4, p.g, extent, kBcDeltaGate)) gate = p.g[at];
                if (bc_global(bc, p.beta + at, 4, p.beta, extent, kBcDeltaGate)) beta = p.beta[at];
            }
        };
        ask(0);
        const FewItem next = look(item + gridDim.x);  // (its loads beside this one's state)
        // Element e of step i: key channel 8 i + 2 t4 + (e & 1), column 16 warp + g + 8 (e >> 1).
        float S[kSteps][4];
        if (n > 0 && len > 0) {
            lost = !kv_wait(landed, phase & 1, abort_flag, err, kDevErrTimeoutDeltaRows);
            ++phase;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 2 * t4 + (e & 1), c = 16 * (warp & 1) + g + 8 * (e >> 1);
                const float* from = sm + C::kS + (warp >> 1) * DK * 32 + r * 32 + ((c >> 2) ^ r) * 4 + (c & 3);
#pragma unroll
                for (int i = 0; i < kSteps; ++i) S[i][e] = from[i * 8 * 32];
            }
        } else {
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[i][e] = 0.f;
        }
        if (__syncthreads_or(lost)) break;  // (all leave together; the last item is done)
        if (tid == 0) {
            // The next state: to L2 now, to shared memory once a product has used all of
            // this one (a barrier alone does not wait for loads on their way to
            // registers, and the copy does not queue behind them).
            if (n == 0) fetch(next);
            else if (next.n > 0 && next.len > 0)
#pragma unroll
                for (int i = 0; i < C::kBoxes; ++i)
                    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(&map_s),
                                 "r"(next.v0 + 32 * i), "r"(next.head * DK), "r"(next.slot)
                                 : "memory");
        }
        if (tid < 3 * TB && next.n > 0) {  // the next item's rows on their way to L2
            const int t = tid / 3, which = tid % 3, nk = next.head / (d.heads / d.key_heads) * DK;
            if (t < next.n) {
                const uint16_t* at = which == 0   ? p.k + (next.row0 + t) * p.k_row_stride + nk
                                     : which == 1 ? p.q + (next.row0 + t) * p.q_row_stride + nk
                                                  : p.v + (next.row0 + t) * p.v_row_stride + next.head * d.value_dim + next.v0;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
                if (which < 2 ? DK > 64 : VS > 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + 64));
            }
        }
        now = next;
        for (int t0 = 0; t0 < n; t0 += TB) {
            const int m = min(TB, n - t0), first = row0 + t0;
            if (t0 > 0) {
                gate = beta = 0.f;
                ask(t0);
                __syncthreads();  // the last block's rows have been used
            }
#pragma unroll
            for (int x = 0; x < kUnits; ++x) {
                const int i = tid + x * C::kThreads, c = i % (DK / 8) * 8, which = i / (DK / 8) % 2, t = i / (DK / 8) / 2;
                if (i >= kAll) break;
                float y[8];
                unpack8(p.bf16, kq[x], y);
                float* const to = sm + (which ? C::kQ : C::kK) + t * C::kPitch + c;
                *reinterpret_cast<float4*>(to) = make_float4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<float4*>(to + 4) = make_float4(y[4], y[5], y[6], y[7]);
            }
            if (tid < TB) {
                sm[C::kGates + tid] = gate;
                sm[C::kGates + TB + tid] = beta;
                seen[tid] = tid >= m ? 0 : p.tree_mask ? (uint32_t)delta_seen(p.tree_mask, p.mask_words, p.rows, row0, tid, bc)
                                                       : (1u << tid) - 1;
            }
            __syncthreads();
            // S^T [K; Q]: columns by rows.  The last warps also [K; Q] K^T: rows by rows,
            // tile y of rows with tile x before or at it.
            {
                float sk[kTiles][3][4] = {}, sq[kTiles][3][4] = {}, pairs[2][4] = {};
                const int pair = kWarps - 1 - warp;  // tiles (0, 0), (1, 0), (1, 1)
                const int ty = pair > 0 ? 1 : 0, tx = pair > 1 ? 1 : 0;
                const bool has_pair = pair < (kTiles == 2 ? 3 : 1);
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    uint32_t hi[4], lo[4];
                    split_tf32_near(S[i][0], hi[0], lo[0]);
                    split_tf32_near(S[i][2], hi[1], lo[1]);
                    split_tf32_near(S[i][1], hi[2], lo[2]);
                    split_tf32_near(S[i][3], hi[3], lo[3]);
                    const int half = i < kSteps / 2 ? 0 : 2;
#pragma unroll
                    for (int x = 0; x < kTiles; ++x) {
                        const uint2 k = *reinterpret_cast<const uint2*>(sm + C::kK + (8 * x + g) * C::kPitch + 8 * i + 2 * t4);
                        const uint2 q = *reinterpret_cast<const uint2*>(sm + C::kQ + (8 * x + g) * C::kPitch + 8 * i + 2 * t4);
                        mma_tf32(sk[x][1], lo, k);
                        mma_tf32(sq[x][1], lo, q);
                        mma_tf32(sk[x][half], hi, k);
                        mma_tf32(sq[x][half], hi, q);
                    }
                    if (has_pair) {
                        const uint2 k = *reinterpret_cast<const uint2*>(sm + C::kK + (8 * ty + g) * C::kPitch + 8 * i + 2 * t4);
                        const uint2 q = *reinterpret_cast<const uint2*>(sm + C::kQ + (8 * ty + g) * C::kPitch + 8 * i + 2 * t4);
                        const uint32_t a[4] = {k.x, q.x, k.y, q.y};
                        mma_tf32(pairs[i & 1], a, *reinterpret_cast<const uint2*>(sm + C::kK + (8 * tx + g) * C::kPitch + 8 * i + 2 * t4));
                    }
                }
#pragma unroll
                for (int x = 0; x < kTiles; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int to = (8 * x + 2 * t4 + (e & 1)) * C::kVPitch + 16 * warp + g + 8 * (e >> 1);
                        sm[C::kU + to] = sk[x][0][e] + (sk[x][1][e] + sk[x][2][e]);
                        sm[C::kO + to] = sq[x][0][e] + (sq[x][1][e] + sq[x][2][e]);
                    }
                if (has_pair) {
                    const int t = 8 * ty + g;
                    const uint32_t with = seen[t] | 1u << t;
                    auto decay_over = [&](uint32_t rows) {
                        float sum = 0.f;
#pragma unroll
                        for (int k = TB - 1; k >= 0; --k) sum += rows >> k & 1 ? sm[C::kGates + k] : 0.f;
                        return expf(sum);
                    };
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int j = 8 * tx + 2 * t4 + e;
                        const bool from = with >> j & 1;
                        const float far = decay_over(with & ~((2u << j) - 1));
                        sm[C::kA + t * TB + j] = from ? sm[C::kGates + TB + t] * far * (pairs[0][e] + pairs[1][e]) : 0.f;
                        sm[C::kP + t * TB + j] = from ? p.scale * far * (pairs[0][2 + e] + pairs[1][2 + e]) : 0.f;
                        if (t == m - 1) sm[C::kGates + 3 * TB + j] = from ? far : 0.f;
                    }
                    if (tx == ty && t4 == 0) sm[C::kGates + 2 * TB + t] = decay_over(with);
                    if (kTiles == 2 && m <= 8 && tx == 0 && t4 == 0) sm[C::kGates + 3 * TB + 8 + g] = 0.f;
                }
            }
            __syncthreads();
            if (t0 == 0 && tid == 0) fetch(next);
            // u, a column a thread.  (A row takes the rows that it comes from, and no
            // others: 0 times NaN is none of its.)
            if (tid < VS) {
                float u[TB];
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    float x = sm[C::kGates + TB + t] * ((p.bf16 ? KvBf16::unpack(v[t]).x : KvF16::unpack(v[t]).x) -
                                                              sm[C::kGates + 2 * TB + t] * sm[C::kU + t * C::kVPitch + tid]);
                    const uint32_t from = seen[t];
#pragma unroll
                    for (int j = 0; j < t; j += 4) {
                        const float4 a = *reinterpret_cast<const float4*>(sm + C::kA + t * TB + j);
                        x = take(from >> j & 1, -a.x, u[j], x);
                        if (j + 1 < t) x = take(from >> (j + 1) & 1, -a.y, u[j + 1], x);
                        if (j + 2 < t) x = take(from >> (j + 2) & 1, -a.z, u[j + 2], x);
                        if (j + 3 < t) x = take(from >> (j + 3) & 1, -a.w, u[j + 3], x);
                    }
                    u[t] = t < m ? x : 0.f;
                }
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    sm[C::kU + t * C::kVPitch + tid] = u[t];
                    float* to = p.u + ((int64_t)(first + t) * d.heads + head) * d.value_dim + v0 + tid;
                    if (!kMoves && t < m && bc_global(bc, to, 4, p.u, 4 * p.rows * values, kBcDeltaU)) *to = u[t];
                }
            }
            __syncthreads();
            // out: a column and every second row a thread
            {
                const int c = tid % VS;
                float u[TB];
#pragma unroll
                for (int t = 0; t < TB; ++t) u[t] = sm[C::kU + t * C::kVPitch + c];
#pragma unroll
                for (int t2 = 0; t2 < TB; t2 += 2) {
                    const int t = t2 + tid / VS;
                    if (t < m) {
                        float x = p.scale * sm[C::kGates + 2 * TB + t] * sm[C::kO + t * C::kVPitch + c];
                        const uint32_t from = seen[t] | 1u << t;
#pragma unroll
                        for (int j = 0; j < t2 + 2; j += 4) {
                            const float4 a = *reinterpret_cast<const float4*>(sm + C::kP + t * TB + j);
                            x = take(from >> j & 1, a.x, u[j], x);
                            if (j + 1 < t2 + 2) x = take(from >> (j + 1) & 1, a.y, u[j + 1], x);
                            if (j + 2 < t2 + 2) x = take(from >> (j + 2) & 1, a.z, u[j + 2], x);
                            if (j + 3 < t2 + 2) x = take(from >> (j + 3) & 1, a.w, u[j + 3], x);
                        }
                        float* to = p.out + (first + t) * p.out_row_stride + head * d.value_dim + v0 + c;
                        if (bc_global(bc, to, 4, p.out, 4 * ((p.rows - 1) * p.out_row_stride + values), kBcDeltaOut)) *to = x;
                    }
                }
            }
            if (kMoves) {
                // S: columns by key channels, the rows between
                uint32_t hi[kTiles][4], lo[kTiles][4];
#pragma unroll
                for (int x = 0; x < kTiles; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = 8 * x + t4 + 4 * (e >> 1);
                        split_tf32_near(sm[C::kGates + 3 * TB + t] * sm[C::kU + t * C::kVPitch + 16 * warp + g + 8 * (e & 1)], hi[x][e], lo[x][e]);
                    }
                const float decay = sm[C::kGates + 2 * TB + m - 1];
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    float add[4] = {};
#pragma unroll
                    for (int x = 0; x < kTiles; ++x) {
                        const float* k = sm + C::kK + (8 * x + t4) * C::kPitch + 8 * i + g;
                        const uint2 k2 = make_uint2(__float_as_uint(k[0]), __float_as_uint(k[4 * C::kPitch]));
                        mma_tf32(add, lo[x], k2);
                        mma_tf32(add, hi[x], k2);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[i][e] = fmaf(decay, S[i][e], add[e]);
                }
            }
            if (!kMoves) break;  // (a tree is one block: no loop that S's parts could be kept over)
        }
        if (kMoves && n > 0) {
            float* const at_s = d.s + p.s_offset + slot * d.s_slot_stride + ((int64_t)head * DK + 2 * t4) * d.value_dim + v0 + 16 * warp + g;
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float* to = at_s + (8 * i + (e & 1)) * d.value_dim + 8 * (e >> 1);
                    if (bc_global(bc, to, 4, d.s, d.s_extent, kBcDeltaS)) *to = S[i][e];
                }
        }
    }
    // No copy may be in flight when the CTA ends; all were waited for, unless a wait ran out.
    if (lost && tid == 0) {
        int no_abort = 0;
        kv_wait(landed, (phase - 1) & 1, &no_abort, err, kDevErrTimeoutDeltaRows);
    }
}

template <int DK, int VS>
cudaError_t launch_row(const DeltaRule& p, const DeltaView& d, const BatchView& b, int* err, cudaStream_t stream) {
    const dim3 grid((unsigned)((int64_t)b.sequences * d.heads * (d.value_dim / VS)));
    return launch_chained(delta_row_kernel<DK, VS>, grid, dim3(kRowThreads), 0, stream, 1, p, d, b, err);
}

template <int DK, int kWarps, int TB, bool kMoves>
cudaError_t launch_few(const DeltaRule& p, const DeltaView& d, const BatchView& b, void* encode, int* err, int num_sms,
                       cudaStream_t stream) {
    using C = FewShape<DK, kWarps, TB>;
    // One map over the layer's states: columns, key channels of all heads, slots.
    CUtensorMap map;
    const int64_t size = (int64_t)d.heads * DK * d.value_dim;
    const cuuint64_t gdim[3] = {(cuuint64_t)d.value_dim, (cuuint64_t)d.heads * DK, (cuuint64_t)d.slots};
    const cuuint64_t gstride[2] = {(cuuint64_t)d.value_dim * 4, (cuuint64_t)(d.slots > 1 ? d.s_slot_stride : size) * 4};
    const cuuint32_t box[3] = {32, DK, 1}, estride[3] = {1, 1, 1};
    if (reinterpret_cast<EncodeTiledFn>(encode)(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, d.s + p.s_offset, gdim, gstride, box,
                                                estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    const cudaError_t e = allow_smem<delta_few_kernel<DK, kWarps, TB, kMoves>>(C::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t items = (int64_t)b.sequences * d.heads * (d.value_dim / C::VS), most = (int64_t)num_sms * (16 / kWarps);
    return launch_chained(delta_few_kernel<DK, kWarps, TB, kMoves>, dim3((unsigned)(items < most ? items : most)), dim3(C::kThreads),
                          C::kSmem, stream, 1, map, p, d, b, (int)items, err);
}

template <int DK>
cudaError_t launch_keys(const DeltaRule& p, const DeltaView& d, const BatchView& b, void* encode, int* err, int num_sms,
                        bool single, int block, cudaStream_t stream) {
    if (single) {
        // 32 columns a CTA while all CTAs are resident at once, else 64 (48 heads:
        // 1 sequence 3.57 and 3.96 us, 3 4.46 and 5.00; 4 6.38 and 5.96, 16 16.1
        // and 13.6, 45 58.7 and 47.0).
        const bool thin = (int64_t)b.sequences * d.heads * (d.value_dim / 32) <= 4 * num_sms;
        return thin ? launch_row<DK, 32>(p, d, b, err, stream) : launch_row<DK, 64>(p, d, b, err, stream);
    }
    // (32 columns a CTA were no faster here, for one sequence either: 6.57 us for
    // 4.95 for a tree of 8.)
    if (p.u == nullptr)
        return d.value_dim == 128 ? launch_few<DK, 8, 8, true>(p, d, b, encode, err, num_sms, stream)
                                  : launch_few<DK, 4, 8, true>(p, d, b, encode, err, num_sms, stream);
    if (block == 8)
        return d.value_dim == 128 ? launch_few<DK, 8, 8, false>(p, d, b, encode, err, num_sms, stream)
                                  : launch_few<DK, 4, 8, false>(p, d, b, encode, err, num_sms, stream);
    return d.value_dim == 128 ? launch_few<DK, 8, 16, false>(p, d, b, encode, err, num_sms, stream)
                              : launch_few<DK, 4, 16, false>(p, d, b, encode, err, num_sms, stream);
}

}  // namespace

// The form follows a sequence's rows (times in us, 48 heads of 128 x 128).
// Row by row up to two on average: 12 chains of 2 13.3 (blocks of 8: 18.1), of 4
// 18.8 (18.4); 48 of 2 59.8 (69.4), of 4 81.6 (70.4).
// Blocks of 8 for chains: 48 of 16 107 (blocks of 16, which have no such form any more,
// 1.2 times as much), of 32 177.  A tree is one block: of 16 from 9 rows on.
// Blocks of 64 from there where they win.  They take 13.6 for a wave of the SMs
// whatever the rows: 3 chains of 16 13.7 (blocks of 8: 13.1), of 20 13.6 (16.5), 1 of 20
// 13.6 (13.0), of 32 13.5 (16.0); in several waves 12 chains of 32 50.8 (44.1), 48
// of 32 221 (177), each 8 rows more 8 and 34.
// A batch whose longest sequence is longer, but not the mean, takes both.
// The same limits for other heads: 48 chains of 16 heads of 128 x 128 of 3 rows 26.7 (row
// by row 20.8), of 4 26.9 (24.6), of 40 80.2 (blocks of 64: 77.8), of 48 80.3 (blocks of 8:
// 94.1).  Narrow heads stay in blocks of 8 for too short: 6 of 64 x 64, one chain of 20
// 10.8 (blocks of 8: 7.1), of 40 10.7 (10.2), 48 of 48 21.2 (16.4), of 64 21.0 (21.1); 16 of
// 128 x 64, 48 of 48 67.3 (52.4), of 64 67.2 (69.7).
cudaError_t launch_delta_rule(DeltaRule p, const DeltaView& d, const BatchView& b, void* encode, int* err, int num_sms,
                              cudaStream_t stream) {
    const bool tree = p.u != nullptr;
    const int64_t sequences = b.sequences;
    const int few = tree || sequences * d.heads <= num_sms ? 16 : 40;
    if (p.max_rows > few && p.rows > few * sequences) return launch_delta_chunk(p, d, b, encode, err, stream);
    const bool both = p.max_rows > few && (tree || p.max_given);
    if (both) {
        p.few_rows = few;
        const cudaError_t e = launch_delta_chunk(p, d, b, encode, err, stream);
        if (e != cudaSuccess) return e;
    } else {
        p.few_rows = p.max_rows;
    }
    const bool single = tree ? p.max_rows == 1 : p.rows <= 2 * sequences && (p.max_rows <= 8 || !p.max_given);
    const int block = tree && p.max_rows > 8 ? 16 : 8;
    return d.key_dim == 64 ? launch_keys<64>(p, d, b, encode, err, num_sms, single, block, stream)
                           : launch_keys<128>(p, d, b, encode, err, num_sms, single, block, stream);
}

}  // namespace iq4xs
