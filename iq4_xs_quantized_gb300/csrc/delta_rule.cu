// delta_rule.cu -- the gated delta rule over few rows a sequence: a decode
// step's single tokens, drafted chains and trees.
//
// A block of rows of one sequence and head at once, S its state before them:
//
//   u_t = beta_t (v_t - G_t S^T k_t) - sum_j A_tj u_j   A_tj = beta_t F_tj k_t.k_j
//   o_t = scale (G_t S^T q_t + sum_j F_tj (q_t.k_j) u_j)
//   S  <- G_n S + sum_j F_nj k_j u_j^T
//
// j over the rows that t comes from (o: and t itself), F_tj = e^(sum of g behind
// j up to t), G_t the same from the block's start.  F is made by walking back
// from t, so that no difference of long sums enters it.
//
// A CTA holds a head's S, or a slice of its columns, in registers for all of a
// sequence's rows: HBM reads it once and, where it moves on, writes it once.
// That traffic bounds decode steps; from about eight rows on it is the fp32
// pipe (4 to 6 operations a value of S and row).
#include "delta.cuh"

namespace iq4xs {
namespace {

constexpr int kStepThreads = 256, kStepWarps = kStepThreads / 32;

// DK key channels; VS of the value channels; blocks of TB rows.
template <int DK, int VS, int TB>
struct StepShape {
    static constexpr int kCols = VS / 4;                  // threads across the columns
    static constexpr int kGroups = kStepThreads / kCols;  // and down the key channels
    static constexpr int kKeys = DK / kGroups;            // key channels a thread
    static constexpr int kRound = TB < 4 ? TB : 4;        // rows summed over the warps at a time
    static constexpr int kPitch = DK + 16;                // (two rows' quarters of 16 channels on all the banks)
    // shared memory, in floats
    static constexpr int kK = 0;                          // [TB][pitch]
    static constexpr int kQ = kK + TB * kPitch;
    static constexpr int kV = kQ + TB * kPitch;           // [TB][VS]
    static constexpr int kSums = kV + TB * VS;            // [TB][S^T k -> u, S^T q][VS]
    static constexpr int kRed = kSums + TB * 2 * VS;      // [warps][round][2][VS]
    static constexpr int kA = kRed + kStepWarps * kRound * 2 * VS;  // [TB][TB]
    static constexpr int kP = kA + TB * TB;
    static constexpr int kFar = kP + TB * TB;
    static constexpr int kGates = kFar + TB * TB;         // [TB] g, beta, G
    static constexpr int kFloats = kGates + 3 * TB;
    static constexpr int kSmem = (kFloats + (kFloats & 1)) * 4 + TB * 8;  // and the rows seen
    static_assert(kKeys >= 1 && kKeys % 2 == 0, "key channels a thread");
    static_assert(TB == 1 || ((kA & 3) == 0 && (kP & 3) == 0), "rows of A and P are read as vectors");
};

__device__ __forceinline__ void axpy(float4& y, float a, const float4& x) {
    y.x = fmaf(a, x.x, y.x);
    y.y = fmaf(a, x.y, y.y);
    y.z = fmaf(a, x.z, y.z);
    y.w = fmaf(a, x.w, y.w);
}

template <int DK, int VS, int TB>
__global__ void __launch_bounds__(kStepThreads, TB == 1 ? 4 : 3) delta_step_kernel(const DeltaRule p, const DeltaView d,
                                                                  const BatchView b, int* err) {
    using C = StepShape<DK, VS, TB>;
    extern __shared__ __align__(16) float sm[];
    uint64_t* seen = reinterpret_cast<uint64_t*>(sm + C::kFloats + (C::kFloats & 1));
    griddep_launch_dependents();
    griddep_wait();
    const Bc bc = bc_open(err);
    const int slices = d.value_dim / VS;
    const int slice = blockIdx.x % slices, head = blockIdx.x / slices % d.heads, s = blockIdx.x / slices / d.heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int col = tid % C::kCols * 4, group = tid / C::kCols;
    int row0;
    const int n = batch_rows(b, s, p.rows, &row0, err);
    const int len = batch_len(b, s, err), slot = delta_slot(d, s, err);
    if (n == 0 || len < 0 || slot < 0) return;
    if (n > p.max_rows) {
        if (tid == 0) data_error(err, kDataCount);
        return;
    }
    const int key_head = head / (d.heads / d.key_heads), v0 = slice * VS;
    float* const at_s = d.s + p.s_offset + slot * d.s_slot_stride +
                        ((int64_t)head * DK + group * C::kKeys) * d.value_dim + v0 + col;
    float4 S[C::kKeys];
#pragma unroll
    for (int i = 0; i < C::kKeys; ++i) {
        const float* from = at_s + i * d.value_dim;
        S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (len > 0 && bc_global(bc, from, 16, d.s, d.s_extent, kBcDeltaS)) S[i] = *reinterpret_cast<const float4*>(from);
    }
    const int64_t keys = (int64_t)d.key_heads * DK, values = (int64_t)d.heads * d.value_dim;
    for (int t0 = 0; t0 < n; t0 += TB) {
        const int m = min(TB, n - t0), first = row0 + t0;
        if (t0 > 0) __syncthreads();  // the last block's rows have been used
        auto put8 = [&](const uint16_t* base, const uint16_t* from, int64_t extent, float* to) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (bc_global(bc, from, 16, base, extent, kBcDeltaQkv)) w = *reinterpret_cast<const uint4*>(from);
            float x[8];
            unpack8(p.bf16, w, x);
            *reinterpret_cast<float4*>(to) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(to + 4) = make_float4(x[4], x[5], x[6], x[7]);
        };
        for (int i = tid; i < m * 2 * (DK / 8); i += kStepThreads) {
            const int c = i % (DK / 8) * 8, which = i / (DK / 8) % 2, t = i / (DK / 8) / 2;
            const uint16_t* base = which ? p.q : p.k;
            const int64_t stride = which ? p.q_row_stride : p.k_row_stride;
            put8(base, base + (first + t) * stride + key_head * DK + c, 2 * ((p.rows - 1) * stride + keys),
                 sm + (which ? C::kQ : C::kK) + t * C::kPitch + c);
        }
        for (int i = kStepThreads - 1 - tid; i < m * (VS / 8); i += kStepThreads) {  // (threads that have no key first)
            const int c = i % (VS / 8) * 8, t = i / (VS / 8);
            put8(p.v, p.v + (first + t) * p.v_row_stride + head * d.value_dim + v0 + c,
                 2 * ((p.rows - 1) * p.v_row_stride + values), sm + C::kV + t * VS + c);
        }
        if (tid < m) {
            const int64_t at = (int64_t)(first + tid) * d.heads + head, extent = 4 * (int64_t)p.rows * d.heads;
            float g = 0.f, beta = 0.f;
            if (bc_global(bc, p.g + at, 4, p.g, extent, kBcDeltaGate)) g = p.g[at];
            if (bc_global(bc, p.beta + at, 4, p.beta, extent, kBcDeltaGate)) beta = p.beta[at];
            sm[C::kGates + tid] = g;
            sm[C::kGates + TB + tid] = beta;
            seen[tid] = p.tree_mask ? delta_seen(p.tree_mask, p.mask_words, p.rows, row0, tid, bc) : (1ull << tid) - 1;
        }
        __syncthreads();
        // Decays by walking back from every row.
        if (tid < m) {
            float run = sm[C::kGates + tid];
            sm[C::kFar + tid * TB + tid] = 1.f;
            for (uint32_t left = (uint32_t)seen[tid]; left != 0;) {
                const int j = 31 - __clz(left);
                left ^= 1u << j;
                sm[C::kFar + tid * TB + j] = expf(run);
                run += sm[C::kGates + j];
            }
            sm[C::kGates + 2 * TB + tid] = expf(run);
        }
        // Products of the rows' keys and queries, four lanes a pair, a quarter of every 16 channels each.
        for (int i0 = 0; i0 < m * TB; i0 += kStepThreads / 4) {
            const int i = i0 + tid / 4, t = i / TB, j = i % TB;
            float kk = 0.f, qk = 0.f;
            if (t < m && j <= t) {
                const float* kt = sm + C::kK + t * C::kPitch + lane % 4 * 4;
                const float* qt = sm + C::kQ + t * C::kPitch + lane % 4 * 4;
                const float* kj = sm + C::kK + j * C::kPitch + lane % 4 * 4;
#pragma unroll
                for (int c = 0; c < DK; c += 16) {
                    const float4 a = *reinterpret_cast<const float4*>(kt + c), q = *reinterpret_cast<const float4*>(qt + c);
                    const float4 e = *reinterpret_cast<const float4*>(kj + c);
                    kk = fmaf(a.x, e.x, fmaf(a.y, e.y, fmaf(a.z, e.z, fmaf(a.w, e.w, kk))));
                    qk = fmaf(q.x, e.x, fmaf(q.y, e.y, fmaf(q.z, e.z, fmaf(q.w, e.w, qk))));
                }
            }
#pragma unroll
            for (int o = 2; o > 0; o >>= 1) {
                kk += __shfl_xor_sync(0xffffffffu, kk, o);
                qk += __shfl_xor_sync(0xffffffffu, qk, o);
            }
            if (lane % 4 == 0 && t < m) {
                sm[C::kA + i] = kk;
                sm[C::kP + i] = qk;
            }
        }
        // S^T k and S^T q, kRound rows at a time.
#pragma unroll 1
        for (int r0 = 0; r0 < m; r0 += C::kRound) {
#pragma unroll
            for (int r = 0; r < C::kRound; ++r) {
                if (r0 + r >= m) break;
                const float* kt = sm + C::kK + (r0 + r) * C::kPitch + group * C::kKeys;
                const float* qt = sm + C::kQ + (r0 + r) * C::kPitch + group * C::kKeys;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f), c = a;
#pragma unroll
                for (int i = 0; i < C::kKeys; i += 2) {
                    const float2 k2 = *reinterpret_cast<const float2*>(kt + i), q2 = *reinterpret_cast<const float2*>(qt + i);
                    axpy(a, k2.x, S[i]);
                    axpy(c, q2.x, S[i]);
                    axpy(a, k2.y, S[i + 1]);
                    axpy(c, q2.y, S[i + 1]);
                }
                // over the warp's groups: the lower lanes the keys' sums, the upper the queries'
                const bool low = lane < 16;
                float4 mine = low ? a : c, other = low ? c : a;
                mine.x += __shfl_xor_sync(0xffffffffu, other.x, 16);
                mine.y += __shfl_xor_sync(0xffffffffu, other.y, 16);
                mine.z += __shfl_xor_sync(0xffffffffu, other.z, 16);
                mine.w += __shfl_xor_sync(0xffffffffu, other.w, 16);
                if (C::kCols == 8) {
                    mine.x += __shfl_xor_sync(0xffffffffu, mine.x, 8);
                    mine.y += __shfl_xor_sync(0xffffffffu, mine.y, 8);
                    mine.z += __shfl_xor_sync(0xffffffffu, mine.z, 8);
                    mine.w += __shfl_xor_sync(0xffffffffu, mine.w, 8);
                }
                if (lane % 16 < C::kCols)
                    *reinterpret_cast<float4*>(sm + C::kRed + ((warp * C::kRound + r) * 2 + (low ? 0 : 1)) * VS + col) = mine;
            }
            __syncthreads();
            const int count = min(C::kRound, m - r0) * 2 * VS;
            for (int i = tid; i < count; i += kStepThreads) {
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < kStepWarps; ++k) sum += sm[C::kRed + k * C::kRound * 2 * VS + i];
                sm[C::kSums + r0 * 2 * VS + i] = sum;
            }
            if (r0 == 0)  // (every decay and product is there)
                for (int i = tid; i < m * TB; i += kStepThreads) {
                    const int t = i / TB, j = i % TB;
                    const bool from = seen[t] >> j & 1;
                    const float far = from || j == t ? sm[C::kFar + i] : 0.f;
                    sm[C::kA + i] = from ? sm[C::kGates + TB + t] * far * sm[C::kA + i] : 0.f;
                    sm[C::kP + i] = from || j == t ? p.scale * far * sm[C::kP + i] : 0.f;
                }
            __syncthreads();
        }
        // u, a column a thread.  (A row takes the rows that it comes from, and no
        // others: 0 times NaN is none of its.)
        if (tid < VS) {
            float u[TB];
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                if (t >= m) break;
                const float beta = sm[C::kGates + TB + t];
                float x = beta * (sm[C::kV + t * VS + tid] - sm[C::kGates + 2 * TB + t] * sm[C::kSums + t * 2 * VS + tid]);
                const uint32_t from = (uint32_t)seen[t];
#pragma unroll
                for (int j = 0; j < t; j += 4) {
                    const float4 a = *reinterpret_cast<const float4*>(sm + C::kA + t * TB + j);
                    if (from >> j & 1) x = fmaf(-a.x, u[j], x);
                    if (j + 1 < t && (from >> (j + 1) & 1)) x = fmaf(-a.y, u[j + 1], x);
                    if (j + 2 < t && (from >> (j + 2) & 1)) x = fmaf(-a.z, u[j + 2], x);
                    if (j + 3 < t && (from >> (j + 3) & 1)) x = fmaf(-a.w, u[j + 3], x);
                }
                u[t] = x;
                sm[C::kSums + t * 2 * VS + tid] = x;
            }
        }
        __syncthreads();
        for (int i = tid; i < m * VS; i += kStepThreads) {
            const int t = i / VS, c = i % VS;
            const float u = sm[C::kSums + 2 * t * VS + c];
            float x = p.scale * sm[C::kGates + 2 * TB + t] * sm[C::kSums + (2 * t + 1) * VS + c];
            const uint32_t from = (uint32_t)seen[t];
#pragma unroll 4
            for (int j = 0; j < t; ++j) {
                const float y = sm[C::kSums + 2 * j * VS + c];
                if (from >> j & 1) x = fmaf(sm[C::kP + t * TB + j], y, x);
            }
            x = fmaf(sm[C::kP + t * TB + t], u, x);
            float* to = p.out + (first + t) * p.out_row_stride + head * d.value_dim + v0 + c;
            if (bc_global(bc, to, 4, p.out, 4 * ((p.rows - 1) * p.out_row_stride + values), kBcDeltaOut)) *to = x;
            if (p.u != nullptr) {
                to = p.u + ((int64_t)(first + t) * d.heads + head) * d.value_dim + v0 + c;
                if (bc_global(bc, to, 4, p.u, 4 * p.rows * values, kBcDeltaU)) *to = u;
            }
        }
        if (p.u == nullptr) {
            const float decay = sm[C::kGates + 2 * TB + m - 1];
#pragma unroll
            for (int i = 0; i < C::kKeys; ++i)
                S[i] = make_float4(decay * S[i].x, decay * S[i].y, decay * S[i].z, decay * S[i].w);
#pragma unroll 2
            for (int j = 0; j < m; ++j) {
                const float far = sm[C::kFar + (m - 1) * TB + j];
                float4 u = *reinterpret_cast<const float4*>(sm + C::kSums + 2 * j * VS + col);
                u = make_float4(far * u.x, far * u.y, far * u.z, far * u.w);
                const float* kj = sm + C::kK + j * C::kPitch + group * C::kKeys;
#pragma unroll
                for (int i = 0; i < C::kKeys; i += 2) {
                    const float2 k2 = *reinterpret_cast<const float2*>(kj + i);
                    axpy(S[i], k2.x, u);
                    axpy(S[i + 1], k2.y, u);
                }
            }
        }
    }
    if (p.u == nullptr) {
#pragma unroll
        for (int i = 0; i < C::kKeys; ++i) {
            float* to = at_s + i * d.value_dim;
            if (bc_global(bc, to, 16, d.s, d.s_extent, kBcDeltaS)) *reinterpret_cast<float4*>(to) = S[i];
        }
    }
}

template <int DK, int VS, int TB>
cudaError_t launch_step(const DeltaRule& p, const DeltaView& d, const BatchView& b, int* err, cudaStream_t stream) {
    using C = StepShape<DK, VS, TB>;
    const cudaError_t e = allow_smem<delta_step_kernel<DK, VS, TB>>(C::kSmem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((int64_t)b.sequences * d.heads * (d.value_dim / VS)));
    return launch_chained(delta_step_kernel<DK, VS, TB>, grid, dim3(kStepThreads), C::kSmem, stream, 1, p, d, b, err);
}

template <int DK, int VS>
cudaError_t launch_rows(const DeltaRule& p, const DeltaView& d, const BatchView& b, int* err, cudaStream_t stream) {
    // Blocks of one row where a sequence has one; a tree is one block.
    if (p.max_rows == 1 || (p.u == nullptr && p.rows <= b.sequences)) return launch_step<DK, VS, 1>(p, d, b, err, stream);
    return p.max_rows <= 8 || (p.u == nullptr && p.rows <= 8 * (int64_t)b.sequences)
               ? launch_step<DK, VS, 8>(p, d, b, err, stream)
               : launch_step<DK, VS, 16>(p, d, b, err, stream);
}

template <int DK>
cudaError_t launch_keys(const DeltaRule& p, const DeltaView& d, const BatchView& b, int* err, int num_sms,
                        cudaStream_t stream) {
    // Slices of 32 columns while that many CTAs find an SM of their own.
    if ((int64_t)b.sequences * d.heads * (d.value_dim / 32) <= 2 * num_sms) return launch_rows<DK, 32>(p, d, b, err, stream);
    return launch_rows<DK, 64>(p, d, b, err, stream);
}

}  // namespace

cudaError_t launch_delta_rule(const DeltaRule& p, const DeltaView& d, const BatchView& b, void* encode, int* err, int num_sms,
                              cudaStream_t stream) {
    // A tree is one block; chains of more than 12 rows on average go in blocks of 64.
    if (p.u != nullptr ? p.max_rows > 16 : p.rows > 12 * (int64_t)b.sequences && p.max_rows > 16)
        return launch_delta_chunk(p, d, b, encode, err, stream);
    return d.key_dim == 64 ? launch_keys<64>(p, d, b, err, num_sms, stream)
                           : launch_keys<128>(p, d, b, err, num_sms, stream);
}

}  // namespace iq4xs
