// delta_commit.cu -- the recurrent layers' states along an accepted path.
//
//   S <- G S + sum_i D_i k_i u_i^T,   D_i = e^(sum of g behind i), G = e^(sum of g)
//
// over the path's rows, in every layer; the convolution's inputs become the
// path's last three.  The rows' k and u are small beside S, which is read once
// and written once: HBM bounds it.  A CTA takes 64 columns of one head of one
// sequence and layer, S in registers; paths of more than kPath rows go in runs.
// 24 layers x 12 sequences x 48 heads of 128 x 128, paths of 5: 306 to 311 us, 6.1 TB/s, 90 % of a
// copy.  Five CTAs an SM keep enough loads in flight (four: 351 us, three 353; six
// spill, 367; slices of 32 columns 381 and more: rows of 128 bytes).  One sequence, four
// layers: 4.7 us, a launch and the chain accepted - path - gates - S.
#include "delta.cuh"

namespace iq4xs {
namespace {

constexpr int kCommitThreads = 256;
constexpr int kPath = 16;  // rows of a path at a time

struct CommitParams {
    const uint16_t* k;
    const float* g;
    const float* u;
    const float* x;
    int64_t k_row_stride, k_layer_stride, g_layer_stride, u_layer_stride, x_row_stride, x_layer_stride;
    const int32_t* paths;
    const int32_t* accepted;
    int path_width, rows, bf16, conv_parts;
};

template <int DK, int DV>
__global__ void __launch_bounds__(kCommitThreads, 5) delta_commit_kernel(const CommitParams p, const DeltaView d,
                                                                      const BatchView b, int* err) {
    constexpr int VS = 64, kCols = VS / 4, kGroups = kCommitThreads / kCols, kKeys = DK / kGroups;
    __shared__ __align__(16) float k_at[kPath][DK];
    __shared__ __align__(16) float u_at[kPath][VS];
    __shared__ int row_at[kPath];
    __shared__ float g_at[kPath], decay[kPath + 1];
    griddep_launch_dependents();
    griddep_wait();
    const Bc bc = bc_open(err);
    constexpr int kSlices = DV / VS;
    const int parts = d.heads * kSlices + p.conv_parts, tid = threadIdx.x;
    const int part = blockIdx.x % parts, s = blockIdx.x / parts % b.sequences, layer = blockIdx.x / parts / b.sequences;
    const int count = p.accepted[s];
    const DeltaSequence seq = delta_sequence(b, d, s, p.rows, err);
    const int row0 = seq.first, n = seq.n, len = seq.len, slot = seq.slot;
    if (len < 0 || slot < 0) return;
    if (count < 0 || count > p.path_width || count > n) {
        if (tid == 0) data_error(err, kDataPath);
        return;
    }
    if (count == 0) return;
    // S is asked for first: what comes behind the path's checks hides under it.
    const bool moves_s = part < d.heads * kSlices;
    const int head = part / kSlices, v0 = part % kSlices * VS, key_head = head / (d.heads / d.key_heads);
    const int col = tid % kCols * 4, group = tid / kCols;
    float* const at_s = d.s + layer * d.s_layer_stride + slot * d.s_slot_stride +
                        ((int64_t)head * DK + group * kKeys) * DV + v0 + col;
    float4 S[kKeys];
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
        S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (moves_s && len > 0 && bc_global(bc, at_s + i * DV, 16, d.s, d.s_extent, kBcDeltaS))
            S[i] = __ldcs(reinterpret_cast<const float4*>(at_s + i * DV));
    }
    const int32_t* path = p.paths + (int64_t)s * p.path_width;
    const int64_t path_extent = 4 * (int64_t)b.sequences * p.path_width;
    bool bad = false;
    for (int i = tid; i < count; i += kCommitThreads) {
        if (!bc_global(bc, path + i, 4, p.paths, path_extent, kBcDeltaPath)) {
            bad = true;
            continue;
        }
        const int t = path[i];
        bad |= t < 0 || t >= n || (i > 0 && t <= path[i - 1]);
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) data_error(err, kDataPath);
        return;
    }
    if (!moves_s) {
        // The last three inputs: of the path, and before it of the state.
        float* const at = d.conv + layer * d.conv_layer_stride + slot * d.conv_slot_stride;
        const float* x = p.x + layer * p.x_layer_stride;
        const int64_t extent = 4 * ((d.layers - 1) * p.x_layer_stride + (p.rows - 1) * p.x_row_stride + d.channels);
        const int c = 4 * ((part - d.heads * kSlices) * kCommitThreads + tid);
        if (c >= d.channels) return;
        float4 in[kConvTaps - 1];
#pragma unroll
        for (int i = 0; i < kConvTaps - 1; ++i) {
            const int on = count - (kConvTaps - 1) + i;  // place on the path
            in[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (on >= 0) {
                const float* from = x + (row0 + path[on]) * p.x_row_stride + c;
                if (bc_global(bc, from, 16, p.x, extent, kBcDeltaX)) in[i] = *reinterpret_cast<const float4*>(from);
            } else if (len > 0) {
                const float* from = at + (int64_t)(on + kConvTaps - 1) * d.channels + c;
                if (bc_global(bc, from, 16, d.conv, d.conv_extent, kBcDeltaConv))
                    in[i] = *reinterpret_cast<const float4*>(from);
            }
        }
#pragma unroll
        for (int i = 0; i < kConvTaps - 1; ++i) {
            float* to = at + (int64_t)i * d.channels + c;
            if (bc_global(bc, to, 16, d.conv, d.conv_extent, kBcDeltaConv)) *reinterpret_cast<float4*>(to) = in[i];
        }
        return;
    }
    const int64_t k_extent = 2 * ((d.layers - 1) * p.k_layer_stride + (p.rows - 1) * p.k_row_stride +
                                  (int64_t)d.key_heads * DK);
    const int64_t g_extent = 4 * ((d.layers - 1) * p.g_layer_stride + (int64_t)p.rows * d.heads);
    const int64_t u_extent = 4 * ((d.layers - 1) * p.u_layer_stride + (int64_t)p.rows * d.heads * DV);
    for (int i0 = 0; i0 < count; i0 += kPath) {
        const int m = min(kPath, count - i0);
        if (i0 > 0) __syncthreads();  // the last run has been used
        if (tid < m) {
            const int row = row0 + path[i0 + tid];
            const float* from = p.g + layer * p.g_layer_stride + (int64_t)row * d.heads + head;
            row_at[tid] = row;
            g_at[tid] = bc_global(bc, from, 4, p.g, g_extent, kBcDeltaGate) ? *from : 0.f;
        }
        __syncthreads();
        for (int i = tid; i < m * (DK / 8); i += kCommitThreads) {
            const int c = i % (DK / 8) * 8, t = i / (DK / 8);
            const uint16_t* from = p.k + layer * p.k_layer_stride + row_at[t] * p.k_row_stride + key_head * DK + c;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (bc_global(bc, from, 16, p.k, k_extent, kBcDeltaQkv)) w = *reinterpret_cast<const uint4*>(from);
            unpack8(p.bf16, w, &k_at[t][c]);
        }
        for (int i = tid; i < m * kCols; i += kCommitThreads) {
            const int c = i % kCols * 4, t = i / kCols;
            const float* from = p.u + layer * p.u_layer_stride + ((int64_t)row_at[t] * d.heads + head) * DV + v0 + c;
            float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
            if (bc_global(bc, from, 16, p.u, u_extent, kBcDeltaU)) w = *reinterpret_cast<const float4*>(from);
            *reinterpret_cast<float4*>(&u_at[t][c]) = w;
        }
        if (tid <= m) {  // decay behind row tid - 1; 0: of S
            float sum = 0.f;
            for (int i = m - 1; i >= tid; --i) sum += g_at[i];
            decay[tid] = expf(sum);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kKeys; ++i)
            S[i] = make_float4(decay[0] * S[i].x, decay[0] * S[i].y, decay[0] * S[i].z, decay[0] * S[i].w);
        for (int t = 0; t < m; ++t) {
            const float f = decay[t + 1];
            float4 u = *reinterpret_cast<const float4*>(&u_at[t][col]);
            u = make_float4(f * u.x, f * u.y, f * u.z, f * u.w);
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                const float k = k_at[t][group * kKeys + i];
                S[i].x = fmaf(k, u.x, S[i].x);
                S[i].y = fmaf(k, u.y, S[i].y);
                S[i].z = fmaf(k, u.z, S[i].z);
                S[i].w = fmaf(k, u.w, S[i].w);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kKeys; ++i)
        if (bc_global(bc, at_s + i * DV, 16, d.s, d.s_extent, kBcDeltaS))
            __stcs(reinterpret_cast<float4*>(at_s + i * DV), S[i]);
}

template <int DK, int DV>
cudaError_t launch(const CommitParams& p, const DeltaView& d, const BatchView& b, int* err, cudaStream_t stream) {
    const int64_t blocks = (int64_t)d.layers * b.sequences * (d.heads * (DV / 64) + p.conv_parts);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    return launch_chained(delta_commit_kernel<DK, DV>, dim3((unsigned)blocks), dim3(kCommitThreads), 0, stream, 1, p, d,
                          b, err);
}

}  // namespace

cudaError_t launch_delta_commit(const iq4xs_delta_commit_args& a, const DeltaView& d, const BatchView& b, int* err,
                                cudaStream_t stream) {
    CommitParams p;
    const bool one = d.layers == 1;
    p.k = static_cast<const uint16_t*>(a.k);
    p.g = a.g;
    p.u = a.u;
    p.x = a.x;
    p.k_row_stride = a.k_row_stride;
    p.k_layer_stride = one ? 0 : a.k_layer_stride;
    p.g_layer_stride = one ? 0 : a.g_layer_stride;
    p.u_layer_stride = one ? 0 : a.u_layer_stride;
    p.x_row_stride = a.x_row_stride;
    p.x_layer_stride = one ? 0 : a.x_layer_stride;
    p.paths = a.paths;
    p.accepted = a.accepted;
    p.path_width = (int)a.path_width;
    p.rows = (int)a.rows;
    p.bf16 = a.dtype == IQ4XS_KV_BF16;
    p.conv_parts = a.x != nullptr ? (d.channels + 4 * kCommitThreads - 1) / (4 * kCommitThreads) : 0;
    if (d.key_dim == 64)
        return d.value_dim == 64 ? launch<64, 64>(p, d, b, err, stream) : launch<64, 128>(p, d, b, err, stream);
    return d.value_dim == 64 ? launch<128, 64>(p, d, b, err, stream) : launch<128, 128>(p, d, b, err, stream);
}

}  // namespace iq4xs
