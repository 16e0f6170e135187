// cache.cuh -- the paged key/value cache and its batch as kernels see them
// (layouts: include/iq4xs.h), with the checks of the values that they read
// from device memory.  Shared by the append, attention and page kernels.
#pragma once

#include <cuda_bf16.h>

#include <atomic>

#include "../../include/iq4xs.h"
#include "internal.cuh"

namespace iq4xs {

struct CacheView {
    uint16_t* k;  // 16-bit elements of either type
    uint16_t* v;
    int64_t layer_stride, page_stride, head_stride, slot_stride;  // elements
    int64_t extent;  // bytes from the first element to behind the last
    int layers, pages, heads, page_size, page_shift, head_dim;
};

struct BatchView {
    const int32_t* row_offsets;
    int32_t* lens;
    int32_t* held;
    int32_t* page_table;
    int64_t table_stride;
    int table_width, sequences;
};

__device__ __forceinline__ void data_error(int* err, int site) { atomicCAS(err, 0, kDevErrData + site); }

// Rows [*first, *first + n) of sequence s among `rows`; n = 0 where the
// offsets are out of order or out of range.
__device__ __forceinline__ int batch_rows(const BatchView& b, int s, int64_t rows, int* first, int* err) {
    const int a = b.row_offsets[s], e = b.row_offsets[s + 1];
    *first = a;
    if (a < 0 || e < a || e > rows) {
        data_error(err, kDataOffsets);
        return 0;
    }
    return e - a;
}
// Cached tokens of sequence s; -1 where its length is out of range.
__device__ __forceinline__ int batch_len(const BatchView& b, int s, int* err) {
    const int n = b.lens[s];
    if (n < 0) data_error(err, kDataLens);
    return n < 0 ? -1 : n;
}
// The page of position p of sequence s, -1 (recorded) where s holds none.
__device__ __forceinline__ int page_of(const CacheView& c, const BatchView& b, int s, int p, int* err) {
    const int j = p >> c.page_shift;
    int page = -1;
    if (j < b.table_width && j < b.held[s]) page = b.page_table[s * b.table_stride + j];
    if (page < 0 || page >= c.pages) {
        data_error(err, kDataPage);
        return -1;
    }
    return page;
}

// fp32 <-> the cache's 16-bit types (RNE).
struct KvF16 {
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ uint32_t pack_rz(float lo, float hi) {  // cut off
        uint32_t w;
        asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
        return w;
    }
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
};
struct KvBf16 {
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
    }
};

// Host-side launchers (csrc/append.cu, csrc/cache_pages.cu, csrc/attention*.cu);
// arguments are checked by the callers in csrc/cache_api.cu.
cudaError_t launch_qk_norm_rope(const iq4xs_qk_norm_rope_args& a, const CacheView& c, const BatchView& b, bool bf16,
                                int* err, int num_sms, cudaStream_t stream);
cudaError_t launch_cache_reserve(const BatchView& b, int page_size, int32_t* refs, int pages, int32_t* status, int* err,
                                 cudaStream_t stream);
cudaError_t launch_cache_commit(const CacheView& c, const BatchView& b, int32_t* refs, const int32_t* paths,
                                int path_width, const int32_t* accepted, int32_t* new_lens, int* err,
                                cudaStream_t stream);
cudaError_t launch_cache_fork(const CacheView& c, const BatchView& b, int32_t* refs, const int32_t* parents,
                              const int32_t* children, int count, int32_t* status, int* err, cudaStream_t stream);
cudaError_t launch_cache_release(const BatchView& b, int32_t* refs, int pages, const int32_t* rows, int count,
                                 int* err, cudaStream_t stream);
cudaError_t launch_cache_copy_pages(const CacheView& c, const int32_t* src, const int32_t* dst, int count, int* err,
                                    cudaStream_t stream);
cudaError_t launch_tree_attention(const iq4xs_tree_attention_args& a, const CacheView& c, const BatchView& b, bool bf16,
                                  void* encode, int* err, int num_sms, int skip_stage, cudaStream_t stream);
int64_t tree_attention_workspace(int64_t rows, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t sequences,
                                 int num_sms);

// Dynamic shared memory of a kernel, once per device.
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// One launch with the library's programmatic dependent launch setting, in
// clusters of `cluster` CTAs (1: none).
template <typename... KArgs, typename... Args>
cudaError_t launch_chained(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                           int cluster, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace iq4xs
