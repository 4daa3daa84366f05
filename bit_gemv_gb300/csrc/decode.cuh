// Shared by the decode-step operators: division by a run-time constant, the
// element types of caches, the checks of a cache description and the launch
// with programmatic dependent launch.
#pragma once

#include <cmath>
#include <cstdint>

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "async.cuh"
#include "common.h"
#include "device.cuh"
#include "ninfer_decode.h"

namespace ninfer {

// Exact n / d for every 32-bit n with one multiplication (Granlund and
// Montgomery, "Division by invariant integers using multiplication", 1994,
// figure 4.1): with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1,
// t = hi32(m n), n / d = (t + ((n - t) >> min(l, 1))) >> max(l - 1, 0).
struct FastDiv {
    uint32_t d, m, sh1, sh2;
    FastDiv() = default;
    explicit FastDiv(uint32_t div) : d(div) {
        uint32_t l = 0;
        while (l < 32 && (1ull << l) < div) ++l;
        m = (uint32_t)((((1ull << l) - div) << 32) / div + 1);
        sh1 = l < 1 ? l : 1;
        sh2 = l > 1 ? l - 1 : 0;
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        const uint32_t t = __umulhi(m, n);
        return (t + ((n - t) >> sh1)) >> sh2;
    }
};

inline bool cache_dtype_valid(int dt) { return dt == NINFER_BF16 || dt == NINFER_F16 || dt == NINFER_E4M3; }
inline uint32_t cache_dtype_size(int dt) { return dt == NINFER_E4M3 ? 1 : 2; }

// The rules of ninfer_kv_cache; `who` begins the error message.
int check_cache(const ninfer_kv_cache *c, const char *who);

// Launch with programmatic dependent launch, in clusters of `cluster` CTAs: the
// kernel calls pdl_wait() before it touches memory.
template <class... P, class... A>
int launch_clusters(const char *who, unsigned cluster, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                    cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) return fail(NINFER_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
    return NINFER_OK;
}

template <class... P, class... A>
int launch_dependent(const char *who, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                     A... args) {
    return launch_clusters(who, 1, kernel, grid, block, smem, stream, args...);
}

}  // namespace ninfer
