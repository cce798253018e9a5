// What the library's other translation units use of the GEMM's host side
// (defined in gemm_f16.cu): the device check, the memory check, the tensor-map
// encoder, the process-wide options and the device status word.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "gemm_f16.h"

namespace gemm_f16_host {

struct Device {
    int sms = 0;
    int* status = nullptr;   // device status word (gemm_f16_device_status)
};

// The current device, GEMM_F16_ERR_UNSUPPORTED_DEVICE unless it is a GB300.
gemm_f16_status current_device(Device* out);

// [p, p + bytes) is device or managed memory of the current device inside one
// allocation.
bool device_range_ok(const void* p, int64_t bytes);

// Span of a strided view in elements (false on overflow); `batch` copies of a
// view of `e` elements `stride` apart.
bool view_extent(int64_t rows, int64_t cols, int64_t s_r, int64_t s_c, int64_t* elems);
bool batch_extent(int64_t e, int64_t n, int64_t stride, int64_t* total);

inline bool overlaps(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + static_cast<uintptr_t>(b_bytes) && y < x + static_cast<uintptr_t>(a_bytes);
}

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// GEMM_F16_OPT_* values (0: default), and the bounded waits' limit.
int64_t option(int o);
uint64_t timeout_ns();

// Launch `kernel` on `stream` with the cluster size (1: none) and, unless
// GEMM_F16_OPT_PDL is 1, as a programmatic dependent of the kernel before it.
template <typename... Params, typename... Args>
gemm_f16_status launch_kernel(void (*kernel)(Params...), dim3 grid, unsigned block, size_t smem, int cluster,
                              cudaStream_t stream, const Args&... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    int n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (option(GEMM_F16_OPT_PDL) != 1) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = static_cast<unsigned>(n);
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_F16_ERR_LAUNCH;
    }
    return GEMM_F16_OK;
}

}  // namespace gemm_f16_host
