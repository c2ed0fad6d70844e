// launch_util.h -- what the entry points of the operators beside the norm
// share (internal): the per-device caches of rmsnorm_api.cu and small host
// helpers.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "rmsnorm.h"

namespace rrn {

// The current device and its SM count.  A status (RMSNORM_OK or RMSNORM_ECUDA).
int current_device_sms(int *dev, int *sms);
// Resident blocks a SM of a kernel (cached per device, kernel and shared memory).
int resident_blocks(int dev, const void *fn, int block, size_t smem, int *blocks);

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline int size_of(int dtype) { return dtype == RMSNORM_BF16 ? 2 : 4; }

inline bool on_boundary(const void *p, int64_t bytes) {
    return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0;
}

// Launch with programmatic stream serialisation (every kernel of the library
// waits for the work before it through griddepcontrol before it touches memory).
// cluster: blocks of a thread-block cluster.
inline int launch_kernel(const void *fn, dim3 grid, int block, size_t smem, rmsnorm_stream_t stream, void **argv,
                         int cluster = 1) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelExC(&cfg, fn, argv) != cudaSuccess) {
        (void)cudaGetLastError();   // clear the non-sticky launch error
        return RMSNORM_ECUDA;
    }
    return RMSNORM_OK;
}

// Opt a kernel in to 226 KB of dynamic shared memory (cached per device and kernel).
int allow_smem(int dev, const void *fn);
// Dynamic shared memory for which that is needed: the limit without it is 48 KB
// together with a kernel's static arrays, 1 KB of them at most.
constexpr size_t kSmemUnasked = 47 * 1024;

// Sums of the columns of partial[rows0 + rows1][ld] into the I/O type: of the
// first rows0 rows to out0, of the rest to out1 (nullable).  partial is 16-byte
// aligned, ld a multiple of 4 (what stands past the cols columns of a row must
// be readable; it is not used).  colsum.cu.
int launch_colsum(const float *partial, int rows0, int rows1, int64_t cols, int64_t ld, void *out0, void *out1,
                  int dtype, rmsnorm_stream_t stream);

}  // namespace rrn
