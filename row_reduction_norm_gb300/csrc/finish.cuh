// finish.cuh -- the second step of a weight's gradient within the launch that
// makes the partial sums, where its blocks are few enough to be one cluster:
// behind a cluster barrier the blocks add the columns up between them, in the
// order of the blocks.  It saves the column sums' launch: half a microsecond of
// the device's time and two of the host's, which such calls wait for (dropout
// gradient bf16 25 x 192 6.4 -> 4.4 us a call, a rotary one of 6 tokens x 8
// heads 10.5 -> 6.1 us).
#pragma once

#include "rmsnorm_kernels.cuh"

namespace rrn {

// Blocks of a gradient at most that are launched as one cluster (the portable size).
constexpr int kFinishBlocks = 8;

// Sums of partial[rows][ld], written by the blocks of this cluster before
// behind_the_cluster(), by `threads` threads of which this is number `first`.
template <typename T>
__device__ __forceinline__ void finish_columns(const float *partial, int rows, int64_t ld, int cols, void *out, int first,
                                               int threads) {
    for (int c = first; c < cols; c += threads) {
        float v[kFinishBlocks];
#pragma unroll
        for (int r = 0; r < kFinishBlocks; ++r) v[r] = r < rows ? __ldcg(partial + r * ld + c) : 0.f;
        st_scalar(out, c, tree_sum(v), T{});
    }
}

__device__ __forceinline__ void behind_the_cluster() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

}  // namespace rrn
