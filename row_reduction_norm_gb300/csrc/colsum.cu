// colsum.cu -- the second step of a weight's gradient: the blocks' partial
// sums [rows][cols] added up column by column and rounded once to the I/O
// type.  32 columns a block (a warp reads 128 consecutive bytes of a row), 32
// warps that take every 32nd row, four running sums a thread, then a fixed
// tree over the warps through shared memory: the order depends on `rows`
// alone.  The partial sums were just written, so they are read from L2.
#include "launch_util.h"
#include "rmsnorm_kernels.cuh"

namespace rrn {
namespace {

constexpr int kColsumWarps = 32;

template <typename T>
__global__ void __launch_bounds__(32 * kColsumWarps)
colsum_kernel(const float *partial, int rows0, int rows1, int64_t cols, void *out0, void *out1) {
    __shared__ float part[kColsumWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + lane;
    const int rows = blockIdx.y ? rows1 : rows0;
    if (blockIdx.y) partial += (int64_t)rows0 * cols;
    void *out = blockIdx.y ? out1 : out0;
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (col < cols) {
        for (int r = warp; r < rows; r += 4 * kColsumWarps) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (r + j * kColsumWarps < rows) v[j] += partial[(int64_t)(r + j * kColsumWarps) * cols + col];
        }
    }
    part[warp][lane] = tree_sum(v);
    __syncthreads();
    // warp w adds up column w of the block
    const int64_t mine = (int64_t)blockIdx.x * 32 + warp;
    const float s = butterfly_sum<32>(part[lane][warp]);
    if (lane == 0 && mine < cols) st_scalar(out, mine, s, T{});
}

}  // namespace

int launch_colsum(const float *partial, int rows0, int rows1, int64_t cols, void *out0, void *out1, int dtype,
                  rmsnorm_stream_t stream) {
    void *argv[] = {&partial, &rows0, &rows1, &cols, &out0, &out1};
    const void *fn = dtype == RMSNORM_BF16 ? reinterpret_cast<const void *>(&colsum_kernel<BF16>)
                                           : reinterpret_cast<const void *>(&colsum_kernel<F32>);
    return launch_kernel(fn, dim3((unsigned)div_up(cols, 32), out1 != nullptr ? 2 : 1), 32 * kColsumWarps, 0, stream, argv);
}

}  // namespace rrn
