// colsum.cu -- the second step of a weight's gradient: the blocks' partial
// sums [rows][ld] added up column by column and rounded once to the I/O type.
// What it costs is latency, not bytes: the sums were just written and are read
// from L2.  So a block takes 8 columns and as many warps (8 to 32) as read all
// rows in one trip: a warp reads 16 rows' 32 bytes at a time, 16 bytes a lane,
// four such reads on their way.  This (in place of 32 columns and 32 warps a
// block) and half the partial rows took the gradient of fp32 1023 x 1001 from
// 8.9 to 6.5 us.  Sums of a lane, of the 16 rows' lanes, of the warps: the
// order depends on `rows` alone.
#include "launch_util.h"
#include "rmsnorm_kernels.cuh"

namespace rrn {
namespace {

constexpr int kColsumWarps = 32, kColsumReads = 4, kColsumCols = 8;   // warps: at most

template <typename T>
__global__ void __launch_bounds__(32 * kColsumWarps)
colsum_kernel(const float *partial, int rows0, int rows1, int64_t cols, int64_t ld, void *out0, void *out1) {
    __shared__ float part[kColsumWarps][kColsumCols];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int rows = blockIdx.y ? rows1 : rows0;
    if (blockIdx.y) partial += (int64_t)rows0 * ld;
    void *out = blockIdx.y ? out1 : out0;
    const int64_t col = (int64_t)blockIdx.x * kColsumCols + (lane % 2) * 4;   // of the lane's four
    const int step = 16 * warps;                                             // rows a read of the block
    const int first = warp * 16 + lane / 2;
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < ld) {   // ld is a multiple of 4; columns cols .. ld - 1 are not written out
        for (int r = first; r < rows; r += kColsumReads * step) {
            float4 v[kColsumReads];
#pragma unroll
            for (int j = 0; j < kColsumReads; ++j) {
                const int row = r + j * step;
                v[j] = row < rows ? *reinterpret_cast<const float4 *>(partial + (int64_t)row * ld + col)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int j = 0; j < kColsumReads; ++j) {
                sum.x += v[j].x;
                sum.y += v[j].y;
                sum.z += v[j].z;
                sum.w += v[j].w;
            }
        }
    }
    float s[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int off = 2; off < 32; off <<= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], off);
        if (lane < 2) part[warp][lane * 4 + k] = s[k];
    }
    __syncthreads();
    // eight threads a column, then their sums
    if (threadIdx.x < 8 * kColsumCols) {
        const int c = threadIdx.x / 8;
        float v = 0.f;
        for (int w = threadIdx.x % 8; w < warps; w += 8) v += part[w][c];
        v = butterfly_sum<8>(v);
        const int64_t mine = (int64_t)blockIdx.x * kColsumCols + c;
        if (threadIdx.x % 8 == 0 && mine < cols) st_scalar(out, mine, v, T{});
    }
}

}  // namespace

int launch_colsum(const float *partial, int rows0, int rows1, int64_t cols, int64_t ld, void *out0, void *out1,
                  int dtype, rmsnorm_stream_t stream) {
    void *argv[] = {&partial, &rows0, &rows1, &cols, &ld, &out0, &out1};
    const void *fn = dtype == RMSNORM_BF16 ? reinterpret_cast<const void *>(&colsum_kernel<BF16>)
                                           : reinterpret_cast<const void *>(&colsum_kernel<F32>);
    const int rows = rows0 > rows1 ? rows0 : rows1;
    int warps = 8;
    while (warps < kColsumWarps && rows > 16 * kColsumReads * warps) warps *= 2;
    return launch_kernel(fn, dim3((unsigned)div_up(cols, kColsumCols), out1 != nullptr ? 2 : 1), 32 * warps, 0, stream,
                         argv);
}

}  // namespace rrn
