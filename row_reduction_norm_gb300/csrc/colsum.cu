// colsum.cu -- the second step of a weight's gradient: the blocks' partial
// sums [rows][ld] added up column by column and rounded once to the I/O type.
// A block takes 32 columns with 32 warps; a warp reads four rows' 128 bytes at
// a time, 16 bytes a lane, up to eight such reads on their way: 1024 rows in
// one trip to L2, where the sums were just written.  It takes 4 to 6 us by
// itself, most of it launch and latency, and half of that as the dependent
// launch it is.  Sums of a lane, of the four rows' lanes, of the warps: the order
// depends on `rows` alone.
#include "launch_util.h"
#include "rmsnorm_kernels.cuh"

namespace rrn {
namespace {

constexpr int kColsumWarps = 32, kColsumReads = 8;

template <typename T>
__global__ void __launch_bounds__(32 * kColsumWarps)
colsum_kernel(const float *partial, int rows0, int rows1, int64_t cols, int64_t ld, void *out0, void *out1) {
    __shared__ float part[kColsumWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rows = blockIdx.y ? rows1 : rows0;
    if (blockIdx.y) partial += (int64_t)rows0 * ld;
    void *out = blockIdx.y ? out1 : out0;
    const int64_t col = (int64_t)blockIdx.x * 32 + (lane % 8) * 4;   // of the lane's four
    const int first = warp * 4 + lane / 8;                          // row
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < ld) {   // ld is a multiple of 4; columns cols .. ld - 1 are not written out
        for (int r = first; r < rows; r += kColsumReads * 4 * kColsumWarps) {
            float4 v[kColsumReads];
#pragma unroll
            for (int j = 0; j < kColsumReads; ++j) {
                const int row = r + j * 4 * kColsumWarps;
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
        s[k] += __shfl_xor_sync(0xffffffffu, s[k], 8);
        s[k] += __shfl_xor_sync(0xffffffffu, s[k], 16);
        if (lane < 8) part[warp][lane * 4 + k] = s[k];
    }
    __syncthreads();
    // warp w adds up column w of the block
    const int64_t mine = (int64_t)blockIdx.x * 32 + warp;
    const float total = butterfly_sum<32>(part[lane][warp]);
    if (lane == 0 && mine < cols) st_scalar(out, mine, total, T{});
}

}  // namespace

int launch_colsum(const float *partial, int rows0, int rows1, int64_t cols, int64_t ld, void *out0, void *out1,
                  int dtype, rmsnorm_stream_t stream) {
    void *argv[] = {&partial, &rows0, &rows1, &cols, &ld, &out0, &out1};
    const void *fn = dtype == RMSNORM_BF16 ? reinterpret_cast<const void *>(&colsum_kernel<BF16>)
                                           : reinterpret_cast<const void *>(&colsum_kernel<F32>);
    return launch_kernel(fn, dim3((unsigned)div_up(cols, 32), out1 != nullptr ? 2 : 1), 32 * kColsumWarps, 0, stream,
                         argv);
}

}  // namespace rrn
