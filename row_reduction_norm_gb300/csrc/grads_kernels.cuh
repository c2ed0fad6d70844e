// grads_kernels.cuh -- the norm of many tensors together, and their clipping:
// norm = sqrt(sum g^2), out = RN(g min(1, max_norm / norm)).
//
// Two launches over the same blocks of 32 KB: sums of squares, then the
// scaling, whose blocks each add up the first launch's partial sums for
// themselves (a few thousand bytes from L2) rather than wait for a launch in
// between.  HBM bandwidth bounds both: every byte is read twice and written
// once.  The scaling goes through the blocks from the last to the first: what
// the norm read last is still in L2.
//
// The tensors' addresses travel as the launch's parameters (up to 32 KB of
// them), so nothing is copied to the device beforehand and a captured call
// replays by itself.
#pragma once

#include "rmsnorm_kernels.cuh"

namespace rrn {

constexpr int kGradThreads = 256, kGradWarps = kGradThreads / 32, kGradChunks = 8;
constexpr int kGradBlock = kGradThreads * kGradChunks * 16;   // bytes of a block of elements
constexpr int kGradPartials = 2048;                           // blocks of the norm's launches at most

// A tensor of a launch: its blocks are first .. the next one's first - 1, cut at
// multiples of 32 KB behind the 16-byte boundary at or before its start.
struct GradEntry {
    const char *grad;
    char *out;
    int64_t count;
    uint32_t first;
    int32_t dtype;
};

// Most tensors of a launch: 32,764 bytes of parameters.
constexpr int kGradSmall = 40, kGradMost = 1020;

template <int CAP>
struct GradTable {
    double *partial;    // of this call, [kGradPartials]
    float *norm;
    int32_t n;          // entries here
    uint32_t blocks;    // of elements, here
    int32_t slot;       // first partial sum of this launch
    int32_t sums;       // partial sums of the whole call
    float max_norm;
    int32_t write_norm;
    GradEntry e[CAP];
};

// The entry that holds block `b`.
template <int CAP>
__device__ __forceinline__ int entry_of(const GradTable<CAP> &t, uint32_t b) {
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.e[mid].first <= b) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// A 16-byte chunk of a tensor on its 16-byte boundaries; what of it lies
// outside the tensor is zero and not read.  i: its first element, maybe negative.
template <typename T>
__device__ __forceinline__ Chunk grad_chunk(const char *grad, int64_t i, int64_t count) {
    constexpr int V = T::kVec, E = 16 / V;
    if (i >= 0 && i + V <= count) return ld_keep_l2_16(grad + i * E);
    Chunk c;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (V == 8) {
            const int64_t a = i + 2 * k, b = a + 1;
            const uint32_t lo = a >= 0 && a < count ? reinterpret_cast<const uint16_t *>(grad)[a] : 0u;
            const uint32_t hi = b >= 0 && b < count ? reinterpret_cast<const uint16_t *>(grad)[b] : 0u;
            c.u[k] = lo | hi << 16;
        } else {
            const int64_t a = i + k;
            c.u[k] = a >= 0 && a < count ? reinterpret_cast<const uint32_t *>(grad)[a] : 0u;
        }
    }
    return c;
}

// Elements before the boundary: the first chunk's place is minus these.
template <typename T>
__device__ __forceinline__ int64_t grad_head(const char *grad) {
    return (int64_t)((reinterpret_cast<uintptr_t>(grad) & 15) / (16 / T::kVec));
}

// Sum of the squares of the thread's chunks of a block, each element times
// `scale` (a power of two) first.
template <typename T>
__device__ __forceinline__ float block_squares(const char *grad, int64_t count, uint32_t block, float scale) {
    constexpr int V = T::kVec;
    const int64_t first = ((int64_t)block * kGradThreads * kGradChunks + threadIdx.x) * V - grad_head<T>(grad);
    Chunk c[kGradChunks];
#pragma unroll
    for (int j = 0; j < kGradChunks; ++j) c[j] = grad_chunk<T>(grad, first + (int64_t)j * kGradThreads * V, count);
    float acc[V] = {};
#pragma unroll
    for (int j = 0; j < kGradChunks; ++j) {
        float x[V];
        unpack(c[j], x, T{});
#pragma unroll
        for (int k = 0; k < V; ++k) x[k] *= scale;
        sq_accumulate(x, acc);
    }
    return tree_sum(acc);
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// The block's threads' values added up, for every thread.
__device__ __forceinline__ double block_sum(double v, double (&part)[kGradWarps]) {
    v = warp_sum(v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    double s = 0.;
#pragma unroll
    for (int w = 0; w < kGradWarps; ++w) s += part[w];
    return s;
}

// Squares of all the blocks this one takes, as fp32 sums of 64 or fewer
// squares, those added up in two parts (a sum and what its roundings lost).
template <int CAP>
__device__ __forceinline__ double grid_squares(const GradTable<CAP> &t, float scale, double back, double (&part)[kGradWarps]) {
    float sum = 0.f, lost = 0.f;
    for (uint32_t b = blockIdx.x; b < t.blocks; b += gridDim.x) {
        const GradEntry &e = t.e[entry_of(t, b)];
        const float v = e.dtype == 1 ? block_squares<BF16>(e.grad, e.count, b - e.first, scale)
                                     : block_squares<F32>(e.grad, e.count, b - e.first, scale);
        const float s = sum + v, w = s - sum;
        lost += (sum - (s - w)) + (v - w);
        sum = s;
    }
    // an infinite sum has lost nothing that can be said
    const double both = isfinite(sum) ? (double)sum + (double)lost : (double)sum;
    return block_sum(both, part) * back;
}

template <int CAP>
__global__ void __launch_bounds__(kGradThreads) grad_squares_kernel(const __grid_constant__ GradTable<CAP> t) {
    __shared__ double part[kGradWarps];
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    double s = grid_squares(t, 1.f, 1., part);
    // Squares past fp32's range, above or below (2^-80: sums so small that
    // squares of 2^-126 count): once more, scaled by a power of two.  All
    // threads of a block see the same sum.
    if (!(s <= 1.7e308) || isinf(s)) s = grid_squares(t, 0x1p-80f, 0x1p160, part);
    else if (s < 0x1p-80) s = grid_squares(t, 0x1p80f, 0x1p-160, part);
    if (threadIdx.x == 0) t.partial[t.slot + blockIdx.x] = s;
}

// The norm from the partial sums, the same in every block that asks.
template <int CAP>
__device__ __forceinline__ double norm_of(const GradTable<CAP> &t, double (&part)[kGradWarps]) {
    double s = 0.;
    for (int i = threadIdx.x; i < t.sums; i += kGradThreads) s += __ldcg(t.partial + i);
    return sqrt(block_sum(s, part));
}

template <int CAP>
__global__ void __launch_bounds__(kGradThreads) grad_norm_kernel(const __grid_constant__ GradTable<CAP> t) {
    __shared__ double part[kGradWarps];
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    const double norm = norm_of(t, part);
    if (threadIdx.x == 0) *t.norm = (float)norm;
}

template <typename T>
__device__ __forceinline__ void scale_block(const GradEntry &e, uint32_t block, float f) {
    constexpr int V = T::kVec, E = 16 / V;
    const int64_t head = grad_head<T>(e.grad);
    const int64_t first = ((int64_t)block * kGradThreads * kGradChunks + threadIdx.x) * V - head;
    const bool alike = ((reinterpret_cast<uintptr_t>(e.grad) ^ reinterpret_cast<uintptr_t>(e.out)) & 15) == 0;
    Chunk c[kGradChunks];
#pragma unroll
    for (int j = 0; j < kGradChunks; ++j) c[j] = grad_chunk<T>(e.grad, first + (int64_t)j * kGradThreads * V, e.count);
#pragma unroll
    for (int j = 0; j < kGradChunks; ++j) {
        const int64_t i = first + (int64_t)j * kGradThreads * V;
        float x[V];
        unpack(c[j], x, T{});
#pragma unroll
        for (int k = 0; k < V; ++k) x[k] *= f;
        if (alike && i >= 0 && i + V <= e.count) {
            st16(e.out + i * E, pack(x, T{}));
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (i + k >= 0 && i + k < e.count) st_scalar(e.out, i + k, x[k], T{});
        }
    }
}

template <int CAP>
__global__ void __launch_bounds__(kGradThreads) grad_scale_kernel(const __grid_constant__ GradTable<CAP> t) {
    __shared__ double part[kGradWarps];
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    const double norm = norm_of(t, part);
    if (t.write_norm && blockIdx.x == 0 && threadIdx.x == 0) *t.norm = (float)norm;
    const float f = norm <= (double)t.max_norm ? 1.f : (float)((double)t.max_norm / norm);
    for (uint32_t b = blockIdx.x; b < t.blocks; b += gridDim.x) {
        const uint32_t block = t.blocks - 1 - b;
        const GradEntry &e = t.e[entry_of(t, block)];
        if (f == 1.f && e.out == e.grad) continue;
        if (e.dtype == 1) scale_block<BF16>(e, block - e.first, f);
        else scale_block<F32>(e, block - e.first, f);
    }
}

}  // namespace rrn
