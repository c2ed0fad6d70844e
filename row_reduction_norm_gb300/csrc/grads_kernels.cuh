// grads_kernels.cuh -- the norm of many tensors together, and their clipping:
// norm = sqrt(sum g^2), out = RN(g min(1, max_norm / norm)).
//
// Two launches over the same parts of 32 KB, a block each: sums of squares, then
// the scaling, whose blocks each add up the first launch's partial sums for
// themselves (a few thousand bytes from L2) rather than wait for a launch in
// between.  HBM bandwidth bounds both: every byte is read twice and written
// once.  The scaling goes through the parts from the last to the first: what
// the norm read last is still in L2.  562 million elements in 25 tensors, a third
// of them fp32: 523 us for what a plain copy of as many bytes would take 504 for.
//
// Up to 2 MB are one launch of one block, or one cluster, in parts of 4 KB, a warp
// each, which stay in registers between the two steps; the blocks' sums meet in
// distributed shared memory (20 tensors of 20,000 elements together 4.3 us, 6.0 in
// two launches; of 1.4 MB 5.8).
//
// The tensors' addresses travel as the launch's parameters (up to 32 KB of
// them), so nothing is copied to the device beforehand and a captured call
// replays by itself.
#pragma once

#include "rmsnorm_cluster.cuh"

namespace rrn {

constexpr int kGradThreads = 256, kGradChunks = 8;
constexpr int kGradPartials = 2048;                             // blocks of the norm's launches at most
constexpr int kGradAlone = 1024, kGradAloneBlocks = 16;   // threads of a block of the single cluster, and blocks

// Bytes of a part that `threads` threads take.
__host__ __device__ constexpr int grad_part(int threads) { return threads * kGradChunks * 16; }

// A tensor of a launch: its parts are first .. the next one's first - 1, cut at
// multiples of their size behind the 16-byte boundary at or before its start.
struct GradEntry {
    const char *grad;
    char *out;
    int64_t count;
    uint32_t first;
    int32_t dtype;
};

// Tensors of a launch at most, 32,764 bytes of parameters.  Parameters cost host
// time (two launches for 60 tensors: 8.8 us with room for 1020), so fewer tensors
// are launched with room for fewer.
constexpr int kGradSmall = 40, kGradSome = 160, kGradMost = 1020;

template <int CAP>
struct GradTable {
    double *partial;    // of this call, [kGradPartials]
    float *norm;
    int32_t n;          // entries here
    uint32_t parts;     // here
    int32_t slot;       // first partial sum of this launch
    int32_t sums;       // partial sums of the whole call
    float max_norm;
    int32_t clip;       // the single cluster's launch: the tensors too, not the norm alone
    GradEntry e[CAP];
};

// The entry that holds part `b`.
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

// Thread t's chunks of a part that THREADS threads take, and the first one's place.
template <typename T, int THREADS>
__device__ __forceinline__ int64_t load_part(Chunk (&c)[kGradChunks], const GradEntry &e, uint32_t part, int t) {
    constexpr int V = T::kVec;
    const int64_t first = ((int64_t)part * THREADS * kGradChunks + t) * V - grad_head<T>(e.grad);
#pragma unroll
    for (int j = 0; j < kGradChunks; ++j) c[j] = grad_chunk<T>(e.grad, first + (int64_t)j * THREADS * V, e.count);
    return first;
}

// Sum of the squares of a thread's chunks, each element times `scale` (a power
// of two) first.
template <typename T>
__device__ __forceinline__ float squares_of(const Chunk (&c)[kGradChunks], float scale) {
    constexpr int V = T::kVec;
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

// A sum and what its roundings lost: fp32 pairs, since the device has two fp64
// lanes an SM (a block's sum, root and quotient in fp64 by every thread took two
// small launches from 5.3 to 7.1 us).
struct Pair {
    float sum, lost;
};
__device__ __forceinline__ void add(Pair &a, float v) {
    const float s = a.sum + v, w = s - a.sum;
    a.lost += (a.sum - (s - w)) + (v - w);
    a.sum = s;
}
__device__ __forceinline__ double whole(const Pair &a) {
    // an infinite sum has lost nothing that can be said
    return isfinite(a.sum) ? (double)a.sum + (double)a.lost : (double)a.sum;
}

// The block's threads' pairs added up, for every thread.
template <int WARPS>
__device__ __forceinline__ Pair block_sum(Pair v, Pair (&sums)[WARPS]) {
    auto lanes = [&](int width) {
        for (int off = width / 2; off > 0; off >>= 1) {
            const Pair w = {__shfl_xor_sync(0xffffffffu, v.sum, off), __shfl_xor_sync(0xffffffffu, v.lost, off)};
            const float s = v.sum + w.sum, d = s - v.sum;
            v.lost = (v.lost + w.lost) + ((v.sum - (s - d)) + (w.sum - d));
            v.sum = s;
        }
    };
    lanes(32);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = v;
    __syncthreads();
    v = sums[threadIdx.x % WARPS];
    lanes(WARPS);
    v.sum = __shfl_sync(0xffffffffu, v.sum, 0);
    v.lost = __shfl_sync(0xffffffffu, v.lost, 0);
    return v;
}

// All of a block's squares, for its first thread; `squares(scale)` gives a
// thread's.  Those past fp32's range, above or below (2^-80: sums so small that
// squares of 2^-126 count), once more, scaled by a power of two.  All threads of
// a block see the same sum.
template <int WARPS, typename F>
__device__ __forceinline__ double block_squares(Pair (&sums)[WARPS], F squares) {
    double back = 1.;
    Pair s = block_sum(squares(1.f), sums);
    if (!isfinite(s.sum) || s.sum < 0x1p-80f) {
        const bool large = !isfinite(s.sum);
        s = block_sum(squares(large ? 0x1p-80f : 0x1p80f), sums);
        back = large ? 0x1p160 : 0x1p-160;
    }
    return threadIdx.x == 0 ? whole(s) * back : 0.;
}

template <int CAP>
__global__ void __launch_bounds__(kGradThreads) grad_squares_kernel(const __grid_constant__ GradTable<CAP> t) {
    __shared__ Pair sums[kGradThreads / 32];
    const int hint = entry_of(t, blockIdx.x);   // (the parameters are there before the wait)
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    const double s = block_squares(sums, [&](float scale) {
        Pair sum = {0.f, 0.f};
        for (uint32_t b = blockIdx.x; b < t.parts; b += gridDim.x) {   // fp32 sums of 64 or fewer squares
            const GradEntry &e = t.e[b == blockIdx.x ? hint : entry_of(t, b)];
            Chunk c[kGradChunks];
            if (e.dtype == 1) {
                load_part<BF16, kGradThreads>(c, e, b - e.first, threadIdx.x);
                add(sum, squares_of<BF16>(c, scale));
            } else {
                load_part<F32, kGradThreads>(c, e, b - e.first, threadIdx.x);
                add(sum, squares_of<F32>(c, scale));
            }
        }
        return sum;
    });
    if (threadIdx.x == 0) t.partial[t.slot + blockIdx.x] = s;
}

// The factor from a norm, for the block's other threads; its first thread calls.
// Below fp32's smallest normal number it would lose bits: there it is 2^126 times
// as large and negative, and store_part multiplies by the power too.
template <int CAP>
__device__ __forceinline__ float factor_of(const GradTable<CAP> &t, double norm) {
    if (norm <= (double)t.max_norm) return 1.f;
    const double q = (double)t.max_norm / norm;
    const float f = (float)q;
    if (__builtin_expect(f < 0x1p-126f, 0)) return (float)(q * -0x1p126);
    return f;
}

// The norm from the partial sums, by the block's first warp, in its lane 0.
template <int CAP>
__device__ __forceinline__ double norm_of(const GradTable<CAP> &t) {
    constexpr int U = 8;
    double s = 0.;
    for (int i = threadIdx.x; i < t.sums; i += 32 * U) {
        double v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = i + 32 * u < t.sums ? __ldcg(t.partial + i + 32 * u) : 0.;
#pragma unroll
        for (int u = 0; u < U; ++u) s += v[u];
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_down_sync(0xffffffffu, s, off);
    return threadIdx.x == 0 ? sqrt(s) : 0.;
}

template <int CAP>
__global__ void __launch_bounds__(32) grad_norm_kernel(const __grid_constant__ GradTable<CAP> t) {
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    const double norm = norm_of(t);
    if (threadIdx.x == 0) *t.norm = (float)norm;
}

// A thread's chunks of a part times the factor (factor_of's), to the tensor's out.
template <typename T, int THREADS>
__device__ __forceinline__ void store_part(const Chunk (&c)[kGradChunks], const GradEntry &e, int64_t first, float f) {
    constexpr int V = T::kVec, E = 16 / V;
    const bool alike = ((reinterpret_cast<uintptr_t>(e.grad) ^ reinterpret_cast<uintptr_t>(e.out)) & 15) == 0;
#pragma unroll
    for (int j = 0; j < kGradChunks; ++j) {
        const int64_t i = first + (int64_t)j * THREADS * V;
        float x[V];
        unpack(c[j], x, T{});
#pragma unroll
        for (int k = 0; k < V; ++k) x[k] *= fabsf(f);
        if (f < 0.f) {
#pragma unroll
            for (int k = 0; k < V; ++k) x[k] *= 0x1p-126f;
        }
        if (alike && i >= 0 && i + V <= e.count) {
            st16(e.out + i * E, pack(x, T{}));
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (i + k >= 0 && i + k < e.count) st_scalar(e.out, i + k, x[k], T{});
        }
    }
}

// The parts from the last to the first.
template <int CAP>
__global__ void __launch_bounds__(kGradThreads) grad_scale_kernel(const __grid_constant__ GradTable<CAP> t) {
    __shared__ float factor;
    const int hint = entry_of(t, t.parts - 1 - blockIdx.x);
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    if (threadIdx.x < 32) {
        const double norm = norm_of(t);
        if (threadIdx.x == 0) {
            factor = factor_of(t, norm);
            if (blockIdx.x == 0) *t.norm = (float)norm;
        }
    }
    __syncthreads();
    const float f = factor;
    for (uint32_t b = blockIdx.x; b < t.parts; b += gridDim.x) {
        const uint32_t part = t.parts - 1 - b;
        const GradEntry &e = t.e[b == blockIdx.x ? hint : entry_of(t, part)];
        if (f == 1.f && e.out == e.grad) continue;
        Chunk c[kGradChunks];
        if (e.dtype == 1) {
            const int64_t first = load_part<BF16, kGradThreads>(c, e, part - e.first, threadIdx.x);
            store_part<BF16, kGradThreads>(c, e, first, f);
        } else {
            const int64_t first = load_part<F32, kGradThreads>(c, e, part - e.first, threadIdx.x);
            store_part<F32, kGradThreads>(c, e, first, f);
        }
    }
}

__device__ __forceinline__ void st_cluster_f64(const double *local, uint32_t rank, double v) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
    uint32_t ra;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.f64 [%0], %1;" : : "r"(ra), "d"(v) : "memory");
}

// Both steps by one cluster, a part a warp.
template <int CAP>
__global__ void __launch_bounds__(kGradAlone, 1) grad_alone_kernel(const __grid_constant__ GradTable<CAP> t) {
    __shared__ Pair sums[kGradAlone / 32];
    __shared__ double of_block[kGradAloneBlocks];
    __shared__ float factor;
    const uint32_t rank = cluster_rank(), blocks = cluster_ctas();
    const uint32_t part = threadIdx.x / 32 * blocks + rank;
    const bool there = part < t.parts;
    const GradEntry &e = t.e[there ? entry_of(t, part) : 0];
    const bool bf16 = e.dtype == 1;
    if (threadIdx.x < kGradAlone / 32) sums[threadIdx.x] = Pair{0.f, 0.f};   // a block may have fewer warps
    // before a block writes to another's shared memory, that has started
    if (blocks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" : : : "memory");
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    Chunk c[kGradChunks] = {};
    int64_t first = 0;
    if (there) first = bf16 ? load_part<BF16, 32>(c, e, part - e.first, threadIdx.x % 32)
                            : load_part<F32, 32>(c, e, part - e.first, threadIdx.x % 32);
    const double s = block_squares(sums, [&](float scale) {
        return Pair{bf16 ? squares_of<BF16>(c, scale) : squares_of<F32>(c, scale), 0.f};
    });
    if (blocks > 1) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" : : : "memory");
        const double mine = __shfl_sync(0xffffffffu, s, 0);
        if (threadIdx.x < blocks) st_cluster_f64(of_block + rank, threadIdx.x, mine);
        __syncwarp();
        cluster_barrier();
    } else if (threadIdx.x == 0) {
        of_block[0] = s;
    }
    if (threadIdx.x == 0) {
        double all = 0.;
        for (uint32_t q = 0; q < blocks; ++q) all += of_block[q];
        const double norm = sqrt(all);
        if (rank == 0) *t.norm = (float)norm;
        factor = factor_of(t, norm);
    }
    __syncthreads();
    const float f = factor;
    if (!t.clip || !there || (f == 1.f && e.out == e.grad)) return;
    if (bf16) store_part<BF16, 32>(c, e, first, f);
    else store_part<F32, 32>(c, e, first, f);
}

}  // namespace rrn
