// row_classes.cuh -- one order of summation for rows of odd widths, whichever
// of two kernels takes them and wherever a row lies on the 16-byte chunks.
//
// Columns fall into W classes, column j into class j mod W, where W is what the
// threads of a shifted row (dropout_shift.cuh) hold in one chunk each.  A
// class is added up by fused multiply-adds over its columns in ascending order;
// then neighbouring classes are added in pairs (0 + 1, 2 + 3, ...), then
// neighbouring pairs, and so on.  W follows from the width and the type, so
// the order does, and a row has the same bits in a batch of any size and at any
// place in it.
//
// Elements one at a time: thread t of GT has columns t, t + GT, ..., so W / GT
// classes.  Shifted chunks: element e of a thread's chunks is always of the
// class t V + e - s, s being the row's shift, so its accumulators are classes
// already; but a pair of classes may be split between two threads, the first
// s accumulators belonging to the thread before's V classes.
//
// What the order costs: a shifted row of more than a warp has a second barrier,
// behind which its warps' last threads take what the next warp's first have.
// Measured on GB300 against sums in whatever order a kernel has its elements:
// bf16 rows of 2047 x 16000 forward 67.7 -> 69.5 us, gradient 86.6 -> 92.5
// (without dropout 58.9 -> 65.2), of 8191 x 6000 119.7 -> 123.0 and 124.9 ->
// 130.4; rows of a warp and single elements within 3 %, or faster (fp32 2047 x
// 16000 gradient 121.7 -> 117.0): the lanes' sums take fewer shuffles.
#pragma once

#include "rmsnorm_kernels.cuh"

namespace rrn {

// K values (a power of two) of each of LANES lanes, neighbouring lanes added in
// pairs; a + b == b + a, so a pair's sum may be made in either lane.  With
// several values the two lanes of a pair share them out, so that K values take
// about K + 4 shuffles and not 5 K: the lane ends with the sum of value
// value_of<K>(lane).
template <int K, int LANES>
__device__ __forceinline__ float lanes_add(float (&v)[K], int lane) {
#pragma unroll
    for (int off = 1, k = K; off < LANES; off <<= 1) {
        if (k > 1) {
            k /= 2;
#pragma unroll
            for (int i = 0; i < K / 2; ++i) {
                if (i < k) {
                    const bool up = lane & off;
                    const float give = up ? v[i] : v[i + k], keep = up ? v[i + k] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
                }
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
        }
    }
    return v[0];
}
template <int K>
__device__ __forceinline__ int value_of(int lane) {
    if constexpr (K == 8) return (lane & 1) * 4 + (lane & 2) + ((lane & 4) >> 2);
    else if constexpr (K == 4) return (lane & 1) * 2 + ((lane & 2) >> 1);
    else return lane & (K - 1);
}

// Sums of M values' N parts each (parts[m * stride + i], in shared memory),
// neighbours added in pairs, for every lane: all of them read by every lane
// (shifted rows, which wait for each other: bf16 16000 x 2047 gradient 92.5 us,
// 96.8 with a part a lane), or a part a lane (rows of single elements: bf16 65536
// x 201 98.5 us, 111.6 when every lane reads them).
template <int N, int M>
__device__ __forceinline__ void parts_read(const float *parts, int stride, float (&sum)[M]) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
        float v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = parts[m * stride + i];
#pragma unroll
        for (int n = N; n > 1; n /= 2)
#pragma unroll
            for (int i = 0; i < n / 2; ++i) v[i] = v[2 * i] + v[2 * i + 1];
        sum[m] = v[0];
    }
}
template <int N, int M>
__device__ __forceinline__ void parts_share(const float *parts, int stride, int lane, float (&sum)[M]) {
    if constexpr (M == 2 && N <= 16) {   // both at once, in the halves of the warp
        float v = parts[(lane >> 4) * stride + (lane & (N - 1))];
#pragma unroll
        for (int off = 1; off < N; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        sum[0] = __shfl_sync(0xffffffffu, v, 0);
        sum[1] = __shfl_sync(0xffffffffu, v, 16);
    } else {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            float v = parts[m * stride + (lane & (N - 1))];
#pragma unroll
            for (int off = 1; off < N; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            sum[m] = v;
        }
    }
}

// --------------------------------------------------------- single elements
// Sums of M products a_m(c) b_m(c) over a row of one block of GT threads with
// CH columns and A classes a thread.  One barrier: what else was written to
// shared memory is behind it.
template <int GT, int CH, int A, int M, typename X, typename Y>
__device__ __forceinline__ void class_sums(X x, Y y, float (*red)[32], int t, float (&sum)[M]) {
    constexpr int WPR = GT / 32, K = A * M;
    static_assert(A * WPR <= 32, "a warp adds the parts up");
    float acc[K];
#pragma unroll
    for (int i = 0; i < K; ++i) acc[i] = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int m = 0; m < M; ++m) {
            float &to = acc[m * A + c % A];
            to = fmaf(x(m, c), y(c), to);
        }
    const float v = lanes_add<K, 32>(acc, t & 31);
    if ((t & 31) < K) {
        const int i = value_of<K>(t & 31);
        red[i / A][i % A * WPR + t / 32] = v;
    }
    __syncthreads();
    parts_share<A * WPR, M>(red[0], 32, t & 31, sum);
}
// With the classes as a number: 1, 2 or, up to 2048 columns, 4.
template <int GT, int CH, int M, typename X, typename Y>
__device__ __forceinline__ void class_sums(int classes, X x, Y y, float (*red)[32], int t, float (&sum)[M]) {
    if (classes == 1) {
        class_sums<GT, CH, 1, M>(x, y, red, t, sum);
    } else if (CH > 8 || classes == 2) {
        class_sums<GT, CH, 2, M>(x, y, red, t, sum);
    } else if constexpr (CH <= 8) {
        class_sums<GT, CH, 4, M>(x, y, red, t, sum);
    }
}

// ---------------------------------------------------------- shifted chunks

// A thread's V accumulators to the sum of the V classes that start among them,
// neighbours in pairs: the last accumulator, to which one value of every level
// is added in turn.  That is last[level], or, where the pair is split (bit
// `level` of the shift), the following thread's first[level].
template <int LEVEL, int N, int L>
__device__ __forceinline__ void pair_up(const float (&v)[N], int s, float (&first)[L], float (&last)[L]) {
    const bool split = (s >> LEVEL) & 1;
    first[LEVEL] = v[0];
    last[LEVEL] = v[N - 2];
    if constexpr (N > 2) {
        float u[N / 2];
#pragma unroll
        for (int i = 0; i + 1 < N / 2; ++i) u[i] = v[2 * i + 1] + (split ? v[2 * i + 2] : v[2 * i]);
        u[N / 2 - 1] = 0.f;   // by what is added in turn
        pair_up<LEVEL + 1>(u, s, first, last);
    }
}

// Shared memory of shifted_sums, a row's: what a warp's first thread has for
// the warp before it, and the warps' sums.
template <int GT, int M>
struct ShiftedSums {
    static constexpr int WPR = GT > 32 ? GT / 32 : 1;
    float4 edge[M][WPR];
    __align__(16) float warp[M][WPR];
};

// Sums of M values over a row's GT threads (every thread of the block calls).
template <int GT, int V, int M>
__device__ __forceinline__ void shifted_sums(const float (&acc)[M][V], int s, ShiftedSums<GT, M> &sh, int t, float (&sum)[M]) {
    constexpr int LANES = GT < 32 ? GT : 32, WPR = GT > 32 ? GT / 32 : 1, L = V == 8 ? 3 : 2;
    const int lane = t & (LANES - 1);
    float first[M][3], last[M][3], v[M];   // of the L levels
#pragma unroll
    for (int m = 0; m < M; ++m) {
        first[m][2] = 0.f;
        pair_up<0>(acc[m], s, first[m], last[m]);
        if (WPR > 1 && lane == 0)
            sh.edge[m][t / 32] = make_float4(first[m][0], first[m][1], first[m][2], 0.f);
#pragma unroll
        for (int l = 0; l < L; ++l) {
            const float beyond = __shfl_sync(0xffffffffu, first[m][l], (lane + 1) & (LANES - 1), LANES);
            last[m][l] = (s >> l) & 1 ? beyond : last[m][l];
        }
    }
    if constexpr (WPR > 1) {
        __syncthreads();
        if (lane == 31) {   // the thread that follows is another warp's
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const float4 e = sh.edge[m][(t / 32 + 1) % WPR];
                if (s & 1) last[m][0] = e.x;
                if (s & 2) last[m][1] = e.y;
                if (L > 2 && (s & 4)) last[m][2] = e.z;
            }
        }
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
        v[m] = acc[m][V - 1];
#pragma unroll
        for (int l = 0; l < L; ++l) v[m] += last[m][l];
    }
    const float all = lanes_add<M, LANES>(v, lane);
    if constexpr (WPR > 1) {
        if (lane < M) sh.warp[lane][t / 32] = all;
        __syncthreads();
        parts_read<WPR, M>(sh.warp[0], WPR, sum);
    } else if constexpr (M == 2) {
        const float other = __shfl_xor_sync(0xffffffffu, all, 1);
        sum[0] = lane & 1 ? other : all;
        sum[1] = lane & 1 ? all : other;
    } else {
        sum[0] = all;
    }
}

}  // namespace rrn
