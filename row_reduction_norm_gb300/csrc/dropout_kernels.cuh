// dropout_kernels.cuh -- residual dropout fused with RMSNorm, and the
// gradient of RMSNorm with and without it.
//
// Forward, per row:   h = RN_T(residual + keep * s * x),  y = RN_T(h r (w + b)),
//                     r = rsqrt(mean(h^2) + eps)
// Gradient, per row:  g = dy (w + b),  d = r (g - h r^2 mean(g h)) + dh
//                     dresidual = RN_T(d),  dx = RN_T(keep * s * d)
//                     dw = sum over rows of dy h r
//
// The mask is never stored: keep is a function of the seed, the offset and
// the element's place, so the gradient makes the same one again.  Elements
// 8 k .. 8 k + 7 of a row share one call of the Philox4x32-10 generator
// (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3",
// SC 2011) at counter (row * ceil(hidden / 8) + k, offset) under key seed: its
// 128 bits are eight 16-bit numbers, element e takes number e % 8, low half
// of a word first, and is kept when that is at least thr = round(65536 p).
// Sixteen bits an element halve the generator's work against 32 (about 8
// integer instructions an element, hidden behind the row's loads); the kept
// elements are scaled by s = 65536 / (65536 - thr), the inverse of the
// probability with which they are really kept, so the mean is exact.
#pragma once

#include "async_copy.cuh"
#include "finish.cuh"
#include "rmsnorm_kernels.cuh"
#include "row_classes.cuh"

namespace rrn {

struct DropParams {
    const void *x, *res, *w;     // forward: x, residual;  w nullable
    const void *dy, *h, *dh;     // gradient: dh (of residual_out) nullable
    void *y, *h_out;             // forward
    void *dres, *dx;             // gradient: dx only with dropout
    float *partial;              // gradient: [blocks][partial_ld] sums of dw, or NULL
    void *dw;                    // gradient of a single cluster: the weight's gradient, or NULL
    int64_t partial_ld;          // row_elems rounded up to a multiple of 4
    const uint64_t *rng;         // seed, offset
    int64_t rows;
    int64_t row_elems, row_bytes;
    int64_t blocks_per_row;      // ceil(row_elems / 8): generator calls a row
    int32_t units;               // loads a row
    uint32_t thr;                // 0: no dropout
    float scale;
    float hidden_f, eps, w_bias;
    int32_t classes;             // rows of single elements: accumulators a thread (row_classes.cuh)
    int32_t acc_in_smem;         // two-pass gradient: dw sums in shared memory, else in partial
};

// The end of a gradient with few blocks, one cluster: the weight's gradient.
template <typename T>
__device__ __forceinline__ void finish_dw(const DropParams &p) {
    if (p.dw == nullptr) return;
    behind_the_cluster();
    finish_columns<T>(p.partial, (int)gridDim.x, p.partial_ld, (int)p.row_elems, p.dw,
                      (int)(blockIdx.x * blockDim.x + threadIdx.x), (int)(gridDim.x * blockDim.x));
}

// --------------------------------------------------------------- generator

// M calls at once: a round's key is made once for all of them.
template <int M>
__device__ __forceinline__ void philox(uint64_t seed, uint64_t offset, const uint64_t (&index)[M], uint32_t (&out)[M][4]) {
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int m = 0; m < M; ++m) {
        out[m][0] = (uint32_t)index[m];
        out[m][1] = (uint32_t)(index[m] >> 32);
        out[m][2] = (uint32_t)offset;
        out[m][3] = (uint32_t)(offset >> 32);
    }
#pragma unroll
    for (int r = 0; r < 10; ++r) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            uint32_t(&c)[4] = out[m];
            const uint64_t p = (uint64_t)c[0] * 0xD2511F53u, q = (uint64_t)c[2] * 0xCD9E8D57u;
            c[0] = (uint32_t)(q >> 32) ^ c[1] ^ k0;
            c[1] = (uint32_t)q;
            c[2] = (uint32_t)(p >> 32) ^ c[3] ^ k1;
            c[3] = (uint32_t)p;
        }
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}

// Whether element e of a block is kept; thr_hi = thr << 16 (the low half of a
// word is compared where the high half stands).
__device__ __forceinline__ bool kept(const uint32_t (&w)[4], int e, uint32_t thr_hi) {
    return ((e & 1) ? w[e / 2] : w[e / 2] << 16) >= thr_hi;
}

// The words of M chunks of a row (chunk u of V elements: a block of 8, or half
// a one, then in words 0 and 1).
template <int V, int M>
__device__ __forceinline__ void chunk_words(uint64_t seed, uint64_t offset, uint64_t row_block, const int (&u)[M],
                                            uint32_t (&w)[M][4]) {
    uint64_t index[M];
#pragma unroll
    for (int m = 0; m < M; ++m) index[m] = row_block + (uint32_t)(V == 8 ? u[m] : u[m] / 2);
    philox<M>(seed, offset, index, w);
    if constexpr (V == 4) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            w[m][0] = (u[m] & 1) ? w[m][2] : w[m][0];
            w[m][1] = (u[m] & 1) ? w[m][3] : w[m][1];
        }
    }
}

// a[e] = kept ? a[e] * scale : 0
template <int V>
__device__ __forceinline__ void drop(float (&a)[V], const uint32_t (&w)[4], uint32_t thr_hi, float scale) {
#pragma unroll
    for (int e = 0; e < V; ++e) a[e] = kept(w, e, thr_hi) ? a[e] * scale : 0.f;
}

// Bit e of the result: whether element e of the 8-element block is kept.
__device__ __forceinline__ uint32_t keep_block(uint64_t seed, uint64_t offset, uint64_t index, uint32_t thr) {
    const uint64_t at[1] = {index};
    uint32_t w[1][4], bits = 0;
    philox<1>(seed, offset, at, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) bits |= (uint32_t)kept(w[0], e, thr << 16) << e;
    return bits;
}

__host__ __device__ constexpr int drop_block_threads(int gt) { return gt >= 256 ? gt : 256; }

// Sums of two values over a row's GT threads (every thread of the block calls).
template <int GT>
__device__ __forceinline__ float2 row_sums(float a, float b, float2 (*red)[GT > 32 ? GT / 32 : 1], int slot, int t) {
    constexpr int LANES = GT < 32 ? GT : 32, WPR = GT > 32 ? GT / 32 : 1;
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, off);
        b += __shfl_xor_sync(0xffffffffu, b, off);
    }
    if constexpr (WPR > 1) {
        if ((t & 31) == 0) red[slot][t / 32] = make_float2(a, b);
        __syncthreads();
        float va[WPR], vb[WPR];
#pragma unroll
        for (int i = 0; i < WPR; ++i) {
            const float2 v = red[slot][i];
            va[i] = v.x;
            vb[i] = v.y;
        }
        a = tree_sum(va);
        b = tree_sum(vb);
    }
    return make_float2(a, b);
}

// ----------------------------------------------------------------- forward
// The register kernel's layout: GT threads a row, CH chunks a thread.
template <typename T, int GT, int CH>
__global__ void __launch_bounds__(drop_block_threads(GT)) drop_fwd_kernel(const DropParams p) {
    constexpr int V = T::kVec, BLOCK = drop_block_threads(GT), RPB = BLOCK / GT;
    __shared__ float2 red[2][RPB][GT > 32 ? GT / 32 : 1];
    const int tid = threadIdx.x, slot = tid / GT, t = tid % GT;
    // the block's first row group into L2 before the wait
    if (tid == 0) prefetch_rows_l2<true>(p.x, p.res, p.row_bytes, p.rows, (int64_t)blockIdx.x * RPB, RPB);
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    uint64_t seed = 0, offset = 0;
    if (p.thr) {
        seed = p.rng[0];
        offset = p.rng[1];
    }
    int parity = 0;
    for (int64_t first = (int64_t)blockIdx.x * RPB; first < p.rows; first += (int64_t)gridDim.x * RPB) {
        const int64_t row = first + slot;
        const bool ok = row < p.rows;
        const int64_t off = row * p.row_bytes;
        Chunk xc[CH], hc[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int u = c * GT + t;
            const bool in = ok && u < p.units;
            xc[c] = in ? ld_stream16(static_cast<const char *>(p.x) + off + (int64_t)u * 16) : Chunk{{0u, 0u, 0u, 0u}};
            hc[c] = in ? ld_stream16(static_cast<const char *>(p.res) + off + (int64_t)u * 16) : Chunk{{0u, 0u, 0u, 0u}};
        }
        float acc[V];
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.f;
        constexpr int M = CH % 2 == 0 ? 2 : 1;   // chunks whose generator calls go together
#pragma unroll
        for (int c0 = 0; c0 < CH; c0 += M) {
            int u[M];
            uint32_t word[M][4];
#pragma unroll
            for (int m = 0; m < M; ++m) u[m] = (c0 + m) * GT + t;
            if (p.thr) chunk_words<V, M>(seed, offset, (uint64_t)(row * p.blocks_per_row), u, word);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const int c = c0 + m;
                float a[V], b[V];
                unpack(xc[c], a, T{});
                unpack(hc[c], b, T{});
                if (p.thr) drop<V>(a, word[m], p.thr << 16, p.scale);
#pragma unroll
                for (int e = 0; e < V; ++e) a[e] = add_round(b[e], a[e], T{});
                hc[c] = pack(a, T{});
                if (ok && u[m] < p.units) st16(static_cast<char *>(p.h_out) + off + (int64_t)u[m] * 16, hc[c]);
                sq_accumulate(a, acc);
            }
        }
        const float sum = row_sums<GT>(tree_sum(acc), 0.f, red[parity], slot, t).x;
        parity ^= 1;
        const float r = rsqrtf(sum / p.hidden_f + p.eps);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int u = c * GT + t;
            if (ok && u < p.units) {
                float a[V], wv[V];
                unpack(hc[c], a, T{});
                if (p.w != nullptr) {
                    unpack(ld_readonly16(static_cast<const char *>(p.w) + (int64_t)u * 16), wv, T{});
                    scale_out_pairs<kWeightBias>(a, r, wv, p.w_bias);
                } else {
                    scale_out_pairs<kNoWeight>(a, r, wv, 0.f);
                }
                st16(static_cast<char *>(p.y) + off + (int64_t)u * 16, pack(a, T{}));
            }
        }
    }
}

// Masks of a row as bits in shared memory (one byte a generator call), by the
// whole block; the caller syncs around it.
__device__ __forceinline__ void stage_mask(const DropParams &p, uint8_t *mask, uint64_t seed, uint64_t offset, int64_t row) {
    for (int k = threadIdx.x; k < (int)p.blocks_per_row; k += blockDim.x)
        mask[k] = (uint8_t)keep_block(seed, offset, (uint64_t)(row * p.blocks_per_row + k), p.thr);
}

// V bits of unit u (VE elements) out of the staged mask.
template <int VE>
__device__ __forceinline__ uint32_t staged_keep(const uint8_t *mask, int64_t u) {
    if constexpr (VE == 8) return mask[u];
    else if constexpr (VE == 4) return mask[u >> 1] >> (4 * (int)(u & 1));
    else return mask[u >> 3] >> (int)(u & 7);
}

// Two passes over a row by a whole block, for rows without 16-byte alignment
// (VE = 1) or too long for registers: the second pass reads h back from L2.
template <typename T, int VE, int BLOCK>
__global__ void __launch_bounds__(BLOCK) drop_fwd_loop_kernel(const DropParams p) {
    using IO = UnitIO<T, VE>;
    using Raw = typename IO::Raw;
    constexpr int U = VE == 1 ? 8 : 2;
    __shared__ float2 red[2][1][BLOCK / 32];
    extern __shared__ uint8_t mask[];   // [blocks_per_row], with dropout
    const int tid = threadIdx.x;
    const int64_t n = p.units;
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    uint64_t seed = 0, offset = 0;
    if (p.thr) {
        seed = p.rng[0];
        offset = p.rng[1];
    }
    int parity = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const int64_t off = row * p.row_bytes;
        const void *xr = static_cast<const char *>(p.x) + off, *rr = static_cast<const char *>(p.res) + off;
        void *hr = static_cast<char *>(p.h_out) + off, *yr = static_cast<char *>(p.y) + off;
        if (p.thr) {
            stage_mask(p, mask, seed, offset, row);   // the last row's readers are behind its sum's barrier
            __syncthreads();
        }
        float acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.f;
        for (int64_t base = tid; base < n; base += (int64_t)BLOCK * U) {
            Raw xa[U], ra[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int64_t u = base + (int64_t)j * BLOCK;
                xa[j] = u < n ? IO::load_last(xr, u) : IO::zero();
                ra[j] = u < n ? IO::load_last(rr, u) : IO::zero();
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int64_t u = base + (int64_t)j * BLOCK;
                if (u >= n) break;
                const uint32_t keep = p.thr ? staged_keep<VE>(mask, u) : 0xffu;
                float a[VE], b[VE];
                IO::widen(xa[j], a);
                IO::widen(ra[j], b);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    a[e] = add_round(b[e], (keep >> e) & 1u ? a[e] * p.scale : 0.f, T{});
                    const int k = (j * VE + e) & 7;
                    acc[k] = fmaf(a[e], a[e], acc[k]);
                }
                IO::store(hr, u, a);
            }
        }
        const float sum = row_sums<BLOCK>(tree_sum(acc), 0.f, red[parity], 0, tid).x;
        parity ^= 1;
        const float r = rsqrtf(sum / p.hidden_f + p.eps);
        for (int64_t base = tid; base < n; base += (int64_t)BLOCK * U) {
            Raw ha[U], wa[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int64_t u = base + (int64_t)j * BLOCK;
                ha[j] = u < n ? IO::load_last(hr, u) : IO::zero();
                wa[j] = u < n && p.w != nullptr ? IO::load_w(p.w, u) : IO::zero();
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int64_t u = base + (int64_t)j * BLOCK;
                if (u >= n) break;
                float a[VE], wv[VE];
                IO::widen(ha[j], a);
                IO::widen(wa[j], wv);
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    a[e] = p.w != nullptr ? (a[e] * r) * (wv[e] + p.w_bias) : a[e] * r;
                IO::store(yr, u, a);
            }
        }
    }
}

// ---------------------------------------------------------------- gradient

// Row groups a block has on their way or in hand.
constexpr int kDropStages = 2;
__host__ __device__ constexpr int drop_ring_bytes(int gt, int ch) {
    return kDropStages * 3 * ch * drop_block_threads(gt) * 16;
}
// Blocks a SM the registers are budgeted for.  (With 112 registers, which leave
// a block of the column sums room beside them, four chunks of bf16 spill: 8000
// x 4096 69.9 us, 55.2 without.)
__host__ __device__ constexpr int drop_bwd_resident(int gt) { return drop_block_threads(gt) == 256 ? 2 : 1; }

template <int N>
__device__ __forceinline__ void mul_pairs(float (&a)[N], const float (&b)[N]) {
#pragma unroll
    for (int k = 0; k < N; k += 2) {
        const float2 v = __fmul2_rn(make_float2(a[k], a[k + 1]), make_float2(b[k], b[k + 1]));
        a[k] = v.x, a[k + 1] = v.y;
    }
}
// acc += a * b
template <int N>
__device__ __forceinline__ void fma_pairs(float (&acc)[N], const float (&a)[N], const float (&b)[N]) {
#pragma unroll
    for (int k = 0; k < N; k += 2) {
        const float2 v = __ffma2_rn(make_float2(a[k], a[k + 1]), make_float2(b[k], b[k + 1]),
                                    make_float2(acc[k], acc[k + 1]));
        acc[k] = v.x, acc[k + 1] = v.y;
    }
}
template <int N>
__device__ __forceinline__ void scale_pairs(float (&a)[N], float r) {
#pragma unroll
    for (int k = 0; k < N; k += 2) {
        const float2 v = __fmul2_rn(make_float2(a[k], a[k + 1]), make_float2(r, r));
        a[k] = v.x, a[k + 1] = v.y;
    }
}

// Persistent blocks of RPB row slots.  A thread copies its own chunks of dy, h
// and dh into its own places of a shared-memory ring, a row group ahead, and
// reads them back where they are used: what is on its way needs no registers
// and no barrier (a thread waits for its own copies only), and what stays in
// registers is the thread's columns' share of dw over all its rows.  The
// slots are added up in order at the end and the block's sums go to
// partial[block].
// ALONE: of a single cluster, with the end of dw; in kernels of their own, since
// its code changes the registers of the loop before it (bf16 12803 x 1856 39.2
// -> 41.1 us).
template <typename T, int GT, int CH, bool DW, bool ALONE = false>
__global__ void __launch_bounds__(drop_block_threads(GT), drop_bwd_resident(GT)) drop_bwd_kernel(const DropParams p) {
    constexpr int V = T::kVec, BLOCK = drop_block_threads(GT), RPB = BLOCK / GT;
    __shared__ float2 red[2][RPB][GT > 32 ? GT / 32 : 1];
    extern __shared__ __align__(16) Chunk ring[];   // [stage][dy, h, dh][CH][BLOCK]
    const int tid = threadIdx.x, slot = tid / GT, t = tid % GT;
    // the block's first row group into L2 before the wait (bf16 8192 x 8192
    // 111.5 -> 109.5 us; two row groups 110.6)
    if (tid == 0) {
        const int64_t r0 = (int64_t)blockIdx.x * RPB;
        prefetch_rows_l2<true>(p.dy, p.h, p.row_bytes, p.rows, r0, RPB);
        if (p.dh != nullptr) prefetch_rows_l2<false>(p.dh, nullptr, p.row_bytes, p.rows, r0, RPB);
    }
    pdl_wait_for_inputs();
    pdl_allow_dependents();

    const int64_t step = (int64_t)gridDim.x * RPB;
    auto place = [&](int stage, int tensor, int c) -> Chunk & { return ring[((stage * 3 + tensor) * CH + c) * BLOCK + tid]; };
    auto issue = [&](int64_t first, int stage) {
        const int64_t row = first + slot;
        if (row < p.rows) {
            const int64_t off = row * p.row_bytes + t * 16;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                if (c * GT + t < p.units) {
                    copy_async<16>(&place(stage, 0, c), static_cast<const char *>(p.dy) + off + c * GT * 16);
                    copy_async<16>(&place(stage, 1, c), static_cast<const char *>(p.h) + off + c * GT * 16);
                    if (p.dh != nullptr)
                        copy_async<16>(&place(stage, 2, c), static_cast<const char *>(p.dh) + off + c * GT * 16);
                }
            }
        }
        copy_async_commit();   // an empty group past the end
    };
    int64_t first = (int64_t)blockIdx.x * RPB;
    issue(first, 0);

    uint64_t seed = 0, offset = 0;
    if (p.thr) {
        seed = p.rng[0];
        offset = p.rng[1];
    }
    const uint32_t thr_hi = p.thr << 16;
    const bool weighted = p.w != nullptr;
    float dw[DW ? CH : 1][V];
#pragma unroll
    for (int c = 0; c < (DW ? CH : 1); ++c)
#pragma unroll
        for (int e = 0; e < V; ++e) dw[c][e] = 0.f;
    Chunk wc[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int u = c * GT + t;
        wc[c] = weighted && u < p.units ? ld_readonly16(static_cast<const char *>(p.w) + (int64_t)u * 16)
                                        : Chunk{{0u, 0u, 0u, 0u}};
    }
    auto weight = [&](int c, float (&w)[V]) {
        unpack(wc[c], w, T{});
        const float2 b2 = make_float2(p.w_bias, p.w_bias);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 v = __fadd2_rn(make_float2(w[e], w[e + 1]), b2);
            w[e] = v.x, w[e + 1] = v.y;
        }
    };

    int parity = 0;
    for (; first < p.rows; first += step) {
        const int64_t row = first + slot;
        const bool ok = row < p.rows;
        const int64_t off = row * p.row_bytes + t * 16;
        issue(first + step, parity ^ 1);
        copy_async_wait<1>();   // this group's copies of this thread are there
        float sq[V], dot[V];
#pragma unroll
        for (int e = 0; e < V; ++e) sq[e] = dot[e] = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (ok && c * GT + t < p.units) {
                float h[V], g[V], w[V];
                unpack(place(parity, 1, c), h, T{});
                unpack(place(parity, 0, c), g, T{});
                sq_accumulate(h, sq);
                if (weighted) {
                    weight(c, w);
                    mul_pairs(g, w);
                }
                fma_pairs(dot, g, h);
            }
        }
        const float2 s = row_sums<GT>(tree_sum(sq), tree_sum(dot), red[parity], slot, t);
        const float r = rsqrtf(s.x / p.hidden_f + p.eps);
        const float m = -(r * (s.y / p.hidden_f));   // d = r (g - (h r) mean(g h) r) + dh
        constexpr int M = CH % 2 == 0 ? 2 : 1;
#pragma unroll
        for (int c0 = 0; c0 < CH; c0 += M) {
            uint32_t word[M][4];
            if (p.thr) {
                int u[M];
#pragma unroll
                for (int k = 0; k < M; ++k) u[k] = (c0 + k) * GT + t;
                chunk_words<V, M>(seed, offset, (uint64_t)(row * p.blocks_per_row), u, word);
            }
#pragma unroll
            for (int k = 0; k < M; ++k) {
                const int c = c0 + k;
                if (ok && c * GT + t < p.units) {
                    float h[V], g[V], w[V], d[V];
                    unpack(place(parity, 1, c), h, T{});
                    unpack(place(parity, 0, c), g, T{});
                    scale_pairs(h, r);
                    if constexpr (DW) fma_pairs(dw[c], g, h);
                    if (weighted) {
                        weight(c, w);
                        mul_pairs(g, w);
                    }
                    float mm[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) mm[e] = m;
                    fma_pairs(g, h, mm);
                    if (p.dh != nullptr) {
                        unpack(place(parity, 2, c), d, T{});
                        float rr[V];
#pragma unroll
                        for (int e = 0; e < V; ++e) rr[e] = r;
                        fma_pairs(d, g, rr);
                    } else {
#pragma unroll
                        for (int e = 0; e < V; ++e) d[e] = g[e];
                        scale_pairs(d, r);
                    }
                    st16(static_cast<char *>(p.dres) + off + c * GT * 16, pack(d, T{}));
                    if (p.dx != nullptr) {
                        if (p.thr) drop<V>(d, word[k], thr_hi, p.scale);
                        st16(static_cast<char *>(p.dx) + off + c * GT * 16, pack(d, T{}));
                    }
                }
            }
        }
        parity ^= 1;
    }
    copy_async_wait<0>();
    if constexpr (DW) {
        float *out = p.partial + (int64_t)blockIdx.x * p.partial_ld;
        if constexpr (RPB > 1) {
            // each slot's sums in a place of its own, then column by column
            // (adding up one slot after another in a single row took bf16
            // 25 x 192, 32 slots, from 3.9 to 9.8 us)
            float *sums = reinterpret_cast<float *>(ring);   // [RPB][GT CH V], at most a third of the ring
            __syncthreads();   // every thread is done with its places
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int e = 0; e < V; e += 4)
                    *reinterpret_cast<float4 *>(sums + (slot * CH * GT + c * GT + t) * V + e) =
                        make_float4(dw[c][e], dw[c][e + 1], dw[c][e + 2], dw[c][e + 3]);
            __syncthreads();
            for (int i = tid; i < (int)p.row_elems; i += BLOCK) {
                float v = 0.f;
#pragma unroll
                for (int s = 0; s < RPB; ++s) v += sums[s * CH * GT * V + i];
                out[i] = v;
            }
        } else {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int u = c * GT + t;
                if (u < p.units)
#pragma unroll
                    for (int e = 0; e < V; e += 4)
                        *reinterpret_cast<float4 *>(out + (int64_t)u * V + e) =
                            make_float4(dw[c][e], dw[c][e + 1], dw[c][e + 2], dw[c][e + 3]);
            }
        }
        if constexpr (ALONE) finish_dw<T>(p);
    }
}

// Two passes over a row by a whole block (rows without 16-byte alignment, or
// too long for registers).  A thread owns the same columns of every row, so
// its sums of dw need no barrier; they sit in shared memory, or, for rows too
// long for it, in the block's own row of `partial` (in L2).
template <typename T, int VE, int BLOCK, bool DW>
__global__ void __launch_bounds__(BLOCK) drop_bwd_loop_kernel(const DropParams p) {
    using IO = UnitIO<T, VE>;
    using Raw = typename IO::Raw;
    constexpr int U = VE == 1 ? 4 : 2;
    __shared__ float2 red[2][1][BLOCK / 32];
    extern __shared__ float sums[];   // [row_elems] with acc_in_smem, then the mask's bytes
    const int tid = threadIdx.x;
    const int64_t n = p.units;
    float *out = DW ? p.partial + (int64_t)blockIdx.x * p.partial_ld : nullptr;
    float *acc = DW && p.acc_in_smem ? sums : out;
    uint8_t *mask = reinterpret_cast<uint8_t *>(sums + (DW && p.acc_in_smem ? p.row_elems : 0));
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    uint64_t seed = 0, offset = 0;
    if (p.thr) {
        seed = p.rng[0];
        offset = p.rng[1];
    }
    if constexpr (DW) {
        for (int64_t u = tid; u < n; u += BLOCK)
#pragma unroll
            for (int e = 0; e < VE; ++e) acc[u * VE + e] = 0.f;
    }
    int parity = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const int64_t off = row * p.row_bytes;
        const void *gr = static_cast<const char *>(p.dy) + off, *hr = static_cast<const char *>(p.h) + off;
        const void *dr = p.dh != nullptr ? static_cast<const char *>(p.dh) + off : nullptr;
        void *outr = static_cast<char *>(p.dres) + off;
        void *xr = p.dx != nullptr ? static_cast<char *>(p.dx) + off : nullptr;
        float sq[8], dot[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) sq[i] = dot[i] = 0.f;
        for (int64_t base = tid; base < n; base += (int64_t)BLOCK * U) {
            Raw ga[U], ha[U], wa[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int64_t u = base + (int64_t)j * BLOCK;
                ga[j] = u < n ? IO::load_first(gr, u) : IO::zero();
                ha[j] = u < n ? IO::load_first(hr, u) : IO::zero();
                wa[j] = u < n && p.w != nullptr ? IO::load_w(p.w, u) : IO::zero();
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                float g[VE], h[VE], w[VE];
                IO::widen(ga[j], g);
                IO::widen(ha[j], h);
                IO::widen(wa[j], w);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    if (p.w != nullptr) g[e] *= w[e] + p.w_bias;
                    const int k = (j * VE + e) & 7;
                    sq[k] = fmaf(h[e], h[e], sq[k]);
                    dot[k] = fmaf(g[e], h[e], dot[k]);
                }
            }
        }
        if (p.thr) stage_mask(p, mask, seed, offset, row);   // read after the sums' barrier
        const float2 s = row_sums<BLOCK>(tree_sum(sq), tree_sum(dot), red[parity], 0, tid);
        parity ^= 1;
        const float r = rsqrtf(s.x / p.hidden_f + p.eps);
        const float m = (r * r) * (s.y / p.hidden_f);
        for (int64_t base = tid; base < n; base += (int64_t)BLOCK * U) {
            Raw ga[U], ha[U], wa[U], da[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int64_t u = base + (int64_t)j * BLOCK;
                ga[j] = u < n ? IO::load_last(gr, u) : IO::zero();
                ha[j] = u < n ? IO::load_last(hr, u) : IO::zero();
                wa[j] = u < n && p.w != nullptr ? IO::load_w(p.w, u) : IO::zero();
                da[j] = u < n && dr != nullptr ? IO::load_last(dr, u) : IO::zero();
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int64_t u = base + (int64_t)j * BLOCK;
                if (u >= n) break;
                float g[VE], h[VE], w[VE], d[VE];
                IO::widen(ga[j], g);
                IO::widen(ha[j], h);
                IO::widen(wa[j], w);
                IO::widen(da[j], d);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    if constexpr (DW) acc[u * VE + e] = fmaf(g[e], h[e] * r, acc[u * VE + e]);
                    if (p.w != nullptr) g[e] *= w[e] + p.w_bias;
                    const float v = r * (g[e] - h[e] * m);
                    d[e] = dr != nullptr ? v + d[e] : v;
                }
                IO::store(outr, u, d);
                if (xr != nullptr) {
                    const uint32_t keep = p.thr ? staged_keep<VE>(mask, u) : 0xffu;
#pragma unroll
                    for (int e = 0; e < VE; ++e) d[e] = (keep >> e) & 1u ? d[e] * p.scale : 0.f;
                    IO::store(xr, u, d);
                }
            }
        }
        if (p.thr) __syncthreads();   // the mask is read before the next row's is staged
    }
    if constexpr (DW) {
        if (p.acc_in_smem) {
            for (int64_t u = tid; u < n; u += BLOCK)
#pragma unroll
                for (int e = 0; e < VE; ++e) out[u * VE + e] = sums[u * VE + e];
        }
        finish_dw<T>(p);
    }
}

// -------------------------------------------------- rows of single elements
// Rows off the 16-byte boundaries (a view that starts anywhere; an odd width
// with few rows, see dropout_shift.cuh for many) that fit a block's registers:
// thread t owns columns t, t + GT, ... (CH of them), so a warp's accesses are
// consecutive, every element is read once, and what a 2-byte access wastes is
// issue slots, not bandwidth.  The mask is made a byte for 8 elements by
// whichever threads, in shared memory.  bf16 16384 x 2047 takes 83 us (49 % of
// the measured copy bandwidth), its gradient 111 (45 %); two passes over the row
// (above) took 102 and 255.  Blocks of 1024 threads for the longer rows measured
// a quarter slower than 512 with twice the columns.

template <typename T, int GT, int CH>
__global__ void __launch_bounds__(GT) drop_fwd_scalar_kernel(const DropParams p) {
    __shared__ __align__(16) float red[2][1][32];
    extern __shared__ uint8_t mask[];   // [blocks_per_row], with dropout
    const int t = threadIdx.x, n = p.units;
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    uint64_t seed = 0, offset = 0;
    if (p.thr) {
        seed = p.rng[0];
        offset = p.rng[1];
    }
    int parity = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const int64_t off = row * p.row_bytes;
        const void *xr = static_cast<const char *>(p.x) + off, *rr = static_cast<const char *>(p.res) + off;
        void *hr = static_cast<char *>(p.h_out) + off, *yr = static_cast<char *>(p.y) + off;
        uint32_t xb[CH], rb[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = c * GT + t;
            xb[c] = e < n ? ld_bits(xr, e, T{}, 1) : 0u;
            rb[c] = e < n ? ld_bits(rr, e, T{}, 1) : 0u;
        }
        if (p.thr) {   // the last row's readers are behind its sum's barrier
            stage_mask(p, mask, seed, offset, row);
            __syncthreads();
        }
        float h[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = c * GT + t;
            const bool keep = !p.thr || (e < n && ((mask[e >> 3] >> (e & 7)) & 1));
            const float x = widen_bits(xb[c], T{});
            h[c] = add_round(widen_bits(rb[c], T{}), p.thr ? (keep ? x * p.scale : 0.f) : x, T{});
            if (e < n) st_scalar(hr, e, h[c], T{});
        }
        float sum[1];
        class_sums<GT, CH, 1>(p.classes, [&](int, int c) { return h[c]; }, [&](int c) { return h[c]; }, red[parity], t, sum);
        parity ^= 1;
        const float r = rsqrtf(sum[0] / p.hidden_f + p.eps);
        if (p.w != nullptr) {
            uint32_t wb[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) wb[c] = c * GT + t < n ? ld_bits(p.w, c * GT + t, T{}, 2) : 0u;
#pragma unroll
            for (int c = 0; c < CH; ++c) h[c] = (h[c] * r) * (widen_bits(wb[c], T{}) + p.w_bias);
        } else {
#pragma unroll
            for (int c = 0; c < CH; ++c) h[c] *= r;
        }
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (c * GT + t < n) st_scalar(yr, c * GT + t, h[c], T{});
    }
}

// An element of dy and one of h: one register for bf16.
struct BothBF16 {
    uint32_t u;
    __device__ __forceinline__ void set(uint32_t g, uint32_t h) { u = (g & 0xffffu) | (h << 16); }
    __device__ __forceinline__ float g() const { return bf16_lo(u); }
    __device__ __forceinline__ float h() const { return bf16_hi(u); }
};
struct BothF32 {
    float a, b;
    __device__ __forceinline__ void set(uint32_t g, uint32_t h) { a = __uint_as_float(g), b = __uint_as_float(h); }
    __device__ __forceinline__ float g() const { return a; }
    __device__ __forceinline__ float h() const { return b; }
};
__device__ __forceinline__ BothBF16 both_of(BF16) { return {}; }
__device__ __forceinline__ BothF32 both_of(F32) { return {}; }

template <typename T, int GT, int CH, bool DW>
__global__ void __launch_bounds__(GT) drop_bwd_scalar_kernel(const DropParams p) {
    using Both = decltype(both_of(T{}));
    __shared__ __align__(16) float red[2][2][32];
    extern __shared__ uint8_t masks[];   // [2][blocks_per_row], with dropout
    const int t = threadIdx.x, n = p.units;
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    uint64_t seed = 0, offset = 0;
    if (p.thr) {
        seed = p.rng[0];
        offset = p.rng[1];
    }
    float dw[DW ? CH : 1];
#pragma unroll
    for (int c = 0; c < (DW ? CH : 1); ++c) dw[c] = 0.f;
    float w[CH];   // the columns' weight, for every row
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int e = c * GT + t;
        w[c] = p.w != nullptr && e < n ? widen_bits(ld_bits(p.w, e, T{}, 2), T{}) + p.w_bias : 1.f;
    }
    int parity = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const int64_t off = row * p.row_bytes;
        const void *dr = p.dh != nullptr ? static_cast<const char *>(p.dh) + off : nullptr;
        void *outr = static_cast<char *>(p.dres) + off;
        void *xr = p.dx != nullptr ? static_cast<char *>(p.dx) + off : nullptr;
        const void *gr = static_cast<const char *>(p.dy) + off, *hr = static_cast<const char *>(p.h) + off;
        Both v[CH];
        uint32_t db[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = c * GT + t;
            const uint32_t g = e < n ? ld_bits(gr, e, T{}, 1) : 0u, h = e < n ? ld_bits(hr, e, T{}, 1) : 0u;
            v[c].set(g, h);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = c * GT + t;
            db[c] = dr != nullptr && e < n ? ld_bits(dr, e, T{}, 1) : 0u;
        }
        uint8_t *mask = masks + parity * p.blocks_per_row;   // the other one may still be read
        if (p.thr) stage_mask(p, mask, seed, offset, row);   // read after the sums' barrier
        float s[2];   // of h h, of g h
        class_sums<GT, CH, 2>(p.classes, [&](int m, int c) { return m ? v[c].g() * w[c] : v[c].h(); },
                              [&](int c) { return v[c].h(); }, red[parity], t, s);
        parity ^= 1;
        const float r = rsqrtf(s[0] / p.hidden_f + p.eps);
        const float m = -(r * (s[1] / p.hidden_f));
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e = c * GT + t;
            if (e < n) {
                const float h = v[c].h() * r;
                const float g = v[c].g();
                if constexpr (DW) dw[c] = fmaf(g, h, dw[c]);
                float d = fmaf(h, m, g * w[c]);
                if (dr != nullptr) {
                    d = fmaf(d, r, widen_bits(db[c], T{}));
                } else {
                    d *= r;
                }
                st_scalar(outr, e, d, T{});
                if (xr != nullptr) {
                    if (p.thr) d = (mask[e >> 3] >> (e & 7)) & 1 ? d * p.scale : 0.f;
                    st_scalar(xr, e, d, T{});
                }
            }
        }
    }
    if constexpr (DW) {
        float *out = p.partial + (int64_t)blockIdx.x * p.partial_ld;
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (c * GT + t < n) out[c * GT + t] = dw[c];
        finish_dw<T>(p);
    }
}

}  // namespace rrn
