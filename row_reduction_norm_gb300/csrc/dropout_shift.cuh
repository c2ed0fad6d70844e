// dropout_shift.cuh -- the register kernels of dropout_kernels.cuh for rows
// whose length is no multiple of 16 bytes (an odd width), in tensors that
// start on a 16-byte boundary.
//
// Rows r and r + V (V elements to 16 bytes) start equally far, `s` elements,
// past a boundary.  The grid strides by a multiple of V rows, so every row of
// a thread has the same s, and a thread works on aligned chunks of memory: its
// chunk u holds the columns u V - s .. u V - s + V - 1, for all its rows.  So
// loads and stores are 16 bytes wide, and the thread's weights and its sums of
// the weight's gradient stay in registers, as with aligned rows.  Only a row's
// first and last chunk hold elements of its neighbours: they are zeroed on the
// way in and left alone on the way out.  A chunk's mask comes out of those of
// two generator calls, which the row's threads leave in shared memory.
#pragma once

#include "dropout_kernels.cuh"
#include "row_classes.cuh"
#include "shift_layout.h"

namespace rrn {

__host__ __device__ constexpr int shift_ring_bytes(int gt, int ch) {
    return drop_ring_bytes(gt, ch) + 2 * (drop_block_threads(gt) / gt) * (gt * ch + 1);
}

// The masks of a row's unshifted chunks (columns k V .. k V + V - 1), a byte
// each: bit e tells whether element e is kept.  Byte k + 1 of `mask` is chunk
// k's, by the thread that has chunk k; warps without one make none.
template <int V, int M>
__device__ __forceinline__ void put_masks(const DropParams &p, uint64_t seed, uint64_t offset, uint64_t row_block,
                                          const int (&k)[M], uint8_t *mask) {
    uint32_t w[M][4];
    chunk_words<V, M>(seed, offset, row_block, k, w);
#pragma unroll
    for (int m = 0; m < M; ++m) {
        uint32_t bits = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) bits |= (uint32_t)kept(w[m], e, p.thr << 16) << e;
        mask[k[m] + 1] = (uint8_t)bits;
    }
}
template <int V, int GT, int CH>
__device__ __forceinline__ void make_masks(const DropParams &p, uint64_t seed, uint64_t offset, int64_t row, int t,
                                           int chunks, uint8_t *mask) {
    const uint64_t row_block = (uint64_t)(row * p.blocks_per_row);
    const int t0 = GT < 32 ? 0 : t & ~31;
#pragma unroll
    for (int c = 0; c < CH; c += 2) {
        if (c + 1 < CH && (c + 1) * GT + t0 < chunks) {
            const int k[2] = {c * GT + t, (c + 1) * GT + t};
            put_masks<V, 2>(p, seed, offset, row_block, k, mask);
        } else if (c * GT + t0 < chunks) {
            const int k[1] = {c * GT + t};
            put_masks<V, 1>(p, seed, offset, row_block, k, mask);
        }
    }
}
// The mask of shifted chunk u (bits 0 .. V - 1), out of the chunk of its number
// and the one before.  Byte 0 is never written: the elements before column 0
// come out of it, and nothing else may.
template <int V>
__device__ __forceinline__ uint32_t shifted_mask(const uint8_t *mask, int u, int s) {
    return (((uint32_t)mask[u] & ((1u << V) - 1u)) | ((uint32_t)mask[u + 1] << V)) >> (V - s);
}

// Chunk of the weight for the columns u V - s and on (0 off its ends).
template <typename T>
__device__ __forceinline__ Chunk shifted_weight(const void *w, int first, int hidden) {
    Chunk c{{0u, 0u, 0u, 0u}};
    constexpr int V = T::kVec;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const int col = first + e, near = col < 0 ? 0 : col < hidden ? col : hidden - 1;   // no branch: the loads go together
        const uint32_t got = ld_bits(w, near, T{}, 2), b = near == col ? got : 0u;
        if constexpr (V == 8) c.u[e / 2] |= b << (16 * (e & 1));
        else c.u[e] = b;
    }
    return c;
}

// Zeros in place of a chunk's elements before lo and from hi on.
template <typename T>
__device__ __forceinline__ void clear_ends(Chunk &c, int lo, int hi) {
    constexpr int V = T::kVec;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if constexpr (V == 8) {
            const uint32_t low = 2 * w >= lo && 2 * w < hi ? 0xffffu : 0u;
            const uint32_t high = 2 * w + 1 >= lo && 2 * w + 1 < hi ? 0xffff0000u : 0u;
            c.u[w] &= low | high;
        } else if (w < lo || w >= hi) {
            c.u[w] = 0u;
        }
    }
}

// Stores a chunk's elements lo .. hi - 1.
template <typename T>
__device__ __forceinline__ void put_chunk(char *at, const float (&v)[T::kVec], int lo, int hi) {
    if (lo == 0 && hi == T::kVec) {
        st16(at, pack(v, T{}));
    } else {
#pragma unroll
        for (int e = 0; e < T::kVec; ++e)
            if (e >= lo && e < hi) st_scalar(at, e, v[e], T{});
    }
}

// bf16 16384 x 2047 takes 71.8 us (82.7 element by element).  Three blocks a SM
// rather than two, with which it took a fifth more.
template <typename T, int GT, int CH>
__global__ void __launch_bounds__(drop_block_threads(GT), GT < 512 ? 3 : 1) drop_fwd_shift_kernel(const DropParams p) {
    constexpr int V = T::kVec, S = 16 / V, BLOCK = drop_block_threads(GT), RPB = BLOCK / GT;
    __shared__ ShiftedSums<GT, 1> red[RPB];
    __shared__ uint8_t masks[2][RPB][GT * CH + 1];
    const int tid = threadIdx.x, slot = tid / GT, t = tid % GT;
    const int hidden = (int)p.row_elems;
    int64_t first = (int64_t)blockIdx.x * RPB;
    ShiftedRow<V> at;
    at.set(first + slot, hidden);
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    uint64_t seed = 0, offset = 0;
    if (p.thr) {
        seed = p.rng[0];
        offset = p.rng[1];
    }
    const bool weighted = p.w != nullptr;
    Chunk wc[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c)
        wc[c] = weighted ? shifted_weight<T>(p.w, (c * GT + t) * V - at.s, hidden) : Chunk{{0u, 0u, 0u, 0u}};
    int parity = 0;
    for (; first < p.rows; first += (int64_t)gridDim.x * RPB) {
        const int64_t row = first + slot;
        const bool ok = row < p.rows;
        const int64_t off = row * p.row_bytes - at.s * S + t * 16;
        const char *xr = static_cast<const char *>(p.x) + off, *rr = static_cast<const char *>(p.res) + off;
        Chunk xc[CH], hc[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int u = c * GT + t;
            xc[c] = hc[c] = Chunk{{0u, 0u, 0u, 0u}};
            if (ok && u < at.chunks) {
                if (at.whole(u, row, p.rows, hidden)) {
                    xc[c] = ld_stream16(xr + c * GT * 16);
                    hc[c] = ld_stream16(rr + c * GT * 16);
                } else {   // the tensors' last elements
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const uint32_t a = e < at.tail ? ld_bits(xr + c * GT * 16, e, T{}, 1) : 0u;
                        const uint32_t b = e < at.tail ? ld_bits(rr + c * GT * 16, e, T{}, 1) : 0u;
                        if constexpr (V == 8) xc[c].u[e / 2] |= a << (16 * (e & 1)), hc[c].u[e / 2] |= b << (16 * (e & 1));
                        else xc[c].u[e] = a, hc[c].u[e] = b;
                    }
                }
            }
        }
        uint8_t *mask = masks[parity][slot];   // the other one may still be read
        if (p.thr) {
            make_masks<V, GT, CH>(p, seed, offset, row, t, at.chunks, mask);
            if constexpr (GT > 32) __syncthreads();
            else __syncwarp();
        }
        float acc[1][V];
#pragma unroll
        for (int e = 0; e < V; ++e) acc[0][e] = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int u = c * GT + t;
            if (ok && u < at.chunks) {
                const int lo = at.lo(u), hi = at.hi(u);
                const uint32_t keep = p.thr ? shifted_mask<V>(mask, u, at.s) : 0u;
                if (lo > 0 || hi < V) {   // not the neighbours' elements
                    clear_ends<T>(xc[c], lo, hi);
                    clear_ends<T>(hc[c], lo, hi);
                }
                float a[V], b[V];
                unpack(xc[c], a, T{});
                unpack(hc[c], b, T{});
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    if (p.thr) a[e] = (keep >> e) & 1u ? a[e] * p.scale : 0.f;
                    a[e] = add_round(b[e], a[e], T{});
                }
                hc[c] = pack(a, T{});
                put_chunk<T>(static_cast<char *>(p.h_out) + off + c * GT * 16, a, lo, hi);
                sq_accumulate(a, acc[0]);
            }
        }
        float sum[1];
        shifted_sums<GT, V, 1>(acc, at.s, red[slot], t, sum);
        parity ^= 1;
        const float r = rsqrtf(sum[0] / p.hidden_f + p.eps);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int u = c * GT + t;
            if (ok && u < at.chunks) {
                float a[V], wv[V];
                unpack(hc[c], a, T{});
                if (weighted) {
                    unpack(wc[c], wv, T{});
                    scale_out_pairs<kWeightBias>(a, r, wv, p.w_bias);
                } else {
                    scale_out_pairs<kNoWeight>(a, r, wv, 0.f);
                }
                put_chunk<T>(static_cast<char *>(p.y) + off + c * GT * 16, a, at.lo(u), at.hi(u));
            }
        }
    }
}

// The gradient (see drop_bwd_kernel).  bf16 8192 x 4095 takes 91 us, 8192 x
// 8191 173 (169 and 343 by single elements; aligned 8192 x 8192 rows 107):
// what bounds it is issue slots, 435 instructions for 32 chunks.
template <typename T, int GT, int CH, bool DW>
__global__ void __launch_bounds__(drop_block_threads(GT), drop_bwd_resident(GT)) drop_bwd_shift_kernel(const DropParams p) {
    constexpr int V = T::kVec, S = 16 / V, BLOCK = drop_block_threads(GT), RPB = BLOCK / GT;
    __shared__ ShiftedSums<GT, 2> red[RPB];
    extern __shared__ __align__(16) Chunk ring[];   // [stage][dy, h, dh][CH][BLOCK], then the masks' bytes [2][RPB][GT CH + 1]
    const int tid = threadIdx.x, slot = tid / GT, t = tid % GT;
    uint8_t *masks = reinterpret_cast<uint8_t *>(ring + kDropStages * 3 * CH * BLOCK);
    const int hidden = (int)p.row_elems;
    int64_t first = (int64_t)blockIdx.x * RPB;
    ShiftedRow<V> at;
    at.set(first + slot, hidden);
    pdl_wait_for_inputs();
    pdl_allow_dependents();

    const int64_t step = (int64_t)gridDim.x * RPB;
    auto place = [&](int stage, int tensor, int c) -> Chunk & { return ring[((stage * 3 + tensor) * CH + c) * BLOCK + tid]; };
    auto issue = [&](int64_t group, int stage) {
        const int64_t row = group + slot;
        if (row < p.rows) {
            const int64_t off = row * p.row_bytes - at.s * S + t * 16;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int u = c * GT + t;
                if (u < at.chunks) {
                    const uint32_t bytes = (uint32_t)(at.hi(u) * S);   // zeros past them
                    copy_async_part(&place(stage, 0, c), static_cast<const char *>(p.dy) + off + c * GT * 16, bytes);
                    copy_async_part(&place(stage, 1, c), static_cast<const char *>(p.h) + off + c * GT * 16, bytes);
                    if (p.dh != nullptr)
                        copy_async_part(&place(stage, 2, c), static_cast<const char *>(p.dh) + off + c * GT * 16, bytes);
                }
            }
        }
        copy_async_commit();   // an empty group past the end
    };
    issue(first, 0);

    uint64_t seed = 0, offset = 0;
    if (p.thr) {
        seed = p.rng[0];
        offset = p.rng[1];
    }
    const bool weighted = p.w != nullptr;
    float dw[DW ? CH : 1][V];
#pragma unroll
    for (int c = 0; c < (DW ? CH : 1); ++c)
#pragma unroll
        for (int e = 0; e < V; ++e) dw[c][e] = 0.f;
    Chunk wc[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c)
        wc[c] = weighted ? shifted_weight<T>(p.w, (c * GT + t) * V - at.s, hidden) : Chunk{{0u, 0u, 0u, 0u}};
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
        const int64_t off = row * p.row_bytes - at.s * S + t * 16;
        issue(first + step, parity ^ 1);
        uint8_t *mask = masks + (parity * RPB + slot) * (GT * CH + 1);   // the other one may still be read
        if (p.thr) make_masks<V, GT, CH>(p, seed, offset, row, t, at.chunks, mask);
        copy_async_wait<1>();   // this group's copies of this thread are there
        if (t == 0 && at.s > 0) {   // not the row before's elements
            clear_ends<T>(place(parity, 0, 0), at.s, V);
            clear_ends<T>(place(parity, 1, 0), at.s, V);
        }
        float acc[2][V];   // of h h, of g h
#pragma unroll
        for (int e = 0; e < V; ++e) acc[0][e] = acc[1][e] = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (ok && c * GT + t < at.chunks) {
                float h[V], g[V], w[V];
                unpack(place(parity, 1, c), h, T{});
                unpack(place(parity, 0, c), g, T{});
                sq_accumulate(h, acc[0]);
                if (weighted) {
                    weight(c, w);
                    mul_pairs(g, w);
                }
                fma_pairs(acc[1], g, h);
            }
        }
        if constexpr (GT <= 32) __syncwarp();
        float sums[2];
        shifted_sums<GT, V, 2>(acc, at.s, red[slot], t, sums);
        const float r = rsqrtf(sums[0] / p.hidden_f + p.eps);
        const float m = -(r * (sums[1] / p.hidden_f));   // d = r (g - (h r) mean(g h) r) + dh
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int u = c * GT + t;
            if (ok && u < at.chunks) {
                float h[V], g[V], w[V], d[V];
                unpack(place(parity, 1, c), h, T{});
                unpack(place(parity, 0, c), g, T{});
                scale_pairs(h, r);
                if constexpr (DW) fma_pairs(dw[c], g, h);
                if (weighted) {
                    weight(c, w);
                    mul_pairs(g, w);
                }
                float mm[V], rr[V];
#pragma unroll
                for (int e = 0; e < V; ++e) mm[e] = m, rr[e] = r;
                fma_pairs(g, h, mm);
                if (p.dh != nullptr) {
                    unpack(place(parity, 2, c), d, T{});
                    fma_pairs(d, g, rr);
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) d[e] = g[e];
                    scale_pairs(d, r);
                }
                const int lo = at.lo(u), hi = at.hi(u);
                put_chunk<T>(static_cast<char *>(p.dres) + off + c * GT * 16, d, lo, hi);
                if (p.dx != nullptr) {
                    if (p.thr) {
                        const uint32_t keep = shifted_mask<V>(mask, u, at.s);
#pragma unroll
                        for (int e = 0; e < V; ++e) d[e] = (keep >> e) & 1u ? d[e] * p.scale : 0.f;
                    }
                    put_chunk<T>(static_cast<char *>(p.dx) + off + c * GT * 16, d, lo, hi);
                }
            }
        }
        parity ^= 1;
    }
    copy_async_wait<0>();
    if constexpr (DW) {
        // each slot's sums in a place of its own, by chunk; then column by column
        float *sums = reinterpret_cast<float *>(ring);   // [RPB][GT CH V], at most a third of the ring
        __syncthreads();                                 // every thread is done with its places
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int e = 0; e < V; e += 4)
                *reinterpret_cast<float4 *>(sums + (slot * CH * GT + c * GT + t) * V + e) =
                    make_float4(dw[c][e], dw[c][e + 1], dw[c][e + 2], dw[c][e + 3]);
        __syncthreads();
        float *out = p.partial + (int64_t)blockIdx.x * p.partial_ld;
        for (int i = tid; i < hidden; i += BLOCK) {
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < RPB; ++k) {
                ShiftedRow<V> of;
                of.set((int64_t)blockIdx.x * RPB + k, hidden);
                v += sums[k * CH * GT * V + of.s + i];
            }
            out[i] = v;
        }
        finish_dw<T>(p);
    }
}

}  // namespace rrn
