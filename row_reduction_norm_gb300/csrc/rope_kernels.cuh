// rope_kernels.cuh -- per-head RMSNorm with rotary positions: the fused
// forward of packed query / key heads, its gradient, and the append of keys
// and values to a paged cache with the same norm and rotation on the way.
//
// Per head row x[D] (D even, R = rot / 2 rotated pairs, weight w):
//   n      = x * rsqrt(mean(x^2) + eps) * (w + bias)      (n = x without the norm)
//   pair i = elements (i, i + R), or (2i, 2i + 1) interleaved
//   theta  = position(axis of i) * inv_freq[i]
//   y_a = n_a cos - n_b sin,  y_b = n_a sin + n_b cos;  elements past rot: y = n
// rounded once.  The gradient, g = dy turned by -theta, dn = g (w + bias):
//   dx = r (dn - x r^2 mean(dn x)),   dw = sum over tokens and heads of g x r.
//
// Work layout.  A lane owns K "units" of a head: unit u is VE pairs, held as
// two pieces of VE elements, so both halves of every pair sit in one lane and
// the rotation needs no exchange.  G lanes share a head, 32 / G heads run
// side by side in a warp, and a warp walks the heads of one token: the
// token's sines and cosines are computed once per warp (each pair by one
// lane) and shared through shared memory behind warp syncs only.
//
// Angles.  Positions are integers, so only the fraction of a turn per step
// matters: inv_freq / 2 pi is held as a 64-bit fixed-point fraction of a turn
// and position * fraction wraps modulo 2^64, exactly modulo one turn.  No
// precision is lost to far positions (|position| (1 + f) 2^-64 turns), no 64-bit
// floating point is used (slow on this GPU), and no table of cosines has to
// be kept or read.
#pragma once

#include "rmsnorm_kernels.cuh"

namespace rrn {

constexpr int kRopeMaxDim = 512;      // head_dim
constexpr int kRopeMaxAxes = 4;
constexpr int kRopeMaxWarps = 8;      // warps a block

struct RopeParams {
    const void *x;            // packed token rows (query, key, [value] heads)
    const void *dy;           // gradient: of the rotated rows
    void *y;                  // rotated rows (append: of the query heads); gradient: dx
    const void *q_w, *k_w;    // nullable
    float *partial;           // gradient: [blocks][2][D] sums of the weights' gradients, or NULL
    int64_t tokens;
    int64_t x_stride, y_stride, dy_stride;   // bytes between token rows
    int32_t q_heads, k_heads, v_heads;       // v_heads: append only
    int32_t head_dim;
    int32_t norm;
    float head_dim_f, eps, w_bias;
    // rotation
    const void *pos;          // [axes][pos_stride], 32 or 64 bit; append: NULL = index in the cache
    int64_t pos_stride;
    int32_t pos64;
    int32_t cut[3];           // first pair of axes 1, 2, 3 (R where there is none)
    const float *inv_freq;    // [R]
    int32_t R;
    int32_t units, rot_units; // pair units of a head, and the rotated ones among them
    int32_t lanes;            // G: lanes a head, a power of two
    int32_t iters;            // head iterations a slice of a token's heads takes
    // paged cache (append)
    const int32_t *cu_tokens, *cache_lens, *page_table;
    int64_t table_stride;
    int32_t seqs, max_pages, num_pages, page_size;
    void *k_cache, *v_cache;
    int64_t page_stride, row_stride, head_stride;   // bytes
    float k_inv, v_inv;       // 8-bit cache: 1 / scale
    int32_t *dropped;
};

// ------------------------------------------------------------------ pieces
// VE consecutive elements as one access of VE * sizeof(T) bytes.

template <int WORDS>
struct RawPiece {
    uint32_t u[WORDS];
};

template <typename T, int VE>
struct Piece {
    static constexpr int kBytes = VE * (int)sizeof(typename T::storage);
    static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
    using Raw = RawPiece<kWords>;

    __device__ static __forceinline__ Raw zero() {
        Raw r;
#pragma unroll
        for (int i = 0; i < kWords; ++i) r.u[i] = 0u;
        return r;
    }
    // Streamed (read once) loads; weights take the read-only path.
    __device__ static __forceinline__ Raw load(const char *p) {
        Raw r;
        if constexpr (kBytes == 16) {
            asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(r.u[0]), "=r"(r.u[1]), "=r"(r.u[2]), "=r"(r.u[3]) : "l"(p));
        } else if constexpr (kBytes == 8) {
            asm volatile("ld.global.cs.v2.u32 {%0, %1}, [%2];" : "=r"(r.u[0]), "=r"(r.u[1]) : "l"(p));
        } else if constexpr (kBytes == 4) {
            asm volatile("ld.global.cs.u32 %0, [%1];" : "=r"(r.u[0]) : "l"(p));
        } else {
            unsigned short h;
            asm volatile("ld.global.cs.u16 %0, [%1];" : "=h"(h) : "l"(p));
            r.u[0] = h;
        }
        return r;
    }
    __device__ static __forceinline__ void widen(const Raw &r, float (&f)[VE]) {
        if constexpr (sizeof(typename T::storage) == 4) {
#pragma unroll
            for (int i = 0; i < VE; ++i) f[i] = __uint_as_float(r.u[i]);
        } else if constexpr (VE == 1) {
            f[0] = bf16_lo(r.u[0]);
        } else {
#pragma unroll
            for (int i = 0; i < VE / 2; ++i) {
                f[2 * i] = bf16_lo(r.u[i]);
                f[2 * i + 1] = bf16_hi(r.u[i]);
            }
        }
    }
    __device__ static __forceinline__ void store(char *p, const float (&f)[VE]) {
        uint32_t u[kWords];
        if constexpr (sizeof(typename T::storage) == 4) {
#pragma unroll
            for (int i = 0; i < VE; ++i) u[i] = __float_as_uint(f[i]);
        } else if constexpr (VE == 1) {
            u[0] = pack_bf16x2(f[0], 0.f);
        } else {
#pragma unroll
            for (int i = 0; i < VE / 2; ++i) u[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
        }
        if constexpr (kBytes == 16) {
            asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};"
                         : : "l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]) : "memory");
        } else if constexpr (kBytes == 8) {
            asm volatile("st.global.v2.u32 [%0], {%1, %2};" : : "l"(p), "r"(u[0]), "r"(u[1]) : "memory");
        } else if constexpr (kBytes == 4) {
            asm volatile("st.global.u32 [%0], %1;" : : "l"(p), "r"(u[0]) : "memory");
        } else {
            asm volatile("st.global.u16 [%0], %1;" : : "l"(p), "h"((unsigned short)u[0]) : "memory");
        }
    }
    // E4M3 codes of f * inv, nearest-even, saturated at 448 (NaN stays NaN).
    __device__ static __forceinline__ void store_e4m3(char *p, const float (&f)[VE], float inv) {
        if constexpr (VE == 1) {
            *reinterpret_cast<uint8_t *>(p) = e4m3_of(f[0] * inv);
        } else {
            uint16_t h[VE / 2];
#pragma unroll
            for (int i = 0; i < VE / 2; ++i) h[i] = e4m3x2(f[2 * i] * inv, f[2 * i + 1] * inv);
            if constexpr (VE == 8) {
                asm volatile("st.global.v2.u32 [%0], {%1, %2};"
                             : : "l"(p), "r"((uint32_t)h[0] | ((uint32_t)h[1] << 16)),
                             "r"((uint32_t)h[2] | ((uint32_t)h[3] << 16)) : "memory");
            } else if constexpr (VE == 4) {
                asm volatile("st.global.u32 [%0], %1;"
                             : : "l"(p), "r"((uint32_t)h[0] | ((uint32_t)h[1] << 16)) : "memory");
            } else {
                asm volatile("st.global.u16 [%0], %1;" : : "l"(p), "h"((unsigned short)h[0]) : "memory");
            }
        }
    }
};

// Element offsets of unit u's two pieces.  Half split: (i, i + R), and what
// is past the rotated part as two halves of its own; interleaved: the 2 VE
// consecutive elements that hold pairs u VE .. u VE + VE - 1.
template <int VE, bool IL>
__device__ __forceinline__ void unit_offsets(const RopeParams &p, int u, int &a, int &b) {
    if constexpr (IL) {
        a = 2 * u * VE;
        b = a + VE;
    } else if (u < p.rot_units) {
        a = u * VE;
        b = p.R + a;
    } else {
        a = 2 * p.R + (u - p.rot_units) * VE;
        b = a + (p.head_dim / 2 - p.R);
    }
}

// Pair j of a unit held as va, vb: interleaved pairs are neighbours.
template <int VE, bool IL>
__device__ __forceinline__ void turn_unit(float (&va)[VE], float (&vb)[VE], const float (&c)[VE], const float (&s)[VE]) {
    if constexpr (IL && VE > 1) {
#pragma unroll
        for (int j = 0; j < VE / 2; ++j) {
            const float a0 = va[2 * j], b0 = va[2 * j + 1], a1 = vb[2 * j], b1 = vb[2 * j + 1];
            va[2 * j] = a0 * c[j] - b0 * s[j];
            va[2 * j + 1] = a0 * s[j] + b0 * c[j];
            vb[2 * j] = a1 * c[VE / 2 + j] - b1 * s[VE / 2 + j];
            vb[2 * j + 1] = a1 * s[VE / 2 + j] + b1 * c[VE / 2 + j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            const float a = va[j], b = vb[j];
            va[j] = a * c[j] - b * s[j];
            vb[j] = a * s[j] + b * c[j];
        }
    }
}

// ------------------------------------------------------------------ angles

// f / 2 pi as a 64-bit fixed-point fraction of a turn (whole turns dropped):
// f = M 2^(E - 150) with a 24-bit M, and M times 2^64 / 2 pi, rounded to an
// integer, is shifted into place.  Off by less than 2^-64 (1 + f) turns.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
    constexpr uint64_t kTurn = 0x28BE60DB9391054Aull;   // 2^64 / (2 pi)
    const uint32_t bits = __float_as_uint(f);
    int e = (int)((bits >> 23) & 0xFFu);
    uint64_t m = bits & 0x7FFFFFu;
    if (e == 0) e = 1; else m |= 0x800000u;
    const uint64_t lo = m * kTurn, hi = __umul64hi(m, kTurn);
    const int s = 150 - e;
    uint64_t t;
    if (s <= 0) t = s > -64 ? lo << -s : 0ull;
    else if (s < 64) t = (lo >> s) | (hi << (64 - s));
    else t = s < 128 ? hi >> (s - 64) : 0ull;
    return (bits >> 31) ? 0ull - t : t;
}

// Sine and cosine of position * fraction turns: the nearest quarter turn is
// taken off in integers, so what is rounded to fp32 is at most an eighth of a
// turn.
__device__ __forceinline__ void sincos_turns(uint64_t phase, float &s, float &c) {
    const uint32_t t = (uint32_t)((phase + 0x80000000ull) >> 32);   // 2^-32 turns
    const uint32_t q = (t + 0x20000000u) >> 30;
    const int32_t rem = (int32_t)(t - (q << 30));                   // [-2^29, 2^29)
    float sr, cr;
    sincospif((float)rem * 4.656612873077392578125e-10f, &sr, &cr); // 2^-31: half turns
    const float ss = (q & 1u) ? cr : sr, cc = (q & 1u) ? sr : cr;
    s = (q & 2u) ? -ss : ss;
    c = ((q + 1u) & 2u) ? -cc : cc;
}

__device__ __forceinline__ int axis_of(const RopeParams &p, int i) {
    return (i >= p.cut[0]) + (i >= p.cut[1]) + (i >= p.cut[2]);
}

__device__ __forceinline__ int64_t position_of(const RopeParams &p, int axis, int64_t token) {
    const int64_t at = (int64_t)axis * p.pos_stride + token;
    return p.pos64 ? static_cast<const int64_t *>(p.pos)[at] : (int64_t)static_cast<const int32_t *>(p.pos)[at];
}

// The token's cosines and sines into the warp's shared memory (cs[0 .. R) and
// cs[R .. 2R)), pair i by lane i % 32.  given: positions come from p.pos,
// else every pair takes `index`.
__device__ __forceinline__ void stage_angles(const RopeParams &p, float *cs, int lane, int64_t token, bool given,
                                             int64_t index) {
    __syncwarp();   // the warp's reads of the previous token's angles are done
    for (int i = lane; i < p.R; i += 32) {
        const int64_t at = given ? position_of(p, axis_of(p, i), token) : index;
        float s, c;
        sincos_turns((uint64_t)at * turn_fraction(p.inv_freq[i]), s, c);
        cs[i] = c;
        cs[p.R + i] = s;
    }
    __syncwarp();
}

// A lane's angles out of the staged ones.
template <int VE, int K>
struct Angles {
    float c[K][VE], s[K][VE];
    __device__ __forceinline__ void read(const RopeParams &p, const float *cs, int t) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int u = t + k * p.lanes;
            if (u < p.rot_units) {
                const float *pc = cs + u * VE, *ps = pc + p.R;
                if constexpr (VE % 4 == 0) {   // R is a multiple of VE: 16-byte aligned
#pragma unroll
                    for (int j = 0; j < VE; j += 4) {
                        const float4 a = *reinterpret_cast<const float4 *>(pc + j);
                        const float4 b = *reinterpret_cast<const float4 *>(ps + j);
                        c[k][j] = a.x, c[k][j + 1] = a.y, c[k][j + 2] = a.z, c[k][j + 3] = a.w;
                        s[k][j] = b.x, s[k][j + 1] = b.y, s[k][j + 2] = b.z, s[k][j + 3] = b.w;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < VE; ++j) {
                        c[k][j] = pc[j];
                        s[k][j] = ps[j];
                    }
                }
            }
        }
    }
};

// Sum over the G lanes of a head (G a power of two, run-time).
__device__ __forceinline__ float lanes_sum(float v, int g) {
    for (int off = g >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// The head weights (w + bias) of a lane's units; 1 without a weight.
template <typename T, int VE, int K, bool IL>
__device__ __forceinline__ void read_weight(const RopeParams &p, const void *w, int t, float (&wa)[K][VE],
                                            float (&wb)[K][VE]) {
    using P = Piece<T, VE>;
    constexpr int S = (int)sizeof(typename T::storage);
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int j = 0; j < VE; ++j) wa[k][j] = wb[k][j] = 1.f;
        const int u = t + k * p.lanes;
        if (w != nullptr && u < p.units) {
            int a, b;
            unit_offsets<VE, IL>(p, u, a, b);
            P::widen(P::load(static_cast<const char *>(w) + (int64_t)a * S), wa[k]);
            P::widen(P::load(static_cast<const char *>(w) + (int64_t)b * S), wb[k]);
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                wa[k][j] += p.w_bias;
                wb[k][j] += p.w_bias;
            }
        }
    }
}

// ------------------------------------------------------------ paged cache

// The sequence of a token: the last s with cu_tokens[s] <= token, found by
// the whole warp 32 ways at a time (a batch of single tokens, where token t
// is sequence t's, is seen at once).  Whatever cu_tokens holds, the answer is
// in [0, seqs).
__device__ __forceinline__ int sequence_of(const RopeParams &p, int64_t token, int lane) {
    if (token < p.seqs && p.cu_tokens[token] <= token && token < p.cu_tokens[token + 1]) return (int)token;
    int lo = 0, hi = p.seqs;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int64_t i = lo + (int64_t)lane * step;
        const bool in = i < hi && p.cu_tokens[i] <= token;
        const int n = __popc(__ballot_sync(0xffffffffu, in));
        const int next = lo + (n > 0 ? n - 1 : 0) * step;
        hi = hi - next < step ? hi : next + step;
        lo = next;
    }
    return lo;
}

// Byte offset of a cache row, or -1 where the page table has no valid page
// for the index (nothing is written there).
__device__ __forceinline__ int64_t cache_row(const RopeParams &p, int seq, int64_t index) {
    if (index < 0 || index > 0x7fffffff) return -1;
    const uint32_t n = (uint32_t)index / (uint32_t)p.page_size;
    if (n >= (uint32_t)p.max_pages) return -1;
    const int32_t page = p.page_table[(int64_t)seq * p.table_stride + n];
    if (page < 0 || page >= p.num_pages) return -1;
    return (int64_t)page * p.page_stride + (int64_t)((uint32_t)index - n * (uint32_t)p.page_size) * p.row_stride;
}

enum RopeMode { kRopePlain = 0, kRopeAppend = 1, kRopeAppendE4m3 = 2 };

// ----------------------------------------------------------------- forward
// grid.x: groups of blockDim / 32 tokens, one a warp; grid.y: slices of a
// token's heads.  UN head iterations are loaded before the first is used.
template <typename T, int VE, int K, bool IL, int MODE, int UN>
__global__ void __launch_bounds__(32 * kRopeMaxWarps) rope_kernel(const RopeParams p) {
    using P = Piece<T, VE>;
    using Raw = typename P::Raw;
    constexpr int S = (int)sizeof(typename T::storage);
    constexpr bool APPEND = MODE != kRopePlain;
    extern __shared__ __align__(16) float cs_all[];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int G = p.lanes, t = lane & (G - 1), group = lane / G, hpw = 32 / G;
    float *cs = cs_all + warp * 2 * p.R;
    const int heads = p.q_heads + p.k_heads + p.v_heads;
    const int turned = p.q_heads + p.k_heads;
    const int first = blockIdx.y * p.iters * hpw;
    const int last = first + p.iters * hpw < heads ? first + p.iters * hpw : heads;

    int oa[K], ob[K];   // byte offsets of the lane's pieces in a head
#pragma unroll
    for (int k = 0; k < K; ++k) {
        int a = 0, b = 0;
        if (t + k * G < p.units) unit_offsets<VE, IL>(p, t + k * G, a, b);
        oa[k] = a;
        ob[k] = b;
    }

    pdl_wait_for_inputs();
    pdl_allow_dependents();

    for (int64_t token = (int64_t)blockIdx.x * warps + warp; token < p.tokens; token += (int64_t)gridDim.x * warps) {
        int64_t index = 0, row = -1;
        if constexpr (APPEND) {
            if (token >= p.cu_tokens[p.seqs]) break;   // behind the last sequence: left as it is
            const int seq = sequence_of(p, token, lane);
            index = (int64_t)p.cache_lens[seq] + (token - p.cu_tokens[seq]);
            row = cache_row(p, seq, index);
            // the slice that holds the first key head counts the token
            if (row < 0 && p.dropped != nullptr && lane == 0 && p.q_heads >= first && p.q_heads < last)
                atomicAdd(p.dropped, 1);
        }
        const char *xr = static_cast<const char *>(p.x) + token * p.x_stride;
        char *yr = static_cast<char *>(p.y) + token * p.y_stride;
        if (first < turned) stage_angles(p, cs, lane, token, p.pos != nullptr, index);
        Angles<VE, K> ang;
        ang.read(p, cs, t);
        float wa[K][VE], wb[K][VE];
        int held = -1;   // whose weights the lane holds: 0 query, 1 key

        for (int h0 = first; h0 < last; h0 += UN * hpw) {
            Raw ra[UN][K], rb[UN][K];
#pragma unroll
            for (int n = 0; n < UN; ++n) {
                const int h = h0 + n * hpw + group;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    ra[n][k] = rb[n][k] = P::zero();
                    if (h < last && t + k * G < p.units) {
                        const char *src = xr + (int64_t)h * p.head_dim * S;
                        ra[n][k] = P::load(src + oa[k] * S);
                        rb[n][k] = P::load(src + ob[k] * S);
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < UN; ++n) {
                if (h0 + n * hpw >= last) break;   // the same for every lane
                const int h = h0 + n * hpw + group;
                const bool value = APPEND && h >= turned;
                float va[K][VE], vb[K][VE];
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    P::widen(ra[n][k], va[k]);
                    P::widen(rb[n][k], vb[k]);
                }
                if (p.norm) {
                    float acc = 0.f;
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        float sq[VE];
#pragma unroll
                        for (int j = 0; j < VE; ++j) sq[j] = fmaf(vb[k][j], vb[k][j], va[k][j] * va[k][j]);
                        acc += tree_sum(sq);
                    }
                    const float r = rsqrtf(lanes_sum(acc, G) / p.head_dim_f + p.eps);
                    if (!value) {
                        const int kind = h >= p.q_heads;
                        if (kind != held) {
                            read_weight<T, VE, K, IL>(p, kind ? p.k_w : p.q_w, t, wa, wb);
                            held = kind;
                        }
#pragma unroll
                        for (int k = 0; k < K; ++k)
#pragma unroll
                            for (int j = 0; j < VE; ++j) {
                                va[k][j] = (va[k][j] * r) * wa[k][j];
                                vb[k][j] = (vb[k][j] * r) * wb[k][j];
                            }
                    }
                }
                if (!value) {
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        if (t + k * G < p.rot_units) turn_unit<VE, IL>(va[k], vb[k], ang.c[k], ang.s[k]);
                }
                if (h >= last) continue;
                if (!APPEND || h < p.q_heads) {
                    char *dst = yr + (int64_t)h * p.head_dim * S;
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        if (t + k * G < p.units) {
                            P::store(dst + oa[k] * S, va[k]);
                            P::store(dst + ob[k] * S, vb[k]);
                        }
                } else if (row >= 0) {
                    const int j = value ? h - turned : h - p.q_heads;
                    char *dst = static_cast<char *>(value ? p.v_cache : p.k_cache) + row + (int64_t)j * p.head_stride;
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        if (t + k * G < p.units) {
                            if constexpr (MODE == kRopeAppendE4m3) {
                                const float inv = value ? p.v_inv : p.k_inv;
                                P::store_e4m3(dst + oa[k], va[k], inv);
                                P::store_e4m3(dst + ob[k], vb[k], inv);
                            } else {
                                P::store(dst + oa[k] * S, va[k]);
                                P::store(dst + ob[k] * S, vb[k]);
                            }
                        }
                }
            }
        }
    }
}

// ---------------------------------------------------------------- gradient
// Persistent blocks.  The query heads of all tokens, then the key heads, are
// a flat list of head iterations (32 / G heads of one token each); every warp
// takes an equal run of it, keeps its share of the weight's gradient in
// registers, and the block's sum goes to partial[block][kind][D].  The order
// of every sum follows from the sizes and the grid: no atomics.
// x is read only with the norm; without it dx = dy turned back.
template <typename T, int VE, int K, bool IL, bool NORM, int UN>
__global__ void __launch_bounds__(32 * kRopeMaxWarps) rope_bwd_kernel(const RopeParams p) {
    using P = Piece<T, VE>;
    using Raw = typename P::Raw;
    constexpr int S = (int)sizeof(typename T::storage);
    extern __shared__ __align__(16) float cs_all[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int G = p.lanes, t = lane & (G - 1), group = lane / G, hpw = 32 / G;
    float *cs = cs_all + warp * 2 * p.R;
    float *sums = cs_all + warps * 2 * p.R;   // [warps][D], with a weight

    int oa[K], ob[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        int a = 0, b = 0;
        if (t + k * G < p.units) unit_offsets<VE, IL>(p, t + k * G, a, b);
        oa[k] = a;
        ob[k] = b;
    }
    pdl_wait_for_inputs();
    pdl_allow_dependents();

    const int64_t all = (int64_t)gridDim.x * warps, me = (int64_t)blockIdx.x * warps + warp;
    for (int kind = 0; kind < 2; ++kind) {
        const int heads = kind ? p.k_heads : p.q_heads, base = kind ? p.q_heads : 0;
        float ga[NORM ? K : 1][VE], gb[NORM ? K : 1][VE];   // the weight's gradient
        if constexpr (NORM) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < VE; ++j) ga[k][j] = gb[k][j] = 0.f;
        }
        if (heads > 0) {
            const int per = (heads + hpw - 1) / hpw;   // iterations a token
            const int64_t total = p.tokens * per, each = total / all, extra = total - each * all;
            int64_t at = me * each + (me < extra ? me : extra);
            const int64_t end = at + each + (me < extra ? 1 : 0);
            float wa[K][VE], wb[K][VE];
            if constexpr (NORM) read_weight<T, VE, K, IL>(p, kind ? p.k_w : p.q_w, t, wa, wb);
            while (at < end) {
                const int64_t token = at / per;
                const int i0 = (int)(at - token * per);
                const int i1 = end - at < per - i0 ? i0 + (int)(end - at) : per;
                at += i1 - i0;
                stage_angles(p, cs, lane, token, true, 0);
                Angles<VE, K> ang;
                ang.read(p, cs, t);
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int j = 0; j < VE; ++j) ang.s[k][j] = -ang.s[k][j];
                const int64_t head0 = (int64_t)base * p.head_dim * S;
                const char *xr = static_cast<const char *>(p.x) + token * p.x_stride + head0;
                const char *gr = static_cast<const char *>(p.dy) + token * p.dy_stride + head0;
                char *yr = static_cast<char *>(p.y) + token * p.y_stride + head0;
                for (int i = i0; i < i1; i += UN) {
                    Raw da[UN][K], db[UN][K], xa[NORM ? UN : 1][K], xb[NORM ? UN : 1][K];
#pragma unroll
                    for (int n = 0; n < UN; ++n) {
                        const int h = (i + n) * hpw + group;
                        const bool in = i + n < i1 && h < heads;
                        const int64_t off = (int64_t)h * p.head_dim * S;
#pragma unroll
                        for (int k = 0; k < K; ++k) {
                            da[n][k] = db[n][k] = P::zero();
                            if constexpr (NORM) xa[n][k] = xb[n][k] = P::zero();
                            if (in && t + k * G < p.units) {
                                da[n][k] = P::load(gr + off + oa[k] * S);
                                db[n][k] = P::load(gr + off + ob[k] * S);
                                if constexpr (NORM) {
                                    xa[n][k] = P::load(xr + off + oa[k] * S);
                                    xb[n][k] = P::load(xr + off + ob[k] * S);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int n = 0; n < UN; ++n) {
                        if (i + n >= i1) break;   // the same for every lane
                        const int h = (i + n) * hpw + group;
                        float va[K][VE], vb[K][VE];
#pragma unroll
                        for (int k = 0; k < K; ++k) {
                            P::widen(da[n][k], va[k]);
                            P::widen(db[n][k], vb[k]);
                            if (t + k * G < p.rot_units) turn_unit<VE, IL>(va[k], vb[k], ang.c[k], ang.s[k]);
                        }
                        if constexpr (NORM) {
                            float fa[K][VE], fb[K][VE];
                            float sq = 0.f, dot = 0.f;
#pragma unroll
                            for (int k = 0; k < K; ++k) {
                                P::widen(xa[n][k], fa[k]);
                                P::widen(xb[n][k], fb[k]);
                                float u[VE], v[VE];
#pragma unroll
                                for (int j = 0; j < VE; ++j) {
                                    u[j] = fmaf(fb[k][j], fb[k][j], fa[k][j] * fa[k][j]);
                                    v[j] = fmaf(vb[k][j] * wb[k][j], fb[k][j], (va[k][j] * wa[k][j]) * fa[k][j]);
                                }
                                sq += tree_sum(u);
                                dot += tree_sum(v);
                            }
                            for (int off = G >> 1; off > 0; off >>= 1) {
                                sq += __shfl_xor_sync(0xffffffffu, sq, off);
                                dot += __shfl_xor_sync(0xffffffffu, dot, off);
                            }
                            // an idle head's zeros must add nothing, whatever eps is
                            const float r = h < heads ? rsqrtf(sq / p.head_dim_f + p.eps) : 0.f;
                            const float m = (r * r) * (dot / p.head_dim_f);
#pragma unroll
                            for (int k = 0; k < K; ++k)
#pragma unroll
                                for (int j = 0; j < VE; ++j) {
                                    ga[k][j] = fmaf(va[k][j], fa[k][j] * r, ga[k][j]);
                                    gb[k][j] = fmaf(vb[k][j], fb[k][j] * r, gb[k][j]);
                                    va[k][j] = r * (va[k][j] * wa[k][j] - fa[k][j] * m);
                                    vb[k][j] = r * (vb[k][j] * wb[k][j] - fb[k][j] * m);
                                }
                        }
                        if (h < heads) {
                            char *dst = yr + (int64_t)h * p.head_dim * S;
#pragma unroll
                            for (int k = 0; k < K; ++k)
                                if (t + k * G < p.units) {
                                    P::store(dst + oa[k] * S, va[k]);
                                    P::store(dst + ob[k] * S, vb[k]);
                                }
                        }
                    }
                }
            }
        }
        if constexpr (NORM) {
            if (p.partial != nullptr) {
                // the heads side by side in the warp, then the block's warps
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int j = 0; j < VE; ++j)
                        for (int off = G; off < 32; off <<= 1) {
                            ga[k][j] += __shfl_xor_sync(0xffffffffu, ga[k][j], off);
                            gb[k][j] += __shfl_xor_sync(0xffffffffu, gb[k][j], off);
                        }
                __syncthreads();   // the previous kind's sums are read
                if (group == 0) {
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        if (t + k * G < p.units)
#pragma unroll
                            for (int j = 0; j < VE; ++j) {
                                sums[warp * p.head_dim + oa[k] + j] = ga[k][j];
                                sums[warp * p.head_dim + ob[k] + j] = gb[k][j];
                            }
                }
                __syncthreads();
                float *out = p.partial + ((int64_t)blockIdx.x * 2 + kind) * p.head_dim;
                for (int d = threadIdx.x; d < p.head_dim; d += blockDim.x) {
                    float v = 0.f;
                    for (int w = 0; w < warps; ++w) v += sums[w * p.head_dim + d];
                    out[d] = v;
                }
            }
        }
    }
}

}  // namespace rrn
