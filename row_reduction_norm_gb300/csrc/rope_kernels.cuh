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
// side by side in a warp (a head iteration), and the batch's iterations are
// cut into equal runs, one a warp, whose next loads are under way while the
// present heads are worked on.  A token's sines and cosines are computed once
// by each warp that is at the token (each pair by one lane) and shared through
// shared memory behind warp syncs only.
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
// Blocks a SM that a shape's registers are budgeted for.
__host__ __device__ constexpr int rope_resident(int ve, int k) { return ve * k <= 8 && ve > 1 && !(ve == 4 && k == 2) ? 2 : 1; }

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
    float inv_dim, eps, w_bias;
    // rotation
    const void *pos;          // [axes][pos_stride], 32 or 64 bit; append: NULL = index in the cache
    int64_t pos_stride;
    int32_t pos64;
    int32_t cut[3];           // first pair of axes 1, 2, 3 (R where there is none)
    const float *inv_freq;    // [R]
    int32_t R;
    int32_t units, rot_units; // pair units of a head, and the rotated ones among them
    int32_t lanes;            // G: lanes a head, a power of two
    int32_t per, per_k;       // head iterations a token (gradient: of its query, its key heads)
    int64_t each, extra, each_k, extra_k;   // a warp's run of them: each, one more for the first `extra`
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
    // Weights: read by every warp, kept in L1.
    __device__ static __forceinline__ Raw load_w(const char *p) {
        Raw r;
        if constexpr (kBytes == 2) {
            r.u[0] = *reinterpret_cast<const uint16_t *>(p);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) r.u[i] = 0u;
            if constexpr (kBytes == 16) {
                const uint4 v = *reinterpret_cast<const uint4 *>(p);
                r.u[0] = v.x, r.u[1] = v.y, r.u[2] = v.z, r.u[3] = v.w;
            } else if constexpr (kBytes == 8) {
                const uint2 v = *reinterpret_cast<const uint2 *>(p);
                r.u[0] = v.x, r.u[1] = v.y;
            } else {
                r.u[0] = *reinterpret_cast<const uint32_t *>(p);
            }
        }
        return r;
    }
    // Streamed (read once) loads.
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

// The 2 x 2 turn of each pair, with whatever weights the caller folded in:
//   y_a = ca x_a + cb x_b,   y_b = cc x_a + cd x_b
// two fp32 operations an instruction.  Half split: the unit's pieces are the
// pairs' first and second elements; interleaved: neighbours are a pair.
template <int VE>
struct Turn {
    float ca[VE], cb[VE], cc[VE], cd[VE];
};

template <int VE, bool IL>
__device__ __forceinline__ void turn_unit(float (&xa)[VE], float (&xb)[VE], const Turn<VE> &m) {
    if constexpr (VE == 1) {
        const float a = xa[0], b = xb[0];
        xa[0] = fmaf(m.ca[0], a, m.cb[0] * b);
        xb[0] = fmaf(m.cc[0], a, m.cd[0] * b);
    } else if constexpr (IL) {
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            float (&x)[VE] = j < VE / 2 ? xa : xb;
            const int e = 2 * (j % (VE / 2));
            const float2 y = __ffma2_rn(make_float2(x[e], x[e]), make_float2(m.ca[j], m.cc[j]),
                                        __fmul2_rn(make_float2(x[e + 1], x[e + 1]), make_float2(m.cb[j], m.cd[j])));
            x[e] = y.x;
            x[e + 1] = y.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < VE; j += 2) {
            const float2 a = make_float2(xa[j], xa[j + 1]), b = make_float2(xb[j], xb[j + 1]);
            const float2 u = __ffma2_rn(make_float2(m.ca[j], m.ca[j + 1]), a,
                                        __fmul2_rn(make_float2(m.cb[j], m.cb[j + 1]), b));
            const float2 v = __ffma2_rn(make_float2(m.cc[j], m.cc[j + 1]), a,
                                        __fmul2_rn(make_float2(m.cd[j], m.cd[j + 1]), b));
            xa[j] = u.x, xa[j + 1] = u.y;
            xb[j] = v.x, xb[j + 1] = v.y;
        }
    }
}

// x *= r, and x *= w elementwise; sums of products.
template <int VE>
__device__ __forceinline__ void scale_by(float (&x)[VE], float r) {
    if constexpr (VE == 1) {
        x[0] *= r;
    } else {
#pragma unroll
        for (int j = 0; j < VE; j += 2) {
            const float2 v = __fmul2_rn(make_float2(x[j], x[j + 1]), make_float2(r, r));
            x[j] = v.x, x[j + 1] = v.y;
        }
    }
}

template <int VE>
__device__ __forceinline__ void times(float (&x)[VE], const float (&w)[VE]) {
    if constexpr (VE == 1) {
        x[0] *= w[0];
    } else {
#pragma unroll
        for (int j = 0; j < VE; j += 2) {
            const float2 v = __fmul2_rn(make_float2(x[j], x[j + 1]), make_float2(w[j], w[j + 1]));
            x[j] = v.x, x[j + 1] = v.y;
        }
    }
}

// acc += x * y, elements of either parity in a sum of their own.
template <int VE>
__device__ __forceinline__ void dot_into(float2 &acc, const float (&x)[VE], const float (&y)[VE]) {
    if constexpr (VE == 1) {
        acc.x = fmaf(x[0], y[0], acc.x);
    } else {
#pragma unroll
        for (int j = 0; j < VE; j += 2)
            acc = __ffma2_rn(make_float2(x[j], x[j + 1]), make_float2(y[j], y[j + 1]), acc);
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
// turn, t in [-pi/4, pi/4], where the Taylor series up to t^9 and t^10 are off
// by t^11 / 11! < 2e-9 and t^12 / 12! < 2e-10.
__device__ __forceinline__ void sincos_turns(uint64_t phase, float &s, float &c) {
    const uint32_t t32 = (uint32_t)((phase + 0x80000000ull) >> 32);   // 2^-32 turns
    const uint32_t q = (t32 + 0x20000000u) >> 30;
    const float t = (float)(int32_t)(t32 - (q << 30)) * 1.46291807926715968e-9f;   // 2 pi / 2^32
    const float z = t * t;
    float sr = fmaf(z, 2.75573192e-6f, -1.98412698e-4f);   // 1/9!, -1/7!, 1/5!, -1/3!
    sr = fmaf(z, sr, 8.33333333e-3f);
    sr = fmaf(z, sr, -1.66666667e-1f);
    sr = fmaf(t * z, sr, t);
    float cr = fmaf(z, -2.75573192e-7f, 2.48015873e-5f);   // -1/10!, 1/8!, -1/6!, 1/4!, -1/2!
    cr = fmaf(z, cr, -1.38888889e-3f);
    cr = fmaf(z, cr, 4.16666667e-2f);
    cr = fmaf(z, cr, -0.5f);
    cr = fmaf(z, cr, 1.f);
    const float ss = (q & 1u) ? cr : sr, cc = (q & 1u) ? sr : cr;
    s = __uint_as_float(__float_as_uint(ss) ^ ((q & 2u) << 30));
    c = __uint_as_float(__float_as_uint(cc) ^ (((q + 1u) & 2u) << 30));
}

__device__ __forceinline__ int axis_of(const RopeParams &p, int i) {
    return (i >= p.cut[0]) + (i >= p.cut[1]) + (i >= p.cut[2]);
}

__device__ __forceinline__ int64_t position_of(const RopeParams &p, int axis, int64_t token) {
    const int64_t at = (int64_t)axis * p.pos_stride + token;
    return p.pos64 ? static_cast<const int64_t *>(p.pos)[at] : (int64_t)static_cast<const int32_t *>(p.pos)[at];
}

// Shared memory of a block: the pairs' turn fractions [R] (once a block),
// then for each warp the cosines and sines [2][R] of the token it is at.
__device__ __forceinline__ void stage_fractions(const RopeParams &p, uint64_t *frac) {
    for (int i = threadIdx.x; i < p.R; i += blockDim.x) frac[i] = turn_fraction(p.inv_freq[i]);
    __syncthreads();
}

// The token's cosines and sines, pair i by lane i % 32.  given: positions
// come from p.pos, else every pair takes `index`.
__device__ __forceinline__ void stage_angles(const RopeParams &p, const uint64_t *frac, float *cs, int lane,
                                             int64_t token, bool given, int64_t index) {
    __syncwarp();   // the warp's reads of the previous token's angles are done
    for (int i = lane; i < p.R; i += 32) {
        const int64_t at = given ? position_of(p, axis_of(p, i), token) : index;
        float s, c;
        sincos_turns((uint64_t)at * frac[i], s, c);
        cs[i] = c;
        cs[p.R + i] = s;
    }
    __syncwarp();
}

// VE consecutive fp32 values out of shared memory (16-byte aligned where VE
// is a multiple of 4: R is then one too).
template <int VE>
__device__ __forceinline__ void read_floats(const float *p, float (&v)[VE]) {
    if constexpr (VE % 4 == 0) {
#pragma unroll
        for (int j = 0; j < VE; j += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(p + j);
            v[j] = a.x, v[j + 1] = a.y, v[j + 2] = a.z, v[j + 3] = a.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < VE; ++j) v[j] = p[j];
    }
}

// Sum over the G lanes of a head (G a power of two, run-time).
__device__ __forceinline__ float lanes_sum(float v, int g) {
    if (g > 1) v += __shfl_xor_sync(0xffffffffu, v, 1);
    if (g > 2) v += __shfl_xor_sync(0xffffffffu, v, 2);
    if (g > 4) v += __shfl_xor_sync(0xffffffffu, v, 4);
    if (g > 8) v += __shfl_xor_sync(0xffffffffu, v, 8);
    if (g > 16) v += __shfl_xor_sync(0xffffffffu, v, 16);
    return v;
}

// The head weights (w + bias) of unit u; 1 without a weight.
template <typename T, int VE, bool IL>
__device__ __forceinline__ void read_weight(const RopeParams &p, const void *w, int u, float (&wa)[VE], float (&wb)[VE]) {
    using P = Piece<T, VE>;
    constexpr int S = (int)sizeof(typename T::storage);
#pragma unroll
    for (int j = 0; j < VE; ++j) wa[j] = wb[j] = 1.f;
    if (w != nullptr && u < p.units) {
        int a, b;
        unit_offsets<VE, IL>(p, u, a, b);
        P::widen(P::load_w(static_cast<const char *>(w) + a * S), wa);
        P::widen(P::load_w(static_cast<const char *>(w) + b * S), wb);
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            wa[j] += p.w_bias;
            wb[j] += p.w_bias;
        }
    }
}

// The turn of unit u with the weight of its elements folded in (y = turn of
// w x); units past the rotated part hold w in ca and cd alone, which the
// caller applies without the cross terms.
template <typename T, int VE, bool IL>
__device__ __forceinline__ void weighted_turn(const RopeParams &p, const float *cs, const void *w, int u, Turn<VE> &m) {
    float wa[VE], wb[VE];
    read_weight<T, VE, IL>(p, w, u, wa, wb);
    if (u < p.rot_units) {
        float c[VE], s[VE];
        read_floats<VE>(cs + u * VE, c);
        read_floats<VE>(cs + p.R + u * VE, s);
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            // the weights of pair j's two elements
            const float w0 = !IL || VE == 1 ? wa[j] : (2 * j < VE ? wa[(2 * j) % VE] : wb[(2 * j) % VE]);
            const float w1 = !IL || VE == 1 ? wb[j] : (2 * j < VE ? wa[(2 * j + 1) % VE] : wb[(2 * j + 1) % VE]);
            m.ca[j] = w0 * c[j];
            m.cb[j] = -w1 * s[j];
            m.cc[j] = w0 * s[j];
            m.cd[j] = w1 * c[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            m.ca[j] = wa[j];
            m.cd[j] = wb[j];
            m.cb[j] = m.cc[j] = 0.f;
        }
    }
}

// The flat list of head iterations (32 / G heads of one token each, `per` a
// token) cut into equal runs, one a warp.
struct Run {
    int64_t token, at, end;
    int it;
    __device__ __forceinline__ void start(int64_t warp, int64_t each, int64_t extra, int per) {
        at = warp * each + (warp < extra ? warp : extra);
        end = at + each + (warp < extra ? 1 : 0);
        token = ((at | per) >> 32) == 0 ? (int64_t)((uint32_t)at / (uint32_t)per) : at / per;
        it = (int)(at - token * per);
    }
    // Iterations of the run from here on that are of this token, at most n.
    __device__ __forceinline__ int count(int per, int n) const {
        const int64_t left = end - at;
        const int c = per - it < n ? per - it : n;
        return left < c ? (int)left : c;
    }
    __device__ __forceinline__ void advance(int n, int per) {
        at += n;
        it += n;
        if (it == per) {
            it = 0;
            ++token;
        }
    }
};

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
// UN head iterations are loaded while the UN before them are worked on.  A
// value's weight is folded into its token's turn, so a head costs its sum of
// squares, one 2 x 2 turn a pair and one product with r.
template <typename T, int VE, int K, bool IL, int MODE, int UN>
__global__ void __launch_bounds__(32 * kRopeMaxWarps, rope_resident(VE, K)) rope_kernel(const RopeParams p) {
    using P = Piece<T, VE>;
    using Raw = typename P::Raw;
    constexpr int S = (int)sizeof(typename T::storage);
    constexpr bool APPEND = MODE != kRopePlain;
    extern __shared__ __align__(16) unsigned char smem[];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int G = p.lanes, t = lane & (G - 1), group = lane / G, hpw = 32 / G;
    uint64_t *frac = reinterpret_cast<uint64_t *>(smem);
    float *cs = reinterpret_cast<float *>(frac + ((p.R + 1) & ~1)) + warp * 2 * p.R;
    const int heads = p.q_heads + p.k_heads + p.v_heads, turned = p.q_heads + p.k_heads;
    const int per = p.per;

    int oa[K], ob[K];   // byte offsets of the lane's pieces in a head; -1: no unit
#pragma unroll
    for (int k = 0; k < K; ++k) {
        oa[k] = ob[k] = -1;
        if (t + k * G < p.units) {
            unit_offsets<VE, IL>(p, t + k * G, oa[k], ob[k]);
            oa[k] *= S;
            ob[k] *= S;
        }
    }
    const int head_bytes = p.head_dim * S;

    Run run;
    run.start((int64_t)blockIdx.x * warps + warp, p.each, p.extra, per);
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    if constexpr (APPEND) {   // rows behind the last sequence are left as they are
        const int64_t valid = p.cu_tokens[p.seqs];
        const int64_t most = (valid < 0 ? 0 : valid) * per;
        if (run.end > most) run.end = most;
    }

    auto load = [&](const Run &r, int n, Raw (&ra)[UN][K], Raw (&rb)[UN][K]) {
        const char *src = static_cast<const char *>(p.x) + r.token * p.x_stride;
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int h = (r.it + i) * hpw + group;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                ra[i][k] = rb[i][k] = P::zero();
                if (i < n && h < heads && oa[k] >= 0) {
                    ra[i][k] = P::load(src + (h * head_bytes + oa[k]));
                    rb[i][k] = P::load(src + (h * head_bytes + ob[k]));
                }
            }
        }
    };

    int64_t row = -1;
    int held = -1;              // whose weights are in m: 0 query, 1 key
    Turn<VE> m[K];
    // One batch: `now` holds it, the next one's loads go into `next`.
    auto step = [&](Raw (&na)[UN][K], Raw (&nb)[UN][K], Raw (&xa)[UN][K], Raw (&xb)[UN][K], bool first) {
        const int n = run.count(per, UN);
        Run ahead = run;
        ahead.advance(n, per);
        const int more = ahead.count(per, UN);
        if (more > 0) load(ahead, more, xa, xb);
        if (first || run.it == 0) {   // a token the warp has not been at
            int64_t index = 0;
            if constexpr (APPEND) {
                const int seq = sequence_of(p, run.token, lane);
                index = (int64_t)p.cache_lens[seq] + (run.token - p.cu_tokens[seq]);
                row = cache_row(p, seq, index);
            }
            if (run.it * hpw < turned) stage_angles(p, frac, cs, lane, run.token, p.pos != nullptr, index);
            held = -1;
        }
        char *yr = static_cast<char *>(p.y) + run.token * p.y_stride;
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            if (i >= n) break;   // the same for every lane
            const int h = (run.it + i) * hpw + group;
            const bool value = APPEND && h >= turned;
            float va[K][VE], vb[K][VE];
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                P::widen(na[i][k], va[k]);
                P::widen(nb[i][k], vb[k]);
                dot_into<VE>(acc, va[k], va[k]);
                dot_into<VE>(acc, vb[k], vb[k]);
            }
            float r = 1.f;
            if (p.norm) r = rsqrtf(fmaf(lanes_sum(acc.x + acc.y, G), p.inv_dim, p.eps));
            if (!value) {
                const int kind = h >= p.q_heads;
                if (kind != held) {
                    held = kind;
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        weighted_turn<T, VE, IL>(p, cs, kind ? p.k_w : p.q_w, t + k * G, m[k]);
                }
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (t + k * G < p.rot_units) {
                        turn_unit<VE, IL>(va[k], vb[k], m[k]);
                    } else {
                        times<VE>(va[k], m[k].ca);
                        times<VE>(vb[k], m[k].cd);
                    }
                    if (p.norm) {
                        scale_by<VE>(va[k], r);
                        scale_by<VE>(vb[k], r);
                    }
                }
            }
            if (!APPEND || h < p.q_heads) {
                char *dst = yr + (int64_t)h * head_bytes;
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (h < heads && oa[k] >= 0) {
                        P::store(dst + oa[k], va[k]);
                        P::store(dst + ob[k], vb[k]);
                    }
            } else {
                if (row < 0) {
                    if (h == p.q_heads && t == 0 && p.dropped != nullptr) atomicAdd(p.dropped, 1);
                } else if (h < heads) {
                    const int j = value ? h - turned : h - p.q_heads;
                    char *dst = static_cast<char *>(value ? p.v_cache : p.k_cache) + row + (int64_t)j * p.head_stride;
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        if (oa[k] >= 0) {
                            if constexpr (MODE == kRopeAppendE4m3) {
                                const float inv = value ? p.v_inv : p.k_inv;
                                P::store_e4m3(dst + oa[k] / S, va[k], inv);
                                P::store_e4m3(dst + ob[k] / S, vb[k], inv);
                            } else {
                                P::store(dst + oa[k], va[k]);
                                P::store(dst + ob[k], vb[k]);
                            }
                        }
                }
            }
        }
        run = ahead;
    };

    // the first loads are on their way while the block prepares its table
    Raw ra[UN][K], rb[UN][K], sa[UN][K], sb[UN][K];
    if (run.at < run.end) load(run, run.count(per, UN), ra, rb);
    stage_fractions(p, frac);
    bool first = true;
    while (run.at < run.end) {
        step(ra, rb, sa, sb, first);
        first = false;
        if (run.at >= run.end) break;
        step(sa, sb, ra, rb, false);
    }
}

// ---------------------------------------------------------------- gradient
// Persistent blocks.  The query heads of all tokens, then the key heads, are
// a flat list of head iterations each; every warp takes an equal run of it,
// keeps its share of the weight's gradient in registers, and the block's sum
// goes to partial[block][kind][D].  The order of every sum follows from the
// sizes and the grid: no atomics.
// x is read only with the norm; without it dx = dy turned back.
template <typename T, int VE, int K, bool IL, bool NORM, int UN>
__global__ void __launch_bounds__(32 * kRopeMaxWarps, rope_resident(VE, K)) rope_bwd_kernel(const RopeParams p) {
    using P = Piece<T, VE>;
    using Raw = typename P::Raw;
    constexpr int S = (int)sizeof(typename T::storage);
    constexpr int KN = NORM ? K : 1, UX = NORM ? UN : 1;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int G = p.lanes, t = lane & (G - 1), group = lane / G, hpw = 32 / G;
    uint64_t *frac = reinterpret_cast<uint64_t *>(smem);
    float *cs_all = reinterpret_cast<float *>(frac + ((p.R + 1) & ~1));
    float *cs = cs_all + warp * 2 * p.R;
    float *wsm = cs_all + warps * 2 * p.R;    // the kind's weight in lane order, with the norm
    float *sums = wsm + (NORM ? K * VE * 64 : 0);   // [warps][D], with a weight's gradient

    int oa[K], ob[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        oa[k] = ob[k] = -1;
        if (t + k * G < p.units) {
            unit_offsets<VE, IL>(p, t + k * G, oa[k], ob[k]);
            oa[k] *= S;
            ob[k] *= S;
        }
    }
    const int head_bytes = p.head_dim * S;
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    stage_fractions(p, frac);

    const int64_t me = (int64_t)blockIdx.x * warps + warp;
    for (int kind = 0; kind < 2; ++kind) {
        const int heads = kind ? p.k_heads : p.q_heads;
        const int per = kind ? p.per_k : p.per;   // iterations a token
        float ga[KN][VE], gb[KN][VE];             // the weight's gradient
#pragma unroll
        for (int k = 0; k < KN; ++k)
#pragma unroll
            for (int j = 0; j < VE; ++j) ga[k][j] = gb[k][j] = 0.f;
        if (heads > 0) {
            Run run;
            run.start(me, kind ? p.each_k : p.each, kind ? p.extra_k : p.extra, per);
            if constexpr (NORM) {   // the kind's weights, unit by unit: 2 VE floats each
                __syncthreads();
                for (int u = threadIdx.x; u < p.units; u += blockDim.x) {
                    float wa[VE], wb[VE];
                    read_weight<T, VE, IL>(p, kind ? p.k_w : p.q_w, u, wa, wb);
#pragma unroll
                    for (int j = 0; j < VE; ++j) {
                        wsm[2 * VE * u + j] = wa[j];
                        wsm[2 * VE * u + VE + j] = wb[j];
                    }
                }
                __syncthreads();
            }
            const int64_t head0 = (int64_t)(kind ? p.q_heads : 0) * head_bytes;
            const char *x0 = static_cast<const char *>(p.x) + head0, *g0 = static_cast<const char *>(p.dy) + head0;
            char *y0 = static_cast<char *>(p.y) + head0;

            auto load = [&](const Run &r, int n, Raw (&da)[UN][K], Raw (&db)[UN][K], Raw (&xa)[UX][K],
                            Raw (&xb)[UX][K]) {
                const char *gr = g0 + r.token * p.dy_stride;
                const char *xr = x0 + r.token * p.x_stride;
#pragma unroll
                for (int i = 0; i < UN; ++i) {
                    const int h = (r.it + i) * hpw + group;
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        da[i][k] = db[i][k] = P::zero();
                        if constexpr (NORM) xa[i][k] = xb[i][k] = P::zero();
                        if (i < n && h < heads && oa[k] >= 0) {
                            da[i][k] = P::load(gr + (h * head_bytes + oa[k]));
                            db[i][k] = P::load(gr + (h * head_bytes + ob[k]));
                            if constexpr (NORM) {
                                xa[i][k] = P::load(xr + (h * head_bytes + oa[k]));
                                xb[i][k] = P::load(xr + (h * head_bytes + ob[k]));
                            }
                        }
                    }
                }
            };

            auto step = [&](Raw (&da)[UN][K], Raw (&db)[UN][K], Raw (&xa)[UX][K], Raw (&xb)[UX][K], Raw (&ea)[UN][K],
                            Raw (&eb)[UN][K], Raw (&za)[UX][K], Raw (&zb)[UX][K], bool first) {
                const int n = run.count(per, UN);
                Run ahead = run;
                ahead.advance(n, per);
                const int more = ahead.count(per, UN);
                if (more > 0) load(ahead, more, ea, eb, za, zb);
                if (first || run.it == 0) {
                    stage_angles(p, frac, cs, lane, run.token, true, 0);
                }
                char *yr = y0 + run.token * p.y_stride;
#pragma unroll
                for (int i = 0; i < UN; ++i) {
                    if (i >= n) break;   // the same for every lane
                    const int h = (run.it + i) * hpw + group;
                    // cosines, sines and weights come from shared memory at each
                    // use: held in registers they spilled (128 a thread)
                    float va[K][VE], vb[K][VE], fa[KN][VE], fb[KN][VE];
                    float2 sq = make_float2(0.f, 0.f), dot = sq;
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        P::widen(da[i][k], va[k]);
                        P::widen(db[i][k], vb[k]);
                        const int u = t + k * G;
                        if (u < p.rot_units) {
                            Turn<VE> m;
                            read_floats<VE>(cs + u * VE, m.ca);
                            read_floats<VE>(cs + p.R + u * VE, m.cb);
#pragma unroll
                            for (int j = 0; j < VE; ++j) {
                                m.cc[j] = -m.cb[j];
                                m.cd[j] = m.ca[j];
                            }
                            turn_unit<VE, IL>(va[k], vb[k], m);
                        }
                        if constexpr (NORM) {
                            float wa[VE], wb[VE];
                            const float *pw = wsm + 2 * VE * (u < p.units ? u : 0);
                            read_floats<VE>(pw, wa);
                            read_floats<VE>(pw + VE, wb);
                            P::widen(xa[i][k], fa[k]);
                            P::widen(xb[i][k], fb[k]);
                            dot_into<VE>(sq, fa[k], fa[k]);
                            dot_into<VE>(sq, fb[k], fb[k]);
                            float ta[VE], tb[VE];
#pragma unroll
                            for (int j = 0; j < VE; ++j) ta[j] = fa[k][j], tb[j] = fb[k][j];
                            times<VE>(ta, va[k]);   // x g, summed with the weight
                            times<VE>(tb, vb[k]);
                            dot_into<VE>(dot, ta, wa);
                            dot_into<VE>(dot, tb, wb);
                        }
                    }
                    if constexpr (NORM) {
                        const float s1 = lanes_sum(sq.x + sq.y, G), s2 = lanes_sum(dot.x + dot.y, G);
                        // an idle head's zeros must add nothing, whatever eps is
                        const float r = h < heads ? rsqrtf(fmaf(s1, p.inv_dim, p.eps)) : 0.f;
                        const float mean = (s2 * p.inv_dim) * r;   // dx = r (w g - (x r) mean)
#pragma unroll
                        for (int k = 0; k < K; ++k) {
                            scale_by<VE>(fa[k], r);
                            scale_by<VE>(fb[k], r);
#pragma unroll
                            for (int j = 0; j < VE; ++j) {
                                ga[k][j] = fmaf(va[k][j], fa[k][j], ga[k][j]);
                                gb[k][j] = fmaf(vb[k][j], fb[k][j], gb[k][j]);
                            }
                            const int u = t + k * G;
                            float wa[VE], wb[VE];
                            const float *pw = wsm + 2 * VE * (u < p.units ? u : 0);
                            read_floats<VE>(pw, wa);
                            read_floats<VE>(pw + VE, wb);
                            times<VE>(va[k], wa);
                            times<VE>(vb[k], wb);
#pragma unroll
                            for (int j = 0; j < VE; ++j) {
                                va[k][j] = fmaf(fa[k][j], -mean, va[k][j]);
                                vb[k][j] = fmaf(fb[k][j], -mean, vb[k][j]);
                            }
                            scale_by<VE>(va[k], r);
                            scale_by<VE>(vb[k], r);
                        }
                    }
                    char *dst = yr + (int64_t)h * head_bytes;
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        if (h < heads && oa[k] >= 0) {
                            P::store(dst + oa[k], va[k]);
                            P::store(dst + ob[k], vb[k]);
                        }
                }
                run = ahead;
            };

            Raw da[UN][K], db[UN][K], xa[UX][K], xb[UX][K], ea[UN][K], eb[UN][K], za[UX][K], zb[UX][K];
            bool first = true;
            if (run.at < run.end) load(run, run.count(per, UN), da, db, xa, xb);
            while (run.at < run.end) {
                step(da, db, xa, xb, ea, eb, za, zb, first);
                first = false;
                if (run.at >= run.end) break;
                step(ea, eb, za, zb, da, db, xa, xb, false);
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
                        if (oa[k] >= 0)
#pragma unroll
                            for (int j = 0; j < VE; ++j) {
                                sums[warp * p.head_dim + oa[k] / S + j] = ga[k][j];
                                sums[warp * p.head_dim + ob[k] / S + j] = gb[k][j];
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
