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
// the rotation needs no exchange.  G lanes share a head (as many as it has
// units), 32 / G heads run side by side in a warp (a head iteration).  A block takes an equal run of
// tokens in tiles of one token a warp: each warp makes its token's table of
// cosines and sines in shared memory, then the tile's head iterations go
// round the warps.  Every factor of a head (cosine, sine, weights) is read
// from shared memory where it is used, so a thread needs few registers and
// many warps hide the loads' latency: with the factors in registers 16 warps
// a SM were resident and bf16 8192 tokens x 40 heads of 128 took 36 us.
//
// Angles.  Positions are integers, so only the fraction of a turn per step
// matters: inv_freq / 2 pi is held as a 64-bit fixed-point fraction of a turn
// and position * fraction wraps modulo 2^64, exactly modulo one turn.  No
// precision is lost to far positions (|position| (1 + f) 2^-64 turns), no 64-bit
// floating point is used (slow on this GPU), and no table of cosines has to
// be kept or read.
#pragma once

#include "async_copy.cuh"
#include "finish.cuh"
#include "rmsnorm_kernels.cuh"

namespace rrn {

constexpr int kRopeMaxDim = 512;      // head_dim
constexpr int kRopeMaxAxes = 4;
constexpr int kRopeMaxWarps = 8;      // warps a block
// Blocks a SM that a shape's registers are budgeted for.  Measured on GB300,
// bf16 8192 tokens x 40 heads of 128, when the factors had moved to shared
// memory: the forward 31.0 us with four blocks (64 registers a thread), 32.5
// with three, 38.7 with five (which spill); the gradient 63.5 us with two, 75.5
// with three.  Kernels of their own for whole heads and the gradient's ring
// took them to 30.4 and 43.9 us.
// bytes: of a piece.
__host__ __device__ constexpr int rope_resident(int bytes, int k) { return bytes * k <= 16 && bytes >= 4 ? 4 : 2; }
// The gradient has 112 registers a thread where two blocks fit: what they leave
// is a block of the column sums' (256 threads of 32), which then stands ready
// when they end.  One register more cost 0.5 us (43.6 -> 44.1 us; 2326 tokens x
// 4 heads 6.7 -> 7.4 us).
__host__ __device__ constexpr int rope_bwd_registers(int bytes, int k) { return bytes * k <= 16 && bytes >= 4 ? 112 : 255; }

struct RopeParams {
    const void *x;            // packed token rows (query, key, [value] heads)
    const void *dy;           // gradient: of the rotated rows
    void *y;                  // rotated rows (append: of the query heads); gradient: dx
    const void *q_w, *k_w;    // nullable
    float *partial;           // gradient: [kind][blocks][partial_ld] sums of the weights' gradients, or NULL
    void *dq_w, *dk_w;        // gradient of a single cluster: the weights' gradients, or NULL
    int32_t partial_ld;
    int64_t tokens;
    int64_t x_stride, y_stride, dy_stride;   // bytes between token rows
    int32_t q_heads, k_heads, v_heads;       // v_heads: append only
    int32_t head_dim;
    int32_t norm;
    float inv_dim, eps, w_bias;
    // rotation
    const void *pos;          // [axes][pos_stride], 32 or 64 bit; append: NULL = index in the cache
    int64_t pos_stride;
    int32_t pos64, axes;
    int32_t cut[3];           // first pair of axes 1, 2, 3 (R where there is none)
    const float *inv_freq;    // [R]
    int32_t R;
    int32_t units, rot_units; // pair units of a head, and the rotated ones among them
    int32_t lanes;            // G: lanes a head
    int32_t heads_a_warp;     // 32 / G, of one head iteration
    int32_t iters, iters_k;   // head iterations a job (gradient: of query heads, of key heads)
    int32_t slices, tile;     // jobs a token; jobs a tile (1 or kRopeMaxWarps)
    int32_t q_warps;          // gradient: warps of a block that take the query heads
    int64_t each, extra;      // a block's run of jobs: each, one more for the first `extra`
    // paged cache (append)
    const int32_t *cu_tokens, *cache_lens, *page_table;
    int64_t table_stride;
    int32_t seqs, max_pages, num_pages, page_size;
    void *k_cache, *v_cache;
    int64_t page_stride, row_stride, head_stride;   // bytes
    float k_inv, v_inv;       // 8-bit cache: 1 / scale, rounded
    float k_scale, v_scale;
    int32_t settle;           // an inverse is not exact
    int32_t *dropped;
};

// ------------------------------------------------------------- 8-bit codes
// What E4M3 code v / scale has, without a division.  v * (1 / scale), both
// rounded, is within 2 steps (2^-23) of the quotient, so its code can be
// another one only next to a point halfway between two codes.  Those points
// have at most four leading bits (the low 19 bits of their mantissa are 0), and
// there one fused multiply-add tells on which side of the point the quotient
// lies: v - point * scale is rounded once, so its sign is exact (scales are
// within 2^-100 .. 2^100: nothing that matters underflows).
__device__ __forceinline__ float settle_quotient(float q, float v, float scale) {
    const uint32_t near = __float_as_uint(q) + 3u;
    if ((near & 0x7FFFFu) > 6u || !(fabsf(q) < 512.f)) return q;
    const uint32_t point = near & ~0x7FFFFu;
    const float over = fmaf(-__uint_as_float(point), scale, v);
    if (over == 0.f) return __uint_as_float(point);
    // one step to the quotient's side of the point
    return __uint_as_float((__float_as_uint(over) ^ point) >> 31 ? point - 1u : point + 1u);
}

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
    // A 16-byte piece into shared memory.
    __device__ static __forceinline__ void give(unsigned char *smem, const Raw &r) {
        static_assert(kBytes == 16, "16-byte pieces");
        *reinterpret_cast<uint4 *>(smem) = make_uint4(r.u[0], r.u[1], r.u[2], r.u[3]);
    }
    // The same piece on its way to shared memory, and read back from there.
    // L1: a lane's other piece is in the same 32 bytes (interleaved pairs).
    template <bool L1>
    __device__ static __forceinline__ void copy(char *smem, const char *p) { copy_async<kBytes, L1>(smem, p); }
    __device__ static __forceinline__ Raw take(const char *smem) {
        Raw r = zero();
        if constexpr (kBytes == 16) {
            const uint4 v = *reinterpret_cast<const uint4 *>(smem);
            r.u[0] = v.x, r.u[1] = v.y, r.u[2] = v.z, r.u[3] = v.w;
        } else if constexpr (kBytes == 8) {
            const uint2 v = *reinterpret_cast<const uint2 *>(smem);
            r.u[0] = v.x, r.u[1] = v.y;
        } else if constexpr (kBytes == 4) {
            r.u[0] = *reinterpret_cast<const uint32_t *>(smem);
        }
        return r;
    }
    // E4M3 codes of the quotients f / scale, nearest-even, saturated at 448 (NaN
    // stays NaN).  SETTLE: inv is not exact.
    template <bool SETTLE>
    __device__ static __forceinline__ void store_e4m3(char *p, const float (&f)[VE], float inv, float scale) {
        float q[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) q[i] = f[i] * inv;
        if constexpr (SETTLE) {
#pragma unroll
            for (int i = 0; i < VE; ++i) q[i] = settle_quotient(q[i], f[i], scale);
        }
        if constexpr (VE == 1) {
            *reinterpret_cast<uint8_t *>(p) = e4m3_of(q[0]);
        } else {
            uint16_t h[VE / 2];
#pragma unroll
            for (int i = 0; i < VE / 2; ++i) h[i] = e4m3x2(q[2 * i], q[2 * i + 1]);
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

// Factors are read for N pairs of a unit at a time, as two runs of N values;
// the elements they go with are two runs of N as well.  Half split: the
// pairs' first elements (q .. q + N - 1 of piece a) and their second ones (of
// piece b).  Interleaved: the 2 N neighbours in order.
__host__ __device__ constexpr int pairs_at_once(int ve) { return ve < 4 ? ve : 4; }
template <int VE, bool IL>
__device__ __forceinline__ constexpr int run_a(int q) { return IL ? 2 * q : q; }
template <int VE, bool IL>
__device__ __forceinline__ constexpr int run_b(int q) { return IL ? 2 * q + pairs_at_once(VE) : VE + q; }

// Where the first run of the N pairs from q on of unit u stands in a table of
// factors; the second run is kRopeTable further.  The lanes of a head read
// consecutive 16 (8, 4) bytes, and every table has as many places whatever the
// head's size (VE * K * 32 lanes at most), so one address serves all of a
// unit's reads.
constexpr int kRopeTable = 256;
template <int VE>
__device__ __forceinline__ constexpr int table_at(int u, int q) {
    constexpr int N = pairs_at_once(VE);
    return (q / N) * 32 * N + u * N;
}
// Where a factor of pair i's first (second) element stands.
template <int VE, bool IL>
__device__ __forceinline__ int factor_at(int i, int second) {
    constexpr int N = pairs_at_once(VE);
    const int j = i % N, at = table_at<VE>(i / VE, i % VE);
    const int place = IL ? 2 * j + second : second * N + j;
    return at + place % N + (place / N) * kRopeTable;
}

template <int N>
__device__ __forceinline__ void read_table(const float *p, float (&v)[N]) {
    if constexpr (N == 4) {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    } else if constexpr (N == 2) {
        const float2 a = *reinterpret_cast<const float2 *>(p);
        v[0] = a.x, v[1] = a.y;
    } else {
        v[0] = p[0];
    }
}

// Two runs of N elements turned by their factors f, g (half split: cosines and
// sines; interleaved: cosine, sine of each pair in turn); BACK: by the
// opposite angle.  Two fp32 operations an instruction.
template <bool IL, bool BACK, int N>
__device__ __forceinline__ void turn_runs(float *a, float *b, const float (&f)[N], const float (&g)[N]) {
    if constexpr (N == 1) {
        const float x = a[0], y = b[0], s = BACK ? -g[0] : g[0];
        a[0] = fmaf(x, f[0], -(y * s));
        b[0] = fmaf(x, s, y * f[0]);
    } else if constexpr (IL) {   // one at a time: packing neighbours both ways costs more than it saves
#pragma unroll
        for (int j = 0; j < 2 * N; j += 2) {
            float *e = j < N ? a + j : b + (j - N);
            const float c = j < N ? f[j % N] : g[j % N], x = e[0], y = e[1];
            const float s = BACK ? -(j < N ? f[j % N + 1] : g[j % N + 1]) : (j < N ? f[j % N + 1] : g[j % N + 1]);
            e[0] = fmaf(x, c, -(y * s));
            e[1] = fmaf(x, s, y * c);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float2 x = make_float2(a[j], a[j + 1]), y = make_float2(b[j], b[j + 1]);
            const float2 c = make_float2(f[j], f[j + 1]), s = make_float2(g[j], g[j + 1]);
            const float2 n = make_float2(-s.x, -s.y);
            const float2 u = __ffma2_rn(x, c, __fmul2_rn(y, BACK ? s : n));
            const float2 v = __ffma2_rn(x, BACK ? n : s, __fmul2_rn(y, c));
            a[j] = u.x, a[j + 1] = u.y;
            b[j] = v.x, b[j + 1] = v.y;
        }
    }
}

// Elementwise on a run of N: x *= y;  x *= r;  acc += x y;  x = fma(y, r, x).
template <int N>
__device__ __forceinline__ void run_times(float *x, const float (&y)[N]) {
    if constexpr (N == 1) {
        x[0] *= y[0];
    } else {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float2 v = __fmul2_rn(make_float2(x[j], x[j + 1]), make_float2(y[j], y[j + 1]));
            x[j] = v.x, x[j + 1] = v.y;
        }
    }
}
template <int N>
__device__ __forceinline__ void run_scale(float *x, float r) {
    float y[N];
#pragma unroll
    for (int j = 0; j < N; ++j) y[j] = r;
    run_times<N>(x, y);
}
template <int N>
__device__ __forceinline__ void run_fma(float *acc, const float *x, const float *y) {
    if constexpr (N == 1) {
        acc[0] = fmaf(x[0], y[0], acc[0]);
    } else {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float2 v = __ffma2_rn(make_float2(x[j], x[j + 1]), make_float2(y[j], y[j + 1]),
                                        make_float2(acc[j], acc[j + 1]));
            acc[j] = v.x, acc[j + 1] = v.y;
        }
    }
}
template <int N>
__device__ __forceinline__ void run_dot(float2 &acc, const float *x, const float *y) {
    if constexpr (N == 1) {
        acc.x = fmaf(x[0], y[0], acc.x);
    } else {
#pragma unroll
        for (int j = 0; j < N; j += 2)
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

// Shared memory of a block: the pairs' turn fractions (64 bits each), the
// weights of the pairs' first and second elements (a table each for query and
// key), then two tiles of a table of cosines and one of sines a token.
// The gradient adds its ring of pieces on their way.
__host__ __device__ constexpr int rope_ring_bytes(int bytes, int k, bool norm) {
    return bytes < 4 ? 0 : 2 * (norm ? 4 : 2) * k * 32 * kRopeMaxWarps * bytes;
}
constexpr int kRopeSmemBytes = 8 * kRopeTable + 4 * (4 * kRopeTable + 2 * kRopeMaxWarps * 2 * kRopeTable);

// A token's position on axis `lane` (lanes past the axes: the last one).
__device__ __forceinline__ int64_t lane_position(const RopeParams &p, int lane, int64_t token) {
    const int64_t at = (int64_t)(lane < p.axes ? lane : p.axes - 1) * p.pos_stride + token;
    return p.pos64 ? static_cast<const int64_t *>(p.pos)[at] : (int64_t)static_cast<const int32_t *>(p.pos)[at];
}

// A token's tables of cosines and sines by one warp, pair i
// by lane i % 32, from the position that lane a holds for axis a.
template <int VE, bool IL>
__device__ __forceinline__ void make_angles(const RopeParams &p, const uint64_t *frac, float *cs, int lane, int64_t pos) {
    for (int i = lane; i - lane < p.R; i += 32) {
        int64_t at = pos;
        if (p.axes > 1) at = __shfl_sync(0xffffffffu, pos, axis_of(p, i));
        if (i < p.R) {
            float s, c;
            sincos_turns((uint64_t)at * frac[i], s, c);
            cs[factor_at<VE, IL>(i, 0)] = c;
            cs[factor_at<VE, IL>(i, 1)] = s;
        }
    }
}

// The turn fractions, and both kinds' head weights (w + bias; 1 without a
// weight), by the whole block.
template <int VE>
__device__ __forceinline__ void make_fractions(const RopeParams &p, uint64_t *frac) {
    for (int i = threadIdx.x; i < p.R; i += blockDim.x) frac[i] = turn_fraction(p.inv_freq[i]);
}

template <typename T, int VE, bool IL>
__device__ __forceinline__ void make_weights(const RopeParams &p, float *wsm) {
    const int D = p.head_dim;
    for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {
        const int kind = i >= D, e = i - kind * D;
        const void *w = kind ? p.k_w : p.q_w;
        // element e: which pair, and whether it is its second element
        int pair, second;
        // (the pairs past the rotated part start with a unit of their own)
        const int tail = p.rot_units * VE;
        if (IL) {
            pair = e >> 1;
            pair = pair < p.R ? pair : tail + pair - p.R;
            second = e & 1;
        } else if (e < 2 * p.R) {
            second = e >= p.R;
            pair = e - second * p.R;
        } else {
            const int half = D / 2 - p.R;
            second = e - 2 * p.R >= half;
            pair = tail + (e - 2 * p.R - second * half);
        }
        float v = 1.f;
        if (w != nullptr) v = widen_bits(ld_bits(w, e, T{}, 2), T{}) + p.w_bias;
        wsm[kind * 2 * kRopeTable + factor_at<VE, IL>(pair, second)] = v;
    }
}

// ------------------------------------------------------------ paged cache

// The sequence of a token: the last s with cu_tokens[s] <= token, by halving
// (a batch of single tokens, where token t is sequence t's, is seen at once).
// Whatever cu_tokens holds, the answer is in [0, seqs).
__device__ __forceinline__ int sequence_of(const RopeParams &p, int64_t token) {
    if (token < p.seqs && p.cu_tokens[token] <= token && token < p.cu_tokens[token + 1]) return (int)token;
    int lo = 0, hi = p.seqs;
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (p.cu_tokens[mid] <= token) lo = mid;
        else hi = mid;
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

// E4m3: scales whose inverses are exact (powers of two); Settled: any.  A kernel
// of its own costs the others nothing: 8192 tokens of 32 + 2 * 8 bf16 heads of
// 128 35.5 us with exact inverses, 37.5 settled, 36.3 and 37.5 from one kernel.
// (The kernels of rope_ragged.cuh look at `settle`.)
enum RopeMode { kRopePlain = 0, kRopeAppend = 1, kRopeAppendE4m3 = 2, kRopeAppendSettled = 3 };
__host__ __device__ constexpr bool rope_codes(int mode) { return mode >= kRopeAppendE4m3; }

// A lane's units of a head: where their pieces start (bytes), and which exist.
// Lanes without a unit take unit 0's place (they load it like a neighbour: no
// branch, no zeroing) and have no part in sums and stores.
// HD: a head size known at compile time (whole heads turned, a power of two
// of lanes a head, K = 1): every lane has a unit, the pieces a fixed distance.
template <int VE, int K, bool IL, int S, int HD>
struct Lane {
    int oa[K], ob[K], unit[K];
    bool act[K], rot[K];
    __device__ __forceinline__ void set(const RopeParams &p, int t, int group) {
        if constexpr (HD > 0) {
            unit[0] = t;
            act[0] = rot[0] = true;
            oa[0] = (IL ? 2 * t * VE : t * VE) * S;
            ob[0] = oa[0] + (IL ? VE : HD / 2) * S;
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                act[k] = t + k * p.lanes < p.units && group < p.heads_a_warp;
                unit[k] = act[k] ? t + k * p.lanes : 0;
                rot[k] = unit[k] < p.rot_units;
                unit_offsets<VE, IL>(p, unit[k], oa[k], ob[k]);
                oa[k] *= S;
                ob[k] *= S;
            }
        }
    }
};

// A block's run of jobs (a token's slice of head iterations; equal runs, one
// more for the first `extra` blocks).
struct Jobs {
    int64_t first, last;
    __device__ __forceinline__ void set(int64_t block, int64_t each, int64_t extra) {
        first = block * each + (block < extra ? block : extra);
        last = first + each + (block < extra ? 1 : 0);
    }
};

template <typename T, int VE>
__device__ __forceinline__ void widen_unit(const typename Piece<T, VE>::Raw &a, const typename Piece<T, VE>::Raw &b,
                                           float (&e)[2 * VE]) {
    float x[VE], y[VE];
    Piece<T, VE>::widen(a, x);
    Piece<T, VE>::widen(b, y);
#pragma unroll
    for (int j = 0; j < VE; ++j) {
        e[j] = x[j];
        e[VE + j] = y[j];
    }
}

// Sums over the g lanes of a head, of M values, for all of them.  t: the
// lane's place in its head.
template <int M>
__device__ __forceinline__ void lanes_sum(float (&v)[M], int g, int t, int lane) {
    auto add = [&](int off) {
#pragma unroll
        for (int i = 0; i < M; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    };
    if ((g & (g - 1)) == 0) {
        if (g >= 8) {   // the usual head sizes: one or two branches
            add(1);
            add(2);
            add(4);
            if (g > 8) {
                add(8);
                if (g > 16) add(16);
            }
        } else if (g > 1) {
            add(1);
            if (g > 2) add(2);
        }
    } else {   // heads of 40, 80, 96 ...: towards the head's first lane and back
        for (int off = 1; off < g; off <<= 1) {
#pragma unroll
            for (int i = 0; i < M; ++i) {
                const float o = __shfl_down_sync(0xffffffffu, v[i], off);
                v[i] += t + off < g ? o : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < M; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], lane - t);
    }
}

// A block's place in its run: tiles of p.tile jobs (one where a token's heads
// are cut in slices, or where token rows lie so far apart that a tile's would
// not be reached with 32 bits), and the warp's head iterations of a tile.
struct Tile {
    int j, i;   // job of the tile, head iteration of the job
    __device__ __forceinline__ void settle(int jobs, int iters) {
        while (i >= iters && j < jobs) {
            i -= iters;
            ++j;
        }
    }
};

// ----------------------------------------------------------------- forward
template <typename T, int VE, int K, bool IL, int MODE, int HD>
__global__ void __launch_bounds__(32 * kRopeMaxWarps, rope_resident(Piece<T, VE>::kBytes, K)) rope_kernel(const RopeParams p) {
    using P = Piece<T, VE>;
    using Raw = typename P::Raw;
    constexpr int S = (int)sizeof(typename T::storage);
    constexpr int N = pairs_at_once(VE);
    constexpr bool APPEND = MODE != kRopePlain;
    extern __shared__ __align__(16) unsigned char smem[];
    // append: where the tokens of kLookUps jobs go (-1: nowhere), and their
    // indices in their sequences, looked up a thread each
    constexpr int kLookUps = 8 * kRopeMaxWarps;
    __shared__ int64_t rows[APPEND ? kLookUps : 1], indices[APPEND ? kLookUps : 1];
    uint64_t *frac = reinterpret_cast<uint64_t *>(smem);
    float *wsm = reinterpret_cast<float *>(smem + 8 * kRopeTable);
    float *tiles = wsm + 4 * kRopeTable;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = HD ? HD / 2 / VE : p.lanes, group = lane / G, t = lane - group * G;
    const int hpw = HD ? 32 / G : p.heads_a_warp;
    const int heads = p.q_heads + p.k_heads + p.v_heads, turned = p.q_heads + p.k_heads;
    const uint32_t head_bytes = (uint32_t)((HD ? HD : p.head_dim) * S);
    Lane<VE, K, IL, S, HD> my;
    my.set(p, t, group);
    Jobs jobs;
    jobs.set(blockIdx.x, p.each, p.extra);

    pdl_wait_for_inputs();
    pdl_allow_dependents();
    if constexpr (APPEND) {   // rows behind the last sequence are left as they are
        const int64_t valid = p.cu_tokens[p.seqs];
        const int64_t most = (valid < 0 ? 0 : valid) * p.slices;
        if (jobs.last > most) jobs.last = most;
    }

    int64_t known = jobs.first;   // first of the jobs looked up
    auto look_up = [&]() {
        const int64_t job = known + threadIdx.x;
        if (threadIdx.x < kLookUps && job < jobs.last) {
            const int64_t token = p.slices > 1 ? job / p.slices : job;
            const int seq = sequence_of(p, token);
            const int64_t index = (int64_t)p.cache_lens[seq] + (token - p.cu_tokens[seq]);
            indices[threadIdx.x] = index;
            rows[threadIdx.x] = cache_row(p, seq, index);
        }
    };

    bool prepared = false;
    int buf = 0;
    for (int64_t base = jobs.first; base < jobs.last; base += p.tile, buf ^= 1) {
        const int n = jobs.last - base < p.tile ? (int)(jobs.last - base) : p.tile;
        const int64_t token0 = p.slices > 1 ? base / p.slices : base;
        const int h0 = p.slices > 1 ? (int)(base - token0 * p.slices) * p.iters * hpw + group : group;
        const char *tx = static_cast<const char *>(p.x) + token0 * p.x_stride;
        char *ty = static_cast<char *>(p.y) + token0 * p.y_stride;
        Tile at{0, warp};
        at.settle(n, p.iters);
        Raw ra[K], rb[K];
        auto load = [&]() {
            int h = h0 + at.i * hpw;
            h = h < heads ? h : heads - 1;
            const uint32_t off = (uint32_t)at.j * (uint32_t)p.x_stride + (uint32_t)h * head_bytes;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const char *src = tx + (off + my.oa[k]);
                ra[k] = P::load(src);
                rb[k] = P::load(src + (HD ? (IL ? VE : HD / 2) * S : my.ob[k] - my.oa[k]));
            }
        };
        if (at.j < n) load();
        if (APPEND && base - known >= kLookUps) {
            __syncthreads();   // what was looked up before is read
            known = base;
            look_up();
            __syncthreads();
        }
        if (!prepared) {
            if constexpr (APPEND) look_up();
            make_fractions<VE>(p, frac);
            make_weights<T, VE, IL>(p, wsm);
            __syncthreads();
            prepared = true;
        }
        if (warp < n) {   // the warp's own token of the tile
            int64_t pos = 0;
            if (!APPEND || p.pos != nullptr) pos = lane_position(p, lane, token0 + warp);
            else pos = indices[base - known + warp];
            make_angles<VE, IL>(p, frac, tiles + (buf * kRopeMaxWarps + warp) * 2 * kRopeTable, lane, pos);
        }
        __syncthreads();   // two buffers: the tile before this one may still be read
        while (at.j < n) {
            Raw ca[K], cb[K];
#pragma unroll
            for (int k = 0; k < K; ++k) ca[k] = ra[k], cb[k] = rb[k];
            const int job = at.j, h = h0 + at.i * hpw;
            at.i += kRopeMaxWarps;
            at.settle(n, p.iters);
            if (at.j < n) load();   // the next heads are on their way
            float r = 1.f;
            if (p.norm) {
                float sum[1] = {0.f};
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    float e[2 * VE];
                    widen_unit<T, VE>(ca[k], cb[k], e);
                    float2 acc = make_float2(0.f, 0.f);
                    run_dot<2 * VE>(acc, e, e);
                    sum[0] += my.act[k] ? acc.x + acc.y : 0.f;
                }
                lanes_sum<1>(sum, G, t, lane);
                r = rsqrtf(fmaf(sum[0], p.inv_dim, p.eps));
            }
            const bool key = h >= p.q_heads, value = APPEND && h >= turned;
            const float *cs = tiles + (buf * kRopeMaxWarps + job) * 2 * kRopeTable;
            const float *w = wsm + (key ? 2 * kRopeTable : 0);
            char *dst = ty + ((uint32_t)job * (uint32_t)p.y_stride + (uint32_t)h * head_bytes);
            bool store = h < heads;
            if (APPEND && key) {
                const int64_t row = rows[base - known + job];
                const int o = value ? h - turned : h - p.q_heads;
                dst = static_cast<char *>(value ? p.v_cache : p.k_cache) + row + (int64_t)o * p.head_stride;
                store = store && row >= 0;
                if (row < 0 && h == p.q_heads && t == 0 && my.act[0] && p.dropped != nullptr) atomicAdd(p.dropped, 1);
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float e[2 * VE];
                widen_unit<T, VE>(ca[k], cb[k], e);
                if (!value) {
                    const float *wu = w + table_at<VE>(my.unit[k], 0), *cu = cs + table_at<VE>(my.unit[k], 0);
                    const bool rot = my.rot[k];
                    if (p.norm) run_scale<2 * VE>(e, r);
#pragma unroll
                    for (int q = 0; q < VE; q += N) {
                        float *a = e + run_a<VE, IL>(q), *b = e + run_b<VE, IL>(q), f[N], g[N];
                        read_table<N>(wu + table_at<VE>(0, q), f);
                        read_table<N>(wu + kRopeTable + table_at<VE>(0, q), g);
                        run_times<N>(a, f);
                        run_times<N>(b, g);
                    }
                    if (rot) {
#pragma unroll
                        for (int q = 0; q < VE; q += N) {
                            float *a = e + run_a<VE, IL>(q), *b = e + run_b<VE, IL>(q), f[N], g[N];
                            read_table<N>(cu + table_at<VE>(0, q), f);
                            read_table<N>(cu + kRopeTable + table_at<VE>(0, q), g);
                            turn_runs<IL, false, N>(a, b, f, g);
                        }
                    }
                }
                if (store && my.act[k]) {
                    float x[VE], y[VE];
#pragma unroll
                    for (int v = 0; v < VE; ++v) x[v] = e[v], y[v] = e[VE + v];
                    const int d = HD ? (IL ? VE : HD / 2) * S : my.ob[k] - my.oa[k];
                    if (rope_codes(MODE) && key) {
                        const float inv = value ? p.v_inv : p.k_inv, scale = value ? p.v_scale : p.k_scale;
                        char *to = dst + my.oa[k] / S;
                        P::template store_e4m3<MODE == kRopeAppendSettled>(to, x, inv, scale);
                        P::template store_e4m3<MODE == kRopeAppendSettled>(to + d / S, y, inv, scale);
                    } else {
                        char *to = dst + my.oa[k];
                        P::store(to, x);
                        P::store(to + d, y);
                    }
                }
            }
        }
    }
}

// ---------------------------------------------------------------- gradient
// A block's first q_warps warps take its tokens' query heads, the rest the
// key heads (so a thread keeps one kind's share of the weight's gradient in
// registers and both kinds share the tokens' angles: with blocks of one kind
// each token's were made twice, 62.5 against 49.5 us for bf16 8192 tokens x 40
// heads of 128).  The block's sums go to partial[kind][block][D], and the
// blocks' are added up by another kernel.  The order of every sum follows from
// the sizes and the grid: no atomics.
// x is read only with the norm; without it dx = dy turned back.
template <typename T, int VE, int K, bool IL, bool NORM, int HD>
__global__ void __maxnreg__(rope_bwd_registers(Piece<T, VE>::kBytes, K)) rope_bwd_kernel(const RopeParams p) {
    using P = Piece<T, VE>;
    using Raw = typename P::Raw;
    constexpr int S = (int)sizeof(typename T::storage);
    constexpr int N = pairs_at_once(VE);
    constexpr int KN = NORM ? K : 1;
    constexpr bool ASYNC = P::kBytes >= 4;
    extern __shared__ __align__(16) unsigned char smem[];
    uint64_t *frac = reinterpret_cast<uint64_t *>(smem);
    float *wsm = reinterpret_cast<float *>(smem + 8 * kRopeTable);
    float *tiles = wsm + 4 * kRopeTable;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = HD ? HD / 2 / VE : p.lanes, group = lane / G, t = lane - group * G;
    const int hpw = HD ? 32 / G : p.heads_a_warp;
    const uint32_t head_bytes = (uint32_t)((HD ? HD : p.head_dim) * S);
    Lane<VE, K, IL, S, HD> my;
    my.set(p, t, group);
    const bool key = warp >= p.q_warps;
    const int heads = key ? p.k_heads : p.q_heads, iters = key ? p.iters_k : p.iters;
    const int mates = key ? kRopeMaxWarps - p.q_warps : p.q_warps;   // warps of the kind
    Jobs jobs;
    jobs.set(blockIdx.x, p.each, p.extra);
    const uint32_t head0 = key ? (uint32_t)p.q_heads * head_bytes : 0u;
    const float *w = wsm + (key ? 2 * kRopeTable : 0);
    // With few tokens a block has one slice of one token's heads: the token is
    // job - skip, the slice's first iteration i0.
    int64_t skip = 0;
    int i0 = 0;
    if (p.slices > 1) {
        const uint32_t token = (uint32_t)jobs.first / (uint32_t)p.slices;
        i0 = (int)((uint32_t)jobs.first - token * (uint32_t)p.slices) * iters;
        skip = jobs.first - token;
    }
    // The block's first token row into L2 before the wait (bf16 8192 tokens x
    // 40 heads of 128 44.6 -> 44.0 us; more rows, or rows in the forward, did
    // not pay).
    if (P::kBytes == 16 && threadIdx.x == 0 && jobs.first < jobs.last) {
        const uint32_t bytes = (uint32_t)(p.q_heads + p.k_heads) * head_bytes;
        prefetch_l2(static_cast<const char *>(p.dy) + (jobs.first - skip) * p.dy_stride, bytes);
        if constexpr (NORM) prefetch_l2(static_cast<const char *>(p.x) + (jobs.first - skip) * p.x_stride, bytes);
    }

    pdl_wait_for_inputs();
    pdl_allow_dependents();

    float gw[KN][2 * VE];   // the weight's gradient
#pragma unroll
    for (int k = 0; k < KN; ++k)
#pragma unroll
        for (int v = 0; v < 2 * VE; ++v) gw[k][v] = 0.f;

    int64_t pos = 0;   // of the warp's token of a tile: axis a's in lane a
    // A thread's own places of the ring [stage][dy a, dy b, x a, x b][K], where
    // pieces are wide enough to be copied asynchronously.
    Raw da[K], db[K], xa[KN], xb[KN];
    int stage = 0;
    auto place = [&](int piece, int k) {
        return reinterpret_cast<char *>(tiles + 2 * kRopeMaxWarps * 2 * kRopeTable) +
               ((((stage * (NORM ? 4 : 2) + piece) * K + k) * 32 * kRopeMaxWarps) + (int)threadIdx.x) * P::kBytes;
    };

    bool prepared = false;
    int buf = 0;
    for (int64_t base = jobs.first; base < jobs.last; base += p.tile, buf ^= 1) {
        const int n = jobs.last - base < p.tile ? (int)(jobs.last - base) : p.tile;
        const int64_t token0 = base - skip;
        const char *tg = static_cast<const char *>(p.dy) + token0 * p.dy_stride + head0;
        const char *tx = static_cast<const char *>(p.x) + token0 * p.x_stride + head0;
        char *ty = static_cast<char *>(p.y) + token0 * p.y_stride + head0;
        Tile at{0, key ? warp - p.q_warps : warp};
        at.settle(n, iters);
        auto load = [&]() {
            int h = (i0 + at.i) * hpw + group;
            h = h < heads ? h : heads - 1;
            const uint32_t go = (uint32_t)at.j * (uint32_t)p.dy_stride + (uint32_t)h * head_bytes;
            const uint32_t xo = (uint32_t)at.j * (uint32_t)p.x_stride + (uint32_t)h * head_bytes;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if constexpr (ASYNC) {
                    const int d = HD ? (IL ? VE : HD / 2) * S : my.ob[k] - my.oa[k];
                    const char *ga = tg + (go + my.oa[k]), *at_x = tx + (xo + my.oa[k]);
                    P::template copy<IL>(place(0, k), ga);
                    P::template copy<IL>(place(1, k), ga + d);
                    if constexpr (NORM) {
                        P::template copy<IL>(place(2, k), at_x);
                        P::template copy<IL>(place(3, k), at_x + d);
                    }
                } else {
                    da[k] = P::load(tg + (go + my.oa[k]));
                    db[k] = P::load(tg + (go + my.ob[k]));
                    if constexpr (NORM) {
                        xa[k] = P::load(tx + (xo + my.oa[k]));
                        xb[k] = P::load(tx + (xo + my.ob[k]));
                    }
                }
            }
        };
        if (at.j < n) load();
        if constexpr (ASYNC) copy_async_commit();
        if (!prepared) {
            if (base + warp < jobs.last) pos = lane_position(p, lane, token0 + warp);
            make_fractions<VE>(p, frac);
            if constexpr (NORM) make_weights<T, VE, IL>(p, wsm);
            __syncthreads();
            prepared = true;
        }
        if (warp < n)
            make_angles<VE, IL>(p, frac, tiles + (buf * kRopeMaxWarps + warp) * 2 * kRopeTable, lane, pos);
        if (base + p.tile + warp < jobs.last) pos = lane_position(p, lane, token0 + p.tile + warp);   // the next tile's
        __syncthreads();   // two buffers: the tile before this one may still be read
        while (at.j < n) {
            Raw ea[K], eb[K], ya[KN], yb[KN];
            if constexpr (!ASYNC) {
#pragma unroll
                for (int k = 0; k < K; ++k) ea[k] = da[k], eb[k] = db[k];
#pragma unroll
                for (int k = 0; k < KN; ++k) ya[k] = xa[k], yb[k] = xb[k];
            }
            const int job = at.j, h = (i0 + at.i) * hpw + group;
            at.i += mates;
            at.settle(n, iters);
            stage ^= 1;
            if (at.j < n) load();   // the next heads are on their way
            if constexpr (ASYNC) {
                copy_async_commit();
                copy_async_wait<1>();   // these heads are there
                stage ^= 1;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    ea[k] = P::take(place(0, k));
                    eb[k] = P::take(place(1, k));
                    if constexpr (NORM) {
                        ya[k] = P::take(place(2, k));
                        yb[k] = P::take(place(3, k));
                    }
                }
                stage ^= 1;
            }
            const float *cs = tiles + (buf * kRopeMaxWarps + job) * 2 * kRopeTable;

            float g[K][2 * VE], x[KN][2 * VE];
            float sums[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < K; ++k) {
                widen_unit<T, VE>(ea[k], eb[k], g[k]);
                const float *wu = w + table_at<VE>(my.unit[k], 0), *cu = cs + table_at<VE>(my.unit[k], 0);
                if (my.rot[k]) {
#pragma unroll
                    for (int q = 0; q < VE; q += N) {
                        float f[N], h2[N];
                        read_table<N>(cu + table_at<VE>(0, q), f);
                        read_table<N>(cu + kRopeTable + table_at<VE>(0, q), h2);
                        turn_runs<IL, true, N>(g[k] + run_a<VE, IL>(q), g[k] + run_b<VE, IL>(q), f, h2);
                    }
                }
                if constexpr (NORM) {
                    widen_unit<T, VE>(ya[k], yb[k], x[k]);
                    float2 sq = make_float2(0.f, 0.f), dot = sq;
                    run_dot<2 * VE>(sq, x[k], x[k]);
#pragma unroll
                    for (int q = 0; q < VE; q += N) {
                        const int a = run_a<VE, IL>(q), b = run_b<VE, IL>(q);
                        float f[N], h2[N];
                        read_table<N>(wu + table_at<VE>(0, q), f);
                        read_table<N>(wu + kRopeTable + table_at<VE>(0, q), h2);
                        run_times<N>(f, reinterpret_cast<const float(&)[N]>(g[k][a]));
                        run_times<N>(h2, reinterpret_cast<const float(&)[N]>(g[k][b]));
                        run_dot<N>(dot, f, x[k] + a);
                        run_dot<N>(dot, h2, x[k] + b);
                    }
                    sums[0] += my.act[k] ? sq.x + sq.y : 0.f;
                    sums[1] += my.act[k] ? dot.x + dot.y : 0.f;
                }
            }
            if constexpr (NORM) {
                lanes_sum<2>(sums, G, t, lane);
                const float r = rsqrtf(fmaf(sums[0], p.inv_dim, p.eps));
                const float mean = -(sums[1] * p.inv_dim) * r;   // dx = r (w g - (x r) mean)
                float mm[2 * VE];
#pragma unroll
                for (int v = 0; v < 2 * VE; ++v) mm[v] = mean;
#pragma unroll
                for (int k = 0; k < K; ++k) run_scale<2 * VE>(x[k], r);
                if (h < heads) {   // an idle head's copy adds nothing
#pragma unroll
                    for (int k = 0; k < K; ++k) run_fma<2 * VE>(gw[k], g[k], x[k]);
                }
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const float *wu = w + table_at<VE>(my.unit[k], 0);
#pragma unroll
                    for (int q = 0; q < VE; q += N) {
                        float f[N], h2[N];
                        read_table<N>(wu + table_at<VE>(0, q), f);
                        read_table<N>(wu + kRopeTable + table_at<VE>(0, q), h2);
                        run_times<N>(g[k] + run_a<VE, IL>(q), f);
                        run_times<N>(g[k] + run_b<VE, IL>(q), h2);
                    }
                    run_fma<2 * VE>(g[k], x[k], mm);
                    run_scale<2 * VE>(g[k], r);
                }
            }
            char *dst = ty + ((uint32_t)job * (uint32_t)p.y_stride + (uint32_t)h * head_bytes);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (h < heads && my.act[k]) {
                    float u[VE], v[VE];
#pragma unroll
                    for (int e = 0; e < VE; ++e) u[e] = g[k][e], v[e] = g[k][VE + e];
                    char *to = dst + my.oa[k];
                    P::store(to, u);
                    P::store(to + (HD ? (IL ? VE : HD / 2) * S : my.ob[k] - my.oa[k]), v);
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
                for (int v = 0; v < 2 * VE; ++v) {
                    const float own = gw[k][v];
                    for (int g = 1; g < hpw; ++g) gw[k][v] += __shfl_sync(0xffffffffu, own, (lane + g * G) & 31);
                }
            __syncthreads();   // the tables are read; their place takes the warps' sums [kRopeMaxWarps][D]
            if (group == 0) {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (my.act[k] && heads > 0)
#pragma unroll
                        for (int v = 0; v < VE; ++v) {
                            wsm[warp * p.head_dim + my.oa[k] / S + v] = gw[k][v];
                            wsm[warp * p.head_dim + my.ob[k] / S + v] = gw[k][VE + v];
                        }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < 2 * p.head_dim; i += blockDim.x) {
                const int kind = i >= p.head_dim, d = i - kind * p.head_dim;
                float v = 0.f;
                for (int k = kind ? p.q_warps : 0; k < (kind ? kRopeMaxWarps : p.q_warps); ++k)
                    v += wsm[k * p.head_dim + d];
                p.partial[((int64_t)kind * gridDim.x + blockIdx.x) * p.partial_ld + d] = v;
            }
            if (p.dq_w != nullptr) {   // few blocks: one cluster
                behind_the_cluster();
                const int mine = (int)(blockIdx.x * blockDim.x + threadIdx.x), all = (int)(gridDim.x * blockDim.x);
                finish_columns<T>(p.partial, (int)gridDim.x, p.partial_ld, p.head_dim, p.dq_w, mine, all);
                finish_columns<T>(p.partial + (int64_t)gridDim.x * p.partial_ld, (int)gridDim.x, p.partial_ld, p.head_dim,
                                  p.dk_w, mine, all);
            }
        }
    }
}

}  // namespace rrn
