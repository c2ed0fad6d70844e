// logprobs_kernels.cuh -- log probabilities of given tokens, entropy and the
// likeliest alternatives of rows of logits, and their gradient.
//
// Forward, one pass: with m the largest logit and z = (x - m) / temperature,
// the sums of exp(z) and z exp(z).  A row is cut into units of 32 lanes x 8
// chunks of 16 bytes (2048 bf16 or 1024 fp32 logits); a warp holds a unit in
// registers, takes its maximum, and sums relative to that, so nothing is ever
// rescaled within a unit.  The units' (maximum, sums) meet in shared memory
// (distributed shared memory where a cluster of blocks shares a row) and are
// added up in one order.  The order follows from the row's length alone,
// however the units are dealt out, so a row has the same bits in every batch.
//
// Alternatives: each thread knows the largest logit it saw.  The k-th largest
// of the maxima of 32 groups of threads is a bound that at least k logits
// reach, so only threads whose maximum reaches it can hold one of the k
// largest; their few chunks are read again (from L2), one a thread, and what
// reaches the bound, a key of value and place, is gathered in shared memory.
// Where that is too much (equal logits, masks, a heap of large ones in one
// place), what was gathered gives a higher bound in the same way, in as many
// rounds as key_search.h allows.  The few that
// are left find their places by counting the larger ones.
//
// Gradient: elementwise, given the forward's statistics.  One read and one
// write of every element; HBM bandwidth bounds both.
//
// bf16 8192 x 131072, 2.1 GB a tensor: forward 294 us (7.3 TB/s), gradient 618
// (6.9); fp32 1001 x 50257 with 5 alternatives: 39.7 (5.1) in rows of 50304, the
// alternatives' look-up and the waves' end bound it, and 45.0 (4.5) in rows that
// begin between the 16-byte boundaries; 8 rows of 131072 with 20 alternatives: 6.9,
// latency.  bf16 8192 x 50257 between the boundaries 166, in rows of 50264 122:
// 1.6 times the instructions an element.
#pragma once

#include "key_search.h"
#include "rmsnorm_cluster.cuh"

namespace rrn {

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32, kLpChunks = 8;
constexpr int kLpTop = 32;   // alternatives at most
constexpr int kLpAhead = 32 * 1024;   // bytes of a row that are asked for ahead
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <typename T>
__host__ __device__ constexpr int lp_unit() {
    return 32 * kLpChunks * T::kVec;
}

struct LogprobParams {
    const char *logits;
    const void *tokens;
    float *logprobs, *stats, *entropy, *top_logprobs;
    int32_t *top_ids;
    int64_t rows, stride;   // bytes
    int32_t vocab, units, top;
    int32_t wide;        // 64-bit tokens
    int32_t warps;       // of a row: 1, 2, 4, 8 (of every block of a cluster)
    int64_t ahead;       // rows that the device holds at once
    float inv_t, c;      // 1 / temperature, and times log2(e)
};

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// The largest of the warp's values (a NaN is passed over).
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Elements i .. i + V - 1 of a row as a chunk, each by itself; -infinity outside
// the row (i may be negative).  Shifted in, for few registers: it is for the
// first and the last chunk of a tensor.
template <typename T>
__device__ __forceinline__ Chunk edge_chunk(const char *row, int i, int vocab) {
    Chunk c = {};
#pragma unroll 4
    for (int k = T::kVec - 1; k >= 0; --k) {
        const bool in = (uint32_t)(i + k) < (uint32_t)vocab;
        if constexpr (T::kVec == 8) {
            const uint32_t v = in ? reinterpret_cast<const uint16_t *>(row)[i + k] : 0xff80u;
            c.u[3] = __funnelshift_l(c.u[2], c.u[3], 16);
            c.u[2] = __funnelshift_l(c.u[1], c.u[2], 16);
            c.u[1] = __funnelshift_l(c.u[0], c.u[1], 16);
            c.u[0] = c.u[0] << 16 | v;
        } else {
            c.u[3] = c.u[2];
            c.u[2] = c.u[1];
            c.u[1] = c.u[0];
            c.u[0] = in ? reinterpret_cast<const uint32_t *>(row)[i + k] : 0xff800000u;
        }
    }
    return c;
}

template <typename T>
__device__ __forceinline__ Chunk minus_infinity() {
    const uint32_t v = T::kVec == 8 ? 0xff80ff80u : 0xff800000u;
    return Chunk{{v, v, v, v}};
}

// -infinity in the places of a chunk, which starts at element i, outside the row.
template <typename T>
__device__ __forceinline__ void mask_chunk(Chunk &c, int i, int vocab) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (T::kVec == 8) {
            if ((uint32_t)(i + 2 * k) >= (uint32_t)vocab) c.u[k] = (c.u[k] & 0xffff0000u) | 0xff80u;
            if ((uint32_t)(i + 2 * k + 1) >= (uint32_t)vocab) c.u[k] = (c.u[k] & 0xffffu) | 0xff800000u;
        } else {
            if ((uint32_t)(i + k) >= (uint32_t)vocab) c.u[k] = 0xff800000u;
        }
    }
}

// Whether 32 bytes before a row's first byte, and behind its last, are the
// tensor's too: chunks that begin or end outside the row may be read whole then.
struct Around {
    bool before, behind;
};
__device__ __forceinline__ Around around(const char *tensor, const char *row, int64_t rows, int64_t stride) {
    return Around{row - tensor >= 32, tensor + (rows - 1) * stride - row >= 32};
}

// A 16-byte load that other lanes read from L1 too.
__device__ __forceinline__ uint4 ld_shared16(const char *p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// 16 bytes that start `off` bytes into a and go on into b.
template <typename T>
__device__ __forceinline__ Chunk across(const uint4 &a, const uint4 &b, int off) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = off & 8 ? w[k + 2] : w[k];
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = off & 4 ? w[k + 1] : w[k];
    Chunk c;
#pragma unroll
    for (int k = 0; k < 4; ++k) c.u[k] = T::kVec == 8 && (off & 2) ? __funnelshift_r(w[k], w[k + 1], 16) : w[k];
    return c;
}

// N chunks of a row `step` elements apart, from element i on; -infinity outside
// the row, and no byte outside the tensor is read.  ALIGNED: they start on
// 16-byte boundaries, else `off` bytes past them: then each lies in two of
// memory's own chunks, the second of which is a neighbouring lane's first and
// comes from L1.
template <typename T, bool ALIGNED, int N>
__device__ __forceinline__ void load_chunks(Chunk (&c)[N], const char *row, int i, int step, int vocab, int off,
                                            Around there) {
    constexpr int V = T::kVec, E = 16 / V;
    // places of chunks that may be read whole, both of memory's where there are two
    const bool two = !ALIGNED && off != 0;
    const int least = there.before ? 1 - V : two ? off / E : 0;
    const int most = there.behind ? vocab - 1 : two ? vocab - 2 * V + off / E : vocab - V;
    if (two) {
        uint4 a[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int at = i + j * step;
            if (at >= least && at <= most) a[j] = ld_shared16(row + (int64_t)at * E - off);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int at = i + j * step;
            if (at >= least && at <= most) c[j] = across<T>(a[j], ld_shared16(row + (int64_t)at * E - off + 16), off);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int at = i + j * step;
            if (at >= least && at <= most) c[j] = ld_keep_l2_16(row + (int64_t)at * E);
        }
    }
    const int last = i + (N - 1) * step;
    if (i >= 0 && i >= least && last <= most && last + V <= vocab) return;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int at = i + j * step;
        if (at < least || at > most) c[j] = edge_chunk<T>(row, at, vocab);
        else if (at < 0 || at + V > vocab) mask_chunk<T>(c[j], at, vocab);
    }
}

// A warp's unit of a row, lane l's chunk j being the unit's chunk 32 j + l;
// -infinity behind the row's end.  Units well within the row are plain loads.  In
// the others addresses are held within the tensor, what lies behind the row is
// masked, and the chunks at the tensor's two ends are put together by themselves.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void load_unit(Chunk (&c)[kLpChunks], const char *row, int unit, int lane, int vocab,
                                          int off, Around there) {
    constexpr int V = T::kVec, E = 16 / V, N = kLpChunks, STEP = 32 * 16;   // bytes between a lane's chunks
    const bool two = !ALIGNED && off != 0;
    const int first = unit * lp_unit<T>(), end = first + lp_unit<T>();
    const char *from = row + (int64_t)first * E + lane * 16;
    const bool inside = end <= vocab && (!two || ((first > 0 || there.before) &&
                                                  (there.behind || end * E + 16 - off <= vocab * E)));
    if (inside) {
        if (two) {
            // the second of memory's chunks is the next lane's first, or the first
            // lane's next
            Chunk a[N], last = {};
#pragma unroll
            for (int j = 0; j < N; ++j) a[j] = ld_keep_l2_16(from - off + j * STEP);
            if (lane == 31) last = ld_keep_l2_16(from - off + 16 + (N - 1) * STEP);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                Chunk b;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t give = j + 1 < N && lane == 0 ? a[j + 1 < N ? j + 1 : j].u[k] : a[j].u[k];
                    b.u[k] = __shfl_sync(0xffffffffu, give, (lane + 1) & 31);
                    if (j == N - 1 && lane == 31) b.u[k] = last.u[k];
                }
                c[j] = across<T>(make_uint4(a[j].u[0], a[j].u[1], a[j].u[2], a[j].u[3]),
                                 make_uint4(b.u[0], b.u[1], b.u[2], b.u[3]), off);
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) c[j] = ld_keep_l2_16(from + j * STEP);
        }
        return;
    }
    // bytes from the row's start at which memory's chunks lie whole in the tensor
    const int low = two ? there.before ? -off : 16 - off : 0;
    const int bytes = vocab * E;
    const int high = ((bytes + off) / 16 - (there.behind ? 0 : 1)) * 16 - off;
    const bool any = high >= low;
    const int at = first * E + lane * 16;
    const int used = (vocab - first + 32 * V - 1) / (32 * V);   // chunks that some lane has in the row
#pragma unroll
    for (int j = 0; j < N; ++j) {
        c[j] = minus_infinity<T>();
        if (j >= used) continue;
        const int a = max(low, min(at + j * STEP - off, high)), b = max(low, min(at + j * STEP - off + 16, high));
        if (!any) continue;
        if (two) c[j] = across<T>(ld_shared16(row + a), ld_shared16(row + b), off);
        else c[j] = ld_keep_l2_16(row + a);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int i = first + j * 32 * V + lane * V;
        if (j < used && i + V > vocab) mask_chunk<T>(c[j], i, vocab);
    }
    if ((there.before || !two) && (there.behind || (!two && vocab % V == 0))) return;
    // the first, the last but one, the last
#pragma unroll 1
    for (int k = there.before || !two ? 2 - two : 0; k < (there.behind ? 1 : 3); ++k) {
        const int i = k == 0 ? 0 : ((vocab - 1) / V - (2 - k)) * V;
        const int mine = i - first - lane * V;
        if (i < 0 || mine < 0 || mine % (32 * V) != 0) continue;
        const Chunk e = edge_chunk<T>(row, i, vocab);
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (mine == j * 32 * V) c[j] = e;
    }
    __syncwarp();
}

// The largest element of the chunks (a NaN is passed over).
template <int N>
__device__ __forceinline__ float chunks_max(const Chunk (&c)[N], BF16) {
    __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162 *>(&c[0].u[0]);
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162 *>(&c[j].u[k]));
    const float a = __low2float(m), b = __high2float(m);
    // a maximum of NaNs alone is one
    return fmaxf(fmaxf(a, b), neg_inf());
}
template <int N>
__device__ __forceinline__ float chunks_max(const Chunk (&c)[N], F32) {
    float m = neg_inf();
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) m = fmaxf(m, __uint_as_float(c[j].u[k]));
    return m;
}

// What orders logits as numbers, largest highest: 32 bits of value (both zeros
// alike, NaN as -infinity), then the place, lowest first.  Never 0.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x != x ? neg_inf() : x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

__device__ __forceinline__ uint64_t key_of(float x, int place) {
    return (uint64_t)order_of(x) << 32 | (uint32_t)~place;
}

// Element k of the chunks.
template <typename T, int N>
__device__ __forceinline__ float element_of(const Chunk (&c)[N], int k) {
    constexpr int V = T::kVec;
    const int word = V == 8 ? k / 2 : k;
    uint32_t w[4 * N];
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) w[i] = c[i / 4].u[i % 4];
#pragma unroll
    for (int half = 2 * N; half > 0; half /= 2)
#pragma unroll
        for (int i = 0; i < half; ++i) w[i] = word & half ? w[i + half] : w[i];
    if constexpr (V == 8) return k & 1 ? bf16_hi(w[0]) : bf16_lo(w[0]);
    return __uint_as_float(w[0]);
}

// The 32 best of two lists of 32 keys, the best in lane 0.
__device__ __forceinline__ void merge_keys(uint64_t &best, uint64_t other, int lane) {
    const uint64_t turned = __shfl_sync(0xffffffffu, other, 31 - lane);
    uint64_t v = best > turned ? best : turned;   // a bitonic run: one half-cleaner after another orders it
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const uint64_t w = __shfl_xor_sync(0xffffffffu, v, off);
        const bool first = (lane & off) == 0;
        v = first == (v > w) ? v : w;
    }
    best = v;
}

__device__ __forceinline__ void st_cluster_u64(const uint64_t *local, uint32_t rank, uint64_t v) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
    uint32_t ra;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.u64 [%0], %1;" : : "r"(ra), "l"(v) : "memory");
}

// (maximum, sum, sum of z exp(z)) of a unit or more, exponents in base 2.
struct Part {
    float m, s, t;
};

// b's sums, formed relative to b.m, relative to m.
__device__ __forceinline__ void add_part(Part &a, const Part &b, float c) {
    if (b.m == neg_inf()) {
        a.s += b.s;   // 0, or a NaN
        return;
    }
    const float d = (b.m - a.m) * c, f = ex2(d);
    a.s = fmaf(f, b.s, a.s);
    // f (t + d s); a part too small to count adds nothing
    if (f > 0.f) a.t = fmaf(f, fmaf(d, b.s, b.t), a.t);
}

// Lists of 32 keys in order, `many` of them (up to 8) `step` apart: the best 32
// of all, by half of the warps at a time.  Every thread of the block calls it.
__device__ __forceinline__ void merge_lists(uint64_t (*lists)[32], int many, int warp, int lane) {
#pragma unroll
    for (int half = 4; half > 0; half /= 2) {
        __syncthreads();
        if (warp < half && warp + half < many) {
            uint64_t best = lists[warp][lane];
            merge_keys(best, lists[warp + half][lane], lane);
            lists[warp][lane] = best;
        }
        if (many > half) many = half;
    }
}

// What a row's units come to.
struct RowSums {
    float m, log, entropy;
    bool none;   // every logit masked
};
template <bool ENT>
__device__ __forceinline__ RowSums sum_units(const float *units, const LogprobParams &p, int lane) {
    float most = neg_inf();
    for (int u = lane; u < p.units; u += 32) most = fmaxf(most, units[u]);
    Part a = {warp_max(most), 0.f, 0.f};
    for (int u = lane; u < p.units; u += 32)
        add_part(a, Part{units[u], units[p.units + u], ENT ? units[2 * p.units + u] : 0.f}, p.c);
    a.s = butterfly_sum<32>(a.s);
    if (ENT) a.t = butterfly_sum<32>(a.t);
    const bool none = a.m == neg_inf() && a.s == 0.f;
    const float log = none ? neg_inf() : logf(a.s);
    return RowSums{a.m, log, !ENT || none ? 0.f : log - kLn2 * a.t / a.s, none};
}

// The `top`-th largest of 32 values (equal ones in their order), lane i's being
// the i-th.
template <typename V>
__device__ __forceinline__ V nth_largest(const V *values, V mine, int top, int lane) {
    int before = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const V v = values[i];
        before += v > mine || (v == mine && i < lane);
    }
    return __shfl_sync(0xffffffffu, mine, __ffs(__ballot_sync(0xffffffffu, before == top - 1)) - 1);
}

// Keys gathered for a row at most; from kLpFew on they give a higher bound.
__host__ __device__ constexpr int lp_room(int warps) { return warps < 2 ? 256 : 128 * warps; }
constexpr int kLpFew = 96;

// Barrier of a row's warps alone.
__device__ __forceinline__ void row_barrier(int slot, int warps) {
    if (warps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" : : "r"(slot + 1), "r"(warps * 32) : "memory");
}

template <typename T, bool ALIGNED, bool ENT, bool TOP>
__global__ void __launch_bounds__(kLpThreads, 4) logprobs_fwd_kernel(const LogprobParams p) {
    constexpr int V = T::kVec, U = 8 / V;
    extern __shared__ float parts[];   // each row's units: maxima, sums, sums of z exp(z)
    __shared__ __align__(16) float maxima[kLpWarps][32];
    __shared__ __align__(16) uint64_t lists[kLpWarps][32], others[kClusterMaxCtas][32];
    __shared__ int flagged_count[kLpWarps], gathered_count[kLpWarps], flagged[kLpThreads];
    __shared__ uint64_t gathered[TOP ? 2048 : 1];   // lp_room(warps) for each row
    __shared__ RowSums row_sums[kLpWarps];
    const int tid = threadIdx.x, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int blocks = (int)cluster_ctas();
    // a block has 8 / warps rows, and a cluster of several blocks one
    const int warps = p.warps, warp = (tid >> 5) % warps, slot = (tid >> 5) / warps;
    const int64_t r = (int64_t)cluster_index() * (kLpWarps / warps) + slot;
    const bool there = r < p.rows;
    const char *row = p.logits + r * p.stride;
    const int off = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(row) & 15);
    const Around space = around(p.logits, row, p.rows, p.stride);
    float *mine = parts + (int64_t)slot * 3 * p.units;
    // before a block writes to the first one's shared memory, that has started
    if (blocks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" : : : "memory");
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    if (TOP && tid < kLpWarps) flagged_count[tid] = gathered_count[tid] = 0;
    // the given token; its logit is on its way with the first unit's
    int64_t token = -1;
    float given = 0.f;
    if (there && rank == 0 && warp == 0 && p.logprobs != nullptr)
        token = p.wide ? static_cast<const int64_t *>(p.tokens)[r]
                       : (int64_t) static_cast<const int32_t *>(p.tokens)[r];
    const int step = blocks * warps, begin = there ? (int)rank * warps + warp : p.units;
    float seen = neg_inf();   // the largest logit of this thread
    for (int unit = begin; unit < p.units; unit += step) {
        Chunk c[kLpChunks];
        load_unit<T, ALIGNED>(c, row, unit, lane, p.vocab, off, space);
        if (unit == 0 && (uint64_t)token < (uint64_t)p.vocab) given = widen_bits(ld_bits(row, token, T{}, 0), T{});
        const float local = chunks_max(c, T{});
        if (TOP) seen = fmaxf(seen, local);
        const float m = warp_max(local);
        const float from = m == neg_inf() ? 0.f : m;
        float2 s = make_float2(0.f, 0.f), t = make_float2(0.f, 0.f);
        const float2 less = make_float2(-from, -from), cc = make_float2(p.c, p.c);
        auto add = [&](const Chunk &chunk) {
            float x[V];
            unpack(chunk, x, T{});
#pragma unroll
            for (int k = 0; k < V; k += 2) {
                const float2 z = __fmul2_rn(__fadd2_rn(make_float2(x[k], x[k + 1]), less), cc);
                const float2 e = make_float2(ex2(z.x), ex2(z.y));
                s = __fadd2_rn(s, e);
                // a masked logit's z is -infinity: no part in the sum
                if (ENT) t = __ffma2_rn(e, make_float2(fmaxf(z.x, -1e4f), fmaxf(z.y, -1e4f)), t);
            }
        };
        // chunks that some lane has in the row
        const int used = (p.vocab - unit * lp_unit<T>() + 32 * V - 1) / (32 * V);
        if (used >= kLpChunks) {
#pragma unroll
            for (int j = 0; j < kLpChunks; ++j) add(c[j]);
        } else {
#pragma unroll
            for (int j = 0; j < kLpChunks; ++j) {
                if (j >= used) break;
                add(c[j]);
            }
        }
        const float sum = butterfly_sum<32>(s.x + s.y);
        const float zsum = ENT ? butterfly_sum<32>(t.x + t.y) : 0.f;
        if (blocks > 1 && unit == begin) {   // (every warp has one, or had none to begin with)
            __syncwarp();
            asm volatile("barrier.cluster.wait.acquire.aligned;" : : : "memory");
        }
        if (lane == 0) {
            if (blocks > 1) {
                st_cluster_f32(mine + unit, 0, m);
                st_cluster_f32(mine + p.units + unit, 0, sum);
                if (ENT) st_cluster_f32(mine + 2 * p.units + unit, 0, zsum);
            } else {
                mine[unit] = m;
                mine[p.units + unit] = sum;
                if (ENT) mine[2 * p.units + unit] = zsum;
            }
        }
    }
    if (blocks > 1 && begin >= p.units) asm volatile("barrier.cluster.wait.acquire.aligned;" : : : "memory");
    // The row that the next block on this SM is likely to take, its first units
    // into L2: blocks end about together, and memory would idle while they do
    // (bf16 1191 x 105656 42.6 -> 41.2 us).
    if (tid == 0 && r + p.ahead < p.rows && blocks == 1) {
        const char *next = p.logits + (r + p.ahead) * p.stride;
        const int64_t bytes = (int64_t)p.vocab * (16 / V), skip = -reinterpret_cast<uintptr_t>(next) & 15;
        const int64_t most = (bytes - skip) / 16 * 16;
        if (most > 0) prefetch_l2(next + skip, (unsigned)(most < kLpAhead ? most : kLpAhead));
    }
    // the units' sums are added up by the row's last warp while others look for alternatives
    const bool early = TOP && blocks == 1 && warps > 1;
    if (TOP) {
        // 32 groups of a row's threads: a lane's of every warp
        maxima[slot * warps + warp][lane] = seen;
        lists[slot * warps + warp][lane] = 0;
        __syncthreads();
        float of_group = neg_inf();
        for (int w = 0; w < warps; ++w) of_group = fmaxf(of_group, maxima[slot * warps + w][lane]);
        row_barrier(slot, warps);
        if (warp == 0) maxima[slot * warps][lane] = of_group;
        row_barrier(slot, warps);
        const float bound = nth_largest(maxima[slot * warps], of_group, p.top, lane);
        const bool lowest = bound == neg_inf();
        KeySearch search;
        search.start(order_of(bound), order_of(warp_max(of_group)));
        if (seen >= bound && begin < p.units)
            flagged[slot * warps * 32 + atomicAdd(flagged_count + slot, 1)] = warp * 32 + lane;   // in any order
        row_barrier(slot, warps);
        const int room = lp_room(warps), threads = warps * 32;
        uint64_t *keys = gathered + slot * room;
        int *count = gathered_count + slot;
        // every chunk of the flagged threads, one a thread
        const int each = begin < p.units + warp ? (p.units - (int)rank * warps + step - 1) / step * kLpChunks : 0;
        const int many = flagged_count[slot] * each;
        // i / each is the product's high word: exact while i < 2^18 and each <= 1024
        const uint32_t inverse = each > 1 ? 0xffffffffu / (uint32_t)each + 1 : 0;
        if (early && warp == warps - 1 && there) {
            const RowSums sums = sum_units<ENT>(mine, p, lane);
            if (lane == 0) row_sums[slot] = sums;
        }
        int found;
        for (;;) {
            for (int i0 = warp * 32; i0 < many; i0 += threads * U) {
                // Other warps add to the count meanwhile: one lane's read of it
                // decides for all, so that they stay together.
                if (__shfl_sync(0xffffffffu, *reinterpret_cast<volatile int *>(count), 0) > room) break;
                Chunk c[U];
                int at[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + u * threads + lane;
                    at[u] = p.vocab;
                    if (i < many) {
                        const int f = (int)__umulhi((uint32_t)i, inverse), j = i - f * each;
                        const int owner = flagged[slot * threads + f];
                        const int unit = (int)rank * warps + (owner >> 5) + j / kLpChunks * step;
                        if (unit < p.units) at[u] = unit * lp_unit<T>() + (j % kLpChunks * 32 + (owner & 31)) * V;
                    }
                    if (at[u] < p.vocab) {
                        Chunk one[1];
                        load_chunks<T, ALIGNED>(one, row, at[u], 0, p.vocab, off, space);
                        c[u] = one[0];
                    }
                }
                // which of them, then places for the warp's all at once
                uint32_t these = 0;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float x[V];
                    unpack(c[u], x, T{});
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        if (reaches(x[k], bound, lowest) && at[u] + k < p.vocab) these |= 1u << (u * V + k);
                }
                if (search.round > 0) {   // a bound that goes by places too
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float x[V];
                        unpack(c[u], x, T{});
#pragma unroll
                        for (int k = 0; k < V; ++k)
                            if (key_of(x[k], at[u] + k) < search.least) these &= ~(1u << (u * V + k));
                    }
                }
                int place = __popc(these), all = place;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int n = __shfl_up_sync(0xffffffffu, all, o);
                    if (lane >= o) all += n;
                }
                int first = 0;
                if (lane == 31 && all > 0) first = atomicAdd(count, all);   // in any order: the keys decide
                place = __shfl_sync(0xffffffffu, first, 31) + all - place;
                for (; these != 0; these &= these - 1, ++place) {
                    if (place >= room) break;
                    const int k = __ffs(these) - 1;
                    const float x = element_of<T>(c, k);
                    int where = at[0];
#pragma unroll
                    for (int u = 1; u < U; ++u) where = k / V == u ? at[u] : where;
                    keys[place] = key_of(x, where + k % V);
                }
            }
            row_barrier(slot, warps);
            found = *count;
            const int held = found < room ? found : room;
            const bool enough = search.enough(found, room, p.top);
            if (enough && found <= kLpFew) break;
            // the bound that 32 groups of these give
            uint64_t best = 0;
            for (int i = lane; i < held; i += 32) best = best > keys[i] ? best : keys[i];
            uint64_t kept[8];   // room / threads at most
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int i = warp * 32 + lane + k * threads;
                kept[k] = i < held ? keys[i] : 0;
            }
            row_barrier(slot, warps);
            if (warp == 0) {
                lists[slot * warps][lane] = best;
                if (lane == 0) *count = 0;
            }
            row_barrier(slot, warps);
            const uint64_t higher = nth_largest(lists[slot * warps], best, p.top, lane);
            if (enough)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (kept[k] >= higher && kept[k] != 0) keys[atomicAdd(count, 1)] = kept[k];
            row_barrier(slot, warps);
            if (warp == 0) lists[slot * warps][lane] = 0;
            if (enough) {
                found = *count;
                row_barrier(slot, warps);
                break;
            }
            search.next(found, room, higher);
            row_barrier(slot, warps);
        }
        // their order, by counting the larger ones
        for (int i = (warp * 32 + lane) / 8; i < (found + 3) / 4 * 4; i += threads / 8) {   // eight lanes a key
            const uint64_t key = i < found ? keys[i] : 0;
            int before = 0;
            for (int j = lane % 8; j < found; j += 8) before += keys[j] > key;
#pragma unroll
            for (int o = 1; o < 8; o *= 2) before += __shfl_xor_sync(0xffffffffu, before, o);
            if (i < found && before < 32 && lane % 8 == 0) {
                if (blocks > 1) st_cluster_u64(&others[rank][before], 0, key);
                else lists[slot * warps][before] = key;
            }
        }
        // where there are fewer than 32
        if (blocks > 1 && warp == 0 && lane >= found) st_cluster_u64(&others[rank][lane], 0, 0);
    }
    if (blocks > 1) {
        __syncwarp();
        cluster_barrier();
    } else {
        __syncthreads();
    }
    if (rank != 0) return;
    if (TOP && blocks > 1) {
        if (warp == kLpWarps - 1) {
            const RowSums sums = sum_units<ENT>(mine, p, lane);
            if (lane == 0) row_sums[slot] = sums;
        }
        merge_lists(others, blocks, warp, lane);   // (barriers of the block)
    }
    if (warp != 0 || !there) return;
    const RowSums sums = TOP && warps > 1 ? row_sums[slot] : sum_units<ENT>(mine, p, lane);
    if (lane == 0) {
        if (p.logprobs != nullptr)
            p.logprobs[r] = (uint64_t)token >= (uint64_t)p.vocab ? 0.f
                            : sums.none                          ? neg_inf()
                                                                 : (given - sums.m) * p.inv_t - sums.log;
        // a NaN takes no part in the maximum, but the row's is NaN where its log is
        if (p.stats != nullptr)
            *reinterpret_cast<float2 *>(p.stats + 2 * r) =
                make_float2(sums.log != sums.log ? sums.log : sums.m, sums.log);
        if (ENT) p.entropy[r] = sums.entropy;
    }
    if (TOP && lane < p.top) {
        const uint64_t best = blocks > 1 ? others[0][lane] : lists[slot * warps][lane];
        p.top_ids[r * p.top + lane] = (int32_t) ~(uint32_t)best;
        p.top_logprobs[r * p.top + lane] =
            sums.none ? neg_inf() : (value_of((uint32_t)(best >> 32)) - sums.m) * p.inv_t - sums.log;
    }
}

// ----------------------------------------------------------------- gradient

struct LogprobBwdParams {
    const char *logits;
    const void *tokens;
    const float *stats, *dlogprobs, *entropy, *dentropy;
    char *dlogits;
    int64_t rows, stride, dstride;   // bytes
    int32_t vocab, slices, turns;    // blocks of a row, and parts of it that each takes
    int32_t shift;                   // 2^shift threads of a row in a block: 32 .. 256
    int32_t wide;
    float inv_t, c;
};

constexpr int kLpBwdChunks = 4;

// d_v = (g [v is the token] - p_v (g + h (log p_v + H))) / temperature, with
// q = log2 p_v:  p (a + b q).  Chunks lie on dlogits' 16-byte boundaries
// (ALIGNED: on both tensors').
template <typename T, bool ALIGNED, bool ENT>
__global__ void __launch_bounds__(kLpThreads, 4) logprobs_bwd_kernel(const LogprobBwdParams p) {
    constexpr int V = T::kVec, E = 16 / V;
    const uint32_t group = blockIdx.x / (uint32_t)p.slices;
    const int slice = (int)(blockIdx.x - group * p.slices);
    const int64_t r = ((int64_t)group << (8 - p.shift)) + (threadIdx.x >> p.shift);
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    if (r >= p.rows) return;
    const char *row = p.logits + r * p.stride;
    char *to = p.dlogits + r * p.dstride;
    const int head = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(to) & 15) / E;
    const int off = ALIGNED ? 0 : (int)((reinterpret_cast<uintptr_t>(row) - head * E) & 15);
    const int step = V << p.shift, turn = kLpBwdChunks * step;
    const int begin = slice * p.turns * turn - head;
    const int place = ((int)threadIdx.x & ((1 << p.shift) - 1)) * V;
    const Around space = around(p.logits, row, p.rows, p.stride);
    // Chunks of a turn: all within the row, with what else is read (32 bytes), or some at its ends.
    Chunk c[kLpBwdChunks];
    auto whole = [&](int first) { return (ALIGNED || first > 0) && first + turn + (ALIGNED ? 0 : 2 * V) <= p.vocab; };
    auto load = [&](int first) {
        if (!whole(first)) {
            load_chunks<T, ALIGNED>(c, row, first + place, step, p.vocab, off, space);
            return;
        }
        const char *from = row + (int64_t)(first + place) * E - off;
        if (ALIGNED || off == 0) {
#pragma unroll
            for (int j = 0; j < kLpBwdChunks; ++j) c[j] = ld_keep_l2_16(from + j * step * E);
        } else {
            uint4 a[kLpBwdChunks];
#pragma unroll
            for (int j = 0; j < kLpBwdChunks; ++j) a[j] = ld_shared16(from + j * step * E);
#pragma unroll
            for (int j = 0; j < kLpBwdChunks; ++j) c[j] = across<T>(a[j], ld_shared16(from + j * step * E + 16), off);
        }
    };
    // The first turn's chunks come with the row's numbers, not behind them (bf16
    // 8192 x 131072: 659 us, and 720 behind them).
    load(begin);
    int token = -1;
    float g = 0.f, h = 0.f, own = 0.f;
    if (p.dlogprobs != nullptr) {
        const float given = p.dlogprobs[r];
        const int64_t id = p.wide ? static_cast<const int64_t *>(p.tokens)[r]
                                  : (int64_t) static_cast<const int32_t *>(p.tokens)[r];
        if ((uint64_t)id < (uint64_t)p.vocab) {
            token = (int)id;
            g = given;
        }
    }
    if (ENT) {
        h = p.dentropy[r];
        own = p.entropy[r];
    }
    const float2 stats = *reinterpret_cast<const float2 *>(p.stats + 2 * r);
    own = h == 0.f ? 0.f : h * own;
    const bool zero = (g == 0.f && h == 0.f) || (stats.x == neg_inf() && stats.y == neg_inf());
    const float2 less = make_float2(-stats.x, -stats.x), cc = make_float2(p.c, p.c);
    const float l = -stats.y * kLog2e, a = -(g + own) * p.inv_t, b = -h * p.inv_t * kLn2;
    for (int first = begin, t = 0;;) {
        const bool inside = whole(first);
#pragma unroll
        for (int j = 0; j < kLpBwdChunks; ++j) {
            const int i = first + place + j * step;
            if (!inside && i >= p.vocab) break;
            float x[V];
            unpack(c[j], x, T{});
#pragma unroll
            for (int k = 0; k < V; k += 2) {
                const float2 q = __ffma2_rn(__fadd2_rn(make_float2(x[k], x[k + 1]), less), cc, make_float2(l, l));
                const float2 e = make_float2(ex2(q.x), ex2(q.y));
                float2 d = make_float2(a, a);
                if (ENT) d = __ffma2_rn(make_float2(b, b), make_float2(fmaxf(q.x, -1e4f), fmaxf(q.y, -1e4f)), d);
                d = __fmul2_rn(e, d);
                x[k] = d.x;
                x[k + 1] = d.y;
            }
            const uint32_t at = (uint32_t)(token - i);
            if (at < (uint32_t)V && token >= 0) {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (at == (uint32_t)k) x[k] += g * p.inv_t;
            }
            const Chunk out = zero ? Chunk{} : pack(x, T{});
            if (inside || (i >= 0 && i + V <= p.vocab)) {
                st16(to + (int64_t)i * E, out);
            } else {
                unpack(out, x, T{});
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (i + k >= 0 && i + k < p.vocab) st_scalar(to, i + k, x[k], T{});
            }
        }
        first += turn;
        if (++t == p.turns || first >= p.vocab) return;
        if (!zero) load(first);   // rows that nothing reaches are not read on
    }
}

}  // namespace rrn
