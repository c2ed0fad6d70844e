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
// largest; their few chunks are read again (from L2) by whole warps, which
// keep the 32 best in order, a key of value and place a lane.
//
// Gradient: elementwise, given the forward's statistics.  One read and one
// write of every element; HBM bandwidth bounds both.
#pragma once

#include "rmsnorm_cluster.cuh"

namespace rrn {

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32, kLpChunks = 8;
constexpr int kLpTop = 32;   // alternatives at most
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
    int64_t stride;      // bytes
    int32_t vocab, units, top;
    int32_t wide;        // 64-bit tokens
    int32_t aligned;     // every row on a 16-byte boundary
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

// Elements i .. i + V - 1 of a row as a chunk; -infinity behind its end.
template <typename T>
__device__ __forceinline__ Chunk logits_chunk(const char *row, int i, int vocab, bool aligned) {
    constexpr int V = T::kVec;
    constexpr int E = 16 / V;
    if (aligned && i + V <= vocab) return ld_keep_l2_16(row + (int64_t)i * E);
    Chunk c;
    if constexpr (V == 8) {
        const uint16_t *at = reinterpret_cast<const uint16_t *>(row) + i;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t lo = i + 2 * k < vocab ? at[2 * k] : 0xff80u;
            const uint32_t hi = i + 2 * k + 1 < vocab ? at[2 * k + 1] : 0xff80u;
            c.u[k] = lo | hi << 16;
        }
    } else {
        const uint32_t *at = reinterpret_cast<const uint32_t *>(row) + i;
#pragma unroll
        for (int k = 0; k < 4; ++k) c.u[k] = i + k < vocab ? at[k] : 0xff800000u;
    }
    return c;
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

// One key more into the warp's 32 best, lane 0 the best (a lower one changes nothing).
__device__ __forceinline__ void insert_key(uint64_t &best, uint64_t key, int lane) {
    const int at = __popc(__ballot_sync(0xffffffffu, best > key));
    const uint64_t above = __shfl_up_sync(0xffffffffu, best, 1);
    if (lane == at) best = key;
    else if (lane > at) best = above;
}

// The 32 best of two such lists.
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

template <typename T, bool ENT, bool TOP>
__global__ void __launch_bounds__(kLpThreads) logprobs_fwd_kernel(const LogprobParams p) {
    constexpr int V = T::kVec;
    extern __shared__ float parts[];   // the row's units: maxima, sums, sums of z exp(z)
    __shared__ float group_max[32];
    __shared__ uint64_t lists[kLpWarps][32], others[kClusterMaxCtas][32];
    __shared__ int flagged_count, flagged[kLpThreads];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const int blocks = (int)cluster_ctas();
    const int64_t r = cluster_index();
    const char *row = p.logits + r * p.stride;
    // before a block writes to the first one's shared memory, that has started
    asm volatile("barrier.cluster.arrive.release.aligned;" : : : "memory");
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    if (TOP && tid == 0) flagged_count = 0;
    // the given token's logit, on its way while the sums are formed
    int64_t token = -1;
    float given = 0.f;
    if (rank == 0 && tid == 0 && p.logprobs != nullptr) {
        token = p.wide ? static_cast<const int64_t *>(p.tokens)[r] : (int64_t) static_cast<const int32_t *>(p.tokens)[r];
        if ((uint64_t)token < (uint64_t)p.vocab)
            given = widen_bits(ld_bits(row, token, T{}, 0), T{});
    }
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" : : : "memory");
    float seen = neg_inf();   // the largest logit of this thread
    const int step = blocks * kLpWarps;
    for (int unit = (int)rank * kLpWarps + warp; unit < p.units; unit += step) {
        Chunk c[kLpChunks];
        const int first = unit * lp_unit<T>() + lane * V;
#pragma unroll
        for (int j = 0; j < kLpChunks; ++j) c[j] = logits_chunk<T>(row, first + j * 32 * V, p.vocab, p.aligned);
        const float local = chunks_max(c, T{});
        if (TOP) seen = fmaxf(seen, local);
        const float m = warp_max(local);
        const float from = m == neg_inf() ? 0.f : m;
        float2 s = make_float2(0.f, 0.f), t = make_float2(0.f, 0.f);
        const float2 off = make_float2(-from, -from), cc = make_float2(p.c, p.c);
#pragma unroll
        for (int j = 0; j < kLpChunks; ++j) {
            float x[V];
            unpack(c[j], x, T{});
#pragma unroll
            for (int k = 0; k < V; k += 2) {
                const float2 z = __fmul2_rn(__fadd2_rn(make_float2(x[k], x[k + 1]), off), cc);
                const float2 e = make_float2(ex2(z.x), ex2(z.y));
                s = __fadd2_rn(s, e);
                // a masked logit's z is -infinity: no part in the sum
                if (ENT) t = __ffma2_rn(e, make_float2(fmaxf(z.x, -1e4f), fmaxf(z.y, -1e4f)), t);
            }
        }
        const float sum = butterfly_sum<32>(s.x + s.y);
        const float zsum = ENT ? butterfly_sum<32>(t.x + t.y) : 0.f;
        if (lane == 0) {
            st_cluster_f32(parts + unit, 0, m);
            st_cluster_f32(parts + p.units + unit, 0, sum);
            if (ENT) st_cluster_f32(parts + 2 * p.units + unit, 0, zsum);
        }
    }
    uint64_t best = 0;
    if (TOP) {
        const float of_group = fmaxf(fmaxf(seen, __shfl_xor_sync(0xffffffffu, seen, 1)), neg_inf());
        const float two = fmaxf(of_group, __shfl_xor_sync(0xffffffffu, of_group, 2));
        const float four = fmaxf(two, __shfl_xor_sync(0xffffffffu, two, 4));
        if (lane % 8 == 0) group_max[warp * 4 + lane / 8] = four;
        __syncthreads();
        // the bound: the group maximum that p.top - 1 others come before
        const float held = group_max[lane];
        int before = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float v = __shfl_sync(0xffffffffu, held, i);
            before += v > held || (v == held && i < lane);
        }
        const float bound = __shfl_sync(0xffffffffu, held, __ffs(__ballot_sync(0xffffffffu, before == p.top - 1)) - 1);
        if (seen >= bound) flagged[atomicAdd(&flagged_count, 1)] = tid;   // in any order: the keys decide
        __syncthreads();
        const uint32_t least = order_of(bound);
        const int many = flagged_count;
        const int mine = p.units / step * kLpChunks + kLpChunks;   // chunks of a thread at most
        for (int f = warp; f < many; f += kLpWarps) {
            const int owner = flagged[f];
            for (int i0 = 0; i0 < mine; i0 += 32) {
                const int i = i0 + lane;
                const int unit = (int)rank * kLpWarps + (owner >> 5) + i / kLpChunks * step;
                const bool there = i < mine && unit < p.units;
                const int at = unit * lp_unit<T>() + (i % kLpChunks * 32 + (owner & 31)) * V;
                float x[V];
                if (there) unpack(logits_chunk<T>(row, at, p.vocab, p.aligned), x, T{});
                const uint64_t worst = __shfl_sync(0xffffffffu, best, p.top - 1);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const uint32_t o = there && at + k < p.vocab ? order_of(x[k]) : 0;
                    const uint64_t key = o >= least ? (uint64_t)o << 32 | (uint32_t)~(at + k) : 0;
                    uint32_t todo = __ballot_sync(0xffffffffu, key > worst);
                    while (todo) {
                        const int from = __ffs(todo) - 1;
                        todo &= todo - 1;
                        insert_key(best, __shfl_sync(0xffffffffu, key, from), lane);
                    }
                }
            }
        }
        lists[warp][lane] = best;
        __syncthreads();
        if (warp == 0) {
            for (int w = 1; w < kLpWarps; ++w) merge_keys(best, lists[w][lane], lane);
            if (rank != 0) st_cluster_u64(&others[rank][lane], 0, best);
        }
    }
    __syncwarp();
    cluster_barrier();
    if (rank != 0 || warp != 0) return;
    float most = neg_inf();
    for (int u = lane; u < p.units; u += 32) most = fmaxf(most, parts[u]);
    Part a = {warp_max(most), 0.f, 0.f};
    for (int u = lane; u < p.units; u += 32)
        add_part(a, Part{parts[u], parts[p.units + u], ENT ? parts[2 * p.units + u] : 0.f}, p.c);
    a.s = butterfly_sum<32>(a.s);
    if (ENT) a.t = butterfly_sum<32>(a.t);
    const bool none = a.m == neg_inf() && a.s == 0.f;   // every logit masked
    const float log = none ? neg_inf() : logf(a.s);
    if (lane == 0) {
        if (p.logprobs != nullptr)
            p.logprobs[r] = (uint64_t)token >= (uint64_t)p.vocab ? 0.f : none ? neg_inf() : (given - a.m) * p.inv_t - log;
        if (p.stats != nullptr) *reinterpret_cast<float2 *>(p.stats + 2 * r) = make_float2(a.m, log);
        if (ENT) p.entropy[r] = none ? 0.f : log - kLn2 * a.t / a.s;
    }
    if (TOP) {
        for (int q = 1; q < blocks; ++q) merge_keys(best, others[q][lane], lane);
        if (lane < p.top) {
            p.top_ids[r * p.top + lane] = (int32_t) ~(uint32_t)best;
            p.top_logprobs[r * p.top + lane] = none ? neg_inf() : (value_of((uint32_t)(best >> 32)) - a.m) * p.inv_t - log;
        }
    }
}

// ----------------------------------------------------------------- gradient

struct LogprobBwdParams {
    const char *logits;
    const void *tokens;
    const float *stats, *dlogprobs, *entropy, *dentropy;
    char *dlogits;
    int64_t stride, dstride;   // bytes
    int32_t vocab, slices;     // blocks of a row
    int32_t wide;
    int32_t aligned;
    float inv_t;
};

constexpr int kLpBwdChunks = 4;

// d_v = (g [v is the token] - p_v (g + h (log p_v + H))) / temperature
template <typename T, bool ENT>
__global__ void __launch_bounds__(kLpThreads) logprobs_bwd_kernel(const LogprobBwdParams p) {
    constexpr int V = T::kVec, E = 16 / V;
    const int64_t r = blockIdx.x / p.slices;
    const int slice = (int)(blockIdx.x - r * p.slices);
    const char *row = p.logits + r * p.stride;
    char *to = p.dlogits + r * p.dstride;
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    int64_t token = -1;
    float g = 0.f, h = 0.f, own = 0.f;
    if (p.dlogprobs != nullptr) {
        token = p.wide ? static_cast<const int64_t *>(p.tokens)[r] : (int64_t) static_cast<const int32_t *>(p.tokens)[r];
        if ((uint64_t)token < (uint64_t)p.vocab) g = p.dlogprobs[r];
        else token = -1;
    }
    if (ENT) h = p.dentropy[r];
    const float2 stats = *reinterpret_cast<const float2 *>(p.stats + 2 * r);
    if (ENT) own = h == 0.f ? 0.f : h * p.entropy[r];
    const bool zero = (g == 0.f && h == 0.f) || (stats.x == neg_inf() && stats.y == neg_inf());
    const float gt = g * p.inv_t;
    const float a = -(g + own) * p.inv_t, b = -h * p.inv_t;   // d = p (a + b log p)
    const float2 off = make_float2(-stats.x, -stats.x), it = make_float2(p.inv_t, p.inv_t);
    const float2 nl = make_float2(-stats.y, -stats.y), l2 = make_float2(kLog2e, kLog2e);
    const float2 a2 = make_float2(a, a), b2 = make_float2(b, b);
    const int first = (slice * kLpBwdChunks * kLpThreads + threadIdx.x) * V;
    Chunk c[kLpBwdChunks];
#pragma unroll
    for (int j = 0; j < kLpBwdChunks; ++j) {
        const int i = first + j * kLpThreads * V;
        if (!zero && i < p.vocab) c[j] = logits_chunk<T>(row, i, p.vocab, p.aligned);
        else c[j] = Chunk{};
    }
#pragma unroll
    for (int j = 0; j < kLpBwdChunks; ++j) {
        const int i = first + j * kLpThreads * V;
        if (i >= p.vocab) return;
        float x[V];
        unpack(c[j], x, T{});
        if (zero) {
#pragma unroll
            for (int k = 0; k < V; ++k) x[k] = 0.f;
        } else {
#pragma unroll
            for (int k = 0; k < V; k += 2) {
                float2 lp = __ffma2_rn(__fadd2_rn(make_float2(x[k], x[k + 1]), off), it, nl);
                const float2 q = __fmul2_rn(lp, l2);
                const float2 e = make_float2(ex2(q.x), ex2(q.y));
                float2 d = a2;
                if (ENT) d = __ffma2_rn(b2, make_float2(fmaxf(lp.x, -1e4f), fmaxf(lp.y, -1e4f)), a2);
                d = __fmul2_rn(e, d);
                x[k] = d.x;
                x[k + 1] = d.y;
            }
            const uint32_t at = (uint32_t)((int)token - i);
            if (at < (uint32_t)V) {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (at == (uint32_t)k) x[k] += gt;
            }
        }
        if (p.aligned && i + V <= p.vocab) {
            st16(to + (int64_t)i * E, pack(x, T{}));
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (i + k < p.vocab) st_scalar(to, i + k, x[k], T{});
        }
    }
}

}  // namespace rrn
