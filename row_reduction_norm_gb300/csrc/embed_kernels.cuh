// embed_kernels.cuh -- the lookup of token embeddings, y[t] = RN(scale *
// table[tokens[t]]), and its gradient, dtable[v] = RN(scale * sum over t with
// tokens[t] = v of dy[t]).  Both are copies with a gather: what bounds them is
// HBM bandwidth, and latency for few tokens.
#pragma once

#include "rmsnorm_cluster.cuh"

namespace rrn {

// -------------------------------------------------------------- pieces
// A row moves in pieces of 16 bytes where everything is aligned to them, else
// of the largest power of two that is: P elements of type T.

template <int BYTES>
struct Raw;
template <>
struct Raw<16> {
    using type = uint4;
};
template <>
struct Raw<8> {
    using type = uint2;
};
template <>
struct Raw<4> {
    using type = uint32_t;
};
template <>
struct Raw<2> {
    using type = uint16_t;
};

template <typename T>
__host__ __device__ constexpr int elem_bytes() {
    return 16 / T::kVec;
}

template <typename T, int P>
struct PieceOf {
    static constexpr int kBytes = P * elem_bytes<T>();
    union {
        typename Raw<kBytes>::type raw;
        typename T::storage e[P];
    };
};

__device__ __forceinline__ float widened(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float widened(float v) { return v; }
__device__ __forceinline__ void narrow(float v, uint16_t &to) {
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    to = *reinterpret_cast<const uint16_t *>(&b);
}
__device__ __forceinline__ void narrow(float v, float &to) { to = v; }

// P values to consecutive elements, in stores of up to 16 bytes.
template <typename T, int P>
__device__ __forceinline__ void store_values(void *to, const float (&v)[P]) {
    constexpr int E = elem_bytes<T>(), W = P * E > 16 ? 16 / E : P;
#pragma unroll
    for (int i = 0; i < P; i += W) {
        PieceOf<T, W> out;
#pragma unroll
        for (int k = 0; k < W; ++k) narrow(v[i + k], out.e[k]);
        reinterpret_cast<decltype(out.raw) *>(to)[i / W] = out.raw;
    }
}
template <typename T, int P>
__device__ __forceinline__ void load_values(const void *from, float (&v)[P]) {
    constexpr int E = elem_bytes<T>(), W = P * E > 16 ? 16 / E : P;
#pragma unroll
    for (int i = 0; i < P; i += W) {
        PieceOf<T, W> in;
        in.raw = reinterpret_cast<const decltype(in.raw) *>(from)[i / W];
#pragma unroll
        for (int k = 0; k < W; ++k) v[i + k] = widened(in.e[k]);
    }
}

__device__ __forceinline__ int64_t token_at(const void *tokens, bool wide, int64_t i) {
    return wide ? static_cast<const int64_t *>(tokens)[i] : (int64_t) static_cast<const int32_t *>(tokens)[i];
}

// -------------------------------------------------------------- forward

struct EmbedParams {
    const void *tokens;
    const char *table;
    char *y;
    int64_t count, vocab;
    int64_t table_stride;   // bytes
    uint32_t pieces;        // of a row
    uint64_t magic;         // floor(2^40 / pieces) + 1
    int32_t wide;           // 64-bit tokens
    float scale;
};

constexpr int kEmbedThreads = 256;

// Pieces of all rows in one flat run, U a thread, so that any width fills the
// threads.  n / pieces by a multiplication: exact while n * pieces < 2^40 (n <
// pieces + U * 256, pieces <= 65536).
template <typename T, int P, int U>
__global__ void __launch_bounds__(kEmbedThreads) embed_fwd_kernel(const EmbedParams p) {
    const int64_t first = (int64_t)blockIdx.x * (kEmbedThreads * U);
    const int64_t t0 = first / p.pieces;
    const uint32_t c0 = (uint32_t)(first - t0 * p.pieces);
    uint32_t col[U];
    int64_t tok[U], id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t n = c0 + u * kEmbedThreads + threadIdx.x;
        const uint32_t q = (uint32_t)(((uint64_t)n * p.magic) >> 40);
        col[u] = n - q * p.pieces;
        tok[u] = t0 + q;
    }
    pdl_wait_for_inputs();
    pdl_allow_dependents();
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = tok[u] < p.count ? token_at(p.tokens, p.wide, tok[u]) : -1;
    PieceOf<T, P> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        v[u].raw = {};
        if ((uint64_t)id[u] < (uint64_t)p.vocab)
            v[u].raw = reinterpret_cast<const decltype(v[u].raw) *>(p.table + id[u] * p.table_stride)[col[u]];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (tok[u] >= p.count) continue;
        float f[P];
#pragma unroll
        for (int k = 0; k < P; ++k) f[k] = widened(v[u].e[k]) * p.scale;
        store_values<T, P>(p.y + (tok[u] * p.pieces + col[u]) * (P * elem_bytes<T>()), f);
    }
}

// ------------------------------------------------------ gradient: the sort
// Tokens sorted by id with their places, stably, by one cluster of blocks:
// digits of up to 10 bits from the lowest, counted and then placed.  A warp
// takes a run of consecutive places, so that counts per warp, summed over the
// warps and blocks before it, say where its next token of a digit belongs.
// Ids outside the table become `vocab`, which sorts behind all others.

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kSortDigits = 1024;
// Shared memory: a warp's counts for every warp, the block's totals and the
// digits' places.
constexpr int sort_smem(int bits) { return ((kSortWarps + 2) * 4) << bits; }

struct SortParams {
    const void *tokens;
    uint2 *a, *b;           // (id, place): passes write a, b, a, ...
    uint32_t *present;      // a bit for each id that occurs, or NULL
    int32_t count, words;   // words of present
    uint32_t vocab;
    int32_t passes, bits;   // bits of a digit
    int32_t wide;
};

__device__ __forceinline__ uint32_t ld_cluster_u32(const uint32_t *local, uint32_t rank) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
    uint32_t ra, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(ra) : "memory");
    return v;
}

__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_kernel(const SortParams p) {
    extern __shared__ uint32_t counts[];   // [warps][digits], total [digits], base [digits]
    __shared__ uint32_t carry[kSortWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), blocks = cluster_ctas();
    const int digits = 1 << p.bits;
    uint32_t *total = counts + kSortWarps * digits, *base = total + digits;
    // the warp's run of places, a multiple of 32 long
    const int64_t per_warp = ((int64_t)p.count + (int64_t)blocks * kSortThreads - 1) / (blocks * kSortThreads) * 32;
    const int64_t begin = (rank * kSortWarps + warp) * per_warp;
    const int64_t end = begin + per_warp < p.count ? begin + per_warp : p.count;
    uint32_t *mine = counts + warp * digits;
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    for (int i = rank * kSortThreads + tid; i < p.words; i += blocks * kSortThreads) p.present[i] = 0;
    for (int pass = 0; pass < p.passes; ++pass) {
        const uint2 *from = pass % 2 ? p.a : p.b;
        uint2 *to = pass % 2 ? p.b : p.a;
        const int shift = pass * p.bits;
        auto item = [&](int64_t i) {
            if (pass > 0) return __ldcg(from + i);
            const int64_t id = token_at(p.tokens, p.wide, i);
            return make_uint2((uint64_t)id < p.vocab ? (uint32_t)id : p.vocab, (uint32_t)i);
        };
        for (int i = lane; i < digits; i += 32) mine[i] = 0;
        __syncwarp();
        constexpr int U = 4;
        for (int64_t i = begin; i < end; i += 32 * U) {
            uint32_t d[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t at = i + u * 32 + lane;
                d[u] = at < end ? (item(at).x >> shift) & (digits - 1) : ~0u;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t same = __match_any_sync(0xffffffffu, d[u]);
                if (d[u] != ~0u && lane == __ffs(same) - 1) mine[d[u]] += __popc(same);
                __syncwarp();
            }
        }
        __syncthreads();
        // of each digit: what the warps before hold, and the block's total
        if (tid < digits) {
            uint32_t sum = 0;
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t n = counts[w * digits + tid];
                counts[w * digits + tid] = sum;
                sum += n;
            }
            total[tid] = sum;
        }
        __syncwarp();
        cluster_barrier();
        uint32_t before = 0, all = 0;
        if (tid < digits)
            for (uint32_t q = 0; q < blocks; ++q) {
                const uint32_t n = ld_cluster_u32(total + tid, q);
                all += n;
                before += q < rank ? n : 0;
            }
        // exclusive sums over the digits
        uint32_t sum = all;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t n = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += n;
        }
        if (lane == 31) carry[warp] = sum;
        __syncthreads();
        uint32_t c = lane < warp ? carry[lane] : 0;
        c = __reduce_add_sync(0xffffffffu, c);
        if (tid < digits) base[tid] = c + sum - all + before;
        __syncthreads();
        for (int64_t i = begin; i < end; i += 32 * U) {
            uint2 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t at = i + u * 32 + lane;
                v[u] = at < end ? item(at) : make_uint2(~0u, 0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool valid = i + u * 32 + lane < end;
                const uint32_t d = valid ? (v[u].x >> shift) & (digits - 1) : ~0u;
                const uint32_t same = __match_any_sync(0xffffffffu, d);
                uint32_t at = 0;
                if (valid) at = mine[d];
                __syncwarp();
                if (valid) {
                    if (lane == __ffs(same) - 1) mine[d] = at + __popc(same);
                    to[base[d] + at + __popc(same & ((1u << lane) - 1))] = v[u];
                    if (pass == 0 && p.present != nullptr && v[u].x < p.vocab)
                        atomicOr(p.present + (v[u].x >> 5), 1u << (v[u].x & 31));
                }
                __syncwarp();
            }
        }
        // the next pass reads what all blocks wrote, and no block reads this
        // one's totals any more
        cluster_barrier();
    }
}

// -------------------------------------------- gradient: sums of sorted runs
// A warp takes a segment of 32 sorted tokens and 256 columns: a lane's eight
// sums stay in registers while it walks the rows of dy, the next U of them on
// their way.  A run of equal ids that lies within the segment is written out;
// one that began before, or goes on behind, leaves its part in the workspace,
// which embed_join_kernel adds up.  Slots 2 s and 2 s + 1 of the workspace: the
// part of a run that segment s did not begin, and of one that it did.

constexpr int kSumThreads = 256, kSumWarps = kSumThreads / 32, kSegment = 32, kTile = 256;

struct SumParams {
    const uint2 *sorted;
    const char *dy;
    char *dtable;
    const uint32_t *present;
    float *partial;
    int64_t dy_stride, table_stride;   // bytes
    int64_t vocab;
    int32_t count, width, segments, tiles;
    int64_t work_blocks;               // of the sums; those behind them write zeros
    float scale;
    int32_t accumulate;
    int32_t zero_bytes;                // zeros are written in pieces of this
};

// Row `id` of the gradient, the lane's eight columns of a tile.
template <typename TG, int P>
__device__ __forceinline__ void write_row(const SumParams &p, uint32_t id, int tile, int lane, const float (&sum)[8]) {
    char *row = p.dtable + (int64_t)id * p.table_stride;
#pragma unroll
    for (int j = 0; j < 8 / P; ++j) {
        const int col = tile * kTile + (j * 32 + lane) * P;
        if (col >= p.width) continue;
        char *at = row + (int64_t)col * elem_bytes<TG>();
        float v[P];
        if (p.accumulate) {
            load_values<TG, P>(at, v);
#pragma unroll
            for (int k = 0; k < P; ++k) v[k] = fmaf(sum[j * P + k], p.scale, v[k]);
        } else {
#pragma unroll
            for (int k = 0; k < P; ++k) v[k] = sum[j * P + k] * p.scale;
        }
        store_values<TG, P>(at, v);
    }
}

__device__ __forceinline__ float4 *partial_slot(const SumParams &p, int64_t slot, int tile, int lane) {
    return reinterpret_cast<float4 *>(p.partial + (slot * p.tiles + tile) * kTile) + lane;
}
__device__ __forceinline__ void write_partial(const SumParams &p, int64_t slot, int tile, int lane, const float (&s)[8]) {
    float4 *to = partial_slot(p, slot, tile, lane);
    to[0] = make_float4(s[0], s[1], s[2], s[3]);
    to[32] = make_float4(s[4], s[5], s[6], s[7]);
}

template <typename RAW>
__device__ __forceinline__ void zero_row(char *row, int64_t bytes, int lane) {
    RAW *to = reinterpret_cast<RAW *>(row);
    const int64_t n = bytes / (int64_t)sizeof(RAW);
    for (int64_t i = lane; i < n; i += 32) to[i] = RAW{};
}

template <typename T, typename TG, int P>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const SumParams p) {
    constexpr int U = P * elem_bytes<T>() * (8 / P) > 16 ? 4 : 8, N = 8 / P;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    if ((int64_t)blockIdx.x >= p.work_blocks) {   // eight rows, a warp each: zeros where no token is
        const int64_t row = ((int64_t)blockIdx.x - p.work_blocks) * kSumWarps + warp;
        if (row >= p.vocab || (p.present[row >> 5] >> (row & 31) & 1)) return;
        char *at = p.dtable + row * p.table_stride;
        const int64_t bytes = (int64_t)p.width * elem_bytes<TG>();
        if (p.zero_bytes == 16) zero_row<uint4>(at, bytes, lane);
        else if (p.zero_bytes == 8) zero_row<uint2>(at, bytes, lane);
        else if (p.zero_bytes == 4) zero_row<uint32_t>(at, bytes, lane);
        else zero_row<uint16_t>(at, bytes, lane);
        return;
    }
    const int64_t item = (int64_t)blockIdx.x * kSumWarps + warp;
    const int64_t seg = item / p.tiles;
    if (seg >= p.segments) return;
    const int tile = (int)(item - seg * p.tiles);
    const int64_t first = seg * kSegment;
    const uint32_t none = (uint32_t)p.vocab;
    const uint2 e = first + lane < p.count ? p.sorted[first + lane] : make_uint2(none, 0);
    const uint32_t before = first > 0 ? p.sorted[first - 1].x : ~0u;
    const uint32_t behind = first + kSegment < p.count ? p.sorted[first + kSegment].x : none;
    uint32_t next = __shfl_down_sync(0xffffffffu, e.x, 1);
    if (lane == 31) next = behind;
    const uint32_t valid = __ballot_sync(0xffffffffu, e.x < none);
    const uint32_t ends = __ballot_sync(0xffffffffu, e.x < none && e.x != next);
    const int n = __popc(valid);   // valid ones come first
    bool began = __shfl_sync(0xffffffffu, e.x, 0) != before;   // this run, here
    float sum[8] = {};
    for (int j = 0; j < n; j += U) {
        PieceOf<T, P> v[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t place = __shfl_sync(0xffffffffu, e.y, (j + u) & 31);
            const char *row = p.dy + (int64_t)place * p.dy_stride;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int col = tile * kTile + (i * 32 + lane) * P;
                v[u][i].raw = {};
                if (j + u < n && col < p.width)
                    v[u][i].raw = *reinterpret_cast<const decltype(v[u][i].raw) *>(row + (int64_t)col * elem_bytes<T>());
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j + u >= n) break;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int k = 0; k < P; ++k) sum[i * P + k] += widened(v[u][i].e[k]);
            if (ends >> (j + u) & 1) {
                const uint32_t id = __shfl_sync(0xffffffffu, e.x, j + u);
                if (began) write_row<TG, P>(p, id, tile, lane, sum);
                else write_partial(p, 2 * seg, tile, lane, sum);
                began = true;
#pragma unroll
                for (int k = 0; k < 8; ++k) sum[k] = 0.f;
            }
        }
    }
    if (n > 0 && !(ends >> (n - 1) & 1)) write_partial(p, 2 * seg + (began ? 1 : 0), tile, lane, sum);
}

// Runs that go on behind the segment that began them: its part and the
// following segments', in their order.
template <typename TG, int P>
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(const SumParams p) {
    constexpr int U = 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t item = (int64_t)blockIdx.x * kSumWarps + warp;
    const int64_t seg = item / p.tiles;
    const int tile = (int)(item - seg * p.tiles);
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    if (seg >= p.segments - 1) return;
    const int64_t last = seg * kSegment + kSegment - 1;
    const uint32_t id = p.sorted[last].x;
    if (id >= (uint32_t)p.vocab || p.sorted[last + 1].x != id) return;
    if (seg > 0 && p.sorted[seg * kSegment].x == id && p.sorted[seg * kSegment - 1].x == id) return;   // begun before
    // segments behind this one that hold more of the run
    int64_t more = 1;
    for (;;) {
        const int64_t at = last + (more + lane) * kSegment;   // the last token of that segment
        const bool on = at + 1 < p.count && p.sorted[at].x == id && p.sorted[at + 1].x == id;
        const uint32_t not_on = ~__ballot_sync(0xffffffffu, on);
        if (not_on) {
            more += __ffs(not_on) - 1;
            break;
        }
        more += 32;
    }
    float sum[8];
    {
        const float4 *at = partial_slot(p, 2 * seg + 1, tile, lane);
        const float4 a = at[0], b = at[32];
        sum[0] = a.x, sum[1] = a.y, sum[2] = a.z, sum[3] = a.w;
        sum[4] = b.x, sum[5] = b.y, sum[6] = b.z, sum[7] = b.w;
    }
    for (int64_t s = 1; s <= more; s += U) {
        float4 a[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            a[u] = b[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (s + u <= more) {
                const float4 *at = partial_slot(p, 2 * (seg + s + u), tile, lane);
                a[u] = at[0];
                b[u] = at[32];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            sum[0] += a[u].x, sum[1] += a[u].y, sum[2] += a[u].z, sum[3] += a[u].w;
            sum[4] += b[u].x, sum[5] += b[u].y, sum[6] += b[u].z, sum[7] += b[u].w;
        }
    }
    write_row<TG, P>(p, id, tile, lane, sum);
}

}  // namespace rrn
