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
// digits of up to 9 bits from the lowest, counted and then placed.  A warp
// takes a run of consecutive places, so that counts per warp, summed over the
// warps and blocks before it, say where its next token of a digit belongs.
// Ids outside the table become `vocab`, which sorts behind all others.  Latency
// bounds it: 16384 tokens of 32768 ids take 12 us, 65536 of them 17 (28,000
// cycles: 5,800 and 4,600 the two passes' placing, 1,000 to 2,200 each of their
// four cluster barriers).  Blocks of 1024 or 256 threads are slower (with the
// sums, us: bf16 1000 x 1024 13.7 and 11.3, 512 threads 9.8; 65536 x 768 47.2 and
// 51.8, 46.3), and so are tokens put in order in shared memory before they are
// stored side by side (5000 x 1024 13.3, 13.0; 65536 x 768 50.0, 49.6).

constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32, kSortMaxBits = 9;
constexpr int kSortBlocks = 16, kSortSteps = 8;   // steps of 32 tokens that a warp holds in registers
// Words of presence bits that a block gathers in shared memory before they go to
// the device's: thousands of tokens of one id there wait for one another (65536
// tokens of 50257 ids: 12,500 cycles for the first pass, 6,400 without).
constexpr int kSortWords = 8192;
// Shared memory: a warp's counts and lanes of each digit for every warp, the
// blocks' totals and the digits' places, and the presence bits.
constexpr int sort_smem(int bits, int words) {
    return (((2 * kSortWarps + kSortBlocks + 1) * 4) << bits) + (words <= kSortWords ? words * 4 : 0);
}

struct SortParams {
    const void *tokens;
    uint2 *a, *b;           // (id, place): passes write a, b, a, ...
    uint32_t *present;      // a bit for each id that occurs, or NULL
    int32_t count, words;   // words of present
    uint32_t vocab;
    int32_t passes, bits;   // bits of a digit
    int32_t wide;
    char *dtable;           // zeros by the blocks behind the sorting ones:
    int64_t table_stride, zero_rows;   // rows 0 .. zero_rows - 1, a stride of bytes
    int32_t row_bytes, zero_bytes;
};

// Zeros in 512 bytes of each of `rows` rows (32 at most), but for those whose
// bit is set: narrower rows several at once.
constexpr int kZeroBytes = 512;
template <typename RAW>
__device__ __forceinline__ void zero_rows(char *first, int64_t stride, int rows, int part, uint32_t but, int row_bytes,
                                          int lane) {
    constexpr int B = (int)sizeof(RAW);
    const int rest = row_bytes - part * kZeroBytes;
    const int pieces = (rest < kZeroBytes ? rest : kZeroBytes) / B;
    int lanes = 1;                       // of a row
    while (lanes < 32 && lanes < pieces) lanes *= 2;
    for (int r = lane / lanes; r < rows; r += 32 / lanes) {
        if (but >> r & 1) continue;
        RAW *to = reinterpret_cast<RAW *>(first + r * stride + part * kZeroBytes);
        for (int i = lane % lanes; i < pieces; i += lanes) to[i] = RAW{};
    }
}
// In pieces of zero_bytes.
__device__ __forceinline__ void zero_rows(char *first, int64_t stride, int rows, int part, uint32_t but, int row_bytes,
                                          int zero_bytes, int lane) {
    if (zero_bytes == 16) zero_rows<uint4>(first, stride, rows, part, but, row_bytes, lane);
    else if (zero_bytes == 8) zero_rows<uint2>(first, stride, rows, part, but, row_bytes, lane);
    else if (zero_bytes == 4) zero_rows<uint32_t>(first, stride, rows, part, but, row_bytes, lane);
    else zero_rows<uint16_t>(first, stride, rows, part, but, row_bytes, lane);
}

__device__ __forceinline__ void st_cluster_u32(const uint32_t *local, uint32_t rank, uint32_t v) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
    uint32_t ra;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" : : "r"(ra), "r"(v) : "memory");
}

__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_kernel(const SortParams p) {
    if (cluster_index() > 0) {   // the sort leaves most SMs idle: they write zeros
        const int lane = threadIdx.x & 31, parts = (p.row_bytes + kZeroBytes - 1) / kZeroBytes;
        const int64_t warps = (int64_t)(gridDim.x - cluster_ctas()) * kSortWarps;
        const int64_t items = (p.zero_rows + 31) / 32 * parts;
        int64_t i = (int64_t)(blockIdx.x - cluster_ctas()) * kSortWarps + (threadIdx.x >> 5);
        pdl_wait_for_inputs();
        pdl_allow_dependents();
        for (; i < items; i += warps) {
            const int64_t row = i / parts * 32, rest = p.zero_rows - row;
            zero_rows(p.dtable + row * p.table_stride, p.table_stride, rest < 32 ? (int)rest : 32, (int)(i % parts), 0,
                      p.row_bytes, p.zero_bytes, lane);
        }
        return;
    }
    extern __shared__ uint32_t counts[];   // [warps][digits], totals [blocks][digits], base [digits], ...
    __shared__ uint32_t carry[kSortWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), blocks = cluster_ctas();
    const int digits = 1 << p.bits;
    uint32_t *totals = counts + kSortWarps * digits, *base = totals + kSortBlocks * digits;
    uint32_t *lanes = base + digits + warp * digits, *bits = base + (kSortWarps + 1) * digits;
    const bool gather = p.words <= kSortWords;
    // the warp's run of places, a multiple of 32 long
    const int64_t per_warp = ((int64_t)p.count + (int64_t)blocks * kSortThreads - 1) / (blocks * kSortThreads) * 32;
    const int64_t begin = (rank * kSortWarps + warp) * per_warp;
    const int64_t end = begin + per_warp < p.count ? begin + per_warp : p.count;
    constexpr int U = kSortSteps;
    const bool held = per_warp <= 32 * U;   // in registers from the count to the placing
    uint32_t *mine = counts + warp * digits;
    // a block writes to another's shared memory once that has started
    if (blocks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" : : : "memory");
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    uint2 v[U];
    auto load = [&](int pass, const uint2 *from, int64_t i) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = i + u * 32 + lane;
            v[u] = make_uint2(~0u, 0);
            if (at >= end) continue;
            if (pass > 0) {
                v[u] = __ldcg(from + at);
            } else {
                const int64_t id = token_at(p.tokens, p.wide, at);
                v[u] = make_uint2((uint64_t)id < p.vocab ? (uint32_t)id : p.vocab, (uint32_t)at);
            }
        }
    };
    for (int pass = 0; pass < p.passes; ++pass) {
        const uint2 *from = pass % 2 ? p.a : p.b;
        uint2 *to = pass % 2 ? p.b : p.a;
        const int shift = pass * p.bits;
        if (held) load(pass, from, begin);
        if (pass == 0) {
            for (int i = rank * kSortThreads + tid; i < p.words; i += blocks * kSortThreads) p.present[i] = 0;
            if (gather)
                for (int i = tid; i < p.words; i += kSortThreads) bits[i] = 0;
        }
        for (int i = lane; i < digits; i += 32) mine[i] = lanes[i] = 0;
        __syncwarp();
        for (int64_t i = begin; i < end; i += 32 * U) {
            if (!held) load(pass, from, i);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i + u * 32 + lane < end) atomicAdd(mine + ((v[u].x >> shift) & (digits - 1)), 1u);
        }
        if (blocks > 1 && pass == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" : : : "memory");
        __syncthreads();
        // of each digit: what the warps before hold, and the block's total, for
        // every block
        if (tid < digits) {
            uint32_t n[kSortWarps], sum = 0;
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) n[w] = counts[w * digits + tid];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                counts[w * digits + tid] = sum;
                sum += n[w];
            }
            for (uint32_t q = 0; q < blocks; ++q) st_cluster_u32(totals + rank * digits + tid, q, sum);
        }
        __syncwarp();
        if (blocks > 1) cluster_barrier();
        uint32_t before = 0, all = 0;
        if (tid < digits) {
#pragma unroll
            for (uint32_t q = 0; q < kSortBlocks; ++q) {
                const uint32_t n = q < blocks ? totals[q * digits + tid] : 0;
                all += n;
                before += q < rank ? n : 0;
            }
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
            if (!held) load(pass, from, i);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i + u * 32 >= end) break;
                const bool valid = i + u * 32 + lane < end;
                const uint32_t d = (v[u].x >> shift) & (digits - 1);
                // The lanes with the same digit, gathered in shared memory: nine
                // votes, or a match of 32 different values, take five times as long.
                if (valid) atomicOr(lanes + d, 1u << lane);
                __syncwarp();
                uint32_t at = 0, same = 1u << lane;
                if (valid) {
                    same = lanes[d];
                    at = mine[d];
                }
                __syncwarp();
                const int lead = __ffs(same) - 1;
                if (valid) {
                    if (lane == lead) {
                        lanes[d] = 0;
                        mine[d] = at + __popc(same);
                    }
                    to[base[d] + at + __popc(same & ((1u << lane) - 1))] = v[u];
                }
                if (pass == 0 && p.present != nullptr) {
                    // the first lane of a digit speaks for those with its id
                    const uint32_t id = __shfl_sync(0xffffffffu, v[u].x, lead);
                    if (valid && v[u].x < p.vocab && (lane == lead || id != v[u].x))
                        atomicOr((gather ? bits : p.present) + (v[u].x >> 5), 1u << (v[u].x & 31));
                }
                __syncwarp();
            }
        }
        if (pass == 0 && gather && p.words > 0) {
            __syncthreads();
            for (int i = tid; i < p.words; i += kSortThreads)
                if (bits[i]) atomicOr(p.present + i, bits[i]);
        }
        // the next pass reads what all blocks wrote, and writes where this
        // one's totals are
        if (pass == p.passes - 1) return;
        if (blocks > 1) cluster_barrier();
        else __syncthreads();
    }
}

// -------------------------------------------------- gradient: what it writes

constexpr int kSumThreads = 256, kSumWarps = kSumThreads / 32, kTile = 256;
constexpr int kDirect = 1024;      // tokens that are added up without a sort at most

struct SumParams {
    const uint2 *sorted;
    const void *tokens;
    const char *dy;
    char *dtable;
    const uint32_t *present;
    float *partial;
    int64_t dy_stride, table_stride;   // bytes
    int64_t vocab;
    int64_t chunks, work_blocks;       // of the sums; the blocks behind them write zeros
    int32_t count, width, tiles;
    int32_t run;                       // sorted tokens of a warp, up to 64; 8 times that are a chunk
    int32_t words, zero_parts;         // 32 rows x 512 bytes each a warp
    int32_t first_word;                // those before are written already
    float scale;
    int32_t accumulate;
    int32_t zero_bytes;                // zeros are written in pieces of this
    int32_t wide;
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

// Rows of dy on their way at once: 32 registers a lane, one at least a piece.
template <typename T, int P>
__host__ __device__ constexpr int rows_ahead() {
    return elem_bytes<T>() == 2 && P > 1 ? 8 : 4;
}

// The lane's eight columns of U rows of dy, those of them below `n`.
template <typename T, int P, int ROWS>
struct RowsOf {
    static constexpr int N = 8 / P, U = ROWS;
    PieceOf<T, P> v[U][N];
    __device__ __forceinline__ void load(const SumParams &p, int tile, int lane, uint32_t place, int first, int n) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (first + u >= n) break;   // the same in every lane
            const char *row = p.dy + (int64_t)__shfl_sync(0xffffffffu, place, first + u) * p.dy_stride;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int col = tile * kTile + (i * 32 + lane) * P;
                v[u][i].raw = {};
                using Whole = decltype(v[u][i].raw);
                if (col < p.width) v[u][i].raw = *reinterpret_cast<const Whole *>(row + (int64_t)col * elem_bytes<T>());
            }
        }
    }
    __device__ __forceinline__ void add(int u, float (&sum)[8]) const {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int k = 0; k < P; ++k) sum[i * P + k] += widened(v[u][i].e[k]);
    }
};

// Zeros in the rows of a word of presence bits that no token has.
template <typename TG>
__device__ __forceinline__ void zero_item(const SumParams &p, int64_t word, int part, uint32_t present, int lane) {
    const int64_t row = word * 32, rest = p.vocab - row;
    zero_rows(p.dtable + row * p.table_stride, p.table_stride, rest < 32 ? (int)rest : 32, part, present,
              p.width * elem_bytes<TG>(), p.zero_bytes, lane);
}

// -------------------------------------------- gradient: sums of sorted runs
// A block takes a chunk of sorted tokens and 256 columns, a warp an eighth of
// the chunk: a lane's eight sums stay in registers while it walks the rows of
// dy, the next U of them on their way.  A run of equal ids within a warp's part
// is written out; parts of runs that cross warps meet in shared memory, and
// those that cross chunks in the workspace, where embed_join_kernel adds them
// up.  HBM bounds it (with the sort, bf16 16384 x 4096 onto fp32 32768 rows 104
// us, 668 MB at 6.4 TB/s) until rows are short and many: 65536 x 768 onto bf16
// 50257 rows 47 us, of which the sort 17.  Slots 2 c and 2 c + 1 of the workspace:
// the part of a run that chunk c did not begin, and of one that it did.

__device__ __forceinline__ float4 *partial_slot(const SumParams &p, int64_t slot, int tile, int lane) {
    return reinterpret_cast<float4 *>(p.partial + (slot * p.tiles + tile) * kTile) + lane;
}
__device__ __forceinline__ void put8(float4 *to, const float (&s)[8]) {
    to[0] = make_float4(s[0], s[1], s[2], s[3]);
    to[32] = make_float4(s[4], s[5], s[6], s[7]);
}
__device__ __forceinline__ void add8(const float4 &a, const float4 &b, float (&s)[8]) {
    s[0] += a.x, s[1] += a.y, s[2] += a.z, s[3] += a.w;
    s[4] += b.x, s[5] += b.y, s[6] += b.z, s[7] += b.w;
}

template <typename T, typename TG, int P>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const SumParams p) {
    __shared__ float4 head[kSumWarps][64], tail[kSumWarps][64];
    __shared__ bool head_ends[kSumWarps], has_tail[kSumWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    if ((int64_t)blockIdx.x >= p.work_blocks) {
        const int64_t item = ((int64_t)blockIdx.x - p.work_blocks) * kSumWarps + warp;
        const int64_t word = p.first_word + item / p.zero_parts;
        if (word < p.words) zero_item<TG>(p, word, (int)(item % p.zero_parts), p.present[word], lane);
        return;
    }
    const int64_t chunk = blockIdx.x / p.tiles;
    const int tile = (int)(blockIdx.x - chunk * p.tiles);
    const int64_t first = (chunk * kSumWarps + warp) * p.run;
    const uint32_t none = (uint32_t)p.vocab;
    auto token = [&](int i) {
        return i < p.run && first + i < p.count ? p.sorted[first + i] : make_uint2(none, 0);
    };
    uint2 e = token(lane);
    const uint2 second = token(32 + lane);   // a warp has up to 64
    const uint32_t before = first > 0 && first <= p.count ? p.sorted[first - 1].x : ~0u;
    const uint32_t behind = first + p.run < p.count ? p.sorted[first + p.run].x : none;
    const uint32_t first_id = __shfl_sync(0xffffffffu, e.x, 0);
    bool began = first_id != before;   // this run, here
    bool goes_on = false, ended = false;
    uint32_t last_id = none;
    float sum[8] = {};
    constexpr int U = rows_ahead<T, P>();
    RowsOf<T, P, U> rows;
    for (int left = p.run;;) {
        const uint32_t after = left > 32 ? __shfl_sync(0xffffffffu, second.x, 0) : behind;
        uint32_t next = __shfl_down_sync(0xffffffffu, e.x, 1);
        if (lane == (left < 32 ? left : 32) - 1) next = after;
        const uint32_t ends = __ballot_sync(0xffffffffu, e.x < none && e.x != next);
        const int n = __popc(__ballot_sync(0xffffffffu, e.x < none));   // valid ones come first
        if (n == 0) break;
        for (int j = 0; j < n; j += U) {
            rows.load(p, tile, lane, e.y, j, n);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (j + u >= n) break;
                rows.add(u, sum);
                if (ends >> (j + u) & 1) {
                    const uint32_t id = __shfl_sync(0xffffffffu, e.x, j + u);
                    if (began) write_row<TG, P>(p, id, tile, lane, sum);
                    else put8(&head[warp][lane], sum);
                    began = true;
#pragma unroll
                    for (int k = 0; k < 8; ++k) sum[k] = 0.f;
                }
            }
        }
        goes_on = !(ends >> (n - 1) & 1);
        ended |= ends != 0;
        last_id = __shfl_sync(0xffffffffu, e.x, n - 1);
        left -= 32;
        if (left <= 0) break;
        e = second;
    }
    if (goes_on) put8(began ? &tail[warp][lane] : &head[warp][lane], sum);
    if (lane == 0) {
        head_ends[warp] = ended;
        has_tail[warp] = goes_on && began;
    }
    __syncthreads();
    // The parts of a run that crosses warps, in their order, by the warp that
    // began it; of one that began before the chunk, by the first.
    auto follow = [&](int w, uint32_t id, int64_t slot, bool ended) {
        for (; !ended && ++w < kSumWarps;) {
            add8(head[w][lane], head[w][lane + 32], sum);
            ended = head_ends[w];
        }
        if (ended && id != none) write_row<TG, P>(p, id, tile, lane, sum);
        else put8(partial_slot(p, slot, tile, lane), sum);
    };
    if (warp == 0 && first_id < none && first_id == before) {
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] = 0.f;
        add8(head[0][lane], head[0][lane + 32], sum);
        follow(0, none, 2 * chunk, head_ends[0]);
    }
    if (has_tail[warp]) {
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] = 0.f;
        add8(tail[warp][lane], tail[warp][lane + 32], sum);
        follow(warp, last_id, 2 * chunk + 1, false);
    }
}

// Runs that go on behind the chunk that began them: its part and the following
// chunks', in their order; a tile a warp, or eight warps side by side where
// the run is long.
constexpr int kLongRun = 64;   // chunks from which on a run is one

template <typename TG, int P>
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(const SumParams p) {
    constexpr int U = 8;
    __shared__ float4 part[kSumWarps][64];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t chunk = blockIdx.x, size = (int64_t)kSumWarps * p.run;
    const int64_t last = (chunk + 1) * size - 1;      // there is a chunk behind this one
    // What follows reads the sorted tokens alone, from L2.  They are complete:
    // this kernel starts once every block of the sums has let it, which each does
    // behind its own wait for the sort.  The sums themselves are waited for below.
    auto id_at = [&](int64_t i) { return __ldcg(&p.sorted[i].x); };
    const uint32_t id = id_at(last), then = id_at(last + 1);
    const uint32_t first = id_at(chunk * size), before = chunk > 0 ? id_at(chunk * size - 1) : ~0u;
    if (id >= (uint32_t)p.vocab || then != id || (first == id && before == id)) {
        pdl_wait_for_inputs();
        return;
    }
    // chunks behind this one that hold more of the run
    int64_t more = 1;
    for (;;) {
        const int64_t at = last + (more + lane) * size;   // the last token of that chunk
        const bool on = at + 1 < p.count && id_at(at) == id && id_at(at + 1) == id;
        const uint32_t not_on = ~__ballot_sync(0xffffffffu, on);
        if (not_on) {
            more += __ffs(not_on) - 1;
            break;
        }
        more += 32;
    }
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    // parts from .. to - 1: slot 2 chunk + 1, then 2 (chunk + s)
    auto parts = [&](int tile, int64_t from, int64_t to, float (&sum)[8]) {
        for (int64_t s = from; s < to; s += U) {
            float4 a[U], b[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                a[u] = b[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (s + u < to) {
                    const float4 *at = partial_slot(p, s + u == 0 ? 2 * chunk + 1 : 2 * (chunk + s + u), tile, lane);
                    a[u] = at[0];
                    b[u] = at[32];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) add8(a[u], b[u], sum);
        }
    };
    if (more < kLongRun) {
        for (int tile = warp; tile < p.tiles; tile += kSumWarps) {
            float sum[8] = {};
            parts(tile, 0, more + 1, sum);
            write_row<TG, P>(p, id, tile, lane, sum);
        }
        return;
    }
    const int64_t each = (more + kSumWarps) / kSumWarps;
    const int64_t from = warp * each, to = from + each < more + 1 ? from + each : more + 1;
    for (int tile = 0; tile < p.tiles; ++tile) {
        float sum[8] = {};
        parts(tile, from, to, sum);
        put8(&part[warp][lane], sum);
        __syncthreads();
        if (warp == tile % kSumWarps) {
            float all[8] = {};
#pragma unroll
            for (int w = 0; w < kSumWarps; ++w) add8(part[w][lane], part[w][lane + 32], all);
            write_row<TG, P>(p, id, tile, lane, all);
        }
        __syncthreads();
    }
}

// ------------------------------------------------- gradient: few tokens
// Without a sort: every block has all the ids in shared memory, a warp takes a
// place and 256 columns.  The first place of an id adds its row up: the warp
// finds the others by comparing 32 ids at a time, and adds their rows in their
// order; of more than 8, eight warps take an eighth of the places each.  A
// block's places are far apart: common ids come early, and eight long rows in
// one block would follow one another.  Latency bounds it: bf16 onto 8192 rows, 64
// x 1024 5.2 us, 256 x 1024 6.1, of which the zeros' 16 MB are 2.5.
constexpr int kDirectAlone = 8;

template <typename T, typename TG, int P>
__global__ void __launch_bounds__(kSumThreads, elem_bytes<T>() == 4 ? 4 : 1) embed_direct_kernel(const SumParams p) {
    __shared__ uint32_t ids[kDirect];
    __shared__ uint32_t list[kSumWarps][32];
    __shared__ float4 part[kSumWarps][64];
    __shared__ int many[kSumWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t none = (uint32_t)p.vocab;
    const int padded = (p.count + 31) / 32 * 32;
    pdl_wait_for_inputs();
    pdl_allow_dependents();
    for (int i = threadIdx.x; i < padded; i += kSumThreads) {
        const int64_t id = i < p.count ? token_at(p.tokens, p.wide, i) : -1;
        ids[i] = (uint64_t)id < (uint64_t)p.vocab ? (uint32_t)id : none;
    }
    __syncthreads();
    if ((int64_t)blockIdx.x >= p.work_blocks) {
        const int64_t item = ((int64_t)blockIdx.x - p.work_blocks) * kSumWarps + warp, word = item / p.zero_parts;
        if (word >= p.words) return;
        uint32_t present = 0;
        for (int i = lane; i < padded; i += 32)
            if ((int64_t)(ids[i] >> 5) == word) present |= 1u << (ids[i] & 31);
        zero_item<TG>(p, word, (int)(item % p.zero_parts), __reduce_or_sync(0xffffffffu, present), lane);
        return;
    }
    const int group = (int)(blockIdx.x / p.tiles), tile = (int)(blockIdx.x - (int64_t)group * p.tiles);
    const int groups = (int)p.chunks, place = warp * groups + group;
    const uint32_t id = place < p.count ? ids[place] : none;
    // the other places of the id, if this is the first
    int n = 0;
    if (id != none)
        for (int i = 0; i < padded; i += 32) {
            const uint32_t same = __ballot_sync(0xffffffffu, ids[i + lane] == id);
            if (i + __ffs(same) - 1 < place && same) {
                n = 0;
                break;
            }
            const int at = n + __popc(same & ((1u << lane) - 1));
            if ((same >> lane & 1) && at < 32) list[warp][at] = i + lane;
            n += __popc(same);
        }
    if (lane == 0) many[warp] = n;
    constexpr int U = rows_ahead<T, P>();
    RowsOf<T, P, U> rows;
    auto add_list = [&](int of, float (&sum)[8]) {
        __syncwarp();
        const uint32_t places = lane < of ? list[warp][lane] : 0;
        for (int j = 0; j < of; j += U) {
            rows.load(p, tile, lane, places, j, of);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j + u < of) rows.add(u, sum);
        }
        __syncwarp();
    };
    if (n > 0 && n <= kDirectAlone) {
        float sum[8] = {};
        add_list(n, sum);
        write_row<TG, P>(p, id, tile, lane, sum);
    }
    __syncthreads();
    for (int w = 0; w < kSumWarps; ++w) {
        if (many[w] <= kDirectAlone) continue;                       // the same in every warp
        const uint32_t of = ids[w * groups + group];
        const int each = (padded / 32 + kSumWarps - 1) / kSumWarps * 32;
        float sum[8] = {};
        int held = 0;
        for (int i = warp * each; i < (warp + 1) * each && i < padded; i += 32) {
            const uint32_t same = __ballot_sync(0xffffffffu, ids[i + lane] == of);
            if (held + __popc(same) > 32) {
                add_list(held, sum);
                held = 0;
            }
            if (same >> lane & 1) list[warp][held + __popc(same & ((1u << lane) - 1))] = i + lane;
            held += __popc(same);
        }
        add_list(held, sum);
        put8(&part[warp][lane], sum);
        __syncthreads();
        if (warp == w) {
            float all[8] = {};
#pragma unroll
            for (int v = 0; v < kSumWarps; ++v) add8(part[v][lane], part[v][lane + 32], all);
            write_row<TG, P>(p, of, tile, lane, all);
        }
        __syncthreads();
    }
}

}  // namespace rrn
