// rope_ragged.cuh -- the rotary kernels for heads whose pairs do not fall on
// 16-byte pieces (a rotated part of 20 of 80 elements, of 50 of 128), while
// the heads themselves do.
//
// The work layout, tables and arithmetic are rope_kernels.cuh's, with units of
// VE pairs of which a part's last one may be short.  What differs is how a
// lane comes by its unit's elements: a warp moves the heads of a head
// iteration, which stand one after another in memory, to and from an image of
// them in its own shared memory, 16 bytes a lane at a time, and picks a
// unit's elements out of the image wherever they stand.  With pieces of 4 or
// 2 bytes straight from global memory the same heads took two to four times as
// long (bf16 8192 tokens x 40 heads of 128, 50 elements of them rotated: 154
// us, 76 here; the gradient 379, 109).  What bounds it is the picking: lanes
// read words 16 bytes apart, four to a bank.
#pragma once

#include "rope_kernels.cuh"

namespace rrn {

constexpr int kRagImage = 1024;   // bytes of a warp's heads: 32 lanes of 2 VE elements
// Shared memory: the tables of rope_kernels.cuh, then an image a warp (two for
// the gradient); a run's last word may reach two bytes past the last image.
constexpr int kRagSmemBytes = kRopeSmemBytes + 2 * kRopeMaxWarps * kRagImage + 16;

// A lane's unit: where its two runs of elements start in a head, and how many
// pairs it has.
template <int VE, bool IL>
struct RagUnit {
    int unit, a, b, pairs;
    bool act, rot;
    __device__ __forceinline__ void set(const RopeParams &p, int t, int group) {
        act = t < p.units && group < p.heads_a_warp;
        unit = act ? t : 0;
        rot = unit < p.rot_units;
        const int half = p.head_dim / 2 - p.R;
        const int first = rot ? unit * VE : (unit - p.rot_units) * VE;   // pair, within its part
        const int left = (rot ? p.R : half) - first;
        pairs = !act ? 0 : left < VE ? left : VE;
        const int part = rot ? 0 : 2 * p.R;
        if (IL) {
            a = part + 2 * first;
            b = a + VE;
        } else {
            a = part + first;
            b = a + (rot ? p.R : half);
        }
    }
    // Elements of the runs that exist.
    __device__ __forceinline__ int in_a() const { return IL ? (2 * pairs < VE ? 2 * pairs : VE) : pairs; }
    __device__ __forceinline__ int in_b() const { return IL ? (2 * pairs > VE ? 2 * pairs - VE : 0) : pairs; }
};

// A run of `n` of VE elements between the image and fp32 registers (0 past
// them).  bf16 moves two elements at a time where they share a word; from an
// odd element on the run's ends are halves of words (what else is in the words
// read there is dropped, and not written).
template <typename T, int VE>
__device__ __forceinline__ void take_run(const unsigned char *img, int first, int n, float *e) {
    if constexpr (sizeof(typename T::storage) == 4) {
        const float *p = reinterpret_cast<const float *>(img) + first;
#pragma unroll
        for (int j = 0; j < VE; ++j) e[j] = j < n ? p[j] : 0.f;
    } else {
        const uint32_t *p = reinterpret_cast<const uint32_t *>(img) + first / 2;
        if (first & 1) {
            float last = bf16_hi(p[0]);
#pragma unroll
            for (int j = 0; j < VE; j += 2) {
                const uint32_t u = j + 1 < n ? p[j / 2 + 1] : 0u;
                e[j] = j < n ? last : 0.f;
                e[j + 1] = j + 1 < n ? bf16_lo(u) : 0.f;
                last = bf16_hi(u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < VE; j += 2) {
                const uint32_t u = j < n ? p[j / 2] : 0u;
                e[j] = bf16_lo(u);
                e[j + 1] = j + 1 < n ? bf16_hi(u) : 0.f;
            }
        }
    }
}
template <typename T, int VE>
__device__ __forceinline__ void put_run(unsigned char *img, int first, int n, const float *e) {
    if constexpr (sizeof(typename T::storage) == 4) {
        float *p = reinterpret_cast<float *>(img) + first;
#pragma unroll
        for (int j = 0; j < VE; ++j)
            if (j < n) p[j] = e[j];
    } else {
        uint16_t *p = reinterpret_cast<uint16_t *>(img) + first;
        const int lone = first & 1;   // elements before the first whole word
        if (lone && n > 0) p[0] = (uint16_t)pack_bf16x2(e[0], 0.f);
#pragma unroll
        for (int j = 0; j < VE; j += 2) {
            const int k = j + lone;   // of this word, within the run
            const float lo = lone ? e[j + 1] : e[j], hi = lone ? (j + 2 < VE ? e[j + 2] : 0.f) : e[j + 1];
            if (k + 1 < n) *reinterpret_cast<uint32_t *>(p + k) = pack_bf16x2(lo, hi);
            else if (k < n) p[k] = (uint16_t)pack_bf16x2(lo, 0.f);
        }
    }
}
template <int VE>
__device__ __forceinline__ void put_codes(unsigned char *img, int first, int n, float inv, float scale, bool settle, const float *e) {
    if (settle) {
#pragma unroll
        for (int j = 0; j < VE; ++j)
            if (j < n) img[first + j] = e4m3_of(settle_quotient(e[j] * inv, e[j], scale));
    } else {
#pragma unroll
        for (int j = 0; j < VE; ++j)
            if (j < n) img[first + j] = e4m3_of(e[j] * inv);
    }
}

// The factors of a unit applied to its runs: times the weights, turned.
template <int VE, bool IL, int N>
__device__ __forceinline__ void rag_weigh(const float *unit, float (&e)[2 * VE]) {
#pragma unroll
    for (int q = 0; q < VE; q += N) {
        float f[N], g[N];
        read_table<N>(unit + table_at<VE>(0, q), f);
        read_table<N>(unit + kRopeTable + table_at<VE>(0, q), g);
        run_times<N>(e + run_a<VE, IL>(q), f);
        run_times<N>(e + run_b<VE, IL>(q), g);
    }
}
template <int VE, bool IL, bool BACK, int N>
__device__ __forceinline__ void rag_turn(const float *unit, float (&e)[2 * VE]) {
#pragma unroll
    for (int q = 0; q < VE; q += N) {
        float f[N], g[N];
        read_table<N>(unit + table_at<VE>(0, q), f);
        read_table<N>(unit + kRopeTable + table_at<VE>(0, q), g);
        turn_runs<IL, BACK, N>(e + run_a<VE, IL>(q), e + run_b<VE, IL>(q), f, g);
    }
}

// Places of short units that no pair fills hold zeros, so that they add
// nothing to a sum; every other place is written before it is read.
__device__ __forceinline__ void clear_tables(float *wsm) {
    for (int i = threadIdx.x; i < 4 * kRopeTable + 2 * kRopeMaxWarps * 2 * kRopeTable; i += blockDim.x) wsm[i] = 0.f;
}

template <typename T, int VE, bool IL, int MODE>
__global__ void __launch_bounds__(32 * kRopeMaxWarps, 4) rope_ragged_kernel(const RopeParams p) {
    using P = Piece<T, VE>;
    using Raw = typename P::Raw;
    constexpr int S = (int)sizeof(typename T::storage);
    constexpr int N = pairs_at_once(VE);
    constexpr bool APPEND = MODE != kRopePlain;
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int kLookUps = 8 * kRopeMaxWarps;
    __shared__ int64_t rows[APPEND ? kLookUps : 1], indices[APPEND ? kLookUps : 1];
    uint64_t *frac = reinterpret_cast<uint64_t *>(smem);
    float *wsm = reinterpret_cast<float *>(smem + 8 * kRopeTable);
    float *tiles = wsm + 4 * kRopeTable;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned char *image = smem + kRopeSmemBytes + warp * kRagImage;

    const int G = p.lanes, group = lane / G, t = lane - group * G, hpw = p.heads_a_warp;
    const int heads = p.q_heads + p.k_heads + p.v_heads, turned = p.q_heads + p.k_heads;
    const uint32_t head_bytes = (uint32_t)(p.head_dim * S);
    const int head_chunks = p.head_dim / VE;   // 16 bytes each
    RagUnit<VE, IL> my;
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
    int64_t known = jobs.first;
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
    clear_tables(wsm);
    __syncthreads();

    bool prepared = false;
    int buf = 0;
    for (int64_t base = jobs.first; base < jobs.last; base += p.tile, buf ^= 1) {
        const int n = jobs.last - base < p.tile ? (int)(jobs.last - base) : p.tile;
        const int64_t token0 = p.slices > 1 ? base / p.slices : base;
        const int h0 = p.slices > 1 ? (int)(base - token0 * p.slices) * p.iters * hpw : 0;
        const char *tx = static_cast<const char *>(p.x) + token0 * p.x_stride;
        char *ty = static_cast<char *>(p.y) + token0 * p.y_stride;
        Tile at{0, warp};
        at.settle(n, p.iters);
        Raw next[2];   // the lane's chunks of the next heads
        auto chunks_at = [&]() {   // of the heads of `at`
            const int left = heads - (h0 + at.i * hpw);
            return (left < hpw ? left : hpw) * head_chunks;
        };
        auto load = [&]() {
            const char *src = tx + ((uint32_t)at.j * (uint32_t)p.x_stride + (uint32_t)(h0 + at.i * hpw) * head_bytes);
            const int n16 = chunks_at();
#pragma unroll
            for (int l = 0; l < 2; ++l)
                if (lane + 32 * l < n16) next[l] = P::load(src + (lane + 32 * l) * 16);
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
            const int job = at.j, first = h0 + at.i * hpw, h = first + group, n16 = chunks_at();
#pragma unroll
            for (int l = 0; l < 2; ++l)
                if (lane + 32 * l < n16) P::give(image + (lane + 32 * l) * 16, next[l]);
            at.i += kRopeMaxWarps;
            at.settle(n, p.iters);
            if (at.j < n) load();   // the next heads are on their way
            __syncwarp();
            const bool mine = h < heads && my.act;
            const bool key = h >= p.q_heads, value = APPEND && h >= turned;
            unsigned char *img = image + (mine ? group : 0) * head_bytes;
            float e[2 * VE];
            take_run<T, VE>(img, my.a, mine ? my.in_a() : 0, e);
            take_run<T, VE>(img, my.b, mine ? my.in_b() : 0, e + VE);
            float r = 1.f;
            if (p.norm) {
                float2 acc = make_float2(0.f, 0.f);
                run_dot<2 * VE>(acc, e, e);
                float sum[1] = {acc.x + acc.y};
                lanes_sum<1>(sum, G, t, lane);
                r = rsqrtf(fmaf(sum[0], p.inv_dim, p.eps));
            }
            if (!value) {
                const int place = table_at<VE>(my.unit, 0);
                if (p.norm) run_scale<2 * VE>(e, r);
                rag_weigh<VE, IL, N>(wsm + (key ? 2 * kRopeTable : 0) + place, e);
                if (my.rot)
                    rag_turn<VE, IL, false, N>(tiles + (buf * kRopeMaxWarps + job) * 2 * kRopeTable + place, e);
            }
            __syncwarp();   // the image is read: it takes the results
            if (mine) {
                if (MODE == kRopeAppendE4m3 && key) {
                    const float inv = value ? p.v_inv : p.k_inv, scale = value ? p.v_scale : p.k_scale;
                    put_codes<VE>(img, my.a, my.in_a(), inv, scale, p.settle, e);
                    put_codes<VE>(img, my.b, my.in_b(), inv, scale, p.settle, e + VE);
                } else {
                    put_run<T, VE>(img, my.a, my.in_a(), e);
                    put_run<T, VE>(img, my.b, my.in_b(), e + VE);
                }
            }
            __syncwarp();
            const int64_t row = APPEND ? rows[base - known + job] : 0;
            if (APPEND && row < 0 && h == p.q_heads && t == 0 && mine && p.dropped != nullptr) atomicAdd(p.dropped, 1);
            char *yr = ty + (uint32_t)job * (uint32_t)p.y_stride;
#pragma unroll
            for (int l = 0; l < 2; ++l) {
                const int c = lane + 32 * l;
                if (c < n16) {
                    const int own = c / head_chunks, g = first + own, in = c - own * head_chunks;
                    const unsigned char *from = image + own * head_bytes;
                    if (!APPEND || g < p.q_heads) {
                        *reinterpret_cast<uint4 *>(yr + ((uint32_t)g * head_bytes + in * 16)) =
                            *reinterpret_cast<const uint4 *>(from + in * 16);
                    } else if (row >= 0) {
                        const bool v = g >= turned;
                        char *dst = static_cast<char *>(v ? p.v_cache : p.k_cache) + row +
                                    (int64_t)(g - (v ? turned : p.q_heads)) * p.head_stride;
                        if constexpr (MODE != kRopeAppendE4m3)
                            *reinterpret_cast<uint4 *>(dst + in * 16) = *reinterpret_cast<const uint4 *>(from + in * 16);
                        else if constexpr (VE == 8)
                            *reinterpret_cast<uint2 *>(dst + in * 8) = *reinterpret_cast<const uint2 *>(from + in * 8);
                        else
                            *reinterpret_cast<uint32_t *>(dst + in * 4) =
                                *reinterpret_cast<const uint32_t *>(from + in * 4);
                    }
                }
            }
            __syncwarp();   // the image is written out before the next heads come in
        }
    }
}

// The gradient (see rope_bwd_kernel): an image for dy, which takes dx, and one
// for x.
template <typename T, int VE, bool IL, bool NORM>
__global__ void __launch_bounds__(32 * kRopeMaxWarps, 2) rope_ragged_bwd_kernel(const RopeParams p) {
    using P = Piece<T, VE>;
    using Raw = typename P::Raw;
    constexpr int S = (int)sizeof(typename T::storage);
    constexpr int N = pairs_at_once(VE);
    extern __shared__ __align__(16) unsigned char smem[];
    uint64_t *frac = reinterpret_cast<uint64_t *>(smem);
    float *wsm = reinterpret_cast<float *>(smem + 8 * kRopeTable);
    float *tiles = wsm + 4 * kRopeTable;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned char *image_g = smem + kRopeSmemBytes + warp * 2 * kRagImage, *image_x = image_g + kRagImage;

    const int G = p.lanes, group = lane / G, t = lane - group * G, hpw = p.heads_a_warp;
    const uint32_t head_bytes = (uint32_t)(p.head_dim * S);
    const int head_chunks = p.head_dim / VE;
    RagUnit<VE, IL> my;
    my.set(p, t, group);
    const bool key = warp >= p.q_warps;
    const int heads = key ? p.k_heads : p.q_heads, iters = key ? p.iters_k : p.iters;
    const int mates = key ? kRopeMaxWarps - p.q_warps : p.q_warps;
    Jobs jobs;
    jobs.set(blockIdx.x, p.each, p.extra);
    const uint32_t head0 = key ? (uint32_t)p.q_heads * head_bytes : 0u;
    const float *w = wsm + (key ? 2 * kRopeTable : 0) + table_at<VE>(my.unit, 0);
    int64_t skip = 0;   // see rope_bwd_kernel
    int i0 = 0;
    if (p.slices > 1) {
        const uint32_t token = (uint32_t)jobs.first / (uint32_t)p.slices;
        i0 = (int)((uint32_t)jobs.first - token * (uint32_t)p.slices) * iters;
        skip = jobs.first - token;
    }

    pdl_wait_for_inputs();
    pdl_allow_dependents();
    clear_tables(wsm);
    __syncthreads();

    float gw[2 * VE];   // the weight's gradient
#pragma unroll
    for (int v = 0; v < 2 * VE; ++v) gw[v] = 0.f;
    int64_t pos = 0;
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
        Raw next_g[2], next_x[2];
        auto chunks_at = [&]() {
            const int left = heads - (i0 + at.i) * hpw;
            return (left < hpw ? left : hpw) * head_chunks;
        };
        auto load = [&]() {
            const uint32_t off = (uint32_t)((i0 + at.i) * hpw) * head_bytes;
            const char *gs = tg + ((uint32_t)at.j * (uint32_t)p.dy_stride + off);
            const char *xs = tx + ((uint32_t)at.j * (uint32_t)p.x_stride + off);
            const int n16 = chunks_at();
#pragma unroll
            for (int l = 0; l < 2; ++l)
                if (lane + 32 * l < n16) {
                    next_g[l] = P::load(gs + (lane + 32 * l) * 16);
                    if constexpr (NORM) next_x[l] = P::load(xs + (lane + 32 * l) * 16);
                }
        };
        if (at.j < n) load();
        if (!prepared) {
            if (base + warp < jobs.last) pos = lane_position(p, lane, token0 + warp);
            make_fractions<VE>(p, frac);
            if constexpr (NORM) make_weights<T, VE, IL>(p, wsm);
            __syncthreads();
            prepared = true;
        }
        if (warp < n)
            make_angles<VE, IL>(p, frac, tiles + (buf * kRopeMaxWarps + warp) * 2 * kRopeTable, lane, pos);
        if (base + p.tile + warp < jobs.last) pos = lane_position(p, lane, token0 + p.tile + warp);
        __syncthreads();   // two buffers: the tile before this one may still be read
        while (at.j < n) {
            const int job = at.j, first = (i0 + at.i) * hpw, h = first + group, n16 = chunks_at();
#pragma unroll
            for (int l = 0; l < 2; ++l)
                if (lane + 32 * l < n16) {
                    P::give(image_g + (lane + 32 * l) * 16, next_g[l]);
                    if constexpr (NORM) P::give(image_x + (lane + 32 * l) * 16, next_x[l]);
                }
            at.i += mates;
            at.settle(n, iters);
            if (at.j < n) load();
            __syncwarp();
            const bool mine = h < heads && my.act;
            const int na = mine ? my.in_a() : 0, nb = mine ? my.in_b() : 0;
            const uint32_t at_head = (mine ? group : 0) * head_bytes;
            float g[2 * VE];
            take_run<T, VE>(image_g + at_head, my.a, na, g);
            take_run<T, VE>(image_g + at_head, my.b, nb, g + VE);
            if (my.rot)
                rag_turn<VE, IL, true, N>(
                    tiles + (buf * kRopeMaxWarps + job) * 2 * kRopeTable + table_at<VE>(my.unit, 0), g);
            if constexpr (NORM) {
                float x[2 * VE], v[2 * VE];
                take_run<T, VE>(image_x + at_head, my.a, na, x);
                take_run<T, VE>(image_x + at_head, my.b, nb, x + VE);
#pragma unroll
                for (int j = 0; j < 2 * VE; ++j) v[j] = g[j];
                rag_weigh<VE, IL, N>(w, v);
                float2 sq = make_float2(0.f, 0.f), dot = sq;
                run_dot<2 * VE>(sq, x, x);
                run_dot<2 * VE>(dot, v, x);
                float sums[2] = {sq.x + sq.y, dot.x + dot.y};
                lanes_sum<2>(sums, G, t, lane);
                const float r = rsqrtf(fmaf(sums[0], p.inv_dim, p.eps));
                const float mean = -(sums[1] * p.inv_dim) * r;
                run_scale<2 * VE>(x, r);
                if (mine) run_fma<2 * VE>(gw, g, x);   // a lane without a head adds nothing, whatever eps is
                float mm[2 * VE];
#pragma unroll
                for (int j = 0; j < 2 * VE; ++j) mm[j] = mean, g[j] = v[j];
                run_fma<2 * VE>(g, x, mm);
                run_scale<2 * VE>(g, r);
            }
            __syncwarp();
            if (mine) {
                put_run<T, VE>(image_g + at_head, my.a, na, g);
                put_run<T, VE>(image_g + at_head, my.b, nb, g + VE);
            }
            __syncwarp();
            char *dst = ty + ((uint32_t)job * (uint32_t)p.y_stride + (uint32_t)first * head_bytes);
#pragma unroll
            for (int l = 0; l < 2; ++l)
                if (lane + 32 * l < n16)
                    *reinterpret_cast<uint4 *>(dst + (lane + 32 * l) * 16) =
                        *reinterpret_cast<const uint4 *>(image_g + (lane + 32 * l) * 16);
            __syncwarp();
        }
    }
    if constexpr (NORM) {
        if (p.partial != nullptr) {
            // the heads side by side in the warp, then the block's warps of the kind
#pragma unroll
            for (int v = 0; v < 2 * VE; ++v) {
                const float own = gw[v];
                for (int g = 1; g < hpw; ++g) gw[v] += __shfl_sync(0xffffffffu, own, (lane + g * G) & 31);
            }
            __syncthreads();   // the tables are read; their place takes the warps' sums [kRopeMaxWarps][D]
            if (group == 0 && my.act && heads > 0) {
                const int na = my.in_a(), nb = my.in_b();
#pragma unroll
                for (int v = 0; v < VE; ++v) {
                    if (v < na) wsm[warp * p.head_dim + my.a + v] = gw[v];
                    if (v < nb) wsm[warp * p.head_dim + my.b + v] = gw[VE + v];
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
