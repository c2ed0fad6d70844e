// rope_api.cu -- entry points of the Q+K head norm with rotary positions, its
// gradient, and the append to a paged cache (declared in include/rmsnorm.h):
// argument checks, the choice of a kernel and its grid, the launch.
#include <climits>
#include <cmath>
#include <cstring>

#include "launch_util.h"
#include "rope_kernels.cuh"
#include "rope_ragged.cuh"
#include "rope_pick.h"

namespace {

using rrn::div_up;

// Blocks of the gradient kernel at most (its workspace is sized for them).
constexpr int kBwdMaxBlocks = 1024;

int check_rope(const rmsnorm_rope_t *rope, int64_t tokens, int64_t head_dim, bool need_positions) {
    if (rope == nullptr) return RMSNORM_EINVAL;
    if (rope->rot_dim < 2 || rope->rot_dim > head_dim || rope->rot_dim % 2 != 0) return RMSNORM_EINVAL;
    if (rope->axes < 1 || rope->axes > rrn::kRopeMaxAxes) return RMSNORM_EINVAL;
    if (rope->interleaved != 0 && rope->interleaved != 1) return RMSNORM_EINVAL;
    if (rope->position_bytes != 4 && rope->position_bytes != 8) return RMSNORM_EINVAL;
    int64_t pairs = 0;
    for (int a = 0; a < rope->axes; ++a) {
        if (rope->section[a] < 0) return RMSNORM_EINVAL;
        pairs += rope->section[a];
    }
    if (pairs != rope->rot_dim / 2) return RMSNORM_EINVAL;
    if (rope->axes > 1 && (rope->position_stride < tokens || rope->position_stride > INT64_MAX / 64)) return RMSNORM_EINVAL;
    if (tokens > 0) {
        if (rope->inv_freq == nullptr || !rrn::on_boundary(rope->inv_freq, 4)) return RMSNORM_EINVAL;
        if (rope->positions == nullptr ? need_positions : !rrn::on_boundary(rope->positions, rope->position_bytes))
            return RMSNORM_EINVAL;
    }
    return RMSNORM_OK;
}

// What every rotary entry point checks and fills in.
int make_rope(int64_t tokens, int64_t x_stride, int32_t q_heads, int32_t k_heads, int32_t v_heads, int64_t head_dim,
              const void *q_w, const void *k_w, float w_bias, float eps, int norm, const rmsnorm_rope_t *rope,
              bool need_positions, int dtype, rrn::RopeParams *p) {
    if (dtype != RMSNORM_F32 && dtype != RMSNORM_BF16) return RMSNORM_EINVAL;
    if (tokens < 0 || head_dim <= 0 || head_dim % 2 != 0) return RMSNORM_EINVAL;
    if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(w_bias)) return RMSNORM_EINVAL;
    if (norm != 0 && norm != 1) return RMSNORM_EINVAL;
    if ((q_w == nullptr) != (k_w == nullptr)) return RMSNORM_EINVAL;
    if (w_bias != 0.f && q_w == nullptr) return RMSNORM_EINVAL;
    if (norm == 0 && q_w != nullptr) return RMSNORM_EINVAL;
    if (q_heads < 0 || k_heads < 0 || (int64_t)q_heads + k_heads < 1) return RMSNORM_EINVAL;
    const int64_t heads = (int64_t)q_heads + k_heads + v_heads;
    if (heads * head_dim > (1 << 28)) return RMSNORM_EUNSUPPORTED;   // a token row within 31 bits
    if (head_dim > rrn::kRopeMaxDim) return RMSNORM_EUNSUPPORTED;
    const int64_t s = rrn::size_of(dtype);
    if (x_stride < heads * head_dim || (tokens > 0 && tokens > INT64_MAX / 8 / x_stride / s)) return RMSNORM_EINVAL;
    const int st = check_rope(rope, tokens, head_dim, need_positions);
    if (st != RMSNORM_OK) return st;
    if (!rrn::on_boundary(q_w, s) || !rrn::on_boundary(k_w, s)) return RMSNORM_EINVAL;
    std::memset(p, 0, sizeof(*p));
    p->q_w = q_w;
    p->k_w = k_w;
    p->tokens = tokens;
    p->x_stride = x_stride * s;
    p->q_heads = q_heads;
    p->k_heads = k_heads;
    p->v_heads = v_heads;
    p->head_dim = (int32_t)head_dim;
    p->norm = norm;
    p->inv_dim = 1.f / (float)head_dim;
    p->eps = eps;
    p->w_bias = w_bias;
    p->pos = rope->positions;
    p->pos_stride = rope->axes > 1 ? rope->position_stride : 0;
    p->pos64 = rope->position_bytes == 8;
    p->axes = rope->axes;
    p->inv_freq = rope->inv_freq;
    p->R = rope->rot_dim / 2;
    int32_t at = 0;
    for (int a = 0; a < 3; ++a) {
        at += a < rope->axes ? rope->section[a] : 0;
        p->cut[a] = a + 1 < rope->axes ? at : p->R;
    }
    return RMSNORM_OK;
}

// A token stride (elements) of another tensor of the call.
bool stride_ok(int64_t stride, int64_t width, int64_t tokens, int64_t s) {
    return stride >= width && (tokens == 0 || tokens <= INT64_MAX / 8 / stride / s);
}

// The widest shape that the head's halves, and every address and stride of
// the call (all multiples of `unit` elements), allow; a head is held by as
// many lanes as it has units (32 at most), so that neighbouring lanes read
// neighbouring pieces and few lanes idle: fp32 heads of 80 (10 units, three
// heads a warp) 4099 tokens x 32 heads 17.9 us, 19.8 with 16 lanes a head.
int pick_shape(int dtype, int64_t unit, rrn::RopeParams *p) {
    const rrn::RopeShape *table = dtype == RMSNORM_BF16 ? rrn::kRopeShapesBf16 : rrn::kRopeShapesF32;
    const int tail = p->head_dim / 2 - p->R;
    for (int i = 0; i < rrn::kRopeShapes; ++i) {
        // Pairs that 16-byte pieces do not hold, nor (bf16) 8-byte ones: whole
        // heads through shared memory, where they come in 16-byte chunks.
        // Measured on GB300, 8192 tokens x 40 heads: bf16 heads of 80, 20 of
        // them rotated, 41.7 us that way, 78.8 in 4-byte pieces; bf16 heads of
        // 72 in 8-byte pieces 28.0 us, 36.7 that way; fp32 heads of 80 (4096
        // tokens) 33.8 us that way, 38.9 in 8-byte pieces.
        if (i == 2 && p->head_dim % table[0].ve == 0 && unit % table[0].ve == 0) {
            const int ve = table[0].ve, turned = (p->R + ve - 1) / ve, units = turned + (tail + ve - 1) / ve;
            if (units <= 32) {
                p->units = p->lanes = units;
                p->rot_units = turned;
                p->heads_a_warp = 32 / units;
                return rrn::kRopeRagged;
            }
        }
        const int ve = table[i].ve, units = p->head_dim / 2 / ve;
        if (p->R % ve != 0 || tail % ve != 0 || unit % ve != 0 || units > 32 * table[i].k) continue;
        p->units = units;
        p->rot_units = p->R / ve;
        p->lanes = units < 32 ? units : 32;
        p->heads_a_warp = 32 / p->lanes;
        return i;
    }
    return -1;   // unreachable: the last shape takes any head
}

// Largest power of two (at most 16) that divides every address and stride
// given, in elements of `s` bytes.  (The weights are read an element at a
// time, into tables, and have no part in it.)
struct Unit {
    uint64_t bits = 16;
    void at(const void *ptr, int64_t s) { bits |= (uint64_t)(reinterpret_cast<uintptr_t>(ptr) / (uintptr_t)s); }
    void step(int64_t elements) { bits |= (uint64_t)elements; }
    int64_t get() const { return (int64_t)(bits & (~bits + 1)); }
};

// Columns of the partial sums' rows.
int64_t partial_ld(int64_t head_dim) { return (head_dim + 3) / 4 * 4; }

// Whether every byte of a tile's token rows is within 31 bits of its first.
bool tile_reaches(int64_t a, int64_t b, int64_t c) {
    const int64_t most = INT32_MAX / rrn::kRopeMaxWarps;
    return a <= most && b <= most && c <= most;
}

// Scales of an 8-bit cache: within 2^-100 .. 2^100 (see settle_quotient).
bool scale_ok(float s) { return s >= 0x1p-100f && s <= 0x1p100f; }
bool power_of_two(float s) {
    int e;
    return std::frexp(s, &e) == 0.5f;
}

int whole_head(const rrn::RopeParams *p) { return 2 * p->R == p->head_dim ? p->head_dim : 0; }

const void *forward_kernel(int dtype, int shape, bool il, int mode, int whole) {
    const int ragged = mode == rrn::kRopeAppendSettled ? (int)rrn::kRopeAppendE4m3 : mode;
    if (shape == rrn::kRopeRagged)
        return dtype == RMSNORM_BF16 ? rrn::rope_ragged_bf16(il, ragged) : rrn::rope_ragged_f32(il, ragged);
    return dtype == RMSNORM_BF16 ? rrn::rope_fwd_bf16(shape, il, mode, whole)
                                 : rrn::rope_fwd_f32(shape, il, mode, whole);
}

const void *backward_kernel(int dtype, int shape, bool il, bool norm, int whole) {
    if (shape == rrn::kRopeRagged)
        return dtype == RMSNORM_BF16 ? rrn::rope_ragged_bwd_bf16(il, norm) : rrn::rope_ragged_bwd_f32(il, norm);
    return dtype == RMSNORM_BF16 ? rrn::rope_bwd_bf16(shape, il, norm, whole)
                                 : rrn::rope_bwd_f32(shape, il, norm, whole);
}

// Shared memory of a gradient block.
size_t backward_smem(int dtype, int shape, bool norm) {
    if (shape == rrn::kRopeRagged) return rrn::kRagSmemBytes;
    const rrn::RopeShape held = (dtype == RMSNORM_BF16 ? rrn::kRopeShapesBf16 : rrn::kRopeShapesF32)[shape];
    return (size_t)rrn::kRopeSmemBytes + rrn::rope_ring_bytes(held.ve * rrn::size_of(dtype), held.k, norm);
}

int launch_forward(rrn::RopeParams *p, int dtype, int64_t unit, bool il, int mode, rmsnorm_stream_t stream) {
    int dev = 0, sms = 0;
    int st = rrn::current_device_sms(&dev, &sms);
    if (st != RMSNORM_OK) return st;
    const int shape = pick_shape(dtype, unit, p);
    const void *fn = forward_kernel(dtype, shape, il, mode, whole_head(p));
    if (fn == nullptr) return RMSNORM_EINVAL;
    // A run of jobs for every resident block.  A job is a token's heads; with
    // fewer tokens than blocks it is a slice of them, one head iteration a
    // warp where that many blocks fit.
    const int64_t iters = div_up((int64_t)p->q_heads + p->k_heads + p->v_heads, p->heads_a_warp);
    const size_t smem = shape == rrn::kRopeRagged ? rrn::kRagSmemBytes : rrn::kRopeSmemBytes;
    int resident = 0;
    if (smem > rrn::kSmemUnasked && (st = rrn::allow_smem(dev, fn)) != RMSNORM_OK) return st;
    if ((st = rrn::resident_blocks(dev, fn, 32 * rrn::kRopeMaxWarps, smem, &resident)) != RMSNORM_OK) return st;
    const int64_t most = (int64_t)sms * resident;
    int64_t slices = 1;
    if (p->tokens < most) {
        slices = most / p->tokens;
        if (slices > div_up(iters, rrn::kRopeMaxWarps)) slices = div_up(iters, rrn::kRopeMaxWarps);
    }
    p->iters = (int32_t)div_up(iters, slices);
    p->slices = (int32_t)div_up(iters, p->iters);
    p->tile = p->slices > 1 || !tile_reaches(p->x_stride, p->y_stride, 0) ? 1 : rrn::kRopeMaxWarps;
    const int64_t jobs = p->tokens * p->slices;
    const int64_t blocks = jobs < most ? jobs : most;
    p->each = jobs / blocks;
    p->extra = jobs % blocks;
    void *argv[] = {p};
    return rrn::launch_kernel(fn, dim3((unsigned)blocks), 32 * rrn::kRopeMaxWarps, smem, stream, argv);
}

}  // namespace

extern "C" {

int rmsnorm_qk_rope_fwd(const void *x, void *y, int64_t tokens, int64_t x_token_stride, int64_t y_token_stride,
                        int32_t q_heads, int32_t k_heads, int64_t head_dim, const void *q_w, const void *k_w,
                        float weight_bias, float eps, int norm, const rmsnorm_rope_t *rope, int dtype,
                        rmsnorm_stream_t stream) {
    rrn::RopeParams p;
    int st = make_rope(tokens, x_token_stride, q_heads, k_heads, 0, head_dim, q_w, k_w, weight_bias, eps, norm, rope,
                       true, dtype, &p);
    if (st != RMSNORM_OK) return st;
    const int64_t s = rrn::size_of(dtype);
    if (!stride_ok(y_token_stride, ((int64_t)q_heads + k_heads) * head_dim, tokens, s)) return RMSNORM_EINVAL;
    if (tokens == 0) return RMSNORM_OK;
    if (x == nullptr || y == nullptr || !rrn::on_boundary(x, s) || !rrn::on_boundary(y, s)) return RMSNORM_EINVAL;
    if (x == y && x_token_stride != y_token_stride) return RMSNORM_EINVAL;
    p.x = x;
    p.y = y;
    p.y_stride = y_token_stride * s;
    Unit u;
    u.at(x, s), u.at(y, s);
    u.step(x_token_stride), u.step(y_token_stride);
    return launch_forward(&p, dtype, u.get(), rope->interleaved == 1, rrn::kRopePlain, stream);
}

int64_t rmsnorm_qk_rope_bwd_workspace_bytes(int64_t head_dim) {
    if (head_dim <= 0 || head_dim % 2 != 0) return RMSNORM_EINVAL;
    if (head_dim > rrn::kRopeMaxDim) return RMSNORM_EUNSUPPORTED;
    return (int64_t)kBwdMaxBlocks * 2 * partial_ld(head_dim) * (int64_t)sizeof(float);
}

int rmsnorm_qk_rope_bwd(const void *dy, const void *x, void *dx, int64_t tokens, int64_t dy_token_stride,
                        int64_t x_token_stride, int64_t dx_token_stride, int32_t q_heads, int32_t k_heads,
                        int64_t head_dim, const void *q_w, const void *k_w, void *dq_w, void *dk_w, float weight_bias,
                        float eps, int norm, const rmsnorm_rope_t *rope, int dtype, void *workspace,
                        uint64_t workspace_bytes, rmsnorm_stream_t stream) {
    rrn::RopeParams p;
    int st = make_rope(tokens, x_token_stride, q_heads, k_heads, 0, head_dim, q_w, k_w, weight_bias, eps, norm, rope,
                       true, dtype, &p);
    if (st != RMSNORM_OK) return st;
    const int64_t s = rrn::size_of(dtype), width = ((int64_t)q_heads + k_heads) * head_dim;
    if (!stride_ok(dy_token_stride, width, tokens, s) || !stride_ok(dx_token_stride, width, tokens, s))
        return RMSNORM_EINVAL;
    if ((dq_w == nullptr) != (dk_w == nullptr) || (dq_w != nullptr && q_w == nullptr)) return RMSNORM_EINVAL;
    if (!rrn::on_boundary(dq_w, s) || !rrn::on_boundary(dk_w, s)) return RMSNORM_EINVAL;
    if (dq_w != nullptr &&
        (workspace == nullptr || !rrn::on_boundary(workspace, 16) ||
         workspace_bytes < (uint64_t)rmsnorm_qk_rope_bwd_workspace_bytes(head_dim)))
        return RMSNORM_EINVAL;
    if (tokens > 0) {
        if (dy == nullptr || dx == nullptr || (norm == 1 && x == nullptr)) return RMSNORM_EINVAL;
        if (!rrn::on_boundary(dy, s) || !rrn::on_boundary(dx, s) || (norm == 1 && !rrn::on_boundary(x, s)))
            return RMSNORM_EINVAL;
        if ((dx == dy && dx_token_stride != dy_token_stride) ||
            (norm == 1 && dx == x && dx_token_stride != x_token_stride))
            return RMSNORM_EINVAL;
    }
    p.dy = dy;
    p.x = x;
    p.y = dx;
    p.dy_stride = dy_token_stride * s;
    p.y_stride = dx_token_stride * s;
    p.partial = static_cast<float *>(dq_w != nullptr ? workspace : nullptr);
    p.partial_ld = (int32_t)partial_ld(head_dim);
    int64_t blocks = 0;
    if (tokens > 0) {
        Unit u;
        u.at(dy, s), u.at(dx, s);
        u.step(dy_token_stride), u.step(dx_token_stride);
        if (norm == 1) u.at(x, s), u.step(x_token_stride);
        int dev = 0, sms = 0;
        if ((st = rrn::current_device_sms(&dev, &sms)) != RMSNORM_OK) return st;
        const int shape = pick_shape(dtype, u.get(), &p);
        const bool il = rope->interleaved == 1;
        const void *fn = backward_kernel(dtype, shape, il, norm == 1, whole_head(&p));
        if (fn == nullptr) return RMSNORM_EINVAL;
        const int64_t iters_q = div_up(q_heads, p.heads_a_warp), iters_k = div_up(k_heads, p.heads_a_warp);
        const size_t smem = backward_smem(dtype, shape, norm == 1);
        int resident = 0;
        if (smem > rrn::kSmemUnasked && (st = rrn::allow_smem(dev, fn)) != RMSNORM_OK) return st;
        if ((st = rrn::resident_blocks(dev, fn, 32 * rrn::kRopeMaxWarps, smem, &resident)) != RMSNORM_OK) return st;
        int64_t most = (int64_t)sms * resident;
        if (most > kBwdMaxBlocks) most = kBwdMaxBlocks;
        // fewer tokens than blocks: a token's heads in slices, one head
        // iteration a warp where that many blocks fit (2 tokens of 56 bf16
        // heads of 128, 10 elements turned: 10.3 -> 7.5 us)
        // With weights, up to two iterations a warp of a single cluster: it
        // adds the weights' gradients up itself.
        const bool alone = dq_w != nullptr && tokens * (iters_q + iters_k) <=
                                                  2 * rrn::kFinishBlocks * rrn::kRopeMaxWarps;
        if (alone && most > rrn::kFinishBlocks) most = rrn::kFinishBlocks;
        int64_t slices = 1;
        if (tokens < most) {
            slices = most / tokens;
            const int64_t enough = div_up(iters_q + iters_k, rrn::kRopeMaxWarps);
            if (slices > enough) slices = enough;
        }
        p.iters = (int32_t)div_up(iters_q, slices);
        p.iters_k = (int32_t)div_up(iters_k, slices);
        p.slices = (int32_t)slices;
        p.tile = slices == 1 && tile_reaches(p.dy_stride, p.y_stride, norm == 1 ? p.x_stride : 0) ? rrn::kRopeMaxWarps : 1;
        blocks = tokens * slices < most ? tokens * slices : most;
        p.each = tokens * slices / blocks;
        p.extra = tokens * slices % blocks;
        // the split of a block's warps that leaves the longer of the two kinds
        // the fewest head iterations a warp and tile
        int64_t best = INT64_MAX;
        for (int qw = q_heads > 0 ? 1 : 0; qw <= rrn::kRopeMaxWarps - (k_heads > 0 ? 1 : 0); ++qw) {
            const int64_t q_turns = q_heads > 0 ? div_up((int64_t)p.tile * p.iters, qw) : 0;
            const int64_t k_turns = k_heads > 0 ? div_up((int64_t)p.tile * p.iters_k, rrn::kRopeMaxWarps - qw) : 0;
            const int64_t turns = q_turns > k_turns ? q_turns : k_turns;
            if (turns < best) {
                best = turns;
                p.q_warps = qw;
            }
        }
        if (alone) p.dq_w = dq_w, p.dk_w = dk_w;
        void *argv[] = {&p};
        st = rrn::launch_kernel(fn, dim3((unsigned)blocks), 32 * rrn::kRopeMaxWarps, smem, stream, argv,
                                alone ? (int)blocks : 1);
        if (st != RMSNORM_OK || alone) return st;
    }
    if (dq_w == nullptr) return RMSNORM_OK;
    return rrn::launch_colsum(static_cast<const float *>(workspace), (int)blocks, (int)blocks, head_dim,
                              partial_ld(head_dim), dq_w, dk_w,
                              dtype, stream);
}

int rmsnorm_qkv_append(const void *x, void *q_out, int64_t tokens, int64_t x_token_stride, int64_t q_token_stride,
                       int32_t q_heads, int32_t kv_heads, int64_t head_dim, const void *q_w, const void *k_w,
                       float weight_bias, float eps, int norm, const rmsnorm_rope_t *rope,
                       const rmsnorm_paged_kv_t *kv, int dtype, rmsnorm_stream_t stream) {
    if (kv_heads < 1) return RMSNORM_EINVAL;
    rrn::RopeParams p;
    int st = make_rope(tokens, x_token_stride, q_heads, kv_heads, kv_heads, head_dim, q_w, k_w, weight_bias, eps, norm,
                       rope, false, dtype, &p);
    if (st != RMSNORM_OK) return st;
    const int64_t s = rrn::size_of(dtype);
    if (q_heads > 0 && !stride_ok(q_token_stride, (int64_t)q_heads * head_dim, tokens, s)) return RMSNORM_EINVAL;
    if (kv == nullptr) return RMSNORM_EINVAL;
    if (rope->positions == nullptr && rope->axes != 1) return RMSNORM_EINVAL;
    const bool e4m3 = kv->cache_dtype == RMSNORM_E4M3;
    if (!e4m3 && kv->cache_dtype != dtype) return RMSNORM_EINVAL;
    if (e4m3 && (!scale_ok(kv->k_scale) || !scale_ok(kv->v_scale))) return RMSNORM_EINVAL;
    if (kv->seqs < 0 || kv->max_pages < 0 || kv->num_pages < 0 || kv->page_size < 1) return RMSNORM_EINVAL;
    if (kv->page_table_stride < kv->max_pages || kv->page_stride < 0 || kv->row_stride < 0 || kv->head_stride < 0)
        return RMSNORM_EINVAL;
    const int64_t c = e4m3 ? 1 : s;
    const int64_t most = INT64_MAX / 8 / c;
    if (kv->num_pages > 0 && kv->page_stride > most / kv->num_pages) return RMSNORM_EINVAL;
    if (kv->row_stride > most / kv->page_size || kv->head_stride > most / kv_heads) return RMSNORM_EINVAL;
    if (kv->seqs > 0 && kv->page_table_stride > INT64_MAX / 8 / kv->seqs) return RMSNORM_EINVAL;
    if (tokens == 0 || kv->seqs == 0) return RMSNORM_OK;
    if (x == nullptr || !rrn::on_boundary(x, s)) return RMSNORM_EINVAL;
    if (q_heads > 0 && (q_out == nullptr || !rrn::on_boundary(q_out, s))) return RMSNORM_EINVAL;
    if (q_heads > 0 && x == q_out && x_token_stride != q_token_stride) return RMSNORM_EINVAL;
    if (kv->cu_tokens == nullptr || kv->cache_lens == nullptr || !rrn::on_boundary(kv->cu_tokens, 4) ||
        !rrn::on_boundary(kv->cache_lens, 4) || !rrn::on_boundary(kv->page_table, 4) ||
        !rrn::on_boundary(kv->dropped, 4))
        return RMSNORM_EINVAL;
    if (kv->max_pages > 0 && kv->page_table == nullptr) return RMSNORM_EINVAL;
    if (kv->max_pages > 0 && kv->num_pages > 0 &&
        (kv->k_cache == nullptr || kv->v_cache == nullptr || !rrn::on_boundary(kv->k_cache, c) ||
         !rrn::on_boundary(kv->v_cache, c)))
        return RMSNORM_EINVAL;
    p.x = x;
    p.y = q_out;
    p.y_stride = q_heads > 0 ? q_token_stride * s : 0;
    p.cu_tokens = kv->cu_tokens;
    p.cache_lens = kv->cache_lens;
    p.page_table = kv->page_table;
    p.table_stride = kv->page_table_stride;
    p.seqs = kv->seqs;
    p.max_pages = kv->max_pages;
    p.num_pages = kv->num_pages;
    p.page_size = kv->page_size;
    p.k_cache = kv->k_cache;
    p.v_cache = kv->v_cache;
    p.page_stride = kv->page_stride * c;
    p.row_stride = kv->row_stride * c;
    p.head_stride = kv->head_stride * c;
    if (e4m3) {
        p.k_inv = (float)(1.0 / (double)kv->k_scale);
        p.v_inv = (float)(1.0 / (double)kv->v_scale);
        p.k_scale = kv->k_scale;
        p.v_scale = kv->v_scale;
        p.settle = !power_of_two(kv->k_scale) || !power_of_two(kv->v_scale);
    }
    p.dropped = kv->dropped;
    Unit u;
    u.at(x, s), u.at(kv->k_cache, c), u.at(kv->v_cache, c);
    u.step(x_token_stride), u.step(kv->page_stride), u.step(kv->row_stride), u.step(kv->head_stride);
    if (q_heads > 0) u.at(q_out, s), u.step(q_token_stride);
    const int mode = !e4m3 ? rrn::kRopeAppend : p.settle ? rrn::kRopeAppendSettled : rrn::kRopeAppendE4m3;
    return launch_forward(&p, dtype, u.get(), rope->interleaved == 1, mode, stream);
}

}  // extern "C"
