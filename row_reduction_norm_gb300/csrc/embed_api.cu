// embed_api.cu -- entry points of the embedding lookup and its gradient
// (declared in include/rmsnorm.h): argument checks, the choice of a kernel and
// its grid, the launches.
#include <climits>
#include <cmath>
#include <cstring>

#include "embed_kernels.cuh"
#include "launch_util.h"

namespace {

constexpr int64_t kMaxWidth = 65536, kMaxCount = 1 << 30;

int check_embedding(const void *tokens, int token_bytes, int64_t count, int64_t vocab, int64_t width,
                    int64_t table_stride, float scale, int dtype) {
    if (dtype != RMSNORM_F32 && dtype != RMSNORM_BF16) return RMSNORM_EINVAL;
    if ((token_bytes != 4 && token_bytes != 8) || count < 0 || vocab <= 0 || width <= 0 || table_stride < width)
        return RMSNORM_EINVAL;
    if (!std::isfinite(scale)) return RMSNORM_EINVAL;
    if (width > kMaxWidth) return RMSNORM_EUNSUPPORTED;
    if (table_stride > INT64_MAX / 8 / vocab || count > INT64_MAX / 8 / width) return RMSNORM_EINVAL;
    if (count > 0 && (tokens == nullptr || !rrn::on_boundary(tokens, token_bytes))) return RMSNORM_EINVAL;
    return RMSNORM_OK;
}

// The largest power of two up to `most` bytes that divides a and b.
int64_t common_bytes(int64_t a, int64_t b, int64_t most) {
    while (most > 1 && (a % most != 0 || b % most != 0)) most /= 2;
    return most;
}

const void *forward_kernel(int dtype, int64_t bytes, bool one) {
#define FWD(T, P) \
    (one ? reinterpret_cast<const void *>(&rrn::embed_fwd_kernel<rrn::T, P, 1>) \
         : reinterpret_cast<const void *>(&rrn::embed_fwd_kernel<rrn::T, P, 4>))
    if (dtype == RMSNORM_BF16)
        return bytes == 16 ? FWD(BF16, 8) : bytes == 8 ? FWD(BF16, 4) : bytes == 4 ? FWD(BF16, 2) : FWD(BF16, 1);
    return bytes == 16 ? FWD(F32, 4) : bytes == 8 ? FWD(F32, 2) : FWD(F32, 1);
#undef FWD
}

const void *sum_kernel(int dtype, int grad_dtype, int64_t p) {
#define SUM(T, TG, P) reinterpret_cast<const void *>(&rrn::embed_sum_kernel<rrn::T, rrn::TG, P>)
    if (dtype == RMSNORM_F32) return p == 4 ? SUM(F32, F32, 4) : p == 2 ? SUM(F32, F32, 2) : SUM(F32, F32, 1);
    if (grad_dtype == RMSNORM_F32)
        return p == 8 ? SUM(BF16, F32, 8) : p == 4 ? SUM(BF16, F32, 4) : p == 2 ? SUM(BF16, F32, 2) : SUM(BF16, F32, 1);
    return p == 8 ? SUM(BF16, BF16, 8) : p == 4 ? SUM(BF16, BF16, 4) : p == 2 ? SUM(BF16, BF16, 2) : SUM(BF16, BF16, 1);
#undef SUM
}

const void *join_kernel(int grad_dtype, int64_t p) {
#define JOIN(TG, P) reinterpret_cast<const void *>(&rrn::embed_join_kernel<rrn::TG, P>)
    if (grad_dtype == RMSNORM_F32) return p == 8 ? JOIN(F32, 8) : p == 4 ? JOIN(F32, 4) : p == 2 ? JOIN(F32, 2) : JOIN(F32, 1);
    return p == 8 ? JOIN(BF16, 8) : p == 4 ? JOIN(BF16, 4) : p == 2 ? JOIN(BF16, 2) : JOIN(BF16, 1);
#undef JOIN
}

// What the gradient's workspace holds, in bytes from its start.
struct Layout {
    int64_t a, b, present, partial, bytes, words, segments, tiles;
    Layout(int64_t count, int64_t vocab, int64_t width) {
        words = rrn::div_up(vocab, 32);
        segments = rrn::div_up(count, rrn::kSegment);
        tiles = rrn::div_up(width, rrn::kTile);
        a = 0;
        b = a + rrn::div_up(count * 8, 16) * 16;
        present = b + rrn::div_up(count * 8, 16) * 16;
        partial = present + rrn::div_up(words * 4, 16) * 16;
        bytes = partial + 2 * segments * tiles * rrn::kTile * 4;
    }
};

// Blocks of the sorting cluster: one while its threads have at most two tokens each.
int sort_blocks(int64_t count) {
    int n = 1;
    while (n < 8 && count > 2048 * n) n *= 2;
    return n;
}

}  // namespace

extern "C" {

int rmsnorm_embedding_fwd(const void *tokens, int token_bytes, const void *table, void *y, int64_t count, int64_t vocab,
                          int64_t width, int64_t table_stride, float scale, int dtype, rmsnorm_stream_t stream) {
    const int st = check_embedding(tokens, token_bytes, count, vocab, width, table_stride, scale, dtype);
    if (st != RMSNORM_OK) return st;
    if (count == 0) return RMSNORM_OK;
    const int64_t s = rrn::size_of(dtype);
    if (table == nullptr || y == nullptr || !rrn::on_boundary(table, s) || !rrn::on_boundary(y, s)) return RMSNORM_EINVAL;
    int64_t bytes = common_bytes(width * s, table_stride * s, 16);
    while (!rrn::on_boundary(table, bytes) || !rrn::on_boundary(y, bytes)) bytes /= 2;
    rrn::EmbedParams p;
    p.tokens = tokens;
    p.table = static_cast<const char *>(table);
    p.y = static_cast<char *>(y);
    p.count = count;
    p.vocab = vocab;
    p.table_stride = table_stride * s;
    p.pieces = (uint32_t)(width * s / bytes);
    p.magic = ((uint64_t)1 << 40) / p.pieces + 1;
    p.wide = token_bytes == 8;
    p.scale = scale;
    int dev = 0, sms = 0;
    const int got = rrn::current_device_sms(&dev, &sms);
    if (got != RMSNORM_OK) return got;
    const int64_t all = count * p.pieces;
    const bool one = all <= (int64_t)sms * rrn::kEmbedThreads * 4;
    const int64_t blocks = rrn::div_up(all, rrn::kEmbedThreads * (one ? 1 : 4));
    if (blocks > INT_MAX) return RMSNORM_EUNSUPPORTED;
    void *argv[] = {&p};
    return rrn::launch_kernel(forward_kernel(dtype, bytes, one), dim3((unsigned)blocks), rrn::kEmbedThreads, 0, stream,
                              argv);
}

int64_t rmsnorm_embedding_bwd_workspace_bytes(int64_t count, int64_t vocab, int64_t width) {
    if (count < 0 || vocab <= 0 || width <= 0) return RMSNORM_EINVAL;
    if (count > kMaxCount || vocab > kMaxCount || width > kMaxWidth) return RMSNORM_EUNSUPPORTED;
    return Layout(count, vocab, width).bytes;
}

int rmsnorm_embedding_bwd(const void *dy, const void *tokens, int token_bytes, void *dtable, int64_t count,
                          int64_t vocab, int64_t width, int64_t table_stride, float scale, int accumulate, int dtype,
                          int grad_dtype, void *workspace, uint64_t workspace_bytes, rmsnorm_stream_t stream) {
    int st = check_embedding(tokens, token_bytes, count, vocab, width, table_stride, scale, dtype);
    if (st != RMSNORM_OK) return st;
    if (grad_dtype != dtype && grad_dtype != RMSNORM_F32) return RMSNORM_EINVAL;
    if (accumulate != 0 && accumulate != 1) return RMSNORM_EINVAL;
    if (count > kMaxCount || vocab > kMaxCount) return RMSNORM_EUNSUPPORTED;
    const int64_t s = rrn::size_of(dtype), sg = rrn::size_of(grad_dtype);
    if (dtable == nullptr || !rrn::on_boundary(dtable, sg)) return RMSNORM_EINVAL;
    if (count > 0 && (dy == nullptr || !rrn::on_boundary(dy, s))) return RMSNORM_EINVAL;
    const Layout at(count, vocab, width);
    if (workspace == nullptr || !rrn::on_boundary(workspace, 16) || workspace_bytes < (uint64_t)at.bytes)
        return RMSNORM_EINVAL;
    if (count == 0 && accumulate) return RMSNORM_OK;
    char *ws = static_cast<char *>(workspace);

    rrn::SortParams q;
    q.tokens = tokens;
    q.a = reinterpret_cast<uint2 *>(ws + at.a);
    q.b = reinterpret_cast<uint2 *>(ws + at.b);
    q.present = accumulate ? nullptr : reinterpret_cast<uint32_t *>(ws + at.present);
    q.words = accumulate ? 0 : (int32_t)at.words;
    q.count = (int32_t)count;
    q.vocab = (uint32_t)vocab;
    int bits = 1;
    while (vocab >> bits) ++bits;   // of 0 .. vocab
    q.passes = (int32_t)rrn::div_up(bits, 10);
    q.bits = (int32_t)rrn::div_up(bits, q.passes);
    q.wide = token_bytes == 8;
    int dev = 0, sms = 0;
    if ((st = rrn::current_device_sms(&dev, &sms)) != RMSNORM_OK) return st;
    const void *sort = reinterpret_cast<const void *>(&rrn::embed_sort_kernel);
    if ((st = rrn::allow_smem(dev, sort)) != RMSNORM_OK) return st;
    void *sort_argv[] = {&q};
    const int cluster = sort_blocks(count);
    st = rrn::launch_kernel(sort, dim3((unsigned)cluster), rrn::kSortThreads,
                            (size_t)rrn::sort_smem(q.bits), stream, sort_argv, cluster);
    if (st != RMSNORM_OK) return st;

    rrn::SumParams p;
    std::memset(&p, 0, sizeof(p));
    p.sorted = q.passes % 2 ? q.a : q.b;
    p.dy = static_cast<const char *>(dy);
    p.dtable = static_cast<char *>(dtable);
    p.present = q.present;
    p.partial = reinterpret_cast<float *>(ws + at.partial);
    p.dy_stride = width * s;
    p.table_stride = table_stride * sg;
    p.vocab = vocab;
    p.count = (int32_t)count;
    p.width = (int32_t)width;
    p.segments = (int32_t)at.segments;
    p.tiles = (int32_t)at.tiles;
    p.scale = scale;
    p.accumulate = accumulate;
    p.work_blocks = rrn::div_up(at.segments * at.tiles, rrn::kSumWarps);
    // elements of a piece: what dy's rows and the gradient's both allow
    int64_t bytes = common_bytes(width * s, 16, 16);
    while (!rrn::on_boundary(dy, bytes)) bytes /= 2;
    int64_t held = common_bytes(table_stride * sg, width * sg, 16);
    while (!rrn::on_boundary(dtable, held)) held /= 2;
    p.zero_bytes = (int32_t)held;
    int64_t piece = bytes / s;
    while (piece * sg > held && held < 16) piece /= 2;
    const int64_t blocks = p.work_blocks + (accumulate ? 0 : rrn::div_up(vocab, rrn::kSumWarps));
    if (blocks > INT_MAX) return RMSNORM_EUNSUPPORTED;
    void *argv[] = {&p};
    st = rrn::launch_kernel(sum_kernel(dtype, grad_dtype, piece), dim3((unsigned)blocks), rrn::kSumThreads, 0, stream,
                            argv);
    if (st != RMSNORM_OK || at.segments < 2) return st;
    return rrn::launch_kernel(join_kernel(grad_dtype, piece),
                              dim3((unsigned)rrn::div_up((at.segments - 1) * at.tiles, rrn::kSumWarps)),
                              rrn::kSumThreads, 0, stream, argv);
}

}  // extern "C"
