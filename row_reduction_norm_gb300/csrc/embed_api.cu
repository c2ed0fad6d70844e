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

// The kernel of the sums over sorted tokens, or over few tokens without a sort.
const void *sum_kernel(int dtype, int grad_dtype, int64_t p, bool direct) {
#define SUM(T, TG, P) \
    (direct ? reinterpret_cast<const void *>(&rrn::embed_direct_kernel<rrn::T, rrn::TG, P>) \
            : reinterpret_cast<const void *>(&rrn::embed_sum_kernel<rrn::T, rrn::TG, P>))
    if (dtype == RMSNORM_F32) return p == 4 ? SUM(F32, F32, 4) : p == 2 ? SUM(F32, F32, 2) : SUM(F32, F32, 1);
    if (grad_dtype == RMSNORM_F32)
        return p == 8 ? SUM(BF16, F32, 8) : p == 4 ? SUM(BF16, F32, 4) : p == 2 ? SUM(BF16, F32, 2) : SUM(BF16, F32, 1);
    return p == 8 ? SUM(BF16, BF16, 8) : p == 4 ? SUM(BF16, BF16, 4) : p == 2 ? SUM(BF16, BF16, 2) : SUM(BF16, BF16, 1);
#undef SUM
}

const void *join_kernel(int grad_dtype, int64_t p) {
#define JOIN(TG, P) reinterpret_cast<const void *>(&rrn::embed_join_kernel<rrn::TG, P>)
    if (grad_dtype == RMSNORM_F32)
        return p == 8 ? JOIN(F32, 8) : p == 4 ? JOIN(F32, 4) : p == 2 ? JOIN(F32, 2) : JOIN(F32, 1);
    return p == 8 ? JOIN(BF16, 8) : p == 4 ? JOIN(BF16, 4) : p == 2 ? JOIN(BF16, 2) : JOIN(BF16, 1);
#undef JOIN
}

// Sorted tokens of a warp: as many, from 4 to 64, as make one wave of blocks,
// three on each of the device's 152 SMs; with more than that to do, 32 (us, bf16
// 65536 x 768: 54, one wave, 46.0, 32 49.5, 16 52.8; 16384 x 4096: 36, two waves,
// 70.7, 32 69.7, 8 80.4; 2000 x 1024: 4 11.3, 32 14.4).  (A constant for the SMs:
// the workspace's size and the order of the sums follow from the sizes alone.)
int run_of(int64_t count, int64_t tiles) {
    constexpr int64_t wave = 3 * 152, least = 4, most = 64, many = 32;
    const int64_t run = rrn::div_up(count, rrn::kSumWarps * (wave / tiles));
    return (int)(run < least ? least : run > most ? many : run);
}

// Whether tokens are added up without a sort: the work of that, every warp
// comparing all ids, grows with the square of their number (without / with a
// sort, us, table of 8192 rows: bf16 256 x 1024 6.1 / 9.3, 512 x 1024 9.5 / 9.4,
// 1000 x 1024 14.2 / 9.8, 1000 x 4096 45.8 / 20.8; fp32 1000 x 256 8.4 / 9.4).
bool direct_sums(int64_t count, int64_t tiles) {
    return count <= rrn::kDirect && count * count * tiles <= 1 << 20;
}

// What the gradient's workspace holds, in bytes from its start.
struct Layout {
    int64_t a, b, present, partial, bytes, words, chunks, tiles;
    int run;
    Layout(int64_t count, int64_t vocab, int64_t width) {
        words = rrn::div_up(vocab, 32);
        tiles = rrn::div_up(width, rrn::kTile);
        run = run_of(count, tiles);
        chunks = rrn::div_up(count, (int64_t)rrn::kSumWarps * run);
        a = 0;
        b = a + rrn::div_up(count * 8, 16) * 16;
        present = b + rrn::div_up(count * 8, 16) * 16;
        partial = present + rrn::div_up(words * 4, 16) * 16;
        bytes = partial + 2 * chunks * tiles * rrn::kTile * 4;
    }
};

// Blocks of the sorting cluster: one while its threads have at most two tokens
// each, and 16 (whose barriers take 2000 cycles, not 800) from eight a thread on
// (8 / 16 blocks, us: bf16 12000 x 256 14.3 / 13.9, 16384 x 4096 69.8 / 72.3, 65536
// x 768 65.5 / 52.8).
int sort_blocks(int64_t count) {
    int n = 1;
    while (n < rrn::kClusterMaxCtas && count > 2 * rrn::kSortThreads * n) n *= 2;
    return count > 8 * rrn::kSortThreads * n ? rrn::kSortBlocks : n;
}

}  // namespace

extern "C" {

int rmsnorm_embedding_fwd(const void *tokens, int token_bytes, const void *table, void *y, int64_t count, int64_t vocab,
                          int64_t width, int64_t table_stride, float scale, int dtype, rmsnorm_stream_t stream) {
    const int st = check_embedding(tokens, token_bytes, count, vocab, width, table_stride, scale, dtype);
    if (st != RMSNORM_OK) return st;
    if (count == 0) return RMSNORM_OK;
    const int64_t s = rrn::size_of(dtype);
    if (table == nullptr || y == nullptr || !rrn::on_boundary(table, s) || !rrn::on_boundary(y, s))
        return RMSNORM_EINVAL;
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
    // a piece a thread, or four: one / four, us, bf16 rows of 4096: 8 rows 1.26 /
    // 1.65, 64 1.32 / 1.64, 200 1.78 / 1.68, 2000 5.1 / 4.1, 16384 41 / 29
    const bool one = all <= (int64_t)sms * rrn::kEmbedThreads * 2;
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

    rrn::SumParams p;
    std::memset(&p, 0, sizeof(p));
    p.tokens = tokens;
    p.wide = token_bytes == 8;
    p.dy = static_cast<const char *>(dy);
    p.dtable = static_cast<char *>(dtable);
    p.dy_stride = width * s;
    p.table_stride = table_stride * sg;
    p.vocab = vocab;
    p.count = (int32_t)count;
    p.width = (int32_t)width;
    p.tiles = (int32_t)at.tiles;
    p.run = at.run;
    p.scale = scale;
    p.accumulate = accumulate;
    // elements of a piece: what dy's rows and the gradient's both allow
    int64_t bytes = common_bytes(width * s, 16, 16);
    while (!rrn::on_boundary(dy, bytes)) bytes /= 2;
    int64_t held = common_bytes(table_stride * sg, width * sg, 16);
    while (!rrn::on_boundary(dtable, held)) held /= 2;
    p.zero_bytes = (int32_t)held;
    int64_t piece = bytes / s;
    while (piece * sg > held && held < 16) piece /= 2;
    const bool direct = direct_sums(count, at.tiles);
    p.words = (int32_t)at.words;
    p.zero_parts = (int32_t)rrn::div_up(width * sg, rrn::kZeroBytes);
    p.chunks = direct ? rrn::div_up(count, rrn::kSumWarps) : at.chunks;
    p.work_blocks = p.chunks * at.tiles;
    int dev = 0, sms = 0;
    if ((st = rrn::current_device_sms(&dev, &sms)) != RMSNORM_OK) return st;
    const void *sort = reinterpret_cast<const void *>(&rrn::embed_sort_kernel);
    if (!direct && (st = rrn::allow_smem(dev, sort)) != RMSNORM_OK) return st;
    int cluster = sort_blocks(count);
    if (!direct && cluster > rrn::kClusterMaxCtas &&
        !rrn::large_cluster(dev, sort, rrn::kSortBlocks, rrn::kSortThreads,
                            (size_t)rrn::sort_smem(rrn::kSortMaxBits, rrn::kSortWords)))
        cluster = rrn::kClusterMaxCtas;
    // Zeros that are written while the tokens are sorted, by as many clusters more
    // as the device has SMs for, and as many bytes as the sort takes time for (12
    // us, and 4 for 65536 tokens more); the sums' blocks write the rest where no
    // token is (bf16 16384 x 4096 75.1 -> 69.8 us, 5000 x 1024 17.7 -> 14.6).
    const int more = direct || accumulate ? 0 : (sms - cluster) / cluster;
    const int64_t row_bytes = width * sg;
    int64_t early = more < 1 ? 0 : (((int64_t)48 << 20) + count * 512) / row_bytes / 32 * 32;
    if (early > vocab) early = vocab;
    p.first_word = (int32_t)rrn::div_up(early, 32);
    const int64_t blocks = p.work_blocks +
                           (accumulate ? 0 : rrn::div_up((at.words - p.first_word) * p.zero_parts, rrn::kSumWarps));
    if (blocks > INT_MAX) return RMSNORM_EUNSUPPORTED;
    void *argv[] = {&p};
    const void *sums = sum_kernel(dtype, grad_dtype, piece, direct);
    if (direct) return rrn::launch_kernel(sums, dim3((unsigned)blocks), rrn::kSumThreads, 0, stream, argv);

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
    q.passes = (int32_t)rrn::div_up(bits, rrn::kSortMaxBits);
    q.bits = (int32_t)rrn::div_up(bits, q.passes);
    q.wide = p.wide;
    q.dtable = p.dtable;
    q.table_stride = p.table_stride;
    q.zero_rows = early;
    q.row_bytes = (int32_t)row_bytes;
    q.zero_bytes = p.zero_bytes;
    void *sort_argv[] = {&q};
    const int sort_blocks_all = cluster * (early > 0 ? 1 + more : 1);
    st = rrn::launch_kernel(sort, dim3((unsigned)sort_blocks_all), rrn::kSortThreads,
                            (size_t)rrn::sort_smem(q.bits, q.words), stream, sort_argv, cluster);
    if (st != RMSNORM_OK) return st;

    p.sorted = q.passes % 2 ? q.a : q.b;
    p.present = q.present;
    p.partial = reinterpret_cast<float *>(ws + at.partial);
    st = rrn::launch_kernel(sums, dim3((unsigned)blocks), rrn::kSumThreads, 0, stream, argv);
    if (st != RMSNORM_OK || at.chunks < 2) return st;
    return rrn::launch_kernel(join_kernel(grad_dtype, piece), dim3((unsigned)(at.chunks - 1)), rrn::kSumThreads, 0,
                              stream, argv);
}

}  // extern "C"
