// logprobs_api.cu -- entry points of the tokens' log probabilities and their
// gradient (declared in include/rmsnorm.h): argument checks, the choice of a
// kernel and its grid, the launch.
#include <climits>
#include <cmath>
#include <cstring>

#include "launch_util.h"
#include "logprobs_kernels.cuh"
#include "logprobs_pick.h"

namespace {

constexpr int64_t kMaxVocab = 1 << 20;

int check_logits(const void *logits, const void *tokens, int token_bytes, int64_t rows, int64_t vocab, int64_t stride,
                 float temperature, int dtype) {
    if (dtype != RMSNORM_F32 && dtype != RMSNORM_BF16) return RMSNORM_EINVAL;
    if ((token_bytes != 4 && token_bytes != 8) || rows < 0 || vocab <= 0 || (rows > 1 && stride < vocab))
        return RMSNORM_EINVAL;
    if (!(temperature > 0.f) || !std::isnormal(temperature) || !std::isnormal((float)(1.0 / (double)temperature)))
        return RMSNORM_EINVAL;
    if (vocab > kMaxVocab) return RMSNORM_EUNSUPPORTED;
    if (rows > 1 && stride > INT64_MAX / 8 / rows) return RMSNORM_EINVAL;
    if (rows > 0 && logits == nullptr) return RMSNORM_EINVAL;
    if (!rrn::on_boundary(logits, rrn::size_of(dtype)) || !rrn::on_boundary(tokens, token_bytes)) return RMSNORM_EINVAL;
    return RMSNORM_OK;
}

template <typename T, bool ALIGNED>
const void *forward_of(bool entropy, bool top) {
    if (entropy)
        return top ? reinterpret_cast<const void *>(&rrn::logprobs_fwd_kernel<T, ALIGNED, true, true>)
                   : reinterpret_cast<const void *>(&rrn::logprobs_fwd_kernel<T, ALIGNED, true, false>);
    return top ? reinterpret_cast<const void *>(&rrn::logprobs_fwd_kernel<T, ALIGNED, false, true>)
               : reinterpret_cast<const void *>(&rrn::logprobs_fwd_kernel<T, ALIGNED, false, false>);
}
const void *forward_kernel(int dtype, bool aligned, bool entropy, bool top) {
    if (dtype == RMSNORM_BF16)
        return aligned ? forward_of<rrn::BF16, true>(entropy, top) : forward_of<rrn::BF16, false>(entropy, top);
    return aligned ? forward_of<rrn::F32, true>(entropy, top) : forward_of<rrn::F32, false>(entropy, top);
}

template <typename T, bool ALIGNED>
const void *backward_of(bool entropy) {
    return entropy ? reinterpret_cast<const void *>(&rrn::logprobs_bwd_kernel<T, ALIGNED, true>)
                   : reinterpret_cast<const void *>(&rrn::logprobs_bwd_kernel<T, ALIGNED, false>);
}
const void *backward_kernel(int dtype, bool aligned, bool entropy) {
    if (dtype == RMSNORM_BF16)
        return aligned ? backward_of<rrn::BF16, true>(entropy) : backward_of<rrn::BF16, false>(entropy);
    return aligned ? backward_of<rrn::F32, true>(entropy) : backward_of<rrn::F32, false>(entropy);
}

}  // namespace

extern "C" {

int rmsnorm_logprobs_fwd(const void *logits, const void *tokens, int token_bytes, float *logprobs, float *stats,
                         float *entropy, float *top_logprobs, int32_t *top_ids, int64_t rows, int64_t vocab,
                         int64_t row_stride, int32_t top, float temperature, int dtype, rmsnorm_stream_t stream) {
    int st = check_logits(logits, tokens, token_bytes, rows, vocab, row_stride, temperature, dtype);
    if (st != RMSNORM_OK) return st;
    if (top < 0 || top > rrn::kLpTop || top > vocab) return RMSNORM_EINVAL;
    if (rows == 0) return RMSNORM_OK;
    if ((logprobs != nullptr && tokens == nullptr) || (top > 0 && (top_logprobs == nullptr || top_ids == nullptr)))
        return RMSNORM_EINVAL;
    const void *fp[] = {logprobs, entropy, top_logprobs, top_ids};
    for (const void *q : fp)
        if (!rrn::on_boundary(q, 4)) return RMSNORM_EINVAL;
    if (!rrn::on_boundary(stats, 8)) return RMSNORM_EINVAL;
    const int64_t s = rrn::size_of(dtype);
    rrn::LogprobParams p;
    std::memset(&p, 0, sizeof(p));
    p.logits = static_cast<const char *>(logits);
    p.tokens = tokens;
    p.logprobs = logprobs;
    p.stats = stats;
    p.entropy = entropy;
    p.top_logprobs = top_logprobs;
    p.top_ids = top_ids;
    p.stride = row_stride * s;
    p.vocab = (int32_t)vocab;
    p.units = (int32_t)rrn::div_up(vocab, dtype == RMSNORM_BF16 ? rrn::lp_unit<rrn::BF16>() : rrn::lp_unit<rrn::F32>());
    p.top = top;
    p.rows = rows;
    p.wide = token_bytes == 8;
    const bool aligned = rrn::on_boundary(logits, 16) && (rows == 1 || p.stride % 16 == 0);
    p.inv_t = (float)(1.0 / (double)temperature);
    p.c = (float)(1.4426950408889634 / (double)temperature);
    int dev = 0, sms = 0;
    if ((st = rrn::current_device_sms(&dev, &sms)) != RMSNORM_OK) return st;
    // a warp a unit, up to the block's eight; short rows several a block, unless
    // there are few and alternatives to be found, which all warps take part in
    // (one warp / eight, us, bf16 rows of 1000 with 5: 8 rows 6.1 / 4.6, 300 6.2 /
    // 5.3, 600 6.4 / 6.2, 2000 7.5 / 19.7)
    p.warps = top > 0 && rows <= 4 * sms ? rrn::kLpWarps : 1;
    while (p.warps < rrn::kLpWarps && p.warps < p.units) p.warps *= 2;
    const int64_t groups = rrn::div_up(rows, rrn::kLpWarps / p.warps);
    // a row over as many blocks as give every SM one, while each of their warps has
    // a unit (alone / together, us, bf16: 8 x 131072 9.7 / 3.1, with 20 alternatives
    // 17.1 / 6.7, 100 x 50264 5.9 / 5.0)
    int cluster = 1;
    while (cluster < 8 && groups * cluster < sms && 2 * cluster * rrn::kLpWarps <= p.units + rrn::kLpWarps - 1)
        cluster *= 2;
    if (groups > INT_MAX / cluster) return RMSNORM_EUNSUPPORTED;
    const void *fn = forward_kernel(dtype, aligned, entropy != nullptr, top > 0);
    const size_t smem = rrn::lp_smem(p.units, rrn::kLpWarps / p.warps);
    int resident = 0;
    if ((st = rrn::resident_blocks(dev, fn, rrn::kLpThreads, smem, &resident)) != RMSNORM_OK) return st;
    p.ahead = (int64_t)resident * sms * (rrn::kLpWarps / p.warps);
    void *argv[] = {&p};
    return rrn::launch_kernel(fn, dim3((unsigned)(groups * cluster)), rrn::kLpThreads, smem, stream, argv, cluster);
}

int rmsnorm_logprobs_bwd(const void *logits, const void *tokens, int token_bytes, const float *stats,
                         const float *dlogprobs, const float *entropy, const float *dentropy, void *dlogits,
                         int64_t rows, int64_t vocab, int64_t row_stride, int64_t dlogits_stride, float temperature,
                         int dtype, rmsnorm_stream_t stream) {
    const int st = check_logits(logits, tokens, token_bytes, rows, vocab, row_stride, temperature, dtype);
    if (st != RMSNORM_OK) return st;
    if (rows > 1 && (dlogits_stride < vocab || dlogits_stride > INT64_MAX / 8 / rows)) return RMSNORM_EINVAL;
    if (rows == 0) return RMSNORM_OK;
    const int64_t s = rrn::size_of(dtype);
    // in place only onto itself: other strides would write rows that are still read
    if (dlogits == logits && rows > 1 && dlogits_stride != row_stride) return RMSNORM_EINVAL;
    if (dlogits == nullptr || !rrn::on_boundary(dlogits, s) || stats == nullptr || !rrn::on_boundary(stats, 8))
        return RMSNORM_EINVAL;
    if ((dlogprobs != nullptr && tokens == nullptr) || (dentropy != nullptr && entropy == nullptr))
        return RMSNORM_EINVAL;
    const void *fp[] = {dlogprobs, entropy, dentropy};
    for (const void *q : fp)
        if (!rrn::on_boundary(q, 4)) return RMSNORM_EINVAL;
    rrn::LogprobBwdParams p;
    std::memset(&p, 0, sizeof(p));
    p.logits = static_cast<const char *>(logits);
    p.tokens = tokens;
    p.stats = stats;
    p.dlogprobs = dlogprobs;
    p.entropy = entropy;
    p.dentropy = dentropy;
    p.dlogits = static_cast<char *>(dlogits);
    p.stride = row_stride * s;
    p.dstride = dlogits_stride * s;
    p.vocab = (int32_t)vocab;
    p.rows = rows;
    p.wide = token_bytes == 8;
    const bool aligned = rrn::on_boundary(logits, 16) && rrn::on_boundary(dlogits, 16) &&
                         (rows == 1 || (p.stride % 16 == 0 && p.dstride % 16 == 0));
    p.inv_t = (float)(1.0 / (double)temperature);
    p.c = (float)(1.4426950408889634 / (double)temperature);
    // chunks of a row, one more where they may start before it
    const int64_t chunks = rrn::div_up(vocab * s, 16) + (aligned ? 0 : 1);
    p.shift = 5;
    while (p.shift < 8 && chunks > rrn::kLpBwdChunks << p.shift) ++p.shift;
    const int64_t groups = rrn::div_up(rows, rrn::kLpThreads >> p.shift);
    const int64_t parts = rrn::div_up(chunks, (int64_t)rrn::kLpBwdChunks << p.shift);
    int dev = 0, sms = 0;
    const int got = rrn::current_device_sms(&dev, &sms);
    if (got != RMSNORM_OK) return got;
    // Parts of a row that a block takes: four where that leaves four waves of
    // blocks (bf16 8192 x 131072: one 700 us, two 635, four 622, sixteen 635).
    const int64_t most = groups * parts / (16 * (int64_t)sms);
    p.turns = most >= 4 ? 4 : most >= 2 ? 2 : 1;
    p.slices = (int32_t)rrn::div_up(parts, p.turns);
    if (groups > INT_MAX / p.slices) return RMSNORM_EUNSUPPORTED;
    void *argv[] = {&p};
    return rrn::launch_kernel(backward_kernel(dtype, aligned, dentropy != nullptr), dim3((unsigned)(groups * p.slices)),
                              rrn::kLpThreads, 0, stream, argv);
}

}  // extern "C"
