// grads_api.cu -- entry points of the norm of many tensors together and their
// clipping (declared in include/rmsnorm.h): argument checks, the launches.
#include <climits>
#include <cmath>
#include <cstddef>
#include <cstring>
#include <memory>
#include <new>

#include "grads_kernels.cuh"
#include "launch_util.h"

namespace {

using rrn::GradEntry;
using rrn::GradTable;

// Parts of a tensor that `threads` threads take one of.
uint32_t parts_of(const rmsnorm_grad_t &g, int threads) {
    const int64_t s = rrn::size_of(g.dtype);
    return (uint32_t)rrn::div_up((int64_t)(reinterpret_cast<uintptr_t>(g.grad) & 15) + g.count * s,
                                 rrn::grad_part(threads));
}

int check_grads(const rmsnorm_grad_t *grads, int64_t n, bool clip, const float *norm, const void *workspace,
                uint64_t workspace_bytes) {
    if (n < 0 || (n > 0 && grads == nullptr) || norm == nullptr || !rrn::on_boundary(norm, 4)) return RMSNORM_EINVAL;
    if (workspace == nullptr || !rrn::on_boundary(workspace, 16) ||
        workspace_bytes < (uint64_t)rmsnorm_grad_norm_workspace_bytes())
        return RMSNORM_EINVAL;
    for (int64_t i = 0; i < n; ++i) {
        const rmsnorm_grad_t &g = grads[i];
        if ((g.dtype != RMSNORM_F32 && g.dtype != RMSNORM_BF16) || g.reserved != 0) return RMSNORM_EINVAL;
        if (g.count < 0 || g.count > INT64_MAX / 8) return RMSNORM_EINVAL;
        if (g.count == 0) continue;
        const int64_t s = rrn::size_of(g.dtype);
        if (g.grad == nullptr || !rrn::on_boundary(g.grad, s)) return RMSNORM_EINVAL;
        if (clip && (g.out == nullptr || !rrn::on_boundary(g.out, s))) return RMSNORM_EINVAL;
        if (g.count > (int64_t)1 << 44) return RMSNORM_EUNSUPPORTED;
    }
    return RMSNORM_OK;
}

// Whether two of the tensors have the same out: they would be scaled twice, or
// once, as it comes.  A status.
int distinct_outs(const rmsnorm_grad_t *grads, int64_t n) {
    if (n <= 24) {
        for (int64_t i = 1; i < n; ++i)
            for (int64_t j = 0; j < i; ++j)
                if (grads[i].out == grads[j].out && grads[i].count > 0 && grads[j].count > 0) return RMSNORM_EINVAL;
        return RMSNORM_OK;
    }
    uint64_t room = 64;
    while (room < 2 * (uint64_t)n) room *= 2;
    const std::unique_ptr<const void *[]> seen(new (std::nothrow) const void *[room]());
    if (seen == nullptr) return RMSNORM_EUNSUPPORTED;
    for (int64_t i = 0; i < n; ++i) {
        if (grads[i].count == 0) continue;
        uint64_t at = (reinterpret_cast<uintptr_t>(grads[i].out) >> 4) * 0x9E3779B97F4A7C15u >> 20 & (room - 1);
        for (; seen[at] != nullptr; at = (at + 1) & (room - 1))
            if (seen[at] == grads[i].out) return RMSNORM_EINVAL;
        seen[at] = grads[i].out;
    }
    return RMSNORM_OK;
}

// One launch's entries, from tensor i on; returns the next one's.
template <int CAP>
int64_t fill(GradTable<CAP> *t, const rmsnorm_grad_t *grads, int64_t i, int64_t n, int threads) {
    t->n = 0;
    t->parts = 0;
    for (; i < n && t->n < CAP; ++i) {
        const rmsnorm_grad_t &g = grads[i];
        if (g.count == 0) continue;
        const uint32_t parts = parts_of(g, threads);
        if (t->n > 0 && parts > (uint32_t)INT_MAX - t->parts) break;
        t->e[t->n++] = GradEntry{static_cast<const char *>(g.grad), static_cast<char *>(g.out), g.count, t->parts,
                                 g.dtype};
        t->parts += parts;
    }
    return i;
}

// Parts of 4 KB that one cluster takes, a warp each, of 8 blocks and of 16 (one
// cluster / two launches, us, device and whole call: one tensor of 1000 2.7 / 5.9;
// 1.6 MB in 20 6.3 and 6.4 / 5.4 and 9.7).
constexpr int64_t kAloneParts = rrn::kClusterMaxCtas * rrn::kGradAlone / 32;
constexpr int64_t kAloneMost = rrn::kGradAloneBlocks * rrn::kGradAlone / 32;

template <int CAP>
int run(const rmsnorm_grad_t *grads, int64_t n, int64_t small_parts, bool clip, float max_norm, float *norm,
        void *workspace, rmsnorm_stream_t stream) {
    int dev = 0, sms = 0, resident = 0;
    int st = rrn::current_device_sms(&dev, &sms);
    if (st != RMSNORM_OK) return st;
    const void *squares = reinterpret_cast<const void *>(&rrn::grad_squares_kernel<CAP>);
    const void *scale = reinterpret_cast<const void *>(&rrn::grad_scale_kernel<CAP>);
    const void *only = reinterpret_cast<const void *>(&rrn::grad_norm_kernel<CAP>);
    GradTable<CAP> t;
    std::memset(&t, 0, offsetof(GradTable<CAP>, e));
    t.partial = static_cast<double *>(workspace);
    t.norm = norm;
    t.max_norm = max_norm;
    t.clip = clip;
    void *argv[] = {&t};
    const void *alone = reinterpret_cast<const void *>(&rrn::grad_alone_kernel<CAP>);
    if (n <= CAP && small_parts <= kAloneMost &&
        (small_parts <= kAloneParts ||
         rrn::large_cluster(dev, alone, rrn::kGradAloneBlocks, rrn::kGradAlone, 0))) {
        fill(&t, grads, 0, n, 32);
        int blocks = 1;
        while (blocks < rrn::kGradAloneBlocks && t.parts > (uint32_t)(blocks * rrn::kGradAlone / 32)) blocks *= 2;
        return rrn::launch_kernel(alone, dim3((unsigned)blocks),
                                  blocks > 1 ? rrn::kGradAlone : 32 * (t.parts > 0 ? (int)t.parts : 1), 0, stream, argv,
                                  blocks);
    }
    if ((st = rrn::resident_blocks(dev, squares, rrn::kGradThreads, 0, &resident)) != RMSNORM_OK) return st;
    // launches of the norm share the partial sums out
    int64_t launches = 0;
    for (int64_t i = 0; i < n; ++launches) i = fill(&t, grads, i, n, rrn::kGradThreads);
    if (launches > rrn::kGradPartials) return RMSNORM_EUNSUPPORTED;
    int64_t most = rrn::kGradPartials / launches;
    if (most > (int64_t)sms * resident) most = (int64_t)sms * resident;
    t.slot = 0;
    for (int64_t i = 0, l = 0; l < launches; ++l) {
        i = fill(&t, grads, i, n, rrn::kGradThreads);
        if (t.parts == 0) continue;
        const unsigned grid = (unsigned)(t.parts < most ? t.parts : most);
        if ((st = rrn::launch_kernel(squares, dim3(grid), rrn::kGradThreads, 0, stream, argv)) != RMSNORM_OK) return st;
        t.slot += (int32_t)grid;
    }
    t.sums = t.slot;
    // the scaling's blocks write the norm; of tensors without elements there are none
    if (!clip || t.sums == 0) return rrn::launch_kernel(only, dim3(1), 32, 0, stream, argv);
    if ((st = rrn::resident_blocks(dev, scale, rrn::kGradThreads, 0, &resident)) != RMSNORM_OK) return st;
    most = (int64_t)sms * resident;
    for (int64_t i = 0, l = 0; l < launches; ++l) {
        i = fill(&t, grads, i, n, rrn::kGradThreads);
        if (t.parts == 0) continue;
        const unsigned grid = (unsigned)(t.parts < most ? t.parts : most);
        if ((st = rrn::launch_kernel(scale, dim3(grid), rrn::kGradThreads, 0, stream, argv)) != RMSNORM_OK) return st;
    }
    return RMSNORM_OK;
}

int norm_and_clip(const rmsnorm_grad_t *grads, int64_t n, bool clip, float max_norm, float *norm, void *workspace,
                  uint64_t workspace_bytes, rmsnorm_stream_t stream) {
    int st = check_grads(grads, n, clip, norm, workspace, workspace_bytes);
    if (st == RMSNORM_OK && clip) st = distinct_outs(grads, n);
    if (st != RMSNORM_OK) return st;
    int64_t parts = 0;
    for (int64_t i = 0; i < n && parts <= kAloneMost; ++i)
        if (grads[i].count > 0) parts += parts_of(grads[i], 32);
    if (n <= rrn::kGradSmall) return run<rrn::kGradSmall>(grads, n, parts, clip, max_norm, norm, workspace, stream);
    if (n <= rrn::kGradSome) return run<rrn::kGradSome>(grads, n, parts, clip, max_norm, norm, workspace, stream);
    return run<rrn::kGradMost>(grads, n, parts, clip, max_norm, norm, workspace, stream);
}

}  // namespace

extern "C" {

int64_t rmsnorm_grad_norm_workspace_bytes(void) { return rrn::kGradPartials * (int64_t)sizeof(double); }

int rmsnorm_grad_norm(const rmsnorm_grad_t *grads, int64_t n, float *norm, void *workspace, uint64_t workspace_bytes,
                      rmsnorm_stream_t stream) {
    return norm_and_clip(grads, n, false, 0.f, norm, workspace, workspace_bytes, stream);
}

int rmsnorm_clip_grads(const rmsnorm_grad_t *grads, int64_t n, float max_norm, float *norm, void *workspace,
                       uint64_t workspace_bytes, rmsnorm_stream_t stream) {
    if (!(max_norm >= 0.f)) return RMSNORM_EINVAL;   // infinity: nothing is clipped
    return norm_and_clip(grads, n, true, max_norm, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
