// dropout_api.cu -- entry points of the residual dropout fused with RMSNorm
// and of RMSNorm's gradient (declared in include/rmsnorm.h): argument checks,
// the choice of a kernel and its grid, the launch.
#include <climits>
#include <cmath>
#include <cstring>

#include "dropout_kernels.cuh"
#include "dropout_pick.h"
#include "dropout_shift.cuh"
#include "launch_util.h"

namespace {

using rrn::div_up;

constexpr int64_t kMaxHidden = 65536;
// Rows the two-pass gradient keeps its sums of dw for in shared memory: 192
// KB of sums and 6 KB of mask bits within the 227 KB of a block.
constexpr int64_t kSmemSums = 49152;   // (208 KB in drop_loop_smem's steps)

// Blocks of the gradient at most: each keeps a row of fp32 sums, which are
// written and read once more.  Four a SM for narrow rows (fp32 1023 x 1001 takes
// 6.5 us with four, 6.6 with three, 7.2 with two), and eight once a block has 16
// of them to read: that is for rows of single elements, in tensors that start off
// the 16-byte boundary (with dropout, eight / four a SM: bf16 32768 x 575 86 /
// 141 us, 65536 x 201 100 / 177, fp32 32768 x 1001 115 / 141).  Aligned rows
// take the same time with either, most of their kernels having fewer blocks
// resident; but the workspace's size is asked for without the addresses.
int64_t most_blocks(int64_t rows, int64_t hidden, int sms) {
    const int64_t few = hidden <= 4096 ? 4 : hidden <= 16384 ? 2 : 1;
    return sms * (hidden <= 1024 && rows >= 16 * 8 * (int64_t)sms ? 8 : few);
}

// Columns of the partial sums' rows.
int64_t partial_ld(int64_t hidden) { return (hidden + 3) / 4 * 4; }

int check_rows(const void *const *ptrs, int n, int64_t rows, int64_t hidden, float eps, float w_bias, const void *w,
               int dtype) {
    if (dtype != RMSNORM_F32 && dtype != RMSNORM_BF16) return RMSNORM_EINVAL;
    if (rows < 0 || hidden <= 0) return RMSNORM_EINVAL;
    if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(w_bias)) return RMSNORM_EINVAL;
    if (hidden > kMaxHidden) return RMSNORM_EUNSUPPORTED;
    if (w_bias != 0.f && w == nullptr) return RMSNORM_EINVAL;
    const int64_t s = rrn::size_of(dtype);
    if (rows > INT64_MAX / 8 / (hidden * s)) return RMSNORM_EINVAL;
    for (int i = 0; i < n; ++i)
        if (!rrn::on_boundary(ptrs[i], s)) return RMSNORM_EINVAL;
    return RMSNORM_OK;
}

bool vec_ok(const void *const *ptrs, int n, int64_t hidden, int dtype) {
    if (hidden * rrn::size_of(dtype) % 16 != 0) return false;
    for (int i = 0; i < n; ++i)
        if (!rrn::on_boundary(ptrs[i], 16)) return false;
    return true;
}

// Dropout probability as the 16-bit threshold it is rounded to.
int threshold_of(float p, uint32_t *thr) {
    if (!(p >= 0.f) || !(p < 1.f)) return RMSNORM_EINVAL;
    const double t = std::floor((double)p * 65536.0 + 0.5);
    if (t > 65535.0) return RMSNORM_EINVAL;
    *thr = (uint32_t)t;
    return RMSNORM_OK;
}

// Threads a row (of those compiled) and chunks a thread that hold `nch`
// chunks, about four a thread; false when they are too many.
bool reg_shape(int64_t nch, int max_ch, int *gt, int *ch) {
    for (int g : rrn::kDropGT) {
        const int64_t need = div_up(nch, g);
        if (need <= 4) {
            *gt = g;
            *ch = (int)need;
            return true;
        }
        if (g == 512 && need <= max_ch) {
            *gt = g;
            *ch = need <= 6 ? 6 : 8;
            return true;
        }
    }
    return false;
}

// Of the shifted kernels' shapes, the first that holds a row of this width
// wherever it starts, or kDropShifts.
int shift_holding(int64_t hidden, int dtype) {
    const int64_t V = 16 / rrn::size_of(dtype), chunks = (hidden + 2 * V - 2) / V;
    int i = 0;
    while (i < rrn::kDropShifts && chunks > (int64_t)rrn::kDropShift[i].gt * rrn::kDropShift[i].ch) ++i;
    return i;
}

// The kernel for rows of a length that is no multiple of 16 bytes, in tensors
// that start on a 16-byte boundary, that holds a row's chunks; or -1 where the
// rows of single elements are faster.  Starting costs the former more (weights
// an element at a time, blocks of several rows) and a row less.  Measured on
// GB300, us, shifted / single elements, dropout 0.1:
//   gradient  bf16 501 x 608 rows 5.2 / 5.5, 1001 x 608 7.4 / 6.6, x 2000 11.7 /
//             12.2, 2047 x 608 9.0 / 8.6, 8191 x 6000 130 / 257; fp32 501 x 608
//             5.8 / 5.1, x 2000 8.4 / 8.8, 1001 x 2000 17.8 / 13.0, x 6000 30.6 /
//             30.7, 3001 x 152 6.6 / 7.6, x 6000 70 / 89; and with a third of
//             the chunks unused, 2047 x 6000 60.0 / 49.3
//   forward   bf16 101 x 2000 4.3 / 3.1, x 6000 5.4 / 6.6, 2047 x 2000 12.8 /
//             11.7, x 6000 30.0 / 32.2, 3001 x 608 6.7 / 7.9, 12001 x 6000 132 /
//             391; fp32 101 x 6000 4.8 / 6.6, 501 x 6000 10.8 / 12.0, and wider
//             rows no faster (1001 x 6000 20.0 / 17.5, 4095 x 6000 93 / 66)
// Rows have the same bits from either (row_classes.cuh).
int shift_shape(const void *const *ptrs, int n, int64_t rows, int64_t hidden, int dtype, bool gradient) {
    for (int i = 0; i < n; ++i)
        if (!rrn::on_boundary(ptrs[i], 16)) return -1;
    const bool bf16 = dtype == RMSNORM_BF16;
    if (gradient) {
        if (!(hidden > 2048 || (hidden <= 512 && rows >= 1024) || rows >= (bf16 ? 1 << 20 : 1 << 22) / hidden)) return -1;
    } else if (!(rows >= 4096 || (bf16 && hidden > 2048))) {
        return -1;
    }
    const int i = shift_holding(hidden, dtype);
    if (i >= (bf16 || gradient ? rrn::kDropShifts : rrn::kDropShiftsF32)) return -1;
    const int64_t V = 16 / rrn::size_of(dtype), chunks = (hidden + 2 * V - 2) / V;
    return bf16 || hidden <= 512 || 10 * chunks >= 7 * (int64_t)rrn::kDropShift[i].gt * rrn::kDropShift[i].ch ? i : -1;
}

// Blocks of `groups` row groups in all, at most `most`, that keep a thread's
// rows equally far past a boundary: a multiple of 8 (any row count is) when
// they take more than one group each.
int64_t shift_blocks(int64_t groups, int64_t most) { return groups <= most ? groups : most < 8 ? 8 : most / 8 * 8; }

// The rows-of-single-elements kernel that holds a row, or -1, and its classes
// of columns a thread: those of the shifted kernel for the width, so that the
// rows have the same bits from either (up to 2048 columns, where the number of
// rows decides between the two).
int scalar_shape(bool vec, int64_t hidden, int dtype, int32_t *classes) {
    if (vec) return -1;
    const int held = shift_holding(hidden, dtype);
    const int64_t all = held < rrn::kDropShifts ? rrn::kDropShift[held].gt * 16 / rrn::size_of(dtype) : INT64_MAX;
    for (int i = 0; i < rrn::kDropScalars; ++i) {
        const int64_t gt = rrn::kDropScalar[i].gt;
        if (hidden > gt * rrn::kDropScalar[i].ch || gt > all) continue;
        const int64_t most = hidden <= 2048 ? 4 : gt < 512 ? 2 : 1;
        *classes = (int32_t)(all / gt < most ? all / gt : most);
        return i;
    }
    return -1;
}

void fill(rrn::DropParams *p, const void *w, int64_t rows, int64_t hidden, float eps, float w_bias, uint32_t thr,
          const uint64_t *rng, int dtype) {
    std::memset(p, 0, sizeof(*p));
    p->w = w;
    p->rng = rng;
    p->rows = rows;
    p->row_elems = hidden;
    p->row_bytes = hidden * rrn::size_of(dtype);
    p->blocks_per_row = div_up(hidden, 8);
    p->thr = thr;
    p->scale = (float)(65536.0 / (65536.0 - (double)thr));
    p->hidden_f = (float)hidden;
    p->eps = eps;
    p->w_bias = w_bias;
}

int backward(const void *dy, const void *h, const void *w, const void *dh, void *dres, void *dx, void *dw, int64_t rows,
             int64_t hidden, float eps, float w_bias, uint32_t thr, const uint64_t *rng, int dtype, void *workspace,
             uint64_t workspace_bytes, rmsnorm_stream_t stream) {
    const void *ptrs[] = {dy, h, w, dh, dres, dx, dw};
    int st = check_rows(ptrs, 7, rows, hidden, eps, w_bias, w, dtype);
    if (st != RMSNORM_OK) return st;
    if (dw != nullptr && w == nullptr) return RMSNORM_EINVAL;
    if (rows > 0 && (dy == nullptr || h == nullptr || dres == nullptr || dx == dres)) return RMSNORM_EINVAL;
    if (rows == 0 && dw == nullptr) return RMSNORM_OK;
    int dev = 0, sms = 0;
    if ((st = rrn::current_device_sms(&dev, &sms)) != RMSNORM_OK) return st;
    const int64_t most = most_blocks(rows, hidden, sms);
    if (dw != nullptr && (workspace == nullptr || !rrn::on_boundary(workspace, 16) ||
                          workspace_bytes < (uint64_t)rmsnorm_bwd_workspace_bytes(rows, hidden, dtype)))
        return RMSNORM_EINVAL;
    int64_t blocks = 0;
    if (rows > 0) {
        rrn::DropParams p;
        fill(&p, w, rows, hidden, eps, w_bias, thr, rng, dtype);
        p.dy = dy;
        p.h = h;
        p.dh = dh;
        p.dres = dres;
        p.dx = dx;
        p.partial = static_cast<float *>(workspace);
        p.partial_ld = partial_ld(hidden);
        const bool vec = vec_ok(ptrs, 6, hidden, dtype);
        const int V = 16 / rrn::size_of(dtype);
        p.units = (int32_t)(vec ? hidden / V : hidden);
        const void *fn;
        int threads, gt = 0, ch = 0;
        int64_t groups = rows;
        size_t smem = 0;
        // the weight may stand anywhere: it is read an element at a time
        const void *rows_of[] = {dy, h, dh, dres, dx};
        const int shift = vec ? -1 : shift_shape(rows_of, 5, rows, hidden, dtype, true);
        if (vec && reg_shape(hidden / V, 4, &gt, &ch)) {
            threads = rrn::drop_block_threads(gt);
            groups = div_up(rows, threads / gt);
            const int part = dw == nullptr ? 0 : groups <= rrn::kFinishBlocks ? 2 : 1;
            if (part == 2) ch = ch <= 2 ? 2 : 4;
            fn = dtype == RMSNORM_BF16 ? rrn::drop_bwd_bf16(gt, ch, part) : rrn::drop_bwd_f32(gt, ch, part);
            smem = (size_t)rrn::drop_ring_bytes(gt, ch);
        } else if (shift >= 0) {
            gt = rrn::kDropShift[shift].gt;
            fn = dtype == RMSNORM_BF16 ? rrn::drop_bwd_shift_bf16(shift, dw != nullptr)
                                       : rrn::drop_bwd_shift_f32(shift, dw != nullptr);
            threads = rrn::drop_block_threads(gt);
            groups = div_up(rows, threads / gt);
            smem = (size_t)rrn::shift_ring_bytes(gt, rrn::kDropShift[shift].ch);
        } else if (const int shape = scalar_shape(vec, hidden, dtype, &p.classes); shape >= 0) {
            threads = rrn::kDropScalar[shape].gt;
            fn = rrn::drop_bwd_scalar(dtype, shape, dw != nullptr);
            smem = rrn::drop_scalar_smem(hidden, thr != 0);
        } else {
            threads = rrn::kDropLoopThreads;
            fn = rrn::drop_bwd_loop(dtype, vec, dw != nullptr);
            p.acc_in_smem = dw != nullptr && hidden <= kSmemSums;
            smem = rrn::drop_loop_smem(hidden, p.acc_in_smem, thr != 0);
        }
        if (fn == nullptr) return RMSNORM_EINVAL;
        if (smem > rrn::kSmemUnasked && (st = rrn::allow_smem(dev, fn)) != RMSNORM_OK) return st;
        int resident = 0;
        if ((st = rrn::resident_blocks(dev, fn, threads, smem, &resident)) != RMSNORM_OK) return st;
        blocks = (int64_t)sms * resident;
        if (dw != nullptr && blocks > most) blocks = most;
        // few row groups, a block each: a single cluster, which adds dw up itself
        const bool alone = dw != nullptr && groups <= rrn::kFinishBlocks;
        blocks = shift >= 0 ? shift_blocks(groups, blocks) : blocks > groups ? groups : blocks;
        if (alone) p.dw = dw;
        void *argv[] = {&p};
        st = rrn::launch_kernel(fn, dim3((unsigned)blocks), threads, smem, stream, argv, alone ? (int)blocks : 1);
        if (st != RMSNORM_OK || alone) return st;
    }
    if (dw == nullptr) return RMSNORM_OK;
    return rrn::launch_colsum(static_cast<const float *>(workspace), (int)blocks, 0, hidden, partial_ld(hidden), dw, nullptr,
                              dtype, stream);
}

}  // namespace

extern "C" {

int rmsnorm_dropout_fwd(const void *x, const void *residual, const void *w, void *y, void *residual_out, int64_t rows,
                        int64_t hidden, float eps, float weight_bias, float p_drop, const uint64_t *rng, int dtype,
                        rmsnorm_stream_t stream) {
    const void *ptrs[] = {x, residual, w, y, residual_out};
    int st = check_rows(ptrs, 5, rows, hidden, eps, weight_bias, w, dtype);
    if (st != RMSNORM_OK) return st;
    uint32_t thr = 0;
    if ((st = threshold_of(p_drop, &thr)) != RMSNORM_OK) return st;
    if (rows == 0) return RMSNORM_OK;
    if (x == nullptr || residual == nullptr || y == nullptr || residual_out == nullptr || y == residual_out)
        return RMSNORM_EINVAL;
    if (thr != 0 && (rng == nullptr || !rrn::on_boundary(rng, 8))) return RMSNORM_EINVAL;
    rrn::DropParams p;
    fill(&p, w, rows, hidden, eps, weight_bias, thr, rng, dtype);
    p.x = x;
    p.res = residual;
    p.y = y;
    p.h_out = residual_out;
    const bool vec = vec_ok(ptrs, 5, hidden, dtype);
    const int V = 16 / rrn::size_of(dtype);
    p.units = (int32_t)(vec ? hidden / V : hidden);
    const void *fn;
    int threads, gt = 0, ch = 0;
    int64_t blocks = rows;
    size_t smem = 0;
    const void *rows_of[] = {x, residual, y, residual_out};
    const int shift = vec ? -1 : shift_shape(rows_of, 4, rows, hidden, dtype, false);
    if (vec && reg_shape(hidden / V, 8, &gt, &ch)) {
        fn = dtype == RMSNORM_BF16 ? rrn::drop_fwd_bf16(gt, ch) : rrn::drop_fwd_f32(gt, ch);
        threads = rrn::drop_block_threads(gt);
        blocks = div_up(rows, threads / gt);
    } else if (shift >= 0) {
        gt = rrn::kDropShift[shift].gt;
        fn = rrn::drop_fwd_shift(dtype, shift);
        threads = rrn::drop_block_threads(gt);
        if (fn == nullptr) return RMSNORM_EINVAL;
        int dev = 0, sms = 0, resident = 0;
        if ((st = rrn::current_device_sms(&dev, &sms)) != RMSNORM_OK) return st;
        if ((st = rrn::resident_blocks(dev, fn, threads, 0, &resident)) != RMSNORM_OK) return st;
        blocks = shift_blocks(div_up(rows, threads / gt), (int64_t)sms * resident);
    } else if (const int shape = scalar_shape(vec, hidden, dtype, &p.classes); shape >= 0) {
        threads = rrn::kDropScalar[shape].gt;
        fn = rrn::drop_fwd_scalar(dtype, shape);
        smem = (size_t)(thr ? p.blocks_per_row : 0);
    } else {
        threads = rrn::kDropLoopThreads;
        fn = rrn::drop_fwd_loop(dtype, vec);
        smem = (size_t)(thr ? p.blocks_per_row : 0);
    }
    if (fn == nullptr) return RMSNORM_EINVAL;
    if (blocks > INT_MAX) blocks = INT_MAX;
    void *argv[] = {&p};
    return rrn::launch_kernel(fn, dim3((unsigned)blocks), threads, smem, stream, argv);
}

int64_t rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t hidden, int dtype) {
    if ((dtype != RMSNORM_F32 && dtype != RMSNORM_BF16) || rows < 0 || hidden <= 0) return RMSNORM_EINVAL;
    if (hidden > kMaxHidden) return RMSNORM_EUNSUPPORTED;
    int dev = 0, sms = 0;
    const int st = rrn::current_device_sms(&dev, &sms);
    if (st != RMSNORM_OK) return st;
    int64_t blocks = most_blocks(rows, hidden, sms);
    if (blocks > rows) blocks = rows > 0 ? rows : 1;
    return blocks * partial_ld(hidden) * (int64_t)sizeof(float);
}

int rmsnorm_bwd(const void *dy, const void *h, const void *w, const void *dresidual_out, void *dx, void *dw,
                int64_t rows, int64_t hidden, float eps, float weight_bias, int dtype, void *workspace,
                uint64_t workspace_bytes, rmsnorm_stream_t stream) {
    return backward(dy, h, w, dresidual_out, dx, nullptr, dw, rows, hidden, eps, weight_bias, 0, nullptr, dtype,
                    workspace, workspace_bytes, stream);
}

int rmsnorm_dropout_bwd(const void *dy, const void *h, const void *w, const void *dresidual_out, void *dresidual,
                        void *dx, void *dw, int64_t rows, int64_t hidden, float eps, float weight_bias, float p_drop,
                        const uint64_t *rng, int dtype, void *workspace, uint64_t workspace_bytes,
                        rmsnorm_stream_t stream) {
    uint32_t thr = 0;
    const int st = threshold_of(p_drop, &thr);
    if (st != RMSNORM_OK) return st;
    if (rows > 0 && (dx == nullptr || (thr != 0 && (rng == nullptr || !rrn::on_boundary(rng, 8)))))
        return RMSNORM_EINVAL;
    return backward(dy, h, w, dresidual_out, dresidual, dx, dw, rows, hidden, eps, weight_bias, thr, rng, dtype,
                    workspace, workspace_bytes, stream);
}

}  // extern "C"
