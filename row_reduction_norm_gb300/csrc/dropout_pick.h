// dropout_pick.h -- the compiled residual-dropout and gradient kernels (internal).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace rrn {

// Threads a row compiled for the register kernels, and chunks a thread: from
// drop_least_ch (with fewer, fewer threads hold the row) to 4, and 6, 8 for the
// forward's 512 threads.
constexpr int kDropGT[6] = {8, 32, 64, 128, 256, 512};
constexpr int drop_least_ch(int gt) { return gt == 8 ? 1 : gt == 32 ? 2 : 3; }

const void *drop_fwd_bf16(int gt, int ch);
const void *drop_fwd_f32(int gt, int ch);
// dw: 0 no gradient of the weight, 1 its partial sums, 2 all of it by a single
// cluster (2 or 4 chunks a thread).
const void *drop_bwd_bf16(int gt, int ch, int dw);
const void *drop_bwd_f32(int gt, int ch, int dw);
// Rows on 16-byte chunks that do not start with one: threads a row, chunks a thread.
struct DropShape {
    int gt, ch;
};
constexpr int kDropShifts = 11, kDropShiftsF32 = 3;   // of these for the fp32 forward
constexpr DropShape kDropShift[kDropShifts] = {{8, 4},   {32, 2},  {32, 4},  {64, 3},  {64, 4}, {128, 3},
                                               {128, 4}, {256, 3}, {256, 4}, {512, 3}, {512, 4}};
const void *drop_fwd_shift(int dtype, int shape);
const void *drop_bwd_shift_bf16(int shape, bool dw);
const void *drop_bwd_shift_f32(int shape, bool dw);
// Rows of single elements in registers: threads a row, elements a thread (the
// second for fp32 alone, whose narrowest rows have 32 classes of columns).
constexpr int kDropScalars = 6;
constexpr DropShape kDropScalar[kDropScalars] = {{64, 4}, {32, 4}, {128, 8}, {256, 8}, {256, 16}, {512, 16}};
const void *drop_fwd_scalar(int dtype, int shape);
const void *drop_bwd_scalar(int dtype, int shape, bool dw);
// Two-pass kernels: blocks of kDropLoopThreads.
constexpr int kDropLoopThreads = 1024;
// Dynamic shared memory of the gradient's kernels whose need follows from the
// width, in steps: it is part of the key under which a kernel's occupancy is
// kept, for every operator of the library, so a process that meets many widths
// must not make a key of each.  The steps cost no resident block: masks are at
// most 8 KB, and of the two-pass kernel's 1024 threads two blocks stand on a SM
// with up to 112 KB each.
constexpr size_t kDropMaskStep = 1024, kDropSumsStep = 16384;
inline size_t drop_smem_in_steps(size_t bytes, size_t step) { return (bytes + step - 1) / step * step; }
// Single elements: two masks, a byte for eight elements, with dropout.
inline size_t drop_scalar_smem(int64_t hidden, bool dropout) {
    return dropout ? drop_smem_in_steps(2 * (size_t)((hidden + 7) / 8), kDropMaskStep) : 0;
}
// Two passes: fp32 sums of the columns, where they are kept there, and a mask.
inline size_t drop_loop_smem(int64_t hidden, bool sums, bool dropout) {
    const size_t mask = dropout ? (size_t)((hidden + 7) / 8) : 0;
    return sums ? drop_smem_in_steps((size_t)hidden * 4 + mask, kDropSumsStep) : drop_smem_in_steps(mask, kDropMaskStep);
}
const void *drop_fwd_loop(int dtype, bool vec);
const void *drop_bwd_loop(int dtype, bool vec, bool dw);

}  // namespace rrn
