// dropout_pick.h -- the compiled residual-dropout and gradient kernels (internal).
#pragma once

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
const void *drop_fwd_loop(int dtype, bool vec);
const void *drop_bwd_loop(int dtype, bool vec, bool dw);

}  // namespace rrn
