// dropout_pick.h -- the compiled residual-dropout and gradient kernels (internal).
#pragma once

namespace rrn {

// Threads a row compiled for the register kernels, and chunks a thread: 1..4
// for each, and 6, 8 for the forward's 512 threads.
constexpr int kDropGT[6] = {8, 32, 64, 128, 256, 512};

const void *drop_fwd_bf16(int gt, int ch);
const void *drop_fwd_f32(int gt, int ch);
const void *drop_bwd_bf16(int gt, int ch, bool dw);
const void *drop_bwd_f32(int gt, int ch, bool dw);
// Rows of single elements in registers: threads a row, elements a thread.
struct DropScalar {
    int gt, ch;
};
constexpr int kDropScalars = 5;
constexpr DropScalar kDropScalar[kDropScalars] = {{64, 4}, {128, 8}, {256, 8}, {256, 16}, {512, 16}};
const void *drop_fwd_scalar(int dtype, int shape);
const void *drop_bwd_scalar(int dtype, int shape, bool dw);
// Two-pass kernels: blocks of 256 (scalar only) or 1024 threads.
const void *drop_fwd_loop(int dtype, bool vec, int block);
const void *drop_bwd_loop(int dtype, bool vec, int block, bool dw);

}  // namespace rrn
