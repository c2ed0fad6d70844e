// rope_pick.h -- the compiled rotary kernels (internal).
#pragma once

namespace rrn {

// Shapes a head can be held in: VE elements a piece, K units a lane.
struct RopeShape {
    int ve, k;
};
constexpr int kRopeShapes = 5;
constexpr RopeShape kRopeShapesBf16[kRopeShapes] = {{8, 1}, {4, 1}, {4, 2}, {2, 2}, {1, 8}};
constexpr RopeShape kRopeShapesF32[kRopeShapes] = {{4, 1}, {4, 2}, {2, 2}, {1, 8}, {1, 8}};

// mode: RopeMode (rope_kernels.cuh); shape: index into the tables above; whole:
// the head size where heads are turned whole (those of 64, 128 and 256 in
// 16-byte pieces have kernels of their own), else 0.
const void *rope_fwd_bf16(int shape, bool interleaved, int mode, int whole);
const void *rope_fwd_f32(int shape, bool interleaved, int mode, int whole);
const void *rope_bwd_bf16(int shape, bool interleaved, bool norm, int whole);
const void *rope_bwd_f32(int shape, bool interleaved, bool norm, int whole);

// Heads in 16-byte chunks whose pairs do not fall on them (rope_ragged.cuh).
constexpr int kRopeRagged = kRopeShapes;
const void *rope_ragged_bf16(bool interleaved, int mode);
const void *rope_ragged_f32(bool interleaved, int mode);
const void *rope_ragged_bwd_bf16(bool interleaved, bool norm);
const void *rope_ragged_bwd_f32(bool interleaved, bool norm);

}  // namespace rrn
