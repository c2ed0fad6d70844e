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

// Floats of shared memory the gradient holds a head's weights in: 32 lanes of
// K units of 2 VE elements.
inline int rope_weight_floats(int dtype, int shape) {
    const RopeShape s = dtype == 1 ? kRopeShapesBf16[shape] : kRopeShapesF32[shape];
    return 64 * s.k * s.ve;
}

// mode: RopeMode (rope_kernels.cuh); shape: index into the tables above.
const void *rope_fwd_bf16(int shape, bool interleaved, int mode);
const void *rope_fwd_f32(int shape, bool interleaved, int mode);
const void *rope_bwd_bf16(int shape, bool interleaved, bool norm);
const void *rope_bwd_f32(int shape, bool interleaved, bool norm);

}  // namespace rrn
