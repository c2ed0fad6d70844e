// Instantiations of the RMSNorm gradient, fp32 rows whose length is no multiple
// of 16 bytes.
#include "dropout_pick.h"
#include "dropout_shift.cuh"

namespace rrn {
namespace {

template <bool DW, int I = 0>
const void *of_shape(int shape) {
    if constexpr (I == kDropShifts) return nullptr;
    else if (shape == I) return reinterpret_cast<const void *>(&drop_bwd_shift_kernel<F32, kDropShift[I].gt, kDropShift[I].ch, DW>);
    else return of_shape<DW, I + 1>(shape);
}

}  // namespace

const void *drop_bwd_shift_f32(int shape, bool dw) { return dw ? of_shape<true>(shape) : of_shape<false>(shape); }

}  // namespace rrn
