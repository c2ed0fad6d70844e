// Instantiations of the residual dropout for rows whose length is no multiple
// of 16 bytes.
#include "dropout_pick.h"
#include "dropout_shift.cuh"

namespace rrn {
namespace {

template <typename T, int I = 0>
const void *of_shape(int shape) {
    if constexpr (I == (T::kVec == 8 ? kDropShifts : kDropShiftsF32)) return nullptr;
    else if (shape == I) return reinterpret_cast<const void *>(&drop_fwd_shift_kernel<T, kDropShift[I].gt, kDropShift[I].ch>);
    else return of_shape<T, I + 1>(shape);
}

}  // namespace

const void *drop_fwd_shift(int dtype, int shape) { return dtype == 1 ? of_shape<BF16>(shape) : of_shape<F32>(shape); }

}  // namespace rrn
