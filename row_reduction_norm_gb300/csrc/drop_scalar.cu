// Instantiations of the residual dropout and of the RMSNorm gradient for rows
// of single elements.
#include "dropout_kernels.cuh"
#include "dropout_pick.h"

namespace rrn {
namespace {

template <typename T, int I = 0>
const void *fwd(int shape) {
    constexpr bool narrow = I == 1;   // fp32 alone
    if constexpr (I == kDropScalars) return nullptr;
    else if constexpr (narrow && T::kVec == 8) return fwd<T, I + 1>(shape);
    else if (shape == I) return reinterpret_cast<const void *>(&drop_fwd_scalar_kernel<T, kDropScalar[I].gt, kDropScalar[I].ch>);
    else return fwd<T, I + 1>(shape);
}

template <typename T, bool DW, int I = 0>
const void *bwd(int shape) {
    constexpr bool narrow = I == 1;
    if constexpr (I == kDropScalars) return nullptr;
    else if constexpr (narrow && T::kVec == 8) return bwd<T, DW, I + 1>(shape);
    else if (shape == I) return reinterpret_cast<const void *>(&drop_bwd_scalar_kernel<T, kDropScalar[I].gt, kDropScalar[I].ch, DW>);
    else return bwd<T, DW, I + 1>(shape);
}

}  // namespace

const void *drop_fwd_scalar(int dtype, int shape) { return dtype == 1 ? fwd<BF16>(shape) : fwd<F32>(shape); }

const void *drop_bwd_scalar(int dtype, int shape, bool dw) {
    if (dtype == 1) return dw ? bwd<BF16, true>(shape) : bwd<BF16, false>(shape);
    return dw ? bwd<F32, true>(shape) : bwd<F32, false>(shape);
}

}  // namespace rrn
