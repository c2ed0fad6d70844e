// Two-pass instantiations of the residual dropout and of the RMSNorm gradient.
#include "dropout_kernels.cuh"
#include "dropout_pick.h"

namespace rrn {
namespace {

template <typename T>
const void *fwd(bool vec) {
    return vec ? reinterpret_cast<const void *>(&drop_fwd_loop_kernel<T, T::kVec, kDropLoopThreads>)
               : reinterpret_cast<const void *>(&drop_fwd_loop_kernel<T, 1, kDropLoopThreads>);
}

template <typename T, bool DW>
const void *bwd(bool vec) {
    return vec ? reinterpret_cast<const void *>(&drop_bwd_loop_kernel<T, T::kVec, kDropLoopThreads, DW>)
               : reinterpret_cast<const void *>(&drop_bwd_loop_kernel<T, 1, kDropLoopThreads, DW>);
}

}  // namespace

const void *drop_fwd_loop(int dtype, bool vec) { return dtype == 1 ? fwd<BF16>(vec) : fwd<F32>(vec); }

const void *drop_bwd_loop(int dtype, bool vec, bool dw) {
    if (dtype == 1) return dw ? bwd<BF16, true>(vec) : bwd<BF16, false>(vec);
    return dw ? bwd<F32, true>(vec) : bwd<F32, false>(vec);
}

}  // namespace rrn
