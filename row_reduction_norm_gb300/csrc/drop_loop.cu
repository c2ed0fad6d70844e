// Two-pass instantiations of the residual dropout and of the RMSNorm gradient.
#include "dropout_kernels.cuh"
#include "dropout_pick.h"

namespace rrn {
namespace {

template <typename T>
const void *fwd(bool vec, int block) {
    if (vec) return block == 1024 ? reinterpret_cast<const void *>(&drop_fwd_loop_kernel<T, T::kVec, 1024>) : nullptr;
    return block == 1024 ? reinterpret_cast<const void *>(&drop_fwd_loop_kernel<T, 1, 1024>)
                         : reinterpret_cast<const void *>(&drop_fwd_loop_kernel<T, 1, 256>);
}

template <typename T, bool DW>
const void *bwd(bool vec, int block) {
    if (vec)
        return block == 1024 ? reinterpret_cast<const void *>(&drop_bwd_loop_kernel<T, T::kVec, 1024, DW>) : nullptr;
    return block == 1024 ? reinterpret_cast<const void *>(&drop_bwd_loop_kernel<T, 1, 1024, DW>)
                         : reinterpret_cast<const void *>(&drop_bwd_loop_kernel<T, 1, 256, DW>);
}

}  // namespace

const void *drop_fwd_loop(int dtype, bool vec, int block) {
    return dtype == 1 ? fwd<BF16>(vec, block) : fwd<F32>(vec, block);
}

const void *drop_bwd_loop(int dtype, bool vec, int block, bool dw) {
    if (dtype == 1) return dw ? bwd<BF16, true>(vec, block) : bwd<BF16, false>(vec, block);
    return dw ? bwd<F32, true>(vec, block) : bwd<F32, false>(vec, block);
}

}  // namespace rrn
