// Instantiations of the residual dropout and of the RMSNorm gradient for rows
// of single elements.
#include "dropout_kernels.cuh"
#include "dropout_pick.h"

namespace rrn {
namespace {

template <typename T>
const void *fwd(int shape) {
    switch (shape) {
        case 0: return reinterpret_cast<const void *>(&drop_fwd_scalar_kernel<T, 64, 4>);
        case 1: return reinterpret_cast<const void *>(&drop_fwd_scalar_kernel<T, 128, 8>);
        case 2: return reinterpret_cast<const void *>(&drop_fwd_scalar_kernel<T, 256, 8>);
        case 3: return reinterpret_cast<const void *>(&drop_fwd_scalar_kernel<T, 256, 16>);
        case 4: return reinterpret_cast<const void *>(&drop_fwd_scalar_kernel<T, 512, 16>);
        default: return nullptr;
    }
}

template <typename T, bool DW>
const void *bwd(int shape) {
    switch (shape) {
        case 0: return reinterpret_cast<const void *>(&drop_bwd_scalar_kernel<T, 64, 4, DW>);
        case 1: return reinterpret_cast<const void *>(&drop_bwd_scalar_kernel<T, 128, 8, DW>);
        case 2: return reinterpret_cast<const void *>(&drop_bwd_scalar_kernel<T, 256, 8, DW>);
        case 3: return reinterpret_cast<const void *>(&drop_bwd_scalar_kernel<T, 256, 16, DW>);
        case 4: return reinterpret_cast<const void *>(&drop_bwd_scalar_kernel<T, 512, 16, DW>);
        default: return nullptr;
    }
}

}  // namespace

const void *drop_fwd_scalar(int dtype, int shape) { return dtype == 1 ? fwd<BF16>(shape) : fwd<F32>(shape); }

const void *drop_bwd_scalar(int dtype, int shape, bool dw) {
    if (dtype == 1) return dw ? bwd<BF16, true>(shape) : bwd<BF16, false>(shape);
    return dw ? bwd<F32, true>(shape) : bwd<F32, false>(shape);
}

}  // namespace rrn
