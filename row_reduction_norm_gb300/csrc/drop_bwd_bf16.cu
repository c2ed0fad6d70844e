// bf16 register-kernel instantiations of the RMSNorm gradient.
#include "dropout_kernels.cuh"
#include "dropout_pick.h"

namespace rrn {
namespace {

template <typename T, int GT, bool DW>
const void *of_ch(int ch) {
    if constexpr (drop_least_ch(GT) <= 1)
        if (ch == 1) return reinterpret_cast<const void *>(&drop_bwd_kernel<T, GT, 1, DW>);
    if constexpr (drop_least_ch(GT) <= 2)
        if (ch == 2) return reinterpret_cast<const void *>(&drop_bwd_kernel<T, GT, 2, DW>);
    switch (ch) {
        case 3: return reinterpret_cast<const void *>(&drop_bwd_kernel<T, GT, 3, DW>);
        case 4: return reinterpret_cast<const void *>(&drop_bwd_kernel<T, GT, 4, DW>);
        default: return nullptr;
    }
}

template <typename T, int GT>
const void *of_dw(int ch, int dw) {
    if constexpr (drop_least_ch(GT) <= 2)
        if (dw == 2 && ch == 2) return reinterpret_cast<const void *>(&drop_bwd_kernel<T, GT, 2, true, true>);
    if (dw == 2) return ch == 4 ? reinterpret_cast<const void *>(&drop_bwd_kernel<T, GT, 4, true, true>) : nullptr;
    return dw ? of_ch<T, GT, true>(ch) : of_ch<T, GT, false>(ch);
}

}  // namespace

const void *drop_bwd_bf16(int gt, int ch, int dw) {
    switch (gt) {
        case 8: return of_dw<BF16, 8>(ch, dw);
        case 32: return of_dw<BF16, 32>(ch, dw);
        case 64: return of_dw<BF16, 64>(ch, dw);
        case 128: return of_dw<BF16, 128>(ch, dw);
        case 256: return of_dw<BF16, 256>(ch, dw);
        case 512: return of_dw<BF16, 512>(ch, dw);
        default: return nullptr;
    }
}

}  // namespace rrn
