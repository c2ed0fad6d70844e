// bf16 register-kernel instantiations of the residual dropout's forward.
#include "dropout_kernels.cuh"
#include "dropout_pick.h"

namespace rrn {
namespace {

template <typename T, int GT>
const void *of_ch(int ch) {
    if constexpr (drop_least_ch(GT) <= 1)
        if (ch == 1) return reinterpret_cast<const void *>(&drop_fwd_kernel<T, GT, 1>);
    if constexpr (drop_least_ch(GT) <= 2)
        if (ch == 2) return reinterpret_cast<const void *>(&drop_fwd_kernel<T, GT, 2>);
    switch (ch) {
        case 3: return reinterpret_cast<const void *>(&drop_fwd_kernel<T, GT, 3>);
        case 4: return reinterpret_cast<const void *>(&drop_fwd_kernel<T, GT, 4>);
        default: return nullptr;
    }
}

}  // namespace

const void *drop_fwd_bf16(int gt, int ch) {
    if (gt == 512 && ch == 6) return reinterpret_cast<const void *>(&drop_fwd_kernel<BF16, 512, 6>);
    if (gt == 512 && ch == 8) return reinterpret_cast<const void *>(&drop_fwd_kernel<BF16, 512, 8>);
    switch (gt) {
        case 8: return of_ch<BF16, 8>(ch);
        case 32: return of_ch<BF16, 32>(ch);
        case 64: return of_ch<BF16, 64>(ch);
        case 128: return of_ch<BF16, 128>(ch);
        case 256: return of_ch<BF16, 256>(ch);
        case 512: return of_ch<BF16, 512>(ch);
        default: return nullptr;
    }
}

}  // namespace rrn
