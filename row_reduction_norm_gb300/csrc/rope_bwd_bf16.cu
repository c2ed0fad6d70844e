// bf16 instantiations of the rotary forward's gradient.
#include "rope_kernels.cuh"
#include "rope_pick.h"

namespace rrn {
namespace {

template <typename T, int VE, int K, bool IL, int HD = 0>
const void *one(bool norm) {
    return norm ? reinterpret_cast<const void *>(&rope_bwd_kernel<T, VE, K, IL, true, HD>)
                : reinterpret_cast<const void *>(&rope_bwd_kernel<T, VE, K, IL, false, HD>);
}

}  // namespace

const void *rope_bwd_bf16(int shape, bool il, bool norm, int whole) {
    if (shape == 0) {
        switch (whole) {
            case 64: return il ? one<BF16, 8, 1, true, 64>(norm) : one<BF16, 8, 1, false, 64>(norm);
            case 128: return il ? one<BF16, 8, 1, true, 128>(norm) : one<BF16, 8, 1, false, 128>(norm);
            case 256: return il ? one<BF16, 8, 1, true, 256>(norm) : one<BF16, 8, 1, false, 256>(norm);
            default: break;
        }
    }
    switch (shape) {
        case 0: return il ? one<BF16, 8, 1, true>(norm) : one<BF16, 8, 1, false>(norm);
        case 1: return il ? one<BF16, 4, 1, true>(norm) : one<BF16, 4, 1, false>(norm);
        case 2: return il ? one<BF16, 4, 2, true>(norm) : one<BF16, 4, 2, false>(norm);
        case 3: return il ? one<BF16, 2, 2, true>(norm) : one<BF16, 2, 2, false>(norm);
        case 4: return il ? one<BF16, 1, 8, true>(norm) : one<BF16, 1, 8, false>(norm);
        default: return nullptr;
    }
}

}  // namespace rrn
