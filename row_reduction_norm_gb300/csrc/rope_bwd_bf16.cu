// bf16 instantiations of the rotary forward's gradient.
#include "rope_kernels.cuh"
#include "rope_pick.h"

namespace rrn {
namespace {

template <typename T, int VE, int K, bool IL>
const void *one(bool norm) {
    return norm ? reinterpret_cast<const void *>(&rope_bwd_kernel<T, VE, K, IL, true>)
                : reinterpret_cast<const void *>(&rope_bwd_kernel<T, VE, K, IL, false>);
}

}  // namespace

const void *rope_bwd_bf16(int shape, bool il, bool norm) {
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
