// f32 instantiations of the rotary forward's gradient.
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

const void *rope_bwd_f32(int shape, bool il, bool norm) {
    switch (shape) {
        case 0: return il ? one<F32, 4, 1, true>(norm) : one<F32, 4, 1, false>(norm);
        case 1: return il ? one<F32, 4, 2, true>(norm) : one<F32, 4, 2, false>(norm);
        case 2: return il ? one<F32, 2, 2, true>(norm) : one<F32, 2, 2, false>(norm);
        case 3: return il ? one<F32, 1, 8, true>(norm) : one<F32, 1, 8, false>(norm);
        default: return nullptr;
    }
}

}  // namespace rrn
