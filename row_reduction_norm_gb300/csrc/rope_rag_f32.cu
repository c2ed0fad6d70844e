// f32 instantiations of the rotary kernels for pairs off the 16-byte pieces.
#include "rope_ragged.cuh"
#include "rope_pick.h"

namespace rrn {
namespace {

template <bool IL>
const void *fwd(int mode) {
    switch (mode) {
        case kRopePlain: return reinterpret_cast<const void *>(&rope_ragged_kernel<F32, 4, IL, kRopePlain>);
        case kRopeAppend: return reinterpret_cast<const void *>(&rope_ragged_kernel<F32, 4, IL, kRopeAppend>);
        case kRopeAppendE4m3: return reinterpret_cast<const void *>(&rope_ragged_kernel<F32, 4, IL, kRopeAppendE4m3>);
        default: return nullptr;
    }
}

template <bool IL>
const void *bwd(bool norm) {
    return norm ? reinterpret_cast<const void *>(&rope_ragged_bwd_kernel<F32, 4, IL, true>)
                : reinterpret_cast<const void *>(&rope_ragged_bwd_kernel<F32, 4, IL, false>);
}

}  // namespace

const void *rope_ragged_f32(bool il, int mode) { return il ? fwd<true>(mode) : fwd<false>(mode); }
const void *rope_ragged_bwd_f32(bool il, bool norm) { return il ? bwd<true>(norm) : bwd<false>(norm); }

}  // namespace rrn
