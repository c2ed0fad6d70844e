// f32 instantiations of the rotary forward and of the paged append.
#include "rope_kernels.cuh"
#include "rope_pick.h"

namespace rrn {
namespace {

template <typename T, int VE, int K, bool IL, int HD = 0>
const void *one(int mode) {
    switch (mode) {
        case kRopePlain: return reinterpret_cast<const void *>(&rope_kernel<T, VE, K, IL, kRopePlain, HD>);
        case kRopeAppend: return reinterpret_cast<const void *>(&rope_kernel<T, VE, K, IL, kRopeAppend, HD>);
        case kRopeAppendE4m3: return reinterpret_cast<const void *>(&rope_kernel<T, VE, K, IL, kRopeAppendE4m3, HD>);
        case kRopeAppendSettled: return reinterpret_cast<const void *>(&rope_kernel<T, VE, K, IL, kRopeAppendSettled, HD>);
        default: return nullptr;
    }
}

template <typename T, int VE, int K>
const void *mode_of(bool il, int mode) {
    return il ? one<T, VE, K, true>(mode) : one<T, VE, K, false>(mode);
}

}  // namespace

const void *rope_fwd_f32(int shape, bool il, int mode, int whole) {
    if (shape == 0) {
        switch (whole) {
            case 64: return il ? one<F32, 4, 1, true, 64>(mode) : one<F32, 4, 1, false, 64>(mode);
            case 128: return il ? one<F32, 4, 1, true, 128>(mode) : one<F32, 4, 1, false, 128>(mode);
            case 256: return il ? one<F32, 4, 1, true, 256>(mode) : one<F32, 4, 1, false, 256>(mode);
            default: break;
        }
    }
    switch (shape) {
        case 0: return mode_of<F32, 4, 1>(il, mode);
        case 1: return mode_of<F32, 4, 2>(il, mode);
        case 2: return mode_of<F32, 2, 2>(il, mode);
        case 3: return mode_of<F32, 1, 8>(il, mode);
        default: return nullptr;
    }
}

}  // namespace rrn
