// logprobs_pick.h -- shared memory of the log probability kernels (internal;
// plain C++ too, so that it can be checked on the host).
#pragma once

#include <stddef.h>

namespace rrn {

// Bytes that a block asks for: three numbers of each of its rows' units, in
// steps, since the amount is part of the key under which a kernel's occupancy is
// kept for every operator of the library and a process that meets many
// vocabularies must not make a key of each.  The steps cost no resident block:
// registers allow four on a SM, and those need less than 40 KB each.
constexpr size_t kLpSmemStep = 4096;
inline size_t lp_smem(int units, int rows) {
    return ((size_t)units * 12 * (size_t)rows + kLpSmemStep - 1) / kLpSmemStep * kLpSmemStep;
}

}  // namespace rrn
