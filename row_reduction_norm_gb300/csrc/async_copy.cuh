// async_copy.cuh -- per-thread asynchronous copies from global to shared
// memory: a thread waits for its own copies only and reads back its own
// places, so a ring of them needs no barrier.
#pragma once

#include <stdint.h>

namespace rrn {

// BYTES: 4, 8 or 16, both addresses aligned to it.  16 bytes pass L1 by unless
// it is asked for (narrower ones cannot): a warp that reads half of each
// 32-byte sector and then the other half fetches it twice without it (the
// gradient of 8192 tokens x 40 interleaved heads of 128: 66.8 us, 45.9 with L1).
template <int BYTES, bool L1 = false>
__device__ __forceinline__ void copy_async(void *smem, const void *global) {
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(smem);
    if constexpr (BYTES == 16 && !L1)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" : : "r"(to), "l"(global) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" : : "r"(to), "l"(global), "n"(BYTES) : "memory");
}
// The first `bytes` of 16, zeros after them.
__device__ __forceinline__ void copy_async_part(void *smem, const void *global, uint32_t bytes) {
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(smem);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" : : "r"(to), "l"(global), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most PENDING of the thread's groups are on their way.
template <int PENDING>
__device__ __forceinline__ void copy_async_wait() {
    asm volatile("cp.async.wait_group %0;" : : "n"(PENDING) : "memory");
}

}  // namespace rrn
