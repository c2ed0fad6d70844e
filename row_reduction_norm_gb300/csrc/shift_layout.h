// shift_layout.h -- how a row of a width that is no multiple of 16 bytes lies
// on the aligned 16-byte chunks of its tensor (internal; plain C++ too, so
// that the bounds can be checked on the host).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define RRN_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define RRN_HOST_DEVICE inline
#endif

namespace rrn {

// Elements of the row before in a row's first chunk, the row's chunks, its
// elements in the last one.
template <int V>
struct ShiftedRow {
    int s, chunks, tail;
    RRN_HOST_DEVICE void set(int64_t row, int64_t hidden) {
        s = (int)(((row & (V - 1)) * (hidden & (V - 1))) & (V - 1));
        chunks = (int)((s + hidden + V - 1) / V);
        tail = (int)(s + hidden - (int64_t)(chunks - 1) * V);
    }
    // Elements lo .. hi - 1 of chunk u are the row's.
    RRN_HOST_DEVICE int lo(int u) const { return u == 0 ? s : 0; }
    RRN_HOST_DEVICE int hi(int u) const { return u == chunks - 1 ? tail : V; }
    // Whether all of chunk u lies within the tensor.  The chunk may hold several
    // rows, or parts of them (rows narrower than a chunk), so this counts
    // elements to the tensor's end, not rows behind this one.
    RRN_HOST_DEVICE bool whole(int u, int64_t row, int64_t rows, int64_t hidden) const {
        return (int64_t)(u + 1) * V <= s + (rows - row) * hidden;
    }
};

}  // namespace rrn
