// key_search.h -- which logits the search for a row's largest gathers, and how
// its bound goes from round to round (internal; plain C++ too, so that it can be
// shown on the host to come to an end).
#pragma once

#include <stdint.h>

#ifndef RRN_HOST_DEVICE
#ifdef __CUDACC__
#define RRN_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define RRN_HOST_DEVICE inline
#endif
#endif

namespace rrn {

// Whether a logit reaches a bound that `top` others reach.  A NaN counts as
// -infinity: it does where the bound is that (`lowest`), and only there.
RRN_HOST_DEVICE bool reaches(float x, float bound, bool lowest) { return x >= bound || lowest; }

// Rounds whose bound comes from a sample alone (KeySearch).  Rows in rising or
// falling order whose largest lie in the way of the first bound take up to nine
// in a model of the gathering.  A row of 2^20 in fp32, falling, 32 alternatives,
// takes 248 us; from the middle after four rounds, not 32, 1024.
constexpr int kSampledRounds = 32;

// The bound on keys (all different) that leaves at least the `top` largest and no
// more than there is room for.  What was gathered before the room ran out gives
// a higher bound that `top` keys reach, so that each round has fewer keys than
// the last.  How many fewer depends on the order in which they came, so after
// kSampledRounds the bound is at least the middle of those still possible: more
// than room keys reach `low`, fewer than top reach `high`, and that distance
// halves.  At most kSampledRounds + 64 rounds, whatever the row holds.
struct KeySearch {
    uint64_t least, low, high;
    int round;
    // The first bound's and the largest logit's high words, without a place.
    RRN_HOST_DEVICE void start(uint32_t first, uint32_t largest) {
        least = low = (uint64_t)first << 32;
        high = ((uint64_t)largest + 1) << 32;   // above every key
        round = 0;
    }
    // Whether the `found` keys that reach `least` hold the largest (the first
    // bound is one that enough keys reach, or there are no more).
    RRN_HOST_DEVICE bool enough(int found, int room, int top) const {
        return found <= room && (found >= top || round == 0);
    }
    // On to the next bound, when they do not.  sample: the top-th largest key of
    // some that reach `least`, where more than room do.
    RRN_HOST_DEVICE void next(int found, int room, uint64_t sample) {
        const bool more = found > room;
        if (more) low = least;
        else high = least;
        const uint64_t middle = low + (high - low) / 2;
        least = more && (round < kSampledRounds || sample > middle) ? sample : middle;
        ++round;
    }
};

}  // namespace rrn
