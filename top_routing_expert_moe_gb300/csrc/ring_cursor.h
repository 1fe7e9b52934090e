// ring_cursor.h -- where a ring of stages stands.  Items 0, 1, 2, ... pass through
// the stages in turn, and the n-th item of a stage completes its barrier's phase of
// parity n & 1.  Plain C++, so that a program on the host can follow it too.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {

struct RingCursor {
    int stages, slot = 0;        // the current item's stage
    uint32_t phase = 0;          // and its parity

    MOE_HD int ahead(int k) const { return slot + k >= stages ? slot + k - stages : slot + k; }   // k < stages
    MOE_HD uint32_t phase_ahead(int k) const { return slot + k >= stages ? phase ^ 1u : phase; }
    MOE_HD void next() {
        if (++slot == stages) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// After items 0 .. sent - 1 have been sent for: the parity of the last of them in
// stage s (s < sent).  It does not depend on how far the cursor went on without new
// items, as it does after a wait that gave up.
MOE_HD uint32_t last_parity(uint32_t sent, uint32_t stages, uint32_t s) {
    return ((sent - 1 - s) / stages) & 1u;
}

}  // namespace moe
