#pragma once

#include <stdint.h>

#include "common.cuh"

namespace qa {

// Waits of a CTA that give up together: the first one that runs out sets
// *abort (in shared memory, 0 before), and from then on every one that would
// block returns at once, so that a CTA whose data never come ends after one
// limit and not after one a wait.  Returns whether the phase is complete.
// more_ns: what a wait may take beyond the limit when all is well.
struct Waits {
    volatile int *abort;
    unsigned int *status;
    unsigned long long limit_ns;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity, unsigned long long more_ns = 0) const {
        if (mbar_try_wait(bar, parity)) return true;
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(bar, parity)) {
            if (*abort) return false;
            if (globaltimer_ns() - t0 > limit_ns + more_ns) {
                atomicOr(status, QA_DEVICE_TIMEOUT);
                *abort = 1;
                return false;
            }
        }
        return true;
    }
};

}  // namespace qa
