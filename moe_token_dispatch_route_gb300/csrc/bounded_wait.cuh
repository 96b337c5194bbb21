// Bounded waits on the mbarriers of the tensor-core kernels' pipelines.
#pragma once

#include "moe_internal.cuh"

namespace moe {

#if defined(__CUDACC__)

struct Wait {
    volatile int* abort;
    int32_t* status;
    long long timeout_ns;
};

__device__ __forceinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, const Wait& w, int where, bool honor_abort) {
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if ((i & 127u) == 0) {
            if (honor_abort && *w.abort) return false;
            if (global_timer_ns() - t0 > (uint64_t)w.timeout_ns) {
                report_error(w.status, kStDevice, where, -1, 0);
                *w.abort = 1;
                return false;
            }
        }
    }
}

// Bounded wait on a barrier of this CTA; false when it gave up or the CTA is leaving.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, const Wait& w, int where, bool honor_abort = true) {
    return mbar_try_wait_cluster(bar, parity) || bar_wait_slow(bar, parity, w, where, honor_abort);
}

#endif  // __CUDACC__

}  // namespace moe
