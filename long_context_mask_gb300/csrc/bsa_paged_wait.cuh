// The bounded waits of the paged forward's warps for one another.
#pragma once

#include <stdint.h>

#include "bsa.h"
#include "bsa_ptx.cuh"

namespace bsa {

constexpr uint64_t kPagedWaitNs = 1000000000ull;  // 1 s per wait

// What the warps of a thread block know of one another (shared memory).
struct Watch {
    uint64_t busy;   // when a key tile of a row computed from its own keys was last done
    int32_t abort;   // a wait of the block has been given up: all others end too
};

// A call that timed out has rows it did not write, where the other codes speak of what
// was left out of an otherwise whole result: it takes their place in the status word.
__device__ __forceinline__ void raise_timeout(int32_t* status) { atomicExch(status, BSA_ERR_TIMEOUT); }
__device__ __forceinline__ void set_abort(Watch* w, int32_t* status) {
    *reinterpret_cast<volatile int32_t*>(&w->abort) = 1;
    raise_timeout(status);
}
// A bounded wait.  While rows are computed from their own keys (busy moves on with
// every key tile of them) those who wait for them have not lost their time yet.  All but
// the first look is out of line: the kernel waits in some twenty places, and a window's
// short rows are sensitive to its length.
template <uint64_t kLimitNs>
__device__ __noinline__ bool paged_wait_on(uint32_t bar, uint32_t parity, const volatile Watch* w,
                                           const volatile int32_t* status) {
    const int64_t t0 = (int64_t)ptx::globaltimer(), limit = (int64_t)kLimitNs;
    uint32_t n = 0;
    while (!ptx::mbar_try_wait(bar, parity)) {
        if ((++n & 255u) == 0) {
            // (busy may move on between the two looks, and be ahead of the clock's)
            const int64_t now = (int64_t)ptx::globaltimer(), last = (int64_t)w->busy;
            if (now - t0 > limit && now - last > limit) return false;
            if (w->abort != 0 || *status == BSA_ERR_TIMEOUT) return false;  // (or one of another block)
        }
    }
    return true;
}
template <uint64_t kLimitNs = kPagedWaitNs>
__device__ __forceinline__ bool paged_wait(uint32_t bar, uint32_t parity, const Watch* w, const int32_t* status) {
    return ptx::mbar_try_wait(bar, parity) || paged_wait_on<kLimitNs>(bar, parity, w, status);
}
// For copies and products in flight, after a failure too.
inline __device__ __noinline__ void paged_drain(uint32_t bar, uint32_t parity, int32_t* status) {
    if (!ptx::mbar_wait(bar, parity, kPagedWaitNs, status, -1)) raise_timeout(status);
}

}  // namespace bsa
