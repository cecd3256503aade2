/*
 * bsa_selftest.h - self-test entry points of libbsa.so.  They check
 * building blocks of the forward calls on the device and are meant for test
 * suites, not for the attention path.  Conventions as in bsa.h.
 */
#ifndef BSA_SELFTEST_H
#define BSA_SELFTEST_H

#include <stdint.h>

#include "bsa.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * bsa_selftest_exp2 - evaluate, for each x[i] (device fp32 [n]), the three
 * 2^x used or mirrored by the softmax: y_fma (the FMA-pipe polynomial that
 * bsa_forward uses for part of its exponentials: Cody-Waite reduction plus a
 * fitted degree-3 minimax polynomial), y_mufu (the hardware ex2.approx) and
 * y_ref (CUDA's exp2f).  All outputs device fp32 [n].  The polynomial is
 * specified for -125 <= x <= 127 (below, clamped to -125).
 */
bsa_status bsa_selftest_exp2(const float* x, float* y_fma, float* y_mufu, float* y_ref, int64_t n,
                             void* stream);

/*
 * bsa_selftest_wait_timeout - launch one thread that waits, bounded by
 * limit_ns (1 us .. 1 s), on an mbarrier that nothing completes, using the
 * same bounded wait as bsa_forward.  When the limit expires the kernel
 * records BSA_ERR_TIMEOUT in the device status word and returns; read it with
 * bsa_device_status().  Nothing faults, traps or hangs.
 */
bsa_status bsa_selftest_wait_timeout(int64_t limit_ns, void* stream);

typedef enum {
    BSA_PAGED_WAIT_NOTHING = 0, /* nothing completes the barrier                            */
    BSA_PAGED_WAIT_BUSY = 1,    /* a second warp completes it after 50 ms of visible progress */
    BSA_PAGED_WAIT_TWO = 2      /* nothing does, and a second warp waits for up to 1 s       */
} bsa_paged_wait_kind;

/*
 * bsa_selftest_paged_wait - launch one warp that waits, for 2 ms at most, on
 * an mbarrier with bsa_forward_paged's wait, which lasts as long as the work
 * it waits for shows progress.  A wait that gives up records BSA_ERR_TIMEOUT
 * in the device status word and ends the other waits of its thread block.
 * Nothing faults, traps or hangs.
 *  elapsed_ns  device int64 [2] out: how long either warp waited, negative
 *              where it gave up (0: it did not wait).
 */
bsa_status bsa_selftest_paged_wait(int32_t kind, int64_t* elapsed_ns, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BSA_SELFTEST_H */
