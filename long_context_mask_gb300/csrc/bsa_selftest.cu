// Self-test entry points (see include/bsa_selftest.h): the FMA-pipe exp2 next
// to CUDA's exp2f, and the bounded mbarrier waits giving up on a barrier that
// nothing will ever complete.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "bsa_internal.h"
#include "bsa_math.cuh"
#include "bsa_paged_wait.cuh"
#include "bsa_ptx.cuh"
#include "bsa_selftest.h"

namespace bsa {
namespace {

__global__ void k_selftest_exp2(const float* x, float* y_fma, float* y_mufu, float* y_ref, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    y_fma[i] = exp2_fma(x[i]);
    y_mufu[i] = ex2(x[i]);
    y_ref[i] = exp2f(x[i]);
}

// One thread waits (bounded) on an mbarrier that expects one arrival that
// never comes; on expiry it records BSA_ERR_TIMEOUT, exactly as the forward
// kernel's waits do.
__global__ void k_selftest_wait(uint64_t limit_ns, int32_t* status) {
    __shared__ uint64_t bar;
    const uint32_t b = ptx::smem_u32(&bar);
    if (threadIdx.x == 0) {
        ptx::mbar_init(b, 1);
        ptx::fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x == 0 && !ptx::mbar_wait(b, 0, limit_ns, status, BSA_ERR_TIMEOUT))
        atomicCAS(status, 0, BSA_ERR_TIMEOUT);
}

// The paged forward's waits: warp 0 waits on an mbarrier (2 ms), warp 1 does what the
// kind says.  out[w]: the ns that warp w waited, negative where it gave up.
constexpr uint64_t kShortNs = 2000000ull, kBusyNs = 50000000ull;
__global__ void k_selftest_paged_wait(int32_t kind, int64_t* out, int32_t* status) {
    __shared__ uint64_t bar[2];
    __shared__ Watch watch;
    const uint32_t b = ptx::smem_u32(&bar[0]);
    if (threadIdx.x == 0) {
        ptx::mbar_init(b, 1);
        ptx::mbar_init(ptx::smem_u32(&bar[1]), 1);
        ptx::fence_mbar_init();
        out[0] = out[1] = 0;
        watch.busy = 0;
        watch.abort = 0;
    }
    __syncthreads();
    const uint64_t t0 = ptx::globaltimer();
    if (threadIdx.x < 32) {
        const bool ok = __all_sync(0xffffffffu, paged_wait<kShortNs>(b, 0, &watch, status));
        const int64_t ns = (int64_t)(ptx::globaltimer() - t0);
        if (threadIdx.x == 0) {
            if (!ok) set_abort(&watch, status);
            out[0] = ok ? ns : -ns;
        }
    } else if (kind == BSA_PAGED_WAIT_TWO) {
        const bool ok = __all_sync(0xffffffffu, paged_wait(ptx::smem_u32(&bar[1]), 0, &watch, status));
        const int64_t ns = (int64_t)(ptx::globaltimer() - t0);
        if (threadIdx.x == 32) out[1] = ok ? ns : -ns;
    } else if (threadIdx.x == 32 && kind == BSA_PAGED_WAIT_BUSY) {
        // what it waits for goes on, and is there after 50 ms (each turn takes 10 ns at the least)
        for (int32_t i = 0; i < 10000000; ++i) {
            const uint64_t now = ptx::globaltimer();
            *reinterpret_cast<volatile uint64_t*>(&watch.busy) = now;
            if (now - t0 > kBusyNs) break;
        }
        ptx::mbar_arrive(b);
    }
}

}  // namespace
}  // namespace bsa

extern "C" {

bsa_status bsa_selftest_exp2(const float* x, float* y_fma, float* y_mufu, float* y_ref, int64_t n,
                             void* stream) {
    if (n < 0 || (n > 0 && (!x || !y_fma || !y_mufu || !y_ref))) return BSA_ERR_INVALID_ARG;
    if (n == 0) return BSA_OK;
    const unsigned grid = (unsigned)((n + 255) / 256);
    bsa::k_selftest_exp2<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(x, y_fma, y_mufu,
                                                                              y_ref, n);
    return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

bsa_status bsa_selftest_wait_timeout(int64_t limit_ns, void* stream) {
    if (limit_ns < 1000 || limit_ns > 1000000000) return BSA_ERR_INVALID_ARG;
    int32_t* status = bsa::status_word_ptr();
    if (!status) return BSA_ERR_CUDA;
    bsa::k_selftest_wait<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>((uint64_t)limit_ns, status);
    return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

bsa_status bsa_selftest_paged_wait(int32_t kind, int64_t* elapsed_ns, void* stream) {
    if (kind < BSA_PAGED_WAIT_NOTHING || kind > BSA_PAGED_WAIT_TWO || !elapsed_ns) return BSA_ERR_INVALID_ARG;
    int32_t* status = bsa::status_word_ptr();
    if (!status) return BSA_ERR_CUDA;
    bsa::k_selftest_paged_wait<<<1, 64, 0, static_cast<cudaStream_t>(stream)>>>(kind, elapsed_ns, status);
    return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // extern "C"
