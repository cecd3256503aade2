// The ragged batch over a paged key/value cache, as the paged kernels read it.
//
// Sequence s owns the new tokens q_start[s] .. q_start[s + 1] - 1 of the
// packed token axis; kv_len[s] tokens of it are in the cache, the new ones
// last, so new token i stands at position kv_len[s] - (number of new tokens)
// + i.  Position p lives in slot p % page of page table[s][p / page].  All of
// this is device data: the host knows only the capacities, so kernels are
// launched for the largest count and find their own work.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "bsa_internal.h"
#include "bsa_ptx.cuh"

namespace bsa {

// Every paged kernel is launched to begin while the kernel before it in the
// stream ends, and waits for that one's results (ptx::wait_primary, in all
// of its blocks and before it touches any tensor) once it has set itself up;
// it lets the next one do the same from its first instruction on.  A decoding
// step is a chain of four to seven short kernels, about 2 us apart otherwise.
template <typename... Params, typename... Args>
cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                           const Args&... args) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct PagedBatch {
    const int32_t* q_start;  // [seqs + 1]
    const int32_t* kv_len;   // [seqs]
    const int32_t* table;    // [seqs, max_pages]
    int32_t seqs, tokens, max_pages;
    int32_t page, n_pages;   // tokens per page (16, 32, 64 or 128); pages of the cache
    int32_t* status;
};

struct PagedSeq {
    int32_t q0, nq, kl;  // first new token, new tokens (0: none, or a bad entry), tokens in the cache
};

// false (and no new tokens) where the entry makes no sense: a negative or
// decreasing start, tokens beyond the packed axis, a length that is negative
// or beyond the table's row.
__device__ __forceinline__ bool paged_seq(const PagedBatch& b, int32_t s, PagedSeq& out) {
    const int32_t a = b.q_start[s], e = b.q_start[s + 1], kl = b.kv_len[s];
    const bool ok = a >= 0 && e >= a && e <= b.tokens && kl >= 0 && (int64_t)kl <= (int64_t)b.max_pages * b.page;
    out.q0 = a;
    out.nq = ok ? e - a : 0;
    out.kl = ok ? kl : 0;
    return ok;
}

// Exclusive prefix sum over the thread block of kThreads; total receives the
// block's sum.  part: kThreads / 32 words of shared memory.
template <int kThreads>
__device__ __forceinline__ int64_t block_prefix(int64_t x, int64_t* part, int64_t& total) {
    constexpr int warps = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t incl = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    __syncthreads();  // an earlier call's readers are done with part
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < warps; ++w) {
        const int64_t v = part[w];
        before += w < warp ? v : 0;
        all += v;
    }
    total = all;
    return before + incl - x;
}

// Unit u of the batch, where sequence s counts count(seq) units: the sequence
// (-1: u is beyond the last), the unit within it and the sequence's entry.
// Called by the whole thread block; the same answer in every thread.  part: see
// block_prefix; hit: 5 words of shared memory.
template <int kThreads, typename Count>
__device__ __forceinline__ int32_t find_unit(const PagedBatch& b, int64_t u, Count&& count, int64_t* part, int32_t* hit,
                                             int32_t& within, PagedSeq& found) {
    if (threadIdx.x == 0) hit[0] = -1;
    int64_t base = 0;
    for (int32_t s0 = 0; s0 < b.seqs; s0 += kThreads) {
        const int32_t s = s0 + threadIdx.x;
        PagedSeq q{0, 0, 0};
        int64_t n = 0;
        if (s < b.seqs) {
            paged_seq(b, s, q);
            n = count(q);
        }
        int64_t total;
        const int64_t at = base + block_prefix<kThreads>(n, part, total);
        if (n > 0 && u >= at && u < at + n) {
            hit[0] = s;
            hit[1] = (int32_t)(u - at);
            hit[2] = q.q0;
            hit[3] = q.nq;
            hit[4] = q.kl;
        }
        base += total;
        if (u < base) break;
    }
    __syncthreads();
    within = hit[1];
    found = PagedSeq{hit[2], hit[3], hit[4]};
    return hit[0];
}

}  // namespace bsa
