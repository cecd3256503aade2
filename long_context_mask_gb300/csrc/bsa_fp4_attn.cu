// Attention of new tokens over a paged key/value cache held in 4 bits.
//
// What it computes is what bsa_paged_attn.cu computes (token i of a sequence at position
// p, query head h, the keys j that causality, a window with sinks or a list of blocks leave):
//     s_j = scale q . k_j,   LSE = ln sum_j exp(s_j),   O = sum_j exp(s_j - LSE) v_j
// with k_j and v_j as bsa_fp4.cuh reads them.
//
// Here: the sequences of few rows (a step of single tokens, a few tokens each); the others are
// bsa_fp4_prompt.cu's.
//
// Rows.  The new tokens of a sequence and the G query heads of a key/value head are rows,
// token by token; a row tile is 8 NT of them (with lists: of one token).  A key tile is 128
// positions.  Few rows want the keys as the long side of the products: with mma m16n8k16,
// S^T = K Q^T has 16 keys by 8 rows, O^T = V^T P^T has 16 values of D by 8 rows.  (The tensor core's
// large tiles have 64 rows or more: a token of 4 rows would leave 15 in 16 unused, and K and V would
// have to be written to shared memory as fp16 first.)  Codes become fp16 operands in registers:
//   K    lane (r, c) = (lane / 4, lane % 4) takes D / 4 values of keys r and r + 8.  The order
//        of the D values in the sum is free, so a byte's two values are one operand register.
//   V^T  lane (r, c) takes D / 8 values of keys 2c, 2c + 1, 2c + 8, 2c + 9.  An operand register
//        holds two keys' values at one place: their nibbles are brought together in a byte
//        before it is converted.
//   P^T  comes out of S^T's accumulators by two 8 x 8 transposes (movmatrix).
// Levels times scales are exact in fp16.  Queries are multiplied by the power of two that
// brings their row's largest value to 2^14, and rounded to fp16 (what a bf16 value loses
// lies 2^39 below the row's largest).  Weights are rounded to fp16: they start at 2^6 (kFp4Start) and are
// kept below 2^16 by raising the row's maximum.
//
// Warps.  One thread block an SM.  Two warps copy K's and V's codes and scales of key tiles into a
// ring of eight, and the query rows of the segments; 16 warps (8 for row tiles of 16, whose state is
// twice as large) multiply, in teams of four that take every fourth (second) tile, 32 keys a warp;
// one warp joins their parts of O in shared memory and stores the rows.  (64 tokens over caches up to
// 8192, 32 + 8 heads of 128, 483 MB of codes and scales: 130 us with eight warps that loaded their 16
// keys of a tile themselves, 95 with one loading warp and two thread blocks an SM, 99 in this
// form, which has two blocks' warps without two blocks' unequal shares of the SM: 2 % faster on 64 tokens over
// 32768 keys each, 15 % on short heads in short pages.)
//
// Split.  All (key/value head, sequence, row tile, key tile) units are laid out in that order
// and cut into equal runs, one for each thread block.  A row tile's part in a run is joined
// over the warps in shared memory; a tile that a cut splits leaves its parts in the workspace
// for k_fp4_join, which adds them in key order.
//
// What bounds it.  The step of 64 tokens: 99 us, 4.9 TB/s, 0.72 of the copy rate.  The conversion of a
// byte of codes runs at 64 lanes a cycle and SM, as do the nibbles' moves: that pipe is busy 53 % of the
// time, issue slots 60 %, and the rest are waits that four warps a scheduler do not cover.  The same copies without
// the arithmetic take 82 us (64 tokens over 32768 keys each: 403 us, 346 without, which is the copy rate).  One token over
// 131072: 38 us, 31 without the arithmetic, 22 at the copy rate: the start, the last parts and the join.
// One token over 1000: 9.7 us, latency: finding the run, the page table, the first tile, the parts, the join.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "bsa_device_setup.h"
#include "bsa_fp4.cuh"
#include "bsa_fp4_runs.cuh"
#include "bsa_internal.h"
#include "bsa_paged.cuh"
#include "bsa_paged_wait.cuh"
#include "bsa_rows.cuh"
#include "bsa_tma_host.h"

namespace bsa {
namespace {

constexpr int32_t kMaxWindow = 1 << 26;  // (positions lie within 2^24 of zero)
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTeam = 4;                     // warps to a key tile, 32 keys each
constexpr int kMaxNT = 2;
constexpr int32_t kFewRows = 16;             // rows of a sequence that are done here
// With lists: so many tokens, where a token is one row tile.  (32 sequences over 16384, 18 random blocks of 129 for each token, 32 + 8
// heads: 16, 24, 32 tokens each by themselves 302, 445, 585 us, as tiles of tokens 241, 262, 276; 64 of 6 tokens, 10 blocks:
// 168, 196.)
constexpr int32_t kFewListed = 8;
// A row tile of n key tiles counts n + kRowCost in a run.
constexpr int32_t kRowCost = 2;
constexpr float kMost = 15.9f;  // log2 of the largest weight (fp16 numbers end at 2^16)

enum { kPlain = 0, kWindow = 1, kListed = 2 };

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t bits(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

// Shared memory of a thread block: a ring of key tiles (codes of keys and of values, then their
// scales), the parts of O that the warps join, query rows, and what the warps tell one another.
template <int D, int NT>
struct Cfg {
    static constexpr int kWarps = NT == 1 ? 16 : 8;      // that compute; two more load, one joins their parts
    static constexpr int kLoadK = kWarps, kLoadV = kWarps + 1, kStore = kWarps + 2;
    static constexpr int kThreads = 32 * (kWarps + 3);
    static constexpr int kTeams = kWarps / kTeam;
    static constexpr int kStages = 8;                    // (a multiple of the teams)
    static constexpr int kCodes = 128 * D / 2, kScales = 128 * D / 16;
    static constexpr int kStage = 2 * (kCodes + kScales);
    static constexpr int kRing = kStages * kStage;
    static constexpr int kRowO = D + 4;                  // a row of O, padded
    static constexpr int kJoin = kWarps * 8 * NT * kRowO * 4;
    static constexpr int kSmem = kRing + kJoin;          // (and 128 bytes to align it)
};

constexpr int kDesc = 3;    // descriptors in flight

template <int D, int NT>
struct Shared {
    __nv_bfloat16 q[kDesc][8 * NT][D];  // the segments' query rows
    uint64_t full[Cfg<D, NT>::kStages], empty[Cfg<D, NT>::kStages];
    uint64_t seg_full[kDesc], seg_empty[kDesc];
    uint64_t joined, freed;           // the warps' parts are there, have been read
    Watch watch;
    Fp4Segment seg[kDesc];
    int32_t key[Cfg<D, NT>::kStages]; // first key of the tile in each slot
    Fp4Start start;
    float2 ml[Cfg<D, NT>::kWarps][8 * NT];
};

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const Watch* w, const int32_t* status) {
    return __all_sync(0xffffffffu, paged_wait(bar, parity, w, status));
}

template <int D, int NT, int kMode>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1) k_fp4_rows(const __grid_constant__ Fp4Params P) {
    using C = Cfg<D, NT>;
    constexpr bool kLists = kMode == kListed;
    constexpr uint32_t S = C::kStages, T = C::kTeams;
    constexpr int kWarps = C::kWarps, kLoadK = C::kLoadK, kLoadV = C::kLoadV, kStore = C::kStore, kThreads = C::kThreads;
    constexpr int R = 8 * NT;
    constexpr int kSteps = D / 16;          // products of S^T for 16 keys; of O^T as well
    constexpr int kKW = D / 32;             // words of a K row that a lane takes
    constexpr int kVW = D / 64;             // words of a V row that a lane takes
    constexpr int kRowO = C::kRowO;
    extern __shared__ uint8_t smem_raw[];
    // (an offset, not a rounded pointer: the compiler has to see that it is shared memory)
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 127u);
    __shared__ __align__(16) Shared<D, NT> sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t* const status = P.b.status;
    if (threadIdx.x == kThreads - 1) {
        for (uint32_t x = 0; x < S; ++x) {
            mbar_init(smem_u32(&sh.full[x]), 2);
            mbar_init(smem_u32(&sh.empty[x]), kTeam);
        }
        for (int x = 0; x < kDesc; ++x) {
            mbar_init(smem_u32(&sh.seg_full[x]), 1);
            mbar_init(smem_u32(&sh.seg_empty[x]), kWarps + 2);
        }
        mbar_init(smem_u32(&sh.joined), kWarps);
        mbar_init(smem_u32(&sh.freed), 1);
        fence_mbar_init();
    }
    launch_dependents();
    wait_primary();
    if (threadIdx.x == kThreads - 1) {
        P.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
        sh.watch.busy = 0;
        // a block of this launch (or an unread earlier one) timed out: abandon
        sh.watch.abort = *reinterpret_cast<const volatile int32_t*>(status) == BSA_ERR_TIMEOUT;
    }

    // ---------------------------------------------------------------- this block's run
    // (its scratch is in the ring, which is free here)
    using Work = Fp4Work<R, kRowCost, kLists>;
    constexpr int kScan = kLists ? kThreads : 128;  // (lists: many counts to read)
    if (threadIdx.x < kScan) Work{P}.template find<kScan>(reinterpret_cast<int32_t*>(smem), sh.start);
    // what was written there by ordinary stores makes room for bulk copies
    fence_proxy_async_smem();
    __syncthreads();
    if (sh.start.any == 0 || sh.watch.abort != 0) return;

    // ---------------------------------------------------------------- loading warps
    // The K (V) tiles of a segment, whose numbers in the run begin at g, four at a time: lane l has page
    // l % N of tile l / N.
    auto load_tiles = [&](const Fp4Segment& sg, bool is_v, uint32_t& g) -> bool {
        constexpr int kAtOnce = 4;
        const int32_t page = P.b.page, N = 128 / page;  // pages of a tile
        const int32_t lane_tile = lane / N, lane_page = lane - lane_tile * N;
        const int32_t j0 = sg.j0, j1 = j0 + sg.n, kvh = sg.kvh;
        const int32_t* table = P.b.table + (int64_t)sg.seq * P.b.max_pages;
        const int32_t* list = kLists ? P.list + Work{P}.list_of(kvh, sg.tile) * P.cap : nullptr;
        const uint8_t *codes = is_v ? P.v : P.k, *scales = is_v ? P.v_scale : P.k_scale;
        const CUtensorMap *map = is_v ? &P.map_v : &P.map_k, *map_s = is_v ? &P.map_vs : &P.map_ks;
        const uint32_t to_codes = smem_u32(smem) + (is_v ? C::kCodes : 0) + lane_page * page * (D / 2);
        const uint32_t to_scales = smem_u32(smem) + 2 * C::kCodes + (is_v ? C::kScales : 0) + lane_page * page * (D / 16);
        // the cache row of this lane's page (-1: behind the sequence's end, or no tile), and the tile's first key
        auto fetch = [&](int32_t jb, int32_t& key) -> int32_t {
            const int32_t j = jb + lane_tile;
            key = 0;
            if (lane_tile >= kAtOnce || j >= j1) return -1;
            if constexpr (kLists) key = list[j] * 128;
            else key = (j < sg.ns ? j : sg.lo + j - sg.ns) * 128;
            const int32_t pg = key / page + lane_page;
            if (pg * page >= sg.kl) return -1;
            int32_t id = table[pg];
            if (id < 0 || id >= P.b.n_pages) {
                raise_status(status, BSA_ERR_BOUNDS);
                id = 0;  // (this row's result is unspecified)
            }
            return (id * P.H_kv + kvh) * page;
        };
        int32_t key_nxt, nxt = fetch(j0, key_nxt);
        for (int32_t jb = j0; jb < j1; jb += kAtOnce) {
            const int32_t row = nxt, key = key_nxt, tiles = min(kAtOnce, j1 - jb);
            nxt = fetch(jb + kAtOnce, key_nxt);
            const bool live = lane_tile < tiles;
            const uint32_t gl = g + (live ? lane_tile : 0), at = gl % S, bar = smem_u32(&sh.full[at]);
            if (!wait_warp(smem_u32(&sh.empty[at]), ((gl / S) & 1u) ^ 1u, &sh.watch, status)) return false;
            const uint32_t held = __ballot_sync(0xffffffffu, row >= 0);
            const int32_t first = __shfl_sync(0xffffffffu, row, lane - lane_page);
            if (live && lane_page == 0) {
                if (!is_v) sh.key[at] = key;
                mbar_arrive_expect_tx(bar, fp4_page_bytes(page, __popc(held >> lane & ((1u << N) - 1u)), D / 2 + D / 16));
            }
            __syncwarp();
            fp4_load_pages(codes, map, page, D / 2, live, row, first, to_codes + at * C::kStage, bar);
            fp4_load_pages(scales, map_s, page, D / 16, live, row, first, to_scales + at * C::kStage, bar);
            __syncwarp();
            g += tiles;
        }
        return true;
    };
    // (every issued copy must land before the block exits)
    auto land = [&](uint32_t g) {
        if (lane == 0)
            for (uint32_t x = g > S ? g - S : 0; x < g; ++x) paged_drain(smem_u32(&sh.full[x % S]), (x / S) & 1u, status);
        __syncwarp();
    };
    uint32_t k = 0;  // segments so far
    bool ok = true;
    if (warp == kLoadK) {
        // ------------------------------------------------------------ segments, query rows and K tiles
        Fp4Walk<R, kRowCost, kLists> walk(P, sh.start);
        Fp4Segment sg;
        uint32_t g = 0;  // tiles so far
        for (; ok && walk.open(sg); walk.advance()) {
            const uint32_t d = k % kDesc, seg_bar = smem_u32(&sh.seg_full[d]);
            if (!wait_warp(smem_u32(&sh.seg_empty[d]), ((k / kDesc) & 1u) ^ 1u, &sh.watch, status)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                sh.seg[d] = sg;
                mbar_arrive_expect_tx(seg_bar, (uint32_t)(sg.nrows * D * 2));
                walk.note(sg);
            }
            __syncwarp();
            if (lane < sg.nrows) {
                const int32_t row = sg.row0 + lane, tok = row / P.group, head = row - tok * P.group;
                bulk_load(smem_u32(sh.q[d][lane]),
                          P.q + ((int64_t)sg.q0 + tok) * P.q_stride + (int64_t)(sg.kvh * P.group + head) * D, D * 2, seg_bar);
            }
            __syncwarp();
            ++k;
            ok = load_tiles(sg, false, g);
        }
        if (ok && wait_warp(smem_u32(&sh.seg_empty[k % kDesc]), ((k / kDesc) & 1u) ^ 1u, &sh.watch, status)) {
            if (lane == 0) {
                sh.seg[k % kDesc].n = -1;
                mbar_arrive(smem_u32(&sh.seg_full[k % kDesc]));
            }
        } else {
            ok = false;
        }
        if (!ok && lane == 0) set_abort(&sh.watch, status);
        land(g);
        if (lane == 0) {
            // (the last descriptor's slot has been handed back: its query rows had landed)
            const uint32_t known = k + (ok ? 1u : 0u);
            for (uint32_t x = known > kDesc ? known - kDesc : 0; x < k; ++x)
                paged_drain(smem_u32(&sh.seg_full[x % kDesc]), (x / kDesc) & 1u, status);
        }
        return;
    }
    if (warp == kLoadV) {
        // ------------------------------------------------------------ V tiles
        uint32_t g = 0;
        for (; ok; ++k) {
            if (!wait_warp(smem_u32(&sh.seg_full[k % kDesc]), (k / kDesc) & 1u, &sh.watch, status)) {
                ok = false;
                break;
            }
            const Fp4Segment sg = sh.seg[k % kDesc];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.seg_empty[k % kDesc]));
            if (sg.n < 0) break;
            ok = load_tiles(sg, true, g);
        }
        if (!ok && lane == 0) set_abort(&sh.watch, status);
        land(g);
        return;
    }

    float* const so = reinterpret_cast<float*>(smem + C::kRing);  // [warp][row][kRowO]
    if (warp == kStore) {
        // ------------------------------------------------------------ joins the warps' parts
        constexpr int kLanes = D / 4, kAbreast = 32 / kLanes;
        const int col = lane % kLanes;
        for (;; ++k) {
            if (!wait_warp(smem_u32(&sh.seg_full[k % kDesc]), (k / kDesc) & 1u, &sh.watch, status)) {
                ok = false;
                break;
            }
            const Fp4Segment sg = sh.seg[k % kDesc];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.seg_empty[k % kDesc]));
            if (sg.n < 0) break;
            const float vg = P.v_gain != nullptr ? P.v_gain[sg.kvh] : 1.0f;
            if (!wait_warp(smem_u32(&sh.joined), k & 1u, &sh.watch, status)) {
                ok = false;
                break;
            }
            for (int32_t row = lane / kLanes; row < sg.nrows; row += kAbreast) {
                float M = -INFINITY, sum = 0.0f, out[4] = {0.f, 0.f, 0.f, 0.f};
                float2 z[kWarps];
#pragma unroll
                for (int y = 0; y < kWarps; ++y) {
                    z[y] = sh.ml[y][row];
                    M = fmaxf(M, z[y].x);
                }
#pragma unroll
                for (int y = 0; y < kWarps; ++y) {
                    if (z[y].y == 0.0f) continue;  // no visible key
                    const float f = ex2(z[y].x - M);
                    sum = fmaf(f, z[y].y, sum);
                    const float4 v = *reinterpret_cast<const float4*>(so + (y * R + row) * kRowO + 4 * col);
                    out[0] = fmaf(f, v.x, out[0]);
                    out[1] = fmaf(f, v.y, out[1]);
                    out[2] = fmaf(f, v.z, out[2]);
                    out[3] = fmaf(f, v.w, out[3]);
                }
                if (sg.part < 0) {
                    // (the gain after the quotient: the smallest gain over a long sum is no normal number)
                    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                    const int32_t x = sg.row0 + row, tok = x / P.group;
                    const int64_t at = ((int64_t)sg.q0 + tok) * P.H + sg.kvh * P.group + (x - tok * P.group);
                    *reinterpret_cast<uint2*>(P.o + at * D + 4 * col) =
                        make_uint2(pack_bf16(out[0] * inv * vg, out[1] * inv * vg), pack_bf16(out[2] * inv * vg, out[3] * inv * vg));
                    if (col == 0) P.lse[at] = sum == 0.0f ? -INFINITY : (M + log2f(sum)) * kFp4Ln2;
                } else {
                    const int64_t at = (int64_t)sg.part * R + row;
                    *reinterpret_cast<float4*>(P.part_o + at * D + 4 * col) = make_float4(out[0], out[1], out[2], out[3]);
                    if (col == 0) P.part_ml[at] = make_float2(M, sum);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.freed));
        }
        if (!ok && lane == 0) set_abort(&sh.watch, status);
        return;
    }

    // ---------------------------------------------------------------- the others: products and softmax
    const int r = lane >> 2, c = lane & 3;
    // which of the sixteen keys is row i of S^T, so that neither lane (r, c)'s rows r and r + 8 of
    // K nor its keys key_of(2 c + (y & 1)) + 8 (y / 2) of V, y < 4, meet those of too many other lanes in a bank
    auto key_of = [](int i) -> int {  // (key_of(i + 8) = key_of(i) + 8)
        return ((i ^ (i >> 1)) & 1) + (i & 2) + (i & 4) + (i & 8);
    };
    const int k_row = key_of(r);
    // this lane's places in a tile: of K and its scales, of V's keys y = 0 and 1 and theirs (the
    // other keys lie eight rows on, the second sixteen sixteen)
    const uint32_t w0 = (warp % kTeam) * 32;
    const uint32_t off_k = (w0 + k_row) * (D / 2) + c * (D / 8);
    const uint32_t off_ks = 2 * C::kCodes + (w0 + k_row) * (D / 16) + (D == 128 ? 2 * c : c);
    const uint32_t v0 = w0 + key_of(2 * c), v1 = w0 + key_of(2 * c + 1);
    const uint32_t off_v[2] = {C::kCodes + v0 * (D / 2) + r * (D / 16), C::kCodes + v1 * (D / 2) + r * (D / 16)};
    const uint32_t at_s = 2 * C::kCodes + C::kScales + (D == 128 ? r : r >> 1);
    const uint32_t off_vs[2] = {at_s + v0 * (D / 16), at_s + v1 * (D / 16)};
    // this warp's team takes every T-th tile of the run: slots team, team + T, ..
    const uint32_t team = warp / kTeam;
    uint32_t slot = team, phase = 0;  // of the team's next tile
    uint32_t g0 = 0;                  // tiles of the segments before
    for (; ok; ++k) {
        if (!wait_warp(smem_u32(&sh.seg_full[k % kDesc]), (k / kDesc) & 1u, &sh.watch, status)) {
            ok = false;
            break;
        }
        const Fp4Segment sg = sh.seg[k % kDesc];
        if (sg.n < 0) break;
        const int32_t row0 = sg.row0, nrows = sg.nrows;

        // queries: lane (r, c) has D / 4 values of rows r, r + 8, ..
        uint32_t qf[NT][kSteps][2];
        float fac[NT][2];               // of the rows of this lane's columns 2 c, 2 c + 1
        int32_t hi[NT][2], lo[NT][2], sk[NT][2];
        auto end = [&](int32_t p) -> int32_t { return P.causal ? min(sg.kl, p + 1) : sg.kl; };
        const float kg = (P.k_gain != nullptr ? P.k_gain[sg.kvh] : 1.0f) * P.scale_log2;
#pragma unroll
        for (int b = 0; b < NT; ++b) {
            // (rows beyond the tile's: any; they are not stored)
            const uint4* src = reinterpret_cast<const uint4*>(sh.q[k % kDesc][min(8 * b + r, nrows - 1)] + c * (D / 4));
            uint4 raw[D / 32];
#pragma unroll
            for (int y = 0; y < D / 32; ++y) raw[y] = src[y];
            const uint32_t* wd = reinterpret_cast<const uint32_t*>(raw);
            uint32_t top = 0u;  // the largest exponent field of a finite value
#pragma unroll
            for (int y = 0; y < D / 8; ++y) {
                const uint32_t e0 = wd[y] >> 7 & 0xffu, e1 = wd[y] >> 23 & 0xffu;
                top = max(top, max(e0 == 0xffu ? 0u : e0, e1 == 0xffu ? 0u : e1));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int32_t e = max((int32_t)top - 127, -100) - 14;
            const float up = __int_as_float((127 - e) << 23);
#pragma unroll
            for (int y = 0; y < D / 8; ++y) {
                const float f0 = __uint_as_float(wd[y] << 16) * up, f1 = __uint_as_float(wd[y] & 0xffff0000u) * up;
                qf[b][y >> 1][y & 1] = bits(__floats2half2_rn(f0, f1));
            }
            const float down = __int_as_float((127 + e) << 23) * kg;
            fac[b][0] = __shfl_sync(0xffffffffu, down, 8 * c);
            fac[b][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int32_t p = sg.pos_of0 + (row0 + min(8 * b + 2 * c + y, nrows - 1)) / P.group;
                hi[b][y] = end(p);
                if constexpr (kMode == kWindow) {
                    lo[b][y] = p - P.window + 1;
                    sk[b][y] = min(P.sinks, hi[b][y]);
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.seg_empty[k % kDesc]));
        const int32_t p_first = sg.pos_of0 + row0 / P.group, p_last = sg.pos_of0 + (row0 + nrows - 1) / P.group;
        const int32_t all_hi = end(p_first), all_lo = p_last - P.window + 1, all_sk = min(P.sinks, all_hi);

        float acc[NT][kSteps][4] = {};
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                m[b][y] = kFp4NoKey;
                l[b][y] = 0.0f;
            }
        const uint32_t first = (team - g0) & (T - 1u);  // the team's first tile of the segment
        g0 += (uint32_t)sg.n;
#pragma unroll 1
        for (int32_t n = sg.n - (int32_t)first; n > 0; n -= (int32_t)T) {
            if (!wait_warp(smem_u32(&sh.full[slot]), phase, &sh.watch, status)) {
                ok = false;
                break;
            }
            const int32_t kb = sh.key[slot] + (int32_t)w0;
            const uint32_t done = smem_u32(&sh.empty[slot]);
            const uint8_t* at = smem + slot * C::kStage;
            slot += T;
            if (slot >= S) {
                slot = team;
                phase ^= 1u;
            }
            if (kb >= sg.kl) {  // behind the sequence's end
                if (lane == 0) mbar_arrive(done);
                continue;
            }
            // S^T = K Q^T, twice sixteen keys
            float sc[2][NT][4] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t kw[2][kKW];
                __half2 s2[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint8_t* src = at + off_k + (16 * h + 8 * y) * (D / 2);
                    const uint8_t* ss = at + off_ks + (16 * h + 8 * y) * (D / 16);
                    if constexpr (D == 128) {
                        *reinterpret_cast<uint4*>(kw[y]) = *reinterpret_cast<const uint4*>(src);
                        s2[y] = fp4_scales(*reinterpret_cast<const uint16_t*>(ss));
                    } else {
                        *reinterpret_cast<uint2*>(kw[y]) = *reinterpret_cast<const uint2*>(src);
                        s2[y] = fp4_scales(*ss);
                    }
                }
#pragma unroll
                for (int wd = 0; wd < kKW; ++wd) {
                    __half2 f[4], e[4];
                    fp4_levels(kw[0][wd], f);
                    fp4_levels(kw[1][wd], e);
                    const __half2 sf = D == 128 && wd >= kKW / 2 ? __high2half2(s2[0]) : __low2half2(s2[0]);
                    const __half2 se = D == 128 && wd >= kKW / 2 ? __high2half2(s2[1]) : __low2half2(s2[1]);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t op[4] = {bits(__hmul2(f[2 * y], sf)), bits(__hmul2(e[2 * y], se)),
                                                bits(__hmul2(f[2 * y + 1], sf)), bits(__hmul2(e[2 * y + 1], se))};
#pragma unroll
                        for (int b = 0; b < NT; ++b) mma16816(sc[h][b], op, qf[b][2 * wd + y][0], qf[b][2 * wd + y][1]);
                    }
                }
            }
            // exponents against the rows' maxima so far
            bool seen = kb + 32 <= all_hi;
            if constexpr (kMode == kWindow) seen = (seen && kb >= all_lo) || kb + 32 <= all_sk;
            auto vis = [&](int h, int b, int y) -> bool {
                const int32_t key = kb + k_row + 16 * h + 8 * (y >> 1);
                bool v = key < hi[b][y & 1];
                if constexpr (kMode == kWindow) v = (v && key >= lo[b][y & 1]) || key < sk[b][y & 1];
                return v;
            };
            float ex[2][NT][4], top = -INFINITY;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int b = 0; b < NT; ++b)
#pragma unroll
                    for (int y = 0; y < 4; ++y) ex[h][b][y] = fmaf(sc[h][b][y], fac[b][y & 1], -m[b][y & 1]);
            if (!seen) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int b = 0; b < NT; ++b)
#pragma unroll
                        for (int y = 0; y < 4; ++y) ex[h][b][y] = vis(h, b, y) ? ex[h][b][y] : -INFINITY;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int b = 0; b < NT; ++b) top = fmax3(fmax3(top, ex[h][b][0], ex[h][b][1]), ex[h][b][2], ex[h][b][3]);
            // A row that passes the limit takes a new maximum; the others' exponents come out as above, bit by bit,
            // so that what one row holds does not show in another.  (The largest exponent of a row is that of its
            // largest product: fmaf rounds in order.)
            if (__any_sync(0xffffffffu, top > kMost)) {
#pragma unroll
                for (int b = 0; b < NT; ++b)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        bool v[4];
                        float best = -INFINITY;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            v[x] = seen || vis(x >> 1, b, y + 2 * (x & 1));
                            best = fmaxf(best, v[x] ? sc[x >> 1][b][y + 2 * (x & 1)] : -INFINITY);
                        }
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, d));
                        const bool raise = fmaf(best, fac[b][y], -m[b][y]) > kMost;
                        const float m_new = raise ? fmaf(best, fac[b][y], -kFp4Start) : m[b][y];
                        const float keep = raise ? ex2(m[b][y] - m_new) : 1.0f;
                        m[b][y] = m_new;
                        l[b][y] *= keep;
#pragma unroll
                        for (int z = 0; z < kSteps; ++z) {
                            acc[b][z][y] *= keep;
                            acc[b][z][y + 2] *= keep;
                        }
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            ex[x >> 1][b][y + 2 * (x & 1)] =
                                v[x] ? fmaf(sc[x >> 1][b][y + 2 * (x & 1)], fac[b][y], -m_new) : -INFINITY;
                    }
            }
            uint32_t pt[2][NT][2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int b = 0; b < NT; ++b) {
                    float p[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        p[y] = ex2(ex[h][b][y]);
                        l[b][y & 1] += p[y];
                    }
                    pt[h][b][0] = transpose8(bits(__floats2half2_rn(p[0], p[1])));
                    pt[h][b][1] = transpose8(bits(__floats2half2_rn(p[2], p[3])));
                }
            // O^T += V^T P^T
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t vw[4][kVW], vs[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const uint8_t* src = at + off_v[y & 1] + (16 * h + 8 * (y >> 1)) * (D / 2);
                    if constexpr (D == 128) *reinterpret_cast<uint2*>(vw[y]) = *reinterpret_cast<const uint2*>(src);
                    else vw[y][0] = *reinterpret_cast<const uint32_t*>(src);
                    vs[y] = at[off_vs[y & 1] + (16 * h + 8 * (y >> 1)) * (D / 16)];
                }
                if (h == 1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(done);
                }
                const __half2 sf = fp4_scales(__byte_perm(vs[0], vs[1], 0x40)), se = fp4_scales(__byte_perm(vs[2], vs[3], 0x40));
                constexpr uint32_t kLow = 0x0f0f0f0fu;
#pragma unroll
                for (int wd = 0; wd < kVW; ++wd) {
                    __half2 f0[4], f1[4], e0[4], e1[4];
                    const uint32_t a0 = vw[0][wd], a1 = vw[1][wd], a2 = vw[2][wd], a3 = vw[3][wd];
                    fp4_levels((a0 & kLow) | (a1 << 4 & ~kLow), f0);
                    fp4_levels((a0 >> 4 & kLow) | (a1 & ~kLow), f1);
                    fp4_levels((a2 & kLow) | (a3 << 4 & ~kLow), e0);
                    fp4_levels((a2 >> 4 & kLow) | (a3 & ~kLow), e1);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint32_t op[4] = {bits(__hmul2(f0[y], sf)), bits(__hmul2(f1[y], sf)), bits(__hmul2(e0[y], se)),
                                                bits(__hmul2(e1[y], se))};
#pragma unroll
                        for (int b = 0; b < NT; ++b) mma16816(acc[b][4 * wd + y], op, pt[h][b][0], pt[h][b][1]);
                    }
                }
            }
        }
        if (!ok) break;

        // ---- this warp's part
        if (!wait_warp(smem_u32(&sh.freed), (k & 1u) ^ 1u, &sh.watch, status)) {
            ok = false;
            break;
        }
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[b][y] += __shfl_xor_sync(0xffffffffu, l[b][y], d);
                const int row = 8 * b + 2 * c + y;
                if (row < nrows) {
                    if (r == 0) sh.ml[warp][row] = make_float2(m[b][y], l[b][y]);
                    float* to = so + (warp * R + row) * kRowO + r * (D / 8);
#pragma unroll
                    for (int z = 0; z < kSteps; z += 2)
                        *reinterpret_cast<float4*>(to + 2 * z) =
                            make_float4(acc[b][z][y], acc[b][z][y + 2], acc[b][z + 1][y], acc[b][z + 1][y + 2]);
                }
            }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.joined));
    }
    if (!ok && lane == 0) set_abort(&sh.watch, status);
}

// ---------------------------------------------------------------- host side
// Workspace: joins, maxima and sums, O parts; then the tokens' lists.
struct Layout {
    size_t joins, ml, o, total;
    struct Lists {  // of tiles of tpt tokens
        size_t cnt, list, who;
        int32_t tpt, rows, cap, words;
    } lists[2];     // few rows, many
};
Layout layout(const PagedForwardArgs& a) {
    Layout L{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at += (bytes + 255) & ~(size_t)255;
        return p;
    };
    // rows of all parts, of either kernel (one comes after the other)
    constexpr size_t few = (size_t)kPagedBlocks * 2 * 8 * kMaxNT, many = (size_t)kPagedBlocks * 2 * kFp4PromptWide;
    L.joins = take(sizeof(int4) * kPagedBlocks);
    L.ml = take(sizeof(float2) * (few > many ? few : many));
    L.o = take(sizeof(float) * (few > many ? few : many) * (size_t)a.D);
    if (a.sel_width > 0) {
        const int64_t blocks = ((int64_t)a.max_pages * a.page + 127) / 128;
        for (int x = 0; x < 2; ++x) {
            Layout::Lists& l = L.lists[x];
            l.tpt = x == 0 ? 1 : kFp4PromptWide / (a.H / a.H_kv);
            const int64_t most = (int64_t)l.tpt * a.sel_width;
            l.cap = (int32_t)(blocks < most ? blocks : most);
            l.words = (l.tpt + 31) / 32;
            l.rows = a.tokens / l.tpt + a.seqs;
            const size_t rows = (size_t)a.H_kv * l.rows;
            l.cnt = take(sizeof(int32_t) * rows);
            l.list = take(sizeof(int32_t) * rows * l.cap);
            l.who = take(sizeof(uint32_t) * rows * l.cap * l.words);
        }
    }
    L.total = at;
    return L;
}

template <int D, int NT, int kMode>
bsa_status launch_rows(const Fp4Params& P, cudaStream_t stream) {
    using C = Cfg<D, NT>;
    constexpr size_t most = 128 + C::kSmem > 3 * sizeof(int32_t) * 16384 ? 128 + C::kSmem : 128 + 3 * sizeof(int32_t) * 16384;  // (of 16384 sequences)
    const size_t lists = 3 * sizeof(int32_t) * (size_t)P.b.seqs;
    const size_t smem = 128 + (C::kSmem > lists ? C::kSmem : lists);
    static DeviceSetup setup;
    static int sms[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
    const bool ready = setup.once(dev, [&] {
        return cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
               cudaFuncSetAttribute(k_fp4_rows<D, NT, kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) ==
                   cudaSuccess;
    });
    if (!ready) return BSA_ERR_CUDA;
    const int grid = sms[dev] < kPagedBlocks ? sms[dev] : kPagedBlocks;
    if (launch_chained(k_fp4_rows<D, NT, kMode>, dim3((unsigned)grid), C::kThreads, smem, stream, P) != cudaSuccess ||
        launch_chained(k_fp4_join<D, 8 * NT, 1>, dim3((unsigned)grid, 8 * NT), kFp4JoinThreads, 0, stream, P) !=
            cudaSuccess)
        return BSA_ERR_CUDA;
    return BSA_OK;
}

template <int kMode>
bsa_status launch_mode(const Fp4Params& P, int32_t D, bool wide, cudaStream_t stream) {
    if (D == 128) return wide ? launch_rows<128, 2, kMode>(P, stream) : launch_rows<128, 1, kMode>(P, stream);
    return wide ? launch_rows<64, 2, kMode>(P, stream) : launch_rows<64, 1, kMode>(P, stream);
}

}  // namespace

size_t fp4_forward_workspace(const PagedForwardArgs& a) { return layout(a).total; }

bsa_status launch_fp4_forward(const Fp4ForwardArgs& x, void* workspace, int32_t* status, cudaStream_t stream) {
    const PagedForwardArgs& a = x.f;
    const Layout L = layout(a);
    Fp4Params P;
    memset(&P, 0, sizeof(P));
    P.b = PagedBatch{a.q_start, a.kv_len, a.table, a.seqs, a.tokens, a.max_pages, a.page, a.n_pages, status};
    P.k = static_cast<const uint8_t*>(a.k_cache);
    P.v = static_cast<const uint8_t*>(a.v_cache);
    P.k_scale = static_cast<const uint8_t*>(x.k_scale);
    P.v_scale = static_cast<const uint8_t*>(x.v_scale);
    P.k_gain = x.k_gain;
    P.v_gain = x.v_gain;
    P.q = static_cast<const __nv_bfloat16*>(a.q);
    P.q_stride = a.q_stride;
    if (a.page < kFp4LongPage) {
        auto enc = get_encode();
        // (in elements of eight bytes: a box is at most 256 of them long)
        auto encode = [&](CUtensorMap* map, const void* base, int32_t row_bytes) {
            const cuuint64_t bytes = (cuuint64_t)a.page * row_bytes, dims[2] = {bytes / 8, (cuuint64_t)a.n_pages * a.H_kv};
            const cuuint32_t box[2] = {(cuuint32_t)(bytes / 8), 1}, ones[2] = {1, 1};
            return enc && enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, 2, const_cast<void*>(base), dims, &bytes, box, ones,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
        };
        if (!encode(&P.map_k, a.k_cache, a.D / 2) || !encode(&P.map_v, a.v_cache, a.D / 2) ||
            !encode(&P.map_ks, x.k_scale, a.D / 16) || !encode(&P.map_vs, x.v_scale, a.D / 16))
            return BSA_ERR_CUDA;
    }
    P.H = a.H;
    P.H_kv = a.H_kv;
    P.group = a.H / a.H_kv;
    P.causal = a.causal;
    P.window = a.window < kMaxWindow ? a.window : kMaxWindow;
    P.sinks = a.sinks;
    P.scale_log2 = (a.scale > 0.f ? a.scale : 1.0f / sqrtf((float)a.D)) * kLog2e;
    P.o = static_cast<__nv_bfloat16*>(a.o);
    P.lse = a.lse;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    P.joins = reinterpret_cast<int4*>(ws + L.joins);
    P.part_ml = reinterpret_cast<float2*>(ws + L.ml);
    P.part_o = reinterpret_cast<float*>(ws + L.o);
    P.least = 1;
    P.most = INT32_MAX;
    // Rows of a sequence, at most, as far as the host knows.  Row tiles of 16 for tokens of more than eight rows and
    // where some sequence has 9 to 16 (64 x 4 tokens of 4 rows over 4096: 110 us, 126 with two tiles of 8), else
    // of 8 (64 tokens over up to 8192: 101 us, 143 with tiles of 16).
    const int64_t most = (int64_t)(x.max_new > 0 && x.max_new < a.tokens ? x.max_new : a.tokens) * P.group;
    const bool wide = P.group > 8 || (a.sel == nullptr && most > 8 && most <= kFewRows);
    // Tokens of few rows take the blocks that they list one by one; of many, a tile of tokens takes what any of them lists,
    // whose bits say who (2048 tokens over 257 blocks, 66 random ones each: 3250 us one by one, 878).
    auto with_lists = [&](int x) -> bsa_status {
        const Layout::Lists& l = L.lists[x];
        int32_t* cnt = reinterpret_cast<int32_t*>(ws + l.cnt);
        int32_t* list = reinterpret_cast<int32_t*>(ws + l.list);
        uint32_t* who = reinterpret_cast<uint32_t*>(ws + l.who);
        P.list = list;
        P.list_cnt = cnt;
        P.who = who;
        P.nt_cap = l.rows;
        P.cap = l.cap;
        P.words = l.words;
        P.tpt = l.tpt;
        return launch_paged_union(a, l.tpt, l.rows, l.cap, l.words, list, cnt, who, status, stream, P.least, P.most);
    };
    // sequences of few rows here, the others on large tiles, unless the host knows of no others (what it
    // was told may be wrong: then all of them are done here)
    // One sequence that may have many: all of it there, whatever it has (two launches less: 64 tokens over 4096 26.9 -> 22.4 us,
    // a prompt of 8192 470 -> 454.  A single token where 256 may come, over 1000 keys, 12.6 us, over 131072 64; whoever
    // tells max_new = 1 has it in 9.7 and 38.)
    const bool lists = a.sel != nullptr;
    const int32_t few = lists && P.group <= 16 ? kFewListed * P.group : kFewRows;
    if (a.seqs == 1 && most > few) {
        if (lists) {
            const bsa_status c = with_lists(1);
            if (c != BSA_OK) return c;
        }
        return launch_fp4_prompt(P, a.D, true, stream);
    }
    P.most = most > few ? few : INT32_MAX;
    bsa_status c = lists ? with_lists(0) : BSA_OK;
    if (c != BSA_OK) return c;
    c = lists          ? launch_mode<kListed>(P, a.D, wide, stream)
        : a.window > 0 ? launch_mode<kWindow>(P, a.D, wide, stream)
                       : launch_mode<kPlain>(P, a.D, wide, stream);
    if (c != BSA_OK || most <= few) return c;
    P.least = few + 1;
    P.most = INT32_MAX;
    if (lists) {
        c = with_lists(1);
        if (c != BSA_OK) return c;
    }
    return launch_fp4_prompt(P, a.D, false, stream);
}

}  // namespace bsa
