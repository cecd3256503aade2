// Attention over a paged key/value cache held in 4 bits, for sequences with many new rows
// (chunks, prompts), on the tensor core's large tiles (tcgen05 + TMEM).  What it computes, and how
// rows are laid out and cut, is bsa_fp4_attn.cu's and bsa_fp4_runs.cuh's.
//
// A row tile is 128 rows, S = Q K^T and O += P V are 128 x 128 (x D) products of fp16 operands.
// Warps (20):
//   0         cuts the run into segments, tells them to the others through a ring of descriptors and
//             loads codes and scales of key tiles (pages of 16: K's, and warp 3 V's)
//   1, 2      issue Q K^T and P V
//   4 .. 11   are the softmax (four threads a row, see bsa_rows.cuh)
//   12 .. 15  unpack V's codes to fp16 tiles in the swizzled layout the products read (levels times
//             scales, exact), and normalise and store a segment's rows while the softmax is at the next
//   16 .. 19  unpack K's codes
//   12 .. 19  put the segment's queries in place, 16 rows each: a row times the power of two that brings
//             its largest value to 2^14, rounded to fp16
// Shared memory: the Q tile, two K and two V tiles (four with D = 64), three tiles of codes.  Tensor memory:
// three score buffers and O.  Tiles are numbered through the whole run, across the borders of segments.
//
// What bounds it.  A prompt of 8192 (32 + 8 heads of 128): 455 us, 1.21 PFLOP/s of visible products, 0.63 of the
// burst rate of a plain product; the tensor pipe is busy half the time.  The softmax takes some 1,750
// cycles a key tile (the products 1,024) beside the unpacking warps, which issue every third
// instruction (issue slots 65 % full): so much where segments are long (a chunk of 1024 over 64512: 781 us,
// 1.40 PFLOP/s, 0.73, 856 key tiles a thread block).  The rest is by row tile: a block of the prompt has 438 key tiles
// and 13.5 row tiles, which leaves some 9,000 cycles for a row tile's start, end and masked tile (queries are put in
// place after the segment before is through with theirs); through a window of 575 + 64 sinks (105 us, 45.5 key tiles and
// 6.7 row tiles a block) it leaves 18,000.
// One set of warps for K, V and the queries took 897 us; K's and V's apart 530; the same
// loop for both, so that it stays in the instruction cache, and each query load in its own register 470.
// Slower, when the prompt took 460: row tiles of 256, each unpacked tile used twice, with one tile of codes and two score
// buffers (510 us: unpacking is not what bounds it, and loads and buffers are missed); queries through the ring
// of codes (484); a segment told and its queries loaded before the end of the one before (485 and 495).
// All warps share 96 registers a thread: what the softmax holds over a tile decides the time (see softmax_rows).
//
// Rounding.  Weights are rounded to fp16 for the product P V; they start at 2^6 (kFp4Start) and stay below 2^16 against
// an earlier maximum of their row (see softmax_rows).  Row sums add them unrounded.
//
// Lists.  A row tile is as many whole tokens as 128 rows hold, and its key tiles are those that any of its tokens
// lists; a bit for each token says whose.  The rows of a token that does not list a tile take no part in it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "bsa_device_setup.h"
#include "bsa_fp4.cuh"
#include "bsa_fp4_runs.cuh"
#include "bsa_internal.h"
#include "bsa_paged.cuh"
#include "bsa_paged_wait.cuh"
#include "bsa_rows.cuh"

namespace bsa {
namespace {

constexpr int kWide = kFp4PromptWide;
// A row tile of n key tiles counts n + row_cost in a run.  (A causal prompt of 8192, whose blocks
// have 8 to 50 row tiles each: 453 us with 4, 471 with 8, 490 with 12; two chunks of 2048 through a window of
// 575, 6 key tiles to a row tile: 117, 110, 107 us.)
constexpr int32_t row_cost(int mode) { return mode == 1 ? 12 : 4; }
constexpr float kSumLimit = 65504.0f;                     // fp16's largest number, see softmax_rows
constexpr int kSBuf = 3;                                  // TMEM score buffers
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 384;
constexpr int kLoad = 0, kMmaQK = 1, kMmaPV = 2, kLoadV = 3, kSoftmax0 = 4, kSoftmaxWarps = 8, kUnpackV0 = 12, kUnpackK0 = 16,
              kUnpackWarps = 4;
constexpr int kThreads = 32 * 20;
constexpr int kDesc = 4;                                  // segment descriptors in flight
constexpr int kReaders = 3 + kSoftmaxWarps + 2 * kUnpackWarps;  // warps that read a descriptor
constexpr int kBox = 128 * 128;                           // 128 rows of 64 fp16

enum { kPlain = 0, kWindow = 1, kListed = 2 };

template <int D>
struct Cfg {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = kBox * kHalves;
    static constexpr int kTiles = D == 128 ? 2 : 4;       // K tiles, and V tiles
    static constexpr int kCodeStages = 3;
    static constexpr int kCodes = 128 * D / 2, kScales = 128 * D / 16;
    static constexpr int kStage = 2 * (kCodes + kScales);
    static constexpr int kTilesData = kTile * (1 + 2 * kTiles) + kCodeStages * kStage;
    static constexpr int kLists = 3 * 4 * 16384;          // three words for each of as many sequences as there may be
    static constexpr int kData = kTilesData > kLists ? kTilesData : kLists;
    static constexpr uint32_t kIdescQK = idesc_f16_f32(128, 128, 0, 0);
    static constexpr uint32_t kIdescPV = idesc_f16_f32(128, D, 0, 1);
};

struct Shared {
    uint64_t code_full[3], code_empty[3];
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
    uint64_t q_ready[kDesc], q_empty;
    uint64_t s_full[kSBuf];   // S_g is there
    uint64_t p_full[kSBuf];   // P_g has been written (and O rescaled)
    uint64_t pv_done[kSBuf];  // O holds P_g V_g
    uint64_t o_free;          // the segment's O has been read
    uint64_t ml_full, ml_empty;  // a segment's maxima and sums are in ml, have been read
    uint64_t mma_done;
    uint64_t seg_full[kDesc], seg_empty[kDesc];
    Watch watch;
    Fp4Segment seg[kDesc];
    float fac[kDesc][kWide];  // of a segment's rows: what turns a product of operands into a score (log2)
    float2 ml[kWide];         // of a segment's rows: maximum (log2) and sum
    Fp4Start start;
    uint32_t tmem_base;
};

__device__ __forceinline__ uint32_t bits(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ void store16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    // (no "memory": what is loaded next need not wait for it; publish() orders it before what reads it)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d));
}

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const Watch* w, const int32_t* status) {
    return __all_sync(0xffffffffu, paged_wait(bar, parity, w, status));
}

// Which of a thread's columns 8 kk and 8 kk + 1 (kk = 0 .. 15; bit 2 kk and the
// next) are below v.
__device__ __forceinline__ uint32_t columns_below(int32_t v) {
    const int32_t n = v <= 0 ? 0 : 2 * (v >> 3) + min(v & 7, 2);
    return n >= 32 ? ~0u : (1u << n) - 1u;
}

// exp_rows of bsa_rows.cuh with a factor for each row and fp16 weights.
__device__ __forceinline__ void exp_rows_f16(uint32_t (&s)[64], const float (&f)[2], float bias_a, float bias_b, float& la,
                                             float& lb) {
    const uint64_t fa = f2pack(f[0], f[0]), fb = f2pack(f[1], f[1]), ba = f2pack(bias_a, bias_a), bb = f2pack(bias_b, bias_b);
    uint64_t acc_a0 = f2pack(0.f, 0.f), acc_a1 = acc_a0, acc_b0 = acc_a0, acc_b1 = acc_a0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        float x[4];
        f2unpack(fma2(f2pack(__uint_as_float(s[4 * k]), __uint_as_float(s[4 * k + 1])), fa, ba), x[0], x[1]);
        f2unpack(fma2(f2pack(__uint_as_float(s[4 * k + 2]), __uint_as_float(s[4 * k + 3])), fb, bb), x[2], x[3]);
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = ex2(x[i]);
        if (k & 1) {
            acc_a1 = add2(acc_a1, f2pack(p[0], p[1]));
            acc_b1 = add2(acc_b1, f2pack(p[2], p[3]));
        } else {
            acc_a0 = add2(acc_a0, f2pack(p[0], p[1]));
            acc_b0 = add2(acc_b0, f2pack(p[2], p[3]));
        }
        s[2 * k] = bits(__floats2half2_rn(p[0], p[1]));
        s[2 * k + 1] = bits(__floats2half2_rn(p[2], p[3]));
    }
    float x0, x1;
    f2unpack(add2(acc_a0, acc_a1), x0, x1);
    la = x0 + x1;
    f2unpack(add2(acc_b0, acc_b1), x0, x1);
    lb = x0 + x1;
}

// One key tile of the online softmax for this thread's shares of rows a and b.
// hidden: the row sees nothing of the tile (its weights are 0).  A row that has seen no key yet has
// m = kFp4NoKey; one that holds no token has scores of 0.  Exponentials are taken against the running maxima
// without computing the tile's own.  Where a row's sums leave fp16's range (its first key makes them infinite) or are
// NaN, the tile is redone with that row's new maximum, and against the maxima that the warp's other rows had,
// to the same bits: what one row holds does not show in another.  first: no row of the warp has seen a key, and
// all take their first maximum at once.  Returns true (warp-uniform) when O must be multiplied by alpha first.
// A tile redone for one row holds up 128, some 600 cycles, most of them the wait for instructions that have left the cache.
// (Prompt of 8192: the votes of both rows kept as they come 456 us; made truth values 492, one mask 454, but lists of 2048
// tokens 878, 914, 936; maxima looked for at tiles 1, 2, 4, .. so that fewer rows pass their limit 510 and more.)
template <typename Reload>
__device__ __forceinline__ bool softmax_rows(uint32_t (&s)[64], const bool (&hidden)[2], const float (&f)[2], bool first, float (&m)[2],
                                             float (&l)[2], float (&alpha)[2], Reload&& reload) {
    alpha[0] = alpha[1] = 1.0f;
    float la, lb;
    uint32_t over[2] = {~0u, ~0u};  // lanes whose share of their row a, b has left the limit
    if (!first) {
        exp_rows_f16(s, f, hidden[0] ? -INFINITY : -m[0], hidden[1] ? -INFINITY : -m[1], la, lb);
        over[0] = __ballot_sync(0xffffffffu, !(la <= kSumLimit));
        over[1] = __ballot_sync(0xffffffffu, !(lb <= kSumLimit));
        if ((over[0] | over[1]) == 0u) {
            l[0] += la;
            l[1] += lb;
            return false;
        }
        reload();
    }
    float mt[2];
    max_rows(s, mt[0], mt[1]);
    bool raised = false;
    float bias[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        mt[i] = fmaf(mt[i], f[i], -kFp4Start);
        // (a row's four threads are neighbours)
        if ((over[i] >> (threadIdx.x & 28u) & 15u) != 0u && !hidden[i] && mt[i] > m[i]) {
            alpha[i] = ex2(m[i] - mt[i]);
            raised |= m[i] != kFp4NoKey;  // (else O and l are 0 still)
            l[i] *= alpha[i];
            m[i] = mt[i];
        }
        bias[i] = hidden[i] ? -INFINITY : -m[i];
    }
    exp_rows_f16(s, f, bias[0], bias[1], la, lb);
    l[0] += la;
    l[1] += lb;
    return !first && __any_sync(0xffffffffu, raised);
}

template <int D, int kMode>
__global__ void __launch_bounds__(kThreads, 1) k_fp4_prompt(const __grid_constant__ Fp4Params P) {
    using C = Cfg<D>;
    constexpr bool kLists = kMode == kListed;
    constexpr uint32_t S = C::kTiles, CS = C::kCodeStages;
    extern __shared__ uint8_t smem_raw[];
    // (an offset, not a rounded pointer: the compiler has to see that it is shared memory)
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    const uint32_t s_q = smem_u32(smem), s_k = s_q + C::kTile, s_v = s_k + S * C::kTile;
    uint8_t* const codes = smem + C::kTile * (1 + 2 * S);
    Shared& sh = *reinterpret_cast<Shared*>(smem + C::kData);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    int32_t* const status = P.b.status;
    // pages of 16 have too many copies for one warp (a prompt of 8192: 531 us with one, 472 with two; pages of 128 454, 459)
    const bool two_load = P.b.page < 32;

    if (threadIdx.x == kThreads - 1) {
        for (int x = 0; x < 3; ++x) {
            mbar_init(smem_u32(&sh.code_full[x]), two_load ? 2 : 1);
            mbar_init(smem_u32(&sh.code_empty[x]), 2 * kUnpackWarps);
        }
        for (int x = 0; x < 4; ++x) {
            mbar_init(smem_u32(&sh.k_full[x]), kUnpackWarps);
            mbar_init(smem_u32(&sh.v_full[x]), kUnpackWarps);
            mbar_init(smem_u32(&sh.k_empty[x]), 1);
            mbar_init(smem_u32(&sh.v_empty[x]), 1);
        }
        for (int x = 0; x < kSBuf; ++x) {
            mbar_init(smem_u32(&sh.s_full[x]), 1);
            mbar_init(smem_u32(&sh.p_full[x]), 32 * kSoftmaxWarps);
            mbar_init(smem_u32(&sh.pv_done[x]), 1);
        }
        mbar_init(smem_u32(&sh.q_empty), 1);
        mbar_init(smem_u32(&sh.o_free), 32 * kUnpackWarps);
        mbar_init(smem_u32(&sh.ml_full), 32 * kSoftmaxWarps);
        mbar_init(smem_u32(&sh.ml_empty), 32 * kUnpackWarps);
        mbar_init(smem_u32(&sh.mma_done), 2);
        for (int x = 0; x < kDesc; ++x) {
            mbar_init(smem_u32(&sh.q_ready[x]), 2 * kUnpackWarps);
            mbar_init(smem_u32(&sh.seg_full[x]), 1);
            mbar_init(smem_u32(&sh.seg_empty[x]), kReaders);
        }
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
    // this block's run (the scratch is in the data area, which is free here)
    constexpr int kScan = 256;
    if (threadIdx.x < kScan)
        Fp4Work<kWide, row_cost(kMode), kLists>{P}.template find<kScan>(reinterpret_cast<int32_t*>(smem), sh.start);
    __syncthreads();
    if (sh.start.any == 0) return;
    const bool abandoned = sh.watch.abort != 0;
    if (warp == kMmaQK && !abandoned) {
        __syncwarp();
        tmem_alloc(smem_u32(&sh.tmem_base), kTmemCols);
        tmem_relinquish();
    }
    // what was written there by ordinary stores makes room for bulk copies
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (abandoned) return;
    const uint32_t tmem = sh.tmem_base;

    // Segment k, for the warps that read descriptors (null: no more); they hand
    // it back when they are through with it.
    auto next_segment = [&](uint32_t k, bool& ok) -> const Fp4Segment* {
        if (!wait_warp(smem_u32(&sh.seg_full[k % kDesc]), (k / kDesc) & 1u, &sh.watch, status)) {
            ok = false;
            return nullptr;
        }
        const Fp4Segment* sg = &sh.seg[k % kDesc];
        return sg->n >= 0 ? sg : nullptr;
    };
    auto hand_back = [&](uint32_t k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.seg_empty[k % kDesc]));
    };
    // No product may still be running when TMEM is freed.
    auto finish_products = [&](bool ok) {
        if (elect_one()) mma_commit(smem_u32(&sh.mma_done));
        __syncwarp();
        if (!ok || !wait_warp(smem_u32(&sh.mma_done), 0, &sh.watch, status)) {
            if (ok && lane == 0) set_abort(&sh.watch, status);
            paged_drain(smem_u32(&sh.mma_done), 0, status);
        }
        __syncwarp();
    };

    if (warp < kSoftmax0) {
        // The codes and scales of a segment's tiles, whose numbers in the run begin at g: K's, V's or both.
        auto load_tiles = [&](const Fp4Segment& sg, bool k_too, bool v_too, uint32_t& g) -> bool {
            const int32_t page = P.b.page, N = 128 / page, per_window = page >> 2;  // pages of a tile; tiles whose pages one read of 32 lanes brings
            const int32_t lane_tile = lane / N, lane_page = lane - lane_tile * N;
            const int32_t j0 = sg.j0, j1 = j0 + sg.n;
            const int32_t* table = P.b.table + (int64_t)sg.seq * P.b.max_pages;
            const int32_t* list = kLists ? P.list + ((int64_t)sg.kvh * P.nt_cap + sg.tile) * P.cap : nullptr;
            const uint32_t to_codes = smem_u32(codes) + lane_page * page * (D / 2);
            const uint32_t to_scales = smem_u32(codes) + 2 * C::kCodes + lane_page * page * (D / 16);
            // lane l of a window: the cache row of page l % N of tile w0 + l / N (-1: behind the
            // sequence's end)
            auto fetch = [&](int32_t w0) -> int32_t {
                const int32_t j = w0 + lane_tile;
                if (j >= j1) return -1;
                int32_t tile;
                if constexpr (kLists) tile = list[j];
                else tile = j < sg.ns ? j : sg.lo + j - sg.ns;
                const int32_t pg = tile * N + lane_page;
                if (pg * page >= sg.kl) return -1;
                int32_t id = table[pg];
                if (id < 0 || id >= P.b.n_pages) {
                    raise_status(status, BSA_ERR_BOUNDS);
                    id = 0;  // (this row's result is unspecified)
                }
                return (id * P.H_kv + sg.kvh) * page;
            };
            int32_t w0 = j0, cur = fetch(j0), nxt = fetch(j0 + per_window);
            for (int32_t j = j0; j < j1; ++j, ++g) {
                if (j >= w0 + per_window) {
                    w0 += per_window;
                    cur = nxt;
                    nxt = fetch(w0 + per_window);
                }
                const bool live = lane_tile == j - w0;
                const int32_t row = live ? cur : -1, first = __shfl_sync(0xffffffffu, cur, (j - w0) * N);
                const int32_t held = __popc(__ballot_sync(0xffffffffu, row >= 0));
                const uint32_t at = g % CS, bar = smem_u32(&sh.code_full[at]), stage = at * C::kStage;
                if (!wait_warp(smem_u32(&sh.code_empty[at]), ((g / CS) & 1u) ^ 1u, &sh.watch, status)) return false;
                if (lane == 0) mbar_arrive_expect_tx(bar, (k_too && v_too ? 2 : 1) * fp4_page_bytes(page, held, D / 2 + D / 16));
                __syncwarp();
                if (k_too) {
                    fp4_load_pages(P.k, &P.map_k, page, D / 2, live, row, first, to_codes + stage, bar);
                    fp4_load_pages(P.k_scale, &P.map_ks, page, D / 16, live, row, first, to_scales + stage, bar);
                }
                if (v_too) {
                    fp4_load_pages(P.v, &P.map_v, page, D / 2, live, row, first, to_codes + stage + C::kCodes, bar);
                    fp4_load_pages(P.v_scale, &P.map_vs, page, D / 16, live, row, first, to_scales + stage + C::kScales, bar);
                }
                __syncwarp();
            }
            return true;
        };
        // (every issued copy must land before the block exits)
        auto land = [&](uint32_t g) {
            if (lane == 0)
                for (uint32_t x = g > CS ? g - CS : 0; x < g; ++x)
                    paged_drain(smem_u32(&sh.code_full[x % CS]), (x / CS) & 1u, status);
            __syncwarp();
        };
        if (warp == kLoad) {
            // -------------------------------------------------------- segments, codes and scales
            Fp4Walk<kWide, row_cost(kMode), kLists> walk(P, sh.start);
            Fp4Segment sg;
            uint32_t k = 0, g = 0;  // segments and tiles so far
            bool ok = true;
            for (; ok && walk.open(sg); walk.advance()) {
                if (!wait_warp(smem_u32(&sh.seg_empty[k % kDesc]), ((k / kDesc) & 1u) ^ 1u, &sh.watch, status)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    sh.seg[k % kDesc] = sg;
                    mbar_arrive(smem_u32(&sh.seg_full[k % kDesc]));
                    walk.note(sg);
                }
                __syncwarp();
                ++k;
                // the queries, which others will wait for, into L2
                for (int32_t row = lane; row < sg.nrows; row += 32) {
                    const int32_t z = sg.row0 + row, tok = z / P.group, head = z - tok * P.group;
                    const __nv_bfloat16* src = P.q + ((int64_t)sg.q0 + tok) * P.q_stride + (int64_t)(sg.kvh * P.group + head) * D;
#pragma unroll
                    for (int d = 0; d < D; d += 64) prefetch_l2(src + d);
                }
                ok = load_tiles(sg, true, !two_load, g);
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
        } else if (warp == kLoadV) {
            // -------------------------------------------------------- V's codes, of short pages
            uint32_t g = 0;
            bool ok = true;
            for (uint32_t k = 0; ok; ++k) {
                const Fp4Segment* sp = next_segment(k, ok);
                if (sp == nullptr) break;
                const Fp4Segment sg = *sp;
                hand_back(k);
                if (two_load) ok = load_tiles(sg, false, true, g);
            }
            if (!ok && lane == 0) set_abort(&sh.watch, status);
            land(g);
        } else if (warp == kMmaQK) {
            // -------------------------------------------------------- S = Q K^T
            // (the whole warp walks the schedule; one elected lane issues a tile's MMAs
            // and their commits)
            const uint64_t dq = smem_desc_sw128(s_q, 16, 1024);
            const uint64_t dk = smem_desc_sw128(s_k, 16, 1024);
            uint32_t g = 0;
            bool ok = true;
            for (uint32_t k = 0; ok; ++k) {
                const Fp4Segment* sp = next_segment(k, ok);
                if (sp == nullptr) break;
                const int32_t n = sp->n;
                // (the descriptor guards q_ready's phase too: handed back before, and with segments behind it that have
                // no key and so nothing of this warp to wait for, the phase could go by unseen)
                if (n > 0) ok = wait_warp(smem_u32(&sh.q_ready[k % kDesc]), (k / kDesc) & 1u, &sh.watch, status);
                hand_back(k);
                if (n == 0) continue;
                for (int32_t j = 0; j < n && ok; ++j, ++g) {
                    // S buffer g % 3 is free once PV_{g-3} has read P_{g-3}
                    if (g >= kSBuf) ok = wait_warp(smem_u32(&sh.pv_done[g % kSBuf]), (g / kSBuf - 1u) & 1u, &sh.watch, status);
                    const uint32_t slot = g % S;
                    ok = ok && wait_warp(smem_u32(&sh.k_full[slot]), (g / S) & 1u, &sh.watch, status);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ks = dk + (uint64_t)((slot * C::kTile) >> 4);
                    const uint32_t d_col = (g % kSBuf) * 128u;
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = ((kk >> 2) * kBox + (kk & 3) * 32) >> 4;
                            mma_ss(tmem + d_col, dq + off, ks + off, C::kIdescQK, kk > 0 ? 1u : 0u);
                        }
                        mma_commit(smem_u32(&sh.s_full[g % kSBuf]));
                        mma_commit(smem_u32(&sh.k_empty[slot]));
                        if (j == n - 1) mma_commit(smem_u32(&sh.q_empty));
                    }
                    __syncwarp();
                }
            }
            if (!ok && lane == 0) set_abort(&sh.watch, status);
            finish_products(ok);
        } else if (warp == kMmaPV) {
            // -------------------------------------------------------- O += P V
            const uint64_t dv = smem_desc_sw128(s_v, kBox, 1024);
            uint32_t g = 0, segs = 0;
            bool ok = true;
            for (uint32_t k = 0; ok; ++k) {
                const Fp4Segment* sp = next_segment(k, ok);
                if (sp == nullptr) break;
                const int32_t n = sp->n;
                hand_back(k);
                if (n == 0) continue;
                for (int32_t j = 0; j < n && ok; ++j, ++g) {
                    const uint32_t slot = g % S;
                    ok = wait_warp(smem_u32(&sh.v_full[slot]), (g / S) & 1u, &sh.watch, status) &&
                         wait_warp(smem_u32(&sh.p_full[g % kSBuf]), (g / kSBuf) & 1u, &sh.watch, status);
                    // a segment's first product overwrites O: the epilogue before must have read it
                    if (ok && j == 0 && segs > 0) ok = wait_warp(smem_u32(&sh.o_free), (segs - 1u) & 1u, &sh.watch, status);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t vs = dv + (uint64_t)((slot * C::kTile) >> 4);
                    const uint32_t p_col = (g % kSBuf) * 128u;
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            mma_ts(tmem + kColO, tmem + p_col + kk * 8, vs + (uint64_t)(kk * 2048 >> 4), C::kIdescPV,
                                   (j > 0 || kk > 0) ? 1u : 0u);
                        mma_commit(smem_u32(&sh.pv_done[g % kSBuf]));
                        mma_commit(smem_u32(&sh.v_empty[slot]));
                    }
                    __syncwarp();
                }
                ++segs;
            }
            if (!ok && lane == 0) set_abort(&sh.watch, status);
            finish_products(ok);
        }
    } else if (warp >= kUnpackV0) {
        // ------------------------------------------------------------ fp16 tiles of K and Q, of V; O and LSE
        const int uw = warp & 3;
        // 32 keys of a tile by this warp, 32 values (a piece) by a lane at a time; eight lanes store to one
        // box and eight places of its lines (no bank conflicts)
        constexpr int PR = D / 32, kRowsOnce = 32 / PR;  // pieces of a row, rows at a time (a multiple of 8)
        const int piece = D == 128 ? (lane & 1) + (lane >> 2 & 2) : lane & 1;
        const int row0 = 32 * uw + (D == 128 ? (lane >> 1 & 3) + (lane >> 2 & 4) : lane >> 1);
        const uint32_t from_at = row0 * (D / 2) + piece * 16, scale_at = row0 * (D / 16) + piece * 2;
        uint32_t to_at[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
            to_at[y] = (uint32_t)(piece >> 1) * kBox + row0 * 128 + ((uint32_t)((4 * (piece & 1) + y) ^ (row0 & 7)) << 4);
        auto unpack = [&](const uint8_t* from, const uint8_t* scales, uint32_t to) {
            uint4 w[PR];
            uint32_t s2[PR];
#pragma unroll
            for (int x = 0; x < PR; ++x) {
                w[x] = *reinterpret_cast<const uint4*>(from + from_at + x * kRowsOnce * (D / 2));
                s2[x] = *reinterpret_cast<const uint16_t*>(scales + scale_at + x * kRowsOnce * (D / 16));
            }
#pragma unroll
            for (int x = 0; x < PR; ++x) {
                const __half2 both = fp4_scales(s2[x]);
                const __half2 sc[2] = {__low2half2(both), __high2half2(both)};
                const uint32_t wd[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    __half2 v[4];
                    fp4_levels(wd[y], v);
                    store16(to + to_at[y] + x * kRowsOnce * 128, bits(__hmul2(v[0], sc[y >> 1])), bits(__hmul2(v[1], sc[y >> 1])),
                            bits(__hmul2(v[2], sc[y >> 1])), bits(__hmul2(v[3], sc[y >> 1])));
                }
            }
        };
        auto publish = [&](uint64_t* bar) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(bar));
        };
        // A segment's queries: D / 8 lanes a row, eight values each; sixteen rows by this warp (loaded
        // ahead, put in place when the segment before is done with the query tile's place)
        constexpr int kLanes = D / 8, kAbreast = 32 / kLanes, kLot = 16 / kAbreast;
        const int qc = lane % kLanes, q_row = 32 * uw + (warp >= kUnpackK0 ? 0 : 16) + lane / kLanes;
        const uint32_t by_group = (65536u + P.group - 1u) / P.group;  // x / group = x by_group >> 16 for x < 256
        // (a short loop, four rows under way: it runs once a segment, and all unrolled it waits for its own instructions)
        constexpr int kAhead = 4;
        uint4 raw[kAhead];
        const __nv_bfloat16* q_src;
        int32_t q_head0, q_rows;
        auto load_row = [&](int x) -> uint4 {
            const int32_t row = q_row + x * kAbreast, z = q_head0 + row, tok = (int32_t)((uint32_t)z * by_group >> 16);
            return x < kLot && row < q_rows ? *reinterpret_cast<const uint4*>(q_src + tok * P.q_stride + (z - tok * P.group) * D)
                                            : make_uint4(0u, 0u, 0u, 0u);
        };
        auto fetch_rows = [&](const Fp4Segment& sg) {
            const int32_t tok0 = sg.row0 / P.group;
            q_head0 = sg.row0 - tok0 * P.group;
            q_rows = sg.nrows;
            q_src = P.q + ((int64_t)sg.q0 + tok0) * P.q_stride + (int64_t)sg.kvh * P.group * D + 8 * qc;
#pragma unroll
            for (int x = 0; x < kAhead; ++x) raw[x] = load_row(x);
        };
        auto place_rows = [&](const Fp4Segment& sg, uint32_t k) {
            const float kg = (P.k_gain != nullptr ? P.k_gain[sg.kvh] : 1.0f) * P.scale_log2;
            const uint32_t line = s_q + (qc >> 3) * kBox;
            float* fac = sh.fac[k % kDesc];
#pragma unroll 1
            for (int x0 = 0; x0 < kLot; x0 += kAhead) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int row = q_row + (x0 + u) * kAbreast;
                    const uint32_t wd[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
                    raw[u] = load_row(x0 + u + kAhead);  // (in its own place: a move would wait for it)
                    // the row's largest magnitude, by its bits (their order is that of the numbers)
                    uint32_t top = 0u;
#pragma unroll
                    for (int y = 0; y < 4; ++y) top = __vmaxu2(top, wd[y] & 0x7fff7fffu);
#pragma unroll
                    for (int d = 1; d < kLanes; d <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, d));
                    top = max(top & 0xffffu, top >> 16) >> 7;
                    // (a row that holds an infinity or a NaN gets NaN scores, whatever its factor)
                    const int32_t e = min(max((int32_t)top - 127, -100), 127) - 14;
                    const float up = __int_as_float((127 - e) << 23);
                    uint32_t h[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        h[y] = bits(__floats2half2_rn(__uint_as_float(wd[y] << 16) * up, __uint_as_float(wd[y] & 0xffff0000u) * up));
                    store16(line + row * 128 + ((uint32_t)((qc & 7) ^ (row & 7)) << 4), h[0], h[1], h[2], h[3]);
                    // (never 0: a hidden score is -inf, and times 0 it would be NaN)
                    if (qc == 0) fac[row] = fmaxf(__int_as_float((127 + e) << 23) * kg, FLT_MIN);
                }
            }
            publish(&sh.q_ready[k % kDesc]);
        };
        bool ok = true;
        // O and LSE of a segment, one thread per row
        const int row = uw * 32 + lane;  // (a warp reaches TMEM lanes 32 (warp % 4) .. + 31)
        const uint32_t t_row = tmem + ((uint32_t)(uw * 32) << 16) + kColO;
        Fp4Segment was;      // a segment whose rows are still to be stored (n > 0), ..
        uint32_t last = 0u;  // .. and its last tile
        was.n = 0;
        auto address = [&](const Fp4Segment& sg) -> int64_t {
            const int32_t x = sg.row0 + (row < sg.nrows ? row : 0), tok = x / P.group;
            return ((int64_t)sg.q0 + tok) * P.H + sg.kvh * P.group + (x - tok * P.group);
        };
        uint32_t stored = 0u;  // segments whose rows have been stored
        auto store_rows = [&]() {
            const bool dead = row >= was.nrows;
            const int64_t at = address(was);
            __nv_bfloat16* orow = P.o + at * D;
            // (the last product is the segment's: the next one waits for o_free)
            ok = wait_warp(smem_u32(&sh.ml_full), stored & 1u, &sh.watch, status) &&
                 wait_warp(smem_u32(&sh.pv_done[last % kSBuf]), (last / kSBuf) & 1u, &sh.watch, status);
            if (!ok) return;
            const float2 ml = sh.ml[row];
            mbar_arrive(smem_u32(&sh.ml_empty));
            tc_fence_after();
            // 1 / l; 0 for a row without a key, NaN where l is
            // (the gain after the quotient: the smallest gain over a long sum is no normal number)
            const float inv = ml.y == 0.0f ? 0.0f : 1.0f / ml.y, vg = P.v_gain != nullptr ? P.v_gain[was.kvh] : 1.0f;
            const int64_t part = (int64_t)max(was.part, 0) * kWide + row;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                __syncwarp();  // the lanes without a row skip the stores below
                tmem_ld32(t_row + c, o);
                tmem_wait_ld();
                if (dead) continue;
                if (was.part < 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t pk[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            pk[y] = pack_bf16(__uint_as_float(o[8 * i + 2 * y]) * inv * vg, __uint_as_float(o[8 * i + 2 * y + 1]) * inv * vg);
                        reinterpret_cast<uint4*>(orow + c)[i] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        reinterpret_cast<uint4*>(P.part_o + part * D + c)[i] =
                            make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
            }
            tc_fence_before();
            mbar_arrive(smem_u32(&sh.o_free));
            if (!dead) {
                if (was.part < 0) P.lse[at] = ml.y == 0.0f ? -INFINITY : (ml.x + log2f(ml.y)) * kFp4Ln2;
                else P.part_ml[part] = ml;
            }
            was.n = 0;
            ++stored;
        };
        // K tiles and V tiles by the same instructions: eight warps run them side by side
        const bool is_v = warp < kUnpackK0;
        const uint32_t tiles = is_v ? s_v : s_k, codes_at = is_v ? C::kCodes : 0, scales_at = 2 * C::kCodes + (is_v ? C::kScales : 0);
        uint64_t *const full = is_v ? sh.v_full : sh.k_full, *const empty = is_v ? sh.v_empty : sh.k_empty;
        uint32_t g = 0, segs = 0;  // tiles, segments with a key so far
        for (uint32_t k = 0; ok; ++k) {
            const Fp4Segment* sp = next_segment(k, ok);
            if (sp == nullptr) break;
            const Fp4Segment sg = *sp;
            if (sg.n == 0) {
                publish(&sh.q_ready[k % kDesc]);  // (its phases go with the descriptors')
                hand_back(k);
                // no key at all: O = 0, LSE = -inf
                if (is_v && row < sg.nrows) {
                    const int64_t at = address(sg);
#pragma unroll 1
                    for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(P.o + at * D + c) = make_uint4(0, 0, 0, 0);
                    P.lse[at] = -INFINITY;
                }
                continue;
            }
            fetch_rows(sg);
            // the queries come before the first V tile, and after the first K tile
            const int32_t q_at = is_v ? 0 : 1;
            for (int32_t x = 0; x <= sg.n; ++x) {
                if (x == q_at) {
                    // (the segment before is done with the query tile's place)
                    if (segs > 0) ok = wait_warp(smem_u32(&sh.q_empty), (segs - 1u) & 1u, &sh.watch, status);
                    if (!ok) break;
                    place_rows(sg, k);
                    hand_back(k);
                    continue;
                }
                const uint32_t cs = g % CS, slot = g % S;
                const uint8_t* at = codes + cs * C::kStage;
                ok = wait_warp(smem_u32(&sh.code_full[cs]), (g / CS) & 1u, &sh.watch, status) &&
                     wait_warp(smem_u32(&empty[slot]), ((g / S) & 1u) ^ 1u, &sh.watch, status);
                if (!ok) break;
                unpack(at + codes_at, at + scales_at, tiles + slot * C::kTile);
                publish(&full[slot]);
                if (lane == 0) mbar_arrive(smem_u32(&sh.code_empty[cs]));
                ++g;
                // the rows of the segment before, which this one's first product waits for
                if (is_v && was.n > 0) store_rows();
                if (!ok) break;
            }
            was = sg;
            if (!is_v) was.n = 0;
            last = g - 1u;
            ++segs;
        }
        if (ok && was.n > 0) store_rows();
        if (!ok && lane == 0) set_abort(&sh.watch, status);
    } else {
        // ------------------------------------------------------------ softmax
        const int qd = warp & 3;  // a warp reaches TMEM lanes 32 (warp % 4) .. + 31
        const int half = (warp - kSoftmax0) >> 2;
        const int row[2] = {qd * 32 + half * 16 + (lane >> 2), qd * 32 + half * 16 + (lane >> 2) + 8};
        const uint32_t t_base = tmem + ((uint32_t)(qd * 32 + half * 16) << 16);
        const int c0 = 2 * (lane & 3);  // this thread's columns: c0 + 8 k, c0 + 8 k + 1
        uint32_t gb0 = 0, segs = 0;  // key tiles, segments with a key so far
        bool ok = true;
        for (uint32_t k = 0;; ++k) {
            const Fp4Segment* sg = next_segment(k, ok);
            if (sg == nullptr) break;
            const int32_t n = sg->n, j0 = sg->j0, lo_t = sg->lo, ns = sg->ns, most = sg->nrows - 1;
            const int64_t list_at = kLists ? ((int64_t)sg->kvh * P.nt_cap + sg->tile) * P.cap : 0;
            if (n == 0) {
                hand_back(k);
                continue;
            }
            const bool dead[2] = {row[0] >= sg->nrows, row[1] >= sg->nrows};
            // Row x sees keys lo[x] .. hi[x] - 1 and 0 .. sk[x] - 1.  Key tiles from
            // some_lo on and below some_hi, or below some_sk, are seen by some row of this
            // warp, from all_lo on and below all_hi, or below all_sk, whole by every row.
            int32_t hi[2], lo[2] = {0, 0}, sk[2] = {0, 0};
            int32_t some_hi, all_hi, some_lo = 0, all_lo = 0, some_sk = 0, all_sk = 0;
            {
                const int32_t kl = sg->kl, p0 = sg->pos_of0, row0 = sg->row0;
                // this warp's first and last row
                const int32_t ra = qd * 32 + half * 16, rb = min(ra + 15, most);
                const int32_t pa = p0 + (row0 + min(ra, most)) / P.group, pb = p0 + (row0 + rb) / P.group;
                auto end = [&](int32_t p) -> int32_t { return P.causal ? min(kl, p + 1) : kl; };
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int32_t p = p0 + (row0 + min(row[x], most)) / P.group;
                    hi[x] = end(p);
                    if constexpr (kMode == kWindow) {
                        lo[x] = p - P.window + 1;
                        sk[x] = min(P.sinks, hi[x]);
                    }
                }
                const bool some = ra <= most;
                all_hi = max(end(pa), 0) >> 7;
                some_hi = some ? (max(end(pb), 0) + 127) >> 7 : 0;
                if constexpr (kMode == kWindow) {
                    all_lo = (max(pb - P.window + 1, 0) + 127) >> 7;
                    some_lo = max(pa - P.window + 1, 0) >> 7;
                    all_sk = min(P.sinks, max(end(pa), 0)) >> 7;
                    some_sk = some ? (min(P.sinks, max(end(pb), 0)) + 127) >> 7 : 0;
                }
            }
            if (__any_sync(0xffffffffu, !paged_wait(smem_u32(&sh.q_ready[k % kDesc]), (k / kDesc) & 1u, &sh.watch, status))) {
                ok = false;
                break;
            }
            const float fac[2] = {sh.fac[k % kDesc][row[0]], sh.fac[k % kDesc][row[1]]};
            hand_back(k);
            float m[2] = {kFp4NoKey, kFp4NoKey};
            float l[2] = {0.0f, 0.0f};  // this thread's share of each row
            bool first = true;
            // lists: the next key tile, and the words that hold this thread's rows' bits
            const int32_t* list = nullptr;
            const uint32_t* who = nullptr;
            int32_t tile_next = 0, tok[2] = {0, 0};
            uint32_t who_next[2] = {0u, 0u};
            auto look = [&](int32_t j) {
                if (j >= n) return;
                tile_next = list[j];
#pragma unroll
                for (int x = 0; x < 2; ++x) who_next[x] = who[(int64_t)j * P.words + (tok[x] >> 5)];
            };
            if constexpr (kLists) {
                list = P.list + list_at + j0;
                who = P.who + (list_at + j0) * P.words;
#pragma unroll
                for (int x = 0; x < 2; ++x) tok[x] = min(row[x], most) / P.group;
                look(0);
            }
            for (int32_t j = 0; j < n; ++j) {
                const uint32_t gb = gb0 + (uint32_t)j;
                const uint32_t sbuf = (gb % kSBuf) * 128u;
                int32_t kt;
                if constexpr (kLists) kt = tile_next;
                else if constexpr (kMode == kWindow) kt = j0 + j < ns ? j0 + j : lo_t + j0 + j - ns;
                else kt = j0 + j;
                const int32_t kb = kt * 128;
                bool hidden[2] = {false, false};
                // bit 2 kk + e of vis[x]: row x sees this thread's column c0 + 8 kk + e
                uint32_t vis[2] = {~0u, ~0u};
                bool visible = (kt < some_hi && kt >= some_lo) || kt < some_sk;
                const bool masked = visible && !((kt < all_hi && kt >= all_lo) || kt < all_sk);
                if constexpr (kLists) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) hidden[x] = dead[x] || (who_next[x] >> (tok[x] & 31) & 1u) == 0u;
                    visible = __any_sync(0xffffffffu, !hidden[0] || !hidden[1]);
                    look(j + 1);
                }
                if (masked) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        vis[x] = columns_below(hi[x] - kb - c0);
                        if constexpr (kMode == kWindow)
                            vis[x] = (vis[x] & ~columns_below(lo[x] - kb - c0)) | columns_below(sk[x] - kb - c0);
                    }
                }
                const bool wt = paged_wait(smem_u32(&sh.s_full[gb % kSBuf]), (gb / kSBuf) & 1u, &sh.watch, status);
                // (a failure elsewhere in the block or in another one ends this wait too)
                if (__any_sync(0xffffffffu, !wt)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (!visible) {
                    // no row of this warp sees a key of the tile: P = 0
                    store_p_zero(t_base + sbuf);
                    tc_fence_before();
                    mbar_arrive(smem_u32(&sh.p_full[gb % kSBuf]));
                    continue;
                }
                uint32_t sc[64];
                auto load_s = [&]() {
                    tmem_ld16x256_x16(t_base + sbuf, sc);
                    tmem_wait_ld();
                    if (masked) {
                        const uint32_t ninf = __float_as_uint(-INFINITY);
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int kk = 0; kk < 16; ++kk)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    sc[4 * kk + 2 * x + e] = (vis[x] >> (2 * kk + e)) & 1u ? sc[4 * kk + 2 * x + e] : ninf;
                    }
                };
                load_s();
                float alpha[2];
                const bool raised = softmax_rows(sc, hidden, fac, first, m, l, alpha, load_s);
                first = false;
                tmem_st16x128_x16(t_base + sbuf, sc);
                if (raised) {
                    // O must hold P_0 .. P_{j-1} V: wait for PV_{j-1}
                    const uint32_t pv = gb - 1u;
                    const bool wv = paged_wait(smem_u32(&sh.pv_done[pv % kSBuf]), (pv / kSBuf) & 1u, &sh.watch, status);
                    if (__any_sync(0xffffffffu, !wv)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    scale_o_rows<D>(t_base + kColO, alpha[0], alpha[1]);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(smem_u32(&sh.p_full[gb % kSBuf]));
            }
            if (!ok) break;
            // maxima and sums of the rows to the storing warps
            const float la = row_sum4(l[0]), lb = row_sum4(l[1]);
            if (__any_sync(0xffffffffu, !paged_wait(smem_u32(&sh.ml_empty), (segs & 1u) ^ 1u, &sh.watch, status))) {
                ok = false;
                break;
            }
            if ((lane & 3) == 0) {
                sh.ml[row[0]] = make_float2(m[0], la);
                sh.ml[row[1]] = make_float2(m[1], lb);
            }
            mbar_arrive(smem_u32(&sh.ml_full));
            ++segs;
            gb0 += (uint32_t)n;
        }
        if (!ok && lane == 0) set_abort(&sh.watch, status);
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaQK) tmem_dealloc(tmem, kTmemCols);
}

template <int D, int kMode>
bsa_status launch_d(const Fp4Params& P, bool first, cudaStream_t stream) {
    constexpr size_t smem = 1024 + Cfg<D>::kData + sizeof(Shared);
    static_assert(smem <= 232448, "shared memory of a thread block");
    static DeviceSetup setup;
    static int sms[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
    const bool ready = setup.once(dev, [&] {
        return cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
               cudaFuncSetAttribute(k_fp4_prompt<D, kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) ==
                   cudaSuccess;
    });
    if (!ready) return BSA_ERR_CUDA;
    const int grid = sms[dev] < kPagedBlocks ? sms[dev] : kPagedBlocks;
    constexpr int kRows = kFp4JoinThreads / (D / 4);
    // As a call's first kernel it does not start beside the one before it, whose SMs its blocks would take as they fall free,
    // in any order (a chunk of 1024 over 64512, again and again: 846 us so, 781 in order).
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    const cudaError_t e = first ? cudaLaunchKernelEx(&cfg, k_fp4_prompt<D, kMode>, P)
                                : launch_chained(k_fp4_prompt<D, kMode>, cfg.gridDim, kThreads, smem, stream, P);
    if (e != cudaSuccess ||
        launch_chained(k_fp4_join<D, kWide, kRows>, dim3((unsigned)grid, kWide / kRows), kFp4JoinThreads, 0, stream, P) != cudaSuccess)
        return BSA_ERR_CUDA;
    return BSA_OK;
}

}  // namespace

bsa_status launch_fp4_prompt(const Fp4Params& P, int32_t D, bool first, cudaStream_t stream) {
    if (P.list != nullptr) return D == 128 ? launch_d<128, kListed>(P, first, stream) : launch_d<64, kListed>(P, first, stream);
    if (P.window > 0) return D == 128 ? launch_d<128, kWindow>(P, first, stream) : launch_d<64, kWindow>(P, first, stream);
    return D == 128 ? launch_d<128, kPlain>(P, first, stream) : launch_d<64, kPlain>(P, first, stream);
}

}  // namespace bsa
