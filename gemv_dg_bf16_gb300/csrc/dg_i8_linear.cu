// dg_i8_linear.cu -- the linear on 8-bit integer weights and activations with a scale for each
// weight row and each token (dg_gemv_i8_rowscale).
//
// sm_103a has no integer tcgen05.mma, and its warp-level integer MMA and dp4a run at 250
// multiply-adds a clock and SM (f16: mma.sync 1020, tcgen05 4096; measured), so the codes are multiplied as
// binary16 numbers, exactly (dg_i8.cuh).  The activations are quantised to binary16 codes
// ahead (i8_quant_kernel); the weights stay bytes until they are in the SM.
//
// Swap-AB: a unit is a tile of 128 weight rows (the MMA's M) with a group of up to MP tokens (its N), taken in
// 128-element blocks of K.  Few units: a cluster of CTAs each, with a range of K a rank.  Many: persistent CTAs, one an
// SM, take one after the other, the next one's blocks under the epilogue of the last.
//   weights      a warp streams 128 x 128 bytes a stage by TMA (128-byte swizzle)
//   MMA          a warp allocates tensor memory; one elected lane issues tcgen05.mma, 8 of K = 16 a block
//   conversion   two or three sets of four warps take the blocks in turn: a lane takes one weight row's 128 bytes from
//                shared memory, turns them into binary16 and stores them in tensor memory, where the MMA reads A,
//                in a ring of 3 or 4 buffers of 64 columns (with two, each conversion waited for an MMA: 790 cycles a
//                block at 128 tokens)
//   epilogue     four warps: every 1024 elements the accumulator (two of them) is taken out of tensor
//                memory, as integers, and added up; then scaled and stored, or folded
//   activations  a warp streams a block of binary16 codes a stage, which the quantisation left in one piece
// Each rank of a K split folds a share of the tokens, and the others write their integers of these into its
// shared memory.
//
// Groups of 64 tokens and more, many units and 16 blocks or more, K not split: a pair of CTAs has a unit of 256
// weight rows, and one MMA (cta_group::2) multiplies both CTAs' 128 rows of A with the N of both, of which each loads
// and holds half.  Of the two the even one issues; what it waits for and what it frees goes through barriers of both.
// What binds it at 128 tokens: the MMAs take 512 cycles a block, its 32 KB 510 at the 64 bytes a clock that an SM takes
// in, and blocks come every 720.
// Measured (calls in turn, quantisation included): 12288 x 4096 at 16 tokens 14.1 us, 3.6 TB/s of weights -- 8 us of
// stream between a quantisation, a first load and a fold; 4099 x 12288 at 77 19.9; 24576 x 4096 at 512 82.1, 1.26
// PFLOP/s.
// Every wait is bounded: on timeout the kernel flags DG_DEVERR_WAIT_TIMEOUT and winds down.
#include <cuda.h>

#include "dg_i8.cuh"
#include "dg_internal.h"
#include "dg_tc_common.cuh"

namespace dg {
namespace {

using tc::cluster_rank;
using tc::cluster_sync_all;
using tc::map_to_rank;

constexpr int kTileRows = 128;                     // MMA M
constexpr int kBlock = 128;                        // K elements a stage: one swizzled row of bytes
constexpr int kWBox = kTileRows * kBlock;          // 16 KB
// Warps of the roles: weights, MMA, activations, then 4 for each converting set and 4 for the epilogue.
template <bool PAIR>
struct Roles {
    static constexpr int kSets = PAIR ? 3 : 2;
    static constexpr int kConvert = PAIR ? 4 : 2, kEpilogue = kConvert + 4 * kSets, kStreamX = PAIR ? 2 : kEpilogue + 4;
    static constexpr int kThreads = PAIR ? 640 : 480;
};
constexpr int kSegBlocks = i8::kSegment / kBlock;
constexpr int kACols = kBlock / 2;                 // tensor-memory columns of a converted block
constexpr int kMaxRanks = 8;
constexpr int kFewTokens = 16;
constexpr int kDone = 8;                           // blocks whose completion is told apart: more than are in flight

struct I8Args {
    int N, K, M;
    int nkb, groups, mp;                           // blocks of K, token groups, tokens of a group (a multiple of 16)
    int units;
    int nsplit, share;                             // ranks of a K split; tokens that each folds (a multiple of 4)
    int sw_stages, sx_stages;
    const uint8_t* x;                              // the activations' codes in tiles (i8::tile_offset), written ahead
    const float* sx;                               // [M], written ahead
    const float* sw;                               // [N]
    uint16_t* y;
    uint8_t* ws;
};

// Four integers into the shared memory of a CTA of the cluster.
__device__ __forceinline__ void st_cluster(uint32_t addr, int a, int b, int c, int d)
{
    asm volatile("st.shared::cluster.v4.s32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// Both barriers' phases complete (the two tests in flight at once; then the bounded waits).
__device__ __forceinline__ bool wait_both(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1, volatile int* abort_flag)
{
    const bool r0 = tc::bar_try(b0, p0), r1 = tc::bar_try(b1, p1);
    return (r0 || tc::bar_wait(b0, p0, abort_flag)) && (r1 || tc::bar_wait(b1, p1, abort_flag));
}

// kind::f16 with binary16 A (tensor memory) and B (shared memory), fp32 accumulate, M = m, N = n.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n)
{
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// PAIR: two CTAs' A (128 rows each) with the N of both CTAs' B (a half each).
template <bool PAIR>
__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
            ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
            ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}

// The barrier at this place (PAIR: in both CTAs) arrives when the MMAs issued so far have finished.
template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
            ::"r"(bar), "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        tc::commit(bar);
}

// Arrival at a barrier of a CTA of the cluster.
__device__ __forceinline__ void arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The phase in which block i is told done.
__device__ __forceinline__ uint32_t done_phase(int i) { return static_cast<uint32_t>(i / kDone) & 1u; }

// Whether a condition holds in all of the 128 epilogue threads (a barrier for them).
__device__ __forceinline__ bool all_of(bool p)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "bar.red.and.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(p))
        : "memory");
    return r != 0;
}

// MP: the most tokens of a group that this instance takes.  PAIR: clusters of two CTAs share a unit of 256 weight rows.
template <int MP, bool PAIR>
__global__ void __launch_bounds__(Roles<PAIR>::kThreads, MP <= 32 ? 2 : 1)
    i8_tc_kernel(const __grid_constant__ CUtensorMap tmW, I8Args a)
{
    constexpr uint32_t kA0 = 2 * MP < 64 ? 64 : 2 * MP;             // first column of the converted blocks
    constexpr uint32_t kCols = MP <= 32 ? 256 : 512;               // two accumulators, kBufs converted blocks
    constexpr int kBufs = MP <= 32 ? 3 : 4;
    constexpr int kSets = Roles<PAIR>::kSets, kConvert = Roles<PAIR>::kConvert;
    constexpr int kEpilogue = Roles<PAIR>::kEpilogue, kStreamX = Roles<PAIR>::kStreamX;
    static_assert(kA0 + kBufs * kACols <= kCols, "tensor memory");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int SW = a.sw_stages, SX = a.sx_stages, xbox = (PAIR ? a.mp / 2 : a.mp) * 128, xstage = 2 * xbox;
    uint8_t* xring = smem + SW * kWBox;
    float* sxs = reinterpret_cast<float*>(xring + SX * xstage);     // [2][MP]
    uint16_t* stage = reinterpret_cast<uint16_t*>(sxs + 2 * MP);    // [2][16 tokens][128 rows] of outputs
    uint64_t* bars = reinterpret_cast<uint64_t*>(stage + 2 * 16 * kTileRows);
    const int nbars = 2 * SW + SX + kDone + kBufs + 4 + (SX + kBufs) % 2;       // (even: 16 bytes)
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + nbars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    // done[i % kDone]: block i is multiplied, its activations' slot and its converted weights' buffer are free
    const uint32_t wfull = tc::su32(bars), wempty = wfull + 8 * SW, xfull = wempty + 8 * SW, done = xfull + 8 * SX;
    const uint32_t afull = done + 8 * kDone, dfull = afull + 8 * kBufs, dempty = dfull + 16;
    // [rank][share / 4][row][4]
    int* fold = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + nbars * 8 + 16);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool split = !PAIR && a.nsplit > 1;
    const int rank = split ? static_cast<int>(cluster_rank()) : 0, half = PAIR ? static_cast<int>(cluster_rank()) : 0;
    constexpr int kUnitRows = PAIR ? 2 * kTileRows : kTileRows;
    // Units `first`, first + stride, ...; groups of one tile run side by side, so that its weights come from memory
    // once.
    const int first = static_cast<int>(blockIdx.x) / (PAIR ? 2 : a.nsplit);
    const int stride = split ? a.units : static_cast<int>(gridDim.x) / (PAIR ? 2 : 1);
    const int kb0 = static_cast<int>(static_cast<long long>(rank) * a.nkb / a.nsplit);
    const int nk = static_cast<int>(static_cast<long long>(rank + 1) * a.nkb / a.nsplit) - kb0;     // blocks of a unit

    if (threadIdx.x == 0) {
        for (int s = 0; s < SW; ++s) {
            tc::bar_init(wfull + 8 * s, 1);
            tc::bar_init(wempty + 8 * s, 4);                        // one per converting warp
        }
        for (int s = 0; s < SX; ++s) {
            tc::bar_init(xfull + 8 * s, 1);
        }
        for (int s = 0; s < kDone; ++s) tc::bar_init(done + 8 * s, 1);
        for (int s = 0; s < kBufs; ++s) tc::bar_init(afull + 8 * s, PAIR ? 8 : 4);
        for (int b = 0; b < 2; ++b) {
            tc::bar_init(dfull + 8 * b, 1);
            tc::bar_init(dempty + 8 * b, PAIR ? 8 : 4);             // one per epilogue warp
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                         ::"r"(tc::su32(tmem_holder)), "r"(kCols));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                         ::"r"(tc::su32(tmem_holder)), "r"(kCols));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    tc::fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();                         // both CTAs' barriers and tensor memory are there
    tc::fence_after();
    const uint32_t tmem = *tmem_holder;
    pdl_launch_dependents();
    if (split) {
        __syncwarp();                                               // (waited for in front of the first remote access)
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    }

    // After a wait that ran out: the copies in flight of a ring whose last `issued` loads went round
    // `stages` slots are waited for, again with a limit, before the CTA may leave.
    auto drain = [&](uint32_t full, int issued, int stages) {
        volatile int own = 0;
        for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
            tc::bar_wait_for(full + 8 * (i % stages), static_cast<uint32_t>(i / stages) & 1u, &own, 100000000ull);
    };

    const int q = warp & 3;                                         // tensor-memory lane quarter
    const uint32_t tlane = tmem + (static_cast<uint32_t>(q * 32) << 16);
    if (warp < kConvert || (!PAIR && warp == kStreamX)) {
        // PAIR: 5 warpgroups of 96 registers become 32 + 3 * 96 + 160.
        if constexpr (PAIR) asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
        if (warp == 0) {
            if (tc::elect_one()) {
                const uint64_t once = tc::policy_evict_first();
                int s = 0, issued = 0;
                uint32_t round = 0;
                // A unit begins at a block of its tile's own, so that not all of them ask for the same activations at
                // a time (24576 x 4096 at 512 tokens 82.0 -> 81.2 us; the order of blocks changes no sum).  Weights
                // have nothing to wait for.
                for (int u = first; u < a.units && !*abort_flag; u += stride) {
                    const int tile = u / a.groups, row = tile * kUnitRows + half * kTileRows;
                    for (int i = 0, kb = tile % nk; i < nk; ++i, kb = kb + 1 < nk ? kb + 1 : 0) {
                        if (round > 0 && !tc::bar_wait(wempty + 8 * s, (round - 1) & 1u, abort_flag)) break;
                        tc::bar_expect_tx(wfull + 8 * s, kWBox);
                        if (a.groups == 1)
                            tc::tma_2d_hint(tc::su32(smem + s * kWBox), &tmW, (kb0 + kb) * kBlock, row,
                                            wfull + 8 * s, once);
                        else
                            tc::tma_2d(tc::su32(smem + s * kWBox), &tmW, (kb0 + kb) * kBlock, row, wfull + 8 * s);
                        ++issued;
                        if (++s == SW) {
                            s = 0;
                            ++round;
                        }
                    }
                }
                if (*abort_flag) drain(wfull, issued, SW);
            }
            __syncwarp();                                           // (a lane in pdl_wait() holds up the whole warp)
            pdl_wait();
        } else if (warp == kStreamX) {
            pdl_wait();
            if (tc::elect_one()) {
                int s = 0, issued = 0;
                uint32_t round = 0;
                for (int u = first; u < a.units && !*abort_flag; u += stride) {
                    // (PAIR: tiles of half a group)
                    const int group = PAIR ? u % a.groups * 2 + half : u % a.groups;
                    const uint8_t* src = a.x + (static_cast<size_t>(group) * a.nkb + kb0) * xstage;
                    for (int i = 0, kb = u / a.groups % nk; i < nk; ++i, kb = kb + 1 < nk ? kb + 1 : 0) {
                        const int before = issued - SX;             // the block that had the slot
                        if (before >= 0 && !tc::bar_wait(done + 8 * (before % kDone), done_phase(before), abort_flag))
                            break;
                        const uint32_t dst = tc::su32(xring + s * xstage);
                        tc::bar_expect_tx(xfull + 8 * s, static_cast<uint32_t>(xstage));
                        tc::bulk_load(dst, src + static_cast<size_t>(kb) * xstage, static_cast<uint32_t>(xstage),
                                      xfull + 8 * s);
                        ++issued;
                        if (++s == SX) {
                            s = 0;
                            ++round;
                        }
                    }
                }
                if (*abort_flag) drain(xfull, issued, SX);
            }
        } else if (warp == 1) {
            if (half == 0 && tc::elect_one()) {
                const uint32_t idesc = idesc_f16(kUnitRows, a.mp);
                const uint64_t box = static_cast<uint64_t>(xbox / 16), ring = tc::sw128_desc(tc::su32(xring));
                int s = 0, b = 0, seg = 0, block = 0;
                uint32_t round = 0, bround = 0;
                for (int u = first; u < a.units && !*abort_flag; u += stride) {
                    for (int i = 0, in = 0; i < nk; ++i, ++block) {     // in: blocks of the segment so far
                        const int d = seg & 1;
                        if constexpr (PAIR) {                       // (whoever converted has seen the activations too)
                            if (!tc::bar_wait(afull + 8 * b, bround & 1u, abort_flag)) break;
                        } else {
                            if (!wait_both(xfull + 8 * s, round & 1u, afull + 8 * b, bround & 1u, abort_flag)) break;
                        }
                        if (in == 0 && seg >= 2 &&
                            !tc::bar_wait(dempty + 8 * d, static_cast<uint32_t>(seg / 2 - 1) & 1u, abort_flag))
                            break;
                        tc::fence_after();
                        const uint64_t x0 = ring + static_cast<uint64_t>(s * (xstage / 16));
#pragma unroll
                        for (int kk = 0; kk < kBlock / 16; ++kk)
                            mma_f16_ta<PAIR>(tmem + static_cast<uint32_t>(d * MP),
                                             tmem + kA0 + static_cast<uint32_t>(b * kACols + kk * 8),
                                             x0 + (kk < 4 ? 0 : box) + static_cast<uint64_t>((kk % 4) * 2), idesc,
                                             (in > 0 || kk > 0) ? 1u : 0u);
                        commit<PAIR>(done + 8 * (block % kDone));
                        if (++in == kSegBlocks || i == nk - 1) {
                            commit<PAIR>(dfull + 8 * d);
                            in = 0;
                            ++seg;
                        }
                        if (++s == SX) {
                            s = 0;
                            ++round;
                        }
                        if (++b == kBufs) {
                            b = 0;
                            ++bround;
                        }
                    }
                }
            }
            __syncwarp();
            pdl_wait();
        } else {
            pdl_wait();
        }
    } else if (warp < kEpilogue) {
        // Convert: this lane's weight row, 16 bytes at a time from their swizzled places.
        const int row = q * 32 + lane, set = (warp - kConvert) / 4;
        const long long blocks = static_cast<long long>(nk) * ((a.units - first + stride - 1) / stride);
        int s = set, b = set;                                       // (SW is even: the slots of a set are its own)
        uint32_t round = 0;
        int xs = set % SX;                                          // PAIR: the activations' slot and its phase
        uint32_t xround = static_cast<uint32_t>(set / SX);
        const uint32_t leader = PAIR ? map_to_rank(afull, 0) : afull;
#pragma unroll 1
        for (int i = set; i < blocks; i += kSets) {
            // (a wait that ran out ends the loop in every lane)
            if (!__all_sync(kFull, tc::bar_wait(wfull + 8 * s, round & 1u, abort_flag))) break;
            const uint8_t* src = smem + s * kWBox;
            uint4 raw[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) raw[c] = *reinterpret_cast<const uint4*>(src + tc::sw128_offset(row, c));
            // Every lane's bytes are read before the slot is handed back: the copy that fills it again writes by
            // another proxy, which an arrival alone does not hold behind these loads.  (Without the fence 12 of 89000
            // calls, all of the instance of 128 tokens on single CTAs, had a few weight rows of a later block; with it
            // none of 450000.  24576 x 4096 at 128 tokens 33.0 -> 33.4 us, 77 tokens 19.4 -> 19.9; handed back behind
            // the stores to tensor memory instead 33.8 and 20.4.)
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) tc::bar_arrive(wempty + 8 * s);
            const int before = i - kBufs;                           // the block that had the buffer
            if (before >= 0 &&
                !__all_sync(kFull, tc::bar_wait(done + 8 * (before % kDone), done_phase(before), abort_flag)))
                break;
            tc::fence_after();
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                uint32_t v[16];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint4 r = raw[2 * h + c];
                    i8::to_halves(r.x, v[8 * c], v[8 * c + 1]);
                    i8::to_halves(r.y, v[8 * c + 2], v[8 * c + 3]);
                    i8::to_halves(r.z, v[8 * c + 4], v[8 * c + 5]);
                    i8::to_halves(r.w, v[8 * c + 6], v[8 * c + 7]);
                }
                tc::tmem_st16(tlane + kA0 + static_cast<uint32_t>(b * kACols + h * 16), v);
            }
            tc::tmem_st_wait();
            tc::fence_before();
            __syncwarp();
            if constexpr (PAIR) {
                // The multiplying CTA hears of this CTA's half of the activations and of its weights at once.
                if (lane == 0 && tc::bar_wait(xfull + 8 * xs, xround & 1u, abort_flag)) arrive_cluster(leader + 8 * b);
                for (xs += kSets; xs >= SX; xs -= SX) ++xround;
            } else {
                if (lane == 0) tc::bar_arrive(afull + 8 * b);
            }
            s += kSets;
            if (s >= SW) {
                s -= SW;
                ++round;
            }
            b += kSets;
            if (b >= kBufs) b -= kBufs;
        }
        pdl_wait();
    } else {
        if constexpr (PAIR) asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
        pdl_wait();
        const int row = q * 32 + lane, nseg = (nk + kSegBlocks - 1) / kSegBlocks;
        int seg = 0;
        bool good = true;
#pragma unroll 1
        for (int u = first, k = 0; u < a.units && good; u += stride, ++k) {
            const int t0 = u % a.groups * a.mp, rows_here = min(a.mp, a.M - t0);
            const int nrow = u / a.groups * kUnitRows + half * kTileRows + row;
            const float sw = a.sw[min(nrow, a.N - 1)];
            float* sxt = sxs + (k & 1) * MP;
            for (int t = threadIdx.x - kEpilogue * 32; t < rows_here; t += 128) sxt[t] = ld_cg_f32(a.sx + t0 + t);
            int tot[MP];
#pragma unroll
            for (int j = 0; j < MP; ++j) tot[j] = 0;
#pragma unroll 1
            for (int e = 0; e < nseg; ++e, ++seg) {
                const int d = seg & 1;
                if (!__all_sync(kFull, tc::bar_wait(dfull + 8 * d, static_cast<uint32_t>(seg / 2) & 1u, abort_flag))) {
                    good = false;
                    break;
                }
                tc::fence_after();
#pragma unroll
                for (int c = 0; c < MP / 16; ++c) {
                    if (c < MP / 16 - 1 || a.mp == MP) {    // (an instance serves mp = MP and, from 64 on, MP - 16)
                        uint32_t v[16];
                        tc::tmem_ld16(tlane + static_cast<uint32_t>(d * MP + c * 16), v);
#pragma unroll
                        for (int j = 0; j < 16; ++j) tot[c * 16 + j] += __float2int_rn(__uint_as_float(v[j]));
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR)
                        arrive_cluster(map_to_rank(dempty + 8 * d, 0));
                    else
                        tc::bar_arrive(dempty + 8 * d);
                }
            }
            // A wait that ran out ends the loop in all 128 threads or in none (they meet here, and the scales are
            // there).
            good = all_of(good && !*abort_flag);
            if (!good) break;
            if (split) {
                // This row's integers, four tokens at a time, to the rank that folds them.
                __syncwarp();
                asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");        // every rank has begun
                int to = 0, at = rank * a.share;
                uint32_t peer = map_to_rank(tc::su32(fold), 0);
#pragma unroll
                for (int j = 0; j < MP; j += 4) {
                    if (j >= a.mp) break;
                    if (at == (rank + 1) * a.share) {
                        at = rank * a.share;
                        peer = map_to_rank(tc::su32(fold), static_cast<uint32_t>(++to));
                    }
                    st_cluster(peer + static_cast<uint32_t>((at * kTileRows + row * 4) * 4), tot[j], tot[j + 1],
                               tot[j + 2], tot[j + 3]);
                    at += 4;
                }
            } else if (a.N % 8 == 0 && nrow - row + kTileRows <= a.N) {
                // Sixteen tokens at a time go through shared memory, [token][row] in turn in two places, and leave 16
                // bytes a lane, 256 of a token's outputs side by side.  (Straight from the lanes, 64 bytes a store, 128
                // tokens took 3.9 us.)
#pragma unroll
                for (int c = 0; c < MP / 16; ++c) {
                    if (c * 16 >= rows_here) break;
                    uint16_t* st = stage + (c & 1) * 16 * kTileRows;
                    uint16_t v[16];         // (all read before the first is written: the compiler keeps their order)
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 sx = *reinterpret_cast<const float4*>(sxt + c * 16 + j);
                        v[j] = i8::output(tot[c * 16 + j], sx.x, sw);
                        v[j + 1] = i8::output(tot[c * 16 + j + 1], sx.y, sw);
                        v[j + 2] = i8::output(tot[c * 16 + j + 2], sx.z, sw);
                        v[j + 3] = i8::output(tot[c * 16 + j + 3], sx.w, sw);
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) st[j * kTileRows + row] = v[j];
                    asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int z = threadIdx.x - kEpilogue * 32 + h * 128, t = c * 16 + z / 16;
                        if (t < rows_here)
                            *reinterpret_cast<uint4*>(a.y + static_cast<size_t>(t0 + t) * a.N + (nrow - row) +
                                                      z % 16 * 8) = *reinterpret_cast<const uint4*>(st + z * 8);
                    }
                }
            } else if (nrow < a.N) {
                uint16_t* dst = a.y + static_cast<size_t>(t0) * a.N + nrow;
#pragma unroll
                for (int c = 0; c < MP; c += 16) {
                    if (c >= rows_here) break;
                    uint16_t v[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = i8::output(tot[c + j], sxt[c + j], sw);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c + j < rows_here) dst[static_cast<size_t>(c + j) * a.N] = v[j];
                }
            }
        }
        if (split && !good) {
            __syncwarp();
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        }
    }
    if (split) {
        if (warp < kEpilogue || warp >= kEpilogue + 4) {
            __syncwarp();
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");            // (the arrival at the start)
        }
        cluster_sync_all();                 // every rank's integers are in place; the last remote access
        if (warp >= kConvert && warp < kEpilogue + 4 && !*abort_flag) {
            // A warp takes 32 rows, the same ones of every third four tokens: a lane adds up a row's over the ranks.
            const int t0 = first % a.groups * a.mp, lo = rank * a.share, rows_here = min(a.mp, a.M - t0);
            const int quads = (max(0, min(rows_here - lo, a.share)) + 3) / 4;
            const int row = (warp - kConvert) % 4 * 32 + lane, nrow = first / a.groups * kTileRows + row;
            const float sw = a.sw[min(nrow, a.N - 1)];
#pragma unroll 1
            for (int z = (warp - kConvert) / 4; z < quads; z += 3) {
                int4 v = make_int4(0, 0, 0, 0);
                for (int r = 0; r < a.nsplit; ++r) {
                    const int4 p = *reinterpret_cast<const int4*>(fold + ((r * a.share + z * 4) * kTileRows + row * 4));
                    v = make_int4(v.x + p.x, v.y + p.y, v.z + p.z, v.w + p.w);
                }
                if (nrow >= a.N) continue;
                const int t = lo + z * 4;
                const float4 sx = *reinterpret_cast<const float4*>(sxs + t);
                const uint16_t out[4] = {i8::output(v.x, sx.x, sw), i8::output(v.y, sx.y, sw),
                                         i8::output(v.z, sx.z, sw), i8::output(v.w, sx.w, sw)};
                uint16_t* dst = a.y + static_cast<size_t>(t0 + t) * a.N + nrow;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (t + j < rows_here) dst[static_cast<size_t>(j) * a.N] = out[j];
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();         // neither leaves while the other's MMAs or arrivals need it
    if (*abort_flag && threadIdx.x == 0) set_status(a.ws, DG_DEVERR_WAIT_TIMEOUT);
    if (warp == 1) {
        tc::fence_after();
        if constexpr (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
    }
}

// ------------------------------------------------------------------------ host

const void* kernel_of(int mp, bool pair)
{
    if (pair)
        return mp == 64   ? reinterpret_cast<const void*>(&i8_tc_kernel<64, true>)
               : mp == 96 ? reinterpret_cast<const void*>(&i8_tc_kernel<96, true>)
                          : reinterpret_cast<const void*>(&i8_tc_kernel<128, true>);
    return mp <= 16   ? reinterpret_cast<const void*>(&i8_tc_kernel<16, false>)
           : mp <= 32 ? reinterpret_cast<const void*>(&i8_tc_kernel<32, false>)
           : mp <= 64 ? reinterpret_cast<const void*>(&i8_tc_kernel<64, false>)
           : mp <= 96 ? reinterpret_cast<const void*>(&i8_tc_kernel<96, false>)
                      : reinterpret_cast<const void*>(&i8_tc_kernel<128, false>);
}

// xt: tokens of a stage of activations; fold: bytes for the integers of a K split.
size_t smem_bytes(int mp, int xt, int sw, int sx, size_t fold)
{
    const size_t most = mp <= 16 ? 16 : mp <= 32 ? 32 : mp <= 64 ? 64 : mp <= 96 ? 96 : 128;
    return 1024 + static_cast<size_t>(sw) * kWBox + static_cast<size_t>(sx) * xt * 256 + most * 8 +
           2 * 16 * kTileRows * 2 + (2 * sw + sx + kDone + 10) * 8 + 16 + fold;
}

// Rows of the last group of up to 128 tokens and elements of the last block are there in full.
size_t code_bytes(int M, int K)
{
    return (static_cast<size_t>(M) + 127) * ((static_cast<size_t>(K) + kBlock - 1) / kBlock * kBlock) * 2;
}

size_t scale_bytes(int M) { return (static_cast<size_t>(M) * 4 + 255) / 256 * 256; }

// Tokens of a group: equal groups of up to `most`, rounded up to the MMA's 16.
int group_tokens(int M, int most)
{
    const int groups = (M - 1) / most + 1;
    return ((M - 1) / groups + 16) / 16 * 16;
}

// What a call of `units` units of mp tokens takes in us with K in ns ranges, roughly, for a choice among them: a
// launch, an epilogue that grows with the tokens, the fold, and 0.4 a block of K of an SM, one CTA after the other on
// it or (K split, up to 32 tokens) two side by side.  Where hardly an SM is left over, the next launch's first loads
// come late.  Fitted to 4.2 us for 64 x 256 at 24 tokens to 21 for 4096 x 4096 at 400: 66 shapes, cuts and counts of
// tokens within a fifth or so.
float estimate(int sms, long long units, int nkb, int mp, int ns)
{
    const long long ctas = units * ns;
    const int blocks = (nkb - 1) / ns + 1;
    const bool two = ns > 1 && mp <= 32;
    const float rounds = two ? (ctas > sms ? static_cast<float>(ctas) / sms : 1.0f) * (mp > 16 ? 1.3f : 1.0f)
                             : static_cast<float>((ctas - 1) / sms + 1);
    float t = 3.6f + (mp == 32 ? 0.7f : 0.031f * (mp - 16)) + 0.4f * blocks * rounds;
    if (ns > 1) t += 1.0f + 0.05f * ns + 0.01f * mp;
    if (mp > 32 ? ctas * 32 > sms * 27ll : ctas * 15 > sms * 26ll) t += 2.5f;
    return t;
}

}  // namespace

size_t i8_workspace_bytes(int M, int K)
{
    return kWsData + code_bytes(M, K) + scale_bytes(M);
}

// How a call is cut, where its choice leaves that open.  Measured, both sides in us at the time:
//   ranks       all that are resident at once; where two CTAs share an SM, at most 263 of the 304 (12288 x 4096 at 16
//               tokens: two ranks 14.0, three 18.5).  None up to 512 elements, where a launch of clusters and the fold
//               cost more than the blocks (256 x 512, one rank / two: 16 tokens 4.65 / 4.9, 64 6.3 / 6.75, 300 8.05 /
//               9.35), nor for groups past 112 tokens, beside whose integers two stages of weights are left.
//   thirds      up to 32 tokens, for a few more units than SMs and long ones: not a second round for some SMs (16
//               tokens, one rank / three: 20480 x 5120 32.3 / 25.5, 24576 x 8192 49.3 / 41.2, 20480 x 12288 71.5 /
//               49.5; not 24576 x 4096 27.3 / 27.3 and at 8 27.2 / 30.0, 26000 x 4096 28.6 / 34.9, 20480 x 2560 18.2 /
//               18.7; at 64 tokens 24576 x 4096 30.7 / 48.7).
//   groups      above 16 tokens the groups and ranks of least estimate (with groups of up to 128 and all the ranks
//               that fit / so: 64 x 256 at 400 tokens 7.1 / 4.5, 1024 x 512 at 200 8.1 / 5.3, 2048 x 1024 at 100 9.6 /
//               7.0, 4096 x 1024 at 200 11.2 / 8.2).
//   pairs       of CTAs for 256 rows, where K is not split and a group has 64 tokens or more.  Each holds half of the
//               activations, so that an SM takes in 32 KB a block at 128 tokens and not 48 (it takes 61 bytes a clock
//               at most), and three sets convert (pair / single CTAs: 24576 x 4096 at 512 tokens 82.1 / 95.0, 256 45.3
//               / 51.7, 128 33.4 / 37.3, 64 29.1 / 31.5; 8192 x 8192 at 256 32.6 / 36.6; groups rounded up to 32
//               tokens: 20480 x 5120 at 160 47.4 / 48.1).  Not for few units or a short K (4096 x 4096 at 200 19.1 /
//               18.0, 2048 x 1024 at 400 11.7 / 10.1).
//   rings       a K split of up to 32 tokens has two CTAs an SM, or leaves room for the next launch's, whose first
//               weights then come under this one's tail (12288 x 4096 at 16 tokens: two ranks 14.0, with deep rings
//               and one CTA an SM 20.7).  Elsewhere they are as deep as an SM holds (19456 x 8192 at 16 tokens: 4
//               stages 39.7, 8 30.1).  Activations wait behind the weights that are on their way: their ring is as
//               long as the weights', or as there is room.
dg_status launch_i8_linear(const DeviceInfo* dev, const dg_choice& c, const void* x, const void* Wq, const float* sw,
                           void* y, int M, int N, int K, void* ws, size_t ws_bytes, cudaStream_t stream)
{
    if (ws_bytes < i8_workspace_bytes(M, K)) return DG_ERR_WORKSPACE_TOO_SMALL;
    for (int i = 0; i < 6; ++i)
        if (c.params[i] < 0 || (i > 3 && c.params[i] != 0)) return DG_ERR_BAD_VARIANT;
    // A multiple of the converting sets as weights' stages: a slot then belongs to one set, which sees its phases in
    // turn.  (A set that waits for a slot's next phase while the one before, another set's, is not complete would pass
    // at once.)
    const int want_stages = c.params[0], want_tokens = c.params[1], want_ranks = c.params[2], want_ctas = c.params[3];
    if (want_stages > 8 || want_stages % 2 != 0 || want_tokens % 16 != 0 || want_tokens > 128 ||
        want_ranks > kMaxRanks || want_ctas > 2)
        return DG_ERR_BAD_VARIANT;
    const int tiles = (N - 1) / kTileRows + 1, nkb = (K - 1) / kBlock + 1;
    const long long sms = dev->sm_count;
    int mp, groups, ns;
    long long units;
    auto cut = [&](int most) {                          // most: tokens of a group
        mp = want_tokens > 0 ? want_tokens : group_tokens(M, most);
        if (mp > (M + 15) / 16 * 16) mp = (M + 15) / 16 * 16;
        groups = (M - 1) / mp + 1;
        units = static_cast<long long>(tiles) * groups;
        ns = want_ranks > 0 ? want_ranks : 1;
        if (want_ranks == 0 && nkb > 4)
            for (int r = 2; r <= kMaxRanks && 2 * r <= nkb; ++r)
                if (units <= tc_cluster_capacity(dev, mp <= 32, r) && (mp > 32 || units * r <= 2 * sms * 13 / 15))
                    ns = r;
        if (want_ranks == 0 && ns == 1 && mp <= 32 && nkb >= 32 && units > sms &&
            (nkb >= 48 ? units * 7 <= sms * 9 : units * 6 <= sms * 7))
            ns = 3;
        if (ns > nkb) ns = nkb;
    };
    cut(128);
    if (ns > 1 && mp > 112) {
        if (want_tokens == 0)
            cut(64);
        else if (want_ranks == 0)
            ns = 1;
    }
    if (M > kFewTokens && want_tokens == 0 && want_ranks == 0 && want_ctas != 2) {
        float best = 0.0f;
        int most_best = 0, ns_best = 1;
        for (int most = 16; most <= 128; most += 16) {
            const int m = group_tokens(M, most);
            const long long u = static_cast<long long>(tiles) * ((M - 1) / m + 1);
            for (int r = 1; r <= kMaxRanks; r += r < 4 ? 1 : 2) {
                if (r > 1 && (nkb <= 4 || 2 * r > nkb || m > 112 || u > tc_cluster_capacity(dev, m <= 32, r))) break;
                const float t = estimate(dev->sm_count, u, nkb, m, r);
                if (most_best == 0 || t < best) {
                    best = t;
                    most_best = m;
                    ns_best = r;
                }
            }
        }
        cut(most_best);
        if (!(ns == 3 && ns_best == 1 && units > sms)) ns = ns_best;     // (thirds stay)
    }
    bool pair = want_ctas == 2;
    if (want_ctas == 0 && ns == 1 && mp >= 64 && nkb >= 16 && units * 8 >= 5 * sms)
        pair = (want_tokens == 0 || mp % 32 == 0) && want_stages % 6 == 0;
    if (pair) {
        // (a group that the rows do not fill is a smaller one, of 64 tokens at least)
        if (want_ranks > 1 || (want_tokens > 0 && (want_tokens < 64 || want_tokens % 32 != 0)) || want_stages % 6 != 0)
            return DG_ERR_BAD_VARIANT;
        mp = mp <= 64 ? 64 : (mp + 31) / 32 * 32;
        groups = (M - 1) / mp + 1;
        units = static_cast<long long>((tiles + 1) / 2) * groups;
        ns = 1;
    }
    const int xt = pair ? mp / 2 : mp;
    const void* fn = kernel_of(mp, pair);
    const int threads = pair ? Roles<true>::kThreads : Roles<false>::kThreads;
    if (units * ns > 0x7fffffffll || units * nkb / sms > 0x3fffffff) return DG_ERR_UNSUPPORTED_SHAPE;
    const int clusters = pair ? tc_cluster_capacity(dev, false, 2) : 0;
    if (pair && clusters < 1) return DG_ERR_UNSUPPORTED_SHAPE;
    const long long grid = pair                     ? 2 * (units < clusters ? units : clusters)
                           : ns > 1 || units < sms ? units * ns
                                                    : sms;
    const int share = ns > 1 ? (mp / 4 + ns - 1) / ns * 4 : mp;
    const size_t fold = ns > 1 ? static_cast<size_t>(ns) * share * kTileRows * 4 : 0;
    const size_t budget = mp <= 32 && ns > 1 ? 112 * 1024 : kMaxDynSmem;
    int stw = want_stages > 0 ? want_stages : mp <= 32 ? 8 : 6, stx = kDone - 1;
    const auto past = [&](size_t room, int x) { return smem_bytes(mp, xt, stw, x, fold) > room; };
    if (want_stages == 0 && !pair)
        while (stw > 4 && past(budget, stw < kDone ? stw : kDone - 1)) stw -= 2;
    while (stx > 2 && past(budget, stx)) --stx;
    if (want_stages == 0 && !pair)
        while (stw > 2 && past(budget, stx)) stw -= 2;
    // A table's pick holds for every row count of its bucket, whose groups and ranks differ, and with them the stages
    // that fit: as deep as this call's (two of each always do; depth changes no bits).
    if (c.from_table && !pair)
        while (stw > 2 && past(kMaxDynSmem, stx)) stw -= 2;
    size_t smem = smem_bytes(mp, xt, stw, stx, fold);
    if (smem > kMaxDynSmem) return DG_ERR_BAD_VARIANT;
    const size_t least = tc::smem_floor(mp <= 32 ? 256 : 512);
    if (smem < least) smem = least;
    if (occupancy(fn, threads, smem) < 1) return DG_ERR_UNSUPPORTED_SHAPE;
    uint8_t* qws = static_cast<uint8_t*>(ws) + kWsData;
    I8Args a{};
    a.N = N;
    a.K = K;
    a.M = M;
    a.nkb = nkb;
    a.groups = groups;
    a.mp = mp;
    a.units = static_cast<int>(units);
    a.nsplit = ns;
    a.share = share;
    a.sw_stages = stw;
    a.sx_stages = stx;
    a.x = qws;
    a.sx = reinterpret_cast<float*>(qws + code_bytes(M, K));
    a.sw = sw;
    a.y = static_cast<uint16_t*>(y);
    a.ws = static_cast<uint8_t*>(ws);
    CUtensorMap tmW;
    if (!encode_2d(&tmW, Wq, static_cast<uint64_t>(K), static_cast<uint64_t>(N), kBlock, kTileRows, true))
        return DG_ERR_CUDA;
    const dg_status st = launch_i8_quant(dev, x, qws, const_cast<float*>(a.sx), M, K, xt, stream);
    if (st != DG_OK) return st;
    void* args[] = {&tmW, &a};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(pair ? 2 : ns);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    if (launch_ordered(cfg, attr, 1, fn, args, Early::kWeights) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

}  // namespace dg
