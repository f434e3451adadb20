// dg_tc_dense.cu -- tcgen05 tensor-core family (DG_VAR_TC) for the bf16 linear and
// the fused gate/up + SiLU.mul (the default from 13 token rows up for the linear and
// from 9 for gate/up, where the tile is a real dense contraction), the A8W8
// block-scaled linear and the A4W4 linear on microscaled 4-bit operands.
//
// Swap-AB: a CTA owns a tile of 128 weight rows (the MMA's M) and one fixed K
// range; the tokens are the MMA's N (M padded to MP in {16, 32, 64, 128, 256};
// calls of 257..512 rows run as chunks of 256), so
// D[128, MP] = W_tile[128, Kr] . x[MP, Kr]^T accumulates in TMEM (fp32).
//   warp 0      TMA producer: 128x64 weight box + MPx64 activation box per stage
//               (128-byte swizzle), into a ring of `stages` shared-memory slots
//   warp 1      allocates TMEM; one elected lane issues tcgen05.mma (4 x K=16 per stage),
//               commits each stage back to its "empty" barrier and the last one
//               to the accumulator barrier
//   warps 2..5  epilogue: tcgen05.ld the accumulator (warp w reads TMEM lanes
//               32*(w%4)..+31), stage the tile in the idle ring and write it out
//               in coalesced pieces (store / pair gate+up), or fold a K-split
// Canonical order of this family: the K range of a tile is cut into `nsplit`
// contiguous ranges of 64-element blocks, a fixed function of (N, K, MP), or of
// (N, K) alone for the fixed split (tc_nsplit below); each range is one MMA chain from zero in ascending k; the
// range partials are folded left in fp32.  The nsplit CTAs of a tile form one
// thread-block cluster and each rank folds a slice of the tile's rows, over all
// ranks in rank order.  Up to 8 tokens the ranks push their rows into the folding
// rank's shared memory (st.async, counted on its mbarrier); beyond that each rank
// parks its partial tile in its own shared memory and, after a cluster barrier,
// the folding ranks read them through distributed shared memory.  Pipeline depth
// and the fold's transport change no bits.
// A4W4 (EPI 3, 4) differs in three places.  A stage holds 256 K elements as e2m1 codes and
// their block scales, which tcgen05.cp takes to TMEM for the block-scaled MMA
// (kind::mxf4 / kind::mxf4nvf4, 64 elements each): y = sum (qx sx)(qw sw) needs no scaling
// of ours but the tensor scales' product.  Tokens are cut into groups of up to 128, a CTA
// (or cluster) each, by a model (a4_plan).  Outputs leave TMEM straight to memory, and a
// K-split's ranks fold tokens, not rows.  Bound: up to some 32 rows the fixed chain (launch,
// first load, fold: 4.8 us for 1 x 4096 x 4096, of whose 9.4 MB the bytes need 1.4); with
// many rows neither memory nor the MMAs (512 x 24576 x 4096: 36 us, DRAM 21 %, tensor pipe
// 36 %) but a CTA's pace: alone it takes 0.30 us a K-block at 16 or 32 tokens, 0.38 at 64 and
// 0.51 to 0.56 at 128 (NV; MX 0.25, 0.30, 0.42), 16 of which and an epilogue make each of the three
// waves that 768 CTAs are.  What sets that pace was not measured.
// Every mbarrier wait is bounded: on timeout the kernel flags
// DG_DEVERR_WAIT_TIMEOUT in the workspace status word and winds down.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstdio>
#include <mutex>

#include "dg_a8.cuh"
#include "dg_fp4.cuh"
#include "dg_internal.h"
#include "dg_tc_common.cuh"

namespace dg {
namespace {

constexpr int kTileRows = 128;                    // MMA M
constexpr int kKB = 64;                           // K per stage: one 128-byte swizzled row
constexpr int kWBox = kTileRows * kKB * 2;        // 16 KB
constexpr int kThreads = 192;
constexpr int kMaxCluster = 8;                    // portable thread-block cluster size
constexpr size_t kCoResidentSmem = 112 * 1024;    // two CTAs per SM
constexpr int kPushMaxTokens = 8;                 // push fold up to this many tokens
constexpr int kWideStages = 4;                    // 256-token tiles: 4 x 48 KB, one CTA per SM

struct TcArgs {
    int N, K, M;
    int nsplit, nkb, tiles;
    int stages;
    int push;             // clustered: ranks push their rows into the owners' shared memory
    int mq;               // tokens pushed per row (M rounded up to 4)
    int slice_max;        // most rows one rank folds
    uint16_t* out;
    int ld_out;
    uint8_t* ws;          // status word only (the K-split fold stays on chip)
    // A8W8 (EPI 2): bf16 activations quantised in the prologue, the weight scales
    // [ceil(N/128)][kbs], and the most K-blocks one rank holds.
    const uint16_t* x;
    const float* sw;
    int kbs;
    int xq_blocks;
    // A8W8 with the quantisation done by a preceding launch: the codes come by TMA
    // (tmX over q [M, K]) and the activation scales from sxg [M, kbs].
    int preq;
    const float* sxg;
    // A4W4 (EPI 3, 4): the tiled block scales of the weights and of the activations, scale
    // tiles along K, and the tensor scales (NULL: 1).
    const uint8_t* sfw;
    const uint8_t* sfx;
    int nkt;
    int groups, tg;        // token groups of tg rows (one CTA or cluster each), M rows in all
    const float* gx;
    const float* gw;
};

constexpr int kA8Bufs = 4;                        // A8W8: per-block accumulators in flight
// A8W8: accumulator full/empty, and one "activations quantised" barrier per K-block a
// rank holds (at most kA8MaxBlocks).  The count stays even: the barrier block must stay a
// multiple of 16 bytes, since the push fold's receive buffer (16-byte st.async / float4
// accesses) follows it.
constexpr int kA8MaxBlocks = 16;
constexpr int kA8Bars = 2 * kA8Bufs + kA8MaxBlocks;
static_assert(kA8Bars % 2 == 0, "keep the barrier block 16-byte aligned");

// A4W4: the "activations quantised" barrier (and one to keep the block a multiple of 16 bytes).
constexpr int kA4Bars = 2;
// A4W4: K elements per stage (128 bytes of codes a row) and the bytes of a stage's block
// scales for 128 rows (NV: 4 tiles of 64 elements, MX: 2 of 128).
constexpr int kA4Block = 256;
__host__ __device__ constexpr int a4_scale_box(bool nv) { return kA4Block / fp4::tile_k(nv) * fp4::kTileBytes; }

// A8W8: bytes after the ring for the quantised activations [block][MP rows x 128 B] and
// the combined scales sx * sw [block][MP].
__host__ __device__ inline size_t a8_extra_bytes(int xq_blocks, int mp)
{
    return static_cast<size_t>(xq_blocks) * mp * (kA8Block + 4);
}

// Every thread of every CTA of the cluster executes this, unconditionally.
__device__ __forceinline__ void cluster_sync_all()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The same barrier in two halves: every thread arrives once, and waits (once) before
// its next arrival or its first access to a peer's shared memory.  The arrival is
// relaxed: the only data a peer reads before the next full barrier are the mbarriers,
// published by fence.mbarrier_init.release.cluster before it.
__device__ __forceinline__ void cluster_arrive()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Token stride (floats) of a parked partial tile: 144 = 128 rows + 16 puts consecutive
// tokens 64 bytes apart modulo 128, so the fold's 16-byte reads of two tokens fall in
// different bank halves (a stride of 128 rows sends every token to the same banks).
constexpr int kPStride = 144;

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t map_to_rank(uint32_t local_addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local_addr), "r"(rank));
    return r;
}

// Rows [lo, hi) of a 128-row tile folded by rank r of an ns-rank cluster
// (multiples of 4, so a (gate, up) row pair never straddles two ranks).
__host__ __device__ inline int slice_lo(int r, int ns) { return (r * (kTileRows / 4) / ns) * 4; }

// Four fp32 into a peer's shared memory; the bytes count on the peer's mbarrier.
__device__ __forceinline__ void st_async_f32x4(uint32_t remote, float a, float b, float c, float d, uint32_t remote_bar)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];"
                 ::"r"(remote), "f"(a), "f"(b), "f"(c), "f"(d), "r"(remote_bar)
                 : "memory");
}

// Four consecutive fp32 from a cluster peer's shared memory (read after a cluster
// barrier; the data does not change afterwards, so loads may be freely reordered).
__device__ __forceinline__ float4 ld_dsmem_f32x4(uint32_t addr)
{
    float4 v;
    asm("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// A4W4: the product of the tensor scales (read after the kernels before this one).
__device__ __forceinline__ float tensor_scale(const TcArgs& a)
{
    return __fmul_rn(a.gx ? *a.gx : 1.0f, a.gw ? *a.gw : 1.0f);
}

// Four consecutive rows n..n+3 of token t held by one thread (n a multiple of 4).
// (A4W4: the tensor scales' product alpha first.)
template <int EPI>
__device__ __forceinline__ void emit4(const TcArgs& a, int t, int n, float4 v, float alpha = 1.0f)
{
    if constexpr (EPI >= 3) v = make_float4(v.x * alpha, v.y * alpha, v.z * alpha, v.w * alpha);
    if constexpr (EPI != 1) {
        uint16_t* dst = a.out + static_cast<size_t>(t) * a.ld_out + n;
        if (n + 3 < a.N && (a.ld_out % 4) == 0) {
            const uint32_t lo = f32_to_bf16_bits(v.x) | (static_cast<uint32_t>(f32_to_bf16_bits(v.y)) << 16);
            const uint32_t hi = f32_to_bf16_bits(v.z) | (static_cast<uint32_t>(f32_to_bf16_bits(v.w)) << 16);
            *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
        } else {
            const float f[4] = {v.x, v.y, v.z, v.w};
            for (int i = 0; i < 4; ++i)
                if (n + i < a.N) dst[i] = f32_to_bf16_bits(f[i]);
        }
    } else {
        // rows (n, n+1) and (n+2, n+3) are (gate, up) pairs of outputs n/2 and n/2 + 1
        const float s0 = v.x / (1.0f + expf(-v.x));
        const float s1 = v.z / (1.0f + expf(-v.z));
        uint16_t* dst = a.out + static_cast<size_t>(t) * a.ld_out + n / 2;
        if (n + 1 < a.N) dst[0] = f32_to_bf16_bits(s0 * v.y);
        if (n + 3 < a.N) dst[1] = f32_to_bf16_bits(s1 * v.w);
    }
}

// Rows [r0, r1) (multiples of 4) of a tile's final fp32 values, staged in shared
// memory as S[t][r - r0] (row stride rs, a multiple of 4), written out by the 128
// epilogue threads (etid) in 8-row pieces (16 bytes of bf16) -- 4-row pieces (the
// 8-byte path of emit4) when the range does not start and end on 8-row boundaries:
// consecutive threads take consecutive pieces of one token's output row, so every
// warp store is contiguous.
template <int EPI>
__device__ __forceinline__ void store_staged(const TcArgs& a, const float* S, int rs, int tile, int r0, int r1,
                                             int etid, float alpha)
{
    // 16-byte pieces need the range to start on an 8-row boundary (rank slices may
    // start at any multiple of 4) and to hold whole 8-row pieces.
    if ((r1 - r0) % 8 != 0 || (r0 % 8) != 0) {
        const int q4 = (r1 - r0) / 4;
#pragma unroll 1
        for (int i = etid; i < a.M * q4; i += 128) {
            const int t = i / q4, c = i - t * q4;
            emit4<EPI>(a, t, tile * kTileRows + r0 + c * 4, *reinterpret_cast<const float4*>(S + t * rs + c * 4),
                       alpha);
        }
        return;
    }
    const int q = (r1 - r0) / 8;                      // 8-row pieces per token
    const int n0 = tile * kTileRows + r0;
    const bool vec = EPI != 1 ? (a.ld_out % 8) == 0 : (a.ld_out % 4) == 0;
#pragma unroll 1
    for (int i = etid; i < a.M * q; i += 128) {
        const int t = i / q, c = i - t * q;
        const float* src = S + t * rs + c * 8;
        float4 lo = *reinterpret_cast<const float4*>(src);
        float4 hi = *reinterpret_cast<const float4*>(src + 4);
        const int n = n0 + c * 8;
        if constexpr (EPI >= 3) {
            lo = make_float4(lo.x * alpha, lo.y * alpha, lo.z * alpha, lo.w * alpha);
            hi = make_float4(hi.x * alpha, hi.y * alpha, hi.z * alpha, hi.w * alpha);
        }
        if constexpr (EPI != 1) {
            if (vec && n + 7 < a.N) {
                uint4 w;
                w.x = f32_to_bf16_bits(lo.x) | (static_cast<uint32_t>(f32_to_bf16_bits(lo.y)) << 16);
                w.y = f32_to_bf16_bits(lo.z) | (static_cast<uint32_t>(f32_to_bf16_bits(lo.w)) << 16);
                w.z = f32_to_bf16_bits(hi.x) | (static_cast<uint32_t>(f32_to_bf16_bits(hi.y)) << 16);
                w.w = f32_to_bf16_bits(hi.z) | (static_cast<uint32_t>(f32_to_bf16_bits(hi.w)) << 16);
                *reinterpret_cast<uint4*>(a.out + static_cast<size_t>(t) * a.ld_out + n) = w;
            } else {
                emit4<EPI>(a, t, n, lo);           // (already scaled)
                emit4<EPI>(a, t, n + 4, hi);
            }
        } else {
            if (vec && n + 7 < a.N) {
                const float g0 = lo.x / (1.0f + expf(-lo.x)), g1 = lo.z / (1.0f + expf(-lo.z));
                const float g2 = hi.x / (1.0f + expf(-hi.x)), g3 = hi.z / (1.0f + expf(-hi.z));
                uint2 w;
                w.x = f32_to_bf16_bits(g0 * lo.y) | (static_cast<uint32_t>(f32_to_bf16_bits(g1 * lo.w)) << 16);
                w.y = f32_to_bf16_bits(g2 * hi.y) | (static_cast<uint32_t>(f32_to_bf16_bits(g3 * hi.w)) << 16);
                *reinterpret_cast<uint2*>(a.out + static_cast<size_t>(t) * a.ld_out + n / 2) = w;
            } else {
                emit4<1>(a, t, n, lo);
                emit4<1>(a, t, n + 4, hi);
            }
        }
    }
}

// A4W4: this rank's share of the tokens (contiguous), folded over the ranks in rank order: a
// warp takes a token's 128 rows, 4 a lane, with the loads of U tokens from all ranks (at
// most R) in flight, and writes 256 bytes of its output row.
template <int EPI, int R, int U>
__device__ __forceinline__ void fold_tokens(const TcArgs& a, uint32_t parked, int rank, int tile, int t0, int rows,
                                            int w, int lane)
{
    const float alpha = tensor_scale(a);
    const int lo = rows * rank / a.nsplit, hi = rows * (rank + 1) / a.nsplit;
    uint32_t peer[R];
#pragma unroll
    for (int r = 0; r < R; ++r) peer[r] = r < a.nsplit ? map_to_rank(parked, r) : 0u;
#pragma unroll 1
    for (int t = lo + w; t < hi; t += 4 * U) {
        float4 p[U][R];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r < a.nsplit && t + 4 * u < hi)
                    p[u][r] = ld_dsmem_f32x4(peer[r] + static_cast<uint32_t>(((t + 4 * u) * kTileRows + lane * 4) * 4));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + 4 * u >= hi) break;
            float4 s = p[u][0];
#pragma unroll
            for (int r = 1; r < R; ++r)
                if (r < a.nsplit) s = make_float4(s.x + p[u][r].x, s.y + p[u][r].y, s.z + p[u][r].z, s.w + p[u][r].w);
            emit4<EPI>(a, t0 + t + 4 * u, tile * kTileRows + lane * 4, s, alpha);
        }
    }
}

template <int MP, int EPI, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    tc_dense_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, TcArgs a)
{
    // EPI 2 (A8W8): e4m3 weights, 128 per stage row; the activations are quantised
    // into shared memory by the epilogue warps, so a stage holds the weight box only.
    // PAIR (256-token tiles without a K-split, more tiles than SMs): the CTA owns two
    // consecutive row tiles, a stage holds both weight boxes beside the one activation
    // box they share, and two TMEM accumulators take the two MMA chains -- one wave of
    // CTAs, each activation box loaded once for 256 weight rows.  Every tile's chain is
    // the same as a CTA of its own would run, so the bits do not change.
    // EPI 3, 4 (A4W4, MX and NV): e2m1 codes of weights and activations, 256 K elements per
    // stage, and the weights' block scales; tcgen05.cp takes the scales to tensor memory in
    // front of the MMAs that use them (two buffers, so a copy need not wait for the previous
    // stage's MMAs).  The activations' codes and scales come with each stage from a launch
    // ahead (preq), or the epilogue warps quantise the rank's whole K range into shared
    // memory beside the ring (few rows), and a stage holds the weights' part only.
    constexpr bool A8 = EPI == 2;
    constexpr bool A4 = EPI >= 3, NV = EPI == 4;
    static_assert(!PAIR || (MP == 256 && !A8 && !A4), "paired tiles are the 256-token bf16 path");
    constexpr int KBE = A4 ? kA4Block : (A8 ? kA8Block : kKB);      // K elements per stage
    constexpr int kXBox = A8 ? 0 : MP * kKB * 2;                    // 128 bytes a row, bf16 or e2m1
    constexpr int kSfBox = A4 ? a4_scale_box(NV) : 0;
    constexpr int kSfTiles = A4 ? kSfBox / fp4::kTileBytes : 1;     // scale tiles along a stage's K
    static_assert(!A4 || MP <= fp4::kTileRows, "one scale tile over a token group");
    constexpr int kWBoxes = PAIR ? 2 : 1;
    constexpr int kXOff = kWBox * kWBoxes + kSfBox;                 // weights, their scales, activations, their scales
    constexpr int kXSf = kXOff + kXBox;
    constexpr int kFullStage = kXSf + kSfBox;
    const int kStage = (A4 && !a.preq) ? kXOff : kFullStage;
    constexpr int kXBlock = kXBox + kSfBox;                         // A4 without preq: one K-block beside the ring
    // A4: accumulator, then two buffers each of the weights' and the activations' scales
    // (4 columns per 128 rows and MMA).
    constexpr uint32_t kSfCols = 4u * (kA4Block / fp4::tile_k(NV));
    constexpr uint32_t kSfw = MP < 32 ? 32 : MP, kSfx = kSfw + 2 * kSfCols;
    constexpr uint32_t kCols = A4   ? (kSfx + 2 * kSfCols <= 128 ? 128 : 256)
                               : A8 ? static_cast<uint32_t>(kA8Bufs * MP)
                                    : (PAIR ? 2 * MP : (MP < 32 ? 32 : MP));
    constexpr uint32_t kIdesc = A4 ? tc::idesc_fp4(MP, NV) : A8 ? tc::idesc_f8(MP) : tc::idesc_bf16(MP);
    constexpr int kKX = A4 ? KBE / 2 : KBE;       // a stage's width in elements of the tensor maps (A4: bytes)
    constexpr int kExtraBars = A8 ? kA8Bars : A4 ? kA4Bars : 0;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int S = a.stages;
    uint8_t* xq = smem + S * kStage;                                            // A8: [block][MP x 128 B]
    float* sxs = reinterpret_cast<float*>(xq + static_cast<size_t>(a.xq_blocks) * MP * kA8Block);   // A8: [block][MP]
    const size_t xtra = A8 ? a8_extra_bytes(a.xq_blocks, MP) : A4 ? static_cast<size_t>(a.xq_blocks) * kXBlock : 0;
    // full[S], empty[S], accum, recv (+ A8: acc_full[4], acc_empty[4], x_ready)
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * kStage + xtra);
    const int nbars = 2 * S + 2 + kExtraBars;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + nbars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    // Push fold: rows pushed here by every rank, [rank][slice row][mq] fp32.
    float* recv = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(bars) + nbars * 8 + 16);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool clustered = a.nsplit > 1;
    // the parked partial tile takes the padded stride when the idle ring holds it
    const int pstride = A4 ? kTileRows : static_cast<size_t>(S) * kStage >= static_cast<size_t>(MP) * kPStride * 4 ? kPStride : kTileRows;
    int tile = PAIR ? 2 * static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x) / a.nsplit;
    // A4: token rows [t0, t0 + rows_here) of the call; groups of one tile run side by side, so
    // the tile's weights come from HBM once.
    int group = 0, t0 = 0, rows_here = a.M;
    if constexpr (A4) {
        group = tile % a.groups;
        tile /= a.groups;
        t0 = group * a.tg;
        rows_here = a.M - t0 < a.tg ? a.M - t0 : a.tg;
    }
    const int ntiles_here = PAIR ? (tile + 1 < a.tiles ? 2 : 1) : 1;
    const int split = clustered ? static_cast<int>(cluster_rank()) : 0;
    const int kb0 = static_cast<int>((static_cast<long long>(split) * a.nkb) / a.nsplit);
    const int kb1 = static_cast<int>((static_cast<long long>(split + 1) * a.nkb) / a.nsplit);
    const int nkb = kb1 - kb0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2 * S + 2; ++s) tc::bar_init(tc::su32(bars + s), 1);
        if constexpr (A8) {
            for (int b = 0; b < kA8Bufs; ++b) {
                tc::bar_init(tc::su32(bars + 2 * S + 2 + b), 1);             // MMA commit
                tc::bar_init(tc::su32(bars + 2 * S + 2 + kA8Bufs + b), 4);   // one per epilogue warp
            }
            for (int i = 0; i < kA8MaxBlocks; ++i) tc::bar_init(tc::su32(bars + 2 * S + 2 + 2 * kA8Bufs + i), 1);
        }
        if constexpr (A4) tc::bar_init(tc::su32(bars + 2 * S + 2), 4);       // one per epilogue warp
        if (clustered && a.push) {
            // every rank pushes this rank's slice of rows, mq tokens each
            const int rows = slice_lo(split + 1, a.nsplit) - slice_lo(split, a.nsplit);
            tc::bar_expect_tx(tc::su32(bars + 2 * S + 1), static_cast<uint32_t>(a.nsplit * rows * a.mq * 4));
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::su32(tmem_holder)),
                     "r"(kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    // Every rank's barriers exist before any remote access: arrive now, wait just before
    // the first access to a peer (the producer streams meanwhile).
    if (clustered) cluster_arrive();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = *tmem_holder;
    const uint32_t full0 = tc::su32(bars), empty0 = tc::su32(bars + S), accum = tc::su32(bars + 2 * S);
    const uint32_t recv_bar = tc::su32(bars + 2 * S + 1);
    const uint32_t accf0 = tc::su32(bars + 2 * S + 2), acce0 = accf0 + 8 * kA8Bufs, xfull0 = accf0 + 16 * kA8Bufs;

    pdl_launch_dependents();
    if (warp == 0) {
        if (tc::elect_one()) {
            // Weight boxes of the first ring fill do not depend on earlier kernels:
            // issue them before waiting, the activation boxes after.
            // Weights are read once: they are the first lines evicted from L2.
            const uint64_t once = tc::policy_evict_first();
            const int pre = nkb < S ? nkb : S;
            // A4: scale tiles of K-block kb, at most kSfBox bytes a side (the last block may have fewer)
            auto sf_bytes = [&](int kb) {
                const int left = a.nkt - kb * kSfTiles;
                return static_cast<uint32_t>((left < kSfTiles ? left : kSfTiles) * fp4::kTileBytes);
            };
            auto stage_tx = [&](int kb) {
                if constexpr (A4)
                    return a.preq ? static_cast<uint32_t>(kWBox + kXBox) + sf_bytes(kb) * 2
                                  : static_cast<uint32_t>(kWBox) + sf_bytes(kb);
                return static_cast<uint32_t>(kFullStage);
            };
            auto load_sfw = [&](uint32_t dst, int kb, uint32_t bar) {
                tc::bulk_load(dst + kWBox,
                              a.sfw + (static_cast<size_t>(tile) * a.nkt + kb * kSfTiles) * fp4::kTileBytes, sf_bytes(kb),
                              bar);
            };
            auto load_sfx = [&](uint32_t dst, int kb, uint32_t bar) {
                // A group's scales start a tile row of their own: the MMA reads them from the first
                // of four tensor-memory columns, which has to be a multiple of four.
                tc::bulk_load(dst + kXSf, a.sfx + (static_cast<size_t>(group) * a.nkt + kb * kSfTiles) * fp4::kTileBytes,
                              sf_bytes(kb), bar);
            };
            for (int i = 0; i < pre; ++i) {
                const uint32_t dst = tc::su32(smem + i * kStage);
                tc::bar_expect_tx(full0 + 8 * i, stage_tx(kb0 + i));
                if constexpr (A4) load_sfw(dst, kb0 + i, full0 + 8 * i);
                tc::tma_2d_hint(dst, &tmW, (kb0 + i) * kKX, tile * kTileRows, full0 + 8 * i, once);
                if constexpr (PAIR)        // (rows past N read as zeros when the tile is the last, odd one)
                    tc::tma_2d_hint(dst + kWBox, &tmW, (kb0 + i) * KBE, (tile + 1) * kTileRows, full0 + 8 * i, once);
            }
            pdl_wait();
            const bool with_x = !A8 && (!A4 || a.preq);
            auto load_x = [&](uint32_t dst, int kb, uint32_t bar) {
                tc::tma_2d(dst + kXOff, &tmX, kb * kKX, t0, bar);
                if constexpr (A4) load_sfx(dst, kb, bar);
            };
            if (with_x)
                for (int i = 0; i < pre; ++i) load_x(tc::su32(smem + i * kStage), kb0 + i, full0 + 8 * i);
            if constexpr (A8)
                if (a.preq)
                    // every block's codes at once (rows M..MP-1 read as zeros), each
                    // completing its own x_full barrier
                    for (int i = 0; i < nkb; ++i) {
                        tc::bar_expect_tx(xfull0 + 8 * i, MP * kA8Block);
                        tc::tma_2d(tc::su32(xq + static_cast<size_t>(i) * MP * kA8Block), &tmX, (kb0 + i) * kA8Block,
                                   0, xfull0 + 8 * i);
                    }
            int s = 0;                       // stage and round of K-block i (pre is S where there is a second round)
            uint32_t round = 1;
            for (int i = pre; i < nkb; ++i) {
                if (!tc::bar_wait(empty0 + 8 * s, (round & 1u) ^ 1u, abort_flag)) break;
                const uint32_t dst = tc::su32(smem + s * kStage);
                tc::bar_expect_tx(full0 + 8 * s, stage_tx(kb0 + i));
                const int k = (kb0 + i) * kKX;
                if constexpr (A4) load_sfw(dst, kb0 + i, full0 + 8 * s);
                tc::tma_2d_hint(dst, &tmW, k, tile * kTileRows, full0 + 8 * s, once);
                if constexpr (PAIR) tc::tma_2d_hint(dst + kWBox, &tmW, k, (tile + 1) * kTileRows, full0 + 8 * s, once);
                if (with_x) load_x(dst, kb0 + i, full0 + 8 * s);
                if (++s == S) {
                    s = 0;
                    ++round;
                }
            }
        } else {
            pdl_wait();
        }
    } else if (warp == 1) {
        pdl_wait();
        if (tc::elect_one()) {
            const uint32_t ring = tc::su32(smem), xring = (A4 && !a.preq) ? tc::su32(xq) : ring + kXOff;
            const uint64_t dw0 = tc::sw128_desc(ring), dx0 = tc::sw128_desc(xring);              // (A4)
            const uint64_t dsw0 = tc::scale_desc(ring + kWBox), dsx0 = tc::scale_desc(xring + kXBox);
            int s = -1;
            uint32_t round = 0;
            for (int i = 0; i < nkb; ++i) {
                if (++s == S) {
                    s = 0;
                    ++round;
                }
                if (!tc::bar_wait(full0 + 8 * s, round & 1u, abort_flag)) break;
                const uint32_t wa = tc::su32(smem + s * kStage);
                if constexpr (A8) {
                    // One K-block (128 elements, 4 x K=32) into accumulator b, from zero;
                    // the epilogue scales and folds it, then frees the accumulator.
                    const int b = i % kA8Bufs;
                    if (!tc::bar_wait(xfull0 + 8 * i, 0, abort_flag)) break;        // block i quantised
                    if (i >= kA8Bufs &&
                        !tc::bar_wait(acce0 + 8 * b, static_cast<uint32_t>(i / kA8Bufs - 1) & 1u, abort_flag))
                        break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t xa = tc::su32(xq + static_cast<size_t>(i) * MP * kA8Block);
#pragma unroll
                    for (int kk = 0; kk < kA8Block / 32; ++kk)
                        tc::mma_f8(tmem + static_cast<uint32_t>(b * MP), tc::sw128_desc(wa + kk * 32),
                                   tc::sw128_desc(xa + kk * 32), kIdesc, kk > 0 ? 1u : 0u);
                    tc::commit(empty0 + 8 * s);
                    tc::commit(accf0 + 8 * b);
                } else if constexpr (A4) {
                    if (!a.preq && i == 0 && !tc::bar_wait(accf0, 0, abort_flag)) break;     // activations quantised
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    // Descriptors count 16-byte units: a stage, a K-block or 64 elements further on
                    // is an addition.
                    const uint32_t ws = static_cast<uint32_t>(s * (kStage / 16));
                    const uint32_t xs = a.preq ? ws : static_cast<uint32_t>(i * (kXBlock / 16));
                    const uint64_t dw = dw0 + ws, dx = dx0 + xs, dsw = dsw0 + ws, dsx = dsx0 + xs;
                    const uint32_t cw = tmem + kSfw + (i & 1) * kSfCols;
                    const uint32_t cx = tmem + kSfx + (i & 1) * kSfCols;
                    const int kleft = a.K - (kb0 + i) * kA4Block;
                    constexpr int kPer = fp4::tile_k(NV) / 64;                                    // MMAs per scale tile
                    // tcgen05.cp and tcgen05.mma of one thread run in order
                    auto scales = [&](int j) {
                        tc::copy_scales(cw + 4 * j, dsw + j * (fp4::kTileBytes / 16));
                        tc::copy_scales(cx + 4 * j, dsx + j * (fp4::kTileBytes / 16));
                    };
                    auto mma = [&](int kk) {
                        const int j = kk / kPer;
                        const uint32_t id = static_cast<uint32_t>(kk % kPer) * 2;                 // MX: byte pair 0 or 2
                        tc::mma_fp4<NV>(tmem, dw + kk * 2, dx + kk * 2, kIdesc | (id << 4) | (id << 29), cw + 4 * j,
                                        cx + 4 * j, (i > 0 || kk > 0) ? 1u : 0u);
                    };
                    if (kleft >= kA4Block) {           // straight: a test in front of each cost 0.1 us a block
#pragma unroll
                        for (int j = 0; j < kSfTiles; ++j) scales(j);
#pragma unroll
                        for (int kk = 0; kk < kA4Block / 64; ++kk) mma(kk);
                    } else {
                        const int steps = (kleft + 63) / 64;
#pragma unroll 1
                        for (int j = 0; j * kPer < steps; ++j) scales(j);
#pragma unroll 1
                        for (int kk = 0; kk < steps; ++kk) mma(kk);
                    }
                    tc::commit(empty0 + 8 * s);
                } else {
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t xa = wa + kWBox * kWBoxes;
#pragma unroll
                    for (int kk = 0; kk < kKB / 16; ++kk)
                        tc::mma_bf16(tmem, tc::sw128_desc(wa + kk * 32), tc::sw128_desc(xa + kk * 32), kIdesc,
                                     (i > 0 || kk > 0) ? 1u : 0u);
                    if constexpr (PAIR)
#pragma unroll
                        for (int kk = 0; kk < kKB / 16; ++kk)
                            tc::mma_bf16(tmem + static_cast<uint32_t>(MP), tc::sw128_desc(wa + kWBox + kk * 32),
                                         tc::sw128_desc(xa + kk * 32), kIdesc, (i > 0 || kk > 0) ? 1u : 0u);
                    tc::commit(empty0 + 8 * s);
                }
            }
            tc::commit(accum);           // fires once every MMA issued above has completed
        }
    } else {
        pdl_wait();
        // Epilogue warps 2..5 -> TMEM lane quarter (warp % 4).
        const int q = warp & 3;
        const int row = q * 32 + lane;
        if constexpr (A4) {
            if (!a.preq) {
                // A warp takes one token's 256 elements of a K-block at a time, 8 a lane: the
                // arithmetic of fp4_quant_kernel, codes into the swizzled rows that the MMA
                // reads, scale words into the scale tile.  Rows M.. stay unset: an MMA column
                // depends on its own row only, and theirs are not stored.
                constexpr int kShare = fp4::block_len(NV) / 8, kWord = 4 * kShare, kU = 4;
                const float g = a.gx ? *a.gx : 1.0f, g6 = __fmul_rn(6.0f, g);
                const int items = nkb * a.M, step_i = 4 / a.M, step_t = 4 - step_i * a.M;
                int gi = q / a.M, gt = q - gi * a.M;                 // (K-block, token) of the warp's next item
#pragma unroll 1
                for (int z0 = q; z0 < items; z0 += 4 * kU) {
                    uint4 raw[kU];
                    int ii[kU], tt[kU];
#pragma unroll
                    for (int u = 0; u < kU; ++u) {
                        const int z = z0 + 4 * u;
                        ii[u] = gi;
                        tt[u] = gt;
                        gi += step_i;
                        gt += step_t;
                        if (gt >= a.M) {
                            gt -= a.M;
                            ++gi;
                        }
                        const int k = (kb0 + ii[u]) * kA4Block + lane * 8;
                        raw[u] = make_uint4(0, 0, 0, 0);
                        if (z < items && k < a.K) raw[u] = ld_stream_after(a.x + static_cast<size_t>(tt[u]) * a.K + k);
                    }
#pragma unroll
                    for (int u = 0; u < kU; ++u) {
                        if (z0 + 4 * u >= items) break;
                        uint32_t m = fp4::amax8(raw[u]);
#pragma unroll
                        for (int o = 1; o < kShare; o <<= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
                        const fp4::Scale bs = fp4::block_scale<NV>(m, g6, g);
                        float v[8];
                        fp4::unpack8(raw[u], v);
                        uint8_t* blk = xq + static_cast<size_t>(ii[u]) * kXBlock;
                        *reinterpret_cast<uint32_t*>(blk + tc::sw128_offset(tt[u], lane / 4) + (lane & 3) * 4) =
                            fp4::encode8<NV>(v, bs);
                        const bool in = (kb0 + ii[u]) * kA4Block + lane * 8 < a.K;      // scales past K are zero
                        uint32_t w = in ? bs.byte << (8 * ((lane / kShare) & 3)) : 0u;
#pragma unroll
                        for (int o = kShare; o < kWord; o <<= 1) w |= __shfl_xor_sync(kFull, w, o);
                        if (lane % kWord == 0)
                            *reinterpret_cast<uint32_t*>(blk + kXBox + (lane / kWord) * fp4::kTileBytes +
                                                         fp4::tile_offset(tt[u], 0)) = w;
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) tc::bar_arrive(accf0);
            }
        }
        if constexpr (A8) {
            const int et = threadIdx.x - 64;
            if (a.preq) {
                // The codes arrive by TMA; the combined scales sx * sw of the live rows.
                for (int z = et; z < nkb * MP; z += 128) {
                    const int i = z / MP, t = z & (MP - 1);
                    sxs[z] = t < a.M ? __fmul_rn(a.sxg[static_cast<size_t>(t) * a.kbs + kb0 + i],
                                                 a.sw[static_cast<size_t>(tile) * a.kbs + kb0 + i])
                                     : 0.0f;
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
            // (1) Rows M..MP-1 of every block get zero codes and scales (their columns
            // are never stored); chunk z = (i * MP + t) * 8 + ch.
            const int live_rows = a.M;
            if (!a.preq && live_rows < MP) {
                for (int z = et; z < nkb * MP * 8; z += 128) {
                    const int ch = z & 7, t = (z >> 3) & (MP - 1), i = z / (MP * 8);
                    if (t < live_rows) continue;
                    *reinterpret_cast<uint4*>(xq + static_cast<size_t>(i) * MP * kA8Block + tc::sw128_offset(t, ch)) =
                        make_uint4(0, 0, 0, 0);
                    if (ch == 0) sxs[i * MP + t] = 0.0f;
                }
            }
            // (2) Quantise the live rows: 8 threads per (block, token) group, 16 elements
            // each, groups in block-major order g = i * M + t, 16 groups per slot of the
            // 128 threads.  Eight slots' loads are issued before any is used; after each
            // slot the blocks it completed are released to the MMA warp (x_full[i]), so
            // the first MMAs overlap the rest of the quantisation.  sxs holds the block's
            // combined scale sx * sw.
            constexpr int kU = 8;
            const int groups = a.preq ? 0 : nkb * live_rows;
            const int step_i = 16 / live_rows, step_t = 16 % live_rows;
            int gi = (et >> 3) / live_rows, gt = (et >> 3) % live_rows;     // (i, t) of this thread's next group
            int released = 0;
#pragma unroll 1
            for (int g0 = 0; g0 < groups; g0 += 16 * kU) {
                uint4 raw[kU][2];
                float swv[kU];
                int ii[kU], tt[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int g = g0 + u * 16 + (et >> 3);
                    ii[u] = gi;
                    tt[u] = gt;
                    gi += step_i;
                    gt += step_t;
                    if (gt >= live_rows) {
                        gt -= live_rows;
                        ++gi;
                    }
                    const int k0 = (kb0 + ii[u]) * kA8Block + (et & 7) * 16;
                    raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
                    swv[u] = 0.0f;
                    if (g < groups) {
                        if (k0 < a.K) {
                            const uint4* src =
                                reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(tt[u]) * a.K + k0);
                            raw[u][0] = src[0];
                            raw[u][1] = src[1];
                        }
                        swv[u] = a.sw[static_cast<size_t>(tile) * a.kbs + kb0 + ii[u]];
                    }
                }
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int g = g0 + u * 16 + (et >> 3);
                    float v[16];
                    a8_unpack16(raw[u][0], raw[u][1], v);
                    const float amax = a8_block_amax(v);          // every lane takes part
                    if (g < groups) {
                        *reinterpret_cast<uint4*>(xq + static_cast<size_t>(ii[u]) * MP * kA8Block +
                                                  tc::sw128_offset(tt[u], et & 7)) = a8_codes(v, a8_recip_scale(amax));
                        if ((et & 7) == 0) sxs[ii[u] * MP + tt[u]] = __fmul_rn(a8_scale(amax), swv[u]);
                    }
                    const int gend = g0 + (u + 1) * 16 < groups ? g0 + (u + 1) * 16 : groups;
                    if ((released + 1) * live_rows <= gend) {     // the same decision in every thread
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        asm volatile("bar.sync 1, 128;" ::: "memory");
                        while ((released + 1) * live_rows <= gend) {
                            if (et == 0) tc::bar_arrive(xfull0 + 8 * released);
                            ++released;
                        }
                    }
                }
            }
            // (2) Fold the blocks in ascending order: tot = fma(p_b, sx_b * sw_b, tot), from 0.
            float tot[MP];
#pragma unroll
            for (int j = 0; j < MP; ++j) tot[j] = 0.0f;
            bool all_in = true;
#pragma unroll 1
            for (int i = 0; i < nkb; ++i) {
                const int b = i % kA8Bufs;
                const bool w = tc::bar_wait(accf0 + 8 * b, static_cast<uint32_t>(i / kA8Bufs) & 1u, abort_flag);
                if (!__all_sync(kFull, w)) {
                    all_in = false;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
                for (int c = 0; c < MP / 16; ++c) {
                    if (c * 16 >= a.M) break;
                    uint32_t v[16];
                    tc::tmem_ld16(tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(b * MP + c * 16), v);
                    const float4* sc4 = reinterpret_cast<const float4*>(sxs + i * MP + c * 16);
#pragma unroll
                    for (int j4 = 0; j4 < 4; ++j4) {
                        const float4 sc = sc4[j4];
                        const int j = c * 16 + 4 * j4;
                        tot[j + 0] = __fmaf_rn(__uint_as_float(v[4 * j4 + 0]), sc.x, tot[j + 0]);
                        tot[j + 1] = __fmaf_rn(__uint_as_float(v[4 * j4 + 1]), sc.y, tot[j + 1]);
                        tot[j + 2] = __fmaf_rn(__uint_as_float(v[4 * j4 + 2]), sc.z, tot[j + 2]);
                        tot[j + 3] = __fmaf_rn(__uint_as_float(v[4 * j4 + 3]), sc.w, tot[j + 3]);
                    }
                }
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) tc::bar_arrive(acce0 + 8 * b);
            }
            // (3) The rank's totals into TMEM columns 0..MP-1, where the tail below reads a
            // finished accumulator (every MMA has completed by now).
            if (all_in) {
#pragma unroll
                for (int c = 0; c < MP / 16; ++c) {
                    uint32_t v[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(tot[c * 16 + j]);
                    tc::tmem_st16(tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(c * 16), v);
                }
                tc::tmem_st_wait();
            }
        }
        const bool ok = tc::bar_wait(accum, 0, abort_flag);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const float alpha = A4 ? tensor_scale(a) : 1.0f;
        // `good` may differ between threads when a wait ran out; every named barrier
        // below is still reached by all 128 epilogue threads.
        const bool good = ok && !*abort_flag;
        if (!good && row == 0) set_status(a.ws, DG_DEVERR_WAIT_TIMEOUT);
        if (A4 && !clustered) {
            // A lane holds one weight row, a warp 32 of them: 64 bytes of one token's output
            // per store, straight from tensor memory.
            const int n = tile * kTileRows + row;
            if (good) {
                constexpr int kC = MP < 32 ? 16 : 32;
                uint16_t* dst = a.out + static_cast<size_t>(t0) * a.ld_out + n;
#pragma unroll 1
                for (int c = 0; c < rows_here; c += kC) {
                    uint32_t v[kC];
                    const uint32_t at = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(c);
                    if constexpr (kC == 16)
                        tc::tmem_ld16(at, v);
                    else
                        tc::tmem_ld32(at, v);
                    const int left = n < a.N ? rows_here - c : 0;
                    if (left >= kC) {
#pragma unroll
                        for (int j = 0; j < kC; ++j)
                            dst[static_cast<size_t>(c + j) * a.ld_out] = f32_to_bf16_bits(__uint_as_float(v[j]) * alpha);
                    } else {
#pragma unroll
                        for (int j = 0; j < kC; ++j)
                            if (j < left)
                                dst[static_cast<size_t>(c + j) * a.ld_out] =
                                    f32_to_bf16_bits(__uint_as_float(v[j]) * alpha);
                    }
                }
            }
        } else if (!clustered) {
            // Stage the tile S[t][row] (fp32) in the now idle stage memory, then write
            // it out in coalesced 16-byte pieces (paired tiles: one after the other).
            float* S = reinterpret_cast<float*>(smem);
#pragma unroll 1
            for (int pt = 0; pt < ntiles_here; ++pt) {
                if (pt > 0) asm volatile("bar.sync 1, 128;" ::: "memory");     // S is free again
                if (good) {
#pragma unroll 1
                    for (int c = 0; c < MP / 16 && c * 16 < a.M; ++c) {
                        uint32_t v[16];
                        tc::tmem_ld16(tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(pt * MP + c * 16), v);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (c * 16 + j < a.M) S[(c * 16 + j) * kTileRows + row] = __uint_as_float(v[j]);
                    }
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (good) store_staged<EPI>(a, S, kTileRows, tile + pt, 0, kTileRows, threadIdx.x - 64, alpha);
            }
        } else if (a.push) {
            // Push row `row` of this rank's partial tile (tokens 0..mq-1) into the
            // shared memory of the rank that folds it.
            cluster_wait();
            if (good) {
                int owner = 0;
                while (owner + 1 < a.nsplit && row >= slice_lo(owner + 1, a.nsplit)) ++owner;
                const uint32_t dst = map_to_rank(tc::su32(recv), static_cast<uint32_t>(owner)) +
                                     static_cast<uint32_t>(((split * a.slice_max + row - slice_lo(owner, a.nsplit)) * a.mq) * 4);
                const uint32_t dbar = map_to_rank(recv_bar, static_cast<uint32_t>(owner));
#pragma unroll 1
                for (int c = 0; c < MP / 16 && c * 16 < a.mq; ++c) {
                    uint32_t v[16];
                    tc::tmem_ld16(tmem + (static_cast<uint32_t>(q * 32) << 16) + c * 16, v);
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        if (c * 16 + j < a.mq)
                            st_async_f32x4(dst + (c * 16 + j) * 4, __uint_as_float(v[j]), __uint_as_float(v[j + 1]),
                                           __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]), dbar);
                }
            }
            // This rank's slice: wait for every rank's rows, fold them in rank order into
            // S[t][r] (the idle stage memory), then coalesced stores.
            const int lo = slice_lo(split, a.nsplit), hi = slice_lo(split + 1, a.nsplit);
            const bool got = good && tc::bar_wait(recv_bar, 0, abort_flag);
            if (good && !got && row == 0) set_status(a.ws, DG_DEVERR_WAIT_TIMEOUT);
            const int r = threadIdx.x - 64;                // 0..127: one folded row per thread
            float* S = reinterpret_cast<float*>(smem);
            const int rs = a.slice_max;
            if (got && r < hi - lo) {
#pragma unroll 1
                for (int t = 0; t < a.mq; t += 4) {
                    float4 acc = *reinterpret_cast<const float4*>(recv + (static_cast<size_t>(r) * a.mq + t));
                    for (int s2 = 1; s2 < a.nsplit; ++s2) {
                        const float4 v = *reinterpret_cast<const float4*>(
                            recv + ((static_cast<size_t>(s2) * a.slice_max + r) * a.mq + t));
                        acc.x = acc.x + v.x;
                        acc.y = acc.y + v.y;
                        acc.z = acc.z + v.z;
                        acc.w = acc.w + v.w;
                    }
                    S[(t + 0) * rs + r] = acc.x;
                    S[(t + 1) * rs + r] = acc.y;
                    S[(t + 2) * rs + r] = acc.z;
                    S[(t + 3) * rs + r] = acc.w;
                }
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (got && !*abort_flag) store_staged<EPI>(a, S, rs, tile, lo, hi, r, alpha);
        } else if (good) {
            // Park this rank's partial tile P[t][row] (fp32) in the now idle stage memory.
            float* P = reinterpret_cast<float*>(smem);
#pragma unroll(A4 ? 2 : 1)
            for (int c = 0; c < MP / 16 && (!A4 || c * 16 < rows_here); ++c) {
                uint32_t v[16];
                tc::tmem_ld16(tmem + (static_cast<uint32_t>(q * 32) << 16) + c * 16, v);
#pragma unroll
                for (int j = 0; j < 16; ++j) P[(c * 16 + j) * pstride + row] = __uint_as_float(v[j]);
            }
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
    if (clustered && !a.push) {
        cluster_wait();                      // (the arrival at the start)
        cluster_sync_all();                  // every rank's partial tile is in place
        if (A4 && warp >= 2) {
            if (!*abort_flag) {
                if (a.nsplit <= 4)
                    fold_tokens<EPI, 4, 4>(a, tc::su32(smem), split, tile, t0, rows_here, warp - 2, lane);
                else
                    fold_tokens<EPI, 8, 2>(a, tc::su32(smem), split, tile, t0, rows_here, warp - 2, lane);
            }
        } else if (warp >= 2) {
            // This rank folds rows [lo, hi) (multiples of 4) for all tokens: P_0 + P_1 + ...
            // in rank order, four rows per thread, read through DSMEM.
            const int etid = threadIdx.x - 64;
            const int lo = (split * (kTileRows / 4) / a.nsplit) * 4;
            const int hi = ((split + 1) * (kTileRows / 4) / a.nsplit) * 4;
            const int w4 = (hi - lo) / 4;
            const int count = w4 * a.M;
            const float alpha = A4 ? tensor_scale(a) : 1.0f;
            const uint32_t pbase = tc::su32(smem);
            uint32_t peer[kMaxCluster];
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) peer[r] = r < a.nsplit ? map_to_rank(pbase, r) : 0u;
            if (!*abort_flag) {
#pragma unroll 1
                for (int base = 0; base < count; base += 2 * 128) {
                    float4 acc[2];
                    int tt[2], rr[2];
                    bool vv[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int e = base + u * 128 + etid;
                        vv[u] = e < count;
                        tt[u] = vv[u] ? e / w4 : 0;
                        rr[u] = lo + 4 * (vv[u] ? e - tt[u] * w4 : 0);
                        const uint32_t off = static_cast<uint32_t>((tt[u] * pstride + rr[u]) * 4);
                        acc[u] = vv[u] ? ld_dsmem_f32x4(peer[0] + off) : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                    // every rank's loads first (they overlap), then the adds in rank order
                    float4 pv[kMaxCluster - 1][2];
#pragma unroll
                    for (int s2 = 1; s2 < kMaxCluster; ++s2)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            pv[s2 - 1][u] = (s2 < a.nsplit && vv[u])
                                ? ld_dsmem_f32x4(peer[s2] + static_cast<uint32_t>((tt[u] * pstride + rr[u]) * 4))
                                : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int s2 = 1; s2 < kMaxCluster; ++s2) {
                        if (s2 >= a.nsplit) break;
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            acc[u].x = acc[u].x + pv[s2 - 1][u].x;
                            acc[u].y = acc[u].y + pv[s2 - 1][u].y;
                            acc[u].z = acc[u].z + pv[s2 - 1][u].z;
                            acc[u].w = acc[u].w + pv[s2 - 1][u].w;
                        }
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        if (vv[u]) emit4<EPI>(a, tt[u], tile * kTileRows + rr[u], acc[u], alpha);
                }
            }
        }
        cluster_sync_all();                  // no rank leaves while others still read its partials
    }
    if (clustered && a.push && warp < 2) cluster_wait();   // (the arrival at the start)
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) set_status(a.ws, DG_DEVERR_WAIT_TIMEOUT);
    if (warp == 1) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
    }
}

// ------------------------------------------------------------------------ host

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

// 2-D tiled map, 128-byte swizzle: bf16 elements, or bytes (e4m3 codes) when `u8`.
bool encode_2d(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer, uint32_t box_inner,
               uint32_t box_outer, bool u8 = false)
{
    std::call_once(g_encode_once, [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
        cudaGetLastError();
    });
    if (!g_encode) return false;
    const cuuint64_t dims[2] = {inner, outer};
    const cuuint64_t strides[1] = {inner * (u8 ? 1 : 2)};
    const cuuint32_t box[2] = {box_inner, box_outer};
    const cuuint32_t estr[2] = {1, 1};
    return g_encode(m, u8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MP, int EPI>
const void* tc_fn()
{
    return reinterpret_cast<const void*>(&tc_dense_kernel<MP, EPI, false>);
}

const void* tc_lookup(int mp, int epi)
{
    switch (mp * 4 + epi) {
    case 16 * 4 + 0: return tc_fn<16, 0>();
    case 16 * 4 + 1: return tc_fn<16, 1>();
    case 16 * 4 + 2: return tc_fn<16, 2>();
    case 32 * 4 + 0: return tc_fn<32, 0>();
    case 32 * 4 + 1: return tc_fn<32, 1>();
    case 32 * 4 + 2: return tc_fn<32, 2>();
    case 64 * 4 + 0: return tc_fn<64, 0>();
    case 64 * 4 + 1: return tc_fn<64, 1>();
    case 64 * 4 + 2: return tc_fn<64, 2>();
    case 128 * 4 + 0: return tc_fn<128, 0>();
    case 128 * 4 + 1: return tc_fn<128, 1>();
    case 256 * 4 + 0: return tc_fn<256, 0>();
    case 256 * 4 + 1: return tc_fn<256, 1>();
    default: return nullptr;
    }
}

// The paired-tile 256-token kernels (bf16 linear, gate/up).
const void* tc_lookup_pair(int epi)
{
    return epi == 0 ? reinterpret_cast<const void*>(&tc_dense_kernel<256, 0, true>)
                    : reinterpret_cast<const void*>(&tc_dense_kernel<256, 1, true>);
}

// The A4W4 kernels.
template <int EPI>
const void* tc_lookup_a4(int mp)
{
    switch (mp) {
    case 16: return tc_fn<16, EPI>();
    case 32: return tc_fn<32, EPI>();
    case 64: return tc_fn<64, EPI>();
    case 128: return tc_fn<128, EPI>();
    default: return nullptr;
    }
}

size_t stage_bytes_pair() { return 2 * static_cast<size_t>(kWBox) + static_cast<size_t>(256) * kKB * 2; }

// Paired 256-token tiles: 3 stages of 64 KB (the epilogue stages a 128 KB tile in them).
constexpr int kPairStages = 3;
size_t smem_bytes_pair(int stages) { return 1024 + stages * stage_bytes_pair() + (2 * stages + 2) * 8 + 16; }

size_t stage_bytes(int mp) { return kWBox + static_cast<size_t>(mp) * kKB * 2; }

// Bytes of the push fold's receive buffer (0 when the tile is not split).
int slice_max(int ns) { return ((kTileRows / 4 + ns - 1) / ns) * 4; }

size_t recv_bytes(int ns, int mq) { return ns > 1 ? static_cast<size_t>(ns) * slice_max(ns) * mq * 4 : 0; }

size_t smem_bytes(int mp, int stages, size_t recv)
{
    return 1024 + stages * stage_bytes(mp) + (2 * stages + 2) * 8 + 16 + recv;
}

// Two CTAs per SM (about 113 KB each) let the next launch's prologue and first
// weight boxes overlap this launch's tail: as many stages as fit that budget
// beside the receive buffer, at most 5.
int default_stages(int mp, size_t recv)
{
    int s = 5;
    while (s > 2 && smem_bytes(mp, s, recv) > kCoResidentSmem) --s;
    return s;
}

}  // namespace

int tc_mp(int M) { return M <= 16 ? 16 : (M <= 32 ? 32 : (M <= 64 ? 64 : (M <= 128 ? 128 : 256))); }

namespace {

// Never launched: stands in for a tensor-core CTA (same block, same dynamic shared
// memory) in the cluster-residency query below.  For the tcgen05 kernels themselves
// the driver's occupancy answer is one CTA per SM at any shared memory size, yet
// their launches hold two per SM at up to 112 KB each (timed on GB300: a K-split
// pays a second wave only once its clusters outnumber the two-per-SM capacity).
__global__ void __launch_bounds__(kThreads, 1) cluster_slot_kernel() {}

// Clusters of `size` tensor-core CTAs that are resident at once with two CTAs per SM
// (up to 128 tokens) or one (256-token tiles).  A cluster's CTAs share one GPC, so
// where the GPCs do not divide evenly this is below SMs x CTAs-per-SM / size: on
// GB300 (152 SMs), one CTA per SM holds 15 clusters of 8, 23 of 6 and 46 of 3.
int cluster_capacity(const DeviceInfo* dev, bool two_per_sm, int size)
{
    static std::mutex mu;
    static int cap[64][2][kMaxCluster + 1];
    static bool attr_set[64] = {};
    const int fallback = (two_per_sm ? 2 : 1) * dev->sm_count / size;
    if (size < 1 || size > kMaxCluster || dev->device < 0 || dev->device >= 64) return fallback;
    std::lock_guard<std::mutex> lk(mu);
    int& c = cap[dev->device][two_per_sm ? 1 : 0][size];
    if (c == 0) {
        const void* fn = reinterpret_cast<const void*>(&cluster_slot_kernel);
        if (!attr_set[dev->device]) {        // the current device is dev->device
            cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxDynSmem));
            attr_set[dev->device] = true;
        }
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(size * dev->sm_count));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = two_per_sm ? kCoResidentSmem : smem_bytes(256, kWideStages, 0);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(size);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        c = n > 0 ? n : fallback;
    }
    return c;
}

}  // namespace

void tc_capacity_init(const DeviceInfo* dev)
{
    for (int size = 1; size <= kMaxCluster; ++size) {
        cluster_capacity(dev, true, size);
        cluster_capacity(dev, false, size);
    }
}

int tc_nsplit(const DeviceInfo* dev, int N, int K, int M, bool fixed)
{
    const int tiles = (N + kTileRows - 1) / kTileRows;
    const int nkb = (K + kKB - 1) / kKB;
    // Up to 128 tokens two CTAs share an SM: the split fills both slots of every SM
    // (measured on GB300 6-11 % faster than about 160 CTAs on the 64-100 MB shapes,
    // where a few doubled-up SMs set the pace).  256-token tiles take one SM each.  A
    // fixed split plans for two CTAs per SM at every row count, so a row's bits do not
    // depend on how many rows share the call.
    const bool two = fixed || tc_mp(M) <= 128;
    int ns = (two ? 2 : 1) * dev->sm_count / tiles;
    if (ns > kMaxCluster) ns = kMaxCluster;
    // At least 4 K-blocks (256 elements) per rank: with less the fold costs more than
    // the streaming it shares (K = 1024 at 128 tokens: 4 ranks 8-18 % faster than 8).
    if (ns > nkb / 4) ns = nkb / 4;
    // One wave: every cluster resident at once.  A split one rank too wide for the
    // GPCs runs a second wave of clusters (2048x4096 at 256 tokens: 8 ranks 26.9 us,
    // 6 ranks 15.7 us).
    while (ns > 1 && tiles > cluster_capacity(dev, two, ns)) --ns;
    // 256-token tiles: a 2-rank fold of a 128 KB partial costs more than halving a
    // rank's stream of at most 32 K-blocks (8192x1024: 16.6 us split, 13.4 us whole).
    if (!two && ns == 2 && nkb <= 32) ns = 1;
    if (ns < 1) ns = 1;
    return ns;
}

// The K-split folds stay on chip, so only the status word is needed.
size_t tc_workspace_bytes(int M, int N, int K)
{
    (void)M;
    (void)N;
    (void)K;
    return kWsData;
}

dg_status launch_tc(bool gate_up, const DeviceInfo* dev, const dg_choice& c, const void* x, const void* W,
                    void* out, int M, int N, int K, int ld_out, void* ws, size_t ws_bytes, cudaStream_t stream)
{
    if (M < 1 || M > kMaxDenseRows) return DG_ERR_UNSUPPORTED_SHAPE;
    if (M > 256) {
        // Mid-M: chunks of 256 token rows (the MMA's widest N), one launch each; the
        // weights stream once per chunk.
        for (int t0 = 0; t0 < M; t0 += 256) {
            const int mc = M - t0 < 256 ? M - t0 : 256;
            const dg_status st = launch_tc(gate_up, dev, c, static_cast<const uint16_t*>(x) + static_cast<size_t>(t0) * K,
                                           W, static_cast<uint16_t*>(out) + static_cast<size_t>(t0) * ld_out, mc, N, K,
                                           ld_out, ws, ws_bytes, stream);
            if (st != DG_OK) return st;
        }
        return DG_OK;
    }
    const int mp = tc_mp(M);
    const int epi = gate_up ? 1 : 0;
    if (c.params[1] != 0 && c.params[1] != 1) return DG_ERR_BAD_VARIANT;
    const int ns = tc_nsplit(dev, N, K, M, c.params[1] == 1);
    const int tiles = (N + kTileRows - 1) / kTileRows;
    // 256-token tiles without a K-split and more tiles than SMs: two tiles per CTA, one
    // wave (the same MMA chains, so the same bits).
    const bool pair = mp == 256 && ns == 1 && tiles > dev->sm_count;
    const void* fn = pair ? tc_lookup_pair(epi) : tc_lookup(mp, epi);
    if (!fn) return DG_ERR_BAD_VARIANT;
    if (pair) {
        const int st = c.params[0] > 0 ? c.params[0] : kPairStages;
        const size_t smem = smem_bytes_pair(st);
        if (st < 2 || st > 8 || smem > kMaxDynSmem) return DG_ERR_BAD_VARIANT;
        if (ws_bytes < tc_workspace_bytes(M, N, K)) return DG_ERR_WORKSPACE_TOO_SMALL;
        TcArgs a{};
        a.N = N;
        a.K = K;
        a.M = M;
        a.tiles = tiles;
        a.nkb = (K + kKB - 1) / kKB;
        a.nsplit = 1;
        a.mq = (M + 3) & ~3;
        a.slice_max = slice_max(1);
        a.stages = st;
        a.out = static_cast<uint16_t*>(out);
        a.ld_out = ld_out;
        a.ws = static_cast<uint8_t*>(ws);
        CUtensorMap tmW, tmX;
        if (!encode_2d(&tmW, W, static_cast<uint64_t>(K), static_cast<uint64_t>(N), kKB, kTileRows) ||
            !encode_2d(&tmX, x, static_cast<uint64_t>(K), static_cast<uint64_t>(M), kKB, 256u))
            return DG_ERR_CUDA;
        if (occupancy(fn, kThreads, smem) < 1) return DG_ERR_UNSUPPORTED_SHAPE;
        void* args[] = {&tmW, &tmX, &a};
        if (launch_kernel(fn, static_cast<unsigned>((tiles + 1) / 2), kThreads, smem, stream, args) != cudaSuccess) {
            cudaGetLastError();
            return DG_ERR_CUDA;
        }
        return DG_OK;
    }
    const int mq = (M + 3) & ~3;
    // K-split fold: ranks push their rows to the folding rank (st.async) for up to 8
    // tokens when the receive buffer costs no pipeline stage; otherwise each rank
    // pulls the others' partials after a cluster barrier (measured on GB300: the
    // push is faster for few tokens, equal or slower beyond).  Same bits either way.
    size_t recv = mq <= kPushMaxTokens ? recv_bytes(ns, mq) : 0;
    int stages = c.params[0] > 0 ? c.params[0] : (mp <= 128 ? default_stages(mp, 0) : kWideStages);
    if (stages < 2 || stages > 8) return DG_ERR_BAD_VARIANT;
    // The epilogue stages the tile (or parks the K-split partial) in the ring.
    if (static_cast<size_t>(stages) * stage_bytes(mp) < static_cast<size_t>(mp) * kTileRows * 4) return DG_ERR_BAD_VARIANT;
    if (recv > 0 && smem_bytes(mp, stages, recv) > (c.params[0] > 0 ? kMaxDynSmem : kCoResidentSmem)) recv = 0;
    const size_t smem = smem_bytes(mp, stages, recv);
    if (smem > kMaxDynSmem) return DG_ERR_BAD_VARIANT;
    if (ws_bytes < tc_workspace_bytes(M, N, K)) return DG_ERR_WORKSPACE_TOO_SMALL;
    TcArgs a{};
    a.N = N;
    a.K = K;
    a.M = M;
    a.tiles = (N + kTileRows - 1) / kTileRows;
    a.nkb = (K + kKB - 1) / kKB;
    a.nsplit = ns;
    a.push = recv > 0 ? 1 : 0;
    a.mq = mq;
    a.slice_max = slice_max(ns);
    const size_t part_bytes = static_cast<size_t>(mp) * kTileRows * 4;
    if (ns > 1 && !a.push && part_bytes > static_cast<size_t>(stages) * stage_bytes(mp)) return DG_ERR_BAD_VARIANT;
    a.stages = stages;
    a.out = static_cast<uint16_t*>(out);
    a.ld_out = ld_out;
    a.ws = static_cast<uint8_t*>(ws);
    CUtensorMap tmW, tmX;
    if (!encode_2d(&tmW, W, static_cast<uint64_t>(K), static_cast<uint64_t>(N), kKB, kTileRows) ||
        !encode_2d(&tmX, x, static_cast<uint64_t>(K), static_cast<uint64_t>(M), kKB, static_cast<uint32_t>(mp)))
        return DG_ERR_CUDA;
    if (occupancy(fn, kThreads, smem) < 1) return DG_ERR_UNSUPPORTED_SHAPE;
    void* args[] = {&tmW, &tmX, &a};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.tiles * a.nsplit));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(a.nsplit);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    if (launch_ordered(cfg, attr, 1, fn, args, Early::kWeights) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

}  // namespace dg

namespace dg {

// ------------------------------------------------------------------ A8W8 blockscale

int tc_a8_nsplit(const DeviceInfo* dev, int N, int K)
{
    const int tiles = (N + kTileRows - 1) / kTileRows;
    const int nkb = (K + kA8Block - 1) / kA8Block;
    // Both CTA slots of every SM, in one wave of clusters, and at most 8 K-blocks of
    // quantised activations per rank (64 KB at 64 tokens); a function of the shape
    // alone, so a row's bits do not depend on how many rows share the call.
    int ns = 2 * dev->sm_count / tiles;
    if (ns > kMaxCluster) ns = kMaxCluster;
    while (ns > 1 && tiles > cluster_capacity(dev, true, ns)) --ns;
    const int by_smem = (nkb + 7) / 8;
    if (ns < by_smem) ns = by_smem;
    if (ns > kMaxCluster) ns = kMaxCluster;
    if (ns > nkb) ns = nkb;
    if (ns < 1) ns = 1;
    return ns;
}

namespace {

size_t smem_bytes_a8(int mp, int stages, size_t recv, int xq_blocks)
{
    return 1024 + static_cast<size_t>(stages) * kWBox + a8_extra_bytes(xq_blocks, mp) +
           (2 * stages + 2 + kA8Bars) * 8 + 16 + recv;
}

}  // namespace

size_t a8_workspace_bytes(int M, int K)
{
    const size_t nb = static_cast<size_t>((K + kA8Block - 1) / kA8Block);
    const size_t q = (static_cast<size_t>(M) * K + 255) / 256 * 256;
    return kWsData + q + (static_cast<size_t>(M) * nb * 4 + 255) / 256 * 256;
}

dg_status launch_tc_a8(const DeviceInfo* dev, const dg_choice& c, const void* x, const void* Wq, const float* sw,
                       void* y, int M, int N, int K, void* ws, size_t ws_bytes, cudaStream_t stream)
{
    (void)dev;
    if (M < 1 || M > kA8MaxRows || K % 16 != 0) return DG_ERR_UNSUPPORTED_SHAPE;
    if (c.params[1] != 0 && c.params[1] != 1) return DG_ERR_BAD_VARIANT;
    for (int i = 2; i < 6; ++i)
        if (c.params[i] != 0) return DG_ERR_BAD_VARIANT;
    // params[1] = 1: quantise in a launch of its own into the workspace, then stream the
    // codes by TMA (the same codes, scales and fold: the same bits).
    const bool preq = c.params[1] == 1;
    const int mp = tc_mp(M);
    const void* fn = tc_lookup(mp, 2);
    if (!fn) return DG_ERR_BAD_VARIANT;
    const int ns = tc_a8_nsplit(dev, N, K);
    const int nkb = (K + kA8Block - 1) / kA8Block;
    const int xq_blocks = (nkb + ns - 1) / ns;
    if (xq_blocks > kA8MaxBlocks) return DG_ERR_UNSUPPORTED_SHAPE;
    const int mq = (M + 3) & ~3;
    size_t recv = mq <= kPushMaxTokens ? recv_bytes(ns, mq) : 0;
    // Two CTAs per SM when at least two stages fit beside the activations, else one
    // CTA per SM with a deeper ring.
    int stages = c.params[0];
    if (stages == 0) {
        stages = 5;
        while (stages > 2 && smem_bytes_a8(mp, stages, recv, xq_blocks) > kCoResidentSmem) --stages;
        if (smem_bytes_a8(mp, stages, recv, xq_blocks) > kCoResidentSmem) {
            stages = 8;
            while (stages > 2 && smem_bytes_a8(mp, stages, recv, xq_blocks) > kMaxDynSmem) --stages;
        }
    }
    if (stages < 2 || stages > 8) return DG_ERR_BAD_VARIANT;
    // The epilogue stages the tile (or parks the K-split partial) in the ring.
    const size_t part_bytes = static_cast<size_t>(mp) * kTileRows * 4;
    if (static_cast<size_t>(stages) * kWBox < part_bytes) return DG_ERR_BAD_VARIANT;
    if (recv > 0 && smem_bytes_a8(mp, stages, recv, xq_blocks) > kMaxDynSmem) recv = 0;
    size_t smem = smem_bytes_a8(mp, stages, recv, xq_blocks);
    if (smem > kMaxDynSmem) return DG_ERR_UNSUPPORTED_SHAPE;
    // Never more co-resident CTAs than their TMEM columns (4 x MP each) fit in the SM's
    // 512: a CTA waiting in tcgen05.alloc while its cluster peers wait for it would hang.
    const size_t per_sm = 228 * 1024;
    const size_t min_smem = per_sm / (512 / (kA8Bufs * mp) + 1) + 1024;
    if (smem < min_smem) smem = min_smem;
    if (ws_bytes < (preq ? a8_workspace_bytes(M, K) : kWsData)) return DG_ERR_WORKSPACE_TOO_SMALL;
    uint8_t* qws = static_cast<uint8_t*>(ws) + kWsData;
    float* sxws = reinterpret_cast<float*>(qws + (static_cast<size_t>(M) * K + 255) / 256 * 256);
    TcArgs a{};
    a.N = N;
    a.K = K;
    a.M = M;
    a.tiles = (N + kTileRows - 1) / kTileRows;
    a.nkb = nkb;
    a.nsplit = ns;
    a.push = recv > 0 ? 1 : 0;
    a.mq = mq;
    a.slice_max = slice_max(ns);
    a.stages = stages;
    a.out = static_cast<uint16_t*>(y);
    a.ld_out = N;
    a.ws = static_cast<uint8_t*>(ws);
    a.x = static_cast<const uint16_t*>(x);
    a.sw = sw;
    a.kbs = nkb;
    a.xq_blocks = xq_blocks;
    a.preq = preq ? 1 : 0;
    a.sxg = sxws;
    CUtensorMap tmW, tmQ;
    if (!encode_2d(&tmW, Wq, static_cast<uint64_t>(K), static_cast<uint64_t>(N), kA8Block, kTileRows, true))
        return DG_ERR_CUDA;
    if (preq && !encode_2d(&tmQ, qws, static_cast<uint64_t>(K), static_cast<uint64_t>(M), kA8Block,
                           static_cast<uint32_t>(mp), true))
        return DG_ERR_CUDA;
    if (occupancy(fn, kThreads, smem) < 1) return DG_ERR_UNSUPPORTED_SHAPE;
    if (preq) {
        const dg_status st = launch_a8_quant(x, qws, sxws, M, K, stream);
        if (st != DG_OK) return st;
    }
    void* args[] = {&tmW, preq ? &tmQ : &tmW, &a};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.tiles * a.nsplit));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(a.nsplit);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    if (launch_ordered(cfg, attr, 1, fn, args, Early::kWeights) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

// ------------------------------------------------------------------ A4W4 blockscale

// How a call is cut: token groups of up to tg rows (the MMA's N) and ns K ranges.
struct A4Plan {
    int tg, ns;
};

// The cheapest cut by a model of what a CTA does, in units of about 10 ns, fitted on GB300 to
// graphs of calls of 1 to 512 rows over 16 weight shapes (44 cases: the one it takes is within
// 0.4 % of the best on average, 8 % at worst): 33 a K-block of 256 elements; kEnd the epilogue
// of a group; with a K-split the fold, kFold + kFoldRank per rank (partials through distributed
// shared memory at about 25 GB/s a CTA).  The constants are of calls as a whole and an earlier
// loop: measured alone, today's K-blocks take 25 to 56 by format and token group (at the top of
// this file), which the model does not tell apart.
// One wave: at most 263 of the 304 CTA slots -- fuller grids leave no room for the next
// launch's CTAs to start under this one's tail (12288 x 4096 at 16 rows: 192 CTAs 7.3 us, 288
// 8.6).  Few rows take few, small groups and a K-split; many rows split tokens instead, and
// the tile's weights come from L2 to each group (128 x 4096 x 4096: one group of 128 and 4
// ranks 11.9 us, 4 groups of 32 and 2 ranks 9.0).
static A4Plan a4_plan(const DeviceInfo* dev, int N, int K, int M, bool fixed)
{
    constexpr int kTg[4] = {16, 32, 64, 128};
    constexpr int kEnd[4] = {0, 20, 180, 260}, kFold[4] = {80, 120, 160, 320}, kFoldRank[4] = {24, 17, 25, 23};
    const int tiles = (N + kTileRows - 1) / kTileRows;
    const int nkb = (K + kA4Block - 1) / kA4Block;
    const long long slots = 2 * dev->sm_count * 13 / 15;
    // the fixed rule: the K ranges that one row would take
    const int ns_fixed = fixed && M > 1 ? a4_plan(dev, N, K, 1, false).ns : 0;
    A4Plan best{128, 1};
    long long best_cost = -1;
    for (int g = 0; g < 4; ++g) {
        const int tg = kTg[g];
        if ((tg == 16 && M > 16) || (tg > 16 && tg / 2 >= M)) continue;
        for (int ns = 1; ns <= kMaxCluster && ns <= nkb; ++ns) {
            if (ns_fixed && ns != ns_fixed) continue;
            const long long ctas = static_cast<long long>(tiles) * ((M + tg - 1) / tg) * ns;
            if (ns > 1 && !ns_fixed && (ctas > slots || ctas / ns > cluster_capacity(dev, true, ns))) continue;
            const long long waves = (ctas + slots - 1) / slots;
            const long long cost = waves * 33 * ((nkb + ns - 1) / ns) + kEnd[g] + (ns > 1 ? kFold[g] + kFoldRank[g] * ns : 0);
            if (best_cost < 0 || cost < best_cost) {
                best_cost = cost;
                best = A4Plan{tg, ns};
            }
        }
    }
    return best;
}

size_t a4_workspace_bytes(int M, int K)
{
    const size_t q = (static_cast<size_t>(M) * K / 2 + 255) / 256 * 256;
    // the wider of the two formats' scales, a tile row for each 32 tokens (the smallest group)
    return kWsData + q +
           static_cast<size_t>(M / 32 + (M % 32 != 0)) * fp4::scale_tiles(K, true) * fp4::kTileBytes;
}

namespace {

// One K-block of activations: codes and scale tiles.
size_t xblock_bytes_a4(int mp, bool nv)
{
    return static_cast<size_t>(mp) * 128 + static_cast<size_t>(a4_scale_box(nv));
}

// xq_blocks: K-blocks of activations kept beside the ring (0: they come with each stage).
size_t stage_bytes_a4(int mp, bool nv, int xq_blocks)
{
    return kWBox + static_cast<size_t>(a4_scale_box(nv)) + (xq_blocks ? 0 : xblock_bytes_a4(mp, nv));
}

size_t smem_bytes_a4(int mp, bool nv, int stages, size_t recv, int xq_blocks)
{
    return 1024 + stages * stage_bytes_a4(mp, nv, xq_blocks) + xq_blocks * xblock_bytes_a4(mp, nv) +
           (2 * stages + 2 + kA4Bars) * 8 + 16 + recv;
}

// The linear's own CTAs quantise the activations where a rank has at most this many
// (row, K-block) pieces: every row tile repeats the work, against a launch of its own (4096 x
// 4096, us fused / apart: 1 row 4.7 / 5.8, 4 rows 5.7 / 5.7, 8 rows 7.6 / 6.3, 16 rows 10.3 /
// 6.1; 12288 x 4096, twice the K-blocks a rank: 1 row 6.9 / 7.7, 4 rows 9.2 / 7.8).
constexpr int kA4FusePieces = 16;

}  // namespace

dg_status launch_tc_a4(const DeviceInfo* dev, const dg_choice& c, bool nv, const void* x, const void* Wq,
                       const void* sw, const float* gx, const float* gw, void* y, int M, int N, int K, void* ws,
                       size_t ws_bytes, cudaStream_t stream)
{
    if (M < 1 || M > kMaxDenseRows || K % 32 != 0) return DG_ERR_UNSUPPORTED_SHAPE;
    if (c.params[1] != 0 && c.params[1] != 1) return DG_ERR_BAD_VARIANT;
    for (int i = 2; i < 6; ++i)
        if (c.params[i] != 0) return DG_ERR_BAD_VARIANT;
    if (ws_bytes < a4_workspace_bytes(M, K)) return DG_ERR_WORKSPACE_TOO_SMALL;
    const A4Plan plan = a4_plan(dev, N, K, M, c.params[1] == 1);
    const int mp = plan.tg, ns = plan.ns, groups = (M + mp - 1) / mp;
    const void* fn = nv ? tc_lookup_a4<4>(mp) : tc_lookup_a4<3>(mp);
    if (!fn) return DG_ERR_BAD_VARIANT;
    const int nkb = (K + kA4Block - 1) / kA4Block;
    const bool fuse = static_cast<long long>(M) * ((nkb + ns - 1) / ns) <= kA4FusePieces;
    const int mq = (M + 3) & ~3;
    const int xq = fuse ? (nkb + ns - 1) / ns : 0;
    const size_t recv = mq <= kPushMaxTokens ? recv_bytes(ns, mq) : 0;
    int stages = c.params[0];
    if (stages == 0) {
        stages = 5;
        while (stages > 2 && smem_bytes_a4(mp, nv, stages, recv, xq) > kCoResidentSmem) --stages;
    } else if (c.from_table) {
        // A pick holds for both formats, every row count of its bucket and both K-split rules, whose
        // stages differ in size: as deep as this call's fit (depth changes no bits).
        while (stages > 2 && smem_bytes_a4(mp, nv, stages, recv, xq) > kMaxDynSmem) --stages;
    }
    if (stages < 2 || stages > 8) return DG_ERR_BAD_VARIANT;
    // A K-split parks its partial tile in the ring.
    if (ns > 1 && !recv && stages * stage_bytes_a4(mp, nv, xq) < static_cast<size_t>(mp) * kTileRows * 4)
        return DG_ERR_BAD_VARIANT;
    size_t smem = smem_bytes_a4(mp, nv, stages, recv, xq);
    if (smem > kMaxDynSmem) return DG_ERR_BAD_VARIANT;
    // Never more co-resident CTAs than their TMEM columns fit in the SM's 512.
    const size_t cols = mp <= 64 ? 128 : 256;
    const size_t min_smem = 228 * 1024 / (512 / cols + 1) + 1024;
    if (smem < min_smem) smem = min_smem;
    if (occupancy(fn, kThreads, smem) < 1) return DG_ERR_UNSUPPORTED_SHAPE;
    uint8_t* qws = static_cast<uint8_t*>(ws) + kWsData;
    uint8_t* sws = qws + (static_cast<size_t>(M) * K / 2 + 255) / 256 * 256;
    TcArgs a{};
    a.N = N;
    a.K = K;
    a.M = M;
    a.tiles = (N + kTileRows - 1) / kTileRows;
    a.nkb = nkb;
    a.nsplit = ns;
    a.push = recv > 0 ? 1 : 0;
    a.mq = mq;
    a.slice_max = slice_max(ns);
    a.stages = stages;
    a.out = static_cast<uint16_t*>(y);
    a.ld_out = N;
    a.ws = static_cast<uint8_t*>(ws);
    a.x = static_cast<const uint16_t*>(x);
    a.preq = fuse ? 0 : 1;
    a.xq_blocks = xq;
    a.nkt = fp4::scale_tiles(K, nv);
    a.sfw = static_cast<const uint8_t*>(sw);
    a.sfx = sws;
    a.groups = groups;
    a.tg = mp;
    a.gx = gx;
    a.gw = gw;
    CUtensorMap tmW, tmX;
    const uint64_t kb = static_cast<uint64_t>(K) / 2;
    if (!encode_2d(&tmW, Wq, kb, static_cast<uint64_t>(N), 128, kTileRows, true)) return DG_ERR_CUDA;
    if (fuse)
        tmX = tmW;                                   // (not read)
    else if (!encode_2d(&tmX, qws, kb, static_cast<uint64_t>(M), 128, static_cast<uint32_t>(mp), true))
        return DG_ERR_CUDA;
    if (!fuse) {
        const dg_status st = launch_fp4_quant(nv, x, qws, sws, gx, M, K, mp, true, stream);
        if (st != DG_OK) return st;
    }
    void* args[] = {&tmW, &tmX, &a};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.tiles * groups * ns));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ns);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    if (launch_ordered(cfg, attr, 1, fn, args, Early::kWeights) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

}  // namespace dg
