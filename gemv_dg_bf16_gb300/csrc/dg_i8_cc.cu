// dg_i8_cc.cu -- the 8-bit integer linear for the fewest tokens (dg_gemv_i8_rowscale) on the CUDA cores: weights
// streamed through registers, dp4a, the activations quantised inside.
//
// dp4a does 250 multiply-adds a clock and SM (measured), as the warp-level integer MMA does; one token
// takes 23 at the rate that weights arrive, so that up to a few tokens nothing is converted.  A CTA owns a
// contiguous range of weight rows; the ks warps of a slot take every ks-th chunk of 512 elements of four rows,
// 16 a lane, and the tokens' codes at the same places serve all four (two: 4096 x 4096 4.97 us, four 4.45).  Sixteen
// loads are in flight a lane: at 4096 x 4096 all that a warp reads.  Lanes are added up by redux.sync and warps by
// shared-memory atomics, one sum for each row and token of the CTA: everything is an exact integer, so no order
// matters, and no barrier holds the stream up before the last one (with one a round of rows 12288 x 4096 took 13.1
// us).
// Measured, weights in turn from memory: 4096 x 4096 5.6 us for one token (from L2 4.5), 6.1 for two, 7.4 for four;
// 12288 x 4096 10.0 (5.0 TB/s), 10.7 and 13.0 (on tensor cores 13.8; for eight 14.2).  A launch, a first load and the
// tokens' quantisation bind the small ones.
// The first loads are on their way before the launch ahead has finished; then every CTA quantises the tokens
// for itself.
#include "dg_i8.cuh"
#include "dg_internal.h"

namespace dg {
namespace {

constexpr int kWarps = 16;
constexpr int kChunk = 512;                      // K elements of a batch, 16 a lane
constexpr int kRows = 4;                         // weight rows of a warp's batch of loads
constexpr int kBatches = 4;                      // batches in flight
constexpr int kHold = 4;                         // 16-byte pieces of a token a lane keeps while it is quantised
constexpr int kMaxTokens = 4;

struct CcArgs {
    const uint16_t* x;
    const uint8_t* W;
    const float* sw;
    uint16_t* y;
    int M, N, K;
    int ks, per_warp;                            // warps that share rows, chunks each of them has
    int stride;                                  // bytes of a token's codes in shared memory
};

// The tokens' codes in shared memory, zeros behind K: `share` warps a token (a power of two), a barrier
// between its maximum and its codes.
__device__ __forceinline__ void quantise(const uint16_t* x, uint8_t* q, float* s, uint32_t* part, int M, int K, int stride)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int share = kWarps;
    while (share > 1 && share * M > kWarps) share >>= 1;
    const int first = (warp % share) * 32 + lane, step = share * 32, nv = K / 8, t = warp / share;
    uint4 raw[kHold];
    uint32_t m = 0;
    const uint16_t* row = x + static_cast<size_t>(t) * K;
    if (t < M) {
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            raw[i] = make_uint4(0, 0, 0, 0);
            if (first + i * step < nv) raw[i] = ld_stream_after(row + 8 * (first + i * step));
        }
#pragma unroll
        for (int i = 0; i < kHold; ++i) m = __vmaxu2(m, i8::amax8(raw[i]));
#pragma unroll 4
        for (int v = first + kHold * step; v < nv; v += step) m = __vmaxu2(m, i8::amax8(ld_stream_after(row + 8 * v)));
    }
    m = __reduce_max_sync(kFull, max(m & 0xffffu, m >> 16));
    if (lane == 0) part[warp] = m;
    __syncthreads();
    if (t < M) {
        for (int i = 0; i < share; ++i) m = max(m, part[t * share + i]);
        const i8::RowScale o = i8::row_scale(m);
        uint8_t* dst = q + t * stride;
#pragma unroll
        for (int i = 0; i < kHold; ++i)
            if (first + i * step < nv) *reinterpret_cast<uint2*>(dst + 8 * (first + i * step)) = i8::codes8(raw[i], o);
#pragma unroll 4
        for (int v = first + kHold * step; v < nv; v += step)
            *reinterpret_cast<uint2*>(dst + 8 * v) = i8::codes8(ld_stream_after(row + 8 * v), o);
        for (int v = nv + first; v < stride / 8; v += step) *reinterpret_cast<uint2*>(dst + 8 * v) = make_uint2(0, 0);
        if (first == 0) s[t] = o.s;
    }
    __syncthreads();
}

template <int MT>
__global__ void __launch_bounds__(kWarps * 32, 1) i8_cc_kernel(CcArgs a)
{
    constexpr int R = kRows;
    extern __shared__ __align__(16) uint8_t sh[];
    uint8_t* xs = sh;                                                        // [M][stride] codes
    uint32_t* part = reinterpret_cast<uint32_t*>(xs + static_cast<size_t>(a.M) * a.stride);
    float* sx = reinterpret_cast<float*>(part + kWarps);                     // [kMaxTokens]
    int* sums = reinterpret_cast<int*>(sx + kMaxTokens);                     // [token][row of the CTA's range]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slots = kWarps / a.ks, slot = warp / a.ks, rank = warp - slot * a.ks;
    const int lo = static_cast<int>(static_cast<long long>(a.N) * blockIdx.x / gridDim.x);
    const int rows = static_cast<int>(static_cast<long long>(a.N) * (blockIdx.x + 1) / gridDim.x) - lo;
    const int groups = (rows + R - 1) / R, mine = (groups - slot + slots - 1) / slots;
    const int last = max(0, rows - R);                                       // where the last group's loads begin

    // Every load is made, from a place that is there (the last group's rows may begin in the one before, codes
    // past K meet zeros): behind a condition it would be waited for at once.
    int ld_row = slot * R, ld_i = 0;
    auto load_batch = [&](uint4 (&b)[R]) {
        const int k = min((rank + a.ks * ld_i) * kChunk + 16 * lane, a.K - 16);
        const uint8_t* p = a.W + static_cast<size_t>(lo + min(ld_row, last)) * a.K + k;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            b[r] = ld_stream(p);
            if (r + 1 < rows) p += a.K;
        }
        ++ld_i;
        const bool next = ld_i == a.per_warp;
        ld_i = next ? 0 : ld_i;
        ld_row = next ? min(ld_row + slots * R, rows) : ld_row;
    };
    uint4 buf[kBatches][R];
#pragma unroll
    for (int b = 0; b < kBatches; ++b) load_batch(buf[b]);
    for (int v = threadIdx.x; v < MT * rows; v += kWarps * 32) sums[v] = 0;
    pdl_launch_dependents();
    pdl_wait();
    quantise(a.x, xs, sx, part, a.M, a.K, a.stride);

    int acc[R][MT], i = 0, row0 = slot * R;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[r][t] = 0;
    auto batch = [&](const uint4 (&w)[R]) {
        const uint8_t* at = xs + (rank + a.ks * i) * kChunk + 16 * lane;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            // (tokens past M repeat the last; theirs are not stored)
            const uint4 x = *reinterpret_cast<const uint4*>(at + min(t, a.M - 1) * a.stride);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                int s = acc[r][t];
                s = __dp4a(static_cast<int>(w[r].x), static_cast<int>(x.x), s);
                s = __dp4a(static_cast<int>(w[r].y), static_cast<int>(x.y), s);
                s = __dp4a(static_cast<int>(w[r].z), static_cast<int>(x.z), s);
                acc[r][t] = __dp4a(static_cast<int>(w[r].w), static_cast<int>(x.w), s);
            }
        }
        if (++i < a.per_warp) return;
        // Lane r * MT + t adds the warp's sum of row r and token t to the CTA's.
        int v = 0;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int s = __reduce_add_sync(kFull, acc[r][t]);
                if (lane == r * MT + t) v = s;
                acc[r][t] = 0;
            }
        const int row = min(row0, last) + lane / MT;
        if (lane < R * MT && row >= row0 && row < rows) atomicAdd(sums + (lane % MT) * rows + row, v);
        i = 0;
        row0 += slots * R;
    };
    const int batches = mine * a.per_warp;
#pragma unroll 1
    for (int b0 = 0; b0 < batches; b0 += kBatches) {
#pragma unroll
        for (int b = 0; b < kBatches; ++b) {
            if (b0 + b < batches) batch(buf[b]);
            load_batch(buf[b]);
        }
    }
    __syncthreads();
    for (int v = threadIdx.x; v < a.M * rows; v += kWarps * 32) {
        const int t = v / rows, n = lo + v - t * rows;
        a.y[static_cast<size_t>(t) * a.N + n] = i8::output(sums[v], sx[t], a.sw[n]);
    }
}

// Warps that share rows and the chunks each has: as many warps as there are chunks, up to 8.
int shared_warps(int K)
{
    const int chunks = (K - 1) / kChunk + 1;
    int ks = 8;
    while (ks > chunks) ks >>= 1;
    return ks;
}

int code_stride(int K)
{
    const int span = shared_warps(K) * kChunk;
    return (K - 1) / span * span + span;
}

// Bytes for the tokens' codes and scales; what is left of a CTA's shared memory holds its sums.
size_t token_bytes(int M, int K) { return static_cast<size_t>(M) * code_stride(K) + kWarps * 4 + kMaxTokens * 4; }

}  // namespace

// Whether a call has room: at most 4 tokens, and their codes beside the sums of 256 rows.
bool i8_cc_takes(int M, int K) { return M <= kMaxTokens && token_bytes(M, K) + kMaxTokens * 256 * 4 <= kMaxDynSmem; }

dg_status launch_i8_cc(const DeviceInfo* dev, const dg_choice& c, const void* x, const void* Wq, const float* sw, void* y, int M, int N,
                       int K, cudaStream_t stream)
{
    for (int i = 0; i < 6; ++i)
        if (c.params[i] != 0) return DG_ERR_BAD_VARIANT;
    if (!i8_cc_takes(M, K)) return DG_ERR_UNSUPPORTED_SHAPE;
    const int mt = M <= 2 ? M : 4;
    // One CTA a SM, or as many more as their sums need.
    const long long most = static_cast<long long>((kMaxDynSmem - token_bytes(M, K)) / (static_cast<size_t>(mt) * 4)) - 1;
    long long grid = N < dev->sm_count ? N : dev->sm_count;
    if ((N + grid - 1) / grid > most) grid = (N + most - 1) / most;
    const size_t smem = token_bytes(M, K) + static_cast<size_t>((N + grid - 1) / grid) * mt * 4;
    const void* fn = mt == 1   ? reinterpret_cast<const void*>(&i8_cc_kernel<1>)
                     : mt == 2 ? reinterpret_cast<const void*>(&i8_cc_kernel<2>)
                               : reinterpret_cast<const void*>(&i8_cc_kernel<4>);
    if (occupancy(fn, kWarps * 32, smem) < 1) return DG_ERR_UNSUPPORTED_SHAPE;
    CcArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.W = static_cast<const uint8_t*>(Wq);
    a.sw = sw;
    a.y = static_cast<uint16_t*>(y);
    a.M = M;
    a.N = N;
    a.K = K;
    a.ks = shared_warps(K);
    a.stride = code_stride(K);
    a.per_warp = a.stride / (a.ks * kChunk);
    void* args[] = {&a};
    if (launch_kernel(fn, static_cast<unsigned>(grid), kWarps * 32, smem, stream, args) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

}  // namespace dg
