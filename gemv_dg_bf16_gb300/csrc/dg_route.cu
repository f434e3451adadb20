// dg_route.cu -- routing of tokens to experts (dg_moe_route).
//
// One warp per token; lane l holds experts j * 32 + l in registers.  The pick compares
// scores (plus the bias) in binary32, so that it is defined to the last bit: sigmoid as
// 1 / (1 + expf(-x)), softmax as expf(x - max) / sum with the sum compensated
// (Knuth's two-sum), which rounds it as the exact sum in all but about 2^-20 of cases
// whatever the order -- the same pick for any arrangement of lanes.
// Bound: latency of topk dependent warp reductions; memory (2 or 4 bytes a logit) is small.
#include "dg_common.cuh"
#include "dg_internal.h"

namespace dg {
namespace {

constexpr int kWarps = 4;

// Total order of floats as unsigned (no NaN, no -0 among scores); -inf is kNone.
__device__ __forceinline__ uint32_t order_key(float f)
{
    const uint32_t b = __float_as_uint(f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
constexpr uint32_t kNone = 0x007fffffu;

// s + e += v, exactly up to the rounding of e.
__device__ __forceinline__ void two_sum(float& s, float& e, float v)
{
    const float t = __fadd_rn(s, v);
    const float z = __fsub_rn(t, s);
    e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(v, z)));
    s = t;
}

struct RouteArgs {
    const void* logits;
    const float* bias;
    int32_t* ids;
    float* w;
    long long ld;
    int M, E;
    int topk, n_group, topk_group, group_top, gsize;
    int sigmoid, renorm;
    float scale;
};

template <bool F32>
__device__ __forceinline__ float load_logit(const RouteArgs& a, long long row, int i)
{
    const long long o = row * a.ld + i;
    if constexpr (F32) return static_cast<const float*>(a.logits)[o];
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(a.logits)[o]) << 16);
}

template <int R, bool F32>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(RouteArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (row >= a.M) return;
    float x[R];
    uint32_t key[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const int i = j * 32 + lane;
        x[j] = i < a.E ? load_logit<F32>(a, row, i) : -INFINITY;
        if (!(x[j] > -INFINITY)) x[j] = -INFINITY;                 // NaN: not available
    }
    float m = 0.0f, sum = 1.0f;
    if (!a.sigmoid) {
        float lm = x[0];
#pragma unroll
        for (int j = 1; j < R; ++j) lm = fmaxf(lm, x[j]);
#pragma unroll
        for (int o = 16; o; o >>= 1) lm = fmaxf(lm, __shfl_xor_sync(kFull, lm, o));
        m = lm;
        float s = 0.0f, e = 0.0f;
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (x[j] > -INFINITY) two_sum(s, e, x[j] == m ? 1.0f : expf(x[j] - m));
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float s2 = __shfl_xor_sync(kFull, s, o), e2 = __shfl_xor_sync(kFull, e, o);
            two_sum(s, e, s2);
            e = __fadd_rn(e, e2);
        }
        sum = __fadd_rn(s, e);
    }
    auto score = [&](float v) {
        if (a.sigmoid) return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-v)));
        return __fdiv_rn(v == m ? 1.0f : expf(v - m), sum);
    };
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const int i = j * 32 + lane;
        key[j] = kNone;
        if (x[j] > -INFINITY) {
            float k = score(x[j]);
            if (a.bias) k = __fadd_rn(k, a.bias[i]);
            if (k > -INFINITY) key[j] = order_key(k);
        }
    }
    if (a.n_group > 1) {
        float gs = -INFINITY;                                      // lane g: the score of group g
        for (int g = 0; g < a.n_group; ++g) {
            uint32_t a1 = kNone, a2 = kNone;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const int i = j * 32 + lane;
                if (i >= g * a.gsize && i < (g + 1) * a.gsize) {
                    a2 = max(a2, min(a1, key[j]));
                    a1 = max(a1, key[j]);
                }
            }
            const uint32_t t1 = __reduce_max_sync(kFull, a1);
            const unsigned own = __ballot_sync(kFull, a1 == t1);
            const uint32_t t2 = __reduce_max_sync(kFull, lane == __ffs(own) - 1 ? a2 : a1);
            const float f1 = __uint_as_float((t1 & 0x80000000u) ? t1 ^ 0x80000000u : ~t1);
            const float f2 = __uint_as_float((t2 & 0x80000000u) ? t2 ^ 0x80000000u : ~t2);
            const float v = t1 == kNone ? -INFINITY : (a.group_top == 2 && t2 != kNone ? __fadd_rn(f1, f2) : f1);
            if (lane == g) gs = v;
        }
        int rank = 0;
        for (int g = 0; g < a.n_group; ++g) {
            const float o = __shfl_sync(kFull, gs, g);
            rank += (o > gs || (o == gs && g < lane)) ? 1 : 0;
        }
        const unsigned keep = __ballot_sync(kFull, lane < a.n_group && rank < a.topk_group);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int i = j * 32 + lane;
            if (i < a.E && !((keep >> (i / a.gsize)) & 1u)) key[j] = kNone;
        }
    }
    int id = -1;                                                   // lane k: slot k
    for (int k = 0; k < a.topk; ++k) {
        uint32_t best = kNone;
        int at = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (key[j] > best) {
                best = key[j];
                at = j * 32 + lane;
            }
        const uint32_t top = __reduce_max_sync(kFull, best);
        if (top == kNone) break;
        const int win = static_cast<int>(__reduce_min_sync(kFull, best == top ? static_cast<unsigned>(at) : 0x7fffffffu));
        if (lane == k) id = win;
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (j * 32 + lane == win) key[j] = kNone;
    }
    float wv = 0.0f;
    if (id >= 0) wv = score(load_logit<F32>(a, row, id));
    if (a.renorm) {
        float t = wv;
#pragma unroll
        for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(kFull, t, o);
        wv = t > 0.0f ? __fdiv_rn(wv, t) : 0.0f;
    }
    if (lane < a.topk) {
        a.ids[row * a.topk + lane] = id;
        a.w[row * a.topk + lane] = __fmul_rn(wv, a.scale);
    }
}

template <bool F32>
const void* route_fn(int E)
{
    const int r = (E + 31) / 32;
    if (r <= 1) return reinterpret_cast<const void*>(&route_kernel<1, F32>);
    if (r <= 2) return reinterpret_cast<const void*>(&route_kernel<2, F32>);
    if (r <= 4) return reinterpret_cast<const void*>(&route_kernel<4, F32>);
    if (r <= 8) return reinterpret_cast<const void*>(&route_kernel<8, F32>);
    if (r <= 16) return reinterpret_cast<const void*>(&route_kernel<16, F32>);
    return reinterpret_cast<const void*>(&route_kernel<32, F32>);
}

}  // namespace

dg_status launch_route(const dg_route_params& p, const void* logits, const float* bias, int32_t* ids, float* w,
                       int M, int E, long long ld, bool f32, cudaStream_t stream)
{
    RouteArgs a{};
    a.logits = logits;
    a.bias = bias;
    a.ids = ids;
    a.w = w;
    a.ld = ld;
    a.M = M;
    a.E = E;
    a.topk = p.topk;
    a.n_group = p.n_group;
    a.topk_group = p.topk_group;
    a.group_top = p.group_top;
    a.gsize = E / p.n_group;
    a.sigmoid = p.score == DG_SCORE_SIGMOID ? 1 : 0;
    a.renorm = p.renorm;
    a.scale = p.scale;
    const void* fn = f32 ? route_fn<true>(E) : route_fn<false>(E);
    void* args[] = {&a};
    const unsigned grid = static_cast<unsigned>((static_cast<long long>(M) + kWarps - 1) / kWarps);
    if (launch_kernel(fn, grid, kWarps * 32, 0, stream, args) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

}  // namespace dg
