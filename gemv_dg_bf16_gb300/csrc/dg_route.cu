// dg_route.cu -- routing of tokens to experts (dg_moe_route).
//
// One warp per token at a time; lane l holds the R consecutive experts l R .. l R + R - 1 in
// registers, so a lower lane is a lower index and a group of experts is a run of lanes.  The
// pick compares scores (plus the bias) in binary32, so that it is defined to the last bit:
// sigmoid as 1 / (1 + expf(-x)), softmax as expf(x - max) / sum with the sum compensated
// (Knuth's two-sum), which rounds it as the exact sum whatever the order, the exact sum's own
// ties included; only a sum within about 2^-43 of a tie from below may go up instead.
//
// Up to 8 experts a lane, each lane sorts its keys (a network of maxima and minima), and a pick
// is one warp maximum over the lanes' heads, a ballot for the lowest lane that holds it, and a
// shift in that lane; which expert each pick was is looked up at the end for all slots at
// once.  A group's best one or two are the heads of its lanes, merged by shuffles.  Warps walk
// over the tokens with the next token's logits already on the way and the bias in registers.
// Bound: instructions, 736 a token of 256 experts with 8 groups and 8 picks (28 of them a pick)
// where memory would be 1 KB a token: 32768 tokens take 29 us at 68 % of the issue slots, 5 us
// of bytes.  With one expert in 32 to a lane and the groups one after the other it took 74 us.  A
// token alone takes 2.8 us.  Past 256 experts a lane searches its experts for each pick: 16 tokens
// of 384 experts 3.7 us without groups and 7.0 with 8, 32768 tokens of 384 62 us and of 512 77.
#include <cfloat>

#include "dg_common.cuh"
#include "dg_internal.h"
#include "dg_route.cuh"

namespace dg {
namespace {

using route::quotient_rn;
using route::recip_rn;

constexpr int kWarps = 4;

struct RouteArgs {
    const void* logits;
    const float* bias;
    int32_t* ids;
    float* w;
    long long ld;
    int M, E;
    int topk, n_group, topk_group, group_top, gsize;
    int group_shift;       // k where groups are aligned runs of 2^k lanes, else -1
    int vec;               // rows start on 16-byte boundaries
    int sigmoid, renorm;
    float scale;
};

// s + e += v, exactly but for the rounding of e, upwards: of a sum next to a tie between two floats
// a trace of further terms (all are positive) stays on the right side, however small.
__device__ __forceinline__ void two_sum(float& s, float& e, float v)
{
    const float t = __fadd_rn(s, v);
    const float z = __fsub_rn(t, s);
    e = __fadd_ru(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(v, z)));
    s = t;
}

__device__ __forceinline__ float warp_max(float v)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Score of a group of experts from its best two keys (-inf: no such key).  NaN marks groups that
// hold no key, and groups already taken: -inf is the score of two keys whose sum is below the
// type's range.
constexpr uint32_t kNoScore = 0x7fc00000u;
__device__ __forceinline__ float group_score(float b1, float b2, int group_top)
{
    if (!(b1 > -INFINITY)) return __uint_as_float(kNoScore);
    return group_top == 2 && b2 > -INFINITY ? __fadd_rn(b1, b2) : b1;
}

template <bool F32>
__device__ __forceinline__ float logit(const RouteArgs& a, long long row, int i)
{
    const long long o = row * a.ld + i;
    if constexpr (F32) return static_cast<const float*>(a.logits)[o];
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(a.logits)[o]) << 16);
}

// The lane's R logits; experts past E and NaN as -inf (not available).
template <int R, bool F32>
__device__ __forceinline__ void load_row(const RouteArgs& a, long long row, int lane, float (&x)[R])
{
    const int i0 = lane * R;
    constexpr int kVec = F32 ? 4 : 8;
    if constexpr (R % kVec == 0) {
        if (a.vec && i0 + R <= a.E) {
            const uint8_t* p = static_cast<const uint8_t*>(a.logits) + (row * a.ld + i0) * (F32 ? 4 : 2);
#pragma unroll
            for (int j = 0; j < R; j += kVec) {
                const uint4 v = *reinterpret_cast<const uint4*>(p + j * (F32 ? 4 : 2));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    if constexpr (F32) {
                        x[j + h] = __uint_as_float(w[h]);
                    } else {
                        x[j + 2 * h] = bf16_lo(w[h]);
                        x[j + 2 * h + 1] = bf16_hi(w[h]);
                    }
                }
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) x[j] = i0 + j < a.E ? logit<F32>(a, row, i0 + j) : -INFINITY;
}

// Descending, values alone (Batcher's odd-even merge sort, two instructions a comparison).
template <int R>
__device__ __forceinline__ void sort_keys(float (&k)[R])
{
#pragma unroll
    for (int p = 1; p < R; p <<= 1)
#pragma unroll
        for (int q = p; q > 0; q >>= 1)
#pragma unroll
            for (int j = q % p; j + q < R; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < R && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const float hi = fmaxf(k[i + j], k[i + j + q]), lo = fminf(k[i + j], k[i + j + q]);
                        k[i + j] = hi;
                        k[i + j + q] = lo;
                    }
}

template <int R, bool F32>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(RouteArgs a)
{
    constexpr bool kSorted = R <= 8;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long step = static_cast<long long>(gridDim.x) * kWarps;
    long long row = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (row >= a.M) return;
    float bias[R];                         // NaN: no key; at most FLT_MAX, as -inf and +inf would make a NaN key
    if (a.bias)
#pragma unroll
        for (int j = 0; j < R; ++j)
            bias[j] = lane * R + j < a.E ? fminf(fmaxf(a.bias[lane * R + j], -INFINITY), FLT_MAX) : 0.0f;
    float next[R];
    load_row<R, F32>(a, row, lane, next);
    for (; row < a.M; row += step) {
        float key[R];                                              // logits, then keys
#pragma unroll
        for (int j = 0; j < R; ++j) key[j] = fmaxf(next[j], -INFINITY);    // (NaN: not available)
        if (row + step < a.M) load_row<R, F32>(a, row + step, lane, next);
        float m = 0.0f, sum = 1.0f;
        if (!a.sigmoid) {
            float lm = key[0];
#pragma unroll
            for (int j = 1; j < R; ++j) lm = fmaxf(lm, key[j]);
            m = warp_max(lm);
            float s = 0.0f, e = 0.0f;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const float t = key[j] == m ? 1.0f : expf(key[j] - m);
                const bool can = key[j] > -INFINITY;
                two_sum(s, e, can ? t : 0.0f);
                key[j] = can ? t : -INFINITY;                              // (the exponential; a score below)
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const float s2 = __shfl_xor_sync(kFull, s, o), e2 = __shfl_xor_sync(kFull, e, o);
                two_sum(s, e, s2);
                e = __fadd_ru(e, e2);
            }
            sum = __fadd_rn(s, e);
        }
        auto score = [&](float v) {
            if (a.sigmoid) return __frcp_rn(__fadd_rn(1.0f, expf(-v)));
            return __fdiv_rn(v == m ? 1.0f : expf(v - m), sum);
        };
        if (a.sigmoid) {
            float low = 0.0f;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const float x = key[j] > -INFINITY ? key[j] : 0.0f;
                low = fminf(low, x);
                const float p = recip_rn(__fadd_rn(1.0f, expf(-x)));
                key[j] = key[j] > -INFINITY ? p : -INFINITY;
            }
            if (low < -86.0f) {                                    // 1 + e^-x past recip_rn's range
                float x[R];
                load_row<R, F32>(a, row, lane, x);
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (x[j] > -INFINITY) key[j] = __frcp_rn(__fadd_rn(1.0f, expf(-x[j])));
            }
        } else {
            const float r = recip_rn(sum);
            float low = 1.0f;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const float e = key[j] > -INFINITY ? key[j] : 1.0f;
                low = fminf(low, e);
                const float p = quotient_rn(e, sum, r);
                key[j] = key[j] > -INFINITY ? p : -INFINITY;
            }
            if (low < route::kLeastE) {
                float x[R];
                load_row<R, F32>(a, row, lane, x);
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (x[j] > -INFINITY) key[j] = __fdiv_rn(x[j] == m ? 1.0f : expf(x[j] - m), sum);
            }
        }
        if (a.bias)
#pragma unroll
            for (int j = 0; j < R; ++j) key[j] = __fadd_rn(key[j], bias[j]);
        float head[R];                                             // the keys in descending order
        if constexpr (kSorted) {
#pragma unroll
            for (int j = 0; j < R; ++j) head[j] = key[j];
            sort_keys<R>(head);
        }

        if (a.n_group > 1) {
            float gs = __uint_as_float(kNoScore);
            if (kSorted && a.group_shift >= 0) {
                // The best two of the lane are its heads; merged over the group's lanes.  Then the
                // best groups one by one, like the picks below.
                float b1 = head[0], b2 = R > 1 ? head[R > 1 ? 1 : 0] : -INFINITY;
                for (int o = 0; o < a.group_shift; ++o) {
                    const float c1 = __shfl_xor_sync(kFull, b1, 1 << o), c2 = __shfl_xor_sync(kFull, b2, 1 << o);
                    b2 = fmaxf(fminf(b1, c1), fmaxf(b2, c2));
                    b1 = fmaxf(b1, c1);
                }
                gs = group_score(b1, b2, a.group_top);
                const int own = lane >> a.group_shift;
                bool keep = false;
                for (int g = 0; g < a.topk_group; ++g) {
                    const float top = warp_max(gs);        // (NaN where no group is left: equal to none)
                    const int src = __ffs(__ballot_sync(kFull, gs == top)) - 1;
                    const bool mine = own == src >> a.group_shift;
                    keep = keep || mine;
                    gs = mine ? __uint_as_float(kNoScore) : gs;
                }
#pragma unroll
                for (int j = 0; j < R; ++j) head[j] = keep ? head[j] : -INFINITY;
            } else {
                // Groups that cut across lanes: one after the other, lane g keeping the score of g.
                for (int g = 0; g < a.n_group; ++g) {
                    float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
                    for (int j = 0; j < R; ++j) {
                        const int i = lane * R + j;
                        if (i >= g * a.gsize && i < (g + 1) * a.gsize) {
                            b2 = fmaxf(b2, fminf(b1, key[j]));
                            b1 = fmaxf(b1, key[j]);
                        }
                    }
                    const float t1 = warp_max(b1);
                    const unsigned who = __ballot_sync(kFull, b1 == t1);
                    const float t2 = warp_max(lane == __ffs(who) - 1 ? b2 : b1);
                    if (lane == g) gs = group_score(t1, t2, a.group_top);
                }
                int rank = 0;
                for (int g = 0; g < a.n_group; ++g) {
                    const float o = __shfl_sync(kFull, gs, g);
                    rank += (o > gs || (o == gs && g < lane)) ? 1 : 0;
                }
                const unsigned keep = __ballot_sync(kFull, lane < a.n_group && rank < a.topk_group);
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    const int i = lane * R + j;
                    if (i < a.E && !((keep >> (i / a.gsize)) & 1u)) key[j] = -INFINITY;
                }
                if constexpr (kSorted) {
#pragma unroll
                    for (int j = 0; j < R; ++j) head[j] = key[j];
                    sort_keys<R>(head);
                }
            }
        }

        int id = -1;                                               // lane k: slot k
        float wv = 0.0f;
        if constexpr (kSorted) {
            // Each pick: the warp's largest head, the lowest lane that has it.  Which of that
            // lane's experts it was is found afterwards, for all slots at once: equal keys of a
            // lane are picked one after the other, so the slot is the `nth` of them.
            float took = -INFINITY;
            int from = 0;
            for (int k = 0; k < a.topk; ++k) {
                const float top = warp_max(head[0]);
                if (!(top > -INFINITY)) break;
                const int src = __ffs(__ballot_sync(kFull, head[0] == top)) - 1;
                took = lane == k ? top : took;
                from = lane == k ? src : from;
                const bool mine = lane == src;
#pragma unroll
                for (int j = 0; j + 1 < R; ++j) head[j] = mine ? head[j + 1] : head[j];
                head[R - 1] = mine ? -INFINITY : head[R - 1];
            }
            // nth: how many slots right before this one took the same key from the same lane
            const float took_before = __shfl_up_sync(kFull, took, 1);
            const int from_before = __shfl_up_sync(kFull, from, 1);
            const unsigned same = __ballot_sync(kFull, lane > 0 && took == took_before && from == from_before);
            int nth = __clz(~(same << (31 - lane)));
            int at = 0;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const float v = __shfl_sync(kFull, key[j], from);
                if (v == took && nth-- == 0) at = j;
            }
            if (took > -INFINITY) {
                id = from * R + at;
                wv = took;
            }
        } else {
            for (int k = 0; k < a.topk; ++k) {
                float best = key[0];
                int at = 0;
#pragma unroll
                for (int j = 1; j < R; ++j)
                    if (key[j] > best) {
                        best = key[j];
                        at = j;
                    }
                const float top = warp_max(best);
                if (!(top > -INFINITY)) break;
                const int src = __ffs(__ballot_sync(kFull, best == top)) - 1;
                const int win = __shfl_sync(kFull, lane * R + at, src);
                if (lane == k) {
                    id = win;
                    wv = top;
                }
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (lane == src && j == at) key[j] = -INFINITY;
            }
        }
        if (a.bias && id >= 0) wv = score(logit<F32>(a, row, id));  // without the bias
        if (a.renorm) {
            float t = wv;
#pragma unroll
            for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(kFull, t, o);
            if (t < route::kLeastY || (wv > 0.0f && wv < route::kLeastE)) {    // where quotient_rn is not exact
                wv = t > 0.0f ? __fdiv_rn(wv, t) : 0.0f;
            } else {
                wv = quotient_rn(wv, t, recip_rn(t));
            }
        }
        if (lane < a.topk) {
            a.ids[row * a.topk + lane] = id;
            a.w[row * a.topk + lane] = __fmul_rn(wv, a.scale);
        }
    }
}

template <bool F32>
const void* route_fn(int r)
{
    switch (r) {
    case 1: return reinterpret_cast<const void*>(&route_kernel<1, F32>);
    case 2: return reinterpret_cast<const void*>(&route_kernel<2, F32>);
    case 4: return reinterpret_cast<const void*>(&route_kernel<4, F32>);
    case 8: return reinterpret_cast<const void*>(&route_kernel<8, F32>);
    case 16: return reinterpret_cast<const void*>(&route_kernel<16, F32>);
    default: return reinterpret_cast<const void*>(&route_kernel<32, F32>);
    }
}

}  // namespace

dg_status launch_route(const dg_route_params& p, const void* logits, const float* bias, int32_t* ids, float* w,
                       int M, int E, long long ld, bool f32, cudaStream_t stream)
{
    dg_status st;
    const DeviceInfo* dev = current_device(&st);
    if (!dev) return st;
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
    const int r = cpow2((E + 31) / 32);
    const int gl = a.gsize % r == 0 ? a.gsize / r : 0;
    a.group_shift = gl > 0 && (gl & (gl - 1)) == 0 ? clog2(gl) : -1;
    a.vec = reinterpret_cast<uintptr_t>(logits) % 16 == 0 && (ld * (f32 ? 4 : 2)) % 16 == 0 ? 1 : 0;
    const void* fn = f32 ? route_fn<true>(r) : route_fn<false>(r);
    const int occ = occupancy(fn, kWarps * 32, 0);
    if (occ < 1) return DG_ERR_CUDA;
    // One token a warp, until every warp slot has some: then they walk.
    long long grid = (static_cast<long long>(M) + kWarps - 1) / kWarps;
    const long long most = static_cast<long long>(dev->sm_count) * occ;
    if (grid > most) grid = most;
    void* args[] = {&a};
    if (launch_kernel(fn, static_cast<unsigned>(grid), kWarps * 32, 0, stream, args, Early::kNothing) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

}  // namespace dg
