// dg_logprobs.cu -- log-probabilities of given tokens, rank, entropy and the top
// alternatives over a row of logits (dg_logprobs).
//
// One pass over the row.  In units of log2 with c = scale * log2(e) and a reference r
// (the largest logit seen so far times c): y = z c - r, s = sum 2^y, t = sum 2^y y; when
// the reference moves by d = r_old - r_new, s <- s 2^d and t <- 2^d (t + s d).  Then
//   logprob = ln 2 (y_token - log2 s),   entropy = ln 2 (log2 s - t / s).
// Every thread keeps its own reference; two terms at a time go through packed binary32
// operations, and bf16 pairs are compared and clamped as they come.  For the alternatives:
// the n-th largest of the 32 parts' largest logits is a bound that at least n logits
// reach, so only the threads whose own largest reaches it are looked at again, with all
// threads of the CTA.
// A row belongs to one CTA, or to a cluster of up to 8 when there are few rows; the others
// write their sums and lists into the first one's shared memory.  The largest, the count and the
// lists do not depend on the split.
// Bound: with many rows memory, 2 or 4 bytes a logit (2048 x 248320 bf16: 176 us, 5.8 TB/s, 85 %
// of the copy rate; 66 % of the issue slots, 8.7 instructions a logit); with few, latencies
// one after the other -- loads, the bound, the gathering, the cluster's join (one row of
// 248320: 7.5 us).  Rows where fewer logits than alternatives are above a value that more than
// kCand share (a mask by the type's lowest value) take a pass for each alternative: 20 of 248320
// with three logits left 105 us for one row and 9.3 ms for 2048, against 6.7 and 166 us where
// the mask is -inf.
#include "dg_common.cuh"
#include "dg_internal.h"

namespace dg {
namespace {

// Threads per CTA (template parameter T).  A row costs a CTA a few us beside its bytes, so many
// short rows take small CTAs, eight or more of them on an SM.
constexpr int kWide = 512, kNarrow = 128;
constexpr int kU = 8;                      // 16-byte loads in flight a thread (two wide CTAs an SM: 4: 184 us, 8: 173)
constexpr int kMaxCs = 8;                  // CTAs of a row
constexpr int kMaxTop = 32;
// Terms that one running sum takes before it is folded away: equal addends between two powers of
// two all round the same way, so the error grows with their number (16384 of them: 2.3e-4).
constexpr int kTerms = 256;
// The vectors that bring them, each half of a packed sum half a vector's elements.
__host__ __device__ constexpr int fold_vectors(bool f32, int threads) { return kTerms * 2 / (f32 ? 4 : 8) * threads; }

constexpr int kCand = 1024;                // candidates held at once
constexpr float kFar = -1.0e30f;           // logits are clamped here (masked ones: 0 * y stays 0)
constexpr float kNear = 1048576.0f;        // |r| up to which z c - r may be off by its rounding (2^-4 at most)
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.442695040888963407f;

struct LpArgs {
    const void* logits;
    long long ld;
    const int64_t* tokens;
    float scale;
    int n_top;
    float* logprob;
    int32_t* rank;
    float* entropy;
    int32_t* top_ids;
    float* top_lp;
    int M, V, cs;
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Two binary32 values in one register pair (packed fused multiply-add, add, multiply).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack(float lo, float hi)
{
    f32x2 v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b)
{
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Pairs of bf16: the larger (a number where one is NaN; NaN where one is), and -1 in the
// halves where a > b.
constexpr uint32_t kFarBf2 = 0xf14af14au;          // about -1e30 twice
__device__ __forceinline__ uint32_t bf2_max(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf2_max_nan(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf2_gt(uint32_t a, uint32_t b)
{
    __nv_bfloat162 x, y;
    memcpy(&x, &a, sizeof x);
    memcpy(&y, &b, sizeof y);
    return __hgt2_mask(x, y);
}

// Order of logits as unsigned: larger is larger, -0 equals +0; 0 for what is never an
// alternative (NaN, -inf).
__device__ __forceinline__ uint32_t order_key(float f)
{
    if (!(f > -INFINITY)) return 0;
    const uint32_t b = __float_as_uint(f + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// Larger logit first, then the lower index.
__device__ __forceinline__ unsigned long long pair_key(uint32_t k, int i)
{
    return (static_cast<unsigned long long>(k) << 32) | static_cast<uint32_t>(~i);
}

template <bool F32>
struct Vec {
    static constexpr int n = F32 ? 4 : 8;
    static __device__ __forceinline__ float at(const void* row, int i)
    {
        if constexpr (F32) return static_cast<const float*>(row)[i];
        return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(row)[i]) << 16);
    }
    static __device__ __forceinline__ void unpack(const uint4& v, float (&z)[n])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (F32) {
                z[i] = __uint_as_float(w[i]);
            } else {
                z[2 * i] = bf16_lo(w[i]);
                z[2 * i + 1] = bf16_hi(w[i]);
            }
        }
    }
};

struct Sums {
    float r, s, t;       // reference, sum 2^y, sum 2^y y
};

// The sums of `b` taken over to the reference of `a` or the other way round.
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b)
{
    const float r = max_nan(a.r, b.r);
    const float da = a.r == r ? 0.0f : a.r - r, db = b.r == r ? 0.0f : b.r - r;
    const float fa = ex2(da), fb = ex2(db);
    return {r, a.s * fa + b.s * fb, fa * (a.t + a.s * da) + fb * (b.t + b.s * db)};
}

template <int T>
struct Shared {
    static constexpr int kW = T / 32;
    static_assert(kW >= 2 && kW <= 32, "the first warp joins the warps' sums, the second finds the bound");
    Sums sums[kW];
    int count[kW];
    float big[kW];
    alignas(16) uint32_t part_key[32];     // largest keys of T / 32 threads each
    Sums total;
    int total_count;
    float total_big;
    int n_list, n_cand;
    uint32_t floor;
    unsigned long long top[kMaxTop];
    // the first CTA of a cluster: what every CTA found
    Sums part[kMaxCs];
    int part_count[kMaxCs];
    float part_big[kMaxCs];
    unsigned long long all[kMaxCs * kMaxTop];
    unsigned long long cand[kCand];
    int list[T];
};

// The row's slice of one CTA: `head` single elements up to a 16-byte boundary (first CTA),
// vectors [v0, v1), `tail` single elements (last CTA).  Single elements belong to the
// threads 0.. in order, vectors to thread (v - v0) % T.
template <bool F32>
struct Slice {
    const void* row;
    const uint4* vec;
    int head, tail, tail0, v0, v1;
    int n_single;

    __device__ int single(int i) const { return i < head ? i : tail0 + i - head; }
    __device__ int index(int v) const { return head0 + v * Vec<F32>::n; }
    int head0;           // element of vector 0
};

// Every (key, index) of this thread's share of `list` that reaches `floor`, to the candidates.
template <bool F32, int T>
__device__ void gather(Shared<T>& sh, const Slice<F32>& sl, uint32_t floor)
{
    const int per = (sl.v1 - sl.v0 + T - 1) / T;
    const int n = sh.n_list * (per + 1);
    for (int q = threadIdx.x; q < n; q += T) {
        const int e = q / (per + 1), k = q - e * (per + 1), t = sh.list[e];
        if (k == per) {
            if (t < sl.n_single) {
                const int i = sl.single(t);
                const uint32_t key = order_key(Vec<F32>::at(sl.row, i));
                if (key >= floor) {
                    const int p = atomicAdd(&sh.n_cand, 1);
                    if (p < kCand) sh.cand[p] = pair_key(key, i);
                }
            }
            continue;
        }
        const int v = sl.v0 + k * T + t;
        if (v >= sl.v1) continue;
        float z[Vec<F32>::n];
        Vec<F32>::unpack(sl.vec[v], z);
#pragma unroll
        for (int j = 0; j < Vec<F32>::n; ++j) {
            const uint32_t key = order_key(z[j]);
            if (key >= floor) {
                const int p = atomicAdd(&sh.n_cand, 1);
                if (p < kCand) sh.cand[p] = pair_key(key, sl.index(v) + j);
            }
        }
    }
}

// The largest pair of the slice below `below`, for every thread.
template <bool F32, int T>
__device__ unsigned long long next_pair(Shared<T>& sh, const Slice<F32>& sl, unsigned long long below)
{
    unsigned long long best = 0;
    auto see = [&](float z, int i) {
        const uint32_t key = order_key(z);
        const unsigned long long p = key ? pair_key(key, i) : 0ull;
        if (p < below && p > best) best = p;
    };
    if (static_cast<int>(threadIdx.x) < sl.n_single) {
        const int i = sl.single(threadIdx.x);
        see(Vec<F32>::at(sl.row, i), i);
    }
    for (int v = sl.v0 + threadIdx.x; v < sl.v1; v += T) {
        float z[Vec<F32>::n];
        Vec<F32>::unpack(sl.vec[v], z);
#pragma unroll
        for (int j = 0; j < Vec<F32>::n; ++j) see(z[j], sl.index(v) + j);
    }
    __syncthreads();
    sh.cand[threadIdx.x] = best;
    __syncthreads();
    for (int o = T / 2; o; o >>= 1) {
        if (static_cast<int>(threadIdx.x) < o)
            sh.cand[threadIdx.x] = max(sh.cand[threadIdx.x], sh.cand[threadIdx.x + o]);
        __syncthreads();
    }
    best = sh.cand[0];
    __syncthreads();
    return best;
}

// The n largest pairs among c, each thread placing its own by counting those ahead.
template <int T>
__device__ void place(const unsigned long long* c, int count, unsigned long long* out, int n)
{
    for (int i = threadIdx.x; i < count; i += T) {
        const unsigned long long p = c[i];
        int ahead = 0;
#pragma unroll 8
        for (int j = 0; j < count; ++j) ahead += c[j] > p ? 1 : 0;
        if (p && ahead < n) out[ahead] = p;
    }
}

// The n largest pairs of `lists` lists of n (lists a power of two; each in descending order, 0
// past its end), in sh.top.  The n-th largest of the lists' first ceil(n / lists) pairs is a
// bound that the n largest reach; few others do, and those place themselves.
template <int T>
__device__ void merge(Shared<T>& sh, const unsigned long long* c, int lists, int n)
{
    const int lane = threadIdx.x & 31, lg = 31 - __clz(lists), k = (n + lists - 1) >> lg;  // lists * k <= 32
    const int at = lane >> lg < k ? (lane & (lists - 1)) * n + (lane >> lg) : -1;
    const unsigned long long v = at >= 0 ? c[at] : 0ull;
    int above = 0;
#pragma unroll 8
    for (int j = 0; j < lists * k; ++j) above += c[(j & (lists - 1)) * n + (j >> lg)] > v ? 1 : 0;
    const bool in = at >= 0 && above < n;
    const uint32_t hi = __reduce_min_sync(kFull, in ? static_cast<uint32_t>(v >> 32) : 0xffffffffu);
    const uint32_t lo = __reduce_min_sync(kFull, in && static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v)
                                                                                            : 0xffffffffu);
    const unsigned long long floor = (static_cast<unsigned long long>(hi) << 32) | lo;
    for (int i = threadIdx.x; i < lists * n; i += T)
        if (c[i] && c[i] >= floor) sh.cand[atomicAdd(&sh.n_cand, 1)] = c[i];
    __syncthreads();
    place<T>(sh.cand, sh.n_cand, sh.top, n);
}
static_assert(kMaxCs * kMaxTop <= kCand, "every pair of the lists fits");

// The slice's n_top largest pairs, in order, in sh.top (0 past the last).  Called with
// sh.part_key and cleared counters visible to all threads.
template <bool F32, int T>
__device__ void slice_top(Shared<T>& sh, const Slice<F32>& sl, uint32_t mine, int n)
{
    static_assert(kMaxTop <= 32, "one alternative a part at least");
    // The n-th largest of the parts' largest, the smallest with fewer than n above it
    // (1: every key that counts); one warp's work, beside the first's sums.
    if (threadIdx.x >> 5 == 1) {
        const uint32_t v = sh.part_key[threadIdx.x & 31];
        int above = 0;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            const uint4 o = *reinterpret_cast<const uint4*>(sh.part_key + j);
            above += (o.x > v ? 1 : 0) + (o.y > v ? 1 : 0) + (o.z > v ? 1 : 0) + (o.w > v ? 1 : 0);
        }
        const uint32_t f = __reduce_min_sync(kFull, above < n ? v : 0xffffffffu);
        if ((threadIdx.x & 31) == 0) sh.floor = f ? f : 1u;
    }
    __syncthreads();
    const uint32_t floor = sh.floor;
    if (mine >= floor) sh.list[atomicAdd(&sh.n_list, 1)] = threadIdx.x;
    __syncthreads();
    gather<F32, T>(sh, sl, floor);
    __syncthreads();
    const int c = sh.n_cand;
    if (c <= kCand) {
        place<T>(sh.cand, c, sh.top, n);
        return;
    }
    // More logits at the bound than are held (rows of equal values): one at a time.
    unsigned long long p = ~0ull;
    for (int k = 0; k < n; ++k) {
        p = next_pair<F32, T>(sh, sl, p);
        if (!p) break;
        if (threadIdx.x == 0) sh.top[k] = p;
    }
}

// Stores into the shared memory of the cluster's first CTA.
__device__ __forceinline__ uint32_t first_cta(const void* p)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))));
    return r;
}

__device__ __forceinline__ void put_f32(float* p, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(first_cta(p)), "f"(v) : "memory");
}

__device__ __forceinline__ void put_u64(unsigned long long* p, unsigned long long v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(first_cta(p)), "l"(v) : "memory");
}

// Long: slices of more than fold_vectors().
template <bool F32, int T, bool Long>
__global__ void __launch_bounds__(T, 1024 / T) logprobs_kernel(LpArgs a)
{
    constexpr int VE = Vec<F32>::n, kW = T / 32;
    __shared__ Shared<T> sh;
    pdl_launch_dependents();
    pdl_wait();
    const int cs = a.cs, rank_in = static_cast<int>(blockIdx.x) % cs;
    const long long m = blockIdx.x / cs;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // (the first CTA runs before others write into it: waited for below)
    if (cs > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

    Slice<F32> sl;
    sl.row = static_cast<const uint8_t*>(a.logits) + m * a.ld * (F32 ? 4 : 2);
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(sl.row) & 15u) / (F32 ? 4 : 2);
    const int head = min(a.V, (VE - off) % VE);
    const int nv = (a.V - head) / VE;
    sl.head0 = head;
    sl.vec = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(sl.row) + head * (F32 ? 4 : 2));
    sl.v0 = static_cast<int>(static_cast<long long>(nv) * rank_in / cs);
    sl.v1 = static_cast<int>(static_cast<long long>(nv) * (rank_in + 1) / cs);
    sl.head = rank_in == 0 ? head : 0;
    sl.tail0 = head + nv * VE;
    sl.tail = rank_in == cs - 1 ? a.V - sl.tail0 : 0;
    sl.n_single = sl.head + sl.tail;

    // kU loads in flight a thread (past the last vector, masked ones), the first of them before
    // the token's logit is looked up: that is two round trips.
    constexpr uint32_t kMasked = F32 ? 0xff800000u : 0xff80ff80u;
    uint4 q[kU];
    auto load = [&](int v) {
#pragma unroll
        for (int i = 0; i < kU; ++i)
            q[i] = v + i * T < sl.v1 ? ld_stream_after(sl.vec + v + i * T)
                                     : make_uint4(kMasked, kMasked, kMasked, kMasked);
    };
    int at = sl.v0 + tid;
    load(at);

    const long long tok = a.tokens ? a.tokens[m] : -1;
    const bool has_tok = tok >= 0 && tok < a.V;
    const float zt = has_tok ? Vec<F32>::at(sl.row, static_cast<int>(tok)) : INFINITY;
    const float c = a.scale * kLog2e;

    // The reference before any logit: far below every one that counts, and yet so far above the
    // clamp below that 2^y of a clamped logit is 0.
    float r = 0.5f * kFar * c, big = -INFINITY;        // (big: largest logit, NaN aside)
    f32x2 s2 = pack(0.0f, 0.0f), t2 = s2, nr = pack(-r, -r);
    const f32x2 c2 = pack(c, c);
    int count = 0;
    uint32_t masks = 0;                    // sum of comparison masks, see below
    auto refer = [&](float z) {            // moves the reference up to z
        const float to = z * c;
        if (to > r) {
            const float d = r - to, f = ex2(d);
            const f32x2 f2 = pack(f, f), d2 = pack(d, d);
            t2 = mul2(f2, fma2(s2, d2, t2));
            s2 = mul2(s2, f2);
            r = to;
            nr = pack(-to, -to);
        }
    };
    auto add = [&](float z0, float z1) {
        const f32x2 y = fma2(pack(z0, z1), c2, nr);
        float y0, y1;
        unpack2(y, y0, y1);
        const f32x2 e = pack(ex2(y0), ex2(y1));
        s2 = add2(s2, e);
        t2 = fma2(e, y, t2);
    };
    if (tid < sl.n_single) {
        const float z = Vec<F32>::at(sl.row, sl.single(tid));
        big = fmaxf(big, z);
        refer(big);
        add(max_nan(z, kFar), kFar);
        count += z > zt ? 1 : 0;
    }
    const uint32_t zt2 = F32 ? 0u : (__float_as_uint(zt) >> 16) * 0x10001u;
    // Two vectors at a time: one test for a new largest, one for logits above the token's.
    auto take = [&](const uint4& p, const uint4& q) {
        const uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
        float vm;
        if constexpr (F32) {
            vm = __uint_as_float(w[0]);
#pragma unroll
            for (int j = 1; j < 8; ++j) vm = fmaxf(vm, __uint_as_float(w[j]));
        } else {
            const uint32_t m2 = bf2_max(bf2_max(bf2_max(w[0], w[1]), bf2_max(w[2], w[3])),
                                        bf2_max(bf2_max(w[4], w[5]), bf2_max(w[6], w[7])));
            vm = fmaxf(bf16_lo(m2), bf16_hi(m2));
        }
        if (vm > big) {
            big = vm;
            refer(vm);
        }
        if (vm > zt) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (F32)
                    count += __uint_as_float(w[j]) > zt ? 1 : 0;
                else               // each mask is -1 in the halves that hold a larger logit: their sum
                    masks += bf2_gt(w[j], zt2);        // mod 2^32 is 2^16 (n_lo - n_hi) - n_lo
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (F32) {
                if (j & 1) add(max_nan(__uint_as_float(w[j - 1]), kFar), max_nan(__uint_as_float(w[j]), kFar));
            } else {
                const uint32_t z = bf2_max_nan(w[j], kFarBf2);
                add(bf16_lo(z), bf16_hi(z));
            }
        }
    };
    auto sums = [&] {
        float s0, s1, t0, t1;
        unpack2(s2, s0, s1);
        unpack2(t2, t0, t1);
        return Sums{r, s0 + s1, t0 + t1};
    };
    // (the candidates' place is idle yet)
    constexpr int kFold = fold_vectors(F32, T);
    static_assert(kFold % (kU * T) == 0 && sizeof(Sums) * T <= sizeof sh.cand, "folds between rounds, in place");
    Sums* const held = reinterpret_cast<Sums*>(sh.cand) + tid;
    const int first = at + kFold;
    int fold = first;
    for (;;) {
#pragma unroll
        for (int i = 0; i < kU; i += 2) take(q[i], q[i + 1]);
        at += kU * T;
        if (at >= sl.v1) break;
        load(at);
        if constexpr (Long)
            if (at == fold) {
                *held = fold == first ? sums() : join(*held, sums());
                s2 = t2 = pack(0.0f, 0.0f);
                fold += kFold;
            }
    }
    if constexpr (!F32) {
        const int lo = static_cast<int>((0u - masks) & 0xffffu);
        count += 2 * lo - (static_cast<int>(masks + static_cast<uint32_t>(lo)) >> 16);
    }
    Sums u = sums();
    if (Long && fold != first) u = join(*held, u);
    const uint32_t mine = order_key(big);

    // CTA totals: warps, then the warps' in the first warp, beside the search for alternatives.
    auto join_lanes = [&](int from) {
        for (int o = from; o; o >>= 1) {
            const Sums v{__shfl_xor_sync(kFull, u.r, o), __shfl_xor_sync(kFull, u.s, o), __shfl_xor_sync(kFull, u.t, o)};
            u = join(u, v);
            count += __shfl_xor_sync(kFull, count, o);
            big = fmaxf(big, __shfl_xor_sync(kFull, big, o));
        }
    };
    uint32_t part = mine;
#pragma unroll
    for (int o = T / 64; o; o >>= 1) part = max(part, __shfl_xor_sync(kFull, part, o));
    join_lanes(16);
    if (tid % (T / 32) == 0) sh.part_key[tid / (T / 32)] = part;
    if (lane == 0) {
        sh.sums[warp] = u;
        sh.count[warp] = count;
        sh.big[warp] = big;
    }
    if (tid < kMaxTop) sh.top[tid] = 0;
    if (tid == 0) sh.n_list = sh.n_cand = 0;
    __syncthreads();
    if (warp == 0) {
        const bool on = lane < kW;
        u = on ? sh.sums[lane] : Sums{kFar, 0.0f, 0.0f};
        count = on ? sh.count[lane] : 0;
        big = on ? sh.big[lane] : -INFINITY;
        join_lanes(kW / 2);
        if (lane == 0) {
            sh.total = u;
            sh.total_count = count;
            sh.total_big = big;
        }
    }
    if (a.n_top > 0) slice_top<F32, T>(sh, sl, mine, a.n_top);
    __syncthreads();
    if (cs > 1) {
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        if (tid < a.n_top) put_u64(&sh.all[rank_in * a.n_top + tid], sh.top[tid]);
        if (tid == 0) {
            put_f32(&sh.part[rank_in].r, sh.total.r);
            put_f32(&sh.part[rank_in].s, sh.total.s);
            put_f32(&sh.part[rank_in].t, sh.total.t);
            put_f32(reinterpret_cast<float*>(&sh.part_count[rank_in]), __int_as_float(sh.total_count));
            put_f32(&sh.part_big[rank_in], sh.total_big);
        }
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (rank_in != 0) return;
        if (tid < kMaxTop) sh.top[tid] = 0;
        if (tid == 0) sh.n_cand = 0;
        if (warp == 0) {
            const bool on = lane < cs;
            u = on ? sh.part[lane] : Sums{kFar, 0.0f, 0.0f};
            count = on ? sh.part_count[lane] : 0;
            big = on ? sh.part_big[lane] : -INFINITY;
            join_lanes(kMaxCs / 2);
            if (lane == 0) {
                sh.total = u;
                sh.total_count = count;
                sh.total_big = big;
            }
        }
        __syncthreads();
        if (a.n_top > 0) merge(sh, sh.all, cs, a.n_top);
        __syncthreads();
    }
    u = sh.total;
    big = sh.total_big;
    const bool near = fabsf(u.r) <= kNear; // y against the reference, else against `big`
    if (!near && big > -INFINITY) {
        // A reference so large that the rounding of z c is no small shift of y any more, or no
        // logit above -1e30 / c: sums against the largest logit itself.
        float s = 0.0f, t = 0.0f;
        for (int i0 = 0; i0 < a.V; i0 += kTerms * T) {
            float sp = 0.0f, tp = 0.0f;
            for (int i = i0 + tid; i < min(a.V, i0 + kTerms * T); i += T) {
                const float z = Vec<F32>::at(sl.row, i);
                if (z == -INFINITY) continue;
                const float y = max_nan((z - big) * c, kFar), e = ex2(y);
                sp += e;
                tp = fmaf(e, y, tp);
            }
            s += sp;
            t += tp;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            s += __shfl_xor_sync(kFull, s, o);
            t += __shfl_xor_sync(kFull, t, o);
        }
        __syncthreads();
        if (lane == 0) sh.sums[warp] = Sums{0.0f, s, t};
        __syncthreads();
        s = t = 0.0f;
        for (int w = 0; w < kW; ++w) {
            s += sh.sums[w].s;
            t += sh.sums[w].t;
        }
        u = Sums{kFar, s, t};
    }
    const bool none = !(big > -INFINITY) && u.s == 0.0f;
    const float l2s = log2f(u.s);
    auto logprob = [&](float z) {
        if (none || z == -INFINITY) return u.s != u.s ? u.s : -INFINITY;
        const float y = near ? fmaf(z, c, -u.r) : (z - big) * c;
        if (y < kFar && l2s == l2s)        // the factor log2(e) may overflow where scale does not, or z - big
            return near ? fmaf(z, a.scale, -u.r * kLn2) : (0.5f * z - 0.5f * big) * a.scale * 2.0f;
        return (y - l2s) * kLn2;
    };
    if (tid == 0) {
        if (a.logprob) a.logprob[m] = has_tok ? logprob(zt) : __uint_as_float(0x7fc00000u);
        if (a.rank) a.rank[m] = has_tok ? sh.total_count : -1;
        if (a.entropy) a.entropy[m] = none ? 0.0f : (l2s - u.t / u.s) * kLn2;
    }
    if (tid < a.n_top) {
        const unsigned long long p = sh.top[tid];
        a.top_ids[m * a.n_top + tid] = p ? static_cast<int32_t>(~static_cast<uint32_t>(p)) : -1;
        a.top_lp[m * a.n_top + tid] = p ? logprob(key_value(static_cast<uint32_t>(p >> 32))) : -INFINITY;
    }
}

template <bool F32>
const void* kernel_for(bool narrow, bool lengthy)
{
    if (narrow) return reinterpret_cast<const void*>(&logprobs_kernel<F32, kNarrow, false>);
    return lengthy ? reinterpret_cast<const void*>(&logprobs_kernel<F32, kWide, true>)
                   : reinterpret_cast<const void*>(&logprobs_kernel<F32, kWide, false>);
}

}  // namespace

dg_status launch_logprobs(const void* logits, bool f32, long long ld, const int64_t* tokens, float scale, int n_top,
                          float* logprob, int32_t* rank, float* entropy, int32_t* top_ids, float* top_logprobs, int M,
                          int V, cudaStream_t stream)
{
    dg_status st;
    const DeviceInfo* dev = current_device(&st);
    if (!dev) return st;
    LpArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.tokens = tokens;
    a.scale = scale;
    a.n_top = n_top;
    a.logprob = logprob;
    a.rank = rank;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_lp = top_logprobs;
    a.M = M;
    a.V = V;
    // CTAs per row: with few rows as many as two for each SM (one CTA alone is bound by its
    // instructions: 248320 logits take it 11 us), but no slice below six vectors a thread, which
    // one round of loads brings (a cluster's join costs about 1.5 us).
    // Many short rows: at most 16 vectors a thread of a wide CTA with four rows for every SM, or 4
    // with two (4096 x 8000: 85 us wide, 24 narrow; 304 x 65536: 11.0 and 15.8).
    const int ve = f32 ? 4 : 8;
    const bool narrow = V <= 16 * kWide * ve && M >= (V <= 4 * kWide * ve ? 2 : 4) * dev->sm_count;
    int cs = 1;
    while (!narrow && cs < kMaxCs && static_cast<long long>(M) * cs * 2 <= 2ll * dev->sm_count &&
           V / (cs * 2) >= 6 * kWide * ve)
        cs *= 2;
    a.cs = cs;
    // Folding running sums away costs 2048 x 248320 bf16, which need none, 1.3 % (176.6 and 178.9 us).
    const bool lengthy = V / ve / cs >= fold_vectors(f32, kWide);
    const void* fn = f32 ? kernel_for<true>(narrow, lengthy) : kernel_for<false>(narrow, lengthy);
    void* args[] = {&a};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(M) * cs));
    cfg.blockDim = dim3(narrow ? kNarrow : kWide);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cs);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    if (launch_ordered(cfg, attr, 1, fn, args, Early::kNothing) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

}  // namespace dg
