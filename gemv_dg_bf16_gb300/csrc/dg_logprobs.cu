// dg_logprobs.cu -- log-probabilities of given tokens, rank, entropy and the top
// alternatives over a row of logits (dg_logprobs).
//
// One pass over the row.  In units of log2 with c = scale * log2(e) and a reference r
// (the largest logit seen so far times c): y = z c - r, s = sum 2^y, t = sum 2^y y; when
// the reference moves by d = r_old - r_new, s <- s 2^d and t <- 2^d (t + s d).  Then
//   logprob = ln 2 (y_token - log2 s),   entropy = ln 2 (log2 s - t / s).
// Every thread keeps its own reference, and its largest logit for the alternatives: the
// n-th largest of the threads' largest is a bound that at least n logits reach, so only
// the threads that reach it are looked at again, with all threads of the CTA.
// A row belongs to one CTA, or to a cluster of up to 8 when there are few rows; the CTAs'
// sums and lists meet in shared memory of the first.  The largest, the count and the
// lists do not depend on the split.
// Bound: memory, 2 or 4 bytes a logit, with many rows; with few, the latency of one
// CTA's slice and the joins.
#include "dg_common.cuh"
#include "dg_internal.h"

namespace dg {
namespace {

constexpr int kT = 512;                    // threads per CTA
constexpr int kW = kT / 32;
constexpr int kMaxTop = 32;
constexpr int kCand = 1024;                // candidates held at once
constexpr float kFar = -1.0e30f;           // reference before any logit; far below it counts as none
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

struct Shared {
    Sums sums[kW];
    int count[kW];
    float big[kW];
    Sums total;
    int total_count;
    float total_big;
    int n_list, n_cand, n_more;
    int list[kT];
    unsigned long long cand[kCand];
    unsigned long long top[kMaxTop];
    unsigned long long all[8 * kMaxTop];
};

// The row's slice of one CTA: `head` single elements up to a 16-byte boundary (first CTA),
// vectors [v0, v1), `tail` single elements (last CTA).  Single elements belong to the
// threads 0.. in order, vectors to thread (v - v0) % kT.
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
template <bool F32>
__device__ void gather(Shared& sh, const Slice<F32>& sl, uint32_t floor)
{
    const int per = (sl.v1 - sl.v0 + kT - 1) / kT;
    const int n = sh.n_list * (per + 1);
    for (int q = threadIdx.x; q < n; q += kT) {
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
        const int v = sl.v0 + k * kT + t;
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
template <bool F32>
__device__ unsigned long long next_pair(Shared& sh, const Slice<F32>& sl, unsigned long long below)
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
    for (int v = sl.v0 + threadIdx.x; v < sl.v1; v += kT) {
        float z[Vec<F32>::n];
        Vec<F32>::unpack(sl.vec[v], z);
#pragma unroll
        for (int j = 0; j < Vec<F32>::n; ++j) see(z[j], sl.index(v) + j);
    }
    __syncthreads();
    sh.cand[threadIdx.x] = best;
    __syncthreads();
    for (int o = kT / 2; o; o >>= 1) {
        if (static_cast<int>(threadIdx.x) < o)
            sh.cand[threadIdx.x] = max(sh.cand[threadIdx.x], sh.cand[threadIdx.x + o]);
        __syncthreads();
    }
    best = sh.cand[0];
    __syncthreads();
    return best;
}

// The n largest pairs among c, each thread placing its own by counting those ahead.
__device__ void place(const unsigned long long* c, int count, unsigned long long* out, int n)
{
    for (int i = threadIdx.x; i < count; i += kT) {
        const unsigned long long p = c[i];
        int ahead = 0;
        for (int j = 0; j < count; ++j) ahead += c[j] > p ? 1 : 0;
        if (p && ahead < n) out[ahead] = p;
    }
}

// The slice's n_top largest pairs, in order, in sh.top (0 past the last).
template <bool F32>
__device__ void slice_top(Shared& sh, const Slice<F32>& sl, uint32_t mine, int n)
{
    if (threadIdx.x < kMaxTop) sh.top[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.n_list = sh.n_cand = 0;
    // The largest bound that n threads reach (1: every key that counts).
    uint32_t floor = 0;
    for (int bit = 31; bit >= (F32 ? 0 : 16); --bit) {
        const uint32_t f = floor | (1u << bit);
        if (__syncthreads_count(mine >= f) >= n) floor = f;
    }
    if (floor == 0) floor = 1;
    if (mine >= floor) sh.list[atomicAdd(&sh.n_list, 1)] = threadIdx.x;
    __syncthreads();
    gather<F32>(sh, sl, floor);
    __syncthreads();
    const int c = sh.n_cand;
    if (c <= kCand) {
        place(sh.cand, c, sh.top, n);
        return;
    }
    // More logits at the bound than are held (rows of equal values): one at a time.
    unsigned long long p = ~0ull;
    for (int k = 0; k < n; ++k) {
        p = next_pair<F32>(sh, sl, p);
        if (!p) break;
        if (threadIdx.x == 0) sh.top[k] = p;
    }
}

__device__ __forceinline__ uint32_t peer(const void* p, int rank)
{
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}

__device__ __forceinline__ float peer_f32(const void* p, int rank)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer(p, rank)));
    return v;
}

__device__ __forceinline__ unsigned long long peer_u64(const void* p, int rank)
{
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(peer(p, rank)));
    return v;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <bool F32>
__global__ void __launch_bounds__(kT) logprobs_kernel(LpArgs a)
{
    constexpr int VE = Vec<F32>::n;
    __shared__ Shared sh;
    pdl_launch_dependents();
    pdl_wait();
    const int cs = a.cs, rank_in = static_cast<int>(blockIdx.x) % cs;
    const long long m = blockIdx.x / cs;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

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

    const long long tok = a.tokens ? a.tokens[m] : -1;
    const bool has_tok = tok >= 0 && tok < a.V;
    const float zt = has_tok ? Vec<F32>::at(sl.row, static_cast<int>(tok)) : INFINITY;
    const float c = a.scale * kLog2e;

    Sums u{kFar, 0.0f, 0.0f};
    float big = -INFINITY;                 // largest logit (NaN aside)
    int count = 0;
    auto refer = [&](float z) {            // moves the reference up to z
        const float r = z * c;
        if (r > u.r) {
            const float d = u.r - r, f = ex2(d);
            u.t = f * (u.t + u.s * d);
            u.s *= f;
            u.r = r;
        }
    };
    auto add = [&](float z) {
        const float y = max_nan(fmaf(z, c, -u.r), kFar);
        const float e = ex2(y);
        u.s += e;
        u.t = fmaf(e, y, u.t);
        count += z > zt ? 1 : 0;
    };
    if (tid < sl.n_single) {
        const float z = Vec<F32>::at(sl.row, sl.single(tid));
        big = fmaxf(big, z);
        refer(big);
        add(z);
    }
#pragma unroll 4
    for (int v = sl.v0 + tid; v < sl.v1; v += kT) {
        float z[VE];
        Vec<F32>::unpack(ld_stream_after(sl.vec + v), z);
        float vm = z[0];
#pragma unroll
        for (int j = 1; j < VE; ++j) vm = fmaxf(vm, z[j]);
        if (vm > big) {
            big = vm;
            refer(vm);
        }
#pragma unroll
        for (int j = 0; j < VE; ++j) add(z[j]);
    }
    const uint32_t mine = order_key(big);

    // CTA totals
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const Sums v{__shfl_xor_sync(kFull, u.r, o), __shfl_xor_sync(kFull, u.s, o), __shfl_xor_sync(kFull, u.t, o)};
        u = join(u, v);
        count += __shfl_xor_sync(kFull, count, o);
        big = fmaxf(big, __shfl_xor_sync(kFull, big, o));
    }
    if (lane == 0) {
        sh.sums[warp] = u;
        sh.count[warp] = count;
        sh.big[warp] = big;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kW; ++w) {
            u = join(u, sh.sums[w]);
            count += sh.count[w];
            big = fmaxf(big, sh.big[w]);
        }
        sh.total = u;
        sh.total_count = count;
        sh.total_big = big;
    }
    if (a.n_top > 0) slice_top<F32>(sh, sl, mine, a.n_top);
    __syncthreads();
    if (cs > 1) {
        cluster_sync();
        if (rank_in == 0) {
            if (tid == 0) {
                for (int r = 1; r < cs; ++r) {
                    u = join(u, Sums{peer_f32(&sh.total.r, r), peer_f32(&sh.total.s, r), peer_f32(&sh.total.t, r)});
                    count += __float_as_int(peer_f32(&sh.total_count, r));
                    big = fmaxf(big, peer_f32(&sh.total_big, r));
                }
                sh.total = u;
                sh.total_count = count;
                sh.total_big = big;
            }
            const int n = cs * a.n_top;
            for (int i = tid; i < n; i += kT) sh.all[i] = peer_u64(&sh.top[i % a.n_top], i / a.n_top);
            __syncthreads();
            if (tid < kMaxTop) sh.top[tid] = 0;
            __syncthreads();
            place(sh.all, n, sh.top, a.n_top);
            __syncthreads();
        }
        cluster_sync();                    // no CTA leaves while the first reads it
        if (rank_in != 0) return;
    }
    u = sh.total;
    big = sh.total_big;
    const bool near = fabsf(u.r) <= kNear; // y against the reference, else against `big`
    if (!near && big > -INFINITY) {
        // A reference so large that the rounding of z c is no small shift of y any more, or no
        // logit above -1e30 / c: sums against the largest logit itself.
        float s = 0.0f, t = 0.0f;
        for (int i = tid; i < a.V; i += kT) {
            const float z = Vec<F32>::at(sl.row, i);
            if (z == -INFINITY) continue;
            const float y = max_nan((z - big) * c, kFar), e = ex2(y);
            s += e;
            t = fmaf(e, y, t);
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
        if (y < kFar && l2s == l2s)        // the factor log2(e) may overflow where scale does not
            return near ? fmaf(z, a.scale, -u.r * kLn2) : (z - big) * a.scale;
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
    // CTAs per row: as many as fill the SMs, no slice below 4 vectors a thread.
    int cs = 1;
    while (cs < 8 && static_cast<long long>(M) * cs * 2 <= dev->sm_count && V / (cs * 2) >= kT * (f32 ? 16 : 32)) cs *= 2;
    a.cs = cs;
    const void* fn = f32 ? reinterpret_cast<const void*>(&logprobs_kernel<true>)
                         : reinterpret_cast<const void*>(&logprobs_kernel<false>);
    void* args[] = {&a};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(M) * cs));
    cfg.blockDim = dim3(kT);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cs);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

}  // namespace dg
