// dg_logits.cu -- penalties for tokens that were used, biases and grammar masks on logits
// (dg_logits_adjust).
//
// A CTA takes a slice of one row's vocabulary and holds one 32-bit counter an entry of it in
// shared memory: how often the sequence has made the token, whether its prompt has it, whether a bias
// is given.  It reads the row's whole list of tokens (a few kilobytes, from L2) and counts
// those in its slice; copies the slice under the mask while the counts come in; and then
// computes the entries that were touched, each once -- whoever swaps a counter for zero has
// it, a biased one belongs to the first of its entries in the list -- from the logit as it came in.
// Counters count whole numbers, so their order does not matter; biases of one token are added
// in list order.  Without a mask and in place nothing but the touched entries is read or written.
// Bound: memory where there are many rows; for one row the chain of list, counters and patches.
#include "dg_internal.h"
#include "dg_common.cuh"

namespace dg {
namespace {

constexpr uint32_t kPrompt = 0x80000000u, kBiased = 0x40000000u, kTimes = 0x3fffffffu;

struct LogitsArgs {
    const uint8_t* in;
    uint8_t* out;
    long long ld, ld_out;                // elements
    dg_logits_edits e;
    int V, slice, slices;
    int copy;                            // out is another buffer
};

template <typename T>
struct Elem;

template <>
struct Elem<float> {
    static constexpr int kPer = 4;                         // per 16 bytes
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
    static __device__ __forceinline__ float none() { return __uint_as_float(0xff800000u); }
    // the elements whose bit is 0 become -inf
    static __device__ __forceinline__ void mask(uint4& v, uint32_t bits)
    {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = (bits >> j) & 1u ? w[j] : 0xff800000u;
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <>
struct Elem<uint16_t> {
    static constexpr int kPer = 8;
    static __device__ __forceinline__ float get(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
    static __device__ __forceinline__ uint16_t put(float v) { return f32_to_bf16_bits(v); }
    static __device__ __forceinline__ uint16_t none() { return 0xff80u; }
    static __device__ __forceinline__ void mask(uint4& v, uint32_t bits)
    {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (!((bits >> (2 * j)) & 1u)) w[j] = (w[j] & 0xffff0000u) | 0xff80u;
            if (!((bits >> (2 * j + 1)) & 1u)) w[j] = (w[j] & 0xffffu) | 0xff800000u;
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

__device__ __forceinline__ bool allowed(const int32_t* mask, int v)
{
    return !mask || ((static_cast<uint32_t>(mask[v >> 5]) >> (v & 31)) & 1u);
}

// The n mask bits of entries v, v + 1, ... (n <= 8, v + n <= V).
__device__ __forceinline__ uint32_t mask_bits(const int32_t* mask, int v, int n)
{
    if (!mask) return 0xffu;
    const int w = v >> 5, o = v & 31;
    const uint32_t lo = static_cast<uint32_t>(mask[w]);
    const uint32_t hi = o + n > 32 ? static_cast<uint32_t>(mask[w + 1]) : 0u;
    return __funnelshift_r(lo, hi, o);
}

// Slice [v0, v1) of a row from `in` to `out` under the mask; in place only what it changes.
template <typename T>
__device__ __forceinline__ void copy_slice(const T* in, T* out, const int32_t* mask, int v0, int v1, bool copy)
{
    constexpr int kPer = Elem<T>::kPer, kU = 4;
    const uintptr_t ai = reinterpret_cast<uintptr_t>(in + v0), ao = reinterpret_cast<uintptr_t>(out + v0);
    int head = v1 - v0;                                    // entries in front of the first whole vector
    if (((ai ^ ao) & 15u) == 0) head = min(head, static_cast<int>(((16u - (ai & 15u)) & 15u) / sizeof(T)));
    auto one = [&](int v) {
        const bool ok = allowed(mask, v);
        if (copy)
            out[v] = ok ? in[v] : Elem<T>::none();
        else if (!ok)
            out[v] = Elem<T>::none();
    };
    for (int v = v0 + threadIdx.x; v < v0 + head; v += blockDim.x) one(v);
    const int vb = v0 + head, nv = (v1 - vb) / kPer;
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < nv; i0 += kU * blockDim.x) {
        uint4 raw[kU];
        uint32_t bits[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = i0 + u * blockDim.x;
            bits[u] = (1u << kPer) - 1;
            if (i < nv) {
                if (copy) raw[u] = ld_stream_after(in + vb + i * kPer);
                bits[u] &= mask_bits(mask, vb + i * kPer, kPer);
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = i0 + u * blockDim.x;
            if (i >= nv) break;
            if (!copy) {
                if (bits[u] == (1u << kPer) - 1) continue;
                raw[u] = bits[u] ? *reinterpret_cast<const uint4*>(in + vb + i * kPer) : make_uint4(0, 0, 0, 0);
            }
            Elem<T>::mask(raw[u], bits[u]);
            *reinterpret_cast<uint4*>(out + vb + i * kPer) = raw[u];
        }
    }
    for (int v = vb + nv * kPer + threadIdx.x; v < v1; v += blockDim.x) one(v);
}

template <typename T>
__global__ void __launch_bounds__(512) logits_kernel(LogitsArgs a)
{
    extern __shared__ uint32_t count[];                    // [slice]
    pdl_launch_dependents();
    pdl_wait();
    const int m = static_cast<int>(blockIdx.x / a.slices);
    const int v0 = static_cast<int>(blockIdx.x % a.slices) * a.slice, v1 = min(a.V, v0 + a.slice);
    const T* in = reinterpret_cast<const T*>(a.in) + m * a.ld;
    T* out = reinterpret_cast<T*>(a.out) + m * a.ld_out;
    const int32_t* mask = a.e.mask ? a.e.mask + m * a.e.ld_mask : nullptr;
    int len = a.e.tokens ? a.e.n_tokens : 0, prompt = 0;
    if (len > 0 && a.e.lengths) len = max(0, min(len, a.e.lengths[m]));
    if (len > 0 && a.e.prompt_lengths) prompt = max(0, min(len, a.e.prompt_lengths[m]));
    const int32_t* tok = a.e.tokens + m * a.e.ld_tokens;
    const int nb = a.e.bias ? a.e.n_bias : 0;
    const int32_t* bid = a.e.bias_ids + static_cast<size_t>(m) * nb;
    const float* bias = a.e.bias + static_cast<size_t>(m) * nb;
    const bool touched = len > 0 || nb > 0;
    if (touched) {
        for (int i = threadIdx.x; i < v1 - v0; i += blockDim.x) count[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < len; i += blockDim.x) {
            const int v = tok[i];
            if (v < v0 || v >= v1) continue;
            if (i < prompt)
                atomicOr(&count[v - v0], kPrompt);
            else
                atomicAdd(&count[v - v0], 1u);
        }
        for (int i = threadIdx.x; i < nb; i += blockDim.x) {
            const int v = bid[i];
            if (v >= v0 && v < v1) atomicOr(&count[v - v0], kBiased);
        }
    }
    if (a.copy || mask) copy_slice(in, out, mask, v0, v1, a.copy != 0);
    if (!touched) return;
    __syncthreads();                                       // counters are complete, the copy is made
    const float rep = a.e.repetition ? a.e.repetition[m] : 1.0f, freq = a.e.frequency ? a.e.frequency[m] : 0.0f;
    const float pres = a.e.presence ? a.e.presence[m] : 0.0f;
    auto apply = [&](int v, uint32_t c, float add) {
        if (!allowed(mask, v)) return;
        float x = Elem<T>::get(in[v]);
        const uint32_t times = c & kTimes;
        if (a.e.repetition && (c & (kPrompt | kTimes))) x = x > 0.0f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
        if (times) {
            if (a.e.frequency) x = __fsub_rn(x, __fmul_rn(freq, static_cast<float>(times)));
            if (a.e.presence) x = __fsub_rn(x, pres);
        }
        if (c & kBiased) x = __fadd_rn(x, add);
        out[v] = Elem<T>::put(x);
    };
    for (int i = threadIdx.x; i < nb; i += blockDim.x) {
        const int v = bid[i];
        if (v < v0 || v >= v1) continue;
        bool first = true;
        float add = bias[i];
        for (int j = 0; j < i; ++j) first &= bid[j] != v;
        if (!first) continue;
        for (int j = i + 1; j < nb; ++j)
            if (bid[j] == v) add = __fadd_rn(add, bias[j]);
        apply(v, count[v - v0], add);
    }
    for (int i = threadIdx.x; i < len; i += blockDim.x) {
        const int v = tok[i];
        if (v < v0 || v >= v1 || (count[v - v0] & kBiased)) continue;
        const uint32_t c = atomicExch(&count[v - v0], 0u);
        if (c) apply(v, c, 0.0f);
    }
}

}  // namespace

dg_status launch_logits_adjust(const DeviceInfo* dev, const void* logits, bool f32, long long ld, void* out, long long ld_out,
                               const dg_logits_edits& e, int M, int V, cudaStream_t stream)
{
    LogitsArgs a{};
    a.in = static_cast<const uint8_t*>(logits);
    a.out = static_cast<uint8_t*>(out);
    a.ld = ld;
    a.ld_out = ld_out;
    a.e = e;
    a.V = V;
    a.copy = out != logits;
    const bool lists = (e.tokens && e.n_tokens > 0) || (e.bias && e.n_bias > 0);
    if (!a.copy && !e.mask && !lists) return DG_OK;        // nothing changes
    // Few rows are cut into more slices, down to 2048 entries, so that two CTAs come on every SM;
    // many rows into slices of 16384 (64 KB of counters, three CTAs an SM).
    int slice = 16384;
    while (slice > 2048 && static_cast<long long>(M) * ((V - 1) / slice + 1) < 2 * dev->sm_count) slice /= 2;
    a.slice = slice;
    a.slices = (V - 1) / slice + 1;
    const long long grid = static_cast<long long>(M) * a.slices;
    if (grid > 0x7fffffffll) return DG_ERR_UNSUPPORTED_SHAPE;
    const int threads = slice >= 8192 ? 512 : 256;
    const size_t smem = lists ? static_cast<size_t>(slice) * 4 : 0;
    const void* fn = f32 ? reinterpret_cast<const void*>(&logits_kernel<float>) : reinterpret_cast<const void*>(&logits_kernel<uint16_t>);
    if (occupancy(fn, threads, smem) < 1) return DG_ERR_UNSUPPORTED_SHAPE;
    void* args[] = {&a};
    if (launch_kernel(fn, static_cast<unsigned>(grid), static_cast<unsigned>(threads), smem, stream, args, Early::kNothing) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

}  // namespace dg
