// dg_logits.cu -- penalties for tokens that were used, biases and grammar masks on logits
// (dg_logits_adjust).
//
// Calls of 2^20 logits or more, and 2048 more for each entry that a row's lists have room for (the lengths are on the
// device), of which there are up to 8192, take two kernels.  The first streams the logits under the mask, a batch of
// 16-byte vectors a thread (in place it writes what the mask changes; without a mask it is left out).  The second
// edits the entries that the lists name, a CTA a row: it counts the row's tokens in a hash table in shared memory --
// how often the sequence has made each, whether its prompt has it, whether a bias is given -- and then edits each
// entry once, from the logit as it came in.  The table has more slots than the lists have entries, so it never fills
// up.  Smaller calls, and longer lists, take one kernel: a CTA a slice of a row's vocabulary, which it streams under
// the mask, with a counter for every entry of the slice; every slice reads the whole list.  Counters count whole
// numbers, so their order does not matter; the biases of one token are added in list order, by the warp that has its
// first place.
// Measured with rows of 248320 bf16, lists of up to 4096 tokens, 64 biases and a mask, one kernel / two: 1 row 5.6 /
// 16.1 us, 8 rows 10.5 / 17.5, 32 rows 20.1 / 20.7, 64 rows 38.1 / 28.2, 256 rows 105 / 61; with 200 tokens 4 rows 4.8 /
// 5.2, 8 rows 7.9 / 6.4; 64 rows of 64000 with 1000 tokens 12.9 / 10.8, 32 rows 9.7 / 10.2.  Of the 61 the stream is 41
// (its bytes 39.5): memory binds it, a chain of list, counters and edits the rest and the small calls.  fp32: 8 rows
// 12.7, 64 rows 38.1, 256 rows 97.3.  Buffers wider than their lists cost: 256 rows of up to 1000 tokens in 32768 columns
// 126, in a view of 1000 54.  (A CTA a row for all of them, the table by the row's own length, longer lists by
// counters over one range of the vocabulary after the other: 62, but 403 where the rows are full, 238 by slices.)
#include "dg_internal.h"
#include "dg_common.cuh"

namespace dg {
namespace {

constexpr uint32_t kPrompt = 0x80000000u, kBiased = 0x40000000u, kTimes = 0x3fffffffu;
constexpr int kThreads = 512;
constexpr int kU = 4;                    // most 16-byte vectors of logits a thread streams
constexpr int kHeld = 8;                 // loads of a list, or of entries to edit, a thread has in flight
constexpr int kListed = 8192;            // longest lists that the hash table takes
constexpr int kFree = -1;                // no token's id

struct LogitsArgs {
    const uint8_t* in;
    uint8_t* out;
    long long ld, ld_out;                // elements
    dg_logits_edits e;
    int V, slice, slices;
    int copy;                            // out is another buffer
    int slots;                           // counters: of the hash table (a power of two), or of a slice
    int stream;                          // logits are copied, or masked
};

template <typename T>
struct Elem;

template <>
struct Elem<float> {
    static constexpr int kPer = 4;                         // entries per 16 bytes
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
    static __device__ __forceinline__ float none() { return __uint_as_float(0xff800000u); }
    // entry j of a vector
    static __device__ __forceinline__ float at(const uint4& v, int j)
    {
        return __uint_as_float(j < 2 ? (j ? v.y : v.x) : (j == 2 ? v.z : v.w));
    }
    static __device__ __forceinline__ void set(uint4& v, int j, float x)
    {
        const uint32_t b = __float_as_uint(x);
        v = make_uint4(j == 0 ? b : v.x, j == 1 ? b : v.y, j == 2 ? b : v.z, j == 3 ? b : v.w);
    }
    // the entries whose bit is 0 become -inf
    static __device__ __forceinline__ void mask(uint4& v, uint32_t bits)
    {
        v = make_uint4(bits & 1u ? v.x : 0xff800000u, bits & 2u ? v.y : 0xff800000u, bits & 4u ? v.z : 0xff800000u,
                       bits & 8u ? v.w : 0xff800000u);
    }
};

template <>
struct Elem<uint16_t> {
    static constexpr int kPer = 8;
    static __device__ __forceinline__ float get(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
    static __device__ __forceinline__ uint16_t put(float v) { return f32_to_bf16_bits(v); }
    static __device__ __forceinline__ uint16_t none() { return 0xff80u; }
    static __device__ __forceinline__ uint16_t at(const uint4& v, int j)
    {
        const uint32_t w = j < 4 ? (j < 2 ? v.x : v.y) : (j < 6 ? v.z : v.w);
        return static_cast<uint16_t>(j & 1 ? w >> 16 : w);
    }
    static __device__ __forceinline__ void set(uint4& v, int j, uint16_t x)
    {
        const uint32_t b = x, sel = j & 1 ? 0x5410u : 0x3254u;             // the new half above, or below
        auto put = [&](uint32_t w) { return __byte_perm(w, b, sel); };
        v = make_uint4(j >> 1 == 0 ? put(v.x) : v.x, j >> 1 == 1 ? put(v.y) : v.y, j >> 1 == 2 ? put(v.z) : v.z,
                       j >> 1 == 3 ? put(v.w) : v.w);
    }
    static __device__ __forceinline__ void mask(uint4& v, uint32_t bits)
    {
        auto two = [](uint32_t w, uint32_t b) {
            const uint32_t keep = (b & 1u ? 0x0000ffffu : 0u) | (b & 2u ? 0xffff0000u : 0u);
            return (w & keep) | (0xff80ff80u & ~keep);
        };
        v = make_uint4(two(v.x, bits), two(v.y, bits >> 2), two(v.z, bits >> 4), two(v.w, bits >> 6));
    }
};

// The mask bits of entries v, v + 1, ..., v + 7, of which those in [0, V) count.  Both words are loaded, from
// places that are there: behind a condition they would be waited for at once (256 x 248320: 26 us).
__device__ __forceinline__ uint32_t mask_bits(const int32_t* mask, int v, int last_word)
{
    const int w = v >> 5;
    return __funnelshift_r(static_cast<uint32_t>(mask[max(0, min(w, last_word))]),
                           static_cast<uint32_t>(mask[min(max(w + 1, 0), last_word)]), v & 31);
}

// What a row's edits are: the parts that every entry shares.
struct Row {
    bool has_rep, has_freq, has_pres;
    float rep, freq, pres;

    __device__ float edit(float x, uint32_t c, float add) const
    {
        const uint32_t times = c & kTimes;
        if (has_rep && (c & (kPrompt | kTimes))) x = x > 0.0f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
        if (times) {
            if (has_freq) x = __fsub_rn(x, __fmul_rn(freq, static_cast<float>(times)));
            if (has_pres) x = __fsub_rn(x, pres);
        }
        return c & kBiased ? __fadd_rn(x, add) : x;
    }
};

// A slice of a row.  Slices begin on the logits' 16-byte boundaries: entry v of the row is entry v + shift of
// the slices'.  (The last slice of a row may be empty: a shift moves the row's end.)
template <typename T>
struct Slice {
    const T* in;
    T* out;
    const int32_t* mask;
    int m, first, v0, v1;

    __device__ explicit Slice(const LogitsArgs& a)
    {
        m = static_cast<int>(blockIdx.x / a.slices);
        in = reinterpret_cast<const T*>(a.in) + m * a.ld;
        out = reinterpret_cast<T*>(a.out) + m * a.ld_out;
        mask = a.e.mask ? a.e.mask + m * a.e.ld_mask : nullptr;
        first = static_cast<int>(blockIdx.x % a.slices) * a.slice - static_cast<int>((reinterpret_cast<uintptr_t>(in) & 15u) / sizeof(T));
        v0 = max(0, first);
        v1 = min(a.V, first + a.slice);
    }
};

// The vectors of a slice that a thread streams, loaded (begin) and stored under the mask (end).
template <typename T>
struct Stream {
    static constexpr int kPer = Elem<T>::kPer;
    static constexpr uint32_t kAll = (1u << kPer) - 1;
    uint4 raw[kU];
    uint32_t bits[kU];

    __device__ __forceinline__ int entry(const Slice<T>& s, int u) const
    {
        return s.first + (static_cast<int>(threadIdx.x) + u * kThreads) * kPer;
    }

    __device__ __forceinline__ void begin(const Slice<T>& s, int V)
    {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int v = entry(s, u);
            if (v >= s.v0 && v + kPer <= s.v1) raw[u] = ld_stream_after(s.in + v);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) bits[u] = s.mask ? mask_bits(s.mask, entry(s, u), (V - 1) >> 5) & kAll : kAll;
    }

    __device__ __forceinline__ void end(const Slice<T>& s, bool copy)
    {
        const bool aligned = ((reinterpret_cast<uintptr_t>(s.out) ^ reinterpret_cast<uintptr_t>(s.in)) & 15u) == 0;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int v = entry(s, u);
            if (v >= s.v1 || v + kPer <= s.v0 || (!copy && bits[u] == kAll)) continue;
            if (v < s.v0 || v + kPer > s.v1) {             // the row begins or ends inside
#pragma unroll 1
                for (int j = 0; j < kPer; ++j)
                    if (v + j >= s.v0 && v + j < s.v1) s.out[v + j] = (bits[u] >> j) & 1u ? s.in[v + j] : Elem<T>::none();
                continue;
            }
            if (bits[u] != kAll) Elem<T>::mask(raw[u], bits[u]);
            if (aligned)
                *reinterpret_cast<uint4*>(s.out + v) = raw[u];
            else
#pragma unroll 1
                for (int j = 0; j < kPer; ++j) s.out[v + j] = Elem<T>::at(raw[u], j);
        }
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) logits_mask_kernel(LogitsArgs a)
{
    pdl_wait();
    // Behind the wait: when the editing kernel begins, what the lists hold has been written.
    pdl_launch_dependents();
    const Slice<T> s(a);
    if (s.v0 >= s.v1) return;
    Stream<T> stream;
    stream.begin(s, a.V);
    stream.end(s, a.copy != 0);
}

// The editing kernel.  HASH: a CTA a row, behind logits_mask_kernel if there is anything to stream; else a CTA a slice,
// which streams it.  Shared memory: the counters [slots], with the hash table its keys [slots]; then the row's biases:
// ids, values, sums, slots [n_bias].
template <typename T, bool HASH>
__global__ void __launch_bounds__(kThreads) logits_edit_kernel(LogitsArgs a)
{
    extern __shared__ __align__(16) uint32_t count[];
    int32_t* key = reinterpret_cast<int32_t*>(count + a.slots);
    const int nb = a.e.bias ? a.e.n_bias : 0, lane = threadIdx.x & 31;
    int32_t* ids = key + (HASH ? a.slots : 0);
    float* values = reinterpret_cast<float*>(ids + nb);
    float* sums = values + nb;
    int32_t* lead = reinterpret_cast<int32_t*>(sums + nb);             // the slot of a token's first bias, else -1
    for (int i = threadIdx.x; i < a.slots / 4; i += kThreads) {
        reinterpret_cast<uint4*>(count)[i] = make_uint4(0, 0, 0, 0);
        if constexpr (HASH) reinterpret_cast<int4*>(key)[i] = make_int4(kFree, kFree, kFree, kFree);
    }
    // Behind the first kernel, which lets this one begin after its own wait, the lists are there already.
    const bool behind = HASH && a.stream;
    if (!behind) pdl_wait();
    pdl_launch_dependents();
    const Slice<T> s(a);                                               // (HASH: the row)
    const int m = s.m, v0 = HASH ? 0 : s.v0, v1 = HASH ? a.V : s.v1;
    if (v0 >= v1) return;
    Stream<T> stream;
    if (!HASH && a.stream) stream.begin(s, a.V);
    int len = a.e.tokens ? a.e.n_tokens : 0, prompt = 0;
    if (len > 0 && a.e.lengths) len = max(0, min(len, ld_cg_s32(a.e.lengths + m)));
    if (len > 0 && a.e.prompt_lengths) prompt = max(0, min(len, ld_cg_s32(a.e.prompt_lengths + m)));
    for (int i = threadIdx.x; i < nb; i += kThreads) {
        ids[i] = ld_cg_s32(a.e.bias_ids + static_cast<size_t>(m) * nb + i);
        values[i] = ld_cg_f32(a.e.bias + static_cast<size_t>(m) * nb + i);
    }
    const Row row{a.e.repetition != nullptr, a.e.frequency != nullptr, a.e.presence != nullptr,
                  a.e.repetition ? ld_cg_f32(a.e.repetition + m) : 1.0f, a.e.frequency ? ld_cg_f32(a.e.frequency + m) : 0.0f,
                  a.e.presence ? ld_cg_f32(a.e.presence + m) : 0.0f};
    __syncthreads();
    // The slot of an entry in [v0, v1), taken if it has none (there are more slots than entries of the lists).
    auto slot = [&](int v) {
        if constexpr (!HASH) {
            return v - s.first;
        } else {
            uint32_t h = (static_cast<uint32_t>(v) * 2654435761u) >> 16;           // (multiplicative hashing)
            for (;; ++h) {
                h &= static_cast<uint32_t>(a.slots - 1);
                int was = *reinterpret_cast<volatile int32_t*>(key + h);
                if (was == kFree) was = atomicCAS(key + h, kFree, v);
                if (was == kFree || was == v) return static_cast<int>(h);
            }
        }
    };
    const int32_t* tok = a.e.tokens + m * a.e.ld_tokens;
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < len; i0 += kHeld * kThreads) {
        int v[kHeld];
#pragma unroll
        for (int u = 0; u < kHeld; ++u) v[u] = i0 + u * kThreads < len ? ld_cg_s32(tok + i0 + u * kThreads) : -1;
#pragma unroll
        for (int u = 0; u < kHeld; ++u) {
            if (v[u] < v0 || v[u] >= v1) continue;
            uint32_t* c = count + slot(v[u]);
            if (i0 + u * kThreads < prompt)
                atomicOr(c, kPrompt);
            else
                atomicAdd(c, 1u);
        }
    }
    // A warp a bias: it looks the whole list over, and adds up if its place is its token's first.
    for (int i = threadIdx.x >> 5; i < nb; i += kThreads / 32) {
        const int v = ids[i];
        bool leads = v >= v0 && v < v1;
        float add = values[i];
        for (int j0 = 0; j0 < nb && leads; j0 += 32) {
            unsigned same = __ballot_sync(kFull, j0 + lane < nb && ids[j0 + lane] == v);
            for (; same; same &= same - 1) {
                const int j = j0 + __ffs(same) - 1;
                if (j < i) leads = false;
                if (j > i) add = __fadd_rn(add, values[j]);
            }
        }
        if (lane == 0) {
            lead[i] = leads ? slot(v) : -1;
            sums[i] = add;
            if (leads) atomicOr(count + lead[i], kBiased);
        }
        __syncwarp();
    }
    if (!HASH && a.stream) stream.end(s, a.copy != 0);
    __syncthreads();                                       // counters are complete, the slice is streamed
    if (behind) pdl_wait();                                // the first kernel's writes are made
    for (int i = threadIdx.x; i < nb; i += kThreads) {
        if (lead[i] < 0) continue;
        const int v = ids[i];
        if (s.mask && !((static_cast<uint32_t>(s.mask[v >> 5]) >> (v & 31)) & 1u)) continue;
        s.out[v] = Elem<T>::put(row.edit(Elem<T>::get(s.in[v]), count[lead[i]], sums[i]));
    }
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < a.slots; i0 += kHeld * kThreads) {
        uint32_t c[kHeld], word[kHeld];
        int v[kHeld];
        T x[kHeld];
#pragma unroll
        for (int u = 0; u < kHeld; ++u) {
            const int i = i0 + u * kThreads;
            c[u] = i < a.slots ? count[i] : 0u;
            if (c[u] & kBiased) c[u] = 0;
            v[u] = c[u] ? (HASH ? key[i] : s.first + i) : v0;          // (an entry that is there)
            x[u] = s.in[v[u]];
            word[u] = s.mask ? static_cast<uint32_t>(s.mask[v[u] >> 5]) : kFull;
        }
#pragma unroll
        for (int u = 0; u < kHeld; ++u)
            if (c[u] && ((word[u] >> (v[u] & 31)) & 1u)) s.out[v[u]] = Elem<T>::put(row.edit(Elem<T>::get(x[u]), c[u], 0.0f));
    }
}

template <typename T>
const void* edit_fn(bool hash)
{
    return hash ? reinterpret_cast<const void*>(&logits_edit_kernel<T, true>) : reinterpret_cast<const void*>(&logits_edit_kernel<T, false>);
}

dg_status launch(const void* fn, LogitsArgs a, int M, size_t smem, cudaStream_t stream)
{
    const long long grid = static_cast<long long>(M) * a.slices;
    if (grid > 0x7fffffffll || occupancy(fn, kThreads, smem) < 1) return DG_ERR_UNSUPPORTED_SHAPE;
    void* args[] = {&a};
    if (launch_kernel(fn, static_cast<unsigned>(grid), kThreads, smem, stream, args, Early::kNothing) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
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
    a.stream = a.copy || e.mask;
    const int listed = (e.tokens ? e.n_tokens : 0) + (e.bias ? e.n_bias : 0);
    if (listed == 0 && !a.stream) return DG_OK;            // nothing changes
    const bool hash = listed <= kListed && static_cast<long long>(M) * V >= (1 << 20) + 2048ll * listed;
    // A slice is what a CTA's threads stream: 512 threads with four vectors each, fewer for few rows, so that two
    // CTAs come on every SM.  (A row's shift moves its end by up to per - 1 entries.)
    const int per = f32 ? Elem<float>::kPer : Elem<uint16_t>::kPer;
    int vectors = kU;
    const auto slices = [&] { return (static_cast<long long>(V) + per - 2) / (kThreads * vectors * per) + 1; };
    while (vectors > 1 && M * slices() < 2 * dev->sm_count) vectors /= 2;
    a.slice = kThreads * vectors * per;
    a.slices = static_cast<int>(slices());
    if ((a.stream && hash) || listed == 0) {
        const void* fn = f32 ? reinterpret_cast<const void*>(&logits_mask_kernel<float>) : reinterpret_cast<const void*>(&logits_mask_kernel<uint16_t>);
        const dg_status st = launch(fn, a, M, 0, stream);
        if (st != DG_OK || listed == 0) return st;
    }
    size_t smem = static_cast<size_t>(e.n_bias) * 16;
    if (hash) {
        a.slices = 1;
        a.slots = 512;
        while (2 * a.slots < 3 * listed) a.slots *= 2;
        smem += static_cast<size_t>(a.slots) * 8;
    } else {
        a.slots = a.slice;
        smem += static_cast<size_t>(a.slots) * 4;
    }
    return launch(f32 ? edit_fn<float>(hash) : edit_fn<uint16_t>(hash), a, M, smem, stream);
}

}  // namespace dg
