// dg_api.cu -- the libdecodegemm C ABI: argument checks, kernel choice, launch.
//
// Nothing here allocates device memory or synchronises the host with a stream
// (dg_device_status excepted, which exists for tests and health checks).
#include <atomic>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <set>
#include <thread>
#include <tuple>
#include <utility>

#include "dg_cc_bulk.cuh"
#include "dg_cc_dense.cuh"
#include "dg_fp4.cuh"
#include "dg_i8.cuh"
#include "dg_internal.h"
#include "dg_moe.cuh"

namespace dg {

namespace {

std::mutex g_mu;
DeviceInfo g_dev[64];
bool g_dev_ok[64];
// Both per device: a kernel's attributes and occupancy belong to the device it runs on.
std::map<std::tuple<int, const void*, int, size_t>, int> g_occ;
std::map<std::pair<int, const void*>, bool> g_attr;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

const DeviceInfo* current_device(dg_status* err)
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        if (err) *err = DG_ERR_NO_DEVICE;
        return nullptr;
    }
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (g_dev_ok[dev]) return &g_dev[dev];
    }
    dg_status s = dg_init(dev);
    if (s != DG_OK) {
        if (err) *err = s;
        return nullptr;
    }
    std::lock_guard<std::mutex> lk(g_mu);
    return &g_dev[dev];
}

namespace {
std::atomic<int> g_launch_flags{DG_LAUNCH_PDL};
}

namespace {

thread_local int t_check_only = 0;

// Streams on which weights were written and no kernel that reads weights early has been
// launched since.  (The default streams go by device, the per-thread one by thread too.)
using StreamKey = std::tuple<int, uintptr_t, std::thread::id>;
std::mutex g_written_mu;
std::set<StreamKey> g_written;
std::atomic<int> g_written_n{0};

StreamKey stream_key(cudaStream_t s)
{
    if (s == nullptr) s = cudaStreamLegacy;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) cudaGetLastError();
    return StreamKey(dev, reinterpret_cast<uintptr_t>(s),
                     s == cudaStreamPerThread ? std::this_thread::get_id() : std::thread::id());
}

}  // namespace

void weights_written(cudaStream_t stream)
{
    std::lock_guard<std::mutex> lk(g_written_mu);
    g_written.insert(stream_key(stream));
    g_written_n = static_cast<int>(g_written.size());
}

cudaError_t launch_ordered(cudaLaunchConfig_t cfg, cudaLaunchAttribute* attr, unsigned n, const void* fn, void** args,
                           Early early)
{
    bool pdl = (g_launch_flags.load(std::memory_order_relaxed) & DG_LAUNCH_PDL) != 0;
    bool written = false;
    if (early == Early::kWeights && g_written_n.load() != 0) {
        std::lock_guard<std::mutex> lk(g_written_mu);
        written = g_written.count(stream_key(cfg.stream)) != 0;
    }
    pdl = pdl && !written;
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = n + 1;
    const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
    if (written && e == cudaSuccess) {
        std::lock_guard<std::mutex> lk(g_written_mu);
        g_written.erase(stream_key(cfg.stream));
        g_written_n = static_cast<int>(g_written.size());
    }
    return e;
}

CheckOnly::CheckOnly() { ++t_check_only; }
CheckOnly::~CheckOnly() { --t_check_only; }

cudaError_t launch_kernel(const void* fn, unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                          void** args, Early early)
{
    if (t_check_only) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    return launch_ordered(cfg, attr, 0, fn, args, early);
}

cudaError_t launch_kernel_cooperative(const void* fn, unsigned grid, unsigned block, size_t smem,
                                      cudaStream_t stream, void** args)
{
    if (t_check_only) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    return launch_ordered(cfg, attr, 1, fn, args, Early::kWeights);
}

int occupancy(const void* fn, int threads, size_t smem)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        dev = 0;
    }
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_attr[std::make_pair(dev, fn)]) {
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxDynSmem));
        g_attr[std::make_pair(dev, fn)] = true;
    }
    auto key = std::make_tuple(dev, fn, threads, smem);
    auto it = g_occ.find(key);
    if (it != g_occ.end()) return it->second;
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, smem) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    g_occ[key] = n;
    return n;
}

void default_choice(dg_op op, int M, int N, int K, dg_choice* out)
{
    std::memset(out, 0, sizeof *out);
    out->variant = DG_VAR_CC_WARP;
    switch (op) {
    case DG_OP_GEMV_BF16:
    case DG_OP_GATE_UP_SILU: {
        const bool lin = op == DG_OP_GEMV_BF16;
        if (M >= kTcMinRows || M > (lin ? kMwMaxRowsLinear : kMwMaxRowsGateUp)) {
            out->variant = DG_VAR_TC;      // a real dense contraction: tcgen05 tiles
            break;
        }
        if (M >= (lin ? kMwMinRowsLinear : kMwMinRowsGateUp)) {
            out->variant = DG_VAR_MMA;     // warp-level tensor cores, geometry derived at launch
            break;
        }
        // Rows per warp [0], warps per CTA [1] and K-split warps [3] as dg_sweep
        // measured them on GB300 for one and two tokens: long rows with few row groups
        // share each group's K segments between warps; many short rows do not.
        const long rows = op == DG_OP_GATE_UP_SILU ? 2L * N : static_cast<long>(N);
        const int nseg = (K + kSeg - 1) / kSeg;
        int R, wpc, ks;
        if (op == DG_OP_GATE_UP_SILU) {
            R = 2;
            wpc = M <= 1 ? 4 : 8;
            ks = M <= 1 ? 4 : 1;
        } else if (rows >= 32768) {
            R = M <= 1 ? 1 : 2;
            wpc = 8;
            ks = 1;
        } else if (rows >= 12288) {
            R = 4;
            wpc = 4;
            ks = M <= 1 ? 4 : 2;
        } else if (rows >= 8192) {
            R = 2;
            wpc = M <= 1 ? 4 : 8;
            ks = 1;
        } else {
            R = (M <= 1 && K <= 4096) ? 2 : 4;
            wpc = 8;
            ks = 2;
        }
        while (ks > 1 && nseg < ks) ks /= 2;          // no warp without a segment
        out->params[0] = R;
        out->params[1] = wpc;
        out->params[3] = ks > 1 ? ks : 0;
        break;
    }
    case DG_OP_HEAD_FP8_ARGMAX:
        if (M >= kTcHeadMinRows && K <= kTcHeadMaxK) {
            out->variant = DG_VAR_TC;      // fp8 MMA on split activations
            break;
        }
        // measured on GB300 (dg_sweep over the 248320 x 4096 head)
        out->params[0] = M == 4 ? 4 : (M <= 3 ? 8 : 4);
        out->params[1] = M <= 4 ? 4 : 8;
        break;
    // MoE: [1] warps per CTA, [3] N-tile (W1: gate/up columns, W2: output rows),
    // [4] pairs per pass -- the GB300 dg_sweep picks per row bucket.
    case DG_OP_MOE_W1:
        if (M >= kTcMoeW1MinRows) {
            out->variant = DG_VAR_TC;
            break;
        }
        if (M <= kMoeRangeMaxRowsW1) {         // one row range of every expert per CTA
            out->params[0] = 4;
            out->params[1] = 4;
            out->params[4] = 2;
            out->params[5] = kMoeOrderRange;
            break;
        }
        out->params[0] = 4;
        out->params[1] = 8;
        out->params[3] = M <= 1 ? 32 : (M <= 2 ? 64 : 0);
        out->params[4] = M <= 2 ? 4 : 2;
        break;
    case DG_OP_MOE_W2:
        if (M >= kTcMoeW2MinRows) {
            out->variant = DG_VAR_TC;
            break;
        }
        if (M <= kMoeRangeMaxRowsW2) {
            out->params[0] = 4;
            out->params[1] = 8;
            out->params[4] = 2;
            out->params[5] = kMoeOrderRange;
            break;
        }
        out->params[0] = 4;
        out->params[1] = M <= 2 ? 8 : 4;
        out->params[3] = M <= 1 ? 64 : (M <= 2 ? 128 : (M <= 4 ? 0 : 64));
        out->params[4] = M <= 1 ? 1 : 2;
        break;
    case DG_OP_GEMV_A8W8:
        out->variant = DG_VAR_TC;          // fp8 MMA on the quantised activations
        // Measured on GB300 (32768x1024, 8192x4096): the fused quantisation ties with a
        // quantisation launch of its own up to 16 rows; beyond, every CTA re-quantising
        // all rows costs more than one extra launch (12.7 -> 9.7 us at 32 rows).
        out->params[1] = M > 16 ? 1 : 0;
        break;
    case DG_OP_GEMV_A4W4:
        out->variant = DG_VAR_TC;          // block-scaled e2m1 MMA
        break;
    case DG_OP_GEMV_I8:
        // dp4a for few tokens whose codes fit in shared memory, else integers as binary16
        out->variant = i8_cc_takes(M, K) ? DG_VAR_CC_WARP : DG_VAR_TC;
        break;
    default:
        break;
    }
}

#ifndef DG_BUILD_ID
#define DG_BUILD_ID "dev"
#endif

const char* build_id() { return DG_BUILD_ID; }

}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_init(int device)
{
    if (device < 0 || device >= 64) return DG_ERR_INVALID_ARG;
    if (cudaSetDevice(device) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_NO_DEVICE;
    }
    cudaDeviceProp prop;
    if (cudaGetDeviceProperties(&prop, device) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_NO_DEVICE;
    }
    if (prop.major != 10 || prop.minor != 3) {
        std::fprintf(stderr, "libdecodegemm: device %d is sm_%d%d; this build runs on sm_103 only\n",
                     device, prop.major, prop.minor);
        return DG_ERR_NO_DEVICE;
    }
    DeviceInfo info;
    info.device = device;
    info.sm_count = prop.multiProcessorCount;
    info.cc_major = prop.major;
    info.cc_minor = prop.minor;
    info.max_smem_optin = static_cast<int>(prop.sharedMemPerBlockOptin);
    cudaDriverGetVersion(&info.driver_version);
    cudaRuntimeGetVersion(&info.runtime_version);
    std::snprintf(info.name, sizeof info.name, "%s", prop.name);
    bool first = false;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        first = !g_dev_ok[device];
        g_dev[device] = info;
        g_dev_ok[device] = true;
    }
    if (first) {
        tc_capacity_init(&info);
        const char* path = std::getenv("DG_TABLE");
        if (path && *path) dg_table_load(path);   // refusal prints one line; defaults stay
    }
    return DG_OK;
}

const char* dg_status_str(dg_status s)
{
    switch (s) {
    case DG_OK: return "ok";
    case DG_ERR_INVALID_ARG: return "invalid argument";
    case DG_ERR_ALIGNMENT: return "pointer not 16-byte aligned";
    case DG_ERR_UNSUPPORTED_SHAPE: return "unsupported shape";
    case DG_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
    case DG_ERR_CUDA: return "CUDA error";
    case DG_ERR_TABLE_REFUSED: return "shape table refused";
    case DG_ERR_NO_DEVICE: return "no usable sm_103 device";
    case DG_ERR_BAD_VARIANT: return "bad kernel variant";
    default: return "unknown status";
    }
}

size_t dg_workspace_bytes(dg_op op, int M, int N, int K, int topk)
{
    (void)K;
    size_t b = kWsData;
    switch (op) {
    case DG_OP_GEMV_BF16:
        if (M > 0 && N > 0 && K > 0) b = tc_workspace_bytes(M, N, K);
        break;
    case DG_OP_GATE_UP_SILU:
        if (M > 0 && N > 0 && K > 0) b = tc_workspace_bytes(M, 2 * N, K);
        break;
    case DG_OP_HEAD_FP8_ARGMAX:
        b += kHeadPartialBytes;
        break;
    case DG_OP_MOE_W2:
        if (M > 0 && topk > 0 && N > 0) b += moe_terms_bytes(M, topk, N);
        break;
    case DG_OP_GEMV_A8W8:
        if (M > 0 && K > 0) b = a8_workspace_bytes(M, K);
        break;
    case DG_OP_GEMV_A4W4:
        if (M > 0 && K > 0) b = a4_workspace_bytes(M, K);
        break;
    case DG_OP_GEMV_I8:
        if (M > 0 && K > 0) b = i8_workspace_bytes(M, K);
        break;
    default:
        break;
    }
    return b;
}

dg_status dg_device_status(const void* ws, int32_t* host_out, dg_stream_t stream)
{
    if (!ws || !host_out) return DG_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cudaMemcpyAsync(host_out, static_cast<const uint8_t*>(ws) + kWsStatus, sizeof(int32_t),
                        cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

dg_status dg_set_launch_flags(unsigned flags)
{
    if (flags & ~static_cast<unsigned>(DG_LAUNCH_PDL)) return DG_ERR_INVALID_ARG;
    g_launch_flags.store(static_cast<int>(flags));
    return DG_OK;
}

unsigned dg_launch_flags(void) { return static_cast<unsigned>(g_launch_flags.load()); }

dg_status dg_device_status_clear(void* ws, dg_stream_t stream)
{
    if (!ws) return DG_ERR_INVALID_ARG;
    if (cudaMemsetAsync(static_cast<uint8_t*>(ws) + kWsStatus, 0, sizeof(int32_t),
                        reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

}  // extern "C"

namespace dg {
namespace {

dg_status resolve_choice(dg_op op, int M, int N, int K, const dg_choice* in, dg_choice* out)
{
    if (in && in->variant != DG_VAR_DEFAULT) {
        *out = *in;
        return DG_OK;
    }
    return dg_select(op, M, N, K, out);
}

// Bulk-staged variant: one (or two) persistent CTAs per SM, a deep shared-memory ring.
dg_status launch_bulk(dg_op op, const DeviceInfo* dev, const dg_choice& c, DenseArgs a, int M, size_t ws_bytes,
                      cudaStream_t stream)
{
    const int esz = (op == DG_OP_HEAD_FP8_ARGMAX) ? 1 : 2;
    const int rw = (op == DG_OP_GATE_UP_SILU) ? 2 : 1;
    const int cps = c.params[2] > 0 ? c.params[2] : 1;
    if (c.params[0] != 0 || c.params[1] < 0 || c.params[1] > 32 || c.params[1] == 1 || cps > 2)
        return DG_ERR_BAD_VARIANT;
    int mt_max = static_cast<int>(kXsBudget / (static_cast<size_t>(a.K) * 2));
    if (mt_max > 8) mt_max = 8;
    if (mt_max < 1) return DG_ERR_UNSUPPORTED_SHAPE;
    if (op == DG_OP_HEAD_FP8_ARGMAX && M > mt_max) return DG_ERR_UNSUPPORTED_SHAPE;
    const size_t stage = static_cast<size_t>(kBulkConsumers) * rw * kSeg * esz;
    const size_t budget = (cps == 1 ? kMaxDynSmem : kMaxDynSmem / 2 - 8 * 1024);
    for (int t0 = 0; t0 < M; t0 += mt_max) {
        const int mt = (M - t0 < mt_max) ? M - t0 : mt_max;
        const void* fn = op == DG_OP_GEMV_BF16      ? bulk_kernel_gemv(mt)
                         : op == DG_OP_GATE_UP_SILU ? bulk_kernel_gateup(mt)
                                                    : bulk_kernel_head(mt);
        if (!fn) return DG_ERR_BAD_VARIANT;
        const size_t xbytes = (static_cast<size_t>(mt) * a.K * 2 + 127) / 128 * 128;
        if (xbytes + 2 * stage + 64 > budget) return DG_ERR_UNSUPPORTED_SHAPE;
        int stages = c.params[1];
        const int fit = static_cast<int>((budget - xbytes - 64) / (stage + 16));
        if (stages == 0) stages = fit < 32 ? fit : 32;
        if (stages < 2 || stages > fit) return DG_ERR_BAD_VARIANT;
        const size_t smem = xbytes + static_cast<size_t>(stages) * (stage + 16);
        const int occ = occupancy(fn, kBulkThreads, smem);
        if (occ < 1) return DG_ERR_UNSUPPORTED_SHAPE;
        const long long grid = static_cast<long long>(dev->sm_count) * (occ < cps ? occ : cps);
        if (op == DG_OP_HEAD_FP8_ARGMAX && ws_bytes < kWsData + static_cast<size_t>(grid) * cpow2(mt) * 8)
            return DG_ERR_WORKSPACE_TOO_SMALL;
        DenseArgs la = a;
        la.t0 = t0;
        void* args[] = {&la, &stages};
        if (launch_kernel(fn, static_cast<unsigned>(grid), kBulkThreads, smem, stream, args) !=
            cudaSuccess) {
            cudaGetLastError();
            return DG_ERR_CUDA;
        }
    }
    return DG_OK;
}

// Launch the dense CUDA-core family over token chunks.
dg_status launch_dense(dg_op op, const DeviceInfo* dev, const dg_choice& c, DenseArgs a, int M,
                       size_t ws_bytes, cudaStream_t stream)
{
    if (c.variant == DG_VAR_CC_BULK) return launch_bulk(op, dev, c, a, M, ws_bytes, stream);
    const int esz = (op == DG_OP_HEAD_FP8_ARGMAX) ? 1 : 2;
    (void)esz;
    int R = c.params[0] > 0 ? c.params[0] : 4;
    const int wpc = c.params[1] > 0 ? c.params[1] : 8;
    const int cap = c.params[2];
    const int ks = c.params[3] > 0 ? c.params[3] : 1;
    if ((R != 1 && R != 2 && R != 4 && R != 8) || wpc < 1 || wpc > 8 || cap < 0)
        return DG_ERR_BAD_VARIANT;
    if ((ks != 1 && ks != 2 && ks != 4 && ks != 8) || wpc % ks != 0) return DG_ERR_BAD_VARIANT;
    if (op == DG_OP_GATE_UP_SILU && R < 2) return DG_ERR_BAD_VARIANT;
    int mt_max = static_cast<int>(kXsBudget / (static_cast<size_t>(a.K) * 2));
    if (mt_max > 8) mt_max = 8;
    if (mt_max < 1) return DG_ERR_UNSUPPORTED_SHAPE;
    if (op == DG_OP_HEAD_FP8_ARGMAX && M > mt_max) return DG_ERR_UNSUPPORTED_SHAPE;
    for (int t0 = 0; t0 < M; t0 += mt_max) {
        const int mt = (M - t0 < mt_max) ? M - t0 : mt_max;
        int r = R;
        while (r > 1 && r * cpow2(mt) > 32) r >>= 1;       // same arithmetic, fewer rows per warp
        if (op == DG_OP_GATE_UP_SILU && r < 2) return DG_ERR_UNSUPPORTED_SHAPE;
        const int kse = mt <= 2 ? ks : 1;                 // K-split kernels exist for 1-2 token chunks
        const void* fn = op == DG_OP_GEMV_BF16      ? dense_kernel_gemv(mt, r, kse > 1)
                         : op == DG_OP_GATE_UP_SILU ? dense_kernel_gateup(mt, r, kse > 1)
                                                    : dense_kernel_head(mt, r, kse > 1);
        if (!fn) return DG_ERR_BAD_VARIANT;
        const int threads = wpc * 32;
        const int slots = wpc / kse;                      // row groups per CTA round
        size_t smem = static_cast<size_t>(mt) * a.K * 2;
        if (kse > 1)                                      // segment partials of the K-split
            smem += static_cast<size_t>(slots) * ((a.K + kSeg - 1) / kSeg) * r * cpow2(mt) * 4;
        if (smem > kMaxDynSmem) return DG_ERR_UNSUPPORTED_SHAPE;
        int occ = occupancy(fn, threads, smem);
        if (occ < 1) return DG_ERR_UNSUPPORTED_SHAPE;
        if (cap > 0 && occ > cap) occ = cap;
        DenseArgs la = a;
        la.t0 = t0;
        la.groups = (a.N + r - 1) / r;
        la.ksplit = kse;
        long long need = (la.groups + slots - 1) / slots;
        long long grid = static_cast<long long>(dev->sm_count) * occ;
        if (grid > need) grid = need;
        if (grid > kMaxGrid) grid = kMaxGrid;
        if (op == DG_OP_HEAD_FP8_ARGMAX &&
            ws_bytes < kWsData + static_cast<size_t>(grid) * cpow2(mt) * 8)
            return DG_ERR_WORKSPACE_TOO_SMALL;
        void* args[] = {&la};
        if (launch_kernel(fn, static_cast<unsigned>(grid), threads, smem, stream, args) !=
            cudaSuccess) {
            cudaGetLastError();
            return DG_ERR_CUDA;
        }
    }
    return DG_OK;
}

dg_status check_common(const void* const* ptrs, int n, void* ws, size_t ws_bytes, size_t ws_need)
{
    for (int i = 0; i < n; ++i)
        if (!ptrs[i]) return DG_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
        if (!aligned16(ptrs[i])) return DG_ERR_ALIGNMENT;
    if (!ws) return DG_ERR_INVALID_ARG;
    if (!aligned16(ws)) return DG_ERR_ALIGNMENT;
    if (ws_bytes < ws_need) return DG_ERR_WORKSPACE_TOO_SMALL;
    return DG_OK;
}

}  // namespace
}  // namespace dg

extern "C" {

dg_status dg_gemv_bf16(const void* x, const void* W, void* y, int M, int N, int K, void* ws,
                       size_t ws_bytes, dg_stream_t stream, const dg_choice* choice)
{
    if (M < 1 || M > kMaxDenseRows || N < 1 || K < 1) return DG_ERR_INVALID_ARG;
    if (K % 8 != 0) return DG_ERR_UNSUPPORTED_SHAPE;
    const void* ptrs[] = {x, W, y};
    dg_status s = check_common(ptrs, 3, ws, ws_bytes, dg_workspace_bytes(DG_OP_GEMV_BF16, M, N, K, 0));
    if (s != DG_OK) return s;
    const DeviceInfo* dev = current_device(&s);
    if (!dev) return s;
    dg_choice c;
    if ((s = resolve_choice(DG_OP_GEMV_BF16, M, N, K, choice, &c)) != DG_OK) return s;
    if (c.variant == DG_VAR_TC)
        return launch_tc(false, dev, c, x, W, y, M, N, K, N, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
    if (c.variant == DG_VAR_MMA) return launch_mw(false, dev, c, x, W, y, M, N, K, N, reinterpret_cast<cudaStream_t>(stream));
    if (c.variant != DG_VAR_CC_WARP && c.variant != DG_VAR_CC_BULK) return DG_ERR_BAD_VARIANT;
    DenseArgs a{};
    a.W = static_cast<const uint8_t*>(W);
    a.x = static_cast<const uint16_t*>(x);
    a.N = N;
    a.K = K;
    a.out = static_cast<uint16_t*>(y);
    a.ld_out = N;
    a.ws = static_cast<uint8_t*>(ws);
    return launch_dense(DG_OP_GEMV_BF16, dev, c, a, M, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

dg_status dg_gate_up_silu(const void* x, const void* W_gu, void* out, int M, int N_half, int K,
                          void* ws, size_t ws_bytes, dg_stream_t stream, const dg_choice* choice)
{
    if (M < 1 || M > kMaxDenseRows || N_half < 1 || K < 1) return DG_ERR_INVALID_ARG;
    if (K % 8 != 0) return DG_ERR_UNSUPPORTED_SHAPE;
    const void* ptrs[] = {x, W_gu, out};
    dg_status s =
        check_common(ptrs, 3, ws, ws_bytes, dg_workspace_bytes(DG_OP_GATE_UP_SILU, M, N_half, K, 0));
    if (s != DG_OK) return s;
    const DeviceInfo* dev = current_device(&s);
    if (!dev) return s;
    dg_choice c;
    if ((s = resolve_choice(DG_OP_GATE_UP_SILU, M, N_half, K, choice, &c)) != DG_OK) return s;
    if (c.variant == DG_VAR_TC)
        return launch_tc(true, dev, c, x, W_gu, out, M, 2 * N_half, K, N_half, ws, ws_bytes,
                         reinterpret_cast<cudaStream_t>(stream));
    if (c.variant == DG_VAR_MMA)
        return launch_mw(true, dev, c, x, W_gu, out, M, 2 * N_half, K, N_half, reinterpret_cast<cudaStream_t>(stream));
    if (c.variant != DG_VAR_CC_WARP && c.variant != DG_VAR_CC_BULK) return DG_ERR_BAD_VARIANT;
    DenseArgs a{};
    a.W = static_cast<const uint8_t*>(W_gu);
    a.x = static_cast<const uint16_t*>(x);
    a.N = 2 * N_half;
    a.K = K;
    a.out = static_cast<uint16_t*>(out);
    a.ld_out = N_half;
    a.ws = static_cast<uint8_t*>(ws);
    return launch_dense(DG_OP_GATE_UP_SILU, dev, c, a, M, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

dg_status dg_head_fp8_argmax(const void* x, const void* Wq, const float* scale, void* logits,
                             int32_t* argmax, int M, int N, int K, void* ws, size_t ws_bytes,
                             dg_stream_t stream, const dg_choice* choice)
{
    if (M < 1 || M > 8 || N < 1 || K < 1) return DG_ERR_INVALID_ARG;
    if (K % 16 != 0) return DG_ERR_UNSUPPORTED_SHAPE;
    if (!scale || !argmax) return DG_ERR_INVALID_ARG;
    if (logits && !aligned16(logits)) return DG_ERR_ALIGNMENT;
    const void* ptrs[] = {x, Wq};
    dg_status s =
        check_common(ptrs, 2, ws, ws_bytes, dg_workspace_bytes(DG_OP_HEAD_FP8_ARGMAX, M, N, K, 0));
    if (s != DG_OK) return s;
    const DeviceInfo* dev = current_device(&s);
    if (!dev) return s;
    dg_choice c;
    if ((s = resolve_choice(DG_OP_HEAD_FP8_ARGMAX, M, N, K, choice, &c)) != DG_OK) return s;
    if (c.variant == DG_VAR_TC)
        return launch_tc_head(dev, c, x, Wq, scale, logits, argmax, M, N, K, ws, ws_bytes,
                              reinterpret_cast<cudaStream_t>(stream));
    if (c.variant != DG_VAR_CC_WARP && c.variant != DG_VAR_CC_BULK) return DG_ERR_BAD_VARIANT;
    DenseArgs a{};
    a.W = static_cast<const uint8_t*>(Wq);
    a.x = static_cast<const uint16_t*>(x);
    a.N = N;
    a.K = K;
    a.out = static_cast<uint16_t*>(logits);
    a.ld_out = N;
    a.scale = scale;
    a.argmax = argmax;
    a.ws = static_cast<uint8_t*>(ws);
    return launch_dense(DG_OP_HEAD_FP8_ARGMAX, dev, c, a, M, ws_bytes,
                        reinterpret_cast<cudaStream_t>(stream));
}

// Row-range order: grid = SMs x CTAs per SM (params[2], else the occupancy limit);
// W2 cuts Nout into equal contiguous ranges (empty CTAs dropped), W1 the flattened
// (expert, column pair) list.
static dg_status launch_moe_range(bool w1, const DeviceInfo* dev, const dg_choice& c, MoeArgs a,
                                  cudaStream_t stream)
{
    const int wpc = c.params[1] > 0 ? c.params[1] : 8;
    const int mtmax = c.params[4] > 0 ? c.params[4] : 2;
    if ((c.params[0] != 0 && c.params[0] != 4) || (wpc != 4 && wpc != 8) || c.params[2] < 0 || c.params[2] > 4 ||
        c.params[3] != 0)
        return DG_ERR_BAD_VARIANT;
    const void* fn = moe_range_kernel_fn(w1, mtmax);
    if (!fn) return DG_ERR_BAD_VARIANT;
    const int threads = wpc * 32;
    const int rows = w1 ? a.I : a.Nout;
    // shared memory at the widest range any grid of >= one CTA per SM gives
    const int rpc_max = w1 ? 0 : (rows + dev->sm_count - 1) / dev->sm_count;
    size_t smem = moe_range_smem(w1, a.M, a.topk, a.K, rpc_max);
    if (smem > kMaxDynSmem) return DG_ERR_UNSUPPORTED_SHAPE;
    int occ = occupancy(fn, threads, smem);
    if (occ < 1) return DG_ERR_UNSUPPORTED_SHAPE;
    if (c.params[2] > 0 && occ > c.params[2]) occ = c.params[2];
    long long grid = static_cast<long long>(dev->sm_count) * occ;
    a.tile = 0;
    if (!w1) {
        if (grid > rows) grid = rows;
        const long long rpc = (rows + grid - 1) / grid;
        grid = (rows + rpc - 1) / rpc;                      // every CTA has rows
        a.tile = static_cast<int>(rpc);
        smem = moe_range_smem(false, a.M, a.topk, a.K, a.tile);
    }
    void* args[] = {&a};
    if (launch_kernel(fn, static_cast<unsigned>(grid), threads, smem, stream, args) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

static dg_status launch_moe(bool w1, const DeviceInfo* dev, const dg_choice& c, MoeArgs a,
                            cudaStream_t stream)
{
    if (c.variant == DG_VAR_TC) return launch_tc_moe(w1, dev, c, a, stream);
    if (c.variant != DG_VAR_CC_WARP) return DG_ERR_BAD_VARIANT;
    if (c.params[5] == kMoeOrderRange) return launch_moe_range(w1, dev, c, a, stream);
    if (c.params[5] != 0 && c.params[5] != kMoeOrderUnits) return DG_ERR_BAD_VARIANT;
    const int wpc = c.params[1] > 0 ? c.params[1] : 8;
    if (c.params[0] != 0 && c.params[0] != 4) return DG_ERR_BAD_VARIANT;
    if (wpc < 1 || wpc > 8 || c.params[2] < 0 || c.params[3] < 0) return DG_ERR_BAD_VARIANT;
    int tile = c.params[3];
    if (tile == 0) tile = w1 ? wpc * 2 : (wpc * 4 < 32 ? 32 : wpc * 4);
    a.tile = tile;
    if (!w1 && moe_tickets(a.M, a.Nout, tile) > kWsMaxCounters) return DG_ERR_BAD_VARIANT;
    const int mtmax = c.params[4] > 0 ? c.params[4] : 2;
    const void* fn = w1 ? moe_w1_kernel(mtmax) : moe_w2_kernel(mtmax);
    if (!fn) return DG_ERR_BAD_VARIANT;
    const int threads = wpc * 32;
    const size_t smem = static_cast<size_t>(mtmax) * a.K * 2;
    if (smem > kMaxDynSmem) return DG_ERR_UNSUPPORTED_SHAPE;
    int occ = occupancy(fn, threads, smem);
    if (occ < 1) return DG_ERR_UNSUPPORTED_SHAPE;
    if (c.params[2] > 0 && occ > c.params[2]) occ = c.params[2];
    const long long grid = static_cast<long long>(dev->sm_count) * occ;
    void* args[] = {&a};
    if (launch_kernel(fn, static_cast<unsigned>(grid), threads, smem, stream, args) !=
        cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

dg_status dg_gemv_a8w8_blockscale(const void* x, const void* Wq, const float* sw, void* y, int M, int N, int K,
                                  void* ws, size_t ws_bytes, dg_stream_t stream, const dg_choice* choice)
{
    if (M < 1 || M > kA8MaxRows || N < 1 || K < 1) return DG_ERR_INVALID_ARG;
    if (K % 16 != 0) return DG_ERR_UNSUPPORTED_SHAPE;
    const void* ptrs[] = {x, Wq, sw, y};
    dg_status s = check_common(ptrs, 4, ws, ws_bytes, dg_workspace_bytes(DG_OP_GEMV_A8W8, M, N, K, 0));
    if (s != DG_OK) return s;
    const DeviceInfo* dev = current_device(&s);
    if (!dev) return s;
    dg_choice c;
    if ((s = resolve_choice(DG_OP_GEMV_A8W8, M, N, K, choice, &c)) != DG_OK) return s;
    if (c.variant != DG_VAR_TC) return DG_ERR_BAD_VARIANT;
    return launch_tc_a8(dev, c, x, Wq, sw, y, M, N, K, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

dg_status dg_quant_a8_blockscale(const void* x, void* q, float* sx, int M, int K, dg_stream_t stream)
{
    if (!x || !q || !sx || M < 1 || K < 1) return DG_ERR_INVALID_ARG;
    if (K % 16 != 0) return DG_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(x) || !aligned16(q) || !aligned16(sx)) return DG_ERR_ALIGNMENT;
    dg_status s;
    if (!current_device(&s)) return s;
    return launch_a8_quant(x, q, sx, M, K, reinterpret_cast<cudaStream_t>(stream));
}

size_t dg_fp4_scale_bytes(int rows, int K, int fmt)
{
    if (rows < 1 || K < 1 || K % 32 != 0 || (fmt != DG_FP4_MX && fmt != DG_FP4_NV)) return 0;
    return fp4::scale_bytes(rows, K, fmt == DG_FP4_NV);
}

static dg_status check_fp4(const void* const* ptrs, int n, const float* g, const float* g2, int M, int K, int fmt)
{
    for (int i = 0; i < n; ++i)
        if (!ptrs[i]) return DG_ERR_INVALID_ARG;
    if (M < 1 || K < 1 || (fmt != DG_FP4_MX && fmt != DG_FP4_NV)) return DG_ERR_INVALID_ARG;
    if (fmt == DG_FP4_MX && (g || g2)) return DG_ERR_INVALID_ARG;
    if (K % 32 != 0 || M > fp4::kMaxLen || K > fp4::kMaxLen) return DG_ERR_UNSUPPORTED_SHAPE;
    for (int i = 0; i < n; ++i)
        if (!aligned16(ptrs[i])) return DG_ERR_ALIGNMENT;
    if ((reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(g2)) & 3u) return DG_ERR_ALIGNMENT;
    return DG_OK;
}

dg_status dg_quant_fp4_blockscale(const void* x, void* q, void* s, const float* g, int M, int K, int fmt,
                                  dg_stream_t stream)
{
    const void* ptrs[] = {x, q, s};
    dg_status st = check_fp4(ptrs, 3, g, nullptr, M, K, fmt);
    if (st != DG_OK) return st;
    if (!current_device(&st)) return st;
    st = launch_fp4_quant(fmt == DG_FP4_NV, x, q, s, g, M, K, fp4::kTileRows, false,
                          reinterpret_cast<cudaStream_t>(stream));
    if (st == DG_OK) weights_written(reinterpret_cast<cudaStream_t>(stream));
    return st;
}

dg_status dg_dequant_fp4_blockscale(const void* q, const void* s, const float* g, void* y, int M, int K, int fmt,
                                    dg_stream_t stream)
{
    const void* ptrs[] = {q, s, y};
    dg_status st = check_fp4(ptrs, 3, g, nullptr, M, K, fmt);
    if (st != DG_OK) return st;
    if (!current_device(&st)) return st;
    st = launch_fp4_dequant(fmt == DG_FP4_NV, q, s, g, y, M, K, reinterpret_cast<cudaStream_t>(stream));
    if (st == DG_OK) weights_written(reinterpret_cast<cudaStream_t>(stream));
    return st;
}

dg_status dg_gemv_a4w4_blockscale(const void* x, const void* Wq, const void* sw, const float* gx, const float* gw,
                                  void* y, int M, int N, int K, int fmt, void* ws, size_t ws_bytes,
                                  dg_stream_t stream, const dg_choice* choice)
{
    if (M < 1 || M > kMaxDenseRows || N < 1) return DG_ERR_INVALID_ARG;
    const void* ptrs[] = {x, Wq, sw, y};
    dg_status s = check_fp4(ptrs, 4, gx, gw, M, K, fmt);
    if (s != DG_OK) return s;
    if (N > fp4::kMaxLen) return DG_ERR_UNSUPPORTED_SHAPE;
    s = check_common(ptrs, 4, ws, ws_bytes, dg_workspace_bytes(DG_OP_GEMV_A4W4, M, N, K, 0));
    if (s != DG_OK) return s;
    const DeviceInfo* dev = current_device(&s);
    if (!dev) return s;
    dg_choice c;
    if ((s = resolve_choice(DG_OP_GEMV_A4W4, M, N, K, choice, &c)) != DG_OK) return s;
    if (c.variant != DG_VAR_TC) return DG_ERR_BAD_VARIANT;
    return launch_tc_a4(dev, c, fmt == DG_FP4_NV, x, Wq, sw, gx, gw, y, M, N, K, ws, ws_bytes,
                        reinterpret_cast<cudaStream_t>(stream));
}

constexpr int kMaxLen = fp4::kMaxLen;      // largest rows and columns of a matrix

dg_status dg_quant_i8_rowscale(const void* x, int8_t* q, float* s, int M, int K, dg_stream_t stream)
{
    if (!x || !q || !s || M < 1 || K < 1) return DG_ERR_INVALID_ARG;
    if (K % 16 != 0 || M > kMaxLen || K > kMaxLen) return DG_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(x) || !aligned16(q) || !aligned16(s)) return DG_ERR_ALIGNMENT;
    dg_status st;
    const DeviceInfo* dev = current_device(&st);
    if (!dev) return st;
    st = launch_i8_quant(dev, x, q, s, M, K, 0, reinterpret_cast<cudaStream_t>(stream));
    if (st == DG_OK) weights_written(reinterpret_cast<cudaStream_t>(stream));
    return st;
}

dg_status dg_gemv_i8_rowscale(const void* x, const int8_t* Wq, const float* sw, void* y, int M, int N, int K, void* ws,
                              size_t ws_bytes, dg_stream_t stream, const dg_choice* choice)
{
    if (M < 1 || M > kMaxDenseRows || N < 1 || K < 1) return DG_ERR_INVALID_ARG;
    if (K % 16 != 0 || K > i8::kMaxK || N > kMaxLen) return DG_ERR_UNSUPPORTED_SHAPE;
    const void* ptrs[] = {x, Wq, sw, y};
    dg_status s = check_common(ptrs, 4, ws, ws_bytes, dg_workspace_bytes(DG_OP_GEMV_I8, M, N, K, 0));
    if (s != DG_OK) return s;
    const DeviceInfo* dev = current_device(&s);
    if (!dev) return s;
    dg_choice c;
    if ((s = resolve_choice(DG_OP_GEMV_I8, M, N, K, choice, &c)) != DG_OK) return s;
    // (a table's pick that has no room for this call's tokens: what is derived without one, the same bits)
    if (c.from_table && c.variant == DG_VAR_CC_WARP && !i8_cc_takes(M, K)) default_choice(DG_OP_GEMV_I8, M, N, K, &c);
    if (c.variant == DG_VAR_CC_WARP) return launch_i8_cc(dev, c, x, Wq, sw, y, M, N, K, reinterpret_cast<cudaStream_t>(stream));
    if (c.variant != DG_VAR_TC) return DG_ERR_BAD_VARIANT;
    return launch_i8_linear(dev, c, x, Wq, sw, y, M, N, K, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

// Logits of either type: a pointer on its element's boundary, rows ld >= n elements apart.
static dg_status check_logits(const void* logits, int type, int64_t ld, int M, int n)
{
    if (!logits || M < 1 || n < 1 || ld < n || (type != DG_LOGITS_BF16 && type != DG_LOGITS_F32))
        return DG_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(logits) & (type == DG_LOGITS_F32 ? 3u : 1u)) return DG_ERR_ALIGNMENT;
    return DG_OK;
}

static bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

dg_status dg_moe_route(const void* logits, int logits_type, int64_t ld, const float* bias, const dg_route_params* p,
                       int32_t* ids, float* w, int M, int E, dg_stream_t stream)
{
    dg_status s = check_logits(logits, logits_type, ld, M, E);
    if (s != DG_OK) return s;
    if (!p || !ids || !w) return DG_ERR_INVALID_ARG;
    if (p->n_group < 1 || p->topk_group < 1 || p->topk_group > p->n_group || p->topk < 1 ||
        (p->group_top != 1 && p->group_top != 2) || (p->renorm != 0 && p->renorm != 1) ||
        (p->score != DG_SCORE_SOFTMAX && p->score != DG_SCORE_SIGMOID))
        return DG_ERR_INVALID_ARG;
    if (E > 1024 || p->topk > 32 || p->n_group > 32 || E % p->n_group != 0 ||
        p->topk > p->topk_group * (E / p->n_group))
        return DG_ERR_UNSUPPORTED_SHAPE;
    if (misaligned(bias, 4) || misaligned(ids, 4) || misaligned(w, 4)) return DG_ERR_ALIGNMENT;
    if (!current_device(&s)) return s;
    return launch_route(*p, logits, bias, ids, w, M, E, ld, logits_type == DG_LOGITS_F32,
                        reinterpret_cast<cudaStream_t>(stream));
}

dg_status dg_moe_sort(const int32_t* ids, int32_t* offsets, int32_t* pos, int32_t* slots, int M, int topk, int E,
                      dg_stream_t stream)
{
    if (!ids || !offsets || !pos || !slots || M < 1 || topk < 1 || E < 1) return DG_ERR_INVALID_ARG;
    if (topk > 32 || E > 1024 || static_cast<long long>(M) * topk > (1 << 30)) return DG_ERR_UNSUPPORTED_SHAPE;
    if (misaligned(ids, 4) || misaligned(offsets, 4) || misaligned(pos, 4) || misaligned(slots, 4)) return DG_ERR_ALIGNMENT;
    dg_status s;
    if (!current_device(&s)) return s;
    return launch_moe_sort(ids, offsets, pos, slots, M, topk, E, reinterpret_cast<cudaStream_t>(stream));
}

// Rows of N bf16 at positions [M, topk].
static dg_status check_rows(const void* const* ptrs, int n, const int32_t* pos, int M, int topk, int P, int N)
{
    for (int i = 0; i < n; ++i)
        if (!ptrs[i]) return DG_ERR_INVALID_ARG;
    if (!pos || M < 1 || topk < 1 || P < 1 || N < 1) return DG_ERR_INVALID_ARG;
    if (topk > 32 || N % 8 != 0) return DG_ERR_UNSUPPORTED_SHAPE;
    for (int i = 0; i < n; ++i)
        if (!aligned16(ptrs[i])) return DG_ERR_ALIGNMENT;
    return misaligned(pos, 4) ? DG_ERR_ALIGNMENT : DG_OK;
}

dg_status dg_moe_gather(const void* x, const int32_t* pos, void* xs, int M, int topk, int P, int64_t row_bytes,
                        dg_stream_t stream)
{
    if (row_bytes < 1) return DG_ERR_INVALID_ARG;
    if (row_bytes % 16 != 0 || row_bytes > (1 << 30)) return DG_ERR_UNSUPPORTED_SHAPE;
    const void* ptrs[] = {x, xs};
    dg_status s = check_rows(ptrs, 2, pos, M, topk, P, 8);
    if (s != DG_OK) return s;
    if (!current_device(&s)) return s;
    return launch_moe_gather(x, pos, xs, M, topk, P, row_bytes, reinterpret_cast<cudaStream_t>(stream));
}

dg_status dg_moe_combine(const void* z, const int32_t* pos, const float* w, void* y, int M, int topk, int P, int N,
                         dg_stream_t stream)
{
    const void* ptrs[] = {z, y};
    dg_status s = check_rows(ptrs, 2, pos, M, topk, P, N);
    if (s != DG_OK) return s;
    if (misaligned(w, 4)) return DG_ERR_ALIGNMENT;
    if (!current_device(&s)) return s;
    return launch_moe_combine(z, pos, w, y, M, topk, P, N, reinterpret_cast<cudaStream_t>(stream));
}

dg_status dg_moe_combine_grad(const void* dy, const void* z, const int32_t* pos, const float* w, void* dz, float* dw,
                              int M, int topk, int P, int N, dg_stream_t stream)
{
    const void* ptrs[] = {dy, z, dz};
    dg_status s = check_rows(ptrs, 3, pos, M, topk, P, N);
    if (s != DG_OK) return s;
    if (!w || !dw) return DG_ERR_INVALID_ARG;
    if (misaligned(w, 4) || misaligned(dw, 4)) return DG_ERR_ALIGNMENT;
    if (!current_device(&s)) return s;
    return launch_moe_combine_grad(dy, z, pos, w, dz, dw, M, topk, P, N, reinterpret_cast<cudaStream_t>(stream));
}

dg_status dg_logits_adjust(const void* logits, int logits_type, int64_t ld, void* out, int64_t ld_out,
                           const dg_logits_edits* e, int M, int V, dg_stream_t stream)
{
    dg_status s = check_logits(logits, logits_type, ld, M, V);
    if (s != DG_OK) return s;
    if ((s = check_logits(out, logits_type, ld_out, M, V)) != DG_OK) return s;
    if (!e || (out == logits && ld_out != ld && M > 1)) return DG_ERR_INVALID_ARG;
    if (e->n_tokens < 0 || e->n_bias < 0 || (e->n_tokens > 0) != (e->tokens != nullptr) ||
        (e->n_bias > 0) != (e->bias != nullptr) || (e->n_bias > 0) != (e->bias_ids != nullptr))
        return DG_ERR_INVALID_ARG;
    if (!e->tokens && (e->lengths || e->prompt_lengths || e->repetition || e->frequency || e->presence))
        return DG_ERR_INVALID_ARG;
    if ((e->tokens && e->ld_tokens < e->n_tokens) || (e->mask && e->ld_mask < (V - 1) / 32 + 1)) return DG_ERR_INVALID_ARG;
    if (V > (1 << 24) || e->n_tokens > (1 << 24) || e->n_bias > 1024) return DG_ERR_UNSUPPORTED_SHAPE;
    if (misaligned(e->tokens, 4) || misaligned(e->lengths, 4) || misaligned(e->prompt_lengths, 4) || misaligned(e->repetition, 4) ||
        misaligned(e->frequency, 4) || misaligned(e->presence, 4) || misaligned(e->bias_ids, 4) || misaligned(e->bias, 4) ||
        misaligned(e->mask, 4))
        return DG_ERR_ALIGNMENT;
    const DeviceInfo* dev = current_device(&s);
    if (!dev) return s;
    return launch_logits_adjust(dev, logits, logits_type == DG_LOGITS_F32, ld, out, ld_out, *e, M, V,
                                reinterpret_cast<cudaStream_t>(stream));
}

dg_status dg_logprobs(const void* logits, int logits_type, int64_t ld, const int64_t* tokens, float scale, int n_top,
                      float* logprob, int32_t* rank, float* entropy, int32_t* top_ids, float* top_logprobs, int M,
                      int V, dg_stream_t stream)
{
    dg_status s = check_logits(logits, logits_type, ld, M, V);
    if (s != DG_OK) return s;
    if (!(scale >= 1e-6f && scale <= 1e6f) || n_top < 0 || (n_top > 0) != (top_ids != nullptr) ||
        (n_top > 0) != (top_logprobs != nullptr) || (!tokens && (logprob || rank)))
        return DG_ERR_INVALID_ARG;
    if (n_top > 32 || M > (1 << 28) || V > (1 << 24)) return DG_ERR_UNSUPPORTED_SHAPE;
    if (misaligned(tokens, 8) || misaligned(logprob, 4) || misaligned(rank, 4) || misaligned(entropy, 4) ||
        misaligned(top_ids, 4) || misaligned(top_logprobs, 4))
        return DG_ERR_ALIGNMENT;
    if (!current_device(&s)) return s;
    return launch_logprobs(logits, logits_type == DG_LOGITS_F32, ld, tokens, scale, n_top, logprob, rank, entropy,
                           top_ids, top_logprobs, M, V, reinterpret_cast<cudaStream_t>(stream));
}

dg_status dg_moe_w1_silu(const void* x, const int32_t* topk_ids, const void* W1, const float* s1,
                         void* a_out, int M, int topk, int E, int I, int K, void* ws, size_t ws_bytes,
                         dg_stream_t stream, const dg_choice* choice)
{
    if (M < 1 || M > 16 || topk < 1 || topk > 8 || E < 1 || E > 1024 || I < 1 || K < 1)
        return DG_ERR_INVALID_ARG;
    if (K % 16 != 0 || I % 8 != 0) return DG_ERR_UNSUPPORTED_SHAPE;
    const void* ptrs[] = {x, topk_ids, W1, s1, a_out};
    dg_status s = check_common(ptrs, 5, ws, ws_bytes, dg_workspace_bytes(DG_OP_MOE_W1, M, I, K, topk));
    if (s != DG_OK) return s;
    const DeviceInfo* dev = current_device(&s);
    if (!dev) return s;
    dg_choice c;
    if ((s = resolve_choice(DG_OP_MOE_W1, M, I, K, choice, &c)) != DG_OK) return s;
    MoeArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.ids = topk_ids;
    a.W = static_cast<const uint8_t*>(W1);
    a.s = s1;
    a.out = static_cast<uint16_t*>(a_out);
    a.ws = static_cast<uint8_t*>(ws);
    a.M = M;
    a.topk = topk;
    a.E = E;
    a.I = I;
    a.K = K;
    a.Nout = 0;
    return launch_moe(true, dev, c, a, reinterpret_cast<cudaStream_t>(stream));
}

dg_status dg_moe_w2(const void* a_in, const int32_t* topk_ids, const float* gw, const void* W2,
                    const float* s2, void* y, int M, int topk, int E, int I, int Nout, void* ws,
                    size_t ws_bytes, dg_stream_t stream, const dg_choice* choice)
{
    if (M < 1 || M > 16 || topk < 1 || topk > 8 || E < 1 || E > 1024 || I < 1 || Nout < 1)
        return DG_ERR_INVALID_ARG;
    if (I % 16 != 0) return DG_ERR_UNSUPPORTED_SHAPE;
    const void* ptrs[] = {a_in, topk_ids, gw, W2, s2, y};
    dg_status s =
        check_common(ptrs, 6, ws, ws_bytes, dg_workspace_bytes(DG_OP_MOE_W2, M, Nout, I, topk));
    if (s != DG_OK) return s;
    const DeviceInfo* dev = current_device(&s);
    if (!dev) return s;
    dg_choice c;
    if ((s = resolve_choice(DG_OP_MOE_W2, M, Nout, I, choice, &c)) != DG_OK) return s;
    MoeArgs a{};
    a.x = static_cast<const uint16_t*>(a_in);
    a.ids = topk_ids;
    a.gw = gw;
    a.W = static_cast<const uint8_t*>(W2);
    a.s = s2;
    a.out = static_cast<uint16_t*>(y);
    a.ws = static_cast<uint8_t*>(ws);
    a.M = M;
    a.topk = topk;
    a.E = E;
    a.I = I;
    a.K = I;
    a.Nout = Nout;
    return launch_moe(false, dev, c, a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
