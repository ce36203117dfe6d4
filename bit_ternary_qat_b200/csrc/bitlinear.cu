// bitlinear.cu -- C ABI of the BitLinear hot path (declared in include/bitlinear.h).
//
// Host side only: argument validation (before any CUDA call, so a bad call launches
// nothing), TMA tensor-map encoding, grid sizing and kernel launches.  All arithmetic
// of the path happens in the kernels included below; nothing here touches the data.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>

#include "../../include/bitlinear.h"
#include "common.cuh"
#include "act_quant.cuh"
#include "weight_quant.cuh"
#include "gemm_tc.cuh"
#include "gemm_simt.cuh"
#include "rmsnorm_bwd.cuh"
#include "gemv.cuh"
#include "optim.cuh"
#include "residual_norm.cuh"
#include "grad_clip.cuh"
#include "weight_quant8.cuh"
#include "gemm_int8.cuh"
#include "gemm_packed.cuh"
#include "gemm_packed2.cuh"
#include "mma_peak.cuh"
#include "read_peak.cuh"

// Scratch of bitlinear_quant_weight_noalloc: the pass-1 partial sums of |W| live in this
// file-scope device array instead of a caller workspace.  Every device that loads the
// library holds it until the process exits.  Host code must not pass the symbol itself to
// a kernel (on the host it names a host-side shadow, not device memory): the device
// address is looked up with cudaGetSymbolAddress once per device and passed instead.
static __device__ __align__(256) double g_quant_scratch[bl::kWqMaxPartials];

namespace {

thread_local std::string g_last_error = "no error";
std::atomic<uint64_t> g_launches{0};
std::atomic<uint64_t> g_wait_ns{2000000000ull};

bl_status fail(bl_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return s;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

#define BL_REQUIRE(cond, status, ...)                  \
    do {                                               \
        if (!(cond)) return fail(status, __VA_ARGS__); \
    } while (0)

#define BL_TRY(expr)                     \
    do {                                 \
        bl_status _s = (expr);           \
        if (_s != BL_OK) return _s;      \
    } while (0)

bl_status check_dims(int64_t T, int64_t N, int64_t K) {
    BL_REQUIRE(T >= 1 && N >= 1 && K >= 1, BL_ERR_INVALID_ARG, "sizes must be positive (T=%lld N=%lld K=%lld)",
               (long long)T, (long long)N, (long long)K);
    BL_REQUIRE(T <= kMaxDim && N <= kMaxDim && K <= kMaxDim, BL_ERR_UNSUPPORTED_SHAPE, "sizes must be < 2^31");
    BL_REQUIRE(K % 32 == 0, BL_ERR_UNSUPPORTED_SHAPE, "K (d_in) must be a multiple of 32, got %lld", (long long)K);
    BL_REQUIRE(N % 16 == 0, BL_ERR_UNSUPPORTED_SHAPE, "N (d_out) must be a multiple of 16, got %lld", (long long)N);
    return BL_OK;
}

bl_status check_ptr(const void* p, const char* name, bool required) {
    if (p == nullptr) {
        BL_REQUIRE(!required, BL_ERR_INVALID_ARG, "%s must not be NULL", name);
        return BL_OK;
    }
    BL_REQUIRE(aligned16(p), BL_ERR_MISALIGNED, "%s must be 16-byte aligned", name);
    return BL_OK;
}

bl_status check_dtype(bl_dtype dt) {
    BL_REQUIRE(dt == BL_F32 || dt == BL_BF16, BL_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
    return BL_OK;
}

// ------------------------------------------------------------------------------------
// device checks
// ------------------------------------------------------------------------------------
struct DeviceInfo {
    int sms = 0;
    int major = 0;
    int max_smem_optin = 0;
};

std::mutex g_dev_mu;
DeviceInfo g_dev[64];
bool g_dev_ok[64] = {};

bl_status current_device(DeviceInfo* out) {
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail(BL_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    BL_REQUIRE(dev >= 0 && dev < 64, BL_ERR_DEVICE, "device index %d out of range", dev);
    std::lock_guard<std::mutex> lk(g_dev_mu);
    if (!g_dev_ok[dev]) {
        DeviceInfo d;
        cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
        cudaDeviceGetAttribute(&d.major, cudaDevAttrComputeCapabilityMajor, dev);
        cudaDeviceGetAttribute(&d.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
        e = cudaGetLastError();
        if (e != cudaSuccess) return fail(BL_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
        if (d.major != 10) return fail(BL_ERR_DEVICE, "device %d is sm_%d0; this library is built for sm_100a", dev, d.major);
        g_dev[dev] = d;
        g_dev_ok[dev] = true;
    }
    *out = g_dev[dev];
    return BL_OK;
}

bl_status launched(const char* what) {
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(BL_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return BL_OK;
}

// Every kernel is launched with programmatic dependent launch: its blocks may be scheduled
// while the previous kernel in the stream drains (each kernel signals this at its start),
// and each kernel runs its set-up (barriers, TMEM, descriptor prefetch) and then waits
// (griddepcontrol.wait) for the previous grid's completion and memory before it touches
// global memory.  After a kernel launched without the attribute the wait is a no-op.
template <typename... KArgs, typename... Args>
void pdl_launch(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);   // errors surface in launched()
}

// ------------------------------------------------------------------------------------
// TMA tensor maps
// ------------------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

enum TmType { kTmU8 = 0, kTmBf16 = 1, kTmF32 = 2, kTmI32 = 3 };

// 2-D row-major tensor [outer x inner] with 128-byte swizzled boxes [box_outer x box_inner]
// (box_inner * element size == 128 bytes).
bl_status make_tmap(CUtensorMap* tm, const void* base, TmType t, uint64_t inner, uint64_t outer,
                    uint32_t box_inner, uint32_t box_outer, bool swizzle128 = true) {
    EncodeTiledFn fn = encode_fn();
    BL_REQUIRE(fn != nullptr, BL_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    const uint64_t esize = t == kTmU8 ? 1 : (t == kTmBf16 ? 2 : 4);
    const CUtensorMapDataType dt = t == kTmU8    ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : t == kTmBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : t == kTmI32  ? CU_TENSOR_MAP_DATA_TYPE_INT32
                                                  : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    cuuint64_t dims[2] = {inner, outer};
    cuuint64_t strides[1] = {inner * esize};
    cuuint32_t box[2] = {box_inner, box_outer};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(tm, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    BL_REQUIRE(r == CUDA_SUCCESS, BL_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return BL_OK;
}

// 3-D map over int32 slices [outer][middle][inner] (no swizzle): the K-split partial sums,
// one box of box_inner x box_middle elements in one slice.
bl_status make_tmap3_i32(CUtensorMap* tm, const void* base, uint64_t inner, uint64_t middle, uint64_t outer,
                         uint32_t box_inner, uint32_t box_middle) {
    EncodeTiledFn fn = encode_fn();
    BL_REQUIRE(fn != nullptr, BL_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    cuuint64_t dims[3] = {inner, middle, outer};
    cuuint64_t strides[2] = {inner * 4, inner * middle * 4};
    cuuint32_t box[3] = {box_inner, box_middle, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_INT32, 3, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    BL_REQUIRE(r == CUDA_SUCCESS, BL_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return BL_OK;
}

// ------------------------------------------------------------------------------------
// tcgen05 GEMM launcher
// ------------------------------------------------------------------------------------
constexpr int kBN = 256;

template <bool kInt8, bool kAMN, bool kBMN, int kEpi>
bl_status launch_tc(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& td, bl::TcGemmArgs a,
                    cudaStream_t st, const DeviceInfo& dev) {
    auto kern = bl::tc_gemm_kernel<kInt8, kAMN, kBMN, kBN, kEpi>;
    const size_t smem = bl::tc_smem_bytes<kBN>();
    BL_REQUIRE((int)smem <= dev.max_smem_optin, BL_ERR_DEVICE, "GEMM needs %zu bytes of shared memory", smem);
    static std::atomic<uint64_t> attr_set{0};   // bit d: attribute set on device d
    int dev_id = 0;
    cudaGetDevice(&dev_id);
    if (!(attr_set.load() & (1ull << dev_id))) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return fail(BL_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        attr_set.fetch_or(1ull << dev_id);
    }
    a.m_tiles = (a.M + bl::kTcBM - 1) / bl::kTcBM;
    a.n_tiles = (a.N + kBN - 1) / kBN;
    const int kb_elems = kInt8 ? 128 : 64;
    a.k_blocks = (a.K + kb_elems - 1) / kb_elems;
    a.wait_ns = g_wait_ns.load();
    const int tiles = a.m_tiles * a.n_tiles;
    const int grid = tiles < dev.sms ? tiles : dev.sms;
    pdl_launch(kern, dim3(grid), dim3(bl::kTcThreads), smem, st, ta, tb, td, a);
    return launched("tc_gemm");
}

// 2-SM variant: clusters of two CTAs, 256 x 256 tiles.  The grid is as many clusters as
// fit on the device at once (queried once per device and kernel), at most one per tile.
template <bool kInt8, bool kAMN, bool kBMN, int kEpi>
bl_status launch_tc2(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& td, bl::TcGemmArgs a,
                     cudaStream_t st, const DeviceInfo& dev) {
    auto kern = bl::tc_gemm2_kernel<kInt8, kAMN, kBMN, kEpi>;
    const size_t smem = bl::tc2_smem_bytes();
    BL_REQUIRE((int)smem <= dev.max_smem_optin, BL_ERR_DEVICE, "GEMM needs %zu bytes of shared memory", smem);
    static std::atomic<int> max_clusters[64] = {};
    int dev_id = 0;
    cudaGetDevice(&dev_id);
    if (dev_id < 0 || dev_id >= 64) return fail(BL_ERR_DEVICE, "device ordinal %d out of range", dev_id);
    int mc = max_clusters[dev_id].load();
    if (mc == 0) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return fail(BL_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * (unsigned)(dev.sms / 2));
        cfg.blockDim = dim3(bl::kTcThreads);
        cfg.dynamicSmemBytes = smem;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
        if (e != cudaSuccess) return fail(BL_ERR_CUDA, "cudaOccupancyMaxActiveClusters: %s", cudaGetErrorString(e));
        if (n < 1) return fail(BL_ERR_DEVICE, "no 2-CTA cluster of the GEMM fits on the device");
        mc = n;
        max_clusters[dev_id].store(mc);
    }
    a.m_tiles = (a.M + 255) / 256;
    a.n_tiles = (a.N + 255) / 256;
    const int kb_elems = kInt8 ? 128 : 64;
    a.k_blocks = (a.K + kb_elems - 1) / kb_elems;
    a.wait_ns = g_wait_ns.load();
    const int tiles = a.m_tiles * a.n_tiles;
    const int clusters = tiles < mc ? tiles : mc;
    pdl_launch(kern, dim3(2 * clusters), dim3(bl::kTcThreads), smem, st, ta, tb, td, a);
    return launched("tc_gemm2");
}

// The 2-SM kernel computes 256-row tiles; for a single 128-row tile the 1-SM kernel wastes
// nothing and needs no partner CTA.
inline bool use_2sm(int64_t M) { return M > bl::kTcBM; }

// ------------------------------------------------------------------------------------
// pieces shared by the entry points (validation already done by the caller)
// ------------------------------------------------------------------------------------
// One row per block (the kernel can take R adjacent rows per block; measured slower here).
template <bool kBf16, int VPT>
void launch_act_quant_v(const void* X, int64_t T, int64_t K, int apply_norm, const float* g, float eps, int8_t* Xq,
                        float* sx, float* rinv, void* Xdq, cudaStream_t st) {
    constexpr int NT = bl::act_threads<kBf16>();
    constexpr int R = 1;
    const unsigned grid = (unsigned)((T + R - 1) / R);
    pdl_launch(bl::act_quant_kernel<kBf16, NT, VPT, R>, dim3(grid), dim3(NT), 0, st, X, (int)T, (int)K, apply_norm, g,
               eps, Xq, sx, rinv, Xdq);
}

// SM count of the current device (cached per device).
int sm_count() {
    static std::atomic<int> cache[64] = {};
    int dev_id = 0;
    cudaGetDevice(&dev_id);
    if (dev_id < 0 || dev_id >= 64) return 148;
    int n = cache[dev_id].load();
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev_id) != cudaSuccess || n <= 0) n = 148;
        cache[dev_id].store(n);
    }
    return n;
}

// Persistent: two blocks of 8 row-warps per SM at most.
template <bool kBf16, int VPL>
void launch_act_quant_w(const void* X, int64_t T, int64_t K, int apply_norm, const float* g, float eps, int8_t* Xq,
                        float* sx, float* rinv, void* Xdq, cudaStream_t st) {
    const int64_t blocks = std::min<int64_t>((T + 7) / 8, 2 * (int64_t)sm_count());
    pdl_launch(bl::act_quant_warp_kernel<kBf16, VPL>, dim3((unsigned)blocks), dim3(256), 0, st, X, (int)T,
               (int)K, apply_norm, g, eps, Xq, sx, rinv, Xdq);
}

// Rows of at most 256 vectors (2048 bf16 / 1024 fp32 elements): warp per row; longer rows:
// block per row.
template <bool kBf16>
void launch_act_quant(const void* X, int64_t T, int64_t K, int apply_norm, const float* g, float eps, int8_t* Xq,
                      float* sx, float* rinv, void* Xdq, cudaStream_t st) {
    constexpr int NT = bl::act_threads<kBf16>();
    const int64_t nvec = K / (kBf16 ? 8 : 4);
    if (nvec <= 32) return launch_act_quant_w<kBf16, 1>(X, T, K, apply_norm, g, eps, Xq, sx, rinv, Xdq, st);
    if (nvec <= 64) return launch_act_quant_w<kBf16, 2>(X, T, K, apply_norm, g, eps, Xq, sx, rinv, Xdq, st);
    if (nvec <= 128) return launch_act_quant_w<kBf16, 4>(X, T, K, apply_norm, g, eps, Xq, sx, rinv, Xdq, st);
    // rows of 129-256 vectors: the warp-per-row kernel, except bf16 rows when there are at
    // most 8192 of them, where the block-per-row kernel's wider concurrency measured faster
    // (4096 x 2048 bf16: 10.0 against 11.2 us back to back; 16384 rows: 36.0 against 34.4 us;
    // fp32 4096 x 1024: 10.9 against 8.0 us)
    if (nvec <= 256 && (!kBf16 || T > 8192))
        return launch_act_quant_w<kBf16, 8>(X, T, K, apply_norm, g, eps, Xq, sx, rinv, Xdq, st);
    const int64_t vpt = (nvec + NT - 1) / NT;
    if (vpt <= 1) launch_act_quant_v<kBf16, 1>(X, T, K, apply_norm, g, eps, Xq, sx, rinv, Xdq, st);
    else if (vpt <= 2) launch_act_quant_v<kBf16, 2>(X, T, K, apply_norm, g, eps, Xq, sx, rinv, Xdq, st);
    else if (vpt <= 4) launch_act_quant_v<kBf16, 4>(X, T, K, apply_norm, g, eps, Xq, sx, rinv, Xdq, st);
    else if (vpt <= 8) launch_act_quant_v<kBf16, 8>(X, T, K, apply_norm, g, eps, Xq, sx, rinv, Xdq, st);
    else if (vpt <= 12) launch_act_quant_v<kBf16, 12>(X, T, K, apply_norm, g, eps, Xq, sx, rinv, Xdq, st);
    else launch_act_quant_v<kBf16, 16>(X, T, K, apply_norm, g, eps, Xq, sx, rinv, Xdq, st);
}

bl_status run_act_quant(const void* X, bl_dtype x_dt, int64_t T, int64_t K, int apply_norm, const float* g,
                        float eps, int8_t* Xq, float* sx, float* rinv, void* Xdq, cudaStream_t st) {
    if (x_dt == BL_BF16)
        launch_act_quant<true>(X, T, K, apply_norm, g, eps, Xq, sx, rinv, Xdq, st);
    else
        launch_act_quant<false>(X, T, K, apply_norm, g, eps, Xq, sx, rinv, Xdq, st);
    return launched("act_quant");
}

bl_status run_linear(const int8_t* Xq, const float* sx, int64_t T, int64_t K, const int8_t* Wq, const float* gamma,
                     int64_t N, void* Y, bl_dtype y_dt, int32_t* acc, cudaStream_t st, const DeviceInfo& dev) {
    CUtensorMap ta, tb, td;
    const bool two = use_2sm(T);
    BL_TRY(make_tmap(&ta, Xq, kTmU8, (uint64_t)K, (uint64_t)T, 128, 128));
    BL_TRY(make_tmap(&tb, Wq, kTmU8, (uint64_t)K, (uint64_t)N, 128, two ? 128 : kBN));
    bl::TcGemmArgs a{};
    a.M = (int)T; a.N = (int)N; a.K = (int)K;
    a.acc_out = acc; a.row_scale = sx; a.gamma = gamma;
    if (y_dt == BL_BF16) {
        BL_TRY(make_tmap(&td, Y, kTmBf16, (uint64_t)N, (uint64_t)T, 64, 32));
        if (two) return launch_tc2<true, false, false, bl::kEpiLinearBf16>(ta, tb, td, a, st, dev);
        return launch_tc<true, false, false, bl::kEpiLinearBf16>(ta, tb, td, a, st, dev);
    }
    BL_TRY(make_tmap(&td, Y, kTmF32, (uint64_t)N, (uint64_t)T, 32, 32));
    if (two) return launch_tc2<true, false, false, bl::kEpiLinearF32>(ta, tb, td, a, st, dev);
    return launch_tc<true, false, false, bl::kEpiLinearF32>(ta, tb, td, a, st, dev);
}

// Per-column scales gamma_n: the 2-SM kernel at every T (its rows past T are zero-filled
// loads and clipped stores).  kInt8: the 8-bit linear's order of the two scales.
template <bool kInt8 = false>
bl_status run_linear_rows(const int8_t* Xq, const float* sx, int64_t T, int64_t K, const int8_t* Wq,
                          const float* gamma_rows, int64_t N, void* Y, bl_dtype y_dt, int32_t* acc, cudaStream_t st,
                          const DeviceInfo& dev) {
    CUtensorMap ta, tb, td;
    BL_TRY(make_tmap(&ta, Xq, kTmU8, (uint64_t)K, (uint64_t)T, 128, 128));
    BL_TRY(make_tmap(&tb, Wq, kTmU8, (uint64_t)K, (uint64_t)N, 128, 128));
    bl::TcGemmArgs a{};
    a.M = (int)T; a.N = (int)N; a.K = (int)K;
    a.acc_out = acc; a.row_scale = sx; a.gamma = gamma_rows;
    if (y_dt == BL_BF16) {
        BL_TRY(make_tmap(&td, Y, kTmBf16, (uint64_t)N, (uint64_t)T, 64, 32));
        return launch_tc2<true, false, false, kInt8 ? bl::kEpiInt8Bf16 : bl::kEpiLinearColBf16>(ta, tb, td, a, st, dev);
    }
    BL_TRY(make_tmap(&td, Y, kTmF32, (uint64_t)N, (uint64_t)T, 32, 32));
    return launch_tc2<true, false, false, kInt8 ? bl::kEpiInt8F32 : bl::kEpiLinearColF32>(ta, tb, td, a, st, dev);
}

bl_status run_grad_input_gemm(const void* dY, bl_dtype dt, const uint16_t* Wq_bf16, const float* gamma, int64_t T,
                              int64_t K, int64_t N, float* dXhat, cudaStream_t st, const DeviceInfo& dev) {
    if (dt == BL_BF16) {
        CUtensorMap ta, tb, td;
        BL_TRY(make_tmap(&ta, dY, kTmBf16, (uint64_t)N, (uint64_t)T, 64, 128));      // dY, K-major (contraction N)
        BL_TRY(make_tmap(&tb, Wq_bf16, kTmBf16, (uint64_t)K, (uint64_t)N, 64, 64));  // W_q, MN-major (rows = N)
        BL_TRY(make_tmap(&td, dXhat, kTmF32, (uint64_t)K, (uint64_t)T, 32, 32));
        bl::TcGemmArgs a{};
        a.M = (int)T; a.N = (int)K; a.K = (int)N;
        a.gamma = gamma;
        if (use_2sm(T)) return launch_tc2<false, false, true, bl::kEpiScaleF32>(ta, tb, td, a, st, dev);
        return launch_tc<false, false, true, bl::kEpiScaleF32>(ta, tb, td, a, st, dev);
    }
    // fp32 layer: CUDA-core fp32 contraction, C[t,k] = gamma * sum_n dY[t,n] W_q[n,k]
    dim3 grid((unsigned)((K + 63) / 64), (unsigned)((T + 63) / 64));
    pdl_launch(bl::simt_gemm_kernel<float, uint16_t>, grid, dim3(256), 0, st, (int)T, (int)K, (int)N,
               static_cast<const float*>(dY), N, (int64_t)1, Wq_bf16, (int64_t)1, K, gamma, dXhat, K);
    return launched("simt_gemm(grad_input)");
}

bl_status run_grad_weight_gemm(const void* dY, const void* Xdq, bl_dtype dt, int64_t T, int64_t K, int64_t N,
                               float* dW, cudaStream_t st, const DeviceInfo& dev) {
    if (dt == BL_BF16) {
        CUtensorMap ta, tb, td;
        BL_TRY(make_tmap(&ta, dY, kTmBf16, (uint64_t)N, (uint64_t)T, 64, 64));    // dY^T: MN-major (n contiguous)
        BL_TRY(make_tmap(&tb, Xdq, kTmBf16, (uint64_t)K, (uint64_t)T, 64, 64));   // X_dq: MN-major (k contiguous)
        BL_TRY(make_tmap(&td, dW, kTmF32, (uint64_t)K, (uint64_t)N, 32, 32));
        bl::TcGemmArgs a{};
        a.M = (int)N; a.N = (int)K; a.K = (int)T;
        if (use_2sm(N)) return launch_tc2<false, true, true, bl::kEpiF32>(ta, tb, td, a, st, dev);
        return launch_tc<false, true, true, bl::kEpiF32>(ta, tb, td, a, st, dev);
    }
    dim3 grid((unsigned)((K + 63) / 64), (unsigned)((N + 63) / 64));
    pdl_launch(bl::simt_gemm_kernel<float, float>, grid, dim3(256), 0, st, (int)N, (int)K, (int)T,
               static_cast<const float*>(dY), (int64_t)1, N, static_cast<const float*>(Xdq), (int64_t)1, K,
               static_cast<const float*>(nullptr), dW, K);
    return launched("simt_gemm(grad_weight)");
}

size_t quant_ws_bytes() { return sizeof(double) * bl::kWqMaxPartials; }

// Weight quantiser pass 2: gamma, threshold and codes (one round of kTqGroups groups per
// thread when the grid covers W).
// tau_factor < 0: the round/clamp threshold; else the zero threshold fl32(tau_factor * gamma).
bl_status run_ternary(const float* W, int64_t n, const double* partials, int parts, int8_t* Wq_i8, uint16_t* Wq_bf16,
                      uint8_t* Wpacked, float* gamma, cudaStream_t st, const DeviceInfo& dev,
                      float tau_factor = -1.0f) {
    const int64_t groups = n / 16;
    const int64_t per_block = (int64_t)bl::kWqThreads * bl::kTqGroups;
    int64_t blocks = (groups + per_block - 1) / per_block;
    const int64_t cap = (int64_t)dev.sms * 4;
    if (blocks > cap) blocks = cap;
    if (tau_factor >= 0.0f) {
        pdl_launch(bl::ternary_quant_kernel<true>, dim3((unsigned)blocks), dim3(bl::kWqThreads), 0, st, W, n,
                   partials, parts, Wq_i8, Wq_bf16, Wpacked, gamma, tau_factor);
        return launched("ternary_quant(tau)");
    }
    pdl_launch(bl::ternary_quant_kernel<false>, dim3((unsigned)blocks), dim3(bl::kWqThreads), 0, st, W, n, partials,
               parts, Wq_i8, Wq_bf16, Wpacked, gamma, 0.0f);
    return launched("ternary_quant");
}

// Weight quantiser: fp64 partial sums of |W| (pass 1), then pass 2.
bl_status run_quant_weight(const float* W, int64_t n, void* scratch, int8_t* Wq_i8, uint16_t* Wq_bf16,
                           uint8_t* Wpacked, float* gamma, cudaStream_t st, const DeviceInfo& dev,
                           float tau_factor = -1.0f) {
    double* partials = static_cast<double*>(scratch);
    const int parts = bl::wq_num_partials(n);
    pdl_launch(bl::absmean_partial_kernel, dim3(parts), dim3(bl::kWqThreads), 0, st, W, n, partials);
    BL_TRY(launched("absmean_partial"));
    return run_ternary(W, n, partials, parts, Wq_i8, Wq_bf16, Wpacked, gamma, st, dev, tau_factor);
}

// Optimizer scratch: dW^2 partials, |W_new| partials, the published step index.
constexpr size_t kOptWpartOffset = sizeof(double) * bl::kWqMaxPartials;
constexpr size_t kOptStepOffset = 2 * sizeof(double) * bl::kWqMaxPartials;
size_t opt_ws_bytes() { return kOptStepOffset + 16; }

size_t dg_ws_bytes(int64_t K) { return sizeof(float) * (size_t)bl::kBwdMaxBlocks * (size_t)K; }

// Persistent grid: as many blocks as are resident at once (queried once per device and
// instantiation), at most kBwdMaxBlocks and at most one per row.
template <bool kBf16X, int NT, int VPT, bool kGain>
int launch_rmsnorm_bwd_v(const void* X, const float* rinv, const float* g, float* dX, int64_t T, int64_t K,
                         float* partial, int sms, cudaStream_t st) {
    auto kern = bl::rmsnorm_bwd_kernel<kBf16X, NT, VPT, kGain>;
    static std::atomic<int> per_sm[64] = {};
    int dev_id = 0;
    cudaGetDevice(&dev_id);
    int b = (dev_id >= 0 && dev_id < 64) ? per_sm[dev_id].load() : 0;
    if (b == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, kern, NT, 0) != cudaSuccess || b < 1) b = 1;
        if (dev_id >= 0 && dev_id < 64) per_sm[dev_id].store(b);
    }
    int64_t grid = (int64_t)b * sms;
    if (grid > bl::kBwdMaxBlocks) grid = bl::kBwdMaxBlocks;
    if (grid > T) grid = T;
    pdl_launch(kern, dim3((unsigned)grid), dim3(NT), 0, st, X, rinv, g, dX, (int)T, (int)K, partial);
    return (int)grid;
}

// Block size: the smallest of 128 / 256 / 512 / 1024 threads that covers a row with at most
// four 16-byte column vectors per thread (K <= 16384).
template <bool kBf16X, bool kGain>
int launch_rmsnorm_bwd_g(const void* X, const float* rinv, const float* g, float* dX, int64_t T, int64_t K,
                         float* partial, int sms, cudaStream_t st) {
    const int64_t nvec = K / 4;
#define BL_BWD(NT)                                                                                              \
    if (nvec <= 4 * (NT)) {                                                                                     \
        const int64_t vpt = (nvec + (NT) - 1) / (NT);                                                          \
        if (vpt <= 1) return launch_rmsnorm_bwd_v<kBf16X, NT, 1, kGain>(X, rinv, g, dX, T, K, partial, sms, st); \
        if (vpt <= 2) return launch_rmsnorm_bwd_v<kBf16X, NT, 2, kGain>(X, rinv, g, dX, T, K, partial, sms, st); \
        if (vpt <= 3) return launch_rmsnorm_bwd_v<kBf16X, NT, 3, kGain>(X, rinv, g, dX, T, K, partial, sms, st); \
        return launch_rmsnorm_bwd_v<kBf16X, NT, 4, kGain>(X, rinv, g, dX, T, K, partial, sms, st);               \
    }
    BL_BWD(128)
    BL_BWD(256)
    BL_BWD(512)
    BL_BWD(1024)
#undef BL_BWD
    return 0;
}

template <bool kBf16X>
int launch_rmsnorm_bwd(const void* X, const float* rinv, const float* g, float* dX, int64_t T, int64_t K,
                       float* partial, int sms, cudaStream_t st) {
    if (g != nullptr) return launch_rmsnorm_bwd_g<kBf16X, true>(X, rinv, g, dX, T, K, partial, sms, st);
    return launch_rmsnorm_bwd_g<kBf16X, false>(X, rinv, g, dX, T, K, partial, sms, st);
}

bl_status run_rmsnorm_bwd(const void* X, bl_dtype dt, const float* rinv, const float* g, float* dX, int64_t T,
                          int64_t K, float* dg, void* ws, int sms, cudaStream_t st) {
    float* partial = dg != nullptr ? static_cast<float*>(ws) : nullptr;
    const int grid = dt == BL_BF16 ? launch_rmsnorm_bwd<true>(X, rinv, g, dX, T, K, partial, sms, st)
                                   : launch_rmsnorm_bwd<false>(X, rinv, g, dX, T, K, partial, sms, st);
    BL_TRY(launched("rmsnorm_bwd"));
    if (dg != nullptr) {
        pdl_launch(bl::dg_reduce_kernel, dim3((unsigned)((K + 31) / 32)), dim3(1024), 0, st,
                   static_cast<const float*>(partial), grid, (int)K, dg);
        BL_TRY(launched("dg_reduce"));
    }
    return BL_OK;
}

// ------------------------------------------------------------------------------------
// packed-weight GEMM: tile shape, K split and launch
// ------------------------------------------------------------------------------------
// Packed-weight GEMM on CTA pairs: 256-row weight tiles x bt tokens
// (bt = T rounded up to 32, at most 256), a K split when the tiles fill at most half the
// pairs, the activation ring, and the packed ring in the rest of shared memory.  The grid is
// as many pairs as fit at once, at most one per unit.
template <bool kBf16Out>
bl_status launch_packed2(const int8_t* Xq, const float* sx, int64_t T, int64_t K, const uint8_t* Wpacked,
                         const float* gamma, int64_t N, void* Y, int32_t* acc, int32_t* scratch,
                         size_t scratch_bytes, cudaStream_t st, const DeviceInfo& dev) {
    bl::Pk2Args a2{};
    bl::PkArgs& a = a2.pk;
    a.T = (int)T; a.N = (int)N; a.K = (int)K;
    int64_t bt = (T + 31) / 32 * 32;
    if (bt > bl::kPkMaxBT) bt = bl::kPkMaxBT;
    a.bt = (int)bt;
    a.t_tiles = (int)((T + bt - 1) / bt);
    a.n_tiles = (int)((N + 2 * bl::kPk2Rows - 1) / (2 * bl::kPk2Rows));
    a.k_blocks = (int)((K + 127) / 128);
    const size_t budget = (size_t)dev.max_smem_optin;
    int pstages = (int)((budget - bl::pk2_smem_bytes((int)bt, 0)) / bl::kPkPBytes);
    pstages = std::min(pstages, bl::kPkMaxPStages);
    // the decoder warps stage their share of the last epilogue (16 x 8 KB) in the packed and
    // activation rings
    BL_REQUIRE(pstages >= 2 && (size_t)pstages * bl::kPkPBytes + (size_t)bl::kPk2DStages * bt * 128 >=
                                   16 * 2 * (size_t)bl::kPk2EpiBuf,
               BL_ERR_DEVICE, "packed GEMM: shared memory too small");
    a.pstages = pstages;
    auto kern = bl::tc_gemm_packed2_kernel<kBf16Out>;
    const size_t smem = bl::pk2_smem_bytes((int)bt, pstages);
    // pairs resident at once, per device and token-tile width (the shared memory differs)
    static std::atomic<int> max_clusters[64][bl::kPkMaxBT / 32] = {};
    int dev_id = 0;
    cudaGetDevice(&dev_id);
    if (dev_id < 0 || dev_id >= 64) return fail(BL_ERR_DEVICE, "device ordinal %d out of range", dev_id);
    std::atomic<int>& mc_slot = max_clusters[dev_id][bt / 32 - 1];
    int mc = mc_slot.load();
    if (mc == 0) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, dev.max_smem_optin);
        if (e != cudaSuccess) return fail(BL_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * (unsigned)(dev.sms / 2));
        cfg.blockDim = dim3(bl::kPk2Threads);
        cfg.dynamicSmemBytes = smem;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
        if (e != cudaSuccess) return fail(BL_ERR_CUDA, "cudaOccupancyMaxActiveClusters: %s", cudaGetErrorString(e));
        if (n < 1) return fail(BL_ERR_DEVICE, "no 2-CTA cluster of the packed GEMM fits on the device");
        mc = n;
        mc_slot.store(mc);
    }
    const int64_t base = (int64_t)a.n_tiles * a.t_tiles;
    int splits = 1;
    if (2 * base <= mc) {
        // the partial sums and their second launch cost more than a second wave of units
        // returns, so K is split only when the tiles fill at most half the pairs, into as many
        // units as one wave holds, each at least 8 k-blocks (4 stages) long
        int64_t sp = std::min<int64_t>(8, (int64_t)mc / base);
        sp = std::min<int64_t>(sp, a.k_blocks / 8);
        sp = std::min<int64_t>(sp, (int64_t)(scratch_bytes / ((size_t)T * N * sizeof(int32_t))));
        splits = (int)std::max<int64_t>(1, sp);
    }
    a.splits = splits;
    a.sx = sx; a.gamma = gamma; a.y = Y;
    a.acc = splits > 1 ? scratch : acc;
    a.wait_ns = g_wait_ns.load();
    CUtensorMap tp, tx, ty, tacc;
    BL_TRY(make_tmap(&tp, Wpacked, kTmU8, (uint64_t)(K / 4), (uint64_t)N, 128, bl::kPk2Rows));
    BL_TRY(make_tmap(&tx, Xq, kTmU8, (uint64_t)K, (uint64_t)T, 128, (uint32_t)(bt / 2)));
    // the epilogue's TMA stores: 32 rows x 32 tokens per box, no swizzle
    BL_TRY(make_tmap(&ty, Y, kBf16Out ? kTmBf16 : kTmF32, (uint64_t)N, (uint64_t)T, 32, 32, false));
    std::memset(&tacc, 0, sizeof(tacc));
    if (splits > 1)
        BL_TRY(make_tmap3_i32(&tacc, scratch, (uint64_t)N, (uint64_t)T, (uint64_t)splits, 32, 32));
    else if (acc != nullptr)
        BL_TRY(make_tmap(&tacc, acc, kTmI32, (uint64_t)N, (uint64_t)T, 32, 32, false));
    const int64_t units = base * splits;
    const unsigned clusters = (unsigned)std::min<int64_t>(units, mc);
    pdl_launch(kern, dim3(2 * clusters), dim3(bl::kPk2Threads), smem, st, tp, tx, ty, tacc, a2);
    BL_TRY(launched("tc_gemm_packed2"));
    if (splits > 1) {
        const int64_t nv = T * N / 4;
        pdl_launch(bl::pk_finalize_kernel<kBf16Out>, dim3((unsigned)std::min<int64_t>((nv + 255) / 256, (int64_t)dev.sms * 8)),
                   dim3(256), 0, st, static_cast<const int32_t*>(scratch), splits, sx, gamma, (int)T, (int)N, Y, acc);
        BL_TRY(launched("pk_finalize"));
    }
    return BL_OK;
}

// Row kernels keep a whole row in registers: d_in is limited to 16384.
constexpr int64_t kMaxRowK = 16384;

// One block per SM (at most one per row group) of 16 warps (12 for two n-tiles, whose
// accumulators need more registers).
template <int NTILES, bool kBf16Out = false>
bl_status launch_gemv(const uint8_t* Wpacked, const float* gamma, int gamma_stride, int64_t N, int64_t K,
                      const int8_t* xq, const float* sx, int64_t B, void* y, int32_t* acc, cudaStream_t st,
                      const DeviceInfo& dev) {
    constexpr int WB = NTILES == 1 ? 16 : 12;
    const int64_t n_rg = N / 16;
    const int64_t nb = n_rg < dev.sms ? n_rg : dev.sms;
    const int max_rgs = (int)((n_rg + nb - 1) / nb);
    const size_t smem = bl::gemv_smem_bytes((int)B, (int)K, max_rgs);
    BL_REQUIRE(smem <= (size_t)dev.max_smem_optin, BL_ERR_UNSUPPORTED_SHAPE,
               "GEMV needs %zu bytes of shared memory for B = %lld, K = %lld; at most %d fit", smem, (long long)B,
               (long long)K, dev.max_smem_optin);
    auto kern = bl::ternary_gemv_kernel<NTILES, WB, kBf16Out>;
    static std::atomic<uint64_t> attr_set{0};   // bit d: attribute set on device d
    int dev_id = 0;
    cudaGetDevice(&dev_id);
    if (dev_id < 0 || dev_id >= 64) return fail(BL_ERR_DEVICE, "device ordinal %d out of range", dev_id);
    if (!(attr_set.load() & (1ull << dev_id))) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, dev.max_smem_optin);
        if (e != cudaSuccess) return fail(BL_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        attr_set.fetch_or(1ull << dev_id);
    }
    pdl_launch(kern, dim3((unsigned)nb), dim3(WB * 32), smem, st, Wpacked, gamma, gamma_stride, (int)N, (int)K, xq,
               sx, (int)B, y, acc, g_wait_ns.load());
    return launched("ternary_gemv");
}

// ------------------------------------------------------------------------------------
// optimizer step, with its own per-matrix clip or with a given coefficient
// ------------------------------------------------------------------------------------
bl_status check_optimizer(const float* W, const float* dW, const float* m, const float* v, int64_t N, int64_t K,
                          float lr, float beta1, float beta2, float eps, float weight_decay, const int32_t* step,
                          const int8_t* Wq_i8, const uint16_t* Wq_bf16, const uint8_t* Wpacked, const float* gamma,
                          const void* ws, size_t ws_bytes) {
    BL_TRY(check_ptr(W, "W", true));
    BL_TRY(check_ptr(dW, "dW", true));
    BL_TRY(check_ptr(m, "m", true));
    BL_TRY(check_ptr(v, "v", true));
    BL_TRY(check_ptr(step, "step", true));
    BL_TRY(check_ptr(gamma, "gamma", false));
    BL_TRY(check_ptr(Wq_i8, "Wq_i8", false));
    BL_TRY(check_ptr(Wq_bf16, "Wq_bf16", false));
    BL_TRY(check_ptr(Wpacked, "Wpacked", false));
    BL_TRY(check_ptr(ws, "ws", true));
    BL_TRY(check_dims(1, N, K));
    BL_REQUIRE(gamma != nullptr || (Wq_i8 == nullptr && Wq_bf16 == nullptr && Wpacked == nullptr), BL_ERR_INVALID_ARG,
               "the next step's codes need gamma");
    BL_REQUIRE(lr >= 0.0f && lr <= 1e30f, BL_ERR_INVALID_ARG, "lr must be finite and >= 0");
    BL_REQUIRE(beta1 >= 0.0f && beta1 < 1.0f && beta2 >= 0.0f && beta2 < 1.0f, BL_ERR_INVALID_ARG,
               "betas must be in [0, 1)");
    BL_REQUIRE(eps > 0.0f && eps <= 1e30f, BL_ERR_INVALID_ARG, "eps must be finite and > 0");
    BL_REQUIRE(weight_decay >= 0.0f && weight_decay <= 1e30f, BL_ERR_INVALID_ARG,
               "weight_decay must be finite and >= 0");
    BL_REQUIRE(ws_bytes >= opt_ws_bytes(), BL_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", opt_ws_bytes(),
               ws_bytes);
    return BL_OK;
}

bl::AdamwArgs adamw_args(float lr, float beta1, float beta2, float eps, float weight_decay, float max_norm) {
    bl::AdamwArgs a{};
    a.lr = lr;
    a.beta1 = beta1;
    a.beta2 = beta2;
    a.eps = eps;
    a.decay = (float)(1.0 - (double)lr * (double)weight_decay);
    a.omb1 = (float)(1.0 - (double)beta1);
    a.omb2 = (float)(1.0 - (double)beta2);
    a.max_norm = max_norm;
    return a;
}

bl_status run_optimizer(float* W, const float* dW, float* m, float* v, int64_t n, const bl::AdamwArgs& a,
                        const float* coef, int32_t* step, int8_t* Wq_i8, uint16_t* Wq_bf16, uint8_t* Wpacked,
                        float* gamma, void* ws, cudaStream_t st, const DeviceInfo& dev) {
    const int parts = bl::wq_num_partials(n);
    uint8_t* wsb = static_cast<uint8_t*>(ws);
    double* gpart = reinterpret_cast<double*>(wsb);
    double* wpart = reinterpret_cast<double*>(wsb + kOptWpartOffset);
    int32_t* step_next = reinterpret_cast<int32_t*>(wsb + kOptStepOffset);
    bl::AdamwScalars* ready = nullptr;
    if (coef != nullptr) {
        static_assert(sizeof(bl::AdamwScalars) <= 16, "the scalars take the published step's place");
        ready = reinterpret_cast<bl::AdamwScalars*>(wsb + kOptStepOffset);
        pdl_launch(bl::adamw_scalars_kernel, dim3(1), dim3(32), 0, st, a, coef, step, ready);
        BL_TRY(launched("adamw_scalars"));
    } else {
        pdl_launch(bl::grad_sumsq_partial_kernel, dim3(parts), dim3(bl::kWqThreads), 0, st, dW, n, gpart,
                   static_cast<const int32_t*>(step), step_next);
        BL_TRY(launched("grad_sumsq_partial"));
    }
    pdl_launch(bl::adamw_clamp_kernel, dim3(parts), dim3(bl::kWqThreads), 0, st, W, dW, m, v, n,
               static_cast<const double*>(gpart), parts, a, static_cast<const int32_t*>(step_next), step,
               static_cast<const bl::AdamwScalars*>(ready), gamma != nullptr ? wpart : static_cast<double*>(nullptr));
    BL_TRY(launched("adamw_clamp"));
    if (gamma == nullptr) return BL_OK;
    // the next step's codes from the |W_new| partials written above (the quantiser's pass 2)
    return run_ternary(W, n, wpart, parts, Wq_i8, Wq_bf16, Wpacked, gamma, st, dev);
}

// ------------------------------------------------------------------------------------
// global gradient norm and clipping
// ------------------------------------------------------------------------------------
size_t gc_ws_bytes() { return sizeof(double) * bl::kGcMaxPartials; }

bl_status check_grads(const void* const* grads, void* const* out, const int64_t* numel, const bl_dtype* dtypes,
                      int64_t count, float max_norm, const float* norm, const float* coef, const void* ws,
                      size_t ws_bytes) {
    BL_REQUIRE(count >= 0 && count <= (1 << 24), BL_ERR_INVALID_ARG, "count must be in [0, 2^24], got %lld",
               (long long)count);
    BL_REQUIRE(count == 0 || (grads != nullptr && numel != nullptr && dtypes != nullptr), BL_ERR_INVALID_ARG,
               "grads, numel and dtypes must not be NULL");
    BL_REQUIRE(max_norm == max_norm && max_norm <= 1e30f, BL_ERR_INVALID_ARG, "max_norm must be finite");
    BL_REQUIRE(norm != nullptr && coef != nullptr, BL_ERR_INVALID_ARG, "norm and coef must not be NULL");
    BL_REQUIRE(((reinterpret_cast<uintptr_t>(norm) | reinterpret_cast<uintptr_t>(coef)) & 3u) == 0,
               BL_ERR_MISALIGNED, "norm and coef must be 4-byte aligned");
    BL_TRY(check_ptr(ws, "ws", true));
    BL_REQUIRE(ws_bytes >= gc_ws_bytes(), BL_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", gc_ws_bytes(),
               ws_bytes);
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) {
        BL_TRY(check_dtype(dtypes[i]));
        BL_REQUIRE(numel[i] >= 0 && numel[i] <= (int64_t(1) << 40), BL_ERR_INVALID_ARG,
                   "gradient %lld: size %lld out of range", (long long)i, (long long)numel[i]);
        if (numel[i] == 0) continue;
        total += numel[i];
        BL_REQUIRE(total <= (int64_t(1) << 40), BL_ERR_UNSUPPORTED_SHAPE, "more than 2^40 elements");
        const uintptr_t mask = dtypes[i] == BL_BF16 ? 1u : 3u;
        BL_REQUIRE(grads[i] != nullptr && (out == nullptr || out[i] != nullptr), BL_ERR_INVALID_ARG,
                   "gradient %lld must not be NULL", (long long)i);
        BL_REQUIRE((reinterpret_cast<uintptr_t>(grads[i]) & mask) == 0 &&
                       (out == nullptr || (reinterpret_cast<uintptr_t>(out[i]) & mask) == 0),
                   BL_ERR_MISALIGNED, "gradient %lld is not aligned to its elements", (long long)i);
    }
    return BL_OK;
}

// Elements per chunk: four chunks a block when every block of the grid has work, between 16 KB
// and 256 KB of fp32, so that a few large matrices and many small tensors both spread evenly.
int64_t gc_chunk(int64_t total, int blocks) {
    int64_t c = 4096;
    while (c < 65536 && total / c > 4 * (int64_t)blocks) c *= 2;
    return c;
}

// One table of the list: gradients [first, ...) as far as they fit, empty ones left out.
// Returns the index behind the last one taken.
template <int kMax>
int64_t gc_fill(bl::GcTable<kMax>& tab, const void* const* grads, void* const* out, const int64_t* numel,
                const bl_dtype* dtypes, int64_t first, int64_t count, int64_t chunk) {
    tab.count = tab.chunks = 0;
    tab.chunk = chunk;
    int64_t i = first;
    for (; i < count; ++i) {
        if (numel[i] == 0) continue;                   // also behind a full table: they need no launch
        if (tab.count == kMax) break;
        bl::GcTensor& t = tab.t[tab.count++];
        t.g = grads[i];
        t.out = out != nullptr ? out[i] : nullptr;
        t.n = numel[i];
        t.first_chunk = tab.chunks;
        t.bf16 = dtypes[i] == BL_BF16;
        tab.chunks += (int32_t)((numel[i] + chunk - 1) / chunk);
    }
    return i;
}

template <int kMax>
bl_status run_grads_t(const void* const* grads, void* const* out, const int64_t* numel, const bl_dtype* dtypes,
                      int64_t count, float max_norm, float* norm, float* coef, double* partials, int blocks,
                      int64_t chunk, cudaStream_t st) {
    bl::GcTable<kMax> tab;
    std::memset(&tab, 0, sizeof(tab));
    int64_t i = 0;
    int add = 0;
    do {
        i = gc_fill(tab, grads, out, numel, dtypes, i, count, chunk);
        pdl_launch(bl::grad_sumsq_kernel<kMax>, dim3((unsigned)blocks), dim3(bl::kGcThreads), 0, st, tab, add,
                   partials);
        BL_TRY(launched("grad_sumsq"));
        add = 1;
    } while (i < count);
    if (out == nullptr) {
        pdl_launch(bl::grad_norm_kernel, dim3(1), dim3(bl::kGcThreads), 0, st, static_cast<const double*>(partials),
                   blocks, max_norm, norm, coef);
        return launched("grad_norm");
    }
    i = 0;
    do {
        i = gc_fill(tab, grads, out, numel, dtypes, i, count, chunk);
        pdl_launch(chunk >= bl::kGcWide ? bl::grad_scale_kernel<kMax, true> : bl::grad_scale_kernel<kMax, false>,
                   dim3((unsigned)blocks), dim3(bl::kGcThreads), 0, st, tab, static_cast<const double*>(partials), blocks,
                   max_norm, norm, coef);
        BL_TRY(launched("grad_scale"));
    } while (i < count);
    return BL_OK;
}

bl_status run_grads(const void* const* grads, void* const* out, const int64_t* numel, const bl_dtype* dtypes,
                    int64_t count, float max_norm, float* norm, float* coef, void* ws, cudaStream_t st,
                    const DeviceInfo& dev) {
    int64_t total = 0, full = 0;
    for (int64_t i = 0; i < count; ++i) {
        total += numel[i];
        full += numel[i] != 0;
    }
    const int most = std::min(4 * dev.sms, (int)bl::kGcMaxPartials);
    const int64_t chunk = gc_chunk(total, most);
    // no more blocks than chunks
    const int blocks = (int)std::max<int64_t>(1, std::min<int64_t>(most, total / chunk + full));
    double* partials = static_cast<double*>(ws);
    if (full <= bl::kGcSmall)
        return run_grads_t<bl::kGcSmall>(grads, out, numel, dtypes, count, max_norm, norm, coef, partials, blocks,
                                         chunk, st);
    return run_grads_t<bl::kGcLarge>(grads, out, numel, dtypes, count, max_norm, norm, coef, partials, blocks, chunk,
                                     st);
}

// ------------------------------------------------------------------------------------
// residual norms
// ------------------------------------------------------------------------------------
bl_status check_residual(bl_dtype x_dt, bl_dtype y_dt, int64_t T, int64_t K, int post_norm, const float* g_post,
                         bl_gate gate_kind, const void* gate, float alpha, float beta) {
    BL_TRY(check_dtype(x_dt));
    BL_TRY(check_dtype(y_dt));
    BL_REQUIRE(x_dt == BL_F32 || y_dt == BL_BF16, BL_ERR_INVALID_ARG, "a bf16 residual takes a bf16 block");
    BL_REQUIRE(T >= 1 && K >= 1, BL_ERR_INVALID_ARG, "sizes must be positive (T=%lld K=%lld)", (long long)T,
               (long long)K);
    BL_REQUIRE(T <= kMaxDim, BL_ERR_UNSUPPORTED_SHAPE, "sizes must be < 2^31");
    BL_REQUIRE(K <= kMaxRowK, BL_ERR_UNSUPPORTED_SHAPE, "K must be <= %lld for the row kernels, got %lld",
               (long long)kMaxRowK, (long long)K);
    BL_REQUIRE((int)gate_kind >= BL_GATE_NONE && (int)gate_kind <= BL_GATE_ELEMENT, BL_ERR_INVALID_ARG,
               "unknown gate kind %d", (int)gate_kind);
    BL_REQUIRE((gate != nullptr) == (gate_kind != BL_GATE_NONE), BL_ERR_INVALID_ARG,
               "gate and gate_kind do not agree");
    BL_TRY(check_ptr(gate, "gate", false));
    BL_TRY(check_ptr(g_post, "g_post", false));
    BL_REQUIRE(g_post == nullptr || post_norm, BL_ERR_INVALID_ARG, "g_post needs post_norm");
    BL_REQUIRE(alpha - alpha == 0.0f && beta - beta == 0.0f, BL_ERR_INVALID_ARG, "alpha and beta must be finite");
    return BL_OK;
}

size_t rn_ws_bytes(int64_t K) {
    return sizeof(double) * bl::kRnMaxBlocks + 2 * sizeof(float) * (size_t)bl::kRnMaxBlocks * (size_t)K;
}

template <bool kBf16X, bool kBf16Y, bool kWarpRow, int E, int NT, int VPT>
void launch_residual_norm_v(const bl::RnFwdArgs& a, cudaStream_t st) {
    constexpr int kRows = kWarpRow ? NT / 32 : 1;
    const dim3 grid((unsigned)(((int64_t)a.T + kRows - 1) / kRows));
    if (a.gate_kind == bl::kGateElement)
        pdl_launch(bl::residual_norm_kernel<kBf16X, kBf16Y, kWarpRow, E, NT, VPT, true>, grid, dim3(NT), 0, st, a);
    else
        pdl_launch(bl::residual_norm_kernel<kBf16X, kBf16Y, kWarpRow, E, NT, VPT, false>, grid, dim3(NT), 0, st, a);
}

constexpr size_t kRnSmem = 224 * 1024;   // dynamic shared memory of a ring block (1 KB static beside it)

// Bytes of a row in the forward's ring, and of the gains beside it.
template <bool kBf16X, bool kBf16Y>
size_t rn_fwd_row(const bl::RnFwdArgs& a) {
    const bool odd = a.K % 8 != 0;
    return bl::rn_pitch(odd, a.K * (kBf16X ? 2u : 4u)) +
           (size_t)bl::rn_pitch(odd, a.K * (kBf16Y ? 2u : 4u)) * (a.gate_kind == bl::kGateElement ? 2 : 1);
}
size_t rn_gain_bytes(int cols) { return 2 * (((size_t)cols * 4 + 15) & ~size_t(15)); }

// The ring kernel: as many row groups, then stages, as shared memory holds beside the gains.
template <bool kBf16X, bool kBf16Y, int TG, int kMaxThreads, int EPT, bool kGateElem, bool kSm, bool kOdd>
bl_status launch_residual_norm_ring_v(const bl::RnFwdArgs& a, cudaStream_t st, const DeviceInfo& dev) {
    auto kern = bl::residual_norm_ring_kernel<kBf16X, kBf16Y, TG, kMaxThreads, EPT, kGateElem, kSm, kOdd>;
    const size_t row = rn_fwd_row<kBf16X, kBf16Y>(a), gains = kSm ? rn_gain_bytes(a.K) : 0;
    constexpr size_t limit = kRnSmem;
    const int groups = (int)std::max<size_t>(1, std::min<size_t>(kMaxThreads / TG, (limit - gains) / row));
    const int stages = (int)std::max<size_t>(1, std::min<size_t>(bl::kRnMaxStages, (limit - gains) / (row * groups)));
    const size_t smem = gains + row * groups * stages;
    BL_REQUIRE(smem <= limit, BL_ERR_DEVICE, "residual norm: shared memory too small");
    static std::atomic<uint64_t> attr_set{0};   // bit d: attribute set on device d
    int dev_id = 0;
    cudaGetDevice(&dev_id);
    if (!(attr_set.load() & (1ull << dev_id))) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)limit);
        if (e != cudaSuccess) return fail(BL_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        attr_set.fetch_or(1ull << dev_id);
    }
    const int64_t blocks = std::min<int64_t>(((int64_t)a.T + groups - 1) / groups, dev.sms);
    pdl_launch(kern, dim3((unsigned)blocks), dim3((unsigned)(TG * groups)), smem, st, a, stages, g_wait_ns.load());
    return launched("residual_norm_ring");
}

template <bool kBf16X, bool kBf16Y, int TG, int kMaxThreads, int EPT, bool kSm = true, bool kOdd = false>
bl_status launch_residual_norm_ring(const bl::RnFwdArgs& a, cudaStream_t st, const DeviceInfo& dev) {
    if (a.gate_kind == bl::kGateElement)
        return launch_residual_norm_ring_v<kBf16X, kBf16Y, TG, kMaxThreads, EPT, true, kSm, kOdd>(a, st, dev);
    return launch_residual_norm_ring_v<kBf16X, kBf16Y, TG, kMaxThreads, EPT, false, kSm, kOdd>(a, st, dev);
}

// Rows of whole 16-byte vectors (8 elements) take the vector kernels, others one element at a
// time; a warp per short row, a block per long one.
template <bool kBf16X, bool kBf16Y>
bl_status launch_residual_norm(const bl::RnFwdArgs& a, cudaStream_t st, const DeviceInfo& dev) {
    const int nvec = a.K / 8;
    // The ring pays from about a million and a half elements on.  Where it begins to depends on the
    // width (us with the ring / without; bf16 alone, then fp32 beside bf16, quantised, inputs beyond L2):
    //   1.26 M elements: 4915 x 256 7.2 / 6.0, 7.9 / 6.6; 1228 x 1024 8.7 / 5.8, 7.9 / 6.2;
    //                    307 x 4096 9.1 / 7.2, 8.6 / 9.2; 76 x 16384 9.0 / 9.6, 10.1 / 10.0
    //   2.5 M:           9830 x 256 10.2 / 9.9, 11.2 / 10.4; 2457 x 1024 10.0 / 9.6, 13.3 / 10.2;
    //                    614 x 4096 10.3 / 11.4, 14.1 / 13.5; 153 x 16384 14.3 / 17.8, 16.1 / 19.0
    // Rows that are no whole vectors (bf16, norm output): 1672 x 1003 9.8 / 10.6, 335 x 5001 14.0 / 21.9,
    // 102 x 16381 16.3 / 21.2, but 25811 x 65 26 / 11 (a warp a row, with a row's copies for 65 elements)
    const bool ring = (int64_t)a.T * a.K >= (3 << 19);
    if (a.K % 8 != 0) {
        if (ring) {
            const size_t row = rn_fwd_row<kBf16X, kBf16Y>(a), gains = rn_gain_bytes(a.K);
            if (a.K <= 512) return launch_residual_norm_ring<kBf16X, kBf16Y, 32, 512, 16, true, true>(a, st, dev);
            if (a.K <= 2048) return launch_residual_norm_ring<kBf16X, kBf16Y, 128, 768, 16, true, true>(a, st, dev);
            if (a.K <= 8192) return launch_residual_norm_ring<kBf16X, kBf16Y, 512, 1024, 16, true, true>(a, st, dev);
            if (row + gains <= kRnSmem)
                return launch_residual_norm_ring<kBf16X, kBf16Y, 1024, 1024, 16, true, true>(a, st, dev);
            return launch_residual_norm_ring<kBf16X, kBf16Y, 1024, 1024, 16, false, true>(a, st, dev);
        }
        if (a.K <= 128) launch_residual_norm_v<kBf16X, kBf16Y, true, 1, 256, 4>(a, st);
        else if (a.K <= 1024) launch_residual_norm_v<kBf16X, kBf16Y, false, 1, 256, 4>(a, st);
        else if (a.K <= 4096) launch_residual_norm_v<kBf16X, kBf16Y, false, 1, 1024, 4>(a, st);
        else launch_residual_norm_v<kBf16X, kBf16Y, false, 1, 1024, 16>(a, st);
        return launched("residual_norm");
    }
    if (ring) {
        // 32 elements a thread amortise a row's reductions and scalars (16384 x 4096, bf16: 117 us
        // against 126 with 16).  Six groups of 128 threads, but four where an fp32 residual stands
        // beside a bf16 block: their rows then have two stages.  16384 rows, us with up to 768 / 512
        // threads, fp32 beside bf16: 1024 columns 44.7 / 41.6, 2048 82.7 / 78.3, 4096 162 / 150, 8192
        // 316 / 271 (5120 the other way: 172 / 206); bf16 alone: 35.6 / 35.2, 62.3 / 64.6, 111 / 122,
        // 215 / 249; fp32 alone: 53.6 / 53.6, 98 / 103, 196 / 202, 390 / 390.
        constexpr int kCap = kBf16X != kBf16Y ? 512 : 768;
        if (nvec <= 32) return launch_residual_norm_ring<kBf16X, kBf16Y, 32, 768, 8>(a, st, dev);
        if (nvec <= 64) return launch_residual_norm_ring<kBf16X, kBf16Y, 32, 768, 16>(a, st, dev);
        if (nvec <= 128) return launch_residual_norm_ring<kBf16X, kBf16Y, 32, kCap, 32>(a, st, dev);
        if (nvec <= 256) return launch_residual_norm_ring<kBf16X, kBf16Y, 64, kCap, 32>(a, st, dev);
        if (nvec <= 512) return launch_residual_norm_ring<kBf16X, kBf16Y, 128, kCap, 32>(a, st, dev);
        if (nvec <= 1024) return launch_residual_norm_ring<kBf16X, kBf16Y, 256, kCap, 32>(a, st, dev);
        // Longer rows: the gains in shared memory if a row fits beside them (4096 x 11008, 100 us
        // against 139 from global memory), two rows at once if two fit (100 against 113 us)
        const size_t row = rn_fwd_row<kBf16X, kBf16Y>(a), gains = rn_gain_bytes(a.K);
        if (2 * row + gains <= kRnSmem) return launch_residual_norm_ring<kBf16X, kBf16Y, 512, 1024, 32>(a, st, dev);
        if (row + gains <= kRnSmem) return launch_residual_norm_ring<kBf16X, kBf16Y, 512, 512, 32>(a, st, dev);
        return launch_residual_norm_ring<kBf16X, kBf16Y, 512, 1024, 32, false>(a, st, dev);
    }
    if (nvec <= 32) launch_residual_norm_v<kBf16X, kBf16Y, true, 8, 256, 1>(a, st);
    else if (nvec <= 64) launch_residual_norm_v<kBf16X, kBf16Y, true, 8, 256, 2>(a, st);
    else if (nvec <= 128) launch_residual_norm_v<kBf16X, kBf16Y, false, 8, 128, 1>(a, st);
    else if (nvec <= 256) launch_residual_norm_v<kBf16X, kBf16Y, false, 8, 256, 1>(a, st);
    else if (nvec <= 512) launch_residual_norm_v<kBf16X, kBf16Y, false, 8, 512, 1>(a, st);
    else if (nvec <= 1024) launch_residual_norm_v<kBf16X, kBf16Y, false, 8, 512, 2>(a, st);
    else launch_residual_norm_v<kBf16X, kBf16Y, false, 8, 1024, 2>(a, st);
    return launched("residual_norm");
}

// Columns of a row that each of cl blocks takes: whole 16-byte vectors of bf16 where the row is.
int rn_cols(int K, int cl) { return K % 8 != 0 ? (K + cl - 1) / cl : (K / 8 + cl - 1) / cl * 8; }

// Bytes of one row in the backward's ring.
template <bool kBf16X, bool kBf16Y>
size_t rn_bwd_row(const bl::RnBwdArgs& a, int cols) {
    const bool odd = a.K % 8 != 0;
    const size_t f = bl::rn_pitch(odd, cols * 4u), x = bl::rn_pitch(odd, cols * (kBf16X ? 2u : 4u)),
                 y = bl::rn_pitch(odd, cols * (kBf16Y ? 2u : 4u));
    return (a.dx != nullptr ? f : 0) + (a.dh != nullptr ? f + x : 0) + y * (a.gate_kind == bl::kGateElement ? 2 : 1);
}

// G: partial rows (blocks, or clusters of kCl); Gs: blocks.
template <bool kBf16X, bool kBf16Y, bool kElem, int TG, int EPT, int kCl, bool kOdd = false>
bl_status launch_residual_norm_bwd_ring(const bl::RnBwdArgs& a, cudaStream_t st, const DeviceInfo& dev, int* G,
                                        int* Gs) {
    auto kern = bl::residual_norm_bwd_ring_kernel<kBf16X, kBf16Y, TG, EPT, kCl, kElem, kOdd>;
    const int cols = rn_cols(a.K, kCl);
    const size_t row = rn_bwd_row<kBf16X, kBf16Y>(a, cols), gains = rn_gain_bytes(cols);
    int groups = 512 / TG;
    while (groups > 1 && gains + 2 * row * groups > kRnSmem) --groups;
    const int stages = (int)std::min<size_t>(bl::kRnMaxStages, (kRnSmem - gains) / (row * groups));
    const size_t smem = std::max(gains + row * groups * stages, gains * groups);   // the groups' sums at the end
    BL_REQUIRE(stages >= 2 && smem <= kRnSmem && cols <= TG * EPT, BL_ERR_DEVICE,
               "residual norm backward: shared memory too small");
    static std::atomic<int> slots[64] = {};
    int dev_id = 0;
    cudaGetDevice(&dev_id);
    int n = dev_id >= 0 && dev_id < 64 ? slots[dev_id].load() : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3((unsigned)(TG * groups));
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCl;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    if (n == 0) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRnSmem);
        if (e != cudaSuccess) return fail(BL_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        n = dev.sms;
        if (kCl > 1) {
            cfg.gridDim = dim3((unsigned)(dev.sms / kCl * kCl));
            cfg.dynamicSmemBytes = kRnSmem;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
            if (e != cudaSuccess)
                return fail(BL_ERR_CUDA, "cudaOccupancyMaxActiveClusters: %s", cudaGetErrorString(e));
            if (n < 1) return fail(BL_ERR_DEVICE, "no cluster of %d blocks of the residual norm fits on the device", kCl);
        }
        if (dev_id >= 0 && dev_id < 64) slots[dev_id].store(n);
    }
    *G = (int)std::min<int64_t>(((int64_t)a.T + groups - 1) / groups, std::min(n, (int)bl::kRnMaxBlocks / kCl));
    *Gs = *G * kCl;
    cfg.gridDim = dim3((unsigned)*Gs);
    cfg.dynamicSmemBytes = smem;
    cfg.numAttrs = 2;
    cudaLaunchKernelEx(&cfg, kern, a, cols, stages, g_wait_ns.load());
    return launched("residual_norm_bwd_ring");
}

template <bool kBf16X, bool kBf16Y, bool kElem>
bl_status launch_residual_norm_bwd_v(const bl::RnBwdArgs& a, cudaStream_t st, const DeviceInfo& dev, int* G, int* Gs) {
    // the gains and two stages (a row's first pass runs before the last row's stage is given back)
    auto fits = [&](int cl, int groups) {
        const int cols = rn_cols(a.K, cl);
        return rn_gain_bytes(cols) + 2 * rn_bwd_row<kBf16X, kBf16Y>(a, cols) * groups <= kRnSmem;
    };
#define BL_RN(...) return launch_residual_norm_bwd_ring<kBf16X, kBf16Y, kElem, __VA_ARGS__>(a, st, dev, G, Gs)
    if (a.K % 8 != 0) {
        if (a.K <= 512) BL_RN(32, 16, 1, true);
        if (a.K <= 2048) BL_RN(128, 16, 1, true);
        if (a.K <= 8192 && fits(1, 1)) BL_RN(512, 16, 1, true);
        if (fits(2, 1)) BL_RN(512, 16, 2, true);
        BL_RN(512, 8, 4, true);
    }
    // 16 columns a thread amortise a row's reduction best (16384 rows of bf16, us against those with 8:
    // 384 columns 30.0 / 32.0, 768 47 / 54, 1536 78 / 93, 4096 185 / 204, 5120 244 / 351), as long as two
    // stages of all the groups fit (fp32, 2048: 131 / 126, 4096: 248 / 241; fp32 beside bf16, 4096:
    // 242 / 212, but 2048: 106 / 112).  Up to 256 columns 8 leave no lane idle (128: 19.3 / 17.9).
    if (a.K <= 256) BL_RN(32, 8, 1);
    if (a.K <= 512) BL_RN(32, 16, 1);
    if (a.K <= 1024 && fits(1, 8)) BL_RN(64, 16, 1);
    if (a.K <= 1024) BL_RN(128, 8, 1);
    if (a.K <= 2048 && fits(1, 4)) BL_RN(128, 16, 1);
    if (a.K <= 2048) BL_RN(256, 8, 1);
    if (a.K <= 4096 && fits(1, 2)) BL_RN(256, 16, 1);
    if (a.K <= 4096) BL_RN(512, 8, 1);
    if (a.K <= 8192 && fits(1, 1)) BL_RN(512, 16, 1);
    if (a.K <= 8192) BL_RN(512, 8, 2);
    if (fits(2, 1)) BL_RN(512, 16, 2);
    BL_RN(512, 8, 4);
#undef BL_RN
}

template <bool kBf16X, bool kBf16Y>
bl_status launch_residual_norm_bwd(const bl::RnBwdArgs& a, cudaStream_t st, const DeviceInfo& dev, int* G, int* Gs) {
    if (a.gate_kind == bl::kGateElement) return launch_residual_norm_bwd_v<kBf16X, kBf16Y, true>(a, st, dev, G, Gs);
    return launch_residual_norm_bwd_v<kBf16X, kBf16Y, false>(a, st, dev, G, Gs);
}

// ------------------------------------------------------------------------------------
// 8-bit linear, few tokens
// ------------------------------------------------------------------------------------
// Clusters of `splits` CTAs (all the shared memory, one CTA per SM) that are resident at once.
template <bool kBf16Out, int kpb>
bl_status i8_slots(int splits, int dev_id, const DeviceInfo& dev, int* out) {
    static std::atomic<int> cache[64][4] = {};
    const int idx = splits == 1 ? 0 : splits == 2 ? 1 : splits == 4 ? 2 : 3;
    int n = cache[dev_id][idx].load();
    if (n == 0) {
        auto kern = bl::gemm_int8_few_kernel<kBf16Out, kpb>;
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, dev.max_smem_optin);
        if (e != cudaSuccess) return fail(BL_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        if (splits == 1) {
            n = dev.sms;
        } else {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)(dev.sms / splits * splits));
            cfg.blockDim = dim3(bl::kI8Threads);
            cfg.dynamicSmemBytes = dev.max_smem_optin;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = (unsigned)splits;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
            if (e != cudaSuccess)
                return fail(BL_ERR_CUDA, "cudaOccupancyMaxActiveClusters: %s", cudaGetErrorString(e));
            if (n < 1) return fail(BL_ERR_DEVICE, "no cluster of %d CTAs of the int8 GEMM fits on the device", splits);
        }
        cache[dev_id][idx].store(n);
    }
    *out = n;
    return BL_OK;
}

template <bool kBf16Out, int kpb>
bl_status launch_int8_few(const CUtensorMap& tw, const CUtensorMap& tx, const bl::I8Args& a, int64_t tiles,
                          cudaStream_t st, int dev_id, const DeviceInfo& dev) {
    auto kern = bl::gemm_int8_few_kernel<kBf16Out, kpb>;
    int slots = 0;
    BL_TRY((i8_slots<kBf16Out, kpb>(a.splits, dev_id, dev, &slots)));   // sets the kernel's attributes
    const size_t smem = bl::i8_smem_bytes(a.stages, kpb, a.a_pitch, a.bt);
    // a split's partial sums lie over the ring
    BL_REQUIRE(smem <= (size_t)dev.max_smem_optin && a.k_steps >= a.splits &&
                   (a.splits == 1 || bl::i8_ring_bytes(a.stages, kpb, a.a_pitch, a.bt) >= (size_t)a.bt * 512),
               BL_ERR_DEVICE, "int8 GEMM: shared memory too small");
    if (a.splits == 1) {
        pdl_launch(kern, dim3((unsigned)std::min<int64_t>(tiles, dev.sms)), dim3(bl::kI8Threads), smem, st, tw, tx, a);
    } else {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(tiles * a.splits));   // one tile per cluster
        cfg.blockDim = dim3(bl::kI8Threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)a.splits;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        cudaLaunchKernelEx(&cfg, kern, tw, tx, a);
    }
    return launched("gemm_int8_few");
}

// Tiles and K split of the few-token kernel, and their cost: the least time on the busiest SM, in rows
// of 128 bytes: of each k-block the weight rows and the tokens, and kStep for issuing it (0.08 us); a
// split pays for its join (two cluster barriers and the way through distributed shared memory, 1 us)
// and for the partial sums' own bytes.  One token: 4096 x 4096 7.2 us split in 4 (128 rows), 7.6 whole
// (28 rows); 11008 x 4096 20.0 split in 4, 10.7 whole (75 rows).
template <bool kBf16Out>
bl_status i8_plan(bl::I8Args& a, int64_t* cost_out, int dev_id, const DeviceInfo& dev) {
    constexpr int64_t kStep = 28, kJoin = 350;
    const int k_blocks = (a.K + 127) / 128;
    a.bt = std::min((a.T + 15) / 16 * 16, bl::kI8MaxTokens);
    a.t_tiles = (a.T + a.bt - 1) / a.bt;
    int64_t best = -1;
    for (int sp = 1; sp <= 8; sp *= 2) {
        if (sp > 1 && k_blocks < 4 * sp) break;
        int slots = 0;
        BL_TRY((i8_slots<kBf16Out, 1>(sp, dev_id, dev, &slots)));
        for (int64_t w = 1;; ++w) {
            const int64_t n_tiles = std::max<int64_t>(1, slots * w / a.t_tiles);
            int64_t rows = (a.N + n_tiles - 1) / n_tiles;
            if (sp > 1) rows = (rows + 3) / 4 * 4;
            if (rows > 128) continue;
            const int64_t kbs = (k_blocks + sp - 1) / sp;
            const int64_t cost = w * (kbs * (rows + a.bt + kStep) + (sp > 1 ? kJoin + 4 * a.bt : 0));
            if (best < 0 || cost < best) {
                best = cost;
                a.rows = (int)rows;
                a.splits = sp;
            }
            break;
        }
    }
    *cost_out = best;
    return BL_OK;
}

// Whether the large tiles (256 tokens x 256 weight rows on a pair of SMs) take T tokens: never up to
// 192, always when they fill half the pairs (256 tokens: 11008 x 4096 18.8 us against 21.3), else when
// the estimates (us) say so (256 tokens: 4096 x 4096 21.6 against 15.3).
bool i8_large(int64_t T, int64_t N, const DeviceInfo& dev) {
    return T > 192 && ((T + 255) / 256) * ((N + 255) / 256) * 4 >= dev.sms;
}
bool i8_few(const bl::I8Args& a, int64_t cost) {
    if (a.T <= 192) return true;
    const double few = 4.0 + 0.0022 * (double)cost;
    const double large = 8.0 + 0.3 * ((a.K + 127) / 128) + 0.5 * (double)a.N * a.K / 6.5e6;
    return few < large;
}

template <bool kBf16Out>
bl_status run_linear_int8(const int8_t* Xq, const float* sx, int64_t T, int64_t K, const int8_t* Wq,
                          const float* gamma_rows, int64_t N, void* Y, int32_t* acc, cudaStream_t st,
                          const DeviceInfo& dev) {
    int dev_id = 0;
    cudaGetDevice(&dev_id);
    if (dev_id < 0 || dev_id >= 64) return fail(BL_ERR_DEVICE, "device ordinal %d out of range", dev_id);
    bl::I8Args a{};
    a.T = (int)T; a.N = (int)N; a.K = (int)K;
    int64_t cost = 0;
    const bool large = i8_large(T, N, dev);
    if (!large) BL_TRY(i8_plan<kBf16Out>(a, &cost, dev_id, dev));
    if (large || !i8_few(a, cost))
        return run_linear_rows<true>(Xq, sx, T, K, Wq, gamma_rows, N, Y, kBf16Out ? BL_BF16 : BL_F32, acc, st, dev);
    const int k_blocks = (int)((K + 127) / 128);
    a.n_tiles = (int)((N + a.rows - 1) / a.rows);
    a.a_pitch = (a.rows + 7) / 8 * 1024;
    const size_t limit = (size_t)dev.max_smem_optin;
    const int kpb = bl::i8_smem_bytes(4, 2, a.a_pitch, a.bt) <= limit ? 2 : 1;
    a.k_steps = (k_blocks + kpb - 1) / kpb;
    a.stages = std::min(bl::kI8MaxStages, std::max(2, a.k_steps));
    while (a.stages > 2 && bl::i8_smem_bytes(a.stages, kpb, a.a_pitch, a.bt) > limit) --a.stages;
    const int64_t per_cta = a.splits > 1 ? 1 : ((int64_t)a.n_tiles * a.t_tiles + dev.sms - 1) / dev.sms;
    a.bufs = per_cta > 1 ? 2 : 1;
    a.sx = sx; a.gamma = gamma_rows; a.y = Y; a.acc = acc;
    a.wait_ns = g_wait_ns.load();
    CUtensorMap tw, tx;
    BL_TRY(make_tmap(&tw, Wq, kTmU8, (uint64_t)K, (uint64_t)N, 128, (uint32_t)a.rows));
    BL_TRY(make_tmap(&tx, Xq, kTmU8, (uint64_t)K, (uint64_t)T, 128, (uint32_t)a.bt));
    const int64_t tiles = (int64_t)a.n_tiles * a.t_tiles;
    if (kpb == 2) return launch_int8_few<kBf16Out, 2>(tw, tx, a, tiles, st, dev_id, dev);
    return launch_int8_few<kBf16Out, 1>(tw, tx, a, tiles, st, dev_id, dev);
}

// |Xq|, |Wq| <= 128: a sum of K products stays below 2^31 for K < 2^17.
constexpr int64_t kMaxInt8K = int64_t(1) << 17;

}  // namespace

// ====================================================================================
// exported C ABI
// ====================================================================================
extern "C" {

int bl_abi_version(void) { return BITLINEAR_ABI_VERSION; }

const char* bl_last_error(void) { return g_last_error.c_str(); }

size_t bitlinear_workspace_bytes(int64_t T, int64_t N, int64_t K) {
    (void)T;
    (void)N;
    if (K < 0) K = 0;
    size_t a = quant_ws_bytes();
    size_t b = dg_ws_bytes(K);
    size_t m = a > b ? a : b;
    if (opt_ws_bytes() > m) m = opt_ws_bytes();
    return (m + 255) & ~size_t(255);
}

void bl_set_wait_limit_ns(uint64_t ns) { g_wait_ns.store(ns == 0 ? 2000000000ull : ns); }

uint64_t bl_launch_count(void) { return g_launches.load(); }

bl_status bl_check_device_status(void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return fail(BL_ERR_CUDA, "cudaStreamSynchronize: %s", cudaGetErrorString(e));
    int v = 0, zero = 0;
    e = cudaMemcpyFromSymbol(&v, bl::g_bl_status, sizeof(int));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(bl::g_bl_status, &zero, sizeof(int));
    if (e != cudaSuccess) return fail(BL_ERR_CUDA, "status word: %s", cudaGetErrorString(e));
    if (v != 0) return fail((bl_status)v, "a kernel reported status %d (bounded wait expired)", v);
    return BL_OK;
}

bl_status bitlinear_quant_weight(const float* W, int64_t N, int64_t K, int8_t* Wq_i8, uint16_t* Wq_bf16,
                                 uint8_t* Wpacked, float* gamma, void* ws, size_t ws_bytes, void* stream) {
    BL_TRY(check_ptr(W, "W", true));
    BL_TRY(check_ptr(gamma, "gamma", true));
    BL_TRY(check_ptr(Wq_i8, "Wq_i8", false));
    BL_TRY(check_ptr(Wq_bf16, "Wq_bf16", false));
    BL_TRY(check_ptr(Wpacked, "Wpacked", false));
    BL_TRY(check_ptr(ws, "ws", true));
    BL_TRY(check_dims(1, N, K));
    BL_REQUIRE(ws_bytes >= quant_ws_bytes(), BL_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu",
               quant_ws_bytes(), ws_bytes);
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return run_quant_weight(W, N * K, ws, Wq_i8, Wq_bf16, Wpacked, gamma, st, dev);
}

bl_status bitlinear_act_quant(const void* X, bl_dtype x_dt, int64_t T, int64_t K, int apply_rmsnorm, const float* g,
                              float eps, int8_t* Xq, float* sx, float* rinv, void* Xdq, void* stream) {
    BL_TRY(check_dtype(x_dt));
    BL_TRY(check_ptr(X, "X", true));
    BL_TRY(check_ptr(Xq, "Xq", true));
    BL_TRY(check_ptr(sx, "sx", true));
    BL_TRY(check_ptr(rinv, "rinv", apply_rmsnorm != 0));
    BL_TRY(check_ptr(g, "g", false));
    BL_TRY(check_ptr(Xdq, "Xdq", false));
    BL_TRY(check_dims(T, 16, K));
    BL_REQUIRE(K <= kMaxRowK, BL_ERR_UNSUPPORTED_SHAPE, "d_in must be <= %lld for the row kernels, got %lld",
               (long long)kMaxRowK, (long long)K);
    BL_REQUIRE(!(eps < 0.0f) && eps == eps, BL_ERR_INVALID_ARG, "eps must be >= 0");
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    return run_act_quant(X, x_dt, T, K, apply_rmsnorm, g, eps, Xq, sx, rinv, Xdq, static_cast<cudaStream_t>(stream));
}

bl_status bitlinear_linear(const int8_t* Xq, const float* sx, int64_t T, int64_t K, const int8_t* Wq_i8,
                           const float* gamma, int64_t N, void* Y, bl_dtype y_dt, int32_t* acc, void* stream) {
    BL_TRY(check_dtype(y_dt));
    BL_TRY(check_ptr(Xq, "Xq", true));
    BL_TRY(check_ptr(sx, "sx", true));
    BL_TRY(check_ptr(Wq_i8, "Wq_i8", true));
    BL_TRY(check_ptr(gamma, "gamma", true));
    BL_TRY(check_ptr(Y, "Y", true));
    BL_TRY(check_ptr(acc, "acc", false));
    BL_TRY(check_dims(T, N, K));
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    return run_linear(Xq, sx, T, K, Wq_i8, gamma, N, Y, y_dt, acc, static_cast<cudaStream_t>(stream), dev);
}

bl_status bitlinear_forward(const void* X, bl_dtype x_dt, int64_t T, int64_t K, const float* g, float eps,
                            const int8_t* Wq_i8, const float* gamma, int64_t N, void* Y, int8_t* Xq, float* sx,
                            float* rinv, void* Xdq, int32_t* acc, void* stream) {
    BL_TRY(check_dtype(x_dt));
    BL_TRY(check_ptr(X, "X", true));
    BL_TRY(check_ptr(g, "g", false));
    BL_TRY(check_ptr(Wq_i8, "Wq_i8", true));
    BL_TRY(check_ptr(gamma, "gamma", true));
    BL_TRY(check_ptr(Y, "Y", true));
    BL_TRY(check_ptr(Xq, "Xq", true));
    BL_TRY(check_ptr(sx, "sx", true));
    BL_TRY(check_ptr(rinv, "rinv", true));
    BL_TRY(check_ptr(Xdq, "Xdq", false));
    BL_TRY(check_ptr(acc, "acc", false));
    BL_TRY(check_dims(T, N, K));
    BL_REQUIRE(K <= kMaxRowK, BL_ERR_UNSUPPORTED_SHAPE, "d_in must be <= %lld for the row kernels, got %lld",
               (long long)kMaxRowK, (long long)K);
    BL_REQUIRE(!(eps < 0.0f) && eps == eps, BL_ERR_INVALID_ARG, "eps must be >= 0");
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    BL_TRY(run_act_quant(X, x_dt, T, K, 1, g, eps, Xq, sx, rinv, Xdq, st));
    return run_linear(Xq, sx, T, K, Wq_i8, gamma, N, Y, x_dt, acc, st, dev);
}

bl_status bitlinear_forward_qat(const void* X, bl_dtype x_dt, int64_t T, int64_t K, const float* g, float eps,
                                const float* W, int64_t N, int8_t* Wq_i8, uint16_t* Wq_bf16, uint8_t* Wpacked,
                                float* gamma, void* Y, int8_t* Xq, float* sx, float* rinv, void* Xdq, int32_t* acc,
                                void* ws, size_t ws_bytes, void* stream) {
    BL_TRY(check_dtype(x_dt));
    BL_TRY(check_ptr(X, "X", true));
    BL_TRY(check_ptr(g, "g", false));
    BL_TRY(check_ptr(W, "W", true));
    BL_TRY(check_ptr(Wq_i8, "Wq_i8", true));
    BL_TRY(check_ptr(Wq_bf16, "Wq_bf16", false));
    BL_TRY(check_ptr(Wpacked, "Wpacked", false));
    BL_TRY(check_ptr(gamma, "gamma", true));
    BL_TRY(check_ptr(Y, "Y", true));
    BL_TRY(check_ptr(Xq, "Xq", true));
    BL_TRY(check_ptr(sx, "sx", true));
    BL_TRY(check_ptr(rinv, "rinv", true));
    BL_TRY(check_ptr(Xdq, "Xdq", false));
    BL_TRY(check_ptr(acc, "acc", false));
    BL_TRY(check_ptr(ws, "ws", true));
    BL_TRY(check_dims(T, N, K));
    BL_REQUIRE(K <= kMaxRowK, BL_ERR_UNSUPPORTED_SHAPE, "d_in must be <= %lld for the row kernels, got %lld",
               (long long)kMaxRowK, (long long)K);
    BL_REQUIRE(!(eps < 0.0f) && eps == eps, BL_ERR_INVALID_ARG, "eps must be >= 0");
    BL_REQUIRE(ws_bytes >= quant_ws_bytes(), BL_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu",
               quant_ws_bytes(), ws_bytes);
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // the |W| partial sums, the ternary codes (their second read of W follows the first
    // directly, so it hits L2 when W fits there), the activation quantiser, then the GEMM
    const int64_t n = N * K;
    const int parts = bl::wq_num_partials(n);
    double* partials = static_cast<double*>(ws);
    pdl_launch(bl::absmean_partial_kernel, dim3(parts), dim3(bl::kWqThreads), 0, st, W, n, partials);
    BL_TRY(launched("absmean_partial"));
    BL_TRY(run_ternary(W, n, partials, parts, Wq_i8, Wq_bf16, Wpacked, gamma, st, dev));
    BL_TRY(run_act_quant(X, x_dt, T, K, 1, g, eps, Xq, sx, rinv, Xdq, st));
    return run_linear(Xq, sx, T, K, Wq_i8, gamma, N, Y, x_dt, acc, st, dev);
}

bl_status bitlinear_backward_input(const void* dY, const void* X, bl_dtype dt, int64_t T, int64_t K, int64_t N,
                                   const float* g, const float* rinv, const uint16_t* Wq_bf16, const float* gamma,
                                   float* dX, float* dg, void* ws, size_t ws_bytes, void* stream) {
    BL_TRY(check_dtype(dt));
    BL_TRY(check_ptr(dY, "dY", true));
    BL_TRY(check_ptr(X, "X", true));
    BL_TRY(check_ptr(g, "g", false));
    BL_TRY(check_ptr(rinv, "rinv", true));
    BL_TRY(check_ptr(Wq_bf16, "Wq_bf16", true));
    BL_TRY(check_ptr(gamma, "gamma", true));
    BL_TRY(check_ptr(dX, "dX", true));
    BL_TRY(check_ptr(dg, "dg", false));
    BL_TRY(check_ptr(ws, "ws", dg != nullptr));
    BL_TRY(check_dims(T, N, K));
    BL_REQUIRE(K <= kMaxRowK, BL_ERR_UNSUPPORTED_SHAPE, "d_in must be <= %lld for the row kernels, got %lld",
               (long long)kMaxRowK, (long long)K);
    if (dg != nullptr)
        BL_REQUIRE(ws_bytes >= dg_ws_bytes(K), BL_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", dg_ws_bytes(K),
                   ws_bytes);
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    BL_TRY(run_grad_input_gemm(dY, dt, Wq_bf16, gamma, T, K, N, dX, st, dev));
    return run_rmsnorm_bwd(X, dt, rinv, g, dX, T, K, dg, ws, dev.sms, st);
}

bl_status bitlinear_grad_input(const void* dY, bl_dtype dt, int64_t T, int64_t K, int64_t N, const uint16_t* Wq_bf16,
                               const float* gamma, float* dXhat, void* stream) {
    BL_TRY(check_dtype(dt));
    BL_TRY(check_ptr(dY, "dY", true));
    BL_TRY(check_ptr(Wq_bf16, "Wq_bf16", true));
    BL_TRY(check_ptr(gamma, "gamma", true));
    BL_TRY(check_ptr(dXhat, "dXhat", true));
    BL_TRY(check_dims(T, N, K));
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    return run_grad_input_gemm(dY, dt, Wq_bf16, gamma, T, K, N, dXhat, static_cast<cudaStream_t>(stream), dev);
}

bl_status bitlinear_rmsnorm_backward(const void* X, bl_dtype dt, int64_t T, int64_t K, const float* g,
                                     const float* rinv, float* dX_inout, float* dg, void* ws, size_t ws_bytes,
                                     void* stream) {
    BL_TRY(check_dtype(dt));
    BL_TRY(check_ptr(X, "X", true));
    BL_TRY(check_ptr(g, "g", false));
    BL_TRY(check_ptr(rinv, "rinv", true));
    BL_TRY(check_ptr(dX_inout, "dX", true));
    BL_TRY(check_ptr(dg, "dg", false));
    BL_TRY(check_ptr(ws, "ws", dg != nullptr));
    BL_TRY(check_dims(T, 16, K));
    BL_REQUIRE(K <= kMaxRowK, BL_ERR_UNSUPPORTED_SHAPE, "d_in must be <= %lld for the row kernels, got %lld",
               (long long)kMaxRowK, (long long)K);
    if (dg != nullptr)
        BL_REQUIRE(ws_bytes >= dg_ws_bytes(K), BL_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", dg_ws_bytes(K),
                   ws_bytes);
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    return run_rmsnorm_bwd(X, dt, rinv, g, dX_inout, T, K, dg, ws, dev.sms, static_cast<cudaStream_t>(stream));
}

bl_status bitlinear_backward_weight(const void* dY, const void* Xdq, bl_dtype dt, int64_t T, int64_t K, int64_t N,
                                    float* dW, void* stream) {
    BL_TRY(check_dtype(dt));
    BL_TRY(check_ptr(dY, "dY", true));
    BL_TRY(check_ptr(Xdq, "Xdq", true));
    BL_TRY(check_ptr(dW, "dW", true));
    BL_TRY(check_dims(T, N, K));
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    return run_grad_weight_gemm(dY, Xdq, dt, T, K, N, dW, static_cast<cudaStream_t>(stream), dev);
}

bl_status bitlinear_backward(const void* dY, const void* X, const void* Xdq, bl_dtype dt, int64_t T, int64_t K,
                             int64_t N, const float* g, const float* rinv, const uint16_t* Wq_bf16, const float* gamma,
                             float* dX, float* dW, float* dg, void* ws, size_t ws_bytes, void* stream) {
    BL_TRY(check_ptr(Xdq, "Xdq", true));
    BL_TRY(check_ptr(dW, "dW", true));
    BL_TRY(bitlinear_backward_input(dY, X, dt, T, K, N, g, rinv, Wq_bf16, gamma, dX, dg, ws, ws_bytes, stream));
    return bitlinear_backward_weight(dY, Xdq, dt, T, K, N, dW, stream);
}

bl_status ternary_pack(const int8_t* Wq_i8, int64_t N, int64_t K, uint8_t* Wpacked, void* stream) {
    BL_TRY(check_ptr(Wq_i8, "Wq_i8", true));
    BL_TRY(check_ptr(Wpacked, "Wpacked", true));
    BL_TRY(check_dims(1, N, K));
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    const int64_t groups = N * K / 16;
    int64_t blocks = (groups + 255) / 256;
    if (blocks > (int64_t)dev.sms * 8) blocks = (int64_t)dev.sms * 8;
    pdl_launch(bl::ternary_pack_kernel, dim3((unsigned)blocks), dim3(256), 0, static_cast<cudaStream_t>(stream), Wq_i8,
               N * K, Wpacked);
    return launched("ternary_pack");
}

bl_status gemv_entry(const uint8_t* Wpacked, const float* gamma, int gamma_stride, int64_t N, int64_t K,
                     const int8_t* xq, const float* sx, int64_t B, float* y, int32_t* acc, void* stream);

bl_status ternary_gemv(const uint8_t* Wpacked, const float* gamma, int64_t N, int64_t K, const int8_t* xq,
                       const float* sx, int64_t B, float* y, int32_t* acc, void* stream) {
    return gemv_entry(Wpacked, gamma, 0, N, K, xq, sx, B, y, acc, stream);
}

bl_status ternary_gemv_rows(const uint8_t* Wpacked, const float* gamma_rows, int64_t N, int64_t K, const int8_t* xq,
                            const float* sx, int64_t B, float* y, int32_t* acc, void* stream) {
    return gemv_entry(Wpacked, gamma_rows, 1, N, K, xq, sx, B, y, acc, stream);
}

bl_status gemv_entry(const uint8_t* Wpacked, const float* gamma, int gamma_stride, int64_t N, int64_t K,
                     const int8_t* xq, const float* sx, int64_t B, float* y, int32_t* acc, void* stream) {
    BL_TRY(check_ptr(Wpacked, "Wpacked", true));
    BL_TRY(check_ptr(gamma, "gamma", true));
    BL_TRY(check_ptr(xq, "xq", true));
    BL_TRY(check_ptr(sx, "sx", true));
    BL_TRY(check_ptr(y, "y", true));
    BL_TRY(check_ptr(acc, "acc", false));
    BL_TRY(check_dims(1, N, K));
    BL_REQUIRE(K % 64 == 0, BL_ERR_UNSUPPORTED_SHAPE,
               "the GEMV reads packed rows in 16-byte pieces: K must be a multiple of 64, got %lld", (long long)K);
    BL_REQUIRE(B >= 1 && B <= 16, BL_ERR_UNSUPPORTED_SHAPE, "batch must be in [1, 16], got %lld", (long long)B);
    BL_REQUIRE(K <= 65536, BL_ERR_UNSUPPORTED_SHAPE, "K must be <= 65536 for the GEMV, got %lld", (long long)K);
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (B <= 8) return launch_gemv<1>(Wpacked, gamma, gamma_stride, N, K, xq, sx, B, y, acc, st, dev);
    return launch_gemv<2>(Wpacked, gamma, gamma_stride, N, K, xq, sx, B, y, acc, st, dev);
}

namespace {
// cuCtxGetCurrent through the runtime's driver entry point (the library does not link libcuda)
typedef CUresult (*CtxGetCurrentFn)(CUcontext*);

CtxGetCurrentFn ctx_get_current_fn() {
    static CtxGetCurrentFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<CtxGetCurrentFn>(p);
    });
    return fn;
}

constexpr int kScratchDevices = 64;
struct ScratchAddr {
    CUcontext ctx;
    void* addr;
};
}  // namespace

bl_status bitlinear_quant_weight_noalloc(const float* W, int64_t N, int64_t K, int8_t* Wq_i8, uint16_t* Wq_bf16,
                                         uint8_t* Wpacked, float* gamma, void* stream) {
    BL_TRY(check_ptr(W, "W", true));
    BL_TRY(check_ptr(gamma, "gamma", true));
    BL_TRY(check_ptr(Wq_i8, "Wq_i8", false));
    BL_TRY(check_ptr(Wq_bf16, "Wq_bf16", false));
    BL_TRY(check_ptr(Wpacked, "Wpacked", false));
    BL_TRY(check_dims(1, N, K));
    const int64_t n = N * K;
    const int parts = bl::wq_num_partials(n);
    BL_REQUIRE(parts <= bl::kWqMaxPartials, BL_ERR_UNSUPPORTED_SHAPE,
               "the built-in scratch holds %d partial sums, this weight needs %d", bl::kWqMaxPartials, parts);
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    // set-up, once per device and context: the device address of the scratch array.  The
    // address belongs to the context that loaded this module, so it is cached together with
    // that context and looked up again when the current context differs (after a
    // cudaDeviceReset the device gets a new primary context and the old address is gone).
    int dev_id = -1;
    cudaError_t e = cudaGetDevice(&dev_id);
    if (e != cudaSuccess) return fail(BL_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    BL_REQUIRE(dev_id >= 0 && dev_id < kScratchDevices, BL_ERR_INVALID_ARG,
               "device index %d is beyond the %d devices the scratch table covers", dev_id, kScratchDevices);
    CtxGetCurrentFn ctx_fn = ctx_get_current_fn();
    BL_REQUIRE(ctx_fn != nullptr, BL_ERR_CUDA, "cuCtxGetCurrent is unavailable");
    CUcontext ctx = nullptr;
    CUresult cr = ctx_fn(&ctx);
    BL_REQUIRE(cr == CUDA_SUCCESS && ctx != nullptr, BL_ERR_CUDA, "cuCtxGetCurrent failed (%d)", (int)cr);
    void* scratch = nullptr;
    {
        static std::mutex mu;
        static ScratchAddr cache[kScratchDevices] = {};
        std::lock_guard<std::mutex> lk(mu);
        if (cache[dev_id].addr == nullptr || cache[dev_id].ctx != ctx) {
            void* p = nullptr;
            e = cudaGetSymbolAddress(&p, g_quant_scratch);
            if (e != cudaSuccess) return fail(BL_ERR_CUDA, "cudaGetSymbolAddress(scratch): %s", cudaGetErrorString(e));
            cache[dev_id].addr = p;
            cache[dev_id].ctx = ctx;
        }
        scratch = cache[dev_id].addr;
    }
    // pass 1 writes every partial that pass 2 reads, so nothing in the scratch needs clearing
    return run_quant_weight(W, n, scratch, Wq_i8, Wq_bf16, Wpacked, gamma, static_cast<cudaStream_t>(stream), dev);
}

// ------------------------------------------------------------------------------------
// quantiser variants
// ------------------------------------------------------------------------------------
bl_status bitlinear_quant_weight_rows(const float* W, int64_t N, int64_t K, int8_t* Wq_i8, uint16_t* Wq_bf16,
                                      uint8_t* Wpacked, float* gamma_rows, void* stream) {
    BL_TRY(check_ptr(W, "W", true));
    BL_TRY(check_ptr(gamma_rows, "gamma_rows", true));
    BL_TRY(check_ptr(Wq_i8, "Wq_i8", false));
    BL_TRY(check_ptr(Wq_bf16, "Wq_bf16", false));
    BL_TRY(check_ptr(Wpacked, "Wpacked", false));
    BL_TRY(check_dims(1, N, K));
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    pdl_launch(bl::ternary_quant_rows_kernel, dim3((unsigned)((N + 7) / 8)), dim3(256), 0,
               static_cast<cudaStream_t>(stream), W, (int)N, (int)K, Wq_i8, Wq_bf16, Wpacked, gamma_rows);
    return launched("ternary_quant_rows");
}

bl_status bitlinear_quant_weight_tau(const float* W, int64_t N, int64_t K, float tau_factor, int8_t* Wq_i8,
                                     uint16_t* Wq_bf16, uint8_t* Wpacked, float* gamma, void* ws, size_t ws_bytes,
                                     void* stream) {
    BL_TRY(check_ptr(W, "W", true));
    BL_TRY(check_ptr(gamma, "gamma", true));
    BL_TRY(check_ptr(Wq_i8, "Wq_i8", false));
    BL_TRY(check_ptr(Wq_bf16, "Wq_bf16", false));
    BL_TRY(check_ptr(Wpacked, "Wpacked", false));
    BL_TRY(check_ptr(ws, "ws", true));
    BL_TRY(check_dims(1, N, K));
    BL_REQUIRE(tau_factor >= 0.0f && tau_factor <= 1e30f, BL_ERR_INVALID_ARG,
               "tau_factor must be finite and >= 0, got %g", (double)tau_factor);
    BL_REQUIRE(ws_bytes >= quant_ws_bytes(), BL_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu",
               quant_ws_bytes(), ws_bytes);
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    return run_quant_weight(W, N * K, ws, Wq_i8, Wq_bf16, Wpacked, gamma, static_cast<cudaStream_t>(stream), dev,
                            tau_factor);
}

bl_status bitlinear_act_quant_tensor(const void* X, bl_dtype x_dt, int64_t T, int64_t K, int apply_rmsnorm,
                                     const float* g, float eps, int8_t* Xq, float* sx, float* rinv, void* Xdq,
                                     void* ws, size_t ws_bytes, void* stream) {
    BL_TRY(check_dtype(x_dt));
    BL_TRY(check_ptr(X, "X", true));
    BL_TRY(check_ptr(Xq, "Xq", true));
    BL_TRY(check_ptr(sx, "sx", true));
    BL_TRY(check_ptr(rinv, "rinv", apply_rmsnorm != 0));
    BL_TRY(check_ptr(g, "g", false));
    BL_TRY(check_ptr(Xdq, "Xdq", false));
    BL_TRY(check_ptr(ws, "ws", true));
    BL_TRY(check_dims(T, 16, K));
    BL_REQUIRE(K <= kMaxRowK, BL_ERR_UNSUPPORTED_SHAPE, "d_in must be <= %lld for the row kernels, got %lld",
               (long long)kMaxRowK, (long long)K);
    BL_REQUIRE(!(eps < 0.0f) && eps == eps, BL_ERR_INVALID_ARG, "eps must be >= 0");
    BL_REQUIRE(ws_bytes >= sizeof(float) * bl::kActMaxPartials, BL_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu",
               sizeof(float) * bl::kActMaxPartials, ws_bytes);
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t row_blocks = (T + 7) / 8;
    const int grid = (int)(row_blocks < bl::kActMaxPartials ? row_blocks : bl::kActMaxPartials);
    float* partials = static_cast<float*>(ws);
    if (x_dt == BL_BF16) {
        pdl_launch(bl::act_tensor_max_kernel<true>, dim3(grid), dim3(256), 0, st, X, (int)T, (int)K, apply_rmsnorm, g,
                   eps, rinv, partials);
        BL_TRY(launched("act_tensor_max"));
        pdl_launch(bl::act_tensor_quant_kernel<true>, dim3(grid), dim3(256), 0, st, X, (int)T, (int)K, apply_rmsnorm,
                   g, static_cast<const float*>(partials), grid, Xq, sx, static_cast<const float*>(rinv), Xdq);
    } else {
        pdl_launch(bl::act_tensor_max_kernel<false>, dim3(grid), dim3(256), 0, st, X, (int)T, (int)K, apply_rmsnorm,
                   g, eps, rinv, partials);
        BL_TRY(launched("act_tensor_max"));
        pdl_launch(bl::act_tensor_quant_kernel<false>, dim3(grid), dim3(256), 0, st, X, (int)T, (int)K, apply_rmsnorm,
                   g, static_cast<const float*>(partials), grid, Xq, sx, static_cast<const float*>(rinv), Xdq);
    }
    return launched("act_tensor_quant");
}

bl_status bitlinear_linear_rows(const int8_t* Xq, const float* sx, int64_t T, int64_t K, const int8_t* Wq_i8,
                                const float* gamma_rows, int64_t N, void* Y, bl_dtype y_dt, int32_t* acc,
                                void* stream) {
    BL_TRY(check_dtype(y_dt));
    BL_TRY(check_ptr(Xq, "Xq", true));
    BL_TRY(check_ptr(sx, "sx", true));
    BL_TRY(check_ptr(Wq_i8, "Wq_i8", true));
    BL_TRY(check_ptr(gamma_rows, "gamma_rows", true));
    BL_TRY(check_ptr(Y, "Y", true));
    BL_TRY(check_ptr(acc, "acc", false));
    BL_TRY(check_dims(T, N, K));
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    return run_linear_rows(Xq, sx, T, K, Wq_i8, gamma_rows, N, Y, y_dt, acc, static_cast<cudaStream_t>(stream), dev);
}

// ------------------------------------------------------------------------------------
// int8 x packed-ternary GEMM (few tokens)
// ------------------------------------------------------------------------------------
bl_status bitlinear_linear_packed(const int8_t* Xq, const float* sx, int64_t T, int64_t K, const uint8_t* Wpacked,
                                  const float* gamma, int64_t N, void* Y, bl_dtype y_dt, int32_t* acc, void* ws,
                                  size_t ws_bytes, void* stream) {
    BL_TRY(check_dtype(y_dt));
    BL_TRY(check_ptr(Xq, "Xq", true));
    BL_TRY(check_ptr(sx, "sx", true));
    BL_TRY(check_ptr(Wpacked, "Wpacked", true));
    BL_TRY(check_ptr(gamma, "gamma", true));
    BL_TRY(check_ptr(Y, "Y", true));
    BL_TRY(check_ptr(acc, "acc", false));
    BL_TRY(check_ptr(ws, "ws", false));
    BL_TRY(check_dims(T, N, K));
    BL_REQUIRE(K % 64 == 0, BL_ERR_UNSUPPORTED_SHAPE,
               "packed rows are read in 16-byte pieces: K must be a multiple of 64, got %lld", (long long)K);
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    int32_t* scratch = static_cast<int32_t*>(ws);
    const size_t scratch_bytes = ws != nullptr ? ws_bytes : 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // Up to 16 tokens whose activation rows fit a block's shared memory: the decode GEMV's
    // kernel (codes decoded in registers, warp-level int8 MMA), which streams the packed
    // weight faster than the tensor-core tile with 16-column MMAs.
    if (T <= 16 && K <= 65536) {
        const int64_t n_rg = N / 16;
        const int64_t nb = n_rg < dev.sms ? n_rg : dev.sms;
        const int max_rgs = (int)((n_rg + nb - 1) / nb);
        if (bl::gemv_smem_bytes((int)T, (int)K, max_rgs) <= (size_t)dev.max_smem_optin) {
            if (y_dt == BL_BF16)
                return T <= 8 ? launch_gemv<1, true>(Wpacked, gamma, 0, N, K, Xq, sx, T, Y, acc, st, dev)
                              : launch_gemv<2, true>(Wpacked, gamma, 0, N, K, Xq, sx, T, Y, acc, st, dev);
            return T <= 8 ? launch_gemv<1, false>(Wpacked, gamma, 0, N, K, Xq, sx, T, Y, acc, st, dev)
                          : launch_gemv<2, false>(Wpacked, gamma, 0, N, K, Xq, sx, T, Y, acc, st, dev);
        }
    }
    // Otherwise (17 tokens or more, or rows too long for the GEMV): 2-SM tiles of 256 weight
    // rows with the decoded codes in tensor memory
    if (y_dt == BL_BF16)
        return launch_packed2<true>(Xq, sx, T, K, Wpacked, gamma, N, Y, acc, scratch, scratch_bytes, st, dev);
    return launch_packed2<false>(Xq, sx, T, K, Wpacked, gamma, N, Y, acc, scratch, scratch_bytes, st, dev);
}

// ------------------------------------------------------------------------------------
// optimizer step
// ------------------------------------------------------------------------------------
bl_status bitlinear_optimizer_step(float* W, const float* dW, float* m, float* v, int64_t N, int64_t K, float lr,
                                   float beta1, float beta2, float eps, float weight_decay, float max_norm,
                                   int32_t* step, int8_t* Wq_i8, uint16_t* Wq_bf16, uint8_t* Wpacked, float* gamma,
                                   void* ws, size_t ws_bytes, void* stream) {
    BL_TRY(check_optimizer(W, dW, m, v, N, K, lr, beta1, beta2, eps, weight_decay, step, Wq_i8, Wq_bf16, Wpacked,
                           gamma, ws, ws_bytes));
    BL_REQUIRE(max_norm == max_norm && max_norm <= 1e30f, BL_ERR_INVALID_ARG, "max_norm must be finite");
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    return run_optimizer(W, dW, m, v, N * K, adamw_args(lr, beta1, beta2, eps, weight_decay, max_norm), nullptr, step,
                         Wq_i8, Wq_bf16, Wpacked, gamma, ws, static_cast<cudaStream_t>(stream), dev);
}

bl_status bitlinear_optimizer_step_coef(float* W, const float* dW, float* m, float* v, int64_t N, int64_t K,
                                        float lr, float beta1, float beta2, float eps, float weight_decay,
                                        const float* coef, int32_t* step, int8_t* Wq_i8, uint16_t* Wq_bf16,
                                        uint8_t* Wpacked, float* gamma, void* ws, size_t ws_bytes, void* stream) {
    BL_TRY(check_optimizer(W, dW, m, v, N, K, lr, beta1, beta2, eps, weight_decay, step, Wq_i8, Wq_bf16, Wpacked,
                           gamma, ws, ws_bytes));
    BL_REQUIRE(coef != nullptr, BL_ERR_INVALID_ARG, "coef must not be NULL");
    BL_REQUIRE((reinterpret_cast<uintptr_t>(coef) & 3u) == 0, BL_ERR_MISALIGNED, "coef must be 4-byte aligned");
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    return run_optimizer(W, dW, m, v, N * K, adamw_args(lr, beta1, beta2, eps, weight_decay, 0.0f), coef, step, Wq_i8,
                         Wq_bf16, Wpacked, gamma, ws, static_cast<cudaStream_t>(stream), dev);
}

// ------------------------------------------------------------------------------------
// global gradient norm and clipping
// ------------------------------------------------------------------------------------
bl_status bitlinear_grad_norm(const void* const* grads, const int64_t* numel, const bl_dtype* dtypes, int64_t count,
                              float max_norm, float* norm, float* coef, void* ws, size_t ws_bytes, void* stream) {
    BL_TRY(check_grads(grads, nullptr, numel, dtypes, count, max_norm, norm, coef, ws, ws_bytes));
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    return run_grads(grads, nullptr, numel, dtypes, count, max_norm, norm, coef, ws, static_cast<cudaStream_t>(stream),
                     dev);
}

bl_status bitlinear_clip_grads(const void* const* grads, void* const* out, const int64_t* numel,
                               const bl_dtype* dtypes, int64_t count, float max_norm, float* norm, float* coef,
                               void* ws, size_t ws_bytes, void* stream) {
    BL_REQUIRE(out != nullptr, BL_ERR_INVALID_ARG, "out must not be NULL");
    BL_TRY(check_grads(grads, out, numel, dtypes, count, max_norm, norm, coef, ws, ws_bytes));
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    return run_grads(grads, out, numel, dtypes, count, max_norm, norm, coef, ws, static_cast<cudaStream_t>(stream),
                     dev);
}

// ------------------------------------------------------------------------------------
// residual norms
// ------------------------------------------------------------------------------------
bl_status bitlinear_residual_norm(const void* X, bl_dtype x_dt, const void* Y, bl_dtype y_dt, int64_t T, int64_t K,
                                  int post_norm, const float* g_post, float eps_post, bl_gate gate_kind,
                                  const void* gate, float alpha, float beta, const float* g_pre, float eps_pre,
                                  void* Xout, float* r_post, float* r_pre, void* H, int8_t* Xq, float* sx, void* Xdq,
                                  void* stream) {
    BL_TRY(check_residual(x_dt, y_dt, T, K, post_norm, g_post, gate_kind, gate, alpha, beta));
    BL_TRY(check_ptr(X, "X", true));
    BL_TRY(check_ptr(Y, "Y", true));
    BL_TRY(check_ptr(Xout, "Xout", true));
    BL_TRY(check_ptr(r_post, "r_post", post_norm != 0));
    BL_TRY(check_ptr(g_pre, "g_pre", false));
    BL_TRY(check_ptr(H, "H", false));
    BL_TRY(check_ptr(Xq, "Xq", false));
    BL_TRY(check_ptr(sx, "sx", Xq != nullptr));
    BL_TRY(check_ptr(Xdq, "Xdq", false));
    BL_TRY(check_ptr(r_pre, "r_pre", H != nullptr || Xq != nullptr));
    BL_REQUIRE(H == nullptr || Xq == nullptr, BL_ERR_INVALID_ARG, "H and Xq exclude each other");
    BL_REQUIRE(Xq != nullptr || Xdq == nullptr, BL_ERR_INVALID_ARG, "Xdq needs Xq");
    BL_REQUIRE(H != nullptr || Xq != nullptr || g_pre == nullptr, BL_ERR_INVALID_ARG, "g_pre needs H or Xq");
    BL_REQUIRE(eps_post >= 0.0f && eps_post <= 1e30f && eps_pre >= 0.0f && eps_pre <= 1e30f, BL_ERR_INVALID_ARG,
               "eps must be finite and >= 0");
    BL_REQUIRE(Xq == nullptr || K % 32 == 0, BL_ERR_UNSUPPORTED_SHAPE,
               "the quantised output needs K to be a multiple of 32, got %lld", (long long)K);
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    bl::RnFwdArgs a{};
    a.x = X; a.y = Y; a.gate = gate; a.g_post = g_post; a.g_pre = g_pre;
    a.xout = Xout; a.r_post = r_post; a.r_pre = (H != nullptr || Xq != nullptr) ? r_pre : nullptr;
    a.h = H; a.xq = Xq; a.sx = sx; a.xdq = Xdq;
    a.T = (int)T; a.K = (int)K;
    a.post = post_norm != 0; a.gate_kind = (int)gate_kind;
    a.alpha = alpha; a.beta = beta; a.eps_post = eps_post; a.eps_pre = eps_pre;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (x_dt == BL_BF16) return launch_residual_norm<true, true>(a, st, dev);
    if (y_dt == BL_BF16) return launch_residual_norm<false, true>(a, st, dev);
    return launch_residual_norm<false, false>(a, st, dev);
}

bl_status bitlinear_residual_norm_backward(const float* dXout, const float* dH, const void* Xout, bl_dtype x_dt,
                                           const void* Y, bl_dtype y_dt, int64_t T, int64_t K, int post_norm,
                                           const float* g_post, const float* r_post, bl_gate gate_kind,
                                           const void* gate, float alpha, float beta, const float* g_pre,
                                           const float* r_pre, float* dX, void* dY, float* dg_post, float* dg_pre,
                                           void* dgate, void* ws, size_t ws_bytes, void* stream) {
    BL_TRY(check_residual(x_dt, y_dt, T, K, post_norm, g_post, gate_kind, gate, alpha, beta));
    BL_TRY(check_ptr(dXout, "dXout", false));
    BL_TRY(check_ptr(dH, "dH", false));
    BL_REQUIRE(dXout != nullptr || dH != nullptr, BL_ERR_INVALID_ARG, "dXout and dH must not both be NULL");
    BL_TRY(check_ptr(Xout, "Xout", dH != nullptr));
    BL_TRY(check_ptr(Y, "Y", true));
    BL_TRY(check_ptr(r_post, "r_post", post_norm != 0));
    BL_TRY(check_ptr(r_pre, "r_pre", dH != nullptr));
    BL_TRY(check_ptr(g_pre, "g_pre", false));
    BL_TRY(check_ptr(dX, "dX", true));
    BL_TRY(check_ptr(dY, "dY", true));
    BL_TRY(check_ptr(dg_post, "dg_post", false));
    BL_TRY(check_ptr(dg_pre, "dg_pre", false));
    BL_TRY(check_ptr(dgate, "dgate", false));
    BL_REQUIRE(dg_post == nullptr || post_norm, BL_ERR_INVALID_ARG, "dg_post needs post_norm");
    BL_REQUIRE(dg_pre == nullptr || dH != nullptr, BL_ERR_INVALID_ARG, "dg_pre needs dH");
    BL_REQUIRE(dgate == nullptr || gate_kind != BL_GATE_NONE, BL_ERR_INVALID_ARG, "dgate needs a gate");
    const bool sums = dg_post != nullptr || dg_pre != nullptr ||
                      (dgate != nullptr && (gate_kind == BL_GATE_SCALAR || gate_kind == BL_GATE_CHANNEL));
    BL_TRY(check_ptr(ws, "ws", sums));
    BL_REQUIRE(!sums || ws_bytes >= rn_ws_bytes(K), BL_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu",
               rn_ws_bytes(K), ws_bytes);
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    bl::RnBwdArgs a{};
    a.dx = dXout; a.dh = dH; a.x = Xout; a.y = Y; a.gate = gate;
    a.r_post = r_post; a.r_pre = r_pre; a.g_post = g_post; a.g_pre = g_pre;
    a.dX = dX; a.dY = dY;
    a.T = (int)T; a.K = (int)K;
    a.post = post_norm != 0; a.gate_kind = (int)gate_kind;
    a.alpha = alpha; a.beta = beta;
    // the scalar's partials first (fp64), then one [blocks x K] array for each column sum
    uint8_t* w = static_cast<uint8_t*>(ws);
    float* part = reinterpret_cast<float*>(w + sizeof(double) * bl::kRnMaxBlocks);
    const bool scalar = dgate != nullptr && gate_kind == BL_GATE_SCALAR;
    const bool channel = dgate != nullptr && gate_kind == BL_GATE_CHANNEL;
    if (dg_pre != nullptr) a.part_pre = part;
    if (dg_post != nullptr || channel) a.part_s = part + bl::kRnMaxBlocks * K;
    if (scalar) a.part_scalar = reinterpret_cast<double*>(w);
    if (!scalar && !channel) a.dgate = dgate;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int G = 0, Gs = 0;
    if (x_dt == BL_BF16) BL_TRY((launch_residual_norm_bwd<true, true>(a, st, dev, &G, &Gs)));
    else if (y_dt == BL_BF16) BL_TRY((launch_residual_norm_bwd<false, true>(a, st, dev, &G, &Gs)));
    else BL_TRY((launch_residual_norm_bwd<false, false>(a, st, dev, &G, &Gs)));
    if (!sums) return BL_OK;
    bl::RnReduceArgs r{};
    r.part_pre = a.part_pre; r.part_s = a.part_s; r.part_scalar = a.part_scalar;
    r.gate = gate_kind == BL_GATE_SCALAR || gate_kind == BL_GATE_CHANNEL ? static_cast<const float*>(gate) : nullptr;
    r.g_post = g_post;
    r.dg_pre = dg_pre; r.dg_post = dg_post; r.dgate = scalar || channel ? static_cast<float*>(dgate) : nullptr;
    r.beta = beta; r.gate_kind = (int)gate_kind;
    r.G = G; r.Gs = Gs; r.K = (int)K;
    pdl_launch(bl::rn_reduce_kernel, dim3((unsigned)((K + 31) / 32), 2), dim3(1024), 0, st, r);
    return launched("residual_norm_reduce");
}

// ------------------------------------------------------------------------------------
// 8-bit linear
// ------------------------------------------------------------------------------------
bl_status bitlinear_quant_weight_int8(const float* W, int64_t N, int64_t K, int8_t* Wq_i8, uint16_t* Wq_bf16,
                                      float* gamma_rows, void* stream) {
    BL_TRY(check_ptr(W, "W", true));
    BL_TRY(check_ptr(gamma_rows, "gamma_rows", true));
    BL_TRY(check_ptr(Wq_i8, "Wq_i8", false));
    BL_TRY(check_ptr(Wq_bf16, "Wq_bf16", false));
    BL_TRY(check_dims(1, N, K));
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    pdl_launch(bl::weight_quant8_kernel, dim3((unsigned)N), dim3(bl::kW8Threads), 0,
               static_cast<cudaStream_t>(stream), W, (int)N, (int)K, Wq_i8, Wq_bf16, gamma_rows);
    return launched("weight_quant8");
}

bl_status bitlinear_linear_int8(const int8_t* Xq, const float* sx, int64_t T, int64_t K, const int8_t* Wq_i8,
                                const float* gamma_rows, int64_t N, void* Y, bl_dtype y_dt, int32_t* acc,
                                void* stream) {
    BL_TRY(check_dtype(y_dt));
    BL_TRY(check_ptr(Xq, "Xq", true));
    BL_TRY(check_ptr(sx, "sx", true));
    BL_TRY(check_ptr(Wq_i8, "Wq_i8", true));
    BL_TRY(check_ptr(gamma_rows, "gamma_rows", true));
    BL_TRY(check_ptr(Y, "Y", true));
    BL_TRY(check_ptr(acc, "acc", false));
    BL_TRY(check_dims(T, N, K));
    BL_REQUIRE(K < kMaxInt8K, BL_ERR_UNSUPPORTED_SHAPE,
               "K must be below %lld: 128 * 128 * K has to fit the int32 accumulator, got %lld", (long long)kMaxInt8K,
               (long long)K);
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (y_dt == BL_BF16) return run_linear_int8<true>(Xq, sx, T, K, Wq_i8, gamma_rows, N, Y, acc, st, dev);
    return run_linear_int8<false>(Xq, sx, T, K, Wq_i8, gamma_rows, N, Y, acc, st, dev);
}

bl_status bl_mma_peak_probe(int kind, int pair, int iters, double* ops_out, void* stream) {
    BL_REQUIRE(kind >= 0 && kind <= 2, BL_ERR_INVALID_ARG, "kind must be 0 (int8), 1 (bf16) or 2 (mma.sync int8), got %d",
               kind);
    BL_REQUIRE(pair == 0 || pair == 1, BL_ERR_INVALID_ARG, "pair must be 0 or 1, got %d", pair);
    BL_REQUIRE(iters >= 1 && iters <= (1 << 20), BL_ERR_INVALID_ARG, "iters must be in [1, 2^20], got %d", iters);
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    if (kind == 2) {
        // per instruction 16 x 8 x 32 multiply-adds; every warp of every SM runs kImmaChains per iteration
        if (ops_out)
            *ops_out = 2.0 * 16 * 8 * 32 * (double)bl::kImmaChains * bl::kImmaWarps * dev.sms * (double)iters;
        pdl_launch(bl::imma_sync_peak_kernel, dim3((unsigned)dev.sms), dim3(bl::kImmaWarps * 32), 0,
                   static_cast<cudaStream_t>(stream), iters);
        return launched("imma_sync_peak");
    }
    BL_REQUIRE(bl::kPeakSmemBytes <= dev.max_smem_optin, BL_ERR_DEVICE, "probe needs %d bytes of shared memory",
               bl::kPeakSmemBytes);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const uint64_t wait_ns = g_wait_ns.load();
    int ctas = pair ? 2 * (dev.sms / 2) : dev.sms;
    void (*kern)(int, uint64_t) = nullptr;
    if (pair) kern = kind == 0 ? bl::mma_peak2_kernel<true> : bl::mma_peak2_kernel<false>;
    else kern = kind == 0 ? bl::mma_peak_kernel<true> : bl::mma_peak_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bl::kPeakSmemBytes);
    if (e != cudaSuccess) return fail(BL_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    if (pair) {
        // no more clusters than can be resident at once: every pair runs in the same wave
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)ctas);
        cfg.blockDim = dim3(bl::kPeakThreads);
        cfg.dynamicSmemBytes = bl::kPeakSmemBytes;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
        if (e != cudaSuccess) return fail(BL_ERR_CUDA, "cudaOccupancyMaxActiveClusters: %s", cudaGetErrorString(e));
        if (n < 1) return fail(BL_ERR_DEVICE, "no 2-CTA cluster of the probe fits on the device");
        ctas = std::min(ctas, 2 * n);
    }
    // multiply-adds x 2 of the launch: per instruction M x N x (32 bytes of K)
    const double k_per_instr = kind == 0 ? 32.0 : 16.0;
    const double per_instr = 2.0 * (pair ? 256.0 * 256.0 : 128.0 * 256.0) * k_per_instr;
    const double units = pair ? ctas / 2 : ctas;
    if (ops_out) *ops_out = units * 4.0 * (double)iters * per_instr;
    pdl_launch(kern, dim3((unsigned)ctas), dim3(bl::kPeakThreads), (size_t)bl::kPeakSmemBytes, st, iters, wait_ns);
    return launched("mma_peak");
}

bl_status bl_read_peak_probe(const uint8_t* buf, int64_t rows, int64_t row_bytes, int pattern, uint32_t* sink,
                             void* stream) {
    BL_TRY(check_ptr(buf, "buf", true));
    BL_TRY(check_ptr(sink, "sink", true));
    BL_REQUIRE(pattern == 0 || pattern == 1, BL_ERR_INVALID_ARG, "pattern must be 0 (GEMV) or 1 (coalesced), got %d",
               pattern);
    BL_REQUIRE(rows >= 16 && rows % 16 == 0 && rows <= (1 << 30), BL_ERR_UNSUPPORTED_SHAPE,
               "rows must be a positive multiple of 16 (at most 2^30), got %lld", (long long)rows);
    BL_REQUIRE(row_bytes >= 64 && row_bytes % 64 == 0 && row_bytes <= (1 << 24), BL_ERR_UNSUPPORTED_SHAPE,
               "row_bytes must be a positive multiple of 64 (at most 2^24), got %lld", (long long)row_bytes);
    // keeps a block's step count (32-bit in the kernel) in range
    BL_REQUIRE(rows * row_bytes <= (int64_t(1) << 40), BL_ERR_UNSUPPORTED_SHAPE, "buffer larger than 2^40 bytes");
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t n_rg = rows / 16;
    if (pattern == 0) {
        // as the GEMV: one block per SM, at most one per row group
        const unsigned nb = (unsigned)std::min<int64_t>(n_rg, dev.sms);
        pdl_launch(bl::read_peak_gemv_kernel, dim3(nb), dim3(bl::kReadWarps * 32), 0, st, buf, (int)rows,
                   (int)row_bytes, sink);
    } else {
        pdl_launch(bl::read_peak_coalesced_kernel, dim3((unsigned)dev.sms), dim3(bl::kReadWarps * 32), 0, st,
                   reinterpret_cast<const uint4*>(buf), rows * row_bytes / 16, sink);
    }
    return launched("read_peak");
}

bl_status bl_selftest_bounded_wait(uint64_t limit_ns, void* stream) {
    BL_REQUIRE(limit_ns > 0 && limit_ns <= 10000000000ull, BL_ERR_INVALID_ARG, "limit must be in (0, 10 s]");
    DeviceInfo dev;
    BL_TRY(current_device(&dev));
    pdl_launch(bl::selftest_wait_kernel, dim3(1), dim3(32), 0, static_cast<cudaStream_t>(stream), limit_ns);
    return launched("selftest_wait");
}

}  // extern "C"
