// grad_clip.cuh -- the global gradient norm over many tensors, and clipping to it.
//
// Restates the pages' model-wide clipping (P3 §6 and P4 §4.1 clip_grad_norm_ over all
// parameters, max_norm 1.0) beside the per-matrix rule of optim.cuh:
//   norm = sqrt( sum_i sum_j g_ij^2 ),   c = min(1, max_norm / (norm + 1e-6)),   g <- c g
// The squares and their sums are fp64 (a product of two fp32 values is exact in fp64 up to its
// 53 bits and cannot overflow there), added in a fixed order: the same tensors give the same
// bits on every call and on every rank that holds the same gradients.
//
// The tensors' addresses and sizes travel as the kernel's parameter, so a call needs no device
// table, no copy to the device and no allocation, and can be captured into a graph.  All
// tensors are cut into chunks of one size; a block finds the tensor of a chunk by bisection in
// the parameter's prefix sums.  HBM-bound: the norm reads 809 MB in 117 us (6.9 TB/s), the scaling
// pass reads and writes them in 268 us (6.0 TB/s); few small tensors cost two launches (4.3 us).
#pragma once
#include "common.cuh"

namespace bl {

constexpr int kGcThreads = 512;
constexpr int kGcMaxPartials = 1184;

struct GcTensor {
    const void* g;
    void* out;
    int64_t n;
    int32_t first_chunk;   // chunks of the tensors before it
    int32_t bf16;
};
// Kernel parameters hold up to 32,764 bytes; the small table keeps the launch of a layer's few
// gradients short.
constexpr int kGcSmall = 64;
constexpr int kGcLarge = 960;
template <int kMax>
struct GcTable {
    int32_t count, chunks;
    int64_t chunk;         // elements
    GcTensor t[kMax];
};

template <int kMax>
__device__ __forceinline__ int gc_find(const GcTable<kMax>& tab, int c) {
    int lo = 0, hi = tab.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.t[mid].first_chunk <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Applies f(value) to every element of a chunk [i0, i1) of a tensor: scalars up to the first
// 16-byte boundary, 16-byte vectors, scalars behind the last.
template <bool kBf16, typename F>
__device__ __forceinline__ void gc_read(const void* __restrict__ g, int64_t i0, int64_t i1, F&& f) {
    constexpr int E = kBf16 ? 8 : 4;
    constexpr int kSize = kBf16 ? 2 : 4;
    const uint8_t* p = static_cast<const uint8_t*>(g) + i0 * kSize;
    int64_t n = i1 - i0;
    auto one = [&](int64_t i) -> float {
        if constexpr (kBf16) return bf16_bits_to_float(__ldg(reinterpret_cast<const uint16_t*>(p) + i));
        else return __ldg(reinterpret_cast<const float*>(p) + i);
    };
    int64_t head = ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / kSize;
    if (head > n) head = n;
    if (threadIdx.x < head) f(one(threadIdx.x));
    const uint4* pv = reinterpret_cast<const uint4*>(p + head * kSize);
    const int64_t nv = (n - head) / E;
    auto vec = [&](const uint4& r) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kBf16) {
                f(__uint_as_float(w[i] << 16));
                f(__uint_as_float(w[i] & 0xFFFF0000u));
            } else {
                f(__uint_as_float(w[i]));
            }
        }
    };
    int64_t i = threadIdx.x;
    for (; i + 3 * kGcThreads < nv; i += 4 * kGcThreads) {
        uint4 r[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) r[u] = __ldg(pv + i + u * kGcThreads);
#pragma unroll
        for (int u = 0; u < 4; ++u) vec(r[u]);
    }
    for (; i < nv; i += kGcThreads) vec(__ldg(pv + i));
    const int64_t tail = head + nv * E;
    if (threadIdx.x < n - tail) f(one(tail + threadIdx.x));
}

template <int kMax>
__global__ void __launch_bounds__(kGcThreads) grad_sumsq_kernel(const __grid_constant__ GcTable<kMax> tab, int add,
                                                                double* __restrict__ partials) {
    __shared__ double red[kGcThreads / 32];
    pdl_trigger_and_wait();
    double acc = 0.0;
    for (int c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
        const GcTensor& t = tab.t[gc_find(tab, c)];
        const int64_t i0 = (c - t.first_chunk) * tab.chunk;
        const int64_t i1 = i0 + tab.chunk < t.n ? i0 + tab.chunk : t.n;
        auto f = [&](float v) { acc = fma(static_cast<double>(v), static_cast<double>(v), acc); };
        if (t.bf16) gc_read<true>(t.g, i0, i1, f);
        else gc_read<false>(t.g, i0, i1, f);
    }
    acc = warp_sum(acc);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = add ? partials[blockIdx.x] : 0.0;   // a list longer than one table adds up
        for (int w = 0; w < kGcThreads / 32; ++w) s += red[w];
        partials[blockIdx.x] = s;
    }
}

// norm and coefficient from the partials, in a fixed order, by every thread of a block.
__device__ __forceinline__ float gc_coef(const double* __restrict__ partials, int nparts, float max_norm,
                                         float* __restrict__ norm_out, float* __restrict__ coef_out, double* red) {
    double acc = 0.0;
    for (int i = threadIdx.x; i < nparts; i += kGcThreads) acc += partials[i];
    acc = warp_sum(acc);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = acc;
    __syncthreads();
    double S = 0.0;
#pragma unroll
    for (int w = 0; w < kGcThreads / 32; ++w) S += red[w];
    const double norm = sqrt(S);
    double c = 1.0;
    if (max_norm > 0.0f) {
        c = static_cast<double>(max_norm) / (norm + 1e-6);
        if (c > 1.0) c = 1.0;                          // a NaN norm stays NaN
    }
    const float cf = static_cast<float>(c);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (norm_out != nullptr) *norm_out = static_cast<float>(norm);
        if (coef_out != nullptr) *coef_out = cf;
    }
    return cf;
}

__global__ void __launch_bounds__(kGcThreads) grad_norm_kernel(const double* __restrict__ partials, int nparts,
                                                               float max_norm, float* __restrict__ norm_out,
                                                               float* __restrict__ coef_out) {
    __shared__ double red[kGcThreads / 32];
    pdl_trigger_and_wait();
    gc_coef(partials, nparts, max_norm, norm_out, coef_out, red);
}

// 32-byte loads and stores (a chunk's bytes are used once: kept out of L1, first to leave L2).
struct GcVec32 {
    uint32_t w[8];
};
__device__ __forceinline__ GcVec32 gc_ld32(const void* p) {
    GcVec32 r;
    asm volatile(
        "ld.global.L1::no_allocate.L2::evict_first.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
        : "l"(p)
        : "memory");
    return r;
}
__device__ __forceinline__ void gc_st32(void* p, const GcVec32& r) {
    asm volatile("st.global.L1::no_allocate.L2::evict_first.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
                 "r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]), "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7])
                 : "memory");
}
// Elements of a chunk from which the 32-byte loop runs (809 MB of fp32: the clip 395 -> 388 us).  Short
// chunks would leave most of their bytes to the 16-byte loop, and the wide kernel's registers keep
// fewer blocks on an SM (15 MB in 50 tensors: 15.8 -> 17.9 us).
constexpr int64_t kGcWide = 32768;

// out = fl(c g) over a chunk; out may be g (each element is read and written by one thread).
template <bool kBf16, bool kWide>
__device__ __forceinline__ void gc_scale(const void* g, void* out, int64_t i0, int64_t i1, float c) {
    constexpr int E = kBf16 ? 8 : 4;
    constexpr int kSize = kBf16 ? 2 : 4;
    const uint8_t* p = static_cast<const uint8_t*>(g) + i0 * kSize;
    uint8_t* q = static_cast<uint8_t*>(out) + i0 * kSize;
    const int64_t n = i1 - i0;
    auto one = [&](int64_t i) {
        if constexpr (kBf16)
            reinterpret_cast<uint16_t*>(q)[i] =
                float_to_bf16_bits(__fmul_rn(bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p)[i]), c));
        else
            reinterpret_cast<float*>(q)[i] = __fmul_rn(reinterpret_cast<const float*>(p)[i], c);
    };
    if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) != 0) {
        // source and destination never meet a 16-byte boundary together
        for (int64_t i = threadIdx.x; i < n; i += kGcThreads) one(i);
        return;
    }
    int64_t head = ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / kSize;
    if (head > n) head = n;
    if (threadIdx.x < head) one(threadIdx.x);
    const uint4* pv = reinterpret_cast<const uint4*>(p + head * kSize);
    uint4* qv = reinterpret_cast<uint4*>(q + head * kSize);
    const int64_t nv = (n - head) / E;
    auto word = [&](uint32_t w) -> uint32_t {
        if constexpr (kBf16)
            return static_cast<uint32_t>(float_to_bf16_bits(__fmul_rn(__uint_as_float(w << 16), c))) |
                   (static_cast<uint32_t>(float_to_bf16_bits(__fmul_rn(__uint_as_float(w & 0xFFFF0000u), c))) << 16);
        else
            return __float_as_uint(__fmul_rn(__uint_as_float(w), c));
    };
    auto vec = [&](const uint4& r) { return make_uint4(word(r.x), word(r.y), word(r.z), word(r.w)); };
    int64_t i = threadIdx.x;
    if (kWide && ((reinterpret_cast<uintptr_t>(pv) | reinterpret_cast<uintptr_t>(qv)) & 31) == 0) {
        // Whole rounds of the block only, the same number for every thread: the loops below give the
        // vectors to other threads, so they have to start behind one border.
        const int64_t n2 = nv / 2;
        int64_t b = 0;
        for (; b + 4 * kGcThreads <= n2; b += 4 * kGcThreads) {
            const int64_t j = b + threadIdx.x;
            GcVec32 r[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) r[u] = gc_ld32(pv + 2 * (j + u * kGcThreads));
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int e = 0; e < 8; ++e) r[u].w[e] = word(r[u].w[e]);
                gc_st32(qv + 2 * (j + u * kGcThreads), r[u]);
            }
        }
        i += 2 * b;
    }
    for (; i + 3 * kGcThreads < nv; i += 4 * kGcThreads) {
        uint4 r[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) r[u] = __ldcs(pv + i + u * kGcThreads);
#pragma unroll
        for (int u = 0; u < 4; ++u) __stcs(qv + i + u * kGcThreads, vec(r[u]));
    }
    for (; i < nv; i += kGcThreads) __stcs(qv + i, vec(__ldcs(pv + i)));
    const int64_t tail = head + nv * E;
    if (threadIdx.x < n - tail) one(tail + threadIdx.x);
}

// The chunks are taken from the last to the first: the norm's pass has just read the last ones,
// so as many of them as L2 holds are not read from memory again.
template <int kMax, bool kWide>
__global__ void __launch_bounds__(kGcThreads) grad_scale_kernel(const __grid_constant__ GcTable<kMax> tab,
                                                                const double* __restrict__ partials, int nparts,
                                                                float max_norm, float* __restrict__ norm_out,
                                                                float* __restrict__ coef_out) {
    __shared__ double red[kGcThreads / 32];
    pdl_trigger_and_wait();
    const float cf = gc_coef(partials, nparts, max_norm, norm_out, coef_out, red);
    for (int b = blockIdx.x; b < tab.chunks; b += gridDim.x) {
        const int c = tab.chunks - 1 - b;
        const GcTensor& t = tab.t[gc_find(tab, c)];
        if (cf == 1.0f && t.out == t.g) continue;      // nothing to change in place
        const int64_t i0 = (c - t.first_chunk) * tab.chunk;
        const int64_t i1 = i0 + tab.chunk < t.n ? i0 + tab.chunk : t.n;
        if (t.bf16) gc_scale<true, kWide>(t.g, t.out, i0, i1, cf);
        else gc_scale<false, kWide>(t.g, t.out, i0, i1, cf);
    }
}

}  // namespace bl
