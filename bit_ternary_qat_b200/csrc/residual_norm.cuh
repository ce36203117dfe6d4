// residual_norm.cuh -- the step between two BitLinears of a residual stack, and its gradient.
//
// Restates P3 ("BitNet 1.5技术解析…") §3.1 (RMSNorm, then the activation quantiser, in front of
// every BitLinear) with the residual branch the layer sits in (P5 keeps the residual stream in
// full precision while the block runs in bf16, so the two have separate types here):
//   n  = y r1 g1        r1_t = 1/sqrt(mean_k y^2 + eps1)      (norm behind the block; optional)
//   x' = alpha x + beta gate n                                 (held in the residual's type)
//   h  = x' r2 g2       r2_t = 1/sqrt(mean_k x'^2 + eps2)     (norm in front of the next block)
// and h is written as it is, or quantised exactly as act_quant.cuh quantises it, or not at all.
//
// Arithmetic of the forward, the same in both kernels: both sums of squares in fp64 (added in another
// order in each: the sums agree to about 2^-46, so that r, and with it a row's codes, can differ by an
// fp32 step between them in one row of some millions; one kernel on one row always gives the same);
// every product and sum of an element in fp32 with one rounding each,
//   x' = fl( fl(x alpha) + fl( fl(y r1) w ) ),   w = fl( fl(gate beta) g1 )
// (w is the same for every row unless the gate is a token's or an element's); x' rounded once to
// the residual's type, and h = fl(fl(x' r2) g2) computed from the rounded x' (what the next layer
// reads).
#pragma once
#include "common.cuh"
#include "act_quant.cuh"
#include "ring_flight.cuh"

namespace bl {

enum RnGate : int { kGateNone = 0, kGateScalar = 1, kGateChannel = 2, kGateToken = 3, kGateElement = 4 };

// E adjacent elements at vector index v, widened exactly to fp32.  E = 8 (16- or 32-byte
// aligned rows) or 1 (rows of any length).
template <bool kBf16, int E>
__device__ __forceinline__ void rn_load(const void* __restrict__ p, int64_t v, float (&f)[E]) {
    static_assert(E == 8 || E == 1, "E");
    if constexpr (E == 8) {
        if constexpr (kBf16) {
            const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p) + v);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        } else {
            const float4 a = __ldcs(reinterpret_cast<const float4*>(p) + 2 * v);
            const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 2 * v + 1);
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
            f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        }
    } else {
        if constexpr (kBf16) f[0] = bf16_bits_to_float(__ldcs(reinterpret_cast<const uint16_t*>(p) + v));
        else f[0] = __ldcs(reinterpret_cast<const float*>(p) + v);
    }
}

// Per-column fp32 gains (kept in L1/L2: every row reads them).
template <int E>
__device__ __forceinline__ void rn_load_gain(const float* __restrict__ g, int v, float (&f)[E]) {
    if constexpr (E >= 4) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(g) + (E / 4) * v + i);
            f[4 * i] = a.x; f[4 * i + 1] = a.y; f[4 * i + 2] = a.z; f[4 * i + 3] = a.w;
        }
    } else {
        f[0] = __ldg(g + v);
    }
}

// Round to the stored type (bf16: once, to nearest even); f becomes the stored values.  E = 4 keeps
// an fp32 warp's 16-byte stores adjacent (8 would write every 32-byte sector in two halves).
template <bool kBf16, int E>
__device__ __forceinline__ void rn_store(void* __restrict__ p, int64_t v, float (&f)[E]) {
    if constexpr (kBf16) {
        uint32_t h[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            h[e] = float_to_bf16_bits(f[e]);
            f[e] = __uint_as_float(h[e] << 16);
        }
        if constexpr (E == 8)
            reinterpret_cast<uint4*>(p)[v] = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16),
                                                        h[4] | (h[5] << 16), h[6] | (h[7] << 16));
        else if constexpr (E == 4)
            reinterpret_cast<uint2*>(p)[v] = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
        else
            reinterpret_cast<uint16_t*>(p)[v] = static_cast<uint16_t>(h[0]);
    } else {
        if constexpr (E >= 4) {
#pragma unroll
            for (int i = 0; i < E / 4; ++i)
                reinterpret_cast<float4*>(p)[(E / 4) * v + i] =
                    make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
        } else {
            reinterpret_cast<float*>(p)[v] = f[0];
        }
    }
}

struct RnFwdArgs {
    const void* x;        // [T x K] residual
    const void* y;        // [T x K] block output
    const void* gate;     // per gate_kind; fp32 except kGateElement (y's type)
    const float* g_post;  // [K] or NULL
    const float* g_pre;   // [K] or NULL
    void* xout;           // [T x K] new residual, x's type (may be x)
    float* r_post;        // [T], with post
    float* r_pre;         // [T], with a norm output
    void* h;              // [T x K] y's type, or NULL
    int8_t* xq;           // [T x K] or NULL
    float* sx;            // [T], with xq
    void* xdq;            // [T x K] y's type, or NULL
    int T, K;
    int post, gate_kind;
    float alpha, beta, eps_post, eps_pre;
};

// r = (mean + eps)^(-1/2) in fp64, rounded once.
__device__ __forceinline__ float rn_rinv(double ss, double invK, float eps) {
    return static_cast<float>(rsqrt(fma(ss, invK, static_cast<double>(eps))));
}

// Sum / maximum over the threads of one row: a warp (kWarpRow) or the whole block.
template <bool kWarpRow, int NT>
__device__ __forceinline__ double rn_row_sum(double v, double* red) {
    v = warp_sum(v);
    if constexpr (kWarpRow) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) s += red[w];
    return s;
}
template <bool kWarpRow, int NT>
__device__ __forceinline__ float rn_row_max(float v, float* red) {
    v = warp_max(v);
    if constexpr (kWarpRow) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = red[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) s = fmaxf(s, red[w]);
    return s;
}

// Forward.  kWarpRow: one warp per row, NT / 32 rows per block; else one row per block.
// Thread i of a row owns vectors i + j * (threads per row), j < VPT; the row is read once and
// stays in registers through its reductions (sum y^2; sum x'^2; max |h|).
template <bool kBf16X, bool kBf16Y, bool kWarpRow, int E, int NT, int VPT, bool kGateElem>
__global__ void __launch_bounds__(NT) residual_norm_kernel(const RnFwdArgs a) {
    constexpr int TPR = kWarpRow ? 32 : NT;
    constexpr int kLutRows = kWarpRow ? NT / 32 : 1;
    using LutT = typename DqLut<kBf16Y>::T;
    __shared__ double red_y[NT / 32], red_x[NT / 32];
    __shared__ float red_m[NT / 32];
    __shared__ LutT lut_all[E == 8 ? kLutRows : 1][E == 8 ? 256 : 1];
    pdl_trigger_and_wait();

    const int tid = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t t = kWarpRow ? static_cast<int64_t>(blockIdx.x) * (NT / 32) + (threadIdx.x >> 5) : blockIdx.x;
    if (t >= a.T) return;                         // warp-uniform (block-uniform for block rows)
    const int nvec = a.K / E;
    const int64_t row0 = t * static_cast<int64_t>(nvec);
    const double invK = 1.0 / static_cast<double>(a.K);

    float x[VPT][E], y[VPT][E], ge[kGateElem ? VPT : 1][E];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = tid + j * TPR;
        if (v < nvec) {
            rn_load<kBf16Y, E>(a.y, row0 + v, y[j]);
            rn_load<kBf16X, E>(a.x, row0 + v, x[j]);
            if constexpr (kGateElem) rn_load<kBf16Y, E>(a.gate, row0 + v, ge[j]);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) y[j][e] = x[j][e] = 0.0f;
        }
    }

    if (a.post) {
        double ss = 0.0;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < E; ++e) ss = fma(static_cast<double>(y[j][e]), static_cast<double>(y[j][e]), ss);
        ss = rn_row_sum<kWarpRow, NT>(ss, red_y);
        const float r1 = rn_rinv(ss, invK, a.eps_post);
        if (tid == 0) a.r_post[t] = r1;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < E; ++e) y[j][e] = __fmul_rn(y[j][e], r1);
    }
    // x' = fl(fl(x alpha) + fl(fl(y r1) w)), rounded to the residual's type and stored
    float gs = 1.0f;
    if (a.gate_kind == kGateScalar) gs = __ldg(static_cast<const float*>(a.gate));
    if (a.gate_kind == kGateToken) gs = __ldg(static_cast<const float*>(a.gate) + t);
    double ss = 0.0;
    float mx = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = tid + j * TPR;
        if (v >= nvec) continue;
        float w[E];
        if constexpr (kGateElem) {
#pragma unroll
            for (int e = 0; e < E; ++e) w[e] = ge[j][e];
        } else if (a.gate_kind == kGateChannel) {
            rn_load_gain<E>(static_cast<const float*>(a.gate), v, w);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) w[e] = gs;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] = __fmul_rn(w[e], a.beta);
        if (a.g_post != nullptr) {
            float g[E];
            rn_load_gain<E>(a.g_post, v, g);
#pragma unroll
            for (int e = 0; e < E; ++e) w[e] = __fmul_rn(w[e], g[e]);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) x[j][e] = __fadd_rn(__fmul_rn(x[j][e], a.alpha), __fmul_rn(y[j][e], w[e]));
        rn_store<kBf16X, E>(a.xout, row0 + v, x[j]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            mx = fmaxf(mx, fabsf(x[j][e]));
            ss = fma(static_cast<double>(x[j][e]), static_cast<double>(x[j][e]), ss);
        }
    }
    if (a.r_pre == nullptr) return;
    ss = rn_row_sum<kWarpRow, NT>(ss, red_x);
    const float r2 = rn_rinv(ss, invK, a.eps_pre);
    if (tid == 0) a.r_pre[t] = r2;
    // h = fl(fl(x' r2) g2)
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = tid + j * TPR;
        if (v >= nvec) continue;
#pragma unroll
        for (int e = 0; e < E; ++e) x[j][e] = __fmul_rn(x[j][e], r2);
        if (a.g_pre != nullptr) {
            float g[E];
            rn_load_gain<E>(a.g_pre, v, g);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                x[j][e] = __fmul_rn(x[j][e], g[e]);
                m = fmaxf(m, fabsf(x[j][e]));
            }
        }
        if (a.h != nullptr) rn_store<kBf16Y, E>(a.h, row0 + v, x[j]);
    }
    if constexpr (E == 8) {
        if (a.xq == nullptr) return;
        // without a gain rounding is monotone: max |fl(x' r2)| = fl(max |x'| r2)
        if (a.g_pre == nullptr) m = __fmul_rn(mx, r2);
        m = rn_row_max<kWarpRow, NT>(m, red_m);
        const float s = __fdiv_rn(127.0f, fmaxf(m, 1e-5f));
        if (tid == 0) a.sx[t] = s;
        LutT* lut = lut_all[kWarpRow ? threadIdx.x >> 5 : 0];
        if (a.xdq != nullptr) {
            const float c = __frcp_rn(s);
            for (int i = tid; i < 256; i += TPR)
                lut[i] = DqLut<kBf16Y>::make(div_by_scale(static_cast<float>(i - 128), s, c));
            if constexpr (kWarpRow) __syncwarp();
            else __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * TPR;
            if (v >= nvec) continue;
            if constexpr (kBf16Y) {
                quant_store_vec<true, 8>(x[j], s, a.xq, a.xdq, row0 + v, lut);
            } else {
                const float lo[4] = {x[j][0], x[j][1], x[j][2], x[j][3]};
                const float hi[4] = {x[j][4], x[j][5], x[j][6], x[j][7]};
                quant_store_vec<false, 4>(lo, s, a.xq, a.xdq, 2 * (row0 + v), lut);
                quant_store_vec<false, 4>(hi, s, a.xq, a.xdq, 2 * (row0 + v) + 1, lut);
            }
        }
    }
}

// ------------------------------------------------------------------------------------
// Rows through a shared-memory ring.  A block is RG groups of TG threads, each group with rows of
// its own (group q of all takes rows q, q + Q, ...) and a ring of whole rows that bulk copies
// (cp.async.bulk) fill while earlier rows are worked on; a group synchronises by its own named
// barrier (a warp by itself), so the groups' barriers and reductions overlap.  A stage is refilled
// by the group's first thread once a barrier of the row shows that every thread has read it.
// Every wait is bounded; after one that ran out the group goes on to its end (with whatever
// is in shared memory: the status word tells), so that no barrier is left waiting, but its first
// thread posts no more copies and at the end waits (with a limit) for those on their way.
// ------------------------------------------------------------------------------------
constexpr int kRnMaxStages = 4;

template <int TG>
__device__ __forceinline__ void rn_group_sync(int g) {
    if constexpr (TG == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "n"(TG) : "memory");
}
// Sum / maximum over a group's threads; `red` (TG / 32 values) is not written again before
// another barrier of the group.
template <int TG, typename V, typename Op>
__device__ __forceinline__ V rn_group_reduce(V v, V* red, int g, Op&& op) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    if constexpr (TG == 32) return v;
    if ((threadIdx.x & 31) == 0) red[(threadIdx.x % TG) >> 5] = v;
    rn_group_sync<TG>(g);
    v = red[0];
#pragma unroll
    for (int w = 1; w < TG / 32; ++w) v = op(v, red[w]);
    return v;
}

// Rows that are no whole 16-byte vectors (kOdd): bulk copies move the aligned bytes around the row,
// and its elements start `rn_shift` bytes into them.  Room for a row of n bytes in a stage:
__host__ __device__ constexpr uint32_t rn_pitch(bool odd, uint32_t n) { return odd ? (n + 30u) & ~15u : n; }
__device__ __forceinline__ uint32_t rn_shift(int64_t first_byte) { return static_cast<uint32_t>(first_byte) & 15u; }

// Where a row's bulk copy reads from: bytes [lo, lo + n) of its array (of `total` bytes, 16-byte
// aligned base), the aligned bytes around [b0, b1).  The last rows of the array stop at the last
// whole 16 bytes inside it; what is behind them is copied by the calling thread (at most 15 bytes).
struct RnSpan {
    int64_t lo;
    uint32_t n;
};
template <int kSize>
__device__ __forceinline__ RnSpan rn_span(uint8_t* dst, const uint8_t* src, int64_t b0, int64_t b1, int64_t total) {
    RnSpan s;
    s.lo = b0 & ~int64_t(15);
    int64_t hi = (b1 + 15) & ~int64_t(15);
    if (hi > total) {
        hi = total & ~int64_t(15);
        if (hi < s.lo) hi = s.lo;
        for (int64_t b = hi > b0 ? hi : b0; b < b1; b += kSize) {
            if constexpr (kSize == 2)
                *reinterpret_cast<uint16_t*>(dst + (b - s.lo)) = *reinterpret_cast<const uint16_t*>(src + b);
            else
                *reinterpret_cast<uint32_t*>(dst + (b - s.lo)) = *reinterpret_cast<const uint32_t*>(src + b);
        }
    }
    s.n = static_cast<uint32_t>(hi - s.lo);
    return s;
}

// E adjacent elements out of shared memory, widened exactly.
template <bool kBf16, int E>
__device__ __forceinline__ void rn_lds(const uint8_t* row, int v, float (&f)[E]) {
    if constexpr (E == 1) {
        if constexpr (kBf16) f[0] = bf16_bits_to_float(reinterpret_cast<const uint16_t*>(row)[v]);
        else f[0] = reinterpret_cast<const float*>(row)[v];
    } else if constexpr (kBf16) {
        uint32_t w[E / 2];
        if constexpr (E == 8) {
            const uint4 a = reinterpret_cast<const uint4*>(row)[v];
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        } else {
            const uint2 a = reinterpret_cast<const uint2*>(row)[v];
            w[0] = a.x; w[1] = a.y;
        }
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            const float4 a = reinterpret_cast<const float4*>(row)[(E / 4) * v + i];
            f[4 * i] = a.x; f[4 * i + 1] = a.y; f[4 * i + 2] = a.z; f[4 * i + 3] = a.w;
        }
    }
}

// Codes of E elements of h with scale s, and their values fl(q / s) rounded to y's type
// (c = fl(1 / s); see div_by_scale).
template <bool kBf16Y, int E>
__device__ __forceinline__ void rn_quant_store(const float (&h)[E], float s, float c, int8_t* xq, void* xdq, int64_t v) {
    uint32_t tb[E];
#pragma unroll
    for (int e = 0; e < E; ++e) tb[e] = quant_bits(h[e], s);
    if constexpr (E == 8)
        reinterpret_cast<uint2*>(xq)[v] =
            make_uint2(gather_low_bytes(tb[0], tb[1], tb[2], tb[3]), gather_low_bytes(tb[4], tb[5], tb[6], tb[7]));
    else
        reinterpret_cast<uint32_t*>(xq)[v] = gather_low_bytes(tb[0], tb[1], tb[2], tb[3]);
    if (xdq != nullptr) {
        float d[E];
#pragma unroll
        for (int e = 0; e < E; ++e) d[e] = div_by_scale(__fsub_rn(__uint_as_float(tb[e]), kRoundMagic), s, c);
        rn_store<kBf16Y, E>(xdq, v, d);
    }
}

// E adjacent gains kept in shared memory (kSm; in E / 4 planes of nvec vectors of 4, so that a
// warp's 16-byte reads are adjacent) or read from global memory.
template <bool kSm, int E>
__device__ __forceinline__ void rn_gain(const float* g, int v, int nvec, float (&f)[E]) {
    if constexpr (kSm && E == 1) {
        f[0] = g[v];
    } else if constexpr (kSm) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            const float4 a = reinterpret_cast<const float4*>(g)[i * nvec + v];
            f[4 * i] = a.x; f[4 * i + 1] = a.y; f[4 * i + 2] = a.z; f[4 * i + 3] = a.w;
        }
    } else {
        rn_load_gain<E>(g, v, f);
    }
}
template <int E>
__device__ __forceinline__ void rn_gain_put(float* g, int v, int nvec, const float (&f)[E]) {
    if constexpr (E == 1) g[v] = f[0];
#pragma unroll
    for (int i = 0; i < E / 4; ++i)
        reinterpret_cast<float4*>(g)[i * nvec + v] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
}

// HBM-bound in bursts, issue-bound at the clock a sustained load leaves: 16384 x 4096, fp32 residual
// beside a bf16 block, quantised, 872 MB in 143 us, up to 152 as the clock falls; bf16 alone, 604 MB,
// 108 to 117 us.  A block per row with direct loads took 241 us.
// Forward: thread i of a group owns vectors i + j * TG of E elements, EPT elements in all (kOdd: the
// rows are no whole 16-byte vectors, E = 1).  kSm:
// the weights w (for a gate that is the same in every row) and g2 are formed once per block in
// shared memory; the rows read them from there.
template <bool kBf16X, bool kBf16Y, int TG, int kMaxThreads, int EPT, bool kGateElem, bool kSm, bool kOdd>
__global__ void __launch_bounds__(kMaxThreads, 1)
    residual_norm_ring_kernel(const RnFwdArgs a, int stages, uint64_t wait_ns) {
    constexpr int E = kOdd ? 1 : kBf16X ? 8 : 4;
    constexpr int VPT = EPT / E;
    constexpr int kRG = kMaxThreads / TG;
    extern __shared__ __align__(128) uint8_t rn_smem[];
    __shared__ uint64_t full[kRG][kRnMaxStages];
    __shared__ double red_y[kRG][2][TG / 32], red_x[kRG][2][TG / 32];
    __shared__ float red_m[kRG][2][TG / 32];
    __shared__ RingFlight flight[kRG];            // each by its group's first thread alone
    __shared__ volatile int abort_flag;
    const int g = threadIdx.x / TG, tid = threadIdx.x % TG;
    const int RG = blockDim.x / TG;
    if (threadIdx.x == 0) abort_flag = 0;
    if (tid == 0) {
        flight[g].reset();
        for (int s = 0; s < stages; ++s) mbar_init(&full[g][s], 1);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_trigger_and_wait();

    const int nvec = a.K / E;
    constexpr int xs = kBf16X ? 2 : 4, ys = kBf16Y ? 2 : 4;
    const uint32_t xb = a.K * xs, yb = a.K * ys;
    const uint32_t o_y = rn_pitch(kOdd, xb), o_g = o_y + rn_pitch(kOdd, yb);
    const uint32_t row_bytes = o_g + (kGateElem ? rn_pitch(kOdd, yb) : 0u);
    const uint32_t gain_bytes = (static_cast<uint32_t>(a.K) * 4u + 15u) & ~15u;
    float* w_sm = reinterpret_cast<float*>(rn_smem);
    float* g_sm = reinterpret_cast<float*>(rn_smem + gain_bytes);
    uint8_t* ring = rn_smem + (kSm ? 2 * gain_bytes : 0) + static_cast<size_t>(g) * stages * row_bytes;
    const int64_t step = static_cast<int64_t>(gridDim.x) * RG;
    const double invK = 1.0 / static_cast<double>(a.K);
    auto issue = [&](int64_t t, int s) {
        uint8_t* dst = ring + static_cast<size_t>(s) * row_bytes;
        uint64_t* bar = &full[g][s];
        const uint8_t *xg = static_cast<const uint8_t*>(a.x), *yg = static_cast<const uint8_t*>(a.y),
                      *gg = static_cast<const uint8_t*>(a.gate);
        if constexpr (kOdd) {
            const int64_t rows = a.T;
            const RnSpan sx = rn_span<xs>(dst, xg, t * xb, (t + 1) * xb, rows * xb);
            const RnSpan sy = rn_span<ys>(dst + o_y, yg, t * yb, (t + 1) * yb, rows * yb);
            RnSpan sg{0, 0};
            if constexpr (kGateElem) sg = rn_span<ys>(dst + o_g, gg, t * yb, (t + 1) * yb, rows * yb);
            mbar_arrive_expect_tx(bar, sx.n + sy.n + sg.n);
            if (sx.n) bulk_load(dst, xg + sx.lo, sx.n, bar);
            if (sy.n) bulk_load(dst + o_y, yg + sy.lo, sy.n, bar);
            if (sg.n) bulk_load(dst + o_g, gg + sg.lo, sg.n, bar);
        } else {
            mbar_arrive_expect_tx(bar, row_bytes);
            bulk_load(dst, xg + t * xb, xb, bar);
            bulk_load(dst + o_y, yg + t * yb, yb, bar);
            if constexpr (kGateElem) bulk_load(dst + o_g, gg + t * yb, yb, bar);
        }
    };
    const int64_t t_first = static_cast<int64_t>(blockIdx.x) * RG + g;
    if (tid == 0)
        for (int s = 0; s < stages; ++s)
            if (t_first + s * step < a.T) issue(t_first + s * step, s);

    // gate * beta where it does not depend on the element of a row
    const bool row_gate = a.gate_kind == kGateToken;
    float gs = a.beta;
    if (a.gate_kind == kGateScalar) gs = __fmul_rn(__ldg(static_cast<const float*>(a.gate)), a.beta);
    // the weights of vector v as far as they are the same in every row
    auto col_weight = [&](int v, float (&w)[E]) {
        if (!kGateElem && a.gate_kind == kGateChannel) {
            rn_load_gain<E>(static_cast<const float*>(a.gate), v, w);
#pragma unroll
            for (int e = 0; e < E; ++e) w[e] = __fmul_rn(w[e], a.beta);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) w[e] = kGateElem || row_gate ? 1.0f : gs;
        }
        if (a.g_post != nullptr) {
            float q[E];
            rn_load_gain<E>(a.g_post, v, q);
#pragma unroll
            for (int e = 0; e < E; ++e) w[e] = __fmul_rn(w[e], q[e]);
        }
    };
    if constexpr (kSm) {
        for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
            float w[E];
            col_weight(v, w);
            rn_gain_put<E>(w_sm, v, nvec, w);
            if (a.g_pre != nullptr) {
                rn_load_gain<E>(a.g_pre, v, w);
                rn_gain_put<E>(g_sm, v, nvec, w);
            }
        }
        __syncthreads();
    }

    int s = 0;
    uint32_t ph = 0, par = 0;
    for (int64_t t = t_first; t < a.T; t += step, par ^= 1u) {
        if (row_gate) gs = __fmul_rn(__ldg(static_cast<const float*>(a.gate) + t), a.beta);
        mbar_wait(&full[g][s], ph, wait_ns, &abort_flag);
        const uint8_t* stage = ring + static_cast<size_t>(s) * row_bytes;
        const uint8_t* xr = stage + (kOdd ? rn_shift(t * xb) : 0u);
        const uint8_t* yr = stage + o_y + (kOdd ? rn_shift(t * yb) : 0u);
        const int64_t row0 = t * nvec;
        float r1 = 1.0f;
        if (a.post) {
            double ss = 0.0;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = tid + j * TG;
                if (v >= nvec) continue;
                float y[E];
                rn_lds<kBf16Y, E>(yr, v, y);
#pragma unroll
                for (int e = 0; e < E; ++e) ss = fma(static_cast<double>(y[e]), static_cast<double>(y[e]), ss);
            }
            ss = rn_group_reduce<TG>(ss, red_y[g][par], g, [](double p, double q) { return p + q; });
            r1 = rn_rinv(ss, invK, a.eps_post);
            if (tid == 0) a.r_post[t] = r1;
        }
        float x[VPT][E];
        double ss = 0.0;
        float mx = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * TG;
            if (v >= nvec) continue;
            float n[E], w[E];
            rn_lds<kBf16X, E>(xr, v, x[j]);
            rn_lds<kBf16Y, E>(yr, v, n);
            if constexpr (kSm) rn_gain<true, E>(w_sm, v, nvec, w);
            else col_weight(v, w);
            if constexpr (kGateElem) {
                float q[E];
                rn_lds<kBf16Y, E>(yr + (o_g - o_y), v, q);
#pragma unroll
                for (int e = 0; e < E; ++e) w[e] = __fmul_rn(__fmul_rn(q[e], a.beta), w[e]);
            } else if (row_gate) {
#pragma unroll
                for (int e = 0; e < E; ++e) w[e] = __fmul_rn(gs, w[e]);
            }
            if (a.post) {
#pragma unroll
                for (int e = 0; e < E; ++e) n[e] = __fmul_rn(n[e], r1);
            }
#pragma unroll
            for (int e = 0; e < E; ++e)
                x[j][e] = __fadd_rn(__fmul_rn(x[j][e], a.alpha), __fmul_rn(n[e], w[e]));
            rn_store<kBf16X, E>(a.xout, row0 + v, x[j]);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                mx = fmaxf(mx, fabsf(x[j][e]));
                ss = fma(static_cast<double>(x[j][e]), static_cast<double>(x[j][e]), ss);
            }
        }
        if (a.r_pre != nullptr) ss = rn_group_reduce<TG>(ss, red_x[g][par], g, [](double p, double q) { return p + q; });
        if (TG == 32 || a.r_pre == nullptr) rn_group_sync<TG>(g);
        // every thread of the group has read the stage
        if (tid == 0 && t + stages * step < a.T) {
            if (abort_flag == 0) issue(t + stages * step, s);
            else flight[g].stop(t);
        }
        if (++s == stages) { s = 0; ph ^= 1u; }
        if (a.r_pre == nullptr) continue;

        const float r2 = rn_rinv(ss, invK, a.eps_pre);
        if (tid == 0) a.r_pre[t] = r2;
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * TG;
            if (v >= nvec) continue;
#pragma unroll
            for (int e = 0; e < E; ++e) x[j][e] = __fmul_rn(x[j][e], r2);
            if (a.g_pre != nullptr) {
                float q[E];
                rn_gain<kSm, E>(kSm ? g_sm : a.g_pre, v, nvec, q);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    x[j][e] = __fmul_rn(x[j][e], q[e]);
                    m = fmaxf(m, fabsf(x[j][e]));
                }
            }
            if (a.h != nullptr) rn_store<kBf16Y, E>(a.h, row0 + v, x[j]);
        }
        if (kOdd || a.xq == nullptr) continue;    // codes need K % 32 == 0
        // without a gain rounding is monotone: max |fl(x' r2)| = fl(max |x'| r2)
        if (a.g_pre == nullptr) m = __fmul_rn(mx, r2);
        m = rn_group_reduce<TG>(m, red_m[g][par], g, [](float p, float q) { return fmaxf(p, q); });
        const float sc = __fdiv_rn(127.0f, fmaxf(m, 1e-5f)), c = __frcp_rn(sc);
        if (tid == 0) a.sx[t] = sc;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * TG;
            if constexpr (!kOdd)
                if (v < nvec) rn_quant_store<kBf16Y, E>(x[j], sc, c, a.xq, a.xdq, row0 + v);
        }
    }
    if (tid == 0 && abort_flag != 0) {
        // loads that had not landed when a wait ran out: let them (briefly) before the block ends
        flight[g].drain(stages, t_first, step, a.T,
                        [&](int q, uint32_t parity) { mbar_wait(&full[g][q], parity, 100000000ull, nullptr); });
    }
}

// ------------------------------------------------------------------------------------
// Backward.  With u1 = y r1, u2 = x' r2:
//   c2 = mean_k(g2 dh u2),   d = dx' + r2 (g2 dh - u2 c2)     gradient of the new residual
//   dX = alpha d
//   dn = beta gate d,  c1 = mean_k(g1 dn u1),  dY = r1 (g1 dn - u1 c1)    (dY = dn without)
//   dg2 = sum_t dh u2,   dg1 = sum_t dn u1,   dgate = sum beta d g1 u1 over what it was given for
// (dx' or dh may be absent).  In the kernels' terms: q = d u1 and
//   w = beta gate g1 where the gate is the same in every row, else beta g1;  f the token's gate or 1
//   dY = f r1 (w d - u1 mean_k(w q)),   token gate's gradient = sum_k w q
// and one column sum S = sum_t f q serves both learned vectors behind the block:
//   dg1 = beta gate S,   dgate = beta g1 S   (channel; its sum over k for a scalar).
// An element's gate multiplies w d and the sums' terms, and its gradient is w q.
// ------------------------------------------------------------------------------------
struct RnBwdArgs {
    const float* dx;      // [T x K] gradient of x' from the residual stream, or NULL
    const float* dh;      // [T x K] gradient of h, or NULL
    const void* x;        // [T x K] x' (residual's type); read only with dh
    const void* y;        // [T x K] block output
    const void* gate;
    const float* r_post;
    const float* r_pre;
    const float* g_post;
    const float* g_pre;
    float* dX;            // [T x K] (may be dx or dh)
    void* dY;             // [T x K] y's type
    void* dgate;          // token: fp32 [T]; element: [T x K] y's type; else NULL
    float* part_pre;      // [G x K] partial sums of dg2, or NULL
    float* part_s;        // [G x K] of S, or NULL
    double* part_scalar;  // [blocks] of sum_k g1 S, or NULL
    int T, K;
    int post, gate_kind;
    float alpha, beta;
};

constexpr int kRnMaxBlocks = 148;   // partial rows

// w of column k as far as it is the same in every row.
__device__ __forceinline__ float rn_col_w(const RnBwdArgs& a, int k) {
    float w = a.beta;
    if (a.gate_kind == kGateScalar) w *= __ldg(static_cast<const float*>(a.gate));
    if (a.gate_kind == kGateChannel) w *= __ldg(static_cast<const float*>(a.gate) + k);
    return a.g_post != nullptr ? w * __ldg(a.g_post + k) : w;
}

// Two sums over the threads of a group, or of a whole cluster, with one barrier.  In a cluster
// every warp sends its sums to every block's slots (8 bytes of distributed shared memory that
// count on that block's mbarrier), so one wait stands for the block barrier and the exchange.
// Slots alternate by row: a block sends row i + 2 only after all warps of all blocks have sent
// row i + 1, hence read row i's slots.
__device__ __forceinline__ void rn_add2(float2& v, int o) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
}
__device__ __forceinline__ void st_async_v2(uint32_t addr, uint32_t bar, float2 v) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(addr),
                 "f"(v.x), "f"(v.y), "r"(bar)
                 : "memory");
}

// Through a ring of rows (see the forward): thread i of a group owns vectors i + j * TG of four
// columns (kOdd: one), EPT columns in all, of every row its group takes, and keeps their column sums
// in registers.  A row is read from shared memory twice (for c2, then for everything else);
// what the last pass needs, w d and u1, stays in registers, so the stage is refilled before it.
// The first pass of the next row runs before the barrier that ends the second pass of this one, so
// a row costs one barrier: its reduction carries this row's sum of w q and c2 of the next.
// HBM-bound: 16384 x 4096 bf16 with a channel gate 186 us for 1.21 GB (6.5 TB/s), 4096 x 16384 fp32
// in clusters of four 252 us for 1.61 GB; three walks over each row took 777 us.
// kCl > 1: a cluster of kCl blocks shares each row, cols columns a block, so that gains and two
// stages always fit.  At the end the groups' sums are joined in shared memory in group order and
// each block (or cluster) writes one partial row.
template <bool kBf16X, bool kBf16Y, int TG, int EPT, int kCl, bool kElem, bool kOdd>
__global__ void __launch_bounds__(512, 1)
    residual_norm_bwd_ring_kernel(const RnBwdArgs a, int cols, int stages, uint64_t wait_ns) {
    constexpr int kThreads = 512;
    constexpr int E = kOdd ? 1 : 4;
    constexpr int VPT = EPT / E;
    constexpr int kRG = kThreads / TG;
    constexpr int kW = TG / 32 * kCl;                 // warps that join a row's sums
    static_assert(kCl == 1 || TG == kThreads, "a cluster's blocks are one group each");
    extern __shared__ __align__(128) uint8_t rn_smem[];
    __shared__ uint64_t full[kRG][kRnMaxStages];
    __shared__ uint64_t xbar[2];
    __shared__ __align__(16) float2 red[kRG][2][kW];
    __shared__ double red_s[kThreads / 32];
    __shared__ RingFlight flight[kRG];            // each by its group's first thread alone
    __shared__ volatile int abort_flag;
    const int g = threadIdx.x / TG, tid = threadIdx.x % TG, lane = threadIdx.x & 31;
    const int RG = blockDim.x / TG;
    const int rank = kCl > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        mbar_init(&xbar[0], 1);
        mbar_init(&xbar[1], 1);
    }
    if (tid == 0) {
        flight[g].reset();
        for (int s = 0; s < stages; ++s) mbar_init(&full[g][s], 1);
        fence_mbar_init();
    }
    if constexpr (kCl > 1) cluster_sync_all();
    else __syncthreads();
    pdl_trigger_and_wait();

    // this block's columns [k0, k0 + cols)
    const int k0 = rank * cols;
    cols = min(cols, a.K - k0);
    const int nvec = cols / E, v0 = k0 / E;
    const int64_t row_vecs = a.K / E;
    const bool has_dx = a.dx != nullptr, has_dh = a.dh != nullptr;
    // a row's arrays in its stage: dx, dh, x, y, gate
    constexpr int xs = kBf16X ? 2 : 4, ys = kBf16Y ? 2 : 4;
    const uint32_t fb = cols * 4u, xb = cols * xs, yb = cols * ys;
    const uint32_t pf = rn_pitch(kOdd, fb), px = rn_pitch(kOdd, xb), py = rn_pitch(kOdd, yb);
    const uint32_t o_dh = has_dx ? pf : 0u, o_x = o_dh + (has_dh ? pf : 0u), o_y = o_x + (has_dh ? px : 0u), o_g = o_y + py;
    const uint32_t row_bytes = o_g + (kElem ? py : 0u);
    const uint32_t gain_bytes = (fb + 15u) & ~15u;
    float* g2_sm = reinterpret_cast<float*>(rn_smem);
    float* w_sm = reinterpret_cast<float*>(rn_smem + gain_bytes);
    uint8_t* ring = rn_smem + 2 * gain_bytes + static_cast<size_t>(g) * stages * row_bytes;
    const int64_t step = static_cast<int64_t>(gridDim.x / kCl) * RG;
    auto issue = [&](int64_t t, int s) {
        uint8_t* dst = ring + static_cast<size_t>(s) * row_bytes;
        uint64_t* bar = &full[g][s];
        const int64_t at = t * a.K + k0;
        const uint8_t *dxg = reinterpret_cast<const uint8_t*>(a.dx), *dhg = reinterpret_cast<const uint8_t*>(a.dh),
                      *xg = static_cast<const uint8_t*>(a.x), *yg = static_cast<const uint8_t*>(a.y),
                      *gg = static_cast<const uint8_t*>(a.gate);
        if constexpr (kOdd) {
            const int64_t all = static_cast<int64_t>(a.T) * a.K;
            RnSpan s1{0, 0}, s2{0, 0}, s3{0, 0}, s5{0, 0};
            if (has_dx) s1 = rn_span<4>(dst, dxg, at * 4, at * 4 + fb, all * 4);
            if (has_dh) {
                s2 = rn_span<4>(dst + o_dh, dhg, at * 4, at * 4 + fb, all * 4);
                s3 = rn_span<xs>(dst + o_x, xg, at * xs, at * xs + xb, all * xs);
            }
            const RnSpan s4 = rn_span<ys>(dst + o_y, yg, at * ys, at * ys + yb, all * ys);
            if constexpr (kElem) s5 = rn_span<ys>(dst + o_g, gg, at * ys, at * ys + yb, all * ys);
            mbar_arrive_expect_tx(bar, s1.n + s2.n + s3.n + s4.n + s5.n);
            if (s1.n) bulk_load(dst, dxg + s1.lo, s1.n, bar);
            if (s2.n) bulk_load(dst + o_dh, dhg + s2.lo, s2.n, bar);
            if (s3.n) bulk_load(dst + o_x, xg + s3.lo, s3.n, bar);
            if (s4.n) bulk_load(dst + o_y, yg + s4.lo, s4.n, bar);
            if (s5.n) bulk_load(dst + o_g, gg + s5.lo, s5.n, bar);
        } else {
            mbar_arrive_expect_tx(bar, row_bytes);
            if (has_dx) bulk_load(dst, dxg + at * 4, fb, bar);
            if (has_dh) {
                bulk_load(dst + o_dh, dhg + at * 4, fb, bar);
                bulk_load(dst + o_x, xg + at * xs, xb, bar);
            }
            bulk_load(dst + o_y, yg + at * ys, yb, bar);
            if constexpr (kElem) bulk_load(dst + o_g, gg + at * ys, yb, bar);
        }
    };
    // byte offsets of row t's elements behind those of the arrays in a stage
    auto shift = [&](int64_t t, int size) -> uint32_t { return kOdd ? rn_shift((t * a.K + k0) * size) : 0u; };
    const int64_t t_first = static_cast<int64_t>(blockIdx.x / kCl) * RG + g;
    if (tid == 0)
        for (int s = 0; s < stages; ++s)
            if (t_first + s * step < a.T) issue(t_first + s * step, s);

    for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
        float f[E];
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = 1.0f;
        if (a.g_pre != nullptr) rn_load_gain<E>(a.g_pre, v0 + v, f);
        rn_gain_put<E>(g2_sm, v, nvec, f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = rn_col_w(a, k0 + E * v + e);
        rn_gain_put<E>(w_sm, v, nvec, f);
    }
    __syncthreads();

    float acc_pre[VPT][E], acc_s[VPT][E];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) acc_pre[j][e] = acc_s[j][e] = 0.0f;
    const float invK = 1.0f / static_cast<float>(a.K);

    uint32_t par = 0, xph = 0;
    bool apart = false;   // this thread's wait for the cluster ran out: it sends and arms nothing more
    auto reduce = [&](float2 v) -> float2 {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) rn_add2(v, o);
        if constexpr (kCl == 1) {
            if constexpr (TG == 32) {
                __syncwarp();
                return v;
            }
            if (lane == 0) red[g][par][tid >> 5] = v;
            rn_group_sync<TG>(g);
        } else {
            if (!apart) {
                if (threadIdx.x == 0) mbar_arrive_expect_tx(&xbar[par], kW * 8u);
                if (lane < kCl)
                    st_async_v2(mapa_shared(smem_u32(&red[0][par][rank * (TG / 32) + (tid >> 5)]), lane),
                                mapa_shared(smem_u32(&xbar[par]), lane), v);
                apart = !mbar_wait(&xbar[par], xph, wait_ns, &abort_flag);
            }
            __syncwarp();
        }
        v = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < (kW + 31) / 32; ++i) {
            const float2 w = red[g][par][(lane & (kW - 1)) + 32 * i];
            v.x += w.x;
            v.y += w.y;
        }
#pragma unroll
        for (int o = (kW < 32 ? kW : 32) / 2; o > 0; o >>= 1) rn_add2(v, o);
        if (par) xph ^= 1u;
        par ^= 1u;
        return v;
    };
    // this thread's part of sum_k g2 dh x, and the column sums of dh u2, of row t in stage s
    auto first_pass = [&](int64_t t, int s, float r2) -> float {
        const uint8_t* row = ring + static_cast<size_t>(s) * row_bytes;
        const uint8_t *dh_r = row + o_dh + shift(t, 4), *x_r = row + o_x + shift(t, xs);
        float c2 = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * TG;
            if (v >= nvec) continue;
            float dh[E], x[E], q[E];
            rn_lds<false, E>(dh_r, v, dh);
            rn_lds<kBf16X, E>(x_r, v, x);
            rn_gain<true, E>(g2_sm, v, nvec, q);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float z = dh[e] * x[e];
                c2 = fmaf(z, q[e], c2);
                acc_pre[j][e] = fmaf(z, r2, acc_pre[j][e]);
            }
        }
        return c2;
    };

    int s = 0;
    uint32_t ph = 0;
    float r2 = 0.0f, c2 = 0.0f;
    if (t_first < a.T && has_dh) {
        r2 = __ldg(a.r_pre + t_first);
        mbar_wait(&full[g][0], 0, wait_ns, &abort_flag);
        c2 = reduce(make_float2(0.0f, first_pass(t_first, 0, r2))).y * invK;
    }
    for (int64_t t = t_first; t < a.T; t += step) {
        const float r1 = a.post ? __ldg(a.r_post + t) : 1.0f;
        const float f = a.gate_kind == kGateToken ? __ldg(static_cast<const float*>(a.gate) + t) : 1.0f;
        const bool more = has_dh && t + step < a.T;
        const float r2n = more ? __ldg(a.r_pre + t + step) : 0.0f;
        if (!has_dh) mbar_wait(&full[g][s], ph, wait_ns, &abort_flag);
        const uint8_t* row = ring + static_cast<size_t>(s) * row_bytes;
        const uint8_t *dx_r = row + shift(t, 4), *dh_r = dx_r + o_dh, *x_r = row + o_x + shift(t, xs),
                      *y_r = row + o_y + shift(t, ys);
        const int64_t row0 = t * row_vecs + v0;
        const float b2 = -r2 * (r2 * c2);         // d = dx + r2 g2 dh + u2 b2 (r2^3 may leave fp32)
        float wd[VPT][E], u1[VPT][E];
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * TG;
            if (v >= nvec) continue;
            float d[E], w[E];
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = 0.0f;
            if (has_dx) rn_lds<false, E>(dx_r, v, d);
            if (has_dh) {
                float dh[E], x[E], g2[E];
                rn_lds<false, E>(dh_r, v, dh);
                rn_lds<kBf16X, E>(x_r, v, x);
                rn_gain<true, E>(g2_sm, v, nvec, g2);
#pragma unroll
                for (int e = 0; e < E; ++e) d[e] = fmaf(x[e] * r2, b2, fmaf(g2[e] * dh[e], r2, d[e]));
            }
            rn_lds<kBf16Y, E>(y_r, v, u1[j]);
            rn_gain<true, E>(w_sm, v, nvec, w);
            if constexpr (kElem) {
                float gt[E], dg[E];
                rn_lds<kBf16Y, E>(y_r + (o_g - o_y), v, gt);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    u1[j][e] *= r1;
                    const float q = d[e] * u1[j][e];
                    dg[e] = w[e] * q;
                    acc_s[j][e] = fmaf(gt[e], q, acc_s[j][e]);
                    wd[j][e] = gt[e] * (w[e] * d[e]);
                    sum.x = fmaf(gt[e], dg[e], sum.x);
                }
                if (a.dgate != nullptr) rn_store<kBf16Y, E>(a.dgate, row0 + v, dg);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    u1[j][e] *= r1;
                    const float q = d[e] * u1[j][e];
                    acc_s[j][e] = fmaf(f, q, acc_s[j][e]);
                    wd[j][e] = w[e] * d[e];
                    sum.x = fmaf(w[e], q, sum.x);
                }
            }
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] *= a.alpha;
            rn_store<false, E>(a.dX, row0 + v, d);
        }
        const int s_row = s;
        if (++s == stages) { s = 0; ph ^= 1u; }
        if (more) {
            mbar_wait(&full[g][s], ph, wait_ns, &abort_flag);
            sum.y = first_pass(t + step, s, r2n);
        }
        sum = reduce(sum);
        // every thread of the group has read the stage
        if (tid == 0 && t + stages * step < a.T) {
            if (abort_flag == 0) issue(t + stages * step, s_row);
            else flight[g].stop(t);
        }
        r2 = r2n;
        c2 = sum.y * invK;
        if (tid == 0 && rank == 0 && a.gate_kind == kGateToken && a.dgate != nullptr)
            static_cast<float*>(a.dgate)[t] = sum.x;
        const float c1 = -sum.x * invK, fr = f * r1;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * TG;
            if (v >= nvec) continue;
#pragma unroll
            for (int e = 0; e < E; ++e) wd[j][e] = fr * (a.post ? fmaf(u1[j][e], c1, wd[j][e]) : wd[j][e]);
            rn_store<kBf16Y, E>(a.dY, row0 + v, wd[j]);
        }
    }
    if (tid == 0 && abort_flag != 0) {
        // loads that had not landed when a wait ran out: let them (briefly) before the block ends
        flight[g].drain(stages, t_first, step, a.T,
                        [&](int q, uint32_t parity) { mbar_wait(&full[g][q], parity, 100000000ull, nullptr); });
    }
    __syncthreads();                              // every group is through its rows and its loads
    // (a load that never landed may still: nothing is written over the ring then)
    if (abort_flag == 0 && (a.part_pre != nullptr || a.part_s != nullptr || a.part_scalar != nullptr)) {
        float* sums = reinterpret_cast<float*>(rn_smem);   // [group][2][cols]
        float* mine = sums + static_cast<size_t>(g) * 2 * cols;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * TG;
            if (v >= nvec) continue;
            rn_gain_put<E>(mine, v, nvec, acc_pre[j]);
            rn_gain_put<E>(mine + cols, v, nvec, acc_s[j]);
        }
        __syncthreads();
        double scalar = 0.0;
        const int64_t out0 = static_cast<int64_t>(blockIdx.x / kCl) * a.K + k0;
        for (int i = threadIdx.x; i < 2 * nvec; i += blockDim.x) {
            const int which = i >= nvec, v = i - which * nvec;
            float tot[E];
            rn_gain<true, E>(sums + static_cast<size_t>(which) * cols, v, nvec, tot);
            for (int q = 1; q < RG; ++q) {
                float w[E];
                rn_gain<true, E>(sums + static_cast<size_t>(q * 2 + which) * cols, v, nvec, w);
#pragma unroll
                for (int e = 0; e < E; ++e) tot[e] += w[e];
            }
            float* part = which ? a.part_s : a.part_pre;
            if (part != nullptr) rn_store<false, E>(part + out0, v, tot);
            if (which && a.part_scalar != nullptr) {
                float q[E];
#pragma unroll
                for (int e = 0; e < E; ++e) q[e] = 1.0f;
                if (a.g_post != nullptr) rn_load_gain<E>(a.g_post, v0 + v, q);
#pragma unroll
                for (int e = 0; e < E; ++e) scalar += static_cast<double>(q[e] * tot[e]);
            }
        }
        if (a.part_scalar != nullptr) {
            scalar = warp_sum(scalar);
            if (lane == 0) red_s[threadIdx.x >> 5] = scalar;
            __syncthreads();
            if (threadIdx.x == 0) {
                double tot = 0.0;
                for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) tot += red_s[w];
                a.part_scalar[blockIdx.x] = tot;
            }
        }
    }
    if constexpr (kCl > 1) {
        __syncwarp();
        cluster_sync_all();                       // no block leaves while another may send to it
    }
}

// The column sums' partials [G x K], added in block order.  blockIdx.y = 0: dg2; 1: S, which gives
// dg1 = beta gate S and a channel gate's beta g1 S.  A block takes 32 columns with 32 warps (lane =
// column, warp w adds partial rows w, w + 32, ..., then warp 0 adds the warps).  A scalar gate's
// partials are added by the first block.
struct RnReduceArgs {
    const float* part_pre;
    const float* part_s;
    const double* part_scalar;
    const float* gate;     // channel or scalar gate, or NULL (the sums hold it)
    const float* g_post;
    float* dg_pre;
    float* dg_post;
    float* dgate;          // channel [K] or scalar [1], or NULL
    float beta;
    int gate_kind;
    int G, Gs, K;          // partial rows, scalar partials
};
__global__ void __launch_bounds__(1024) rn_reduce_kernel(const RnReduceArgs a) {
    __shared__ float red[32][33];
    pdl_trigger_and_wait();
    const int c = threadIdx.x & 31, w = threadIdx.x >> 5;
    if (blockIdx.y == 1 && blockIdx.x == 0 && a.part_scalar != nullptr && w == 0) {
        double s = 0.0;
        for (int p = c; p < a.Gs; p += 32) s += a.part_scalar[p];
        s = warp_sum(s);
        if (c == 0) *a.dgate = static_cast<float>(static_cast<double>(a.beta) * s);
    }
    const float* part = blockIdx.y ? a.part_s : a.part_pre;
    if (part == nullptr) return;
    const int k = blockIdx.x * 32 + c;
    float v[(kRnMaxBlocks + 31) / 32];
#pragma unroll
    for (int i = 0; i < (kRnMaxBlocks + 31) / 32; ++i) {
        const int p = w + 32 * i;
        v[i] = (k < a.K && p < a.G) ? __ldcs(part + static_cast<int64_t>(p) * a.K + k) : 0.0f;
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < (kRnMaxBlocks + 31) / 32; ++i) s += v[i];
    red[w][c] = s;
    __syncthreads();
    if (w != 0 || k >= a.K) return;
    float tot = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) tot += red[i][c];
    if (blockIdx.y == 0) {
        a.dg_pre[k] = tot;
        return;
    }
    tot *= a.beta;
    if (a.dg_post != nullptr)
        a.dg_post[k] = a.gate_kind == kGateChannel  ? tot * __ldg(a.gate + k)
                       : a.gate_kind == kGateScalar ? tot * __ldg(a.gate)
                                                    : tot;
    if (a.dgate != nullptr && a.gate_kind == kGateChannel)
        a.dgate[k] = a.g_post != nullptr ? tot * __ldg(a.g_post + k) : tot;
}

}  // namespace bl
