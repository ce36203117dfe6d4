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
// Arithmetic of the forward (the same in both kernels, so that the 8-bit codes are reproducible):
// both sums of squares in fp64; every product and sum of an element in fp32 with one rounding each,
//   x' = fl( fl(x alpha) + fl( fl(y r1) w ) ),   w = fl( fl(gate beta) g1 )
// (w is the same for every row unless the gate is a token's or an element's); x' rounded once to
// the residual's type, and h = fl(fl(x' r2) g2) computed from the rounded x' (what the next layer
// reads).
#pragma once
#include "common.cuh"
#include "act_quant.cuh"

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
// is in shared memory: the status word tells), so that no barrier is left waiting.
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

// E adjacent elements out of shared memory, widened exactly.
template <bool kBf16, int E>
__device__ __forceinline__ void rn_lds(const uint8_t* row, int v, float (&f)[E]) {
    if constexpr (kBf16) {
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
    if constexpr (kSm) {
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
#pragma unroll
    for (int i = 0; i < E / 4; ++i)
        reinterpret_cast<float4*>(g)[i * nvec + v] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
}

// Forward for rows of whole vectors: thread i of a group owns vectors i + j * TG of E elements,
// EPT elements in all.  kSm:
// the weights w (for a gate that is the same in every row) and g2 are formed once per block in
// shared memory; the rows read them from there.
template <bool kBf16X, bool kBf16Y, int TG, int kMaxThreads, int EPT, bool kGateElem, bool kSm>
__global__ void __launch_bounds__(kMaxThreads, 1)
    residual_norm_ring_kernel(const RnFwdArgs a, int stages, uint64_t wait_ns) {
    constexpr int E = kBf16X ? 8 : 4;
    constexpr int VPT = EPT / E;
    constexpr int kRG = kMaxThreads / TG;
    extern __shared__ __align__(128) uint8_t rn_smem[];
    __shared__ uint64_t full[kRG][kRnMaxStages];
    __shared__ double red_y[kRG][2][TG / 32], red_x[kRG][2][TG / 32];
    __shared__ float red_m[kRG][2][TG / 32];
    __shared__ int abort_flag;
    const int g = threadIdx.x / TG, tid = threadIdx.x % TG;
    const int RG = blockDim.x / TG;
    if (threadIdx.x == 0) abort_flag = 0;
    if (tid == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&full[g][s], 1);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_trigger_and_wait();

    const int nvec = a.K / E;
    const uint32_t xb = a.K * (kBf16X ? 2u : 4u), yb = a.K * (kBf16Y ? 2u : 4u);
    const uint32_t row_bytes = xb + (kGateElem ? 2 * yb : yb);
    float* w_sm = reinterpret_cast<float*>(rn_smem);
    float* g_sm = w_sm + a.K;
    uint8_t* ring = rn_smem + (kSm ? static_cast<size_t>(a.K) * 8 : 0) + static_cast<size_t>(g) * stages * row_bytes;
    const int64_t step = static_cast<int64_t>(gridDim.x) * RG;
    const double invK = 1.0 / static_cast<double>(a.K);
    auto issue = [&](int64_t t, int s) {
        uint8_t* dst = ring + static_cast<size_t>(s) * row_bytes;
        mbar_arrive_expect_tx(&full[g][s], row_bytes);
        bulk_load(dst, static_cast<const uint8_t*>(a.x) + t * xb, xb, &full[g][s]);
        bulk_load(dst + xb, static_cast<const uint8_t*>(a.y) + t * yb, yb, &full[g][s]);
        if constexpr (kGateElem)
            bulk_load(dst + xb + yb, static_cast<const uint8_t*>(a.gate) + t * yb, yb, &full[g][s]);
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
        const uint8_t* xs = ring + static_cast<size_t>(s) * row_bytes;
        const uint8_t* ys = xs + xb;
        const int64_t row0 = t * nvec;
        float r1 = 1.0f;
        if (a.post) {
            double ss = 0.0;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = tid + j * TG;
                if (v >= nvec) continue;
                float y[E];
                rn_lds<kBf16Y, E>(ys, v, y);
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
            rn_lds<kBf16X, E>(xs, v, x[j]);
            rn_lds<kBf16Y, E>(ys, v, n);
            if constexpr (kSm) rn_gain<true, E>(w_sm, v, nvec, w);
            else col_weight(v, w);
            if constexpr (kGateElem) {
                float q[E];
                rn_lds<kBf16Y, E>(ys + yb, v, q);
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
        if (tid == 0 && t + stages * step < a.T) issue(t + stages * step, s);
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
        if (a.xq == nullptr) continue;
        // without a gain rounding is monotone: max |fl(x' r2)| = fl(max |x'| r2)
        if (a.g_pre == nullptr) m = __fmul_rn(mx, r2);
        m = rn_group_reduce<TG>(m, red_m[g][par], g, [](float p, float q) { return fmaxf(p, q); });
        const float sc = __fdiv_rn(127.0f, fmaxf(m, 1e-5f)), c = __frcp_rn(sc);
        if (tid == 0) a.sx[t] = sc;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * TG;
            if (v < nvec) rn_quant_store<kBf16Y, E>(x[j], sc, c, a.xq, a.xdq, row0 + v);
        }
    }
    if (tid == 0 && abort_flag != 0) {
        // loads that had not landed when the wait ran out: let them (briefly) before the block ends
        for (int q = 0; q < stages; ++q) {
            mbar_wait(&full[g][s], ph, 100000000ull, nullptr);
            if (++s == stages) { s = 0; ph ^= 1u; }
        }
    }
}

// ------------------------------------------------------------------------------------
// Backward.  With u1 = y r1, n = u1 g1 (n = y without the post norm), u2 = x' r2:
//   e  = g2 dh,  c2 = mean_k(e u2)
//   d  = dx' + r2 (e - u2 c2)          gradient of the new residual (dx' or dh may be absent)
//   dX = alpha d;   p = beta d
//   dgate = sum p n over what the gate was broadcast over
//   dn = p gate;  e1 = g1 dn,  c1 = mean_k(e1 u1);  dY = r1 (e1 - u1 c1)   (dY = dn without)
//   dg2 = sum_t dh u2,   dg1 = sum_t dn u1
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
    void* dgate;          // token: fp32 [T]; element: [T x K] y's type (channel / scalar: through the partials)
    float* part_pre;      // [G x K] partial sums of dg2, or NULL
    float* part_post;     // [G x K] of dg1, or NULL
    float* part_gate;     // [G x K] of the channel gate's gradient, or NULL
    double* part_scalar;  // [G] of the scalar gate's gradient, or NULL
    int T, K;
    int post, gate_kind;
    float alpha, beta;
};

constexpr int kRnMaxBlocks = 148;   // partial rows: three gains' partials fit the RMSNorm backward's workspace

template <int NT>
__device__ __forceinline__ void rn_block_sum2(float& a, float& b, float (*red)[NT / 32]) {
    a = warp_sum(a);
    b = warp_sum(b);
    if ((threadIdx.x & 31) == 0) {
        red[0][threadIdx.x >> 5] = a;
        red[1][threadIdx.x >> 5] = b;
    }
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        a += red[0][w];
        b += red[1][w];
    }
}

// Any row length: the row is walked three times (the second and third time out of L2), and the
// column sums sit in shared memory, each element owned by one thread.  Block b takes rows b,
// b + G, ...; the reductions' order is fixed.
template <bool kBf16X, bool kBf16Y, int E, int NT>
__global__ void __launch_bounds__(NT) residual_norm_bwd_walk_kernel(const RnBwdArgs a) {
    extern __shared__ float acc[];               // [3][K]: dg2, dg1, channel gate
    __shared__ float red[2][2][NT / 32];
    __shared__ double red_s[NT / 32];
    pdl_trigger_and_wait();
    float* acc_pre = acc;
    float* acc_post = acc + a.K;
    float* acc_gate = acc + 2 * static_cast<int64_t>(a.K);
    const int nvec = a.K / E;
    const float K = static_cast<float>(a.K);
    for (int i = threadIdx.x; i < 3 * nvec; i += NT)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[i * E + e] = 0.0f;
    __syncthreads();
    double scalar = 0.0;

    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t row0 = static_cast<int64_t>(t) * nvec;
        const float r2 = a.dh != nullptr ? __ldg(a.r_pre + t) : 0.0f;
        const float r1 = a.post ? __ldg(a.r_post + t) : 1.0f;
        float gs = 1.0f;
        if (a.gate_kind == kGateScalar) gs = __ldg(static_cast<const float*>(a.gate));
        if (a.gate_kind == kGateToken) gs = __ldg(static_cast<const float*>(a.gate) + t);
        float c2 = 0.0f, c1 = 0.0f, tok = 0.0f;
        if (a.dh != nullptr) {
            float unused = 0.0f;
            for (int v = threadIdx.x; v < nvec; v += NT) {
                float dh[E], x[E], g[E];
                rn_load<false, E>(a.dh, row0 + v, dh);
                rn_load<kBf16X, E>(a.x, row0 + v, x);
#pragma unroll
                for (int e = 0; e < E; ++e) g[e] = 1.0f;
                if (a.g_pre != nullptr) rn_load_gain<E>(a.g_pre, v, g);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float u = x[e] * r2;
                    c2 = fmaf(g[e] * dh[e], u, c2);
                    if (a.part_pre != nullptr) acc_pre[v * E + e] = fmaf(dh[e], u, acc_pre[v * E + e]);
                }
            }
            rn_block_sum2<NT>(c2, unused, red[0]);
            c2 /= K;
        }
        // the gradient d of the new residual at vector v, and what follows from it: n, dn
        auto at = [&](int v, float (&d)[E], float (&u1)[E], float (&n)[E], float (&dn)[E]) {
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = 0.0f;
            if (a.dx != nullptr) rn_load<false, E>(a.dx, row0 + v, d);
            if (a.dh != nullptr) {
                float dh[E], x[E], g[E];
                rn_load<false, E>(a.dh, row0 + v, dh);
                rn_load<kBf16X, E>(a.x, row0 + v, x);
#pragma unroll
                for (int e = 0; e < E; ++e) g[e] = 1.0f;
                if (a.g_pre != nullptr) rn_load_gain<E>(a.g_pre, v, g);
#pragma unroll
                for (int e = 0; e < E; ++e) d[e] += r2 * (g[e] * dh[e] - x[e] * r2 * c2);
            }
            float g[E];
            rn_load<kBf16Y, E>(a.y, row0 + v, u1);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (a.post) u1[e] *= r1;
                n[e] = u1[e];
            }
            if (a.g_post != nullptr) {
                rn_load_gain<E>(a.g_post, v, g);
#pragma unroll
                for (int e = 0; e < E; ++e) n[e] *= g[e];
            }
#pragma unroll
            for (int e = 0; e < E; ++e) g[e] = gs;
            if (a.gate_kind == kGateChannel) rn_load_gain<E>(static_cast<const float*>(a.gate), v, g);
            if (a.gate_kind == kGateElement) rn_load<kBf16Y, E>(a.gate, row0 + v, g);
#pragma unroll
            for (int e = 0; e < E; ++e) dn[e] = a.beta * d[e] * g[e];
        };
        if (a.post || a.gate_kind != kGateNone) {
            for (int v = threadIdx.x; v < nvec; v += NT) {
                float d[E], u1[E], n[E], dn[E], g[E];
                at(v, d, u1, n, dn);
#pragma unroll
                for (int e = 0; e < E; ++e) g[e] = 1.0f;
                if (a.g_post != nullptr) rn_load_gain<E>(a.g_post, v, g);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float pn = a.beta * d[e] * n[e];
                    tok += pn;
                    if (a.part_gate != nullptr) acc_gate[v * E + e] += pn;
                    c1 = fmaf(g[e] * dn[e], u1[e], c1);
                    if (a.part_post != nullptr) acc_post[v * E + e] = fmaf(dn[e], u1[e], acc_post[v * E + e]);
                }
            }
            scalar += static_cast<double>(tok);
            rn_block_sum2<NT>(c1, tok, red[1]);
            c1 /= K;
            if (a.gate_kind == kGateToken && a.dgate != nullptr && threadIdx.x == 0)
                static_cast<float*>(a.dgate)[t] = tok;
        }
        for (int v = threadIdx.x; v < nvec; v += NT) {
            float d[E], u1[E], n[E], dn[E], g[E];
            at(v, d, u1, n, dn);
#pragma unroll
            for (int e = 0; e < E; ++e) g[e] = 1.0f;
            if (a.g_post != nullptr) rn_load_gain<E>(a.g_post, v, g);
            if (a.gate_kind == kGateElement && a.dgate != nullptr) {
#pragma unroll
                for (int e = 0; e < E; ++e) n[e] *= a.beta * d[e];
                rn_store<kBf16Y, E>(a.dgate, row0 + v, n);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                d[e] *= a.alpha;
                if (a.post) dn[e] = r1 * (g[e] * dn[e] - u1[e] * c1);
            }
            rn_store<false, E>(a.dX, row0 + v, d);
            rn_store<kBf16Y, E>(a.dY, row0 + v, dn);
        }
        __syncthreads();                          // the sums in red[] are read before the next row's
    }
    for (int v = threadIdx.x; v < nvec; v += NT)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int64_t k = static_cast<int64_t>(v) * E + e, o = static_cast<int64_t>(blockIdx.x) * a.K + k;
            if (a.part_pre != nullptr) a.part_pre[o] = acc_pre[k];
            if (a.part_post != nullptr) a.part_post[o] = acc_post[k];
            if (a.part_gate != nullptr) a.part_gate[o] = acc_gate[k];
        }
    if (a.part_scalar != nullptr) {
        const double s = warp_sum(scalar);
        if ((threadIdx.x & 31) == 0) red_s[threadIdx.x >> 5] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            double tot = 0.0;
            for (int w = 0; w < NT / 32; ++w) tot += red_s[w];
            a.part_scalar[blockIdx.x] = tot;
        }
    }
}

// The same through a ring of rows (see the forward): thread i of a group owns vectors of four
// columns i + j * TG, j < EPT / 4, of every row its group takes, and keeps their column sums in
// registers.  A row is read from shared memory twice (c2 first, then everything else); what the
// last pass needs, e1 (dn without the post norm) and u1, stays in registers, so the stage is
// refilled before it.  At the end the groups' sums are joined in shared memory in group order and
// the block writes one partial row for each.
template <bool kBf16X, bool kBf16Y, int TG, int kMaxThreads, int EPT, bool kSm>
__global__ void __launch_bounds__(kMaxThreads, 1)
    residual_norm_bwd_ring_kernel(const RnBwdArgs a, int stages, uint64_t wait_ns) {
    constexpr int VPT = EPT / 4;
    constexpr int kRG = kMaxThreads / TG;
    extern __shared__ __align__(128) uint8_t rn_smem[];
    __shared__ uint64_t full[kRG][kRnMaxStages];
    __shared__ float red_2[kRG][2][TG / 32], red_1[kRG][2][TG / 32], red_t[kRG][2][TG / 32];
    __shared__ double red_s[kMaxThreads / 32];
    __shared__ int abort_flag;
    const int g = threadIdx.x / TG, tid = threadIdx.x % TG;
    const int RG = blockDim.x / TG;
    if (threadIdx.x == 0) abort_flag = 0;
    if (tid == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&full[g][s], 1);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_trigger_and_wait();

    const int nvec = a.K / 4;
    const bool has_dx = a.dx != nullptr, has_dh = a.dh != nullptr, elem = a.gate_kind == kGateElement;
    // a row's arrays in its stage: dx, dh, x, y, gate
    const uint32_t fb = a.K * 4u, xb = a.K * (kBf16X ? 2u : 4u), yb = a.K * (kBf16Y ? 2u : 4u);
    const uint32_t o_dh = has_dx ? fb : 0u, o_x = o_dh + (has_dh ? fb : 0u), o_y = o_x + (has_dh ? xb : 0u), o_g = o_y + yb;
    const uint32_t row_bytes = o_g + (elem ? yb : 0u);
    float* g2_sm = reinterpret_cast<float*>(rn_smem);
    float* g1_sm = g2_sm + a.K;
    float* gt_sm = g1_sm + a.K;
    uint8_t* ring = rn_smem + (kSm ? static_cast<size_t>(a.K) * 12 : 0) + static_cast<size_t>(g) * stages * row_bytes;
    const int64_t step = static_cast<int64_t>(gridDim.x) * RG;
    auto issue = [&](int64_t t, int s) {
        uint8_t* dst = ring + static_cast<size_t>(s) * row_bytes;
        uint64_t* bar = &full[g][s];
        mbar_arrive_expect_tx(bar, row_bytes);
        if (has_dx) bulk_load(dst, reinterpret_cast<const uint8_t*>(a.dx) + t * fb, fb, bar);
        if (has_dh) {
            bulk_load(dst + o_dh, reinterpret_cast<const uint8_t*>(a.dh) + t * fb, fb, bar);
            bulk_load(dst + o_x, static_cast<const uint8_t*>(a.x) + t * xb, xb, bar);
        }
        bulk_load(dst + o_y, static_cast<const uint8_t*>(a.y) + t * yb, yb, bar);
        if (elem) bulk_load(dst + o_g, static_cast<const uint8_t*>(a.gate) + t * yb, yb, bar);
    };
    const int64_t t_first = static_cast<int64_t>(blockIdx.x) * RG + g;
    if (tid == 0)
        for (int s = 0; s < stages; ++s)
            if (t_first + s * step < a.T) issue(t_first + s * step, s);

    auto ones = [](float (&f)[4]) { f[0] = f[1] = f[2] = f[3] = 1.0f; };
    if constexpr (kSm) {
        for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
            float f[4];
            ones(f);
            if (a.g_pre != nullptr) rn_load_gain<4>(a.g_pre, v, f);
            rn_gain_put<4>(g2_sm, v, nvec, f);
            ones(f);
            if (a.g_post != nullptr) rn_load_gain<4>(a.g_post, v, f);
            rn_gain_put<4>(g1_sm, v, nvec, f);
            ones(f);
            if (a.gate_kind == kGateChannel) rn_load_gain<4>(static_cast<const float*>(a.gate), v, f);
            rn_gain_put<4>(gt_sm, v, nvec, f);
        }
        __syncthreads();
    }
    auto gain = [&](const float* sm, const float* gm, bool have, int v, float (&f)[4]) {
        if constexpr (kSm) {
            rn_gain<true, 4>(sm, v, nvec, f);
        } else {
            ones(f);
            if (have) rn_load_gain<4>(gm, v, f);
        }
    };

    float acc_pre[VPT][4], acc_post[VPT][4], acc_gate[VPT][4];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc_pre[j][e] = acc_post[j][e] = acc_gate[j][e] = 0.0f;
    const float invK = 1.0f / static_cast<float>(a.K);
    const bool want_tok = a.gate_kind == kGateToken && a.dgate != nullptr;
    double scalar = 0.0;
    float gs = 1.0f;
    if (a.gate_kind == kGateScalar) gs = __ldg(static_cast<const float*>(a.gate));

    int s = 0;
    uint32_t ph = 0, par = 0;
    for (int64_t t = t_first; t < a.T; t += step, par ^= 1u) {
        const float r2 = has_dh ? __ldg(a.r_pre + t) : 0.0f;
        const float r1 = a.post ? __ldg(a.r_post + t) : 1.0f;
        if (a.gate_kind == kGateToken) gs = __ldg(static_cast<const float*>(a.gate) + t);
        mbar_wait(&full[g][s], ph, wait_ns, &abort_flag);
        const uint8_t* row = ring + static_cast<size_t>(s) * row_bytes;
        const int64_t row0 = t * nvec;
        float c2 = 0.0f;
        if (has_dh) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = tid + j * TG;
                if (v >= nvec) continue;
                float dh[4], x[4], q[4];
                rn_lds<false, 4>(row + o_dh, v, dh);
                rn_lds<kBf16X, 4>(row + o_x, v, x);
                gain(g2_sm, a.g_pre, a.g_pre != nullptr, v, q);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float u = x[e] * r2;
                    c2 = fmaf(q[e] * dh[e], u, c2);
                    acc_pre[j][e] = fmaf(dh[e], u, acc_pre[j][e]);
                }
            }
            c2 = rn_group_reduce<TG>(c2, red_2[g][par], g, [](float p, float q) { return p + q; }) * invK;
        }
        const float b2 = -r2 * c2;                // d = dx + r2 (e - u2 c2)
        float e1[VPT][4], u1[VPT][4];
        float c1 = 0.0f, tok = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * TG;
            if (v >= nvec) continue;
            float d[4], q[4], gt[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = 0.0f;
            if (has_dx) rn_lds<false, 4>(row, v, d);
            if (has_dh) {
                float dh[4], x[4];
                rn_lds<false, 4>(row + o_dh, v, dh);
                rn_lds<kBf16X, 4>(row + o_x, v, x);
                gain(g2_sm, a.g_pre, a.g_pre != nullptr, v, q);
#pragma unroll
                for (int e = 0; e < 4; ++e) d[e] = fmaf(r2, fmaf(x[e], b2, q[e] * dh[e]), d[e]);
            }
            rn_lds<kBf16Y, 4>(row + o_y, v, u1[j]);
            gain(g1_sm, a.g_post, a.g_post != nullptr, v, q);
            if (elem) {
                rn_lds<kBf16Y, 4>(row + o_g, v, gt);
            } else if (a.gate_kind == kGateChannel) {
                gain(gt_sm, static_cast<const float*>(a.gate), true, v, gt);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) gt[e] = gs;
            }
            float dg[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                u1[j][e] *= r1;
                const float p = a.beta * d[e];
                dg[e] = p * (u1[j][e] * q[e]);
                tok += dg[e];
                acc_gate[j][e] += dg[e];
                const float dn = p * gt[e];
                acc_post[j][e] = fmaf(dn, u1[j][e], acc_post[j][e]);
                e1[j][e] = q[e] * dn;
                c1 = fmaf(e1[j][e], u1[j][e], c1);
                d[e] *= a.alpha;
            }
            rn_store<false, 4>(a.dX, row0 + v, d);
            if (elem && a.dgate != nullptr) rn_store<kBf16Y, 4>(a.dgate, row0 + v, dg);
        }
        scalar += static_cast<double>(tok);
        if (a.post) c1 = rn_group_reduce<TG>(c1, red_1[g][par], g, [](float p, float q) { return p + q; }) * invK;
        if (want_tok) {
            tok = rn_group_reduce<TG>(tok, red_t[g][par], g, [](float p, float q) { return p + q; });
            if (tid == 0) static_cast<float*>(a.dgate)[t] = tok;
        }
        if (TG == 32 || (!a.post && !want_tok)) rn_group_sync<TG>(g);
        // every thread of the group has read the stage
        if (tid == 0 && t + stages * step < a.T) issue(t + stages * step, s);
        if (++s == stages) { s = 0; ph ^= 1u; }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * TG;
            if (v >= nvec) continue;
            if (a.post) {
#pragma unroll
                for (int e = 0; e < 4; ++e) e1[j][e] = r1 * fmaf(-u1[j][e], c1, e1[j][e]);
            }
            rn_store<kBf16Y, 4>(a.dY, row0 + v, e1[j]);
        }
    }
    if (tid == 0 && abort_flag != 0) {
        // loads that had not landed when the wait ran out: let them (briefly) before the block ends
        for (int q = 0; q < stages; ++q) {
            mbar_wait(&full[g][s], ph, 100000000ull, nullptr);
            if (++s == stages) { s = 0; ph ^= 1u; }
        }
    }
    if (a.part_scalar != nullptr) {
        const double w = warp_sum(scalar);
        if ((threadIdx.x & 31) == 0) red_s[threadIdx.x >> 5] = w;
    }
    __syncthreads();                              // every group is through its rows and its loads
    if (a.part_scalar != nullptr && threadIdx.x == 0) {
        double tot = 0.0;
        for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) tot += red_s[w];
        a.part_scalar[blockIdx.x] = tot;
    }
    if (a.part_pre == nullptr && a.part_post == nullptr && a.part_gate == nullptr) return;
    float* sums = reinterpret_cast<float*>(rn_smem);   // [group][3][K]
    float* mine = sums + static_cast<size_t>(g) * 3 * a.K;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = tid + j * TG;
        if (v >= nvec) continue;
        rn_gain_put<4>(mine, v, nvec, acc_pre[j]);
        rn_gain_put<4>(mine + a.K, v, nvec, acc_post[j]);
        rn_gain_put<4>(mine + 2 * a.K, v, nvec, acc_gate[j]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 3 * nvec; i += blockDim.x) {
        const int which = i / nvec, v = i - which * nvec;
        float* part = which == 0 ? a.part_pre : which == 1 ? a.part_post : a.part_gate;
        if (part == nullptr) continue;
        float4 tot = reinterpret_cast<const float4*>(sums + static_cast<size_t>(which) * a.K)[v];
        for (int q = 1; q < RG; ++q) {
            const float4 w = reinterpret_cast<const float4*>(sums + static_cast<size_t>(q * 3 + which) * a.K)[v];
            tot.x += w.x; tot.y += w.y; tot.z += w.z; tot.w += w.w;
        }
        reinterpret_cast<float4*>(part + static_cast<int64_t>(blockIdx.x) * a.K)[v] = tot;
    }
}

// The column sums' partials [G x K], added in block order: blockIdx.y picks the gradient
// (dg2, dg1, channel gate), a block takes 32 columns with 32 warps (lane = column, warp w adds
// partial rows w, w + 32, ..., then warp 0 adds the warps).  The scalar gate's partials are
// added by the first block of the third.
struct RnReduceArgs {
    const float* part[3];
    float* out[3];
    const double* part_scalar;
    float* dscalar;
    int G, K;
};
__global__ void __launch_bounds__(1024) rn_reduce_kernel(const RnReduceArgs a) {
    __shared__ float red[32][33];
    pdl_trigger_and_wait();
    const int c = threadIdx.x & 31, w = threadIdx.x >> 5;
    if (blockIdx.y == 2 && blockIdx.x == 0 && a.part_scalar != nullptr && w == 0) {
        double s = 0.0;
        for (int p = c; p < a.G; p += 32) s += a.part_scalar[p];
        s = warp_sum(s);
        if (c == 0) *a.dscalar = static_cast<float>(s);
    }
    const float* part = a.part[blockIdx.y];
    if (part == nullptr) return;
    const int k = blockIdx.x * 32 + c;
    float s = 0.0f;
    for (int p = w; p < a.G; p += 32) s += k < a.K ? __ldcs(part + static_cast<int64_t>(p) * a.K + k) : 0.0f;
    red[w][c] = s;
    __syncthreads();
    if (w == 0 && k < a.K) {
        float tot = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) tot += red[i][c];
        a.out[blockIdx.y][k] = tot;
    }
}

}  // namespace bl
