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
// Arithmetic of the forward (fixed, so that the 8-bit codes are reproducible): both sums of
// squares in fp64; every product and sum of an element in fp32 with one rounding each, in the
// order  fl(fl(y r1) g1), fl(n gate), fl(n beta), fl(fl(x alpha) + n);  x' rounded once to the
// residual's type, and h computed from the rounded x' (what the next layer reads).
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
    if constexpr (E == 8) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(g) + 2 * v);
        const float4 b = __ldg(reinterpret_cast<const float4*>(g) + 2 * v + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        f[0] = __ldg(g + v);
    }
}

// Round to the stored type (bf16: once, to nearest even); f becomes the stored values.
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
        else
            reinterpret_cast<uint16_t*>(p)[v] = static_cast<uint16_t>(h[0]);
    } else {
        if constexpr (E == 8) {
            reinterpret_cast<float4*>(p)[2 * v] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4*>(p)[2 * v + 1] = make_float4(f[4], f[5], f[6], f[7]);
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
    const double invK = static_cast<double>(a.K);

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

    // n = fl(fl(y r1) g1)
    if (a.post) {
        double ss = 0.0;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < E; ++e) ss = fma(static_cast<double>(y[j][e]), static_cast<double>(y[j][e]), ss);
        ss = rn_row_sum<kWarpRow, NT>(ss, red_y);
        const float r1 = static_cast<float>(1.0 / sqrt(ss / invK + static_cast<double>(a.eps_post)));
        if (tid == 0) a.r_post[t] = r1;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * TPR;
#pragma unroll
            for (int e = 0; e < E; ++e) y[j][e] = __fmul_rn(y[j][e], r1);
            if (a.g_post != nullptr && v < nvec) {
                float g[E];
                rn_load_gain<E>(a.g_post, v, g);
#pragma unroll
                for (int e = 0; e < E; ++e) y[j][e] = __fmul_rn(y[j][e], g[e]);
            }
        }
    }
    // x' = fl(fl(x alpha) + fl(fl(n gate) beta)), rounded to the residual's type and stored
    float gs = 1.0f;
    if (a.gate_kind == kGateScalar) gs = __ldg(static_cast<const float*>(a.gate));
    if (a.gate_kind == kGateToken) gs = __ldg(static_cast<const float*>(a.gate) + t);
    double ss = 0.0;
    float mx = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = tid + j * TPR;
        if (v >= nvec) continue;
        float g[E];
        if constexpr (kGateElem) {
#pragma unroll
            for (int e = 0; e < E; ++e) g[e] = ge[j][e];
        } else if (a.gate_kind == kGateChannel) {
            rn_load_gain<E>(static_cast<const float*>(a.gate), v, g);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) g[e] = gs;
        }
#pragma unroll
        for (int e = 0; e < E; ++e)
            x[j][e] = __fadd_rn(__fmul_rn(x[j][e], a.alpha), __fmul_rn(__fmul_rn(y[j][e], g[e]), a.beta));
        rn_store<kBf16X, E>(a.xout, row0 + v, x[j]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            mx = fmaxf(mx, fabsf(x[j][e]));
            ss = fma(static_cast<double>(x[j][e]), static_cast<double>(x[j][e]), ss);
        }
    }
    if (a.r_pre == nullptr) return;
    ss = rn_row_sum<kWarpRow, NT>(ss, red_x);
    const float r2 = static_cast<float>(1.0 / sqrt(ss / invK + static_cast<double>(a.eps_pre)));
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
