// weight_quant8.cuh -- 8-bit weight quantiser with one scale per output channel (weight row).
//
// The activation quantiser's rule (P3 §2.2: 127 / row absmax clamped at 1e-5, round half to
// even) applied to the rows of a latent weight, for the layers that a ternary model keeps in
// 8 bits (P4 / P5 "mixed 8-bit layers"):
//   m_n = max(max_k |W[n,k]|, 1e-5),  s_n = fl(127 / m_n),  gamma_n = fl(m_n / 127)
//   W_q[n,k] = rint(fl(W[n,k] s_n))   in [-127, 127]
// and the backward's operand W_q * bf16(gamma_n) in bf16.  A row is read twice, the second time
// out of L1 / L2; HBM-bound on one read of W and the outputs (11008 x 4096: 48.4 us for 316 MB, 6.5 TB/s;
// rows of 32768 leave L1 between the reads: 4096 x 32768 217 us for 940 MB).
#pragma once
#include "common.cuh"
#include "act_quant.cuh"

namespace bl {

constexpr int kW8Threads = 256;

// One block per row.  K % 32 == 0, rows 16-byte aligned.
__global__ void __launch_bounds__(kW8Threads) weight_quant8_kernel(const float* __restrict__ W, int N, int K,
                                                                   int8_t* __restrict__ Wq,
                                                                   uint16_t* __restrict__ Wbf,
                                                                   float* __restrict__ gamma_rows) {
    __shared__ float red[kW8Threads / 32];
    pdl_trigger_and_wait();
    const int nvec = K / 8;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * nvec;
    const float4* w4 = reinterpret_cast<const float4*>(W);
    float m = 0.0f;
    for (int v = threadIdx.x; v < nvec; v += kW8Threads) {
        const float4 a = __ldg(w4 + 2 * (row0 + v)), b = __ldg(w4 + 2 * (row0 + v) + 1);
        m = fmaxf(m, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))));
        m = fmaxf(m, fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))));
    }
    m = warp_max(m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int w = 1; w < kW8Threads / 32; ++w) m = fmaxf(m, red[w]);
    m = fmaxf(m, 1e-5f);
    const float s = __fdiv_rn(127.0f, m);
    const float gm = __fdiv_rn(m, 127.0f);
    if (threadIdx.x == 0) gamma_rows[blockIdx.x] = gm;
    const float gb = bf16_bits_to_float(float_to_bf16_bits(gm));
    for (int v = threadIdx.x; v < nvec; v += kW8Threads) {
        const float4 a = __ldg(w4 + 2 * (row0 + v)), b = __ldg(w4 + 2 * (row0 + v) + 1);
        const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t tb[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) tb[e] = quant_bits(f[e], s);
        if (Wq != nullptr)
            reinterpret_cast<uint2*>(Wq)[row0 + v] = make_uint2(gather_low_bytes(tb[0], tb[1], tb[2], tb[3]),
                                                                gather_low_bytes(tb[4], tb[5], tb[6], tb[7]));
        if (Wbf != nullptr) {
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = float_to_bf16_bits(__fmul_rn(__fsub_rn(__uint_as_float(tb[e]), kRoundMagic), gb));
            reinterpret_cast<uint4*>(Wbf)[row0 + v] = make_uint4(o[0] | (o[1] << 16), o[2] | (o[3] << 16),
                                                                 o[4] | (o[5] << 16), o[6] | (o[7] << 16));
        }
    }
}

}  // namespace bl
