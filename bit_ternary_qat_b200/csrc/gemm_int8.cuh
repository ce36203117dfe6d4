// gemm_int8.cuh -- the 8-bit linear for few tokens (single decoded tokens to a few hundred).
//
//   acc[t, n] = sum_k X_q[t, k] W_q[n, k]       y = fl( fl(acc gamma_n) r_t ),  r_t = fl(1 / s_t)
//
// With few tokens the product reads the weight once and is bound by HBM, so the tiles are cut
// for the read, not for the tensor core: the weight rows are the M side of tcgen05.mma (kind::i8,
// M = 128) and the tokens, rounded up to 16, its N side.  A tile has R <= 128 weight rows, any
// number: the TMA box loads R rows of each 128-byte k-block and the MMA's other rows multiply
// whatever lies behind them in shared memory into accumulators that nobody reads.  R is chosen so
// that the tiles divide evenly over the SMs (28672 rows: 296 tiles of 97 rows, two per SM).  When
// the rows alone give too few bytes per token-side byte, K is split over the CTAs of a cluster
// and the int32 partial sums are added through distributed shared memory (whole numbers: any
// order gives the same sum).  No workspace, one launch.
//
// Roles as in gemm_tc.cuh: warp 0 TMA producer, warp 1 MMA issuer, warps 2..9 epilogue (two to a
// quadrant of TMEM lanes, taking 16 tokens in turn: with few rows a tile only some quadrants hold
// rows, and with 256 tokens an epilogue of four warps that divided by s_t took longer than the
// loads: 11008 x 4096, 41 us, 14 without it, 21 as it is).  Every mbarrier wait is bounded, and a
// block that gives up still reaches the cluster barriers.
#pragma once
#include <cuda.h>
#include "common.cuh"

namespace bl {

constexpr int kI8Threads = 320;
constexpr int kI8MaxStages = 24;
constexpr int kI8MaxTokens = 256;      // token side of one tile

struct I8Args {
    int T, N, K;
    int rows;          // R: weight rows per tile
    int bt;            // token tile (multiple of 16)
    int n_tiles, t_tiles;
    int k_steps;       // stages' worth of K
    int stages;
    int bufs;          // tiles whose accumulators fit TMEM at once: 1 or 2
    int a_pitch;       // bytes of a k-block's weight slot (multiple of 1024)
    int splits;        // cluster size along K
    const float* sx;
    const float* gamma;
    void* y;
    int32_t* acc;
    uint64_t wait_ns;
};

// Shared memory behind the 1024-byte aligned start: weight slots, token slots, barriers.  The
// MMA reads 128 rows from each weight slot's start, so 16 KB must be readable behind the last.
__host__ __device__ inline size_t i8_ring_bytes(int stages, int kpb, int a_pitch, int bt) {
    const size_t a = (size_t)stages * kpb * a_pitch, b = (size_t)stages * kpb * bt * 128;
    const size_t need = (size_t)(stages * kpb - 1) * a_pitch + 16384;
    return a + b < need ? need : a + b;
}
__host__ __device__ inline size_t i8_smem_bytes(int stages, int kpb, int a_pitch, int bt) {
    return 1024 + i8_ring_bytes(stages, kpb, a_pitch, bt) + (2 * kI8MaxStages + 4) * sizeof(uint64_t) + 16;
}

// 16 consecutive columns of 32 TMEM lanes.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ int4 ld_cluster_v4(uint32_t addr) {
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

template <bool kBf16Out>
__device__ __forceinline__ void i8_store(const I8Args& a, int64_t o, int32_t acc, float gm, float r) {
    const float v = __fmul_rn(__fmul_rn(static_cast<float>(acc), gm), r);
    if constexpr (kBf16Out) static_cast<uint16_t*>(a.y)[o] = float_to_bf16_bits(v);
    else static_cast<float*>(a.y)[o] = v;
    if (a.acc != nullptr) a.acc[o] = acc;
}

// kpb: k-blocks of 128 bytes in a stage.  A stage costs its waits, its expect and its commit (about
// 300 cycles, whatever it carries), so it carries as many as leave four stages; fixed at compile time,
// since the two issuing threads' own instructions are what counts (2048 x 16384, one token, without a
// K split: 24.7 us with 1, 17.5 with 2; 23.3 with 2 when the loops take it from the arguments).
template <bool kBf16Out, int kpb>
__global__ void __launch_bounds__(kI8Threads, 1)
    gemm_int8_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                         const I8Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align1024(smem_raw);
    uint8_t* sA = smem;
    uint8_t* sB = smem + static_cast<size_t>(a.stages) * kpb * a.a_pitch;
    const uint32_t a_stage = static_cast<uint32_t>(kpb * a.a_pitch), b_kb = static_cast<uint32_t>(a.bt) * 128u,
                   b_stage = kpb * b_kb;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + i8_ring_bytes(a.stages, kpb, a.a_pitch, a.bt));
    uint64_t* empty = full + kI8MaxStages;
    uint64_t* tfull = empty + kI8MaxStages;
    uint64_t* tempty = tfull + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    uint32_t tmem_cols = 32;
    while (tmem_cols < static_cast<uint32_t>(a.bt * a.bufs)) tmem_cols *= 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 8);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_trigger_and_wait();

    const uint64_t lim = a.wait_ns;
    const int rank = a.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int unit0 = blockIdx.x / a.splits, units = gridDim.x / a.splits;
    const int tiles = a.n_tiles * a.t_tiles;
    const int kb0 = static_cast<int>(static_cast<int64_t>(a.k_steps) * rank / a.splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(a.k_steps) * (rank + 1) / a.splits);
    const uint32_t stage_tx = static_cast<uint32_t>(a.rows + a.bt) * (128u * kpb);

    if (warp == 0) {
        // ----------------------------------------------------------------- producer
        if (elect_one()) {
            int s = 0;
            uint32_t ph = 0;
            int posted = 0;
            bool ok = true;
            for (int tile = unit0; tile < tiles && ok; tile += units) {
                const int n0 = (tile / a.t_tiles) * a.rows, t0 = (tile % a.t_tiles) * a.bt;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(&empty[s], ph ^ 1u, lim, abort_flag)) { ok = false; break; }
                    mbar_arrive_expect_tx(&full[s], stage_tx);
#pragma unroll
                    for (int q = 0; q < kpb; ++q) {   // past the end of K the boxes are filled with zeros
                        tma_load_2d(sA + s * a_stage + q * a.a_pitch, &tmW, &full[s], (kb * kpb + q) * 128, n0);
                        tma_load_2d(sB + s * b_stage + q * b_kb, &tmX, &full[s], (kb * kpb + q) * 128, t0);
                    }
                    ++posted;
                    if (++s == a.stages) { s = 0; ph ^= 1u; }
                }
            }
            if (!ok) {
                // wait (briefly) for the loads that are still on their way
                for (int i = 0; i < a.stages && i < posted; ++i) {
                    if (--s < 0) { s = a.stages - 1; ph ^= 1u; }
                    mbar_wait(&full[s], ph, 100000000ull, nullptr);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ----------------------------------------------------------------- MMA issuer
        if (elect_one()) {
            const uint32_t idesc = umma_idesc(true, false, false, 128, a.bt);
            int s = 0;
            uint32_t ph = 0;
            int tcount = 0;
            bool ok = true;
            for (int tile = unit0; tile < tiles && ok; tile += units, ++tcount) {
                const int b = a.bufs == 2 ? tcount & 1 : 0;
                const uint32_t tph = static_cast<uint32_t>(a.bufs == 2 ? tcount >> 1 : tcount) & 1u;
                if (!mbar_wait(&tempty[b], tph ^ 1u, lim, abort_flag)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(b * a.bt);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(&full[s], ph, lim, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a_base = smem_u32(sA) + s * a_stage, b_base = smem_u32(sB) + s * b_stage;
#pragma unroll
                    for (int q = 0; q < kpb; ++q) {
                        const uint64_t ad = umma_desc_sw128(a_base + q * a.a_pitch, 16, 1024),
                                       bd = umma_desc_sw128(b_base + q * b_kb, 16, 1024);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)      // 32 bytes of K: 2 in the descriptors' address fields
                            tc_mma<true>(d_tmem, ad + 2 * kk, bd + 2 * kk, idesc,
                                         (kb != kb0 || q != 0 || kk != 0) ? 1u : 0u);
                    }
                    tc_commit(&empty[s]);
                    if (++s == a.stages) { s = 0; ph ^= 1u; }
                }
                if (!ok) break;
                tc_commit(&tfull[b]);
            }
            if (!ok) {
                const int b = a.bufs == 2 ? tcount & 1 : 0;
                tc_commit(&tfull[b]);
                mbar_wait(&tfull[b], static_cast<uint32_t>(a.bufs == 2 ? tcount >> 1 : tcount) & 1u, 100000000ull,
                          nullptr);
            }
        }
        __syncwarp();
    } else {
        // ----------------------------------------------------------------- epilogue
        const int quad = warp & 3;              // TMEM lanes [32 quad, 32 quad + 32): weight rows
        const int half = (warp - 2) >> 2;       // 16-token chunks half, half + 2, ...
        const int r = quad * 32 + lane;
        int tcount = 0;
        for (int tile = unit0; tile < tiles; tile += units, ++tcount) {
            const int b = a.bufs == 2 ? tcount & 1 : 0;
            const uint32_t tph = static_cast<uint32_t>(a.bufs == 2 ? tcount >> 1 : tcount) & 1u;
            if (!mbar_wait_warp(&tfull[b], tph, lim, abort_flag)) break;
            tc_fence_after();
            const int n0 = (tile / a.t_tiles) * a.rows, t0 = (tile % a.t_tiles) * a.bt;
            const int n = n0 + r;
            const bool live = r < a.rows && n < a.N;
            const int tend = min(a.bt, a.T - t0);
            const float gm = a.splits == 1 && live ? __ldg(a.gamma + n) : 0.0f;
            const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) +
                                   static_cast<uint32_t>(b * a.bt);
            if (quad * 32 < a.rows) {
                for (int c0 = half * 16; c0 < tend; c0 += 32) {
                    uint32_t v[16];
                    float rt[16];
                    __syncwarp();
                    tmem_ld_32x32b_x16(t_row + c0, v);
                    if (a.splits == 1) {
                        // 1 / s_t of the chunk's tokens: a lane computes one, the warp reads all
                        const float mine = c0 + (lane & 15) < tend ? __frcp_rn(__ldg(a.sx + t0 + c0 + (lane & 15))) : 0.0f;
#pragma unroll
                        for (int i = 0; i < 16; ++i) rt[i] = __shfl_sync(0xffffffffu, mine, i);
                    }
                    tmem_ld_wait();
                    if (a.splits == 1) {
                        const int64_t o = static_cast<int64_t>(t0 + c0) * a.N + n;
                        if (live) {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (c0 + i < tend)
                                    i8_store<kBf16Out>(a, o + static_cast<int64_t>(i) * a.N, static_cast<int32_t>(v[i]),
                                                       gm, rt[i]);
                        }
                    } else {
                        // this CTA's partial sums [token][row], over the ring: every load has been
                        // consumed once the tile's last MMA is done, and with a split a CTA has one tile
                        int32_t* part = reinterpret_cast<int32_t*>(smem);
#pragma unroll
                        for (int i = 0; i < 16; ++i) part[(c0 + i) * 128 + r] = static_cast<int32_t>(v[i]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[b]);
        }
    }

    if (a.splits > 1) {
        __syncwarp();
        cluster_sync_all();                     // every CTA's partial sums are in its shared memory
        const int n0 = (unit0 / a.t_tiles) * a.rows, t0 = (unit0 % a.t_tiles) * a.bt;
        const int tend = min(a.bt, a.T - t0);
        if (*abort_flag == 0) {
            // token t is joined by rank t % splits: a warp takes a token, a lane four rows
            const uint32_t part = smem_u32(smem);
            for (int c = rank + a.splits * warp; c < tend; c += a.splits * (kI8Threads / 32)) {
                const uint32_t off = part + static_cast<uint32_t>(c * 128 + lane * 4) * 4u;
                int4 v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q < a.splits) v[q] = ld_cluster_v4(mapa_shared(off, static_cast<uint32_t>(q)));
                int4 sum = make_int4(0, 0, 0, 0);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q < a.splits) {
                        sum.x += v[q].x; sum.y += v[q].y; sum.z += v[q].z; sum.w += v[q].w;
                    }
                const float rt = __frcp_rn(__ldg(a.sx + t0 + c));
                const int64_t o = static_cast<int64_t>(t0 + c) * a.N + n0 + lane * 4;
                const int32_t e[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = lane * 4 + i;
                    if (r < a.rows && n0 + r < a.N) i8_store<kBf16Out>(a, o + i, e[i], __ldg(a.gamma + n0 + r), rt);
                }
            }
        }
        __syncwarp();
        cluster_sync_all();                     // no CTA leaves while another reads its shared memory
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, tmem_cols);
    }
}

}  // namespace bl
