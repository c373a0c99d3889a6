// The epilogue linear for a few dozen to a few hundred tokens, where reading
// the weights once sets the pace and the tiles of the output alone do not
// fill the GPU.
//
//   acc[n, m] = sum_k W[n, k] X[m, k]     (TMEM: lane = weight row, column = token)
//   y[m, n]   = bf16_rne( residual[m, n] + act( (float(acc) * sx[m]) * sw[n] + bias[n] ) )
//
// Swap-AB: 128 weight rows are the A operand of tcgen05.mma.kind::i8, a block
// of BN tokens the B operand, so shared memory takes no more token rows than
// there are.  A cluster of S CTAs shares a tile's k blocks (S fills the SMs'
// two slots); each keeps its int32 partial sums in shared memory, over the
// drained ring, and CTA r adds those of tokens r, r + S, ... across the cluster
// -- integer sums, exact in any order -- with no workspace, counter or second
// launch.  The weights' loads start before the activation quant ends
// (programmatic launch); weights and tokens are issued by a thread each.
// After the join a warp holds one token's 128 columns, four a lane, so
// residual and output move in 256-byte rows.
//
// Roles (384 threads): warp 0 weight loads, warp 1 TMEM and MMA, warp 2 token
// loads, warps 4..11 TMEM to shared memory; all 12 finish.  All waits are
// bounded.
#pragma once

#include "common.cuh"
#include "epilogue.cuh"
#include "gemm_tc.cuh"

namespace w8a8 {

constexpr int kSpThreads = 384;
constexpr int kKernelIdSplit = 12;

template <int BN>
struct SpSmem {
    static constexpr int kW = 128 * kTcBK;              // 16 KB a stage
    static constexpr int kX = BN * kTcBK;
    static constexpr int kStage = kW + kX;
    static constexpr int kStages = (100 * 1024) / kStage;   // 5, 4 or 3: two CTAs an SM
    static constexpr int kTiles = kStages * kStage;
    static constexpr int kBars = (2 * kStages + 2) * 8;
    static constexpr int kBytes = 1024 + kTiles + kBars + 16;
    static_assert(BN * 128 * 4 <= kTiles, "the partial sums lie over the ring");
    static_assert(2 * (kBytes + 1024) <= 228 * 1024, "two CTAs an SM");
};

struct SpArgs {
    const float* sx;      // [M]
    const float* sw;      // [N]
    uint16_t* y;
    EpiFused f;
    int M, N, nkb;
    int mtiles;           // blocks of BN tokens
};

template <int BN>
__global__ void __launch_bounds__(kSpThreads, 2)
    gemm_split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, SpArgs a) {
    using SM = SpSmem<BN>;
    constexpr int ST = SM::kStages;
    constexpr int kCols = BN < 32 ? 32 : BN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::kTiles);
    uint64_t* empty = full + ST;
    uint64_t* done = empty + ST;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t S;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
    const uint32_t r = cluster_ctarank();
    const int tile = blockIdx.x / S;                       // token blocks of a weight tile side by side
    const int n0 = tile / a.mtiles * 128, m0 = tile % a.mtiles * BN;
    const int kb0 = (int)((int64_t)a.nkb * r / S), kb1 = (int)((int64_t)a.nkb * (r + 1) / S);
    const int mv = min(BN, a.M - m0);                      // tokens of the block

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(&full[s], 2);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0 || warp == 2) {
        // ---------------------------------------------------------- weight and token loads
        if (lane == 0) {
            const CUtensorMap* map = warp == 0 ? &tmW : &tmX;
            prefetch_tensormap(map);
            const int off = warp == 0 ? 0 : SM::kW, row = warp == 0 ? n0 : m0;
            const uint32_t bytes = warp == 0 ? SM::kW : SM::kX;
            if (warp == 2) asm volatile("griddepcontrol.wait;" ::: "memory");   // the codes come from the kernel before
            int stage = 0;
            uint32_t phase = 0, issued = 0, last_phase = 0;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, (kKernelIdSplit << 16) | 1)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&full[stage], bytes);
                tma_load_2d(smem + stage * SM::kStage + off, map, &full[stage], kb * kTcBK, row);
                issued |= 1u << stage;
                last_phase = (last_phase & ~(1u << stage)) | (phase << stage);
                if (++stage == ST) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) {
                // every copy lands (or both threads' waits run out) before the CTA exits
                for (int s = 0; s < ST; ++s)
                    if (issued & (1u << s))
                        mbar_wait_bounded(&full[s], (last_phase >> s) & 1u, nullptr, (kKernelIdSplit << 16) | 2, 100000000ull);
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_i8(128, BN);
            int stage = 0;
            uint32_t phase = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait_bounded(&full[stage], phase, abort_flag, (kKernelIdSplit << 16) | 3)) break;
                tc_fence_after();
                const uint32_t w0 = smem_u32(smem + stage * SM::kStage), x0 = w0 + SM::kW;
#pragma unroll
                for (int kk = 0; kk < kTcBK / 32; ++kk)
                    tc_mma_i8(tmem_base, smem_desc_k_sw128(w0 + kk * 32), smem_desc_k_sw128(x0 + kk * 32), idesc,
                              (kb > kb0 || kk > 0) ? 1u : 0u);
                tc_commit(&empty[stage]);
                if (++stage == ST) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            tc_commit(done);
        }
    } else if (a.f.res) {
        // ---------------------------------------------------------- bring this CTA's residual rows towards the SM
        asm volatile("griddepcontrol.wait;" ::: "memory");
        for (int i = (int)r + (int)S * (warp - 3); i < mv; i += 9 * (int)S)
            if (lane < 2 && n0 + 64 * lane < a.N)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(a.f.res + (int64_t)(m0 + i) * a.f.ldr + n0 + 64 * lane));
    }
    const int n = n0 + 4 * lane;
    float4 sw = make_float4(0.0f, 0.0f, 0.0f, 0.0f), bias = sw;
    if (n < a.N) {
        sw = __ldg(reinterpret_cast<const float4*>(a.sw + n));
        if (a.f.bias) bias = __ldg(reinterpret_cast<const float4*>(a.f.bias + n));
    }
    // the sums are complete, and with them every read of the ring
    if (warp >= 4) {
        const bool ok = mbar_wait_bounded(done, 0u, abort_flag, (kKernelIdSplit << 16) | 4);
        tc_fence_after();
        if (ok) {
            const int quarter = warp & 3, half = (warp - 4) >> 2;
            int* part = reinterpret_cast<int*>(smem) + quarter * 32 + lane;
            const uint32_t tq = tmem_base + ((uint32_t)(quarter * 32) << 16);
#pragma unroll
            for (int c = 0; c < BN / 2; c += 16) {
                const int col = half * (BN / 2) + c;
                if (col >= mv) break;
                uint32_t v[16];
                tmem_ld_32x32b_x16(tq + (uint32_t)col, v);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) part[(col + j) * 128] = (int)v[j];
            }
        }
        tc_fence_before();
    }
    __syncthreads();      // the warps whose first lane had a role are whole again
    cluster_sync_all();   // every CTA's sums are in its shared memory
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (n < a.N) {
        const uint32_t own = smem_u32(smem) + 16 * lane;
        constexpr int kWarps = kSpThreads / 32, U = 4;     // U tokens of a warp at a time
        for (int i0 = (int)r + (int)S * warp; i0 < mv; i0 += (int)S * kWarps * U) {
            uint2 res[U];
            float sx[U];
            int4 acc[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int i = i0 + (int)S * kWarps * j;
                res[j] = make_uint2(0, 0);
                acc[j] = make_int4(0, 0, 0, 0);
                sx[j] = 0.0f;
                if (i < mv) {
                    if (a.f.res) res[j] = __ldcg(reinterpret_cast<const uint2*>(a.f.res + (int64_t)(m0 + i) * a.f.ldr + n));
                    sx[j] = __ldcg(a.sx + m0 + i);
                }
            }
            for (uint32_t p = 0; p < S; ++p) {
                const uint32_t from = mapa_shared(own, p);
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int i = i0 + (int)S * kWarps * j;
                    if (i < mv) {
                        int4 v;
                        asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                     : "r"(from + (uint32_t)i * 512));
                        acc[j].x += v.x;
                        acc[j].y += v.y;
                        acc[j].z += v.z;
                        acc[j].w += v.w;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int i = i0 + (int)S * kWarps * j;
                if (i < mv)
                    *reinterpret_cast<uint2*>(a.y + (int64_t)(m0 + i) * a.f.ldy + n) =
                        epi_fused4(acc[j], sx[j], sw, bias, res[j], a.f.act);
            }
        }
    }
    cluster_sync_all();   // no CTA leaves while another reads its sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, kCols);
    }
}

}  // namespace w8a8
