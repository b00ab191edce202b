// Grouped W4A16 GEMM on the sm_100a tensor cores: bf16 rows sorted by expert
// times the expert's packed 4-bit weight, dequantized to bf16 inside the tile
// ("Kimi 2.7 MoE, 4-bit storage to INT8" §4.4 step 4 for the grouping,
// "Inference Quantization ch.1" §2-§3.2 for the weight-only product):
//   w_hat[e,k,n] = bf16( fp32( s_w[e,g,n] * (q[e,k,n] - z[e,g,n]) ) )  g = k / group
//   y[r,n]       = bf16( sum_k x[r,k] * w_hat[e,k,n] )   e = expert of row r, fp32 sums
//
// The tile kernel (many rows for each expert).  The pipeline of the dense
// W4A16 kernel (gemm_w4a16.cuh: weight ring, activation ring, eight warps that
// dequantize into a swizzled A ring, one MMA thread, two accumulators in TMEM)
// over the tile list of the grouped W8A8 kernel (gemm_w8a8_grouped.cuh): every
// CTA derives tiles from the device offsets, hands them out round-robin, sets
// the MMA's N to the tile's rows and loads no more activation boxes than they
// need.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "gemm_w4a16.cuh"
#include "gemm_w8a8_grouped.cuh"

namespace w4a8 {

struct W16GroupedParams {
    int N, K, KB;                // KB = K / 64 k-blocks
    int E, R, G, group;
    int n_tiles;                 // ceil(N / 128)
    const int32_t* offsets;      // [E + 1] device
    const uint8_t* packed;       // E stacked packed weights
    long long packed_estride;    // bytes between experts
    int sg_rows;                 // rows (groups) of the scale / zero-point boxes
    uint16_t* Y;
    int ldy;
    int vec16;
    int32_t* status;
    unsigned long long wait_ns;
};

template <int BN>
struct W16GCfg : W16Cfg<BN> {
    using B = W16Cfg<BN>;
    static constexpr int XROWS = BN < 128 ? BN : 128;       // rows per activation request
    static constexpr int STG = 4 * 2048;                    // output staging: 32 tokens x 32 columns per warp
    static constexpr int OFF_BAR = B::OFF_Y + STG;
    static constexpr int OFF_TABLE = OFF_BAR + B::NUM_BARS * 8;
    static constexpr int TABLE = 3 * (kGroupedMaxExperts + 1) * 4;
    static constexpr int OFF_MISC = OFF_TABLE + TABLE;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int BN, bool SYM>
__global__ void __launch_bounds__(kW16Threads, 1)
    w4a16_grouped_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_s,
                         const __grid_constant__ CUtensorMap tmap_z, const W16GroupedParams p) {
    using C = W16GCfg<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* w_full = bars;                   // [NW] codes, scales, zero-points landed
    uint64_t* w_empty = w_full + C::NW;        // [NW] the 8 dequant warps read them
    uint64_t* x_full = w_empty + C::NW;        // [NX] activation boxes landed
    uint64_t* x_empty = x_full + C::NX;        // [NX] their MMAs completed
    uint64_t* a_full = x_empty + C::NX;        // [NA] bf16 weight tile written
    uint64_t* a_empty = a_full + C::NA;        // [NA] its MMAs completed
    uint64_t* acc_full = a_empty + C::NA;      // [2]
    uint64_t* acc_empty = acc_full + 2;        // [2]
    uint64_t* drain = acc_empty + 2;           // [1]
    GroupTable g;
    g.beg = reinterpret_cast<int32_t*>(smem + C::OFF_TABLE);
    g.cnt = g.beg + kGroupedMaxExperts + 1;
    g.mt = g.cnt + kGroupedMaxExperts + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    int* abort_flag = reinterpret_cast<int*>(smem + C::OFF_MISC + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        pdl_launch_dependents();
        for (int i = 0; i < C::NW; ++i) {
            mbar_init(&w_full[i], 1);
            mbar_init(&w_empty[i], kW16DqWarps);
        }
        for (int i = 0; i < C::NX; ++i) {
            mbar_init(&x_full[i], 1);
            mbar_init(&x_empty[i], 1);
        }
        for (int i = 0; i < C::NA; ++i) {
            mbar_init(&a_full[i], kW16DqWarps);
            mbar_init(&a_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
        prefetch_tmap(&tmap_x);
        prefetch_tmap(&tmap_s);
        if (!SYM) prefetch_tmap(&tmap_z);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    // offsets and rows may come from the kernel launched just before
    pdl_wait_prerequisites();
    build_group_table(g, p.offsets, p.E, p.R, BN, blockIdx.x == 0 ? p.status : nullptr);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const WaitCtx wc{abort_flag, p.status, wait_cycles_for_ns(p.wait_ns)};
    GroupedWalk walk(g, p.E, p.n_tiles, p.KB, 0);
    const int KB = p.KB;
    const int kb_shift = p.group == 128 ? 1 : 0;   // k-blocks of 64 per group: 1 << kb_shift
    long long tile;
    int kb_first, kb_end;                           // always 0 and KB: whole tiles

    if (warp == 0) {
        // ------------------------------------------ producer: weight ring --
        if (lane == 0) {
            Ring rw;
            long long issued = 0;
            bool ok = true;
            while (ok && walk.next(tile, kb_first, kb_end)) {
                const GroupedTile gt(g, p.E, p.n_tiles, BN, tile);
                const int halves = min(128, p.N - gt.nt * 128) / 64;
                const uint8_t* codes = p.packed + gt.e * p.packed_estride;
                for (int kb = 0; kb < KB; kb += kW16KSW) {
                    const int len = min(kW16KSW, KB - kb);
                    if (!wait_bounded(&w_empty[rw.idx], rw.phase ^ 1u, wc)) { ok = false; break; }
                    uint32_t bytes = halves * len * 2048 + p.sg_rows * 512;
                    if (!SYM) bytes += p.sg_rows * 128;
                    mbar_arrive_expect_tx(&w_full[rw.idx], bytes);
                    uint8_t* st = smem + C::OFF_W + rw.idx * C::W_STAGE;
                    // 64 columns x 32 k are 1 KB; a column block's chunks follow one another over all of K
                    for (int hf = 0; hf < halves; ++hf)
                        bulk_load(st + hf * C::PK_HALF, codes + ((long long)(gt.nt * 2 + hf) * KB + kb) * 2048,
                                  len * 2048, &w_full[rw.idx]);
                    const int g0 = gt.e * p.G + (kb >> kb_shift);
                    tma_load_2d(st + C::W_S, &tmap_s, &w_full[rw.idx], gt.nt * 128, g0);
                    if (!SYM) tma_load_2d(st + C::W_Z, &tmap_z, &w_full[rw.idx], gt.nt * 128, g0);
                    rw.next(C::NW);
                    ++issued;
                }
            }
            WaitCtx wd = wc;
            volatile int no_abort = 0;
            wd.abort = &no_abort;
            Ring d = rw;
            for (long long k = 0; k < issued && k < C::NW; ++k) {
                ring_back(d, C::NW);
                (void)wait_bounded(&w_full[d.idx], d.phase, wd);
            }
        }
    } else if (warp == kW16XWarp) {
        // -------------------------------------- producer: activation ring --
        if (lane == 0) {
            Ring rx;
            long long issued = 0;
            bool ok = true;
            while (ok && walk.next(tile, kb_first, kb_end)) {
                const GroupedTile gt(g, p.E, p.n_tiles, BN, tile);
                const int boxes = gt.rows > C::XROWS ? 2 : 1;
                for (int kb = 0; kb < KB; kb += C::KX) {
                    if (!wait_bounded(&x_empty[rx.idx], rx.phase ^ 1u, wc)) { ok = false; break; }
                    uint8_t* st = smem + C::OFF_X + rx.idx * C::X_STAGE;
                    mbar_arrive_expect_tx(&x_full[rx.idx], boxes * (C::KX * C::XROWS * 128));
                    tma_load_3d(st, &tmap_x, &x_full[rx.idx], 0, gt.row0, kb);
                    // BN > XROWS only where a stage is one k-block, so the second box follows the first
                    if (boxes == 2)
                        tma_load_3d(st + C::XROWS * 128, &tmap_x, &x_full[rx.idx], 0, gt.row0 + C::XROWS, kb);
                    rx.next(C::NX);
                    ++issued;
                }
            }
            WaitCtx wd = wc;
            volatile int no_abort = 0;
            wd.abort = &no_abort;
            Ring d = rx;
            for (long long k = 0; k < issued && k < C::NX; ++k) {
                ring_back(d, C::NX);
                (void)wait_bounded(&x_full[d.idx], d.phase, wd);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issue --
        if (lane == 0) {
            Ring rx, ra, rc;
            bool ok = true;
            while (ok && walk.next(tile, kb_first, kb_end)) {
                const GroupedTile gt(g, p.E, p.n_tiles, BN, tile);
                const uint32_t idesc = idesc_bf16((gt.rows + 15) & ~15);
                if (!wait_bounded(&acc_empty[rc.idx], rc.phase ^ 1u, wc)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + rc.idx * BN;
                int xo = 0;   // offset of the next k-block in its activation stage
                for (int kb = 0; kb < KB && ok; kb += C::KA) {
                    const int len = min(C::KA, KB - kb);
                    if (!wait_bounded(&a_full[ra.idx], ra.phase, wc)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t adesc0 = umma_desc_kmajor(smem_u32(smem + C::OFF_A + ra.idx * C::A_STAGE), 128);
#pragma unroll
                    for (int j = 0; j < C::KA; ++j) {
                        if (j < len) {
                            if (xo == 0) {
                                if (!wait_bounded(&x_full[rx.idx], rx.phase, wc)) { ok = false; break; }
                                tc_fence_after();
                            }
                            const uint64_t adesc = adesc0 + (uint64_t)(j * (C::A_BYTES >> 4));
                            const uint64_t bdesc =
                                umma_desc_kmajor(smem_u32(smem + C::OFF_X + rx.idx * C::X_STAGE + xo * C::XB), 128);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_bf16(d_tmem, adesc + 2 * kk, bdesc + 2 * kk, idesc,
                                         (kb > 0 || j > 0 || kk > 0) ? 1u : 0u);
                            if (xo + 1 == C::KX || kb + j + 1 == KB) {
                                tc_commit(&x_empty[rx.idx]);
                                rx.next(C::NX);
                                xo = 0;
                            } else {
                                ++xo;
                            }
                        }
                    }
                    if (!ok) break;
                    tc_commit(&a_empty[ra.idx]);
                    ra.next(C::NA);
                }
                if (!ok) break;
                tc_commit(&acc_full[rc.idx]);
                rc.next(2);
            }
            // drain: every MMA issued above completes before TMEM is freed
            tc_commit(drain);
            WaitCtx wd = wc;
            volatile int no_abort = 0;
            wd.abort = &no_abort;
            (void)wait_bounded(drain, 0, wd);
        }
    } else if (warp >= kW16DqWarp0 && warp < kW16DqWarp0 + kW16DqWarps) {
        // ----------------------------------------------------- dequantize --
        const int dt = threadIdx.x - kW16DqWarp0 * 32;  // 0..255
        const int r = dt & 127;                          // weight column within the tile = A row
        const int cc = dt >> 7;                          // 32-k chunk of the k-block
        const int hf = r >> 6;
        const uint32_t row_addr = smem_u32(smem + C::OFF_A) + r * 128;
        Ring rw, ra;
        uint64_t A[5], S[5];
        bool ok = true;
        while (ok && walk.next(tile, kb_first, kb_end)) {
            const GroupedTile gt(g, p.E, p.n_tiles, BN, tile);
            const bool valid = hf * 64 < min(128, p.N - gt.nt * 128);
            int wo = 0;               // offset of the next k-block in its weight stage
            int g0 = 0, g_prev = -1;
            for (int kb = 0; kb < KB; kb += C::KA) {
                const int len = min(C::KA, KB - kb);
                if (wo == 0) {
                    ok = warp_wait_bounded(&w_full[rw.idx], rw.phase, wc);
                    g0 = kb >> kb_shift;
                }
                if (ok) ok = warp_wait_bounded(&a_empty[ra.idx], ra.phase ^ 1u, wc);
                if (!ok) break;
                const uint8_t* st = smem + C::OFF_W + rw.idx * C::W_STAGE;
                uint4 c[C::KA];
#pragma unroll
                for (int j = 0; j < C::KA; ++j)
                    c[j] = (valid && j < len)
                               ? *reinterpret_cast<const uint4*>(st + hf * C::PK_HALF + (wo + j) * 2048 + cc * 1024 +
                                                                 (r & 63) * 16)
                               : make_uint4(0u, 0u, 0u, 0u);
                uint4 out[C::KA][4];
#pragma unroll
                for (int j = 0; j < C::KA; ++j) {
                    if (valid && j < len) {
                        const int gi = (kb + j) >> kb_shift;
                        if (gi != g_prev) {
                            const float sv = reinterpret_cast<const float*>(st + C::W_S)[(gi - g0) * 128 + r];
                            const float zc = SYM ? 8.0f : (float)st[C::W_Z + (gi - g0) * 128 + r];
#pragma unroll
                            for (int q = 0; q < 5; ++q) {
                                const float sc = (float)(1 << (4 * q));
                                A[q] = f2_splat(-(8388608.0f + zc * sc));
                                S[q] = f2_splat(sv * (1.0f / sc));
                            }
                            g_prev = gi;
                        }
                        dequant_chunk<SYM>(c[j], A, S, out[j]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) out[j][i] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                wo += len;
                if (wo == kW16KSW || kb + len == KB) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&w_empty[rw.idx]);
                    rw.next(C::NW);
                    wo = 0;
                }
                const uint32_t a_row = row_addr + ra.idx * C::A_STAGE;
#pragma unroll
                for (int j = 0; j < C::KA; ++j) {
                    if (j < len) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int jj = cc * 4 + i;
                            const uint32_t addr = a_row + j * C::A_BYTES + ((jj ^ (r & 7)) << 4);
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(out[j][i].x),
                                         "r"(out[j][i].y), "r"(out[j][i].z), "r"(out[j][i].w)
                                         : "memory");
                        }
                    }
                }
                fence_proxy_async_smem();  // generic-proxy writes -> visible to the tensor core
                __syncwarp();
                if (lane == 0) mbar_arrive(&a_full[ra.idx]);
                ra.next(C::NA);
            }
        }
    } else if (warp >= kW16EpiWarp0 && warp < kW16EpiWarp0 + 4) {
        // ------------------------------------------------------- epilogue --
        const int q = warp & 3;                 // TMEM lane quadrant
        const uint32_t lane_addr = ((uint32_t)(q * 32)) << 16;
        uint16_t* stg = reinterpret_cast<uint16_t*>(smem + C::OFF_Y) + (warp - kW16EpiWarp0) * 1024;
        constexpr int LB = C::LB;
        Ring ra;
        while (walk.next(tile, kb_first, kb_end)) {
            const GroupedTile gt(g, p.E, p.n_tiles, BN, tile);
            if (!warp_wait_bounded(&acc_full[ra.idx], ra.phase, wc)) break;
            tc_fence_after();
            const uint32_t tacc = tmem_base + lane_addr + ra.idx * BN;
            const int col0 = gt.nt * 128 + q * 32;
            if (col0 < p.N) {
#pragma unroll 1
                for (int c0 = 0; c0 < gt.rows; c0 += LB) {
                    uint32_t v[LB];
                    tmem_ld32<LB>(tacc + c0, v);
                    tmem_wait_ld();
                    __syncwarp();  // the previous batch's copy-out is done with the staging
#pragma unroll
                    for (int j = 0; j < LB; ++j) stg[j * 32 + lane] = f32_to_bf16_bits(__uint_as_float(v[j]));
                    __syncwarp();
#pragma unroll
                    for (int i = lane; i < LB * 4; i += 32) {
                        const int j = i >> 2;
                        if (c0 + j < gt.rows) {
                            const uint4 val = *reinterpret_cast<const uint4*>(stg + j * 32 + (i & 3) * 8);
                            uint16_t* dst = p.Y + (long long)(gt.row0 + c0 + j) * p.ldy + col0 + (i & 3) * 8;
                            if (p.vec16) {
                                *reinterpret_cast<uint4*>(dst) = val;
                            } else {
                                const uint32_t w4[4] = {val.x, val.y, val.z, val.w};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    dst[2 * k] = (uint16_t)(w4[k] & 0xFFFFu);
                                    dst[2 * k + 1] = (uint16_t)(w4[k] >> 16);
                                }
                            }
                        }
                    }
                }
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[ra.idx]);
            ra.next(2);
        }
    }

    // ----------------------------------------------------------- teardown --
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

// Launches the grouped W4A16 tile kernel for a tile of BN in {16, 32, 64, 128,
// 256} rows (defined in gemm_w4a16_grouped.cu).  Status codes as in w4a8.h.
int launch_w4a16_grouped(int bn, bool sym, const CUtensorMap& tmap_x, const CUtensorMap& tmap_s,
                         const CUtensorMap& tmap_z, const W16GroupedParams& p, int grid, cudaStream_t stream);

// Rows of one activation request of a tile of bn rows.
inline int w4a16_grouped_xrows(int bn) { return bn < 128 ? bn : 128; }

}  // namespace w4a8
