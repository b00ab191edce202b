// Grouped W4A16 GEMM on the sm_100a tensor cores: bf16 rows sorted by expert
// times the expert's packed 4-bit weight, dequantized to bf16 inside the tile
// ("Kimi 2.7 MoE, 4-bit storage to INT8" §4.4 step 4 for the grouping,
// "Inference Quantization ch.1" §2-§3.2 for the weight-only product):
//   w_hat[e,k,n] = bf16( fp32( s_w[e,g,n] * (q[e,k,n] - z[e,g,n]) ) )  g = k / group
//   y[r,n]       = bf16( sum_k x[r,k] * w_hat[e,k,n] )   e = expert of row r, fp32 sums
//
// Design (B200): the tiles of the grouped W8A8 kernel (gemm_w8a8_grouped.cuh:
// every CTA derives them from the device offsets; whole tiles round-robin, or
// equal ranges of k with partial tiles added by the CTA that comes last) around
// the dequantization of the dense W4A16 kernel (gemm_w4a16.cuh).
//   * Swap-AB: 128 weight columns are the MMA's rows, up to BN tokens its
//     columns; its N is set to the tile's rows, and few rows take small
//     activation boxes.
//   * A unit is two k-blocks of 64.  The dequantized bf16 weights go straight
//     to TMEM (the MMA's A operand: lane = column, 32 TMEM columns for a
//     k-block), so they need neither shared memory nor a proxy fence; with A in
//     shared memory the stores and the fence took 500 of a k-block's 2,400
//     cycles (512 rows over 32 experts, K = 7168, N = 4096: 264 -> 245 us).
//   * 8 warps dequantize, two teams of 4, units in turn, so that one team's
//     waits and stores overlap the other's arithmetic.  A thread takes one
//     column's 128 k and gives the stage of packed weights back as soon as the
//     codes are in registers (16 warps with 64 k each: 222 us to 214).
//   * Activations come in stages of their own, longer in k where the rows are
//     few: two units of them on their way left the pipeline without arithmetic
//     at 180 us, these at 145.
//   * The MMA warp's pace is the kernel's: of 1,030 cycles for a unit, whatever
//     its rows, it waited 250 on barriers that were complete and issued for
//     390, slowed by the dequantizing warps beside it.  So it has one wait for
//     a unit (another warp sees the activations land: 210 -> 201 us), and
//     descriptors advance by additions.
//   * The producers and the MMA warp run converged, one lane issuing: a lone
//     lane moves every descriptor and address to uniform registers one by one,
//     135 cycles for each MMA instead of 32, 300 for each copy.
//   * The dequantization takes 22 instructions for 8 weights, 13 of them at
//     half rate: 26 cycles measured alone, 94 of the 201 us.  A mask is an
//     immediate and 2^23 a register; a second constant for the flipped bit
//     would cost each mask a move.  At 144 rows and more the activations come at
//     47 bytes a cycle for each SM, the bound of that case.
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda.h>
#include <cuda_bf16.h>

#include "gemm_w4a16.cuh"
#include "gemm_w8a8_grouped.cuh"

namespace w4a8 {

struct W16GroupedParams {
    int N;
    int units;                   // stages of two k-blocks of a tile
    int E, R, G, group;
    int n_tiles;                 // ceil(N / 128)
    int KB;                      // k-blocks of 64
    const int32_t* offsets;      // [E + 1] device
    const uint8_t* packed;       // E stacked packed weights
    long long packed_estride;    // bytes between experts
    uint16_t* Y;
    int ldy;
    int vec16;
    int split_tiles;             // tiles below which units may be split (0: never)
    float* partial;              // [2 * grid][BN][128] fp32 partial tiles
    unsigned long long* counts;  // [split_tiles] arrivals of this launch
    unsigned long long epoch;
    int32_t* status;
    unsigned long long wait_ns;
};

constexpr int kW16GEpiWarp0 = 3;       // after the two producers and the MMA warp
constexpr int kW16GXSeenWarp = 7;
constexpr int kW16GDqWarp0 = 8;        // a multiple of 4: a warp's TMEM lanes follow from its number
constexpr int kW16GKSW = 2;            // k-blocks of 64 per stage of packed weights: a unit's

// Activation boxes: 32 rows x 8 k-blocks (tiles of 16 rows: 16 x 2), 64 rows
// x 4, or, for tiles of more than 64 rows, the rows below x 1.
__host__ __device__ constexpr int w4a16_grouped_rows0(int bn) { return bn == 16 ? 16 : 32; }
__host__ __device__ constexpr int w4a16_grouped_kb0(int bn) { return bn == 16 ? 2 : 8; }
constexpr int kW16GRows1 = 64, kW16GKb1 = 4;
__host__ __device__ constexpr int w4a16_grouped_xrows(int bn) { return bn == 192 ? 96 : 128; }

template <int BN>
struct W16GCfg {
    // A stage of activations: 8 k-blocks of 32 rows, 4 of 64, 2 of BN.  Few rows take long stages, so that enough
    // of k is on its way whatever the tile.
    static constexpr int XSTAGE = BN <= 128 ? 32768 : 2 * BN * 128;
    static constexpr int NX = BN <= 128 ? 4 : 3;
    static constexpr int NS = BN <= 128 ? 4 : 2;           // stages of dequantized weights: the CTA's units in turn
    // Teams of 4 dequantizing warps, a unit each in turn.  At most NS: a team that is P units ahead has seen
    // unit - P - NS released, and a barrier's parity tells two uses of a stage apart, not three.
    static constexpr int TEAMS = 2;
    static constexpr int DQ_WARPS = 4 * TEAMS;
    static constexpr int THREADS = 32 * (kW16GDqWarp0 + DQ_WARPS);
    static_assert(TEAMS <= NS, "a team's lead");
    static constexpr int XROWS = w4a16_grouped_xrows(BN);  // rows of the largest activation box
    static constexpr int KSW = kW16GKSW;
    static constexpr int PK_HALF = KSW * 2048;             // codes of one 64-column half
    static constexpr int W_S = 2 * PK_HALF;                // fp32 scales [KSW][128]
    static constexpr int W_Z = W_S + KSW * 512;            // zero-points [KSW][128]
    static constexpr int W_STAGE = W_Z + KSW * 128;
    // Stages of packed weights, the CTA's units in turn.  A multiple of TEAMS: a stage's readers are always the same
    // team, which has seen its last use (copies of different stages may land out of order).
    static constexpr int NW = 2 * TEAMS;
    static constexpr int STG = 4 * 1024;                   // output staging: 16 tokens x 32 columns per warp
    static constexpr int OFF_W = NX * XSTAGE;
    static constexpr int OFF_Y = OFF_W + NW * W_STAGE;
    static constexpr int OFF_BAR = OFF_Y + STG;
    static constexpr int NUM_BARS = 2 * NW + 2 * NS + 2 * NX + 5;
    static constexpr int OFF_TABLE = OFF_BAR + NUM_BARS * 8;
    static constexpr int TABLE = 3 * (kGroupedMaxExperts + 1) * 4;
    static constexpr int OFF_MISC = OFF_TABLE + TABLE;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    // TMEM: two accumulators, then the dequantized weights: 64 columns (two k-blocks of 64 bf16) per stage
    static constexpr int A_COL0 = 2 * BN;
    static constexpr uint32_t TMEM_COLS = A_COL0 + 64 * NS <= 256 ? 256 : A_COL0 + 64 * NS <= 512 ? 512 : 1024;
    static_assert(TMEM_COLS <= 512, "TMEM");
    // a part of a split tile, in units / 16: 0.3 + 0.05 for each row (four warps add the parts)
    static constexpr int PART0 = 5, PART1 = 13;
    static constexpr int LB = 16;                        // tokens per epilogue batch
    static_assert(BN == 16 || BN == 32 || BN == 64 || BN == 128 || BN == 192, "BN");
    static_assert(W_S % 128 == 0 && W_STAGE % 128 == 0, "TMA destinations");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

// The activation stages of a tile: units to a stage, and bytes from one k-block
// to the next.
template <int BN>
struct XPlan {
    int units, kstride;
    __device__ __forceinline__ explicit XPlan(int rows) {
        if (BN <= 32 || rows <= w4a16_grouped_rows0(BN)) {
            units = w4a16_grouped_kb0(BN) / 2;
            kstride = w4a16_grouped_rows0(BN) * 128;
        } else if (BN <= 64 || rows <= kW16GRows1) {
            units = kW16GKb1 / 2;
            kstride = kW16GRows1 * 128;
        } else {
            units = 1;
            kstride = BN * 128;
        }
    }
};

// Scale and zero-point of a column's group for dequant_word32: pairs for the
// nibbles of the first and of the second byte of a halfword (a = -(2^23 + z
// 16^p): a paired subtraction would negate its operand first).
template <bool SYM>
struct NibblePairs {
    uint64_t s01, s23, a01, a23;
    __device__ __forceinline__ void set(float s, uint32_t z) {
        s01 = f2_from_bits(__float_as_uint(s), __float_as_uint(s * 0x1p-4f));
        s23 = f2_from_bits(__float_as_uint(s * 0x1p-8f), __float_as_uint(s * 0x1p-12f));
        const uint32_t zc = SYM ? 8u : z;
        a01 = f2_from_bits(0xCB000000u | zc, 0xCB000000u | (zc << 4));
        a23 = f2_from_bits(0xCB000000u | (zc << 8), 0xCB000000u | (zc << 12));
    }
};

// The bits of w under mask in the mantissa of 2^23.  The mask is an immediate
// and 2^23 a register; a second constant would cost a move each time.
template <uint32_t MASK>
__device__ __forceinline__ uint32_t magic_bits(uint32_t w) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "n"(MASK), "r"(0x4B000000u));  // (w & mask) | 2^23
    return d;
}

// dequant_chunk's arithmetic for one word (bytes 0-3): lo / hi = its low and
// high nibbles' weights, two bf16 pairs each in byte order.  Symmetric codes
// are two's complement; with bit 3 flipped they are q + 8.
template <bool SYM>
__device__ __forceinline__ void dequant_word32(uint32_t w, const NibblePairs<SYM>& q, uint32_t* lo, uint32_t* hi) {
    if (SYM) w ^= 0x88888888u;
    const uint32_t v = w >> 16;
    float l0, l1, l2, l3, h0, h1, h2, h3;
    f2_split(f2_mul(f2_add(f2_from_bits(magic_bits<0xFu>(w), magic_bits<0xF0u>(w)), q.a01), q.s01), l0, h0);
    f2_split(f2_mul(f2_add(f2_from_bits(magic_bits<0xF00u>(w), magic_bits<0xF000u>(w)), q.a23), q.s23), l1, h1);
    f2_split(f2_mul(f2_add(f2_from_bits(magic_bits<0xFu>(v), magic_bits<0xF0u>(v)), q.a01), q.s01), l2, h2);
    f2_split(f2_mul(f2_add(f2_from_bits(magic_bits<0xF00u>(v), magic_bits<0xF000u>(v)), q.a23), q.s23), l3, h3);
    lo[0] = pack_bf16x2(l0, l1);
    lo[1] = pack_bf16x2(l2, l3);
    hi[0] = pack_bf16x2(h0, h1);
    hi[1] = pack_bf16x2(h2, h3);
}

// D[tmem] (+)= A[tmem] * B[smem]^T, bf16 x bf16 -> fp32, K = 16; the A tile
// sits in TMEM (lane = row, 2 consecutive k per 32-bit column).
__device__ __forceinline__ void mma_bf16_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <int BN, bool SYM>
__global__ void __launch_bounds__(W16GCfg<BN>::THREADS, 1)
    w4a16_grouped_kernel(const __grid_constant__ CUtensorMap tmap_x0, const __grid_constant__ CUtensorMap tmap_x1,
                         const __grid_constant__ CUtensorMap tmap_x2, const __grid_constant__ CUtensorMap tmap_s, const __grid_constant__ CUtensorMap tmap_z, const W16GroupedParams p) {
    using C = W16GCfg<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* w_full = bars;                   // [NW] codes, scales, zero-points landed
    uint64_t* w_empty = w_full + C::NW;        // [NW] a team read them
    uint64_t* full = w_empty + C::NW;          // [NS] dequantized weights written by a team, activations landed
    uint64_t* empty = full + C::NS;            // [NS] their MMAs completed
    uint64_t* x_full = empty + C::NS;          // [NX] activations landed
    uint64_t* x_empty = x_full + C::NX;        // [NX] their MMAs completed
    uint64_t* acc_full = x_empty + C::NX;      // [2]
    uint64_t* acc_empty = acc_full + 2;        // [2]
    uint64_t* drain = acc_empty + 2;           // [1]
    GroupTable g;
    g.beg = reinterpret_cast<int32_t*>(smem + C::OFF_TABLE);
    g.cnt = g.beg + kGroupedMaxExperts + 1;
    g.mt = g.cnt + kGroupedMaxExperts + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    int* abort_flag = reinterpret_cast<int*>(smem + C::OFF_MISC + 4);
    int* last_flag = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        pdl_launch_dependents();
        for (int i = 0; i < C::NW; ++i) {
            mbar_init(&w_full[i], 1);
            mbar_init(&w_empty[i], 4);
        }
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(&full[i], 4 + 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < C::NX; ++i) {
            mbar_init(&x_full[i], 1);
            mbar_init(&x_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
        prefetch_tmap(&tmap_x0);
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
    GroupedWalk walk(g, p.E, p.n_tiles, p.units, p.split_tiles, grouped_part(C::PART0, C::PART1, BN, p.R, g.mt[p.E]));
    const int KB = p.KB;
    const int kb_shift = p.group == 128 ? 1 : 0;   // k-blocks of 64 per group: 1 << kb_shift
    long long tile;
    int u0, u1;                                     // the segment's stages

    if (warp == 0) {
        // ------------------------------------------ producer: weight ring --
        const bool leader = elect_one();
        uint32_t phases = 0u;    // parity of every stage's next fill
        uint32_t used = 0u;      // stages that have been filled
        uint32_t seq = 0u;       // units of this CTA so far
        bool ok = true;
        const int sg_rows = C::KSW >> kb_shift;
        while (ok && walk.next(tile, u0, u1)) {
            const GroupedTile gt(g, p.E, p.n_tiles, BN, tile);
            const int halves = min(128, p.N - gt.nt * 128) / 64;
            const uint8_t* codes = p.packed + gt.e * p.packed_estride + (long long)gt.nt * 2 * KB * 2048;
            for (int u = u0; u < u1; ++u, ++seq) {
                const int kb = 2 * u, len = min(C::KSW, KB - kb);
                const int slot = seq % C::NW;
                ok = warp_wait_bounded(&w_empty[slot], ((phases >> slot) & 1u) ^ 1u, wc);
                if (!ok) break;
                if (leader) {
                    uint32_t bytes = halves * len * 2048 + sg_rows * 512;
                    if (!SYM) bytes += sg_rows * 128;
                    mbar_arrive_expect_tx(&w_full[slot], bytes);
                    uint8_t* st = smem + C::OFF_W + slot * C::W_STAGE;
                    // 64 columns x 32 k are 1 KB; a column block's chunks follow one another over all of K
                    bulk_load(st, codes + (long long)kb * 2048, len * 2048, &w_full[slot]);
                    if (halves == 2)
                        bulk_load(st + C::PK_HALF, codes + (long long)(KB + kb) * 2048, len * 2048, &w_full[slot]);
                    const int g0 = gt.e * p.G + (kb >> kb_shift);
                    tma_load_2d(st + C::W_S, &tmap_s, &w_full[slot], gt.nt * 128, g0);
                    if (!SYM) tma_load_2d(st + C::W_Z, &tmap_z, &w_full[slot], gt.nt * 128, g0);
                }
                __syncwarp();
                used |= 1u << slot;
                phases ^= 1u << slot;
            }
        }
        // copies in flight land before the CTA leaves
        if (leader) {
            WaitCtx wd = wc;
            volatile int no_abort = 0;
            wd.abort = &no_abort;
            for (int i = 0; i < C::NW; ++i)   // parity of a stage's last fill
                if ((used >> i) & 1u) (void)wait_bounded(&w_full[i], ((phases >> i) & 1u) ^ 1u, wd);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------- producer: activations --
        const bool leader = elect_one();
        Ring rx;
        long long issued = 0;
        bool ok = true;
        while (ok && walk.next(tile, u0, u1)) {
            const GroupedTile gt(g, p.E, p.n_tiles, BN, tile);
            const XPlan<BN> x(gt.rows);
            const int boxes = gt.rows > C::XROWS ? 2 : 1;
            for (int u = u0; u < u1; u += x.units) {
                const int kb = 2 * u;
                ok = warp_wait_bounded(&x_empty[rx.idx], rx.phase ^ 1u, wc);
                if (!ok) break;
                if (leader) {
                    uint8_t* st = smem + rx.idx * C::XSTAGE;
                    uint64_t* bar = &x_full[rx.idx];
                    // a box's k-blocks past the tile's last are loaded (zeros past K), not used
                    if (BN <= 32 || x.units == w4a16_grouped_kb0(BN) / 2) {
                        mbar_arrive_expect_tx(bar, w4a16_grouped_rows0(BN) * w4a16_grouped_kb0(BN) * 128);
                        tma_load_3d(st, &tmap_x0, bar, 0, gt.row0, kb);
                    } else if (BN <= 64 || x.units == kW16GKb1 / 2) {
                        mbar_arrive_expect_tx(bar, kW16GRows1 * kW16GKb1 * 128);
                        tma_load_3d(st, &tmap_x1, bar, 0, gt.row0, kb);
                    } else {
                        const int len = min(2, KB - kb);
                        mbar_arrive_expect_tx(bar, len * boxes * (C::XROWS * 128));
                        for (int i = 0; i < len; ++i, st += BN * 128) {
                            tma_load_3d(st, &tmap_x2, bar, 0, gt.row0, kb + i);
                            if (boxes == 2)
                                tma_load_3d(st + C::XROWS * 128, &tmap_x2, bar, 0, gt.row0 + C::XROWS, kb + i);
                        }
                    }
                }
                __syncwarp();
                rx.next(C::NX);
                ++issued;
            }
        }
        // copies in flight land before the CTA leaves
        if (leader) {
            WaitCtx wd = wc;
            volatile int no_abort = 0;
            wd.abort = &no_abort;
            for (long long k = 0; k < issued && k < C::NX; ++k) {
                ring_back(rx, C::NX);
                (void)wait_bounded(&x_full[rx.idx], rx.phase, wd);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issue --
        // The whole warp runs the loop and one lane issues: with every value
        // uniform over the warp, an MMA's descriptors sit in uniform registers
        // instead of being moved there one by one.
        {
            const bool leader = elect_one();
            Ring rc, rx, ra;
            bool ok = true;
            while (ok && walk.next(tile, u0, u1)) {
                const GroupedTile gt(g, p.E, p.n_tiles, BN, tile);
                const uint32_t idesc = idesc_bf16((gt.rows + 15) & ~15);
                const XPlan<BN> x(gt.rows);
                const uint32_t kstep = (uint32_t)x.kstride >> 4;     // in descriptor units
                if (!warp_wait_bounded(&acc_empty[rc.idx], rc.phase ^ 1u, wc)) { ok = false; break; }
                const uint32_t d_tmem = tmem_base + rc.idx * BN;
                uint32_t more = 0u;                                  // 0: the tile's first MMA
                int left = u1 - u0, kbs = KB - 2 * u0;
                while (left > 0) {
                    // one activation stage
                    uint64_t bdesc = umma_desc_kmajor(smem_u32(smem + rx.idx * C::XSTAGE), 128);
                    const int n = min(left, x.units);
                    left -= n;
                    for (int i = n; i > 0; --i) {
                        ok = warp_wait_bounded(&full[ra.idx], ra.phase, wc);
                        if (!ok) break;
                        tc_fence_after();
                        if (leader) {
                            const uint32_t a = tmem_base + C::A_COL0 + ra.idx * 64;
                            mma_bf16_tmem_a(d_tmem, a, bdesc, idesc, more);
#pragma unroll
                            for (int kk = 1; kk < 4; ++kk)
                                mma_bf16_tmem_a(d_tmem, a + 8 * kk, bdesc + 2 * kk, idesc, 1u);
                            if (kbs > 1) {
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    mma_bf16_tmem_a(d_tmem, a + 32 + 8 * kk, bdesc + kstep + 2 * kk, idesc, 1u);
                            }
                            tc_commit(&empty[ra.idx]);
                        }
                        __syncwarp();
                        more = 1u;
                        kbs -= 2;
                        bdesc += 2 * kstep;
                        ra.next(C::NS);
                    }
                    if (!ok) break;
                    if (leader) tc_commit(&x_empty[rx.idx]);
                    __syncwarp();
                    rx.next(C::NX);
                }
                if (!ok) break;
                if (leader) tc_commit(&acc_full[rc.idx]);
                __syncwarp();
                rc.next(2);
            }
            // drain: every MMA issued above completes before TMEM is freed
            if (leader) {
                tc_commit(drain);
                WaitCtx wd = wc;
                volatile int no_abort = 0;
                wd.abort = &no_abort;
                (void)wait_bounded(drain, 0, wd);
            }
            __syncwarp();
        }
    } else if (warp == kW16GXSeenWarp) {
        // ------------------------------------ activations seen to have landed --
        // Counts them in at each unit's stage of weights, so that the MMA warp,
        // whose pace is the kernel's, has one wait for a unit.
        Ring rx, ra;
        bool ok = true;
        while (ok && walk.next(tile, u0, u1)) {
            const GroupedTile gt(g, p.E, p.n_tiles, BN, tile);
            const XPlan<BN> x(gt.rows);
            for (int u = u0, xu = 0; u < u1; ++u) {
                ok = (xu > 0 || warp_wait_bounded(&x_full[rx.idx], rx.phase, wc)) &&
                     warp_wait_bounded(&empty[ra.idx], ra.phase ^ 1u, wc);
                if (!ok) break;
                if (lane == 0) mbar_arrive(&full[ra.idx]);
                ra.next(C::NS);
                if (++xu == x.units || u == u1 - 1) {
                    xu = 0;
                    rx.next(C::NX);
                }
            }
        }
    } else if (warp >= kW16GDqWarp0) {
        // ----------------------------------------------------- dequantize --
        // The teams take units in turn, so that one's waits and hand-over
        // overlap the other's arithmetic.  A thread takes one column's 128 k.
        const int team = (warp - kW16GDqWarp0) >> 2;
        const int r = (warp & 3) * 32 + lane;            // weight column within the tile = A row = TMEM lane
        const int hf = r >> 6;
        const uint32_t a_tmem = tmem_base + (((uint32_t)(warp & 3) * 32) << 16) + C::A_COL0;
        const uint32_t off_c = hf * C::PK_HALF + (r & 63) * 16;
        const int g1 = 1 >> kb_shift;                    // the second k-block's group row
        uint32_t seq = 0u;                               // units of this CTA so far
        uint32_t own = team;                             // the team's next among them: every TEAMS-th
        bool ok = true;
        while (ok && walk.next(tile, u0, u1)) {
            const GroupedTile gt(g, p.E, p.n_tiles, BN, tile);
            const bool valid = hf * 64 < min(128, p.N - gt.nt * 128);
            const uint32_t end = seq + (uint32_t)(u1 - u0);
            for (; own < end; own += C::TEAMS) {
                const int u = u0 + (int)(own - seq);
                const uint32_t slot = own % C::NW;
                ok = warp_wait_bounded(&w_full[slot], (own / C::NW) & 1u, wc);
                if (!ok) break;
                const bool two = 2 * u + 1 < KB;         // warp-uniform
                const uint8_t* st = smem + C::OFF_W + slot * C::W_STAGE;
                // everything this thread needs of the stage, which is then free again
                uint4 c[4] = {};                         // columns past N: scale 0
                float s0 = 0.0f, s1 = 0.0f;
                uint32_t z0 = 0u, z1 = 0u;
                if (valid) {
                    c[0] = *reinterpret_cast<const uint4*>(st + off_c);
                    c[1] = *reinterpret_cast<const uint4*>(st + off_c + 1024);
                    s0 = *reinterpret_cast<const float*>(st + C::W_S + r * 4);
                    if (!SYM) z0 = st[C::W_Z + r];
                    if (two) {
                        c[2] = *reinterpret_cast<const uint4*>(st + off_c + 2 * 1024);
                        c[3] = *reinterpret_cast<const uint4*>(st + off_c + 3 * 1024);
                        s1 = *reinterpret_cast<const float*>(st + C::W_S + (g1 * 128 + r) * 4);
                        if (!SYM) z1 = st[C::W_Z + g1 * 128 + r];
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&w_empty[slot]);
                const uint32_t as = own % C::NS;
                uint32_t out[16];                        // 32 k of the column, bf16 pairs in k order
                NibblePairs<SYM> q;
                q.set(s0, z0);
                auto chunk = [&](const uint4& c) {
                    dequant_word32<SYM>(c.x, q, out, out + 8);
                    dequant_word32<SYM>(c.y, q, out + 2, out + 10);
                    dequant_word32<SYM>(c.z, q, out + 4, out + 12);
                    dequant_word32<SYM>(c.w, q, out + 6, out + 14);
                };
                chunk(c[0]);
                ok = warp_wait_bounded(&empty[as], ((own / C::NS) & 1u) ^ 1u, wc);
                if (!ok) break;
                tc_fence_after();
                tmem_st32<16>(a_tmem + as * 64, out);
                chunk(c[1]);
                tmem_st32<16>(a_tmem + as * 64 + 16, out);
                if (two) {
                    if (kb_shift == 0) q.set(s1, z1);
                    chunk(c[2]);
                    tmem_st32<16>(a_tmem + as * 64 + 32, out);
                    chunk(c[3]);
                    tmem_st32<16>(a_tmem + as * 64 + 48, out);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[as]);
            }
            seq = end;
        }
    } else if (warp >= kW16GEpiWarp0 && warp < kW16GEpiWarp0 + 4) {
        // ------------------------------------------------------- epilogue --
        const int q = warp & 3;                 // TMEM lane quadrant
        const uint32_t lane_addr = ((uint32_t)(q * 32)) << 16;
        uint16_t* stg = reinterpret_cast<uint16_t*>(smem + C::OFF_Y) + (warp - kW16GEpiWarp0) * (C::STG / 8);
        constexpr int LB = C::LB;
        const int c_in = q * 32 + lane;         // column within the tile
        Ring ra;
        while (walk.next(tile, u0, u1)) {
            const GroupedTile gt(g, p.E, p.n_tiles, BN, tile);
            bool ok = warp_wait_bounded(&acc_full[ra.idx], ra.phase, wc);
            if (walk.split) ok = !named_bar_or(1, 128, !ok);  // one decision before the barriers below
            if (!ok) break;
            tc_fence_after();
            const uint32_t tacc = tmem_base + lane_addr + ra.idx * BN;
            const int col0 = gt.nt * 128 + q * 32;
            const bool live = col0 < p.N;       // warp-uniform
            bool write = live, parts = false;
            int nparts = 0, c_first = 0;
            constexpr long long kTile = (long long)BN * 128;
            if (walk.split && (u0 > 0 || u1 < p.units)) {
                // part of a tile: the raw sums go to this CTA's slot (0: the tile began in an earlier CTA)
                float* dst = p.partial + (2LL * blockIdx.x + (u0 > 0 ? 0 : 1)) * kTile + c_in;
                if (live) {
#pragma unroll 1
                    for (int c0 = 0; c0 < gt.rows; c0 += LB) {
                        uint32_t v[LB];
                        tmem_ld32<LB>(tacc + c0, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < LB; ++i) dst[(c0 + i) * 128] = __uint_as_float(v[i]);
                    }
                }
                tc_fence_before();
                const int t0 = (int)tile * p.units;
                c_first = t0 / walk.Q;
                nparts = (t0 + p.units - 1) / walk.Q - c_first + 1;
                named_bar_sync(1, 128);
                if (threadIdx.x == kW16GEpiWarp0 * 32) {
                    __threadfence();
                    *last_flag = count_in(p.counts + tile, p.epoch, nparts) == nparts - 1;
                    __threadfence();
                }
                named_bar_sync(1, 128);
                write = live && *reinterpret_cast<volatile int*>(last_flag) != 0;
                parts = true;
            }
            if (write) {
#pragma unroll 1
                for (int c0 = 0; c0 < gt.rows; c0 += LB) {
                    uint32_t v[LB];
                    if (parts) {
                        // in the order of k, whoever came last: the same sum in every run
#pragma unroll
                        for (int i = 0; i < LB; ++i) v[i] = 0u;
#pragma unroll 2
                        for (int k = 0; k < nparts; ++k) {
                            const int c = c_first + k;
                            const int slot = c * walk.Q > (int)tile * p.units ? 0 : 1;
                            const float* src = p.partial + (2LL * c + slot) * kTile + c0 * 128 + c_in;
#pragma unroll
                            for (int i = 0; i < LB; ++i)
                                v[i] = __float_as_uint(__uint_as_float(v[i]) + __ldcg(src + i * 128));
                        }
                    } else {
                        tmem_ld32<LB>(tacc + c0, v);
                        tmem_wait_ld();
                    }
                    __syncwarp();  // the previous batch's copy-out is done with the staging
#pragma unroll
                    for (int i = 0; i < LB; ++i) stg[i * 32 + lane] = f32_to_bf16_bits(__uint_as_float(v[i]));
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
// 192} rows (defined in gemm_w4a16_grouped.cu).  tmap_x: the three activation
// boxes.  Status codes as in w4a8.h.
int launch_w4a16_grouped(int bn, bool sym, const CUtensorMap (&tmap_x)[3], const CUtensorMap& tmap_s,
                         const CUtensorMap& tmap_z, const W16GroupedParams& p, int grid, cudaStream_t stream);

}  // namespace w4a8
