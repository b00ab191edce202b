// Grouped W8A8 GEMM on the sm_100a tensor cores: rows sorted by expert, each
// run of rows times its expert's INT8 weight ("Kimi 2.7 MoE, 4-bit storage to
// INT8" §4.4 step 4 with the INT8 x INT8 product of "Inference Quantization
// ch.1" §4 and the scales of §8.2-8.3):
//   acc[r,n] = sum_k q_x[r,k] q_w[e,n,k]        e = expert of row r, exact int32
//   y[r,n]   = s_x[r] * (s_w[e,n] * acc[r,n])   fp32, one bf16 rounding
// and, for the gate_up product (columns [0, I) gate, [I, 2I) up),
//   h[r,i]   = silu(y[r,i]) * y[r,I+i]          fp32, one bf16 rounding.
//
// Design (B200):
//   * Swap-AB as in the other GEMMs here: the 128 MMA rows are weight columns
//     n, the MMA N dimension is tokens.  A tile is a PAIR of 128-column weight
//     boxes times up to BN rows of one expert, each box with its own TMEM
//     accumulator: 256 consecutive columns, or 128 gate columns and the same
//     128 up columns, so that the thread that drains gate column i also holds
//     up column i and silu(gate) * up needs no exchange.  Per 128 k a stage
//     moves 32 KB of weights and BN * 128 bytes of rows for 2 x 128 x BN
//     products: the traffic of a 256-wide tile at half its row granularity,
//     which ragged groups waste less of.
//   * One 4-D tensor map (k, column, half, expert) brings both boxes in one
//     request; columns past the expert's last are filled with zeros instead of
//     the next expert's weights.
//   * Rows of a tile past its expert's last are loaded (they belong to the next
//     expert) but neither multiplied, beyond a multiple of 16 (the MMA's N is
//     set per tile), nor stored: every output row has one writer.
//   * The host does not know the offsets, so every CTA derives the tile list:
//     m-tiles per expert, their prefix sum in shared memory, tile -> (expert,
//     n-tile, m-tile) by binary search.  m-tiles run inside n-tiles, so tiles
//     that share a weight box run side by side.
//   * Persistent.  Enough tiles: handed out round-robin.  Few tiles (a decode
//     step of few experts): the (tile, k-block) units are cut into equal
//     ranges, at most one for each CTA.  A CTA that holds part of a tile stores its
//     int32 partial tile and counts itself in; the one that completes the
//     count adds all parts and writes the output.  Integer sums are exact in
//     any order, so results do not depend on who comes last, and no CTA ever
//     waits for another.
//   * One warp streams weights, one rows, two issue the MMAs (one accumulator
//     each), 16 warps drain (32 columns each, staged in shared memory of its
//     own and written as 16-byte pieces; with 8 warps the drain took 8,400 of a
//     tile's 11,000 cycles at K = 1408).  Two accumulator pairs alternate, so a
//     drain overlaps the next tile's MMAs.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace w4a8 {

struct W8GroupedParams {
    int N;                       // output columns (gate_up: I)
    int KB;                      // k-blocks of 128
    int E, R;
    int halves;                  // boxes of 128 columns to a tile: 2, plain and few tiles: 1
    int n_tiles;                 // ceil(N / (128 halves)), gate_up: ceil(I / 128)
    const int32_t* offsets;      // [E + 1] device
    const float* s_w;            // [E][N], gate_up: [E][2I]
    const float* s_x;            // [R]
    uint16_t* Y;
    int ldy;
    int vec16;                   // Y and ldy allow 16-byte row stores
    int early;                   // offsets are final before the preceding kernel is complete
    int split_tiles;             // tiles below which units may be split (0: never)
    int32_t* partial;            // [2 * grid][2][BN][128] int32 partial tiles
    unsigned long long* counts;  // [split_tiles] arrivals of this launch
    unsigned long long epoch;
    int32_t* status;
    unsigned long long wait_ns;
};

constexpr int kW8GEpiWarps = 16;     // four groups, each with every quarter of the 128 columns
constexpr int kW8GThreads = 32 * (kW8GEpiWarps + 4);   // and 2 producers, 2 MMA warps
constexpr int kW8GEpiWarp0 = 2;
constexpr int kW8GXWarp = kW8GEpiWarp0 + kW8GEpiWarps;
constexpr int kW8GMma2Warp = kW8GXWarp + 1;
constexpr int kGroupedMaxExperts = 512;

template <int BN>
struct W8GCfg {
    static constexpr int A_STAGE = 256 * 128;               // two weight boxes of 128 columns x 128 k
    static constexpr int XBOX = BN < 64 ? BN : 64;          // rows per activation request
    static constexpr int B_STAGE = BN * 128;
    static constexpr int STAGE = A_STAGE + B_STAGE;
    static constexpr int LB = BN < 32 ? 8 : 16;             // tokens per epilogue batch
    static constexpr int STG = kW8GEpiWarps * 1024;         // output staging: 16 tokens x 32 columns per warp
    static constexpr int TABLE = 3 * (kGroupedMaxExperts + 1) * 4;
    static constexpr int NST_RAW = (227 * 1024 - 1024 - STG - TABLE - 512) / STAGE;
    static constexpr int NST = NST_RAW > 8 ? 8 : NST_RAW;
    static constexpr int OFF_STG = NST * STAGE;
    static constexpr int OFF_BAR = OFF_STG + STG;
    static constexpr int NUM_BARS = 3 * NST + 6;
    static constexpr int OFF_TABLE = OFF_BAR + NUM_BARS * 8;
    static constexpr int OFF_MISC = OFF_TABLE + TABLE;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static constexpr int ACC_COLS = 4 * BN;                 // two pairs of accumulators
    static constexpr uint32_t TMEM_COLS = ACC_COLS;
    // a part of a split tile, in k-blocks / 16: 0.8 + 0.027 for each row
    static constexpr int PART0 = 13, PART1 = 7;
    static_assert(BN == 16 || BN == 32 || BN == 64 || BN == 128, "BN");
    static_assert(NST >= 3, "stages");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

// 4-D tiled tensor load (coordinates innermost first).
__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z, int32_t w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// Rows and m-tiles of every expert, in shared memory.
struct GroupTable {
    int32_t* beg;   // [E] first row
    int32_t* cnt;   // [E] rows
    int32_t* mt;    // [E + 1] prefix of m-tiles
};

// Fills the table from the device offsets (all threads of the CTA; ends with
// a barrier).  Offsets outside [0, R] or decreasing are reported and clamped,
// so that no row index derived from them leaves [0, R).
__device__ __forceinline__ void build_group_table(const GroupTable& g, const int32_t* offsets, int E, int R, int bn,
                                                  int32_t* status) {
    const int tid = threadIdx.x, nthr = blockDim.x;
    for (int e = tid; e < E; e += nthr) {
        const int32_t o0 = __ldcg(offsets + e), o1 = __ldcg(offsets + e + 1);
        if ((o0 < 0) | (o1 > R) | (o1 < o0)) report_status(status, 1);
        const int32_t a = min(max(o0, 0), R), b = min(max(o1, 0), R);
        const int32_t c = max(b - a, 0);
        g.beg[e] = a;
        g.cnt[e] = c;
        g.mt[e + 1] = (c + bn - 1) / bn;
    }
    __syncthreads();
    if (tid < 32) {  // inclusive scan, one run of consecutive experts per lane
        const int per = (E + 31) / 32;
        const int e0 = min(tid * per, E), e1 = min(e0 + per, E);
        int32_t sum = 0;
        for (int e = e0; e < e1; ++e) sum += g.mt[e + 1];
        int32_t inc = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, off);
            if (tid >= off) inc += v;
        }
        int32_t run = inc - sum;
        for (int e = e0; e < e1; ++e) {
            run += g.mt[e + 1];
            g.mt[e + 1] = run;
        }
        if (tid == 0) g.mt[0] = 0;
    }
    __syncthreads();
}

// How `tiles` tiles of KB units go to `grid` CTAs: 0 for whole tiles in turn,
// else the length of the equal ranges of units that the CTAs take.  cost: the
// longest CTA's units x 16.  A range costs 2 units beside its own (two ends),
// and each of a tile's parts `part` / 16 units when the CTA that comes last
// adds them all (as written and read: 200 rows, K = N = 1024 in tiles of 128
// rows, 8 parts each: 28.8 us, whole 9); so ranges longer than the shortest
// ones, in fewer CTAs, are looked at too.
// (T: 32 bits on the device, where every division counts: 64-bit ones put 0.7
// us on a launch of 13.)
template <typename T>
__host__ __device__ inline int grouped_split(T tiles, T KB, T grid, T part, T& cost) {
    const T first = (tiles * KB + grid - 1) / grid;
    cost = (tiles + grid - 1) / grid * KB * 16;
    T best = 0;
    for (T q = first; q > 0 && (q == first || q < KB); q *= 2) {
        const T parts = (KB + q - 1) / q;
        const T c = 16 * q + 32 + (parts * q != KB ? parts + 1 : parts) * part;
        if (c < cost) {
            cost = c;
            best = q;
        }
    }
    return (int)best;
}

// The price of a tile's part (PART0 + PART1 / 16 for each of its rows), from
// the mean rows of M tiles of at most bn.
__host__ __device__ inline int grouped_part(int part0, int part1, int bn, unsigned R, unsigned M) {
    const unsigned rows = M > 0 ? (R + M - 1) / M : 0;
    return part0 + (int)(rows < (unsigned)bn ? rows : bn) * part1 / 16;
}

// A CTA's share of the work, as segments: k-blocks [kb0, kb1) of a tile.
struct GroupedWalk {
    long long tiles, t;          // whole tiles: next tile (strided by the grid)
    int u, u1, Q, KB;            // split: unit range
    bool split;

    __device__ __forceinline__ GroupedWalk(const GroupTable& g, int E, int n_tiles, int KB_, int split_tiles, int part) {
        KB = KB_;
        tiles = (long long)g.mt[E] * n_tiles;
        t = blockIdx.x;
        Q = 0;
        u = u1 = 0;
        if (tiles < split_tiles) {
            unsigned cost;
            Q = grouped_split<unsigned>((unsigned)tiles, KB, gridDim.x, part, cost);
        }
        split = Q > 0;
        if (split) {
            const int U = (int)tiles * KB;  // below split_tiles * 2^10
            u = min((int)blockIdx.x * Q, U);
            u1 = min(u + Q, U);
        }
    }
    // next segment; false at the end
    __device__ __forceinline__ bool next(long long& tile, int& kb0, int& kb1) {
        if (split) {
            if (u >= u1) return false;
            const int ti = u / KB;
            tile = ti;
            kb0 = u - ti * KB;
            kb1 = min(KB, kb0 + (u1 - u));
            u += kb1 - kb0;
            return true;
        }
        if (t >= tiles) return false;
        tile = t;
        kb0 = 0;
        kb1 = KB;
        t += gridDim.x;
        return true;
    }
};

struct GroupedTile {
    int e, nt, row0, rows;
    __device__ __forceinline__ GroupedTile(const GroupTable& g, int E, int n_tiles, int bn, long long tile) {
        const int m = (int)(tile / n_tiles);   // in [mt[e], mt[e + 1])
        int lo = 0, hi = E - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (g.mt[mid + 1] <= m) lo = mid + 1; else hi = mid;
        }
        e = lo;
        const int m0 = g.mt[lo], mc = g.mt[lo + 1] - m0;
        const int local = (int)(tile - (long long)m0 * n_tiles);
        nt = local / mc;
        const int mi = local - nt * mc;
        row0 = g.beg[lo] + mi * bn;
        rows = min(bn, g.cnt[lo] - mi * bn);
    }
};

// Counts this CTA in at a tile's arrival word and returns how many were there
// before it.  The word holds (epoch, count); any other epoch's content counts
// as zero, so the word needs no initialisation.  The last of `n` arrivals
// clears it, so that a replayed graph (same epoch) starts over.
__device__ __forceinline__ int count_in(unsigned long long* word, unsigned long long epoch, int n) {
    const unsigned long long base = epoch << 8;
    unsigned long long cur = *reinterpret_cast<volatile unsigned long long*>(word);
    while (true) {
        const int before = (cur >> 8) == (base >> 8) ? (int)(cur & 0xFFu) : 0;
        const unsigned long long want = before + 1 == n ? 0ull : base | (unsigned long long)(before + 1);
        const unsigned long long got = atomicCAS(word, cur, want);
        if (got == cur) return before;
        cur = got;
    }
}

// silu(y) = y / (1 + e^-y), as y e^y / (1 + e^y) for y < 0: the power never
// overflows and the quotient's divisor stays in [1, 2], so gates below -87 keep
// their value down to fp32's subnormals.  h's bf16 rounding is 2^-8; the power
// is within 2^-17 (its argument's rounding, 2^-24 of up to 88, and ex2's 2^-22)
// and the fast quotient within 2^-22.  With expf and the correctly rounded
// quotient the epilogue, not the MMAs, set the pace (13,000 of 15,000 cycles a
// tile at K = 2048).
__device__ __forceinline__ float silu_fast(float y) {
    float e;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(-1.442695041f * fabsf(y)));
    return __fdividef(y < 0.0f ? y * e : y, 1.0f + e);
}

template <int BN, bool GATEUP>
__global__ void __launch_bounds__(kW8GThreads, 1)
    w8a8_grouped_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                        const W8GroupedParams p) {
    using C = W8GCfg<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* w_full = bars;                // [NST] weight boxes landed
    uint64_t* x_full = w_full + C::NST;     // [NST] rows landed
    uint64_t* empty = x_full + C::NST;      // [NST] their MMAs completed
    uint64_t* acc_full = empty + C::NST;    // [2] accumulator pair's MMAs completed
    uint64_t* acc_empty = acc_full + 2;     // [2] drained by the epilogue warps
    uint64_t* drain = acc_empty + 2;        // [2] every MMA of a warp completed
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
        for (int i = 0; i < C::NST; ++i) {
            mbar_init(&w_full[i], 1);
            mbar_init(&x_full[i], 1);
            mbar_init(&empty[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 2);
            mbar_init(&acc_empty[i], kW8GEpiWarps);
        }
        mbar_init(&drain[0], 1);
        mbar_init(&drain[1], 1);
        *abort_flag = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
        prefetch_tmap(&tmap_w);
        prefetch_tmap(&tmap_x);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    // The rows, and the offsets too unless `early`, may come from the kernel
    // launched just before; the weights do not, and stream meanwhile.
    if (!p.early) pdl_wait_prerequisites();
    build_group_table(g, p.offsets, p.E, p.R, BN, blockIdx.x == 0 ? p.status : nullptr);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const WaitCtx wc{abort_flag, p.status, wait_cycles_for_ns(p.wait_ns)};
    GroupedWalk walk(g, p.E, p.n_tiles, p.KB, p.split_tiles, grouped_part(C::PART0, C::PART1, BN, p.R, g.mt[p.E]));
    long long tile;
    int kb0, kb1;

    if (warp == 0 || warp == kW8GXWarp) {
        // ------------------------------------------------------ producers --
        // Converged, one lane issuing, like the MMA warps below.
        const bool is_w = warp == 0;
        const bool leader = elect_one();
        uint64_t* full = is_w ? w_full : x_full;
        if (!is_w) pdl_wait_prerequisites();
        Ring rs;
        long long issued = 0;
        bool ok = true;
        while (ok && walk.next(tile, kb0, kb1)) {
            const GroupedTile gt(g, p.E, p.n_tiles, BN, tile);
            const int boxes = gt.rows > C::XBOX ? 2 : 1;
            const int col = gt.nt * (GATEUP ? 128 : 128 * p.halves);
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = warp_wait_bounded(&empty[rs.idx], rs.phase ^ 1u, wc);
                if (!ok) break;
                if (leader) {
                    uint8_t* st = smem + rs.idx * C::STAGE;
                    if (is_w) {
                        mbar_arrive_expect_tx(&full[rs.idx], p.halves * (C::A_STAGE / 2));
                        tma_load_4d(st, &tmap_w, &full[rs.idx], kb * 128, col, 0, gt.e);
                    } else {
                        mbar_arrive_expect_tx(&full[rs.idx], boxes * (C::XBOX * 128));
                        st += C::A_STAGE;
                        tma_load_2d(st, &tmap_x, &full[rs.idx], kb * 128, gt.row0);
                        if (boxes == 2)
                            tma_load_2d(st + C::XBOX * 128, &tmap_x, &full[rs.idx], kb * 128, gt.row0 + C::XBOX);
                    }
                }
                __syncwarp();
                rs.next(C::NST);
                ++issued;
            }
        }
        // copies in flight land before the CTA leaves
        if (leader) {
            WaitCtx wd = wc;
            volatile int no_abort = 0;
            wd.abort = &no_abort;
            Ring d = rs;
            for (long long k = 0; k < issued && k < C::NST; ++k) {
                ring_back(d, C::NST);
                (void)wait_bounded(&full[d.idx], d.phase, wd);
            }
        }
        __syncwarp();
    } else if (warp == 1 || warp == kW8GMma2Warp) {
        // ------------------------------------------------------ MMA issue --
        // One warp for each of the pair's accumulators: what a warp spends between
        // two stages (commit, wait) is covered by the other's MMAs.
        // The whole warp runs the loop and one lane issues: with every value
        // uniform over the warp, an MMA's descriptors sit in uniform registers
        // instead of being moved there one by one (measured in the W4A16
        // kernel: 135 -> 32 cycles for each MMA).
        // A wait costs its latency even when the stage is there, and the MMA
        // queue holds little more than a stage: so the next stage is asked for
        // before this one's MMAs are issued.
        const int half = warp == 1 ? 0 : 1;
        const bool leader = elect_one();
        Ring rs, ra;
        bool there = false;   // the stage's copies were seen to have landed
        bool ok = true;
        while (ok && walk.next(tile, kb0, kb1)) {
            const GroupedTile gt(g, p.E, p.n_tiles, BN, tile);
            const uint32_t idesc = idesc_i8((gt.rows + 15) & ~15);
            // some of the box's columns exist
            const bool mine = half == 0 || GATEUP || (p.halves == 2 && p.N - gt.nt * 256 > 128);
            ok = warp_wait_bounded(&acc_empty[ra.idx], ra.phase ^ 1u, wc);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem_base + ra.idx * (2 * BN) + half * BN;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!there) {
                    ok = warp_wait_bounded(&w_full[rs.idx], rs.phase, wc) &&
                         warp_wait_bounded(&x_full[rs.idx], rs.phase, wc);
                    if (!ok) break;
                }
                tc_fence_after();
                const uint32_t a_addr = smem_u32(smem + rs.idx * C::STAGE);
                uint64_t* const done = &empty[rs.idx];
                rs.next(C::NST);
                const bool next_w = mbar_test_wait(&w_full[rs.idx], rs.phase);
                const bool next_x = mbar_test_wait(&x_full[rs.idx], rs.phase);
                if (leader) {
                    const uint64_t adesc = umma_desc_kmajor(a_addr + half * (128 * 128), 128);
                    const uint64_t bdesc = umma_desc_kmajor(a_addr + C::A_STAGE, 128);
                    if (mine) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_i8(d, adesc + 2 * kk, bdesc + 2 * kk, idesc, (kb > kb0 || kk > 0) ? 1u : 0u);
                    }
                    tc_commit(done);
                }
                there = __all_sync(0xFFFFFFFFu, next_w && next_x) != 0;
            }
            if (!ok) break;
            if (leader) tc_commit(&acc_full[ra.idx]);
            __syncwarp();
            ra.next(2);
        }
        // drain: every MMA issued above completes before TMEM is freed
        if (leader) {
            tc_commit(&drain[half]);
            WaitCtx wd = wc;
            volatile int no_abort = 0;
            wd.abort = &no_abort;
            (void)wait_bounded(&drain[half], 0, wd);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------- epilogue --
        const int q = warp & 3;                          // TMEM lane quadrant
        const int grp = (warp - kW8GEpiWarp0) >> 2;      // plain: column half and every other batch; gate_up: every 4th
        const uint32_t lane_addr = ((uint32_t)(q * 32)) << 16;
        uint16_t* stg = reinterpret_cast<uint16_t*>(smem + C::OFF_STG) + (warp - kW8GEpiWarp0) * 512;
        constexpr int LB = C::LB;                        // a thread holds LB accumulators (gate_up: LB pairs)
        constexpr int STEP = GATEUP ? 4 * LB : 2 * LB;
        constexpr int kEpiThreads = 32 * kW8GEpiWarps;
        const int et = threadIdx.x - kW8GEpiWarp0 * 32;
        pdl_wait_prerequisites();
        Ring ra;
        while (walk.next(tile, kb0, kb1)) {
            const GroupedTile gt(g, p.E, p.n_tiles, BN, tile);
            bool ok = warp_wait_bounded(&acc_full[ra.idx], ra.phase, wc);
            if (walk.split) ok = !named_bar_or(1, kEpiThreads, !ok);  // one decision before the barriers below
            if (!ok) break;
            tc_fence_after();
            const uint32_t tacc = tmem_base + lane_addr + ra.idx * (2 * BN);
            const int half = GATEUP ? 0 : grp & 1;
            const int c_in = q * 32 + lane;                                      // column within the 128
            // the warp's first column
            const int col0 = GATEUP ? gt.nt * 128 + q * 32 : (gt.nt * p.halves + half) * 128 + q * 32;
            const int first = GATEUP ? grp * LB : (grp >> 1) * LB;               // the warp's first token batch
            const bool live = half < p.halves && col0 < p.N;                     // warp-uniform
            const int32_t* parts = nullptr;   // the tile's partial tiles, when this CTA adds them
            int nparts = 0, c_first = 0;
            bool write = live;
            if (walk.split && (kb0 > 0 || kb1 < p.KB)) {
                // part of a tile: the raw sums go to this CTA's slot
                const long long tile_ints = 2LL * BN * 128;
                int32_t* dst = p.partial + (2LL * blockIdx.x + (kb0 > 0 ? 0 : 1)) * tile_ints;
                if (live) {
#pragma unroll 1
                    for (int c0 = first; c0 < gt.rows; c0 += STEP) {
#pragma unroll
                        for (int hh = 0; hh < (GATEUP ? 2 : 1); ++hh) {
                            const int hf = GATEUP ? hh : half;
                            uint32_t v[LB];
                            tmem_ld32<LB>(tacc + hf * BN + c0, v);
                            tmem_wait_ld();
                            int32_t* d = dst + (hf * BN + c0) * 128 + c_in;
#pragma unroll
                            for (int j = 0; j < LB; ++j) d[j * 128] = (int32_t)v[j];
                        }
                    }
                }
                tc_fence_before();
                const int t0 = (int)tile * p.KB;
                c_first = t0 / walk.Q;
                nparts = (t0 + p.KB - 1) / walk.Q - c_first + 1;
                named_bar_sync(1, kEpiThreads);
                if (et == 0) {
                    __threadfence();
                    *last_flag = count_in(p.counts + tile, p.epoch, nparts) == nparts - 1;
                    __threadfence();
                }
                named_bar_sync(1, kEpiThreads);
                write = live && *reinterpret_cast<volatile int*>(last_flag) != 0;
                // the CTA holding the tile's first k-blocks stored to its slot 1, the others to slot 0
                parts = p.partial;
            }
            if (write) {
                const float* sw = p.s_w + (long long)gt.e * (GATEUP ? 2 * p.N : p.N);
                const int n = col0 + lane;
                const bool n_ok = n < p.N;
                const float sw0 = n_ok ? __ldg(sw + n) : 0.0f;
                const float sw1 = GATEUP && n_ok ? __ldg(sw + p.N + n) : 0.0f;
                auto load = [&](int hf, int c0, uint32_t* v) {
                    if (parts) {
                        const long long tile_ints = 2LL * BN * 128;
#pragma unroll
                        for (int j = 0; j < LB; ++j) v[j] = 0u;
#pragma unroll 2
                        for (int k = 0; k < nparts; ++k) {
                            const int c = c_first + k;
                            const int slot = c * walk.Q > (int)tile * p.KB ? 0 : 1;
                            const int32_t* s = parts + (2LL * c + slot) * tile_ints + (hf * BN + c0) * 128 + c_in;
#pragma unroll
                            for (int j = 0; j < LB; ++j) v[j] += (uint32_t)__ldcg(s + j * 128);
                        }
                    } else {
                        tmem_ld32<LB>(tacc + hf * BN + c0, v);
                    }
                };
#pragma unroll 1
                for (int c0 = first; c0 < gt.rows; c0 += STEP) {
                    uint32_t a[LB], b[GATEUP ? LB : 1];
                    load(GATEUP ? 0 : half, c0, a);
                    if constexpr (GATEUP) load(1, c0, b);
                    const float sxl = lane < LB && c0 + lane < gt.rows ? __ldg(p.s_x + gt.row0 + c0 + lane) : 0.0f;
                    if (!parts) tmem_wait_ld();
                    __syncwarp();  // the previous batch's copy-out is done with the staging
#pragma unroll
                    for (int j = 0; j < LB; ++j) {
                        const float sx = __shfl_sync(0xFFFFFFFFu, sxl, j);
                        float y = sx * (sw0 * (float)(int32_t)a[j]);
                        if constexpr (GATEUP) {
                            const float up = sx * (sw1 * (float)(int32_t)b[j]);
                            y = silu_fast(y) * up;
                        }
                        stg[j * 32 + lane] = f32_to_bf16_bits(y);
                    }
                    __syncwarp();
                    // LB rows of 32 columns: 16-byte pieces
#pragma unroll
                    for (int i = lane; i < LB * 4; i += 32) {
                        const int j = i >> 2, col = col0 + (i & 3) * 8;
                        if (c0 + j < gt.rows && col < p.N) {
                            const uint4 val = *reinterpret_cast<const uint4*>(stg + j * 32 + (i & 3) * 8);
                            uint16_t* dst = p.Y + (long long)(gt.row0 + c0 + j) * p.ldy + col;
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
            // the accumulator pair is free for the MMA's next tile
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

// Launches the grouped W8A8 kernel for a tile of BN in {16, 32, 64, 128} rows
// (defined in gemm_w8a8_grouped.cu).  Status codes as in w4a8.h.
int launch_w8a8_grouped(int bn, bool gate_up, const CUtensorMap& tmap_w, const CUtensorMap& tmap_x,
                        const W8GroupedParams& p, int grid, cudaStream_t stream);

// Rows of one activation request of a tile of bn rows.
inline int w8a8_grouped_xbox(int bn) { return bn < 64 ? bn : 64; }

}  // namespace w4a8
