// FP8 E4M3 TN GEMM with an fp32 scale per 128 elements of K, plain and grouped:
//
//   D[m][n] = C[m][n] + sum_b sa(m, b) sb(n, b) sum_{k in block b} A[m][k] B[n][k]
//
// The tensor cores sum one block's 128 products in fp32 (four MMAs of 32) into a TMEM
// accumulator of its own; the promotion warps read it, scale it and add it to their
// registers, which hold the tile's running fp32 sums, while the MMAs fill the next
// accumulator.  Nothing is scaled before the sum of a block, so the scales cost no
// precision, and there is one rounding, at the store.
//
// Tile: (128 * PAIR) rows x BN columns.  "Rows" are the MMA's M side: the rows of A, or,
// swapped, the rows of B (the weights), so that a few rows of A become a narrow N.
//   MODE_ROWS   rows of A, whose scale is the thread's own (sa, times the 128-block's sb)
//   MODE_BOTH   rows of A; a scale per row and one per column (both operands FP8_ROWS)
//   MODE_SWAP   rows of B; the scale of a column (a row of A) times the tile's sb
//
// Warps: 0 and 2 issue the row and column operands' TMA boxes (128 bytes of K, KSUB of
// them per stage), 1 the MMAs, 3 fills a ring with the tile's scales, KC blocks of K per
// slot; 4 .. 4 + EW - 1 promote and store, in G = EW / 4 groups of columns, four warps (the
// TMEM lane quarters) each.
// Barriers: `full` per stage (both operands' bytes), `done` per stage (one tcgen05.commit:
// the accumulator is ready, the stage is free), `free` per accumulator (every promotion
// warp has read it).  The MMA warp polls `full` and `free` in one instruction, each lane
// parity its own: a second wait of one thread would cost it ~200 of a block's 512 cycles.
// The promotion warps' time is the critical part: a block of a CTA's 128 x 256 sums takes the
// tensor cores 512 cycles, the fp32 pipes 256 (a scale per row and column: 512) and the TMEM
// loads 140 (257), and the store waits for the sums; so all else is kept off these warps.
// Scales read lane by lane from global memory took 75 of 303 us (8192 x 8192 x 4096),
// copied by these warps with cp.async 60; hence the ring and its warp.
// 8192 x 8192 x 4096, bf16: 177 us on codes of -1 to 1 (3.11 PFLOP/s), 190 to 194 on normal
// values, whose power takes the clock down (8192^3, new inputs each pass: 403 to 419 us, 2.62 to
// 2.73 PFLOP/s at ~1690 MHz).  Builds that skip work, at 180 us: no additions and TMEM loads 159,
// no store either 135, no operand loads either 125; the MMAs alone are 119.  The same of 4096 x
// 8192 x 4096 with a scale per row and column, fp32: 140, 95, 71, 67, 60.  No one part bounds it.
// Work: persistent units over whole tiles, or, for few tiles, a cluster of 2, 4 or 8 CTAs
// per tile that share its k-blocks and add their sums through distributed shared memory.
// Every wait is bounded, as in the other kernels of the library.
#pragma once

#include <cuda_bf16.h>

#include "experts.h"
#include "gemm_kernel.cuh"

namespace tn {

enum Fp8Mode : int { MODE_ROWS = 0, MODE_BOTH = 1, MODE_SWAP = 2 };

struct Fp8Params {
    int M, N, K;  // grouped: M = rows of A in all
    int nkb;      // 128-blocks of K
    int num_m, num_n, raster_group;  // plain: tiles along the rows of A and of B
    int split;                       // CTAs per tile (cluster split), 1 = off
    const float* sfa;
    const float* sfb;
    const int32_t* offsets;  // grouped: first row of each expert
    int experts;             // grouped; plain: 0
    const void* C;
    void* D;
    bool f32_out;
    unsigned int* err;
};

template <int MODE_, int PAIR_, int BN_, int STAGES_, int KSUB_, int ACC_BUFS_, int EW_, bool GROUPED_>
struct Fp8Config {
    static constexpr int MODE = MODE_;
    static constexpr bool kSwap = MODE == MODE_SWAP;
    static constexpr bool kColScale = MODE != MODE_ROWS;
    // How a promotion warp holds its 32 rows x W sums: a row per lane, or (with a scale per row
    // and per column) in 4-column fragments, four rows and W / 4 columns per lane, which needs
    // W / 4 column scales per lane and block instead of W: shared memory returns 128 bytes a
    // cycle, and reading every lane all scales took 1024 cycles of a block.  (Eight warps read
    // 128 x 256 accumulators in 140 cycles a row per lane, in 257 by 4-column fragments and in
    // 512 by 8-column ones.)
    static constexpr bool kFrag = MODE == MODE_BOTH;
    static constexpr bool kGrouped = GROUPED_;
    static constexpr int PAIR = PAIR_, BN = BN_, STAGES = STAGES_, KSUB = KSUB_, ACC_BUFS = ACC_BUFS_, EW = EW_;
    static constexpr int BN_CTA = BN / PAIR;
    static constexpr int TM = kSwap ? BN : 128 * PAIR;  // rows of A per tile
    static constexpr int TN = kSwap ? 128 * PAIR : BN;  // rows of B per tile
    static constexpr int THREADS = 128 + 32 * EW;
    static constexpr int G = EW / 4;  // promotion groups of four warps
    static constexpr int W = BN / G;  // columns of one group
    static constexpr bool kSplit = PAIR == 1 && !GROUPED_;
    // Eight promotion warps with 128 sums per thread take registers from the other four.
    static constexpr bool kRegSplit = W == 128;
    static constexpr int kRegsLaunch = 168, kRegsIssue = 56, kRegsPromote = 224;
    static_assert(!kRegSplit || (EW == 8 && 128 * kRegsIssue + 32 * EW * kRegsPromote <= THREADS * kRegsLaunch),
                  "register split within the launch's");
    static constexpr int TMEM_USED = ACC_BUFS * KSUB * BN;
    static constexpr int TMEM_COLS = TMEM_USED <= 32 ? 32 : TMEM_USED <= 64 ? 64 : TMEM_USED <= 128 ? 128 : TMEM_USED <= 256 ? 256 : 512;
    static_assert(TMEM_USED <= 512, "TMEM holds 512 columns");
    static_assert(EW == 4 || EW == 8, "whole groups of four promotion warps");
    static_assert(BN % (16 * PAIR) == 0 && BN <= 256 && W % 8 == 0, "MMA N, whole 16-byte vectors of D");
    static_assert(MODE != MODE_ROWS || (W <= 128 && 128 % W == 0), "one 128-block of B rows per group");

    static constexpr int ROW_SUB = 128 * 128, COL_SUB = BN_CTA * 128;  // bytes of one box
    static constexpr int ROW_BYTES = KSUB * ROW_SUB, COL_BYTES = KSUB * COL_SUB;
    // Scale ring: a slot holds, for KC blocks of K, [block][line]: per row of the tile its
    // scale (MODE_ROWS: times that of each group's 128-block of B, [group][row]), and per
    // column its scale (MODE_SWAP: times that of this CTA's rows of B).
    // (A single CTA's 128 x 256 tiles leave room for half the slots.)
    static constexpr int KC = PAIR_ == 1 && BN_ == 256 ? 4 : 8, SC_SLOTS = 2;
    static_assert(KC % KSUB_ == 0, "a scale chunk ends with a stage");
    static constexpr int SC_ROWS = MODE == MODE_ROWS ? G * 128 : MODE == MODE_BOTH ? 128 : 0;
    // Fragments: a group's columns 0, 4, 8, .. first, then 1, 5, .., so that a lane reads four of
    // its scales at once; the four runs start 4 banks apart.
    static constexpr int SC_RUN = W / 4 + 4;
    static constexpr int SC_COLS = kFrag ? G * 4 * SC_RUN : kColScale ? BN : 0;
    static_assert(!kFrag || KC == 8, "a lane of the scale warp keeps to one run");
    // floats; 4 apart from whole rows of banks, and a tile's place (m0, m_end, n0) in those of
    // its first slot's first block
    static constexpr int SC_PITCH = SC_ROWS + SC_COLS + 4;
    static constexpr int SC_SLOT = KC * SC_PITCH * 4;
    static_assert(SC_PITCH % 4 == 0, "16-byte aligned column scales");
    static constexpr int OFF_ROW = 0;
    static constexpr int OFF_COL = OFF_ROW + STAGES * ROW_BYTES;
    // Staging of the store (rows of A), and of C before it: boxes of 32 rows x 128 bytes per
    // promotion warp, 128B swizzle; as many as its columns take in bf16.  C's first boxes come
    // while the tile is summed.  4096 x 8192 x 8208 with a scale per row and column, fp32:
    // without C 266 to 281 us, added in place 273 to 285, another C 291 to 304 (318 read by the
    // lanes at the store).
    static constexpr int OFF_STG = OFF_COL + STAGES * COL_BYTES;
    static constexpr int STG_BUFS = W > 64 ? 2 : 1;
    static constexpr int STG_WARP = kSwap ? 0 : STG_BUFS * 4096;
    static constexpr int OFF_SC = OFF_STG + EW * STG_WARP;
    static constexpr int OFF_GRP = OFF_SC + SC_SLOTS * SC_SLOT;  // grouped: first rows, first tiles
    static constexpr int GRP_BYTES = GROUPED_ ? 2 * (kMaxExperts + 1) * 4 : 0;
    static constexpr int OFF_BAR = (OFF_GRP + GRP_BYTES + 7) / 8 * 8;
    // A cluster of `ways` CTAs cuts every promotion warp's columns into whole vectors of D.
    __host__ __device__ static constexpr bool split_fits(int ways) { return kSplit && W % ways == 0 && (kSwap || W / ways % 8 == 0); }
    static constexpr int BAR_FULL = 0, BAR_DONE = STAGES, BAR_FREE = 2 * STAGES, BAR_SCFULL = BAR_FREE + ACC_BUFS;
    static constexpr int BAR_SCFREE = BAR_SCFULL + SC_SLOTS, BAR_DRAIN = BAR_SCFREE + SC_SLOTS, BAR_C = BAR_DRAIN + 1;
    static constexpr bool kBoxC = !kSwap && !GROUPED_;  // C comes in boxes through the staging buffers
    static constexpr int NUM_BARS = BAR_C + (kBoxC ? EW * STG_BUFS : 0);
    static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
    static_assert(SMEM_BYTES <= 232448, "227 KB of dynamic shared memory per CTA");
    static_assert(COL_SUB % 1024 == 0, "operand boxes start on swizzle atoms");
    static_assert(!kSplit || 128 * BN * 4 <= STAGES * (ROW_BYTES + COL_BYTES), "a cluster's partial sums fit the idle stages");
};

// Each thread of the warp reads 16 consecutive 32-bit columns of its own TMEM lane.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// 16 TMEM lanes x 32 columns as 4-column fragments: thread l holds, of column 4i + l % 4, rows
// l / 4 (r[2i]) and l / 4 + 8 (r[2i + 1]).
__device__ __forceinline__ void tmem_ld_16x128b_x8(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x128b.x8.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// tmem_ld_wait for a load into r: the registers pass through the wait, so that no use of
// them moves before it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// Non-blocking parity test (CTA scope).
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Bounded parity wait that polls without suspending.
__device__ __forceinline__ bool wait_spin(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned int* err) {
    if (mbar_test_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_test_wait(bar, parity)) return true;
        if ((i & 1023u) == 0) {
            if (*abort_flag) return false;
            if (global_timer_ns() - t0 > kWaitLimitNs) {
                *abort_flag = 1;
                atomicOr(err, 1u);
                return false;
            }
        }
    }
}

// Bounded wait of a whole warp for two barriers: even lanes poll the first, odd the second.
template <bool kCluster>
__device__ __forceinline__ bool wait_two(uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1, int lane,
                                         volatile int* abort_flag, unsigned int* err) {
    const uint32_t bar = lane & 1 ? bar1 : bar0, parity = lane & 1 ? parity1 : parity0;
    auto poll = [&]() {
        return __all_sync(0xffffffffu, kCluster ? mbar_test_wait_cluster(bar, parity) : mbar_test_wait(bar, parity)) != 0;
    };
    if (poll()) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1;; ++i) {
        if (poll()) return true;
        if ((i & 1023u) == 0) {
            const bool late = global_timer_ns() - t0 > kWaitLimitNs;
            if (__any_sync(0xffffffffu, late)) {
                if (lane == 0) {
                    *abort_flag = 1;
                    atomicOr(err, 1u);
                }
                __syncwarp();
            }
            if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
        }
    }
}

// a[0..1] += t[0..1] * f * s[0..1], in packed fp32 arithmetic: half the instructions of the
// same rate, and the promotion is held up by its instructions.
__device__ __forceinline__ void scale_add2(float* a, const uint32_t* t, float f, float2 s) {
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%5, %6};\n\tmul.rn.f32x2 x, x, y;\n\t"
        "mov.b64 y, {%4, %4};\n\tmov.b64 z, {%0, %1};\n\tfma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "+f"(a[0]), "+f"(a[1])
        : "r"(t[0]), "r"(t[1]), "f"(f), "f"(s.x), "f"(s.y));
}
// a[0..1] += t[0..1] * f
__device__ __forceinline__ void add_scaled2(float* a, const uint32_t* t, float2 f) {
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%0, %1};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "+f"(a[0]), "+f"(a[1])
        : "r"(t[0]), "r"(t[1]), "f"(f.x), "f"(f.y));
}

// Copy 4 bytes (or, where `in` is false, four zero bytes) to shared memory, asynchronously.
__device__ __forceinline__ void cp_async_f32(uint32_t dst, const float* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// `bytes` (a multiple of 16) from global memory into L2.
__device__ __forceinline__ void l2_prefetch(const void* p, int bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// 2-D tiled store that adds the box to global memory (fp32).
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y) {
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y)
                 : "memory");
}

// Where one tile lies.
struct Fp8Tile {
    int m0, m_end;  // first row of A, end of its expert's (or of all) rows
    int n0;         // first row of B within its expert
    int expert;
};

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    gemm_fp8_block_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                          const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmD, const Fp8Params p) {
    constexpr int PAIR = Cfg::PAIR, STAGES = Cfg::STAGES, KSUB = Cfg::KSUB, EW = Cfg::EW, W = Cfg::W, BN = Cfg::BN;
    constexpr int ACC = Cfg::ACC_BUFS, KC = Cfg::KC;
    constexpr bool kPair = PAIR == 2, kSwap = Cfg::kSwap;

    extern __shared__ uint8_t smem_raw[];
    // (an offset, not an address rounded as an integer: the compiler then still knows that what
    // is read through it is shared memory)
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = kPair ? cluster_ctarank() : 0u;  // 0 = leader
    const bool leader = rank == 0;
    const int unit = static_cast<int>(blockIdx.x) / PAIR, units = static_cast<int>(gridDim.x) / PAIR;
    auto bar = [&](int i) -> uint32_t { return sbase + Cfg::OFF_BAR + 8 * i; };
    auto leader_bar = [&](int i) -> uint32_t { return kPair ? mapa_shared(bar(i), 0u) : bar(i); };
    volatile uint32_t* tmem_base_slot = reinterpret_cast<volatile uint32_t*>(smem + Cfg::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC + 4);
    int* first_row = reinterpret_cast<int*>(smem + Cfg::OFF_GRP);  // [experts + 1]
    int* first_tile = first_row + kMaxExperts + 1;                 // [experts + 1]

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar(Cfg::BAR_FULL + s), 2);
            mbar_init(bar(Cfg::BAR_DONE + s), 1);
        }
        for (int i = 0; i < ACC; ++i) mbar_init(bar(Cfg::BAR_FREE + i), EW * PAIR);
        for (int i = 0; i < Cfg::SC_SLOTS; ++i) {
            mbar_init(bar(Cfg::BAR_SCFULL + i), 1);
            mbar_init(bar(Cfg::BAR_SCFREE + i), EW);
        }
        mbar_init(bar(Cfg::BAR_DRAIN), 1);
        for (int i = Cfg::BAR_C; i < Cfg::NUM_BARS; ++i) mbar_init(bar(i), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        if (!kSwap) tma_prefetch_desc(&tmD);
        if (Cfg::kBoxC && p.C != nullptr) tma_prefetch_desc(&tmC);
    }
    if (warp == 1) {
        if constexpr (kPair) {
            tmem_alloc_pair(sbase + Cfg::OFF_MISC, Cfg::TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(sbase + Cfg::OFF_MISC, Cfg::TMEM_COLS);
            tmem_relinquish();
        }
    }
    griddep_launch_dependents();
    if constexpr (Cfg::kGrouped) {
        // Each expert's rows and tiles.  One warp makes the offsets ascending and within
        // 0 .. M (a running maximum) and sums the tiles.
        griddep_wait();
        for (int e = threadIdx.x; e <= p.experts; e += Cfg::THREADS) first_row[e] = min(max(p.offsets[e], 0), p.M);
        __syncthreads();
        if (warp == 2) {
            int high = 0, tiles = 0;
            for (int e0 = 0; e0 <= p.experts; e0 += 32) {
                const int e = e0 + lane;
                int r = e <= p.experts ? first_row[e] : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(0xffffffffu, r, o);
                    if (lane >= o) r = max(r, u);
                }
                r = max(r, high);
                int prev = __shfl_up_sync(0xffffffffu, r, 1);  // first row of expert e - 1
                if (lane == 0) prev = high;
                high = __shfl_sync(0xffffffffu, r, 31);
                int t = e >= 1 && e <= p.experts ? (r - prev + Cfg::TM - 1) / Cfg::TM * p.num_n : 0;  // tiles of expert e - 1
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(0xffffffffu, t, o);
                    if (lane >= o) t += u;
                }
                t += tiles;
                tiles = __shfl_sync(0xffffffffu, t, 31);
                if (e <= p.experts) {
                    first_row[e] = r;
                    first_tile[e] = t;
                }
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (kPair || (Cfg::kSplit && p.split > 1)) cluster_sync_all();  // every CTA's barriers exist before any cross-CTA signal
    tc_fence_after_sync();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_base_slot, 0);  // known to be one value per warp

    const int tiles = Cfg::kGrouped ? first_tile[p.experts] : p.num_m * p.num_n;
    // this unit's first tile and its share of a tile's stages
    const int nst = (p.nkb + KSUB - 1) / KSUB;
    const int split = Cfg::kSplit ? p.split : 1;
    const int part = split > 1 ? unit % split : 0;
    const int tile0 = split > 1 ? unit / split : unit;
    const int step = split > 1 ? tiles : units;  // a split tile is its cluster's only one
    const int st0 = static_cast<int>(static_cast<int64_t>(nst) * part / split);
    const int st1 = static_cast<int>(static_cast<int64_t>(nst) * (part + 1) / split);

    auto locate = [&](int tile) {
        Fp8Tile t;
        if constexpr (Cfg::kGrouped) {
            int lo = 0, hi = p.experts;  // first_tile[lo] <= tile < first_tile[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (first_tile[mid] <= tile)
                    lo = mid;
                else
                    hi = mid;
            }
            const int begin = first_row[lo], end = first_row[lo + 1];
            const int blocks = (end - begin + Cfg::TM - 1) / Cfg::TM;
            const int local = tile - first_tile[lo];
            // down the rows of A first: tiles that run at one time share the rows of B
            t.m0 = begin + local % blocks * Cfg::TM;
            t.m_end = end;
            t.n0 = local / blocks * Cfg::TN;
            t.expert = lo;
        } else {
            int mb, nb;
            tile_coords(tile, p.num_m, p.num_n, p.raster_group, mb, nb);
            t.m0 = mb * Cfg::TM;
            t.m_end = p.M;
            t.n0 = nb * Cfg::TN;
            t.expert = 0;
        }
        return t;
    };

    // ------------------------------------------------------------------ TMA issuers
    auto issue_loop = [&](const bool rows) {
        int s = 0;
        uint32_t ph = 0;
        bool ok = true, dep_done = false;
        const bool of_a = rows != kSwap;  // which matrix this warp loads
        const CUtensorMap* map = of_a ? &tmA : &tmB;
        // B is read once where a single tile of rows of A covers it: it goes first in L2
        const bool once = Cfg::kGrouped ? kSwap : p.num_m == 1;
        const bool hinted = of_a || once;
        const uint64_t policy = of_a ? l2_policy_evict_last() : l2_policy_evict_first();
        for (int tile = tile0; ok && tile < tiles; tile += step) {
            const Fp8Tile t = locate(tile);
            int y = of_a ? t.m0 : t.expert * p.N + t.n0;
            y += static_cast<int>(rank) * (rows ? 128 : Cfg::BN_CTA);
            for (int st = st0; st < st1; ++st) {
                ok = wait_bar(bar(Cfg::BAR_DONE + s), ph ^ 1u, abort_flag, p.err);
                if (!ok) break;
                if (!dep_done) {
                    griddep_wait();
                    dep_done = true;
                }
                const uint32_t sub = rows ? Cfg::ROW_SUB : Cfg::COL_SUB;
                const uint32_t dst = sbase + (rows ? Cfg::OFF_ROW + s * Cfg::ROW_BYTES : Cfg::OFF_COL + s * Cfg::COL_BYTES);
                const int subs = min(KSUB, p.nkb - st * KSUB);
                if (leader) mbar_arrive_expect_tx(bar(Cfg::BAR_FULL + s), PAIR * subs * sub);
#ifdef TN_TIMEOUT_INJECT
                // Test build only: CTA 0's first box of rows is withheld.
                if (rows && blockIdx.x == 0 && tile == tile0 && st == st0) {
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                    continue;
                }
#endif
#pragma unroll
                for (int j = 0; j < KSUB; ++j) {
                    if (KSUB > 1 && j >= subs) break;
                    const int x = (st * KSUB + j) * 128;
                    if constexpr (kPair) {
                        if (hinted)
                            tma_load_2d_pair_hint(dst + j * sub, map, leader_bar(Cfg::BAR_FULL + s), x, y, policy);
                        else
                            tma_load_2d_pair(dst + j * sub, map, leader_bar(Cfg::BAR_FULL + s), x, y);
                    } else {
                        if (hinted)
                            tma_load_2d_hint(dst + j * sub, map, bar(Cfg::BAR_FULL + s), x, y, policy);
                        else
                            tma_load_2d(dst + j * sub, map, bar(Cfg::BAR_FULL + s), x, y);
                    }
                }
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (ok && rows) {
            // every stage's MMAs done: no commit is in flight when the CTA exits
            for (int i = 0; i < STAGES && ok; ++i) {
                ok = wait_bar(bar(Cfg::BAR_DONE + s), ph ^ 1u, abort_flag, p.err);
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok) {
            // Abandoning: give every issued copy time to land.
            pause_ns(kDrainLimitNs / 4);
        }
    };

    // ------------------------------------------------------------------ MMA issuer
    // The warp waits, its lane 0 issues.
    auto mma_role = [&]() {
        if (!leader) return;
        const uint64_t rdesc0 = layout::umma_smem_desc_kmajor(sbase + Cfg::OFF_ROW, 128);
        const uint64_t cdesc0 = layout::umma_smem_desc_kmajor(sbase + Cfg::OFF_COL, 128);
        constexpr uint32_t idesc = idesc_dense(128 * PAIR, BN, true, 0u);
        bool ok = true;
        int s = 0, buf = 0;
        uint32_t ph = 0, bufph = 0;
        for (int tile = tile0; ok && tile < tiles; tile += step) {
            for (int st = st0; st < st1; ++st) {
                // operands landed; the accumulator was read by every promotion warp
                ok = wait_two<kPair>(bar(Cfg::BAR_FULL + s), ph, bar(Cfg::BAR_FREE + buf), bufph ^ 1u, lane, abort_flag, p.err);
                if (!ok) break;
                tc_fence_after_sync();
                const int subs = min(KSUB, p.nkb - st * KSUB);
                if (lane == 0) {
#pragma unroll
                    for (int j = 0; j < KSUB; ++j) {
                        if (KSUB > 1 && j >= subs) break;
                        const uint32_t d = tmem_base + static_cast<uint32_t>((buf * KSUB + j) * BN);
                        const uint64_t rd = rdesc0 + static_cast<uint64_t>((s * Cfg::ROW_BYTES + j * Cfg::ROW_SUB) >> 4);
                        const uint64_t cd = cdesc0 + static_cast<uint64_t>((s * Cfg::COL_BYTES + j * Cfg::COL_SUB) >> 4);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if constexpr (kPair)
                                mma_f8f6f4_pair(d, rd + 2 * i, cd + 2 * i, idesc, i != 0);
                            else
                                mma_f8f6f4(d, rd + 2 * i, cd + 2 * i, idesc, i != 0);
                        }
                    }
                    if constexpr (kPair)
                        tc_commit_pair(bar(Cfg::BAR_DONE + s), 0x3);
                    else
                        tc_commit(bar(Cfg::BAR_DONE + s));
                }
                __syncwarp();
                if (++buf == ACC) {
                    buf = 0;
                    bufph ^= 1u;
                }
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) {
            if constexpr (kPair)
                tc_commit_pair(bar(Cfg::BAR_DRAIN), 0x1);
            else
                tc_commit(bar(Cfg::BAR_DRAIN));
            wait_bar_drain(bar(Cfg::BAR_DRAIN), 0u);
        }
        __syncwarp();
    };

    // ------------------------------------------------------------------ scales
    // One warp copies the scales of KC blocks of K into each ring slot; what lies outside the
    // matrices is 0.  Lane l takes block l % KC of line l / KC of every 32 / KC lines, 4 KC
    // bytes of a scale row per access whatever the row's alignment.
    const int kb0 = st0 * KSUB, kb1 = min(st1 * KSUB, p.nkb);
    auto scale_role = [&]() {
        griddep_wait();
        constexpr int LINES = 32 / KC;
        const int nbs = static_cast<int>((static_cast<uint32_t>(p.N) + 127u) >> 7);
        const int line = lane / KC;
        int slot = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int tile = tile0; ok && tile < tiles; tile += step) {
            const Fp8Tile t = locate(tile);
            if (!kSwap && p.C != nullptr && (split > 1 || (p.f32_out && p.C != p.D))) {
                // the tile's C into L2: what does not fit the staging buffers is read at the store
                const int bytes = p.f32_out ? 4 : 2, cols = min(BN, p.N - t.n0);
                for (int r = lane; r < 128; r += 32) {
                    const int m = t.m0 + static_cast<int>(rank) * 128 + r;
                    if (m < t.m_end)
                        l2_prefetch(static_cast<const char*>(p.C) + (static_cast<int64_t>(m) * p.N + t.n0) * bytes, cols * bytes);
                }
                __syncwarp();
            }
            for (int kb = kb0; kb < kb1; kb += KC) {
                ok = __all_sync(0xffffffffu, wait_bar(bar(Cfg::BAR_SCFREE + slot), ph ^ 1u, abort_flag, p.err));
                if (!ok) break;
                const int k = kb + lane % KC;
                const bool k_in = k < kb1;
                float* out = reinterpret_cast<float*>(smem + Cfg::OFF_SC + slot * Cfg::SC_SLOT) + (lane % KC) * Cfg::SC_PITCH + line;
                // Scale rows first .. first + N - 1 of sf (those from `end` on are 0), times each of f
                // where there are factors.  All loads are in flight at once, in registers or (no
                // factors) copied to shared memory asynchronously.
                auto copy = [&](const float* sf, int first, int end, auto count, auto factors, const float* f) {
                    constexpr int N = decltype(count)::value, F = decltype(factors)::value, U = N / LINES;
                    const float* src = sf + static_cast<int64_t>(first + line) * p.nkb + k;
                    const int left = k_in ? end - first - line : 0;
                    if constexpr (F == 0) {
#pragma unroll 8
                        for (int u = 0; u < U; ++u) {
                            const bool in = u * LINES < left;
                            cp_async_f32(smem_u32(out + u * LINES), in ? src : sf, in);
                            src += static_cast<int64_t>(LINES) * p.nkb;
                        }
                        out += N;
                    } else {
                        static_assert(U <= 32, "one register per load");
                        float v[U];
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            v[u] = u * LINES < left ? __ldg(src) : 0.0f;
                            src += static_cast<int64_t>(LINES) * p.nkb;
                        }
#pragma unroll
                        for (int u = 0; u < U; ++u)
#pragma unroll
                            for (int j = 0; j < F; ++j) out[j * N + u * LINES] = v[u] * f[j];
                        out += F * N;
                    }
                };
                const int row0 = static_cast<int>(rank) * 128;
                using std::integral_constant;
                // the scales of a 128-block of B: of each group's columns, or (swapped) this CTA's rows
                constexpr int F = Cfg::MODE == MODE_ROWS ? Cfg::G : 1;
                float blk[F];
#pragma unroll
                for (int j = 0; j < F; ++j) {
                    const int nb = (kSwap ? t.n0 + row0 : t.n0 + j * W) >> 7;
                    const bool in = Cfg::MODE != MODE_BOTH && k_in && nb < nbs;
                    blk[j] = in ? __ldg(p.sfb + (static_cast<int64_t>(t.expert) * nbs + nb) * p.nkb + k) : 0.0f;
                }
                if constexpr (Cfg::MODE == MODE_ROWS) copy(p.sfa, t.m0 + row0, t.m_end, integral_constant<int, 128>{}, integral_constant<int, F>{}, blk);
                if constexpr (kSwap) copy(p.sfa, t.m0, t.m_end, integral_constant<int, BN>{}, integral_constant<int, 1>{}, blk);
                if constexpr (Cfg::MODE == MODE_BOTH) {
                    copy(p.sfa, t.m0 + row0, t.m_end, integral_constant<int, 128>{}, integral_constant<int, 0>{}, blk);
                    const float* src = p.sfb + static_cast<int64_t>(t.n0 + line) * p.nkb + k;
                    const int left = k_in ? p.N - t.n0 - line : 0;
                    out += line * (Cfg::SC_RUN - 1);  // line l of every four: run l
#pragma unroll
                    for (int g = 0; g < Cfg::G; ++g)
#pragma unroll 8
                        for (int u = 0; u < W / 4; ++u) {
                            const bool in = g * W + 4 * u < left;
                            cp_async_f32(smem_u32(out + g * 4 * Cfg::SC_RUN + u), in ? src : p.sfb, in);
                            src += static_cast<int64_t>(4) * p.nkb;
                        }
                    cp_async_wait_all();
                }
                if (kb == kb0 && lane == 0)
                    *reinterpret_cast<int4*>(smem + Cfg::OFF_SC + slot * Cfg::SC_SLOT + (Cfg::SC_ROWS + Cfg::SC_COLS) * 4) =
                        make_int4(t.m0, t.m_end, t.n0, t.expert);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(Cfg::BAR_SCFULL + slot));
                if (++slot == Cfg::SC_SLOTS) {
                    slot = 0;
                    ph ^= 1u;
                }
            }
        }
    };

    // ------------------------------------------------------------------ promotion, store
    auto promote_role = [&]() {
        griddep_wait();
        const int q = warp & 3, e = warp - 4, g = e >> 2;
        const int c0 = g * W;  // this warp's columns
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(c0);
        // Columns per TMEM load.  32 and 64 at a time, or half of the columns on their way while
        // the others are added, ran the same (180 to 183 us, 8192 x 8192 x 4096).
        constexpr int CH = 16;
        static_assert(W % CH == 0, "whole loads");
        int s = 0, buf = 0, slot = 0;
        uint32_t ph = 0, scph = 0;
        bool ok = true;
        float acc[W];
        const uint32_t done0 = bar(Cfg::BAR_DONE), free0 = mapa_shared(bar(Cfg::BAR_FREE), kPair ? 0u : cluster_ctarank());
        const int sc_row = Cfg::kFrag ? q * 32 + lane / 4 : g * 128 + q * 32 + lane;
        constexpr int RS = Cfg::kFrag ? 4 : 1;  // rows of the thread
        // a barrier that has mostly completed already: one test, else the bounded wait
        auto wait = [&](uint32_t b, uint32_t parity) {
            if (__all_sync(0xffffffffu, mbar_test_wait(b, parity))) return true;
            return __all_sync(0xffffffffu, wait_spin(b, parity, abort_flag, p.err)) != 0;
        };

        // this thread's sums v[0 .. NC-1] of the warp's rows and columns cb .. cb+NC-1 of the tile,
        // plus C, to D.  In fragments, each four of them are of one column of four: rows l / 4,
        // + 8, + 16, + 24.
        // staged_c: C's first boxes are in the staging buffers, or on their way (fetch_c).
        // the copy engine adds: one addition and one rounding per element, subnormals kept (measured)
        const bool add = p.f32_out && p.C == p.D;
        const bool c_boxes = Cfg::kBoxC && p.C != nullptr && !add;
        const int box_cols = p.f32_out ? 32 : 64;
        uint32_t cph = 0;  // parity of each buffer's C barrier
        auto c_bar = [&](int i) { return bar(Cfg::BAR_C + e * Cfg::STG_BUFS + i % Cfg::STG_BUFS); };
        // C's box i of the warp's columns into its buffer, once the copies out of it have read it
        auto fetch_c = [&](const Fp8Tile& t, int i) {
            const int m_warp = t.m0 + static_cast<int>(rank) * 128 + q * 32, n = t.n0 + c0 + i * box_cols;
            if (lane == 0 && n < p.N && m_warp < t.m_end) {
                bulk_wait_group_read<0>();
                mbar_arrive_expect_tx(c_bar(i), 4096);
                tma_load_2d(sbase + Cfg::OFF_STG + e * Cfg::STG_WARP + i % Cfg::STG_BUFS * 4096, &tmC, c_bar(i), n, m_warp);
            }
            __syncwarp();
        };
        auto store = [&](const Fp8Tile& t, int cb, auto count, auto staged_c, const float* v) {
            constexpr int NC = decltype(count)::value;
            [[maybe_unused]] constexpr bool kStagedC = Cfg::kBoxC && decltype(staged_c)::value;
            if constexpr (kSwap) {
                // columns are rows of A: 32 lanes write 32 neighbours of one row of D
                const int n = t.n0 + static_cast<int>(rank) * 128 + q * 32 + lane;
                if (n >= p.N) return;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    const int m = t.m0 + cb + i;
                    if (m >= t.m_end) break;
                    const int64_t at = static_cast<int64_t>(m) * p.N + n;
                    if (p.f32_out) {
                        const float c = p.C ? static_cast<const float*>(p.C)[at] : 0.0f;
                        static_cast<float*>(p.D)[at] = v[i] + c;
                    } else {
                        const float c = p.C ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.C)[at]) : 0.0f;
                        static_cast<__nv_bfloat16*>(p.D)[at] = __float2bfloat16_rn(v[i] + c);
                    }
                }
            } else {
                // Through the warp's 32 x 128-byte staging buffers (16-byte vector j of row r at
                // vector j ^ (r % 8)).  A C that is D itself in fp32 is added by the copy engine
                // (each element once, one rounding); another C comes into the buffers the same
                // way the sums leave them and is added there.  The copies leave the SM
                // asynchronously, and clip at the matrix's edges.  Rows that end inside the
                // warp's 32 (a grouped tile's last) and a cluster's parts with C are written by
                // the lanes.
                const int m_warp = t.m0 + static_cast<int>(rank) * 128 + q * 32;
                if (m_warp >= t.m_end) return;
                const bool with_c = kStagedC && c_boxes;
                const bool boxes = (!Cfg::kGrouped || m_warp + 32 <= t.m_end) && (p.C == nullptr || add || with_c);
                uint8_t* stg = smem + Cfg::OFF_STG + e * Cfg::STG_WARP;
                uint32_t stg_u32 = sbase + Cfg::OFF_STG + e * Cfg::STG_WARP;
                // box i's staging buffer, once its last copy has read it, or C has come
                auto next_box = [&](int i, int n) {
                    const int buf = i % Cfg::STG_BUFS;
                    stg = smem + Cfg::OFF_STG + e * Cfg::STG_WARP + buf * 4096;
                    stg_u32 = sbase + Cfg::OFF_STG + e * Cfg::STG_WARP + buf * 4096;
                    if (with_c) {
                        if (Cfg::STG_BUFS == 1 && i > 0) fetch_c(t, i);
                        if (n < p.N) {
                            if (ok) ok = wait(c_bar(i), cph >> buf & 1u);
                            cph ^= 1u << buf;
                        } else {
                            // no C comes past the columns, and so no wait with it: an earlier box may
                            // still be leaving this buffer, which the sums are written to all the same
                            if (lane == 0) bulk_wait_group_read<0>();
                            __syncwarp();
                        }
                    } else {
                        // (boxes are one group per buffer, in turn; the lanes' passes are none, so
                        // that the last group may be of this buffer)
                        if (lane == 0) {
                            if (boxes)
                                bulk_wait_group_read<Cfg::STG_BUFS - 1>();
                            else
                                bulk_wait_group_read<0>();
                        }
                        __syncwarp();
                    }
                };
                // the box is filled: C for the other buffer, whose copy has had this box's time
                auto after_box = [&](int i, int boxes) {
                    if (with_c && Cfg::STG_BUFS == 2 && i >= 1 && i + 1 < boxes) fetch_c(t, i + 1);
                    fence_proxy_async_smem();
                    __syncwarp();
                };
                auto vec = [&](int row, int j) { return reinterpret_cast<float4*>(stg + row * 128 + ((j ^ (row & 7)) << 4)); };
                if (boxes && !p.f32_out && NC % 64 == 0) {
#pragma unroll
                    for (int i = 0; i < NC; i += 64) {
                        const int n = t.n0 + cb + i;
                        next_box(i / 64, n);
#pragma unroll
                        for (int j = 0; j < 64 && i + j < NC; j += 8) {
                            if constexpr (Cfg::kFrag) {
#pragma unroll
                                for (int u = 0; u < 8; ++u) {
                                    __nv_bfloat16& d = reinterpret_cast<__nv_bfloat16*>(vec(lane / 4 + 8 * (u & 3), j / 8))[(u & 4) + (lane & 3)];
                                    d = __float2bfloat16_rn(with_c ? v[i + j + u] + __bfloat162float(d) : v[i + j + u]);
                                }
                            } else {
                                float f[8], c[8];
#pragma unroll
                                for (int u = 0; u < 8; ++u) f[u] = v[i + j + u];
                                if (with_c) {
                                    unpack8<KIND_FP8_E4M3>(*reinterpret_cast<const uint4*>(vec(lane, j / 8)), c);
#pragma unroll
                                    for (int u = 0; u < 8; ++u) f[u] += c[u];
                                }
                                *reinterpret_cast<uint4*>(vec(lane, j / 8)) = pack8<KIND_FP8_E4M3>(f);
                            }
                        }
                        after_box(i / 64, NC / 64);
                        if (lane == 0) {
                            if (n < p.N) tma_store_2d(&tmD, stg_u32, n, m_warp);
                            bulk_commit_group();  // empty past the columns: one group per buffer, in turn
                        }
                    }
                    return;
                }
                constexpr int SC = NC < 32 ? NC : 32;  // columns per pass
                constexpr int RL = SC / 4;             // lanes per row
#pragma unroll
                for (int i = 0; i < NC; i += SC) {
                    const int n = t.n0 + cb + i;
                    next_box(i / SC, n);
#pragma unroll
                    for (int j = 0; j < SC; j += 8) {
                        if constexpr (Cfg::kFrag) {
#pragma unroll
                            for (int u = 0; u < 8; ++u) {
                                float& d = reinterpret_cast<float*>(vec(lane / 4 + 8 * (u & 3), j / 4 + u / 4))[lane & 3];
                                d = with_c ? v[i + j + u] + d : v[i + j + u];
                            }
                        } else {
#pragma unroll
                            for (int u = 0; u < 8; u += 4) {
                                float4* d = vec(lane, (j + u) / 4);
                                float4 f = make_float4(v[i + j + u], v[i + j + u + 1], v[i + j + u + 2], v[i + j + u + 3]);
                                if (with_c) f.x += d->x, f.y += d->y, f.z += d->z, f.w += d->w;
                                *d = f;
                            }
                        }
                    }
                    if (boxes && p.f32_out && SC == 32) {
                        after_box(i / SC, NC / SC);
                        if (lane == 0) {
                            if (n < p.N && add) tma_add_2d(&tmD, stg_u32, n, m_warp);
                            if (n < p.N && !add) tma_store_2d(&tmD, stg_u32, n, m_warp);
                            bulk_commit_group();
                        }
                        continue;
                    }
                    __syncwarp();
                    const int col = n + 4 * (lane % RL), r0 = lane / RL;
                    if (col < p.N) {
                        constexpr int RSTEP = 32 / RL, ROWS = 32 / RSTEP;  // rows per lane
                        const int64_t at0 = static_cast<int64_t>(m_warp + r0) * p.N + col;
                        float4 c[ROWS];  // C, all of the lane's rows in flight at once
#pragma unroll
                        for (int i = 0; i < ROWS; ++i) {
                            c[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            if (p.C && m_warp + r0 + i * RSTEP < t.m_end) {
                                const int64_t at = at0 + static_cast<int64_t>(i * RSTEP) * p.N;
                                if (p.f32_out) {
                                    c[i] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.C) + at);
                                } else {
                                    const uint2 b = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.C) + at);
                                    c[i] = make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xFFFF0000u),
                                                       __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xFFFF0000u));
                                }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < ROWS; ++i) {
                            const int r = r0 + i * RSTEP;
                            if (m_warp + r >= t.m_end) break;
                            const int64_t at = at0 + static_cast<int64_t>(i * RSTEP) * p.N;
                            float4 f = *vec(r, lane % RL);
                            f.x += c[i].x, f.y += c[i].y, f.z += c[i].z, f.w += c[i].w;
                            if (p.f32_out) {
                                *reinterpret_cast<float4*>(static_cast<float*>(p.D) + at) = f;
                            } else {
                                const __nv_bfloat162 lo = __floats2bfloat162_rn(f.x, f.y), hi = __floats2bfloat162_rn(f.z, f.w);
                                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.D) + at) =
                                    make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                            }
                        }
                    }
                    __syncwarp();
                }
            }
        };

        for (int tile = tile0; ok && tile < tiles; tile += step) {
#pragma unroll
            for (int i = 0; i < W; ++i) acc[i] = 0.0f;
            int in_chunk = 0;
            bool fetched = false;
            Fp8Tile t{};  // where the tile lies: the scale warp's word, off this warp's path
            for (int st = st0; st < st1; ++st) {
                const int kb_st = st * KSUB, subs = min(KSUB, p.nkb - kb_st);
                const float* sc = reinterpret_cast<const float*>(smem + Cfg::OFF_SC + slot * Cfg::SC_SLOT) + in_chunk * Cfg::SC_PITCH;
                if (in_chunk == 0) {
                    ok = wait(bar(Cfg::BAR_SCFULL + slot), scph);
                    if (!ok) break;
                    if (st == st0) {
                        const int4 v = *reinterpret_cast<const int4*>(sc + Cfg::SC_ROWS + Cfg::SC_COLS);
                        t = Fp8Tile{v.x, v.y, v.z, v.w};
                        if (c_boxes && split == 1) {
#pragma unroll
                            for (int i = 0; i < Cfg::STG_BUFS; ++i) fetch_c(t, i);
                            fetched = true;
                        }
                    }
                }
                float rs[KSUB][RS];  // the scales of the thread's rows in this stage's blocks
#pragma unroll
                for (int j = 0; j < KSUB; ++j)
#pragma unroll
                    for (int i = 0; i < RS; ++i) rs[j][i] = kSwap ? 1.0f : sc[j * Cfg::SC_PITCH + sc_row + 8 * i];
                ok = wait(done0 + 8 * s, ph);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t tacc = lane_base + static_cast<uint32_t>(buf * KSUB * BN);
                auto release = [&]() {
                    // the accumulator is in registers: the MMAs may have it
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive_cluster_relaxed(free0 + 8 * buf);  // relaxed: what is handed over is TMEM
                    }
                };
#pragma unroll
                for (int j = 0; j < KSUB; ++j) {
                    if (KSUB > 1 && j >= subs) break;
                    const float* cs = sc + j * Cfg::SC_PITCH + Cfg::SC_ROWS + (Cfg::kFrag ? (g * 4 + (lane & 3)) * Cfg::SC_RUN : c0);
                    if constexpr (Cfg::kFrag) {
                        // 32 columns in flight while 32 are added; [0], [1]: lanes 0-15, 16-31 of the quarter
                        uint32_t rr[2][2][16];
                        auto load = [&](int c, uint32_t (&r)[2][16]) {
                            tmem_ld_16x128b_x8(tacc + j * BN + c, r[0]);
                            tmem_ld_16x128b_x8(tacc + j * BN + c + (16u << 16), r[1]);
                        };
                        load(0, rr[0]);
#pragma unroll
                        for (int c = 0; c < W; c += 32) {
                            uint32_t(&r)[2][16] = rr[c / 32 & 1];
                            float4 f[2];
#pragma unroll
                            for (int i = 0; i < 2; ++i) f[i] = *reinterpret_cast<const float4*>(cs + c / 4 + 4 * i);
                            tmem_ld_wait_for(r[0]);
                            tmem_ld_wait_for(r[1]);
                            if (c + 32 < W) load(c + 32, rr[c / 32 + 1 & 1]);
                            if (c + 32 >= W && j + 1 >= subs) release();
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float fi = i % 4 == 0 ? f[i / 4].x : i % 4 == 1 ? f[i / 4].y : i % 4 == 2 ? f[i / 4].z : f[i / 4].w;
                                scale_add2(&acc[c + 4 * i], &r[0][2 * i], fi, make_float2(rs[j][0], rs[j][1]));
                                scale_add2(&acc[c + 4 * i + 2], &r[1][2 * i], fi, make_float2(rs[j][2], rs[j][3]));
                            }
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < W; c += CH) {
                            uint32_t r[CH];
                            tmem_ld_32x32b_x16(tacc + j * BN + c, r);
                            tmem_ld_wait_for(r);
                            if (c + CH >= W && j + 1 >= subs) release();
#pragma unroll
                            for (int i = 0; i < CH; i += 4) {
                                float4 f = make_float4(rs[j][0], rs[j][0], rs[j][0], rs[j][0]);
                                if constexpr (kSwap) f = *reinterpret_cast<const float4*>(cs + c + i);
                                add_scaled2(&acc[c + i], &r[i], make_float2(f.x, f.y));
                                add_scaled2(&acc[c + i + 2], &r[i + 2], make_float2(f.z, f.w));
                            }
                        }
                    }
                }
                in_chunk += KSUB;
                if (in_chunk == KC || kb_st + KSUB >= kb1) {
                    in_chunk = 0;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(Cfg::BAR_SCFREE + slot));
                    if (++slot == Cfg::SC_SLOTS) {
                        slot = 0;
                        scph ^= 1u;
                    }
                }
                if (++buf == ACC) buf = 0;
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (ok && split == 1) store(t, c0, std::integral_constant<int, W>{}, std::true_type{}, acc);
            if (!ok && fetched) pause_ns(kDrainLimitNs / 4);  // abandoning: give C's boxes time to land
        }
        if constexpr (Cfg::kSplit) {
            if (split > 1) {
                // Each CTA of the cluster owns 1/split of every warp's columns.  The stages are
                // idle once all CTAs are past their main loops (first barrier): a slot of each
                // owner holds [source CTA][warp][column][lane] sums, added in source order.
                cluster_sync_all();
                auto reduce = [&](auto ways) {
                    constexpr int S = decltype(ways)::value;
                    constexpr int P = W / S;
                    if constexpr (Cfg::split_fits(S)) {
                        if (ok) {
#pragma unroll
                            for (int o = 0; o < S; ++o) {
                                const uint32_t at = static_cast<uint32_t>(Cfg::OFF_ROW + ((part * EW + e) * P * 32 + lane) * 4);
                                const uint32_t dst = mapa_shared(sbase + at, static_cast<uint32_t>(o));
#pragma unroll
                                for (int i = 0; i < P; ++i) {
                                    const int c = o * P + i;
                                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst + i * 128), "f"(acc[c]) : "memory");
                                }
                            }
                        }
                        __syncwarp();
                        cluster_sync_all();
                        if (ok && *abort_flag == 0) {
                            const Fp8Tile t = locate(tile0);
                            const float* in = reinterpret_cast<const float*>(smem + Cfg::OFF_ROW) + e * P * 32 + lane;
                            float v[P];
#pragma unroll
                            for (int i = 0; i < P; ++i) v[i] = 0.0f;
#pragma unroll
                            for (int r = 0; r < S; ++r)
#pragma unroll
                                for (int i = 0; i < P; ++i) v[i] += in[(r * EW * P + i) * 32];
                            store(t, c0 + part * P, std::integral_constant<int, P>{}, std::false_type{}, v);
                        }
                    }
                };
                if (split == 2)
                    reduce(std::integral_constant<int, 2>{});
                else if (split == 4)
                    reduce(std::integral_constant<int, 4>{});
                else
                    reduce(std::integral_constant<int, 8>{});
            }
        }
    };

    auto finish_stores = [&]() {
        if (!kSwap && lane == 0) bulk_wait_group_all();
        __syncwarp();
    };
    auto other_role = [&]() {
        if (warp == 1)
            mma_role();
        else if (warp == 3)
            scale_role();
        else if (lane == 0)
            issue_loop(warp == 0);
        __syncwarp();
        if (split > 1) {  // the two barriers of the cluster's reduction
            fence_proxy_async_smem();
            cluster_sync_all();
            cluster_sync_all();
        }
    };
    if constexpr (Cfg::kRegSplit) {
        if (warp < 4) {
            setmaxnreg_dec<Cfg::kRegsIssue>();
            other_role();
        } else {
            setmaxnreg_inc<Cfg::kRegsPromote>();
            promote_role();
            finish_stores();
        }
    } else {
        if (warp < 4)
            other_role();
        else {
            promote_role();
            finish_stores();
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    if constexpr (kPair)
        cluster_sync_all();  // no CTA leaves while its peer may still signal it
    else
        __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after_sync();
        if constexpr (kPair)
            tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
        else
            tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
    }
}

}  // namespace tn
